// tree_verify.cu - sampled acceptance along a tree of drafted nodes from given random numbers (dspark_tree_verify).
//
// openvino.genai PR #4847, commit on exact sampled speculative decoding: accept with min(1, p / q), otherwise draw from
// norm(max(0, p - q)). With several children at a node the residual takes the target's place for the next child; written out,
// the residual after any number of refusals is max(0, p - a q) / b with two numbers a and b, so that a refusal needs one sum over
// the vocabulary and nothing is stored.
#include "dspark_common.cuh"
#include "host_common.h"
#include "rowsample.cuh"

namespace {

using rs::FF;

constexpr int TV_MAXT = 512;
constexpr int TV_MAXC = 8;                   // blocks of a cluster

struct TvArgs {
  const float *p, *q;
  int64_t ldp, ldq, V;
  const int32_t *tokens, *parent, *n_nodes;
  const double *ua, *ud;
  int32_t T;
  int64_t seg;                               // ids of a warp's stretch of a row, a multiple of 4
  int32_t *out_tokens, *n_accepted, *path, *status;
};

// A block's share of what the whole cluster adds up, and what thread 0 asks of the others.
template <int WARPS>
struct TvShared {
  int32_t par[TV_MAXT], tok[TV_MAXT], first[TV_MAXT], next[TV_MAXT], path[TV_MAXT], dup[TV_MAXT];
  float px[TV_MAXT], qx[TV_MAXT];
  FF warp[WARPS], part[2][TV_MAXC];       // stretches of this block; shares of all blocks, two rounds of them
  uint32_t filter[64];                       // a bit for every refused id modulo 2048 (q absent)
  FF a;
  int32_t cur, done, refused, depth;         // row asked for; whether the walk ended; first refused child (q absent), depth
};

DS_DEV FF tv_pair(double x) {
  const float h = float(x);
  return FF{h, float(x - double(h))};
}

// max(0, p - a q) as a float pair; a number that is not one stays.
template <bool Q>
DS_DEV FF tv_term(float p, float q, const FF& a) {
  FF t{p, 0.0f};
  if (Q) {
    const float m = __fmul_rn(a.hi, q), e = __fmaf_rn(a.lo, q, __fmaf_rn(a.hi, q, -m));
    const float s = __fsub_rn(p, m), bb = __fsub_rn(s, p);
    t.hi = s;
    t.lo = __fsub_rn(__fadd_rn(__fsub_rn(p, __fsub_rn(s, bb)), __fsub_rn(-m, bb)), e);
  }
  const float v = __fadd_rn(t.hi, t.lo);
  if (v <= 0.0f) t.hi = t.lo = 0.0f;
  return t;
}
DS_DEV void tv_add(FF& acc, const FF& t) {
  rs::ff_add(acc, t.hi);
  acc.lo = __fadd_rn(acc.lo, t.lo);
}

// Entries i .. i + 3 of a row (VEC 4: 16-byte aligned, i a multiple of 4), 0 from `hi` on.
template <int VEC>
DS_DEV float4 tv_load(const float* row, int64_t i, int64_t hi) {
  if (VEC == 4 && i + 4 <= hi) return __ldg(reinterpret_cast<const float4*>(row + i));
  return make_float4(i < hi ? row[i] : 0.0f, i + 1 < hi ? row[i + 1] : 0.0f, i + 2 < hi ? row[i + 2] : 0.0f, i + 3 < hi ? row[i + 3] : 0.0f);
}

DS_DEV void tv_put_remote(FF* at, int rank, const FF& x) {      // the same place of another block of the cluster
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(ds_mapa(ds_smem_addr(at), uint32_t(rank))), "f"(x.hi), "f"(x.lo) : "memory");
}
// It stands behind branches on the thread's number and loops that end by the data, so the warp meets first: the barrier's aligned form wants it together.
// (One tree 16.4 us; with the form that each thread may reach for itself 17.7 us, means of ten runs.)
DS_DEV void tv_cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
DS_DEV int tv_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return int(r);
}
DS_DEV int tv_ranks() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_nctaid.x;" : "=r"(r));
  return int(r);
}

// One cluster per request. Every block keeps the tree (first child, next sibling, p and q of every node's token at its parent's row, gathered
// at once) and walks it by itself, with the same arithmetic, so no decision has to be sent; what the blocks share is the sum over
// a row, each warp of the cluster taking one stretch of it. The stretches' sums then also say where the draw's target lies: the warp whose
// stretch holds it reads it once more. Sums are float pairs, 2Sum and FMA, 48 bits: a token is drawn where a sum passes a border, and with
// 10^5 ids a float32 sum would put one draw in a hundred on the other side. Bound by the sums that follow one another, one for a refusal that the
// bound on b does not settle and one for the draw, each a pass over a row and a barrier of the cluster. Vocabularies of 151,936 ids: one tree without q 16 us
// (with the call), 64 trees of 24 nodes with q 55 us (49-59 in eight runs), 1.4 TB/s of the rows that a draw cannot do without.
template <bool Q, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) tree_verify_kernel(const TvArgs a) {
  constexpr int WARPS = THREADS / 32;
  __shared__ TvShared<WARPS> s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = tv_rank(), ranks = tv_ranks();
  const int64_t r = blockIdx.x / uint32_t(ranks);
  const int T = a.T;
  ds_pdl_trigger();
  ds_pdl_wait();
  int32_t n = a.n_nodes ? a.n_nodes[r] : T;
  if (n < 0 || n > T) {
    if (tid == 0) ds_set_error(a.status, DSPARK_EINVAL);
    n = 0;
  }
  for (int i = tid; i < T; i += THREADS) {
    int32_t par = -1, tok = -1;
    if (i > 0 && i < n) {
      par = a.parent ? a.parent[r * T + i] : i - 1;
      if (par >= i || par < 0) par = -1;                // never reached
      tok = a.tokens[r * T + i];
      if (tok < 0 || tok >= a.V) tok = -1;
    }
    s.par[i] = par;
    s.tok[i] = tok;
    s.first[i] = TV_MAXT;
    s.px[i] = par >= 0 && tok >= 0 ? a.p[(r * T + par) * a.ldp + tok] : 0.0f;
    s.qx[i] = Q && par >= 0 && tok >= 0 ? a.q[(r * T + par) * a.ldq + tok] : 1.0f;
  }
  __syncthreads();
  for (int i = tid; i < n; i += THREADS) {
    const int32_t par = s.par[i], tok = s.tok[i];
    if (par < 0) continue;
    atomicMin(&s.first[par], i);
    int next = TV_MAXT, dup = 0;
    if (!Q) {
      for (int k = par + 1; k < i; ++k) dup |= s.par[k] == par && s.tok[k] == tok;      // refused before, when i is tested
    }
    for (int k = i + 1; k < n; ++k) {
      if (s.par[k] == par) {
        next = k;
        break;
      }
    }
    s.next[i] = next;
    s.dup[i] = dup;
  }
  if (ranks > 1) tv_cluster_sync();                    // also: every block has begun before another writes to it
  else __syncthreads();
  // thread 0's state of the walk
  int cur = 0, child = 0, depth = 0;
  double da = 0.0, db = 1.0;
  bool open = false;                                   // b of this a is not known yet; db is the one before
  if (tid == 0 && n > 0) {
    s.path[0] = 0;
    child = s.first[0];
  }
  int round = 0;
  FF total{0.0f, 0.0f};
  int64_t lo = 0, hi = 0;
  bool plain = false;                   // plain: a residual without mass, replaced by p
  if (n > 0) {
    for (;;) {
      if (tid == 0) {
        int done = 0;
        if (open && round > 0 && !plain) {             // the sum that the test of `child` asked for
          db = rs::ff_value(total);
          open = false;
        }
        for (;;) {
          if (child >= TV_MAXT || plain) {
            done = 1;
            break;
          }
          const int x = child;
          const int32_t tok = s.tok[x];
          if (tok < 0) {
            ds_set_error(a.status, DSPARK_ERANGE);
            child = s.next[x];
            continue;
          }
          const double px = double(s.px[x]), u = a.ua[r * T + x];
          const double left = Q ? fmax(0.0, px - da * double(s.qx[x])) : (s.dup[x] ? 0.0 : px);
          // While b is not known it is at most the one before (a little more, where p was rounded and does not quite sum to 1): a child that would
          // be accepted with that one needs no sum.
          if (u * (open ? db * 1.015625 : db) * (Q ? double(s.qx[x]) : 1.0) < left) {
            cur = x;
            s.path[++depth] = x;
            child = s.first[x];
            da = 0.0;
            db = 1.0;
            open = false;
            continue;
          }
          if (open) break;                             // the others are needed for b
          child = s.next[x];
          if (Q) {
            da += db;
            open = true;
          } else {
            db -= left;
          }
        }
        s.cur = cur;
        s.done = done;
        s.depth = depth;
        s.refused = s.first[cur];
        s.a = tv_pair(da);
      }
      __syncthreads();
      const bool done = s.done != 0;
      const FF fa = s.a;
      if constexpr (!Q) {                              // only the draw's sum leaves ids out: the walk has ended
        if (tid < 64) s.filter[tid] = 0u;
        __syncthreads();
        for (int k = tid; k < n; k += THREADS)
          if (!plain && s.par[k] == s.cur && s.tok[k] >= 0) atomicOr(&s.filter[(s.tok[k] >> 5) & 63], 1u << (s.tok[k] & 31));
        __syncthreads();
      }
      const int64_t row = r * T + s.cur;
      const float* pr = a.p + row * a.ldp;
      const float* qr = Q ? a.q + row * a.ldq : nullptr;
      lo = min(a.V, (int64_t(rank) * WARPS + warp) * a.seg);
      hi = min(a.V, lo + a.seg);
      const bool minus = Q && (fa.hi != 0.0f || fa.lo != 0.0f) && !plain;
      // refused children of this node, without q: their ids count as 0
      auto gone = [&](int64_t id) {
        if constexpr (!Q) {
          if (((s.filter[(id >> 5) & 63] >> (id & 31)) & 1u) == 0u) return false;
          for (int k = plain ? TV_MAXT : s.refused; k < TV_MAXT; k = s.next[k])
            if (s.tok[k] == id) return true;
        }
        return false;
      };
      auto span = [&](int64_t i0, int64_t i1) {        // whether any refused id lies there
        if constexpr (!Q) {
          for (int k = plain ? TV_MAXT : s.refused; k < TV_MAXT; k = s.next[k])
            if (s.tok[k] >= i0 && s.tok[k] < i1) return true;
        }
        return false;
      };
      const bool some = span(lo, hi);
      FF acc[4] = {};
      // four vectors of each row on their way together
      for (int64_t i = lo + lane * 4; i < hi; i += 32 * 16) {
        float4 x[4], y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = tv_load<VEC>(pr, i + 128 * c, hi);
          if (minus) y[c] = tv_load<VEC>(qr, i + 128 * c, hi);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (some) {
            const int64_t id = i + 128 * c;
            x[c] = make_float4(gone(id) ? 0.0f : x[c].x, gone(id + 1) ? 0.0f : x[c].y, gone(id + 2) ? 0.0f : x[c].z, gone(id + 3) ? 0.0f : x[c].w);
          }
          if (minus) {
            tv_add(acc[0], tv_term<true>(x[c].x, y[c].x, fa));
            tv_add(acc[1], tv_term<true>(x[c].y, y[c].y, fa));
            tv_add(acc[2], tv_term<true>(x[c].z, y[c].z, fa));
            tv_add(acc[3], tv_term<true>(x[c].w, y[c].w, fa));
          } else {
            tv_add(acc[0], tv_term<false>(x[c].x, 0.0f, fa));
            tv_add(acc[1], tv_term<false>(x[c].y, 0.0f, fa));
            tv_add(acc[2], tv_term<false>(x[c].z, 0.0f, fa));
            tv_add(acc[3], tv_term<false>(x[c].w, 0.0f, fa));
          }
        }
      }
      rs::ff_acc(acc[0], acc[1]);
      rs::ff_acc(acc[2], acc[3]);
      rs::ff_acc(acc[0], acc[2]);
      const FF w = rs::warp_ff_reduce(acc[0]);
      if (lane == 0) s.warp[warp] = w;
      __syncthreads();
      if (tid < ranks) {
        FF sum = s.warp[0];
        for (int k = 1; k < WARPS; ++k) rs::ff_acc(sum, s.warp[k]);
        if (ranks > 1) tv_put_remote(&s.part[round & 1][rank], tid, sum);
        else s.part[round & 1][0] = sum;
      }
      if (ranks > 1) tv_cluster_sync();
      else __syncthreads();
      total = FF{0.0f, 0.0f};
      for (int k = 0; k < ranks; ++k) rs::ff_acc(total, s.part[round & 1][k]);
      ++round;
      if (!done) continue;
      const float mass = __fadd_rn(total.hi, total.lo);
      if (!(mass > 0.0f) && mass == mass && !plain) {  // nothing left: p itself
        plain = true;
        __syncthreads();
        continue;
      }
      // ---- the draw ----
      if (!(mass > 0.0f && mass < INFINITY)) {
        if (rank == 0 && tid == 0) {
          ds_set_error(a.status, DSPARK_ENONFINITE);
          a.out_tokens[r * T + s.depth] = -1;
        }
        break;
      }
      const FF target = rs::ff_mul(tv_pair(a.ud[r]), total);
      // the block, then the warp, whose running sum passes the target first; if rounding leaves none, the last with mass
      const FF* part = s.part[(round - 1) & 1];
      auto find = [&](const FF* v, int count, FF& run, bool& last) {
        int at = -1, some = -1;
        FF pre = run;
        for (int k = 0; k < count && at < 0; ++k) {
          FF upto = run;
          rs::ff_acc(upto, v[k]);
          if (__fadd_rn(v[k].hi, v[k].lo) > 0.0f) {
            some = k;
            pre = run;
            if (!last && rs::ff_diff(upto, target) > 0.0f) at = k;
          }
          run = upto;
        }
        if (at < 0) {
          at = some;
          last = true;
        }
        run = pre;
        return at;
      };
      FF run{0.0f, 0.0f};
      bool last = false;
      const int block = find(part, ranks, run, last);
      if (block == rank) {
        const int w = find(s.warp, WARPS, run, last);
        if (w == warp) {
          // 128 ids at a time, four of the stretch's vectors on their way together; where the target lies in them, the lane that passes it,
          // and the id in the lane
          int64_t pick = -1;                           // last id above 0 so far, in case rounding leaves none
          bool found = false;
          for (int64_t i0 = lo; i0 < hi && !found; i0 += 512) {
            float4 x[4], y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              x[c] = tv_load<VEC>(pr, i0 + 128 * c + lane * 4, hi);
              y[c] = minus ? tv_load<VEC>(qr, i0 + 128 * c + lane * 4, hi) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (found) continue;
              const int64_t id = i0 + 128 * c + lane * 4;
              const float px[4] = {x[c].x, x[c].y, x[c].z, x[c].w}, qx[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
              FF t[4], mine{0.0f, 0.0f};
              int top = -1;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                t[e] = minus ? tv_term<true>(px[e], qx[e], fa) : tv_term<false>(id + e < hi && gone(id + e) ? 0.0f : px[e], 0.0f, fa);
                tv_add(mine, t[e]);
                if (__fadd_rn(t[e].hi, t[e].lo) > 0.0f) top = e;
              }
              FF upto = mine;                          // inclusive over the lanes
#pragma unroll
              for (int d = 1; d < 32; d <<= 1) {
                const FF nb{__shfl_up_sync(0xFFFFFFFFu, upto.hi, d), __shfl_up_sync(0xFFFFFFFFu, upto.lo, d)};
                if (lane >= d) rs::ff_acc(upto, nb);
              }
              FF before{__shfl_up_sync(0xFFFFFFFFu, upto.hi, 1), __shfl_up_sync(0xFFFFFFFFu, upto.lo, 1)};
              if (lane == 0) before = FF{0.0f, 0.0f};
              rs::ff_acc(before, run);
              FF all = upto;
              rs::ff_acc(all, run);
              const unsigned past = __ballot_sync(0xFFFFFFFFu, !last && top >= 0 && rs::ff_diff(all, target) > 0.0f);
              const unsigned some = __ballot_sync(0xFFFFFFFFu, top >= 0);
              if (past) {
                const int at = __ffs(int(past)) - 1;
                int e = top;                           // the lane's last above 0 if rounding leaves none
                FF sum = before;
#pragma unroll
                for (int k = 3; k >= 0; --k) {         // first of the four whose running sum passes
                  FF s4 = sum;
                  for (int j = 0; j <= k; ++j) tv_add(s4, t[j]);
                  if (__fadd_rn(t[k].hi, t[k].lo) > 0.0f && rs::ff_diff(s4, target) > 0.0f) e = k;
                }
                pick = __shfl_sync(0xFFFFFFFFu, id + e, at);
                found = true;
              } else {
                if (some) pick = __shfl_sync(0xFFFFFFFFu, id + top, 31 - __clz(int(some)));
                run = FF{__shfl_sync(0xFFFFFFFFu, all.hi, 31), __shfl_sync(0xFFFFFFFFu, all.lo, 31)};
              }
            }
          }
          if (lane == 0) a.out_tokens[r * T + s.depth] = int32_t(pick);
        }
      }
      break;
    }
  }
  if (rank == 0) {
    __syncthreads();
    const int depth_ = n > 0 ? s.depth : -1;
    if (tid == 0) a.n_accepted[r] = depth_;
    for (int i = tid; i < T; i += THREADS) {
      a.path[r * T + i] = i <= depth_ ? s.path[i] : -1;
      if (i != depth_ || n == 0) a.out_tokens[r * T + i] = i < depth_ ? s.tok[s.path[i + 1]] : -1;
    }
  }
  // no block leaves while another may still write to its shares
  if (ranks > 1) tv_cluster_sync();
}

template <bool Q, int VEC, int THREADS>
cudaError_t tv_launch(const TvArgs& a, int64_t R, int ranks, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(R * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ranks);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<Q, VEC, THREADS>, a);
}

template <int THREADS>
cudaError_t tv_dispatch(const TvArgs& a, int64_t R, int ranks, bool vec, cudaStream_t st) {
  if (a.q) return vec ? tv_launch<true, 4, THREADS>(a, R, ranks, st) : tv_launch<true, 1, THREADS>(a, R, ranks, st);
  return vec ? tv_launch<false, 4, THREADS>(a, R, ranks, st) : tv_launch<false, 1, THREADS>(a, R, ranks, st);
}

}  // namespace

extern "C" dspark_status dspark_tree_verify(const float* p, int64_t ldp, const float* q, int64_t ldq, int64_t V, const int32_t* tokens,
                                            const int32_t* parent, const int32_t* n_nodes, const double* u_accept,
                                            const double* u_draw, int64_t R, int32_t T, int32_t* out_tokens, int32_t* n_accepted,
                                            int32_t* path, int32_t* dev_status, dspark_stream_t stream) {
  DS_REQUIRE(R >= 0 && R <= INT32_MAX / TV_MAXC && T >= 1 && T <= TV_MAXT && V >= 1 && V <= (int64_t(1) << 30) && ldp >= V);
  DS_REQUIRE(!q || ldq >= V);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(p && tokens && u_accept && u_draw && out_tokens && n_accepted && path && dev_status);
  DS_REQUIRE(ds_aligned(p, 4) && ds_aligned(q, 4) && ds_aligned(u_accept, 8) && ds_aligned(u_draw, 8));
  // Blocks for a request: as many as one wave of 1,024 threads an SM holds. With more requests than eight blocks of 512 threads each let into a
  // wave, blocks have 256 threads: 64 trees of 24 nodes 55 us, with 512 threads 59 us (means of eight runs); one tree 16 us with 512 threads, 21 us with 256. With four
  // blocks at most: one tree 23 us, 16 trees 47 us (36 us with eight), 64 trees 77 us; with one: 75, 140 and 219 us.
  const int64_t sms = ds_num_sms();
  const int threads = R * TV_MAXC > 2 * sms ? 256 : 512;
  int ranks = TV_MAXC;
  while (ranks > 1 && R * ranks > 1024 / threads * sms) ranks >>= 1;
  TvArgs a{p, q, ldp, ldq, V, tokens, parent, n_nodes, u_accept, u_draw, T, 0, out_tokens, n_accepted, path, dev_status};
  a.seg = ds_ceil_div(ds_ceil_div(V, int64_t(ranks) * (threads / 32)), 4) * 4;
  const bool vec = ds_aligned(p, 16) && ldp % 4 == 0 && (!q || (ds_aligned(q, 16) && ldq % 4 == 0));
  DS_CUDA_TRY(threads == 512 ? tv_dispatch<512>(a, R, ranks, vec, stream) : tv_dispatch<256>(a, R, ranks, vec, stream));
  return DSPARK_OK;
}
