// tree_attn.cu - attention of drafted nodes over a paged key/value cache (dspark_tree_attention):
// the bf16 tensor-core kernel, the join of partial results and the entry point.
//
// openvino.genai PR #4847, Fixes > Split validation windows, and optimum-intel PR #2098 (paged
// attention targets): the target's pass over the drafted candidates of several requests at once.
//
// tree_attn_tc_kernel. One block per SM works through its share of the line of tiles (tree_attn.cuh).
// The T * G query rows that read one key head lie on the 128 lanes of tensor memory, so the G query
// heads of a group and all drafted nodes share every key and value that is loaded:
//   S[128 rows, 128 keys] = Q K^T          (tcgen05.mma, K-major tiles in 128-byte swizzle)
//   P = 2^(x - m)  in bf16, over S in tensor memory (one thread per row, running maximum m and sum)
//   O[128 rows, D] += P V                  (A from tensor memory, V as it lies: D-major)
// Two softmax groups of four warps alternate so that the tensor pipe works on one while the other
// computes weights: with more than 128 rows they hold different rows of the same key tile, else the
// even and the odd key tiles of the same rows, joined through tensor memory at the end. O is rescaled
// only when a row's maximum rises by more than 2^8 (the weights stay below 256; sums are relative to
// the same reference, so the result is the same softmax).
//
// Roles: warp 0 copies key and value tiles with TMA, one box per page piece, into a ring of stages;
// warp 1 issues the MMAs; warps 2-3 copy the query rows; warps 4-7 and 8-11 are the softmax groups.
// Bound: HBM (2 D bytes of keys and of values per cached token and key head) up to about 270 query
// rows per key head, the tensor pipe above.
#include "tree_attn.cuh"

extern "C" size_t dspark_internal_ws_tree_attention(int64_t R, int32_t T, int64_t cols, int32_t heads);

namespace {

constexpr int TA_KT = 128;                 // keys per tile
constexpr int TA_THREADS = 384;
constexpr int TA_QTHREADS = 64;
constexpr uint32_t TA_CHUNK = 128 * 128;   // bytes of 128 rows x 64 bf16 columns
constexpr float TA_RISE = 8.0f;            // log2 rise of the maximum that rescales O

template <int DP, bool TWO>
__host__ __device__ constexpr int ta_stages() {
  return DP == 128 ? (TWO ? 4 : 5) : 8;
}
template <int DP, bool TWO>
__host__ __device__ constexpr size_t ta_smem() {
  return 1024 + size_t(DP / 64) * TA_CHUNK * ((TWO ? 2 : 1) + ta_stages<DP, TWO>());
}

// 4-D tiled TMA load (column, place in page, head, page); what lies outside the tensor reads as zero.
DS_DEV void ta_tma_load(void* dst, const void* tmap, int32_t d, int32_t t, int32_t h, int32_t p, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(ds_smem_addr(dst)),
      "l"(tmap), "r"(d), "r"(t), "r"(h), "r"(p), "r"(ds_smem_addr(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16; one thread.
DS_DEV void ta_umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of an operand whose N index is contiguous (V: rows are keys, 64 columns of D to a
// 128-byte row): 64-column blocks lie TA_CHUNK apart, groups of eight keys 1024 bytes apart.
DS_DEV uint64_t ta_desc_nmajor(uint32_t saddr) {
  uint64_t d = 0;
  d |= uint64_t((saddr & 0x3FFFFu) >> 4);
  d |= uint64_t(TA_CHUNK >> 4) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

DS_DEV void ta_tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
DS_DEV void ta_tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

DS_DEV uint32_t ta_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The row again in plain float32, every key looked at by itself: used for a row whose result came out
// not finite where drafted nodes are among the keys. The product P V adds 0 * v for a node that the
// row does not see, and that is not a number when v is not finite; here such a node is passed over.
// One warp per row; writes columns [d0, d1) relative to the reference maximum `mref`, times `mul`.
__device__ __noinline__ void ta_row_again(const TaArgs& a, int r, int hk, int m, int64_t k0, int64_t k1, float mref,
                                          float mul, int d0, int d1, __nv_bfloat16* out, float4* part) {
  const int lane = threadIdx.x & 31;
  int32_t ctx, n;
  ta_lens(a, r, ctx, n);
  const int i = m / a.G, h = hk * a.G + m % a.G, D = a.c.head_dim;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t(r) * a.T + i) * a.ldq + int64_t(h) * D;
  const __nv_bfloat16* kc = reinterpret_cast<const __nv_bfloat16*>(a.c.k) + hk * a.c.head_stride;
  const __nv_bfloat16* vc = reinterpret_cast<const __nv_bfloat16*>(a.c.v) + hk * a.c.head_stride;
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  k1 = min(k1, int64_t(ctx) + n);
  for (int64_t j = k0; j < k1; ++j) {
    if (!(ta_mask32(a, r, i, n, j - ctx) & 1u)) continue;
    const int64_t at = ta_slot(a, r, j);
    float s = 0.0f;
    if (at >= 0)
      for (int d = lane; d < D; d += 32) s = __fmaf_rn(__bfloat162float(q[d]), __bfloat162float(kc[at + d]), s);
    s = ds_warp_sumf(s);
    const float x = a.softcap > 0.0f ? ta_tanh(s * (a.scale * 2.0f * TA_LOG2E / a.softcap), a.softcap * TA_LOG2E)
                                     : s * (a.scale * TA_LOG2E);
    const float p = ta_ex2(x - mref);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int d = d0 + lane + 32 * u;
      if (d < d1) acc[u] = __fmaf_rn(p, at >= 0 ? __bfloat162float(vc[at + d]) : 0.0f, acc[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int d = d0 + lane + 32 * u;
    if (d >= d1) continue;
    if (out) out[d] = __float2bfloat16_rn(acc[u] * mul);
    else reinterpret_cast<float*>(part + int64_t(d >> 2) * a.rs)[d & 3] = acc[u];
  }
}

template <int DP, bool TWO, bool CAP>
__global__ void __launch_bounds__(TA_THREADS, 1) tree_attn_tc_kernel(const TaArgs a,
                                                                     const __grid_constant__ CUtensorMap tmK,
                                                                     const __grid_constant__ CUtensorMap tmV) {
  constexpr int NS = ta_stages<DP, TWO>();
  constexpr int NC = DP / 64;                          // 64-column chunks
  constexpr uint32_t STAGE = NC * TA_CHUNK;
  constexpr uint32_t TS = 0, TO = 256;                 // tensor memory: S of group g at 128 g, O at 256 + DP g
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[NS], s_empty[NS], s_qfull, s_qempty, s_sfull[2], s_pfull[2], s_ofull, s_ofree, s_mlfull, s_drain;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int32_t s_pref[TA_MAXR + 1];
  __shared__ float2 s_ml[2][2][128];                   // [piece parity][group][row]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sR = sQ + (TWO ? 2 : 1) * STAGE;            // the ring (a query tile has a stage's size)

  ds_pdl_trigger();
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      ds_mbar_init(&s_full[s], 1);
      ds_mbar_init(&s_empty[s], 1);
    }
    ds_mbar_init(&s_qfull, TA_QTHREADS);
    ds_mbar_init(&s_qempty, 1);
    for (int g = 0; g < 2; ++g) {
      ds_mbar_init(&s_sfull[g], 1);
      ds_mbar_init(&s_pfull[g], 4);
    }
    ds_mbar_init(&s_ofull, 1);
    ds_mbar_init(&s_ofree, 8);
    ds_mbar_init(&s_mlfull, 8);
    ds_mbar_init(&s_drain, 1);
    ds_fence_mbar_init_cluster();
    s_abort = 0;
  }
  ds_pdl_wait();
  if (warp == 1) ds_tmem_alloc(&s_tmem, 512);
  ds_tc_fence_before();
  ta_prefix(a, s_pref);                                // synchronises the block
  ds_tc_fence_after();
  const uint32_t tmem = s_tmem;
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t limit) {
    if (!ds_mbar_wait_or_abort(bar, parity & 1u, limit, &s_abort)) {
      if (!aborted()) ds_set_error(a.status, DSPARK_ETIMEOUT);
      s_abort = 1;
    }
    return !aborted();
  };
  TaWalk walk;
  walk.init(s_pref, a, blockIdx.x, gridDim.x);
  TaPiece p;

  if (warp == 0) {
    // ---- key and value tiles: lane b copies box b (keys b * box ..) of a tile; the copy of a box past
    // the last key, or of a page that does not exist, names a page past the last and reads zeros ----
    const int box = a.box, nbox = TA_KT / box;
    uint32_t seq = 0;
    bool ok = true;
    while (ok && walk.next(s_pref, a, p)) {
      int32_t ctx, n;
      ta_lens(a, p.r, ctx, n);
      const int64_t len = int64_t(ctx) + n;
      const int32_t* table = a.c.page_table + int64_t(p.r) * a.c.ld_table;
      int32_t place = 0;
      auto page_of = [&](int t) -> int64_t {           // (page, place) of this lane's box of tile t
        int32_t pg = int32_t(a.c.num_pages);
        const int64_t key = int64_t(t) * TA_KT + lane * box;
        if (lane < nbox && t < p.t1 && key < len) {
          const int64_t e = key / a.c.page_size;
          place = int32_t(key - e * a.c.page_size);
          pg = table[e];
          if (pg < 0 || pg >= a.c.num_pages) {
            ds_set_error(a.status, DSPARK_ERANGE);
            pg = int32_t(a.c.num_pages);
          }
        }
        return (int64_t(place) << 32) | uint32_t(pg);
      };
      auto load = [&](const CUtensorMap* tm, int64_t at) {
        const uint32_t s = seq % NS, ph = (seq / NS) & 1u;
        ok = wait(&s_empty[s], ph ^ 1u, DS_WAIT_LIMIT);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return;
        if (lane == 0) ds_mbar_arrive_expect_tx(&s_full[s], STAGE);
        __syncwarp();
        if (lane < nbox) {
          uint8_t* dst = sR + s * STAGE + lane * box * 128;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            ta_tma_load(dst + c * TA_CHUNK, tm, c * 64, int32_t(at >> 32), p.hk, int32_t(at), &s_full[s]);
        }
        __syncwarp();
        ++seq;
      };
      // the order in which the MMA warp consumes them
      int64_t pa = page_of(p.t0), pb = page_of(p.t0 + 1);
      load(&tmK, pa);
      if (!TWO && ok && p.t0 + 1 < p.t1) load(&tmK, pb);
      for (int t = p.t0; ok && t < p.t1; ++t) {
        const int64_t pc = page_of(t + 2);
        load(&tmV, pa);
        if (ok && TWO && t + 1 < p.t1) load(&tmK, pb);
        if (ok && !TWO && t + 2 < p.t1) load(&tmK, pc);
        pa = pb;
        pb = pc;
      }
    }
    if (lane == 0)                                     // every copy lands before the block leaves
      for (uint32_t k = (seq > uint32_t(NS) ? seq - NS : 0); k < seq; ++k)
        (void)ds_mbar_wait(&s_full[k % NS], (k / NS) & 1u, DS_WAIT_LIMIT);
    __syncwarp();
  } else if (warp == 1) {
    // ---- one thread issues the MMAs. QK of a group's next tile follows the group's PV: S and P share
    // tensor memory, and the MMAs of one thread run in order ----
    if (lane == 0) {
      constexpr uint32_t idS = ds_idesc_bf16_f32(128, TA_KT);
      constexpr uint32_t idO = ds_idesc_bf16_f32(128, DP) | (1u << 16);   // B is N-major
      const uint32_t qaddr = ds_smem_addr(sQ), raddr = ds_smem_addr(sR);
      uint32_t seq = 0, np = 0, pn[2] = {0, 0};
      bool ok = true;
      auto full = [&](uint32_t sq) {
        ok = ok && wait(&s_full[sq % NS], sq / NS, DS_WAIT_LIMIT);
        ds_tc_fence_after();
        return ok;
      };
      auto release = [&](uint32_t sq) { ds_umma_commit(&s_empty[sq % NS]); };
      auto qk = [&](int g, uint32_t sq) {
        const uint32_t q0 = qaddr + (TWO ? g : 0) * STAGE, k0 = raddr + (sq % NS) * STAGE;
#pragma unroll
        for (int kb = 0; kb < DP / 16; ++kb) {
          const uint32_t off = (kb >> 2) * TA_CHUNK + (kb & 3) * 32;
          ds_umma_f16(tmem + TS + 128 * g, ds_smem_desc_sw128(q0 + off), ds_smem_desc_sw128(k0 + off), idS, kb != 0);
        }
        ds_umma_commit(&s_sfull[g]);
      };
      auto pv = [&](int g, uint32_t sq, bool acc) {
        const uint32_t v0 = raddr + (sq % NS) * STAGE;
#pragma unroll
        for (int kb = 0; kb < TA_KT / 16; ++kb)
          ta_umma_ts(tmem + TO + DP * g, tmem + TS + 128 * g + kb * 8, ta_desc_nmajor(v0 + kb * 2048), idO, acc || kb != 0);
      };
      auto weights = [&](int g, bool first) {          // P of group g is written; at first O must be free too
        ok = ok && wait(&s_pfull[g], pn[g]++, DS_WAIT_LIMIT);
        if (first && np > 0) ok = ok && wait(&s_ofree, np - 1, DS_WAIT_LIMIT);
        ds_tc_fence_after();
        return ok;
      };
      while (ok && walk.next(s_pref, a, p)) {
        const int nt = p.t1 - p.t0;
        ok = wait(&s_qfull, np, DS_WAIT_LIMIT);
        if (!ok) break;
        ds_tc_fence_after();
        if (TWO) {                                     // ring order: K0, then V_t, K_{t+1}
          if (!full(seq)) break;
          qk(0, seq);
          qk(1, seq);
          release(seq++);
          if (nt == 1) ds_umma_commit(&s_qempty);
          for (int t = 0; t < nt; ++t) {
            const bool more = t + 1 < nt;
            if (!weights(0, t == 0) || !full(seq)) break;
            pv(0, seq, t > 0);
            if (more) {
              if (!full(seq + 1)) break;
              qk(0, seq + 1);
            }
            if (!weights(1, false)) break;
            pv(1, seq, t > 0);
            release(seq++);
            if (more) {
              qk(1, seq);
              release(seq++);
              if (t + 2 == nt) ds_umma_commit(&s_qempty);
            }
          }
        } else {                                       // ring order: K0, K1, then V_t, K_{t+2}
          for (int t = 0; t < min(2, nt); ++t) {
            if (!full(seq)) break;
            qk(t, seq);
            release(seq++);
          }
          if (nt <= 2) ds_umma_commit(&s_qempty);
          for (int t = 0; ok && t < nt; ++t) {
            const int g = t & 1;
            if (!weights(g, t == 0) || !full(seq)) break;
            pv(g, seq, t >= 2);
            release(seq++);
            if (t + 2 < nt) {
              if (!full(seq)) break;
              qk(g, seq);
              release(seq++);
              if (t + 3 == nt) ds_umma_commit(&s_qempty);
            }
          }
        }
        if (!ok) break;
        ds_umma_commit(&s_ofull);
        ++np;
      }
      ds_umma_commit(&s_drain);                        // the MMAs are done before tensor memory goes
      (void)ds_mbar_wait(&s_drain, 0, DS_WAIT_LIMIT);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ---- query rows of each piece into the swizzled layout; columns past head_dim are zero (the key
    // tile's are too), rows that do not exist keep what was there: a row only reaches its own results ----
    const int qt = tid - 64, cpr = DP / 8, D = a.c.head_dim;
    uint32_t np = 0;
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q);
    while (walk.next(s_pref, a, p)) {
      if (np > 0 && !wait(&s_qempty, np - 1, DS_WAIT_LIMIT)) break;
      const int m0 = p.g * a.rpg, cnt = min(a.rpg, a.rows - m0);
#pragma unroll 4
      for (int u = qt; u < cnt * cpr; u += TA_QTHREADS) {
        const int lr = u / cpr, c = u % cpr, m = m0 + lr, i = m / a.G;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (c * 8 < D)
          x = __ldg(reinterpret_cast<const uint4*>(q + (int64_t(p.r) * a.T + i) * a.ldq +
                                                   int64_t(p.hk * a.G + (m - i * a.G)) * D + c * 8));
        const int row = lr & 127;
        *reinterpret_cast<uint4*>(sQ + (lr >> 7) * STAGE + (c >> 3) * TA_CHUNK + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x;
      }
      ds_fence_proxy_async_smem();
      ds_mbar_arrive(&s_qfull);
      ++np;
    }
  } else {
    // ---- softmax: group g, one thread per row ----
    const int g = (warp - 4) >> 2, quarter = warp & 3, lr = quarter * 32 + lane;
    const uint32_t tl = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t tS = tl + TS + 128 * g, tO = tl + TO + DP * g;
    const float sc = CAP ? a.scale * 2.0f * TA_LOG2E / a.softcap : a.scale * TA_LOG2E;
    const float cap2 = a.softcap * TA_LOG2E;
    const int D = a.c.head_dim;
    uint32_t np = 0, ns = 0, seq = 0;
    bool first = true, ok = true;
    while (ok && walk.next(s_pref, a, p)) {
      int32_t ctx, n;
      ta_lens(a, p.r, ctx, n);
      const int64_t len = int64_t(ctx) + n;
      const int npt = p.t1 - p.t0;
      const int m = p.g * a.rpg + (TWO ? g * 128 : 0) + lr;    // this thread's row
      const bool live = p.g * a.rpg + (TWO ? g * 128 : 0) + quarter * 32 < a.rows;   // any row of this warp
      const int i = min(m, a.rows - 1) / a.G;
      float mref = -INFINITY, l = 0.0f;
      bool has = false;                                        // O holds an earlier tile
      for (int t = TWO ? 0 : g; t < npt; t += TWO ? 1 : 2) {
        ok = wait(&s_sfull[g], ns++, first ? a.first_wait : DS_WAIT_LIMIT);
        ok = __all_sync(0xFFFFFFFFu, ok);
        first = false;
        if (!ok) break;
        ds_tc_fence_after();
        const int64_t key0 = int64_t(p.t0 + t) * TA_KT;
        if (key0 + TA_KT > len) {
          // the item's last tile: values past the last key may be anything in the page, and 0 times
          // that need not be 0
          const uint32_t sv = seq + (TWO ? 2 * t + 1 : min(npt, t + 2) + t);
          ok = __all_sync(0xFFFFFFFFu, wait(&s_full[sv % NS], sv / NS, DS_WAIT_LIMIT));
          if (!ok) break;
          const int k0 = int(len - key0), k1 = min(TA_KT, (k0 + a.box - 1) / a.box * a.box);
          uint8_t* st = sR + (sv % NS) * STAGE;
          for (int u = lr; u < (k1 - k0) * NC * 8; u += 128) {
            const int key = k0 + u / (NC * 8), c = u % (NC * 8);
            *reinterpret_cast<uint4*>(st + (c >> 3) * TA_CHUNK + key * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
          ds_fence_proxy_async_smem();
        }
        if (live) {
          const bool masked = key0 + TA_KT > ctx;              // drafted nodes, or the end, among the keys
          uint32_t bits[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
          if (masked) {
#pragma unroll
            for (int w = 0; w < 4; ++w) bits[w] = ta_mask32(a, p.r, i, n, key0 + 32 * w - ctx);
          }
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            ds_tmem_ld_32x32b_x32(tS + 32 * c, v);
            if (masked) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = (bits[c] >> e) & 1u ? v[e] : -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 32; e += 2) mx = fmaxf(mx, fmaxf(v[e], v[e + 1]));
          }
          const float m2 = mx == -INFINITY ? -INFINITY : CAP ? ta_tanh(mx * sc, cap2) : mx * sc;
          const bool up = m2 > mref + TA_RISE || (mref == -INFINITY && m2 > -INFINITY);
          if (__any_sync(0xFFFFFFFFu, up)) {
            const float f = up ? ta_ex2(mref - m2) : 1.0f;     // 0 from -inf
            if (has) {
#pragma unroll
              for (int c = 0; c < DP / 16; ++c) {
                float o[16];
                uint32_t w[16];
                ds_tmem_ld_32x32b_x16(tO + 16 * c, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * f);
                ta_tmem_st_x16(tO + 16 * c, w);
              }
            }
            l *= f;
            if (up) mref = m2;
          }
          const float mu = mref == -INFINITY ? 0.0f : mref;
          const uint64_t sc2 = ds_f2(sc, sc), nm2 = ds_f2(-mu, -mu);
          uint64_t sum = ds_f2(0.0f, 0.0f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float v[32];
            uint32_t w[16];
            ds_tmem_ld_32x32b_x32(tS + 32 * c, v);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              if (CAP) {
                x0 = ta_tanh(v[e] * sc, cap2) - mu;
                x1 = ta_tanh(v[e + 1] * sc, cap2) - mu;
              } else {
                const uint64_t x = ds_fma2(ds_f2(v[e], v[e + 1]), sc2, nm2);
                x0 = ds_f2lo(x);
                x1 = ds_f2hi(x);
              }
              if (masked) {
                x0 = (bits[c] >> e) & 1u ? x0 : -INFINITY;
                x1 = (bits[c] >> (e + 1)) & 1u ? x1 : -INFINITY;
              }
              x0 = ta_ex2(x0);
              x1 = ta_ex2(x1);
              sum = ds_add2(sum, ds_f2(x0, x1));
              w[e >> 1] = ta_pack(x0, x1);
            }
            ta_tmem_st_x16(tS + 16 * c, w);
          }
          l += ds_f2lo(sum) + ds_f2hi(sum);
          ta_tmem_wait_st();
        }
        has = true;
        ds_tc_fence_before();
        __syncwarp();
        if (lane == 0) ds_mbar_arrive(&s_pfull[g]);
      }
      if (!ok) break;
      // ---- the piece's result ----
      if (!TWO) {
        s_ml[np & 1][g][lr] = make_float2(mref, l);
        __syncwarp();
        if (lane == 0) ds_mbar_arrive(&s_mlfull);
      }
      ok = wait(&s_ofull, np, DS_WAIT_LIMIT) && (TWO || wait(&s_mlfull, np, DS_WAIT_LIMIT));
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      ds_tc_fence_after();
      if (live) {
        const bool valid = m < a.rows && i < n;
        float w0 = 1.0f, w1 = 0.0f;
        if (!TWO) {
          const float2 x = s_ml[np & 1][0][lr], y = s_ml[np & 1][1][lr];
          mref = fmaxf(x.x, y.x);
          w0 = x.x == -INFINITY ? 0.0f : ta_ex2(x.x - mref);
          w1 = y.x == -INFINITY ? 0.0f : ta_ex2(y.x - mref);
          l = w0 * x.y + w1 * y.y;
        }
        const bool any = valid && l != 0.0f;                   // also when l is not a number
        const float inv = any ? 1.0f / l : 0.0f;
        const bool whole = p.whole();
        const int d0 = TWO ? 0 : g * (DP / 2), d1 = TWO ? DP : d0 + DP / 2;
        const int64_t slot = p.slot(blockIdx.x);
        const int h = p.hk * a.G + m - i * a.G;
        const int64_t row = int64_t(p.r) * a.T + i;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.ldo + int64_t(h) * D;
        float4* part = a.part_o + slot * (D / 4) * a.rs + (m - p.g * a.rpg);
        float chk = 0.0f;
#pragma unroll
        for (int c = 0; c < (TWO ? DP : DP / 2) / 16; ++c) {
          const int d = d0 + 16 * c;
          float o[16];
          __syncwarp();
          if (TWO) {
            ds_tmem_ld_32x32b_x16(tO + 16 * c, o);
          } else {
            ds_tmem_ld_32x32b_x16(tl + TO + d, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= w0;
            if (npt > 1) {
              float y[16];
              ds_tmem_ld_32x32b_x16(tl + TO + DP + d, y);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __fmaf_rn(w1, y[e], o[e]);
            }
          }
          if (d < D && m < a.rows) {
#pragma unroll
            for (int e = 0; e < 16; ++e) chk = __fmaf_rn(o[e], 0.0f, chk);
            if (whole) {
#pragma unroll
              for (int e = 0; e < 16; e += 8) {
                uint4 y;
                y.x = any ? ta_pack(o[e] * inv, o[e + 1] * inv) : 0u;
                y.y = any ? ta_pack(o[e + 2] * inv, o[e + 3] * inv) : 0u;
                y.z = any ? ta_pack(o[e + 4] * inv, o[e + 5] * inv) : 0u;
                y.w = any ? ta_pack(o[e + 6] * inv, o[e + 7] * inv) : 0u;
                if (d + e < D) *reinterpret_cast<uint4*>(out + d + e) = y;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                if (d + e < D) part[int64_t((d + e) >> 2) * a.rs] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
        __syncwarp();
        if (m < a.rows && (TWO || g == 0)) {
          if (!whole) a.part_ml[slot * a.rs + m - p.g * a.rpg] = valid ? make_float2(mref, l) : make_float2(-INFINITY, 0.0f);
          else if (a.lse) a.lse[row * a.Hq + h] = any ? (mref + log2f(l)) * TA_LN2 : -INFINITY;
        }
        // rows that came out not finite with nodes among the keys
        uint32_t redo = __ballot_sync(0xFFFFFFFFu, any && !(chk == 0.0f) && int64_t(p.t1) * TA_KT > ctx);
        while (redo) {
          const int src = __ffs(int(redo)) - 1;
          redo &= redo - 1;
          const int mm = __shfl_sync(0xFFFFFFFFu, m, src);
          const float mr = __shfl_sync(0xFFFFFFFFu, mref, src), iv = __shfl_sync(0xFFFFFFFFu, inv, src);
          const int ii = mm / a.G;
          ta_row_again(a, p.r, p.hk, mm, int64_t(p.t0) * TA_KT, int64_t(p.t1) * TA_KT, mr, iv, d0, min(d1, D),
                       whole ? reinterpret_cast<__nv_bfloat16*>(a.out) + (int64_t(p.r) * a.T + ii) * a.ldo +
                                   int64_t(p.hk * a.G + mm - ii * a.G) * D
                             : nullptr,
                       a.part_o + slot * (D / 4) * a.rs + (mm - p.g * a.rpg));
        }
      }
      ds_tc_fence_before();
      __syncwarp();
      if (lane == 0) ds_mbar_arrive(&s_ofree);
      seq += 2 * npt;
      ++np;
    }
  }
  __syncthreads();
  if (warp == 1) {
    ds_tc_fence_after();
    ds_tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of one item's rows: thread (row, four columns), the parts in the order of
// the blocks that left them. Blocks whose item was finished by one block alone leave at once.
template <typename T>
__global__ void __launch_bounds__(256) tree_attn_join_kernel(const TaArgs a, int32_t grid, int32_t nrb) {
  ds_pdl_trigger();
  ds_pdl_wait();
  const int64_t item = blockIdx.x / nrb;
  const int rb = int(blockIdx.x - item * nrb);
  const int64_t hm = int64_t(a.c.heads) * a.mg;
  const int r = int(item / hm);
  const int64_t sub = item - r * hm;
  const int hk = int(sub / a.mg), g = int(sub - int64_t(hk) * a.mg);
  const int64_t total = int64_t(a.pref[a.R]) * hm, nt = a.pref[r + 1] - a.pref[r], g0 = int64_t(a.pref[r]) * hm + sub * nt;
  const int64_t b0 = ((g0 + 1) * grid + total - 1) / total - 1;          // block that holds tile g0
  if (total * (b0 + 1) / grid >= g0 + nt) return;                       // whole
  const int64_t b1 = ((g0 + nt) * grid + total - 1) / total - 1;        // block of the last tile
  const int D = a.c.head_dim;
  const int lrow = rb * 8 + (threadIdx.x & 7), m = g * a.rpg + lrow;
  if (lrow >= a.rpg || m >= a.rows) return;
  float M = -INFINITY;
  for (int64_t b = b0; b <= b1; ++b) {
    if (total * (b + 1) / grid == total * b / grid) continue;
    M = fmaxf(M, a.part_ml[(2 * b + (total * b / grid > g0 ? 0 : 1)) * a.rs + lrow].x);
  }
  const int i = m / a.G, h = hk * a.G + m - i * a.G;
  const int64_t row = int64_t(r) * a.T + i;
  for (int c = threadIdx.x >> 3; c < D / 4; c += 32) {
    float L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t b = b0; b <= b1; ++b) {
      if (total * (b + 1) / grid == total * b / grid) continue;
      const int64_t slot = 2 * b + (total * b / grid > g0 ? 0 : 1);
      const float2 ml = a.part_ml[slot * a.rs + lrow];
      if (ml.y == 0.0f) continue;                      // nothing seen (a sum that is not a number goes on)
      const float w = ta_ex2(ml.x - M);
      const float4 x = a.part_o[(slot * (D / 4) + c) * a.rs + lrow];
      L = __fmaf_rn(w, ml.y, L);
      o.x = __fmaf_rn(w, x.x, o.x);
      o.y = __fmaf_rn(w, x.y, o.y);
      o.z = __fmaf_rn(w, x.z, o.z);
      o.w = __fmaf_rn(w, x.w, o.w);
    }
    const bool any = L != 0.0f;
    const float inv = any ? 1.0f / L : 0.0f;
    T* out = reinterpret_cast<T*>(a.out) + row * a.ldo + int64_t(h) * D + 4 * c;
    const float y[4] = {any ? o.x * inv : 0.0f, any ? o.y * inv : 0.0f, any ? o.z * inv : 0.0f, any ? o.w * inv : 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 2) out[e] = __float2bfloat16_rn(y[e]);
      else out[e] = y[e];
    }
    if (c == 0 && a.lse) a.lse[row * a.Hq + h] = any ? (M + log2f(L)) * TA_LN2 : -INFINITY;
  }
}

// Tensor map of one buffer of the cache: (column, place, head, page), boxes of 64 columns x `box` places.
bool ta_tensor_map(CUtensorMap* m, void* base, const dspark_kvcache& c, int box) {
  const DsEncodeFn fn = ds_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.page_size), cuuint64_t(c.heads), cuuint64_t(c.num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(c.token_stride) * 2, cuuint64_t(c.head_stride) * 2, cuuint64_t(c.page_stride) * 2};
  const cuuint32_t bx[4] = {64, cuuint32_t(box), 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DP, bool TWO, bool CAP>
cudaError_t ta_launch_tc(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  constexpr size_t smem = ta_smem<DP, TWO>();
  const cudaError_t e = ds_ensure_smem(reinterpret_cast<const void*>(tree_attn_tc_kernel<DP, TWO, CAP>), smem);
  if (e != cudaSuccess) return e;
  return ds_launch(tree_attn_tc_kernel<DP, TWO, CAP>, dim3(unsigned(grid)), dim3(TA_THREADS), smem, st, a, k, v);
}

template <int DP>
cudaError_t ta_dispatch_tc(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (a.rpg > 128) return a.softcap > 0.0f ? ta_launch_tc<DP, true, true>(a, grid, k, v, st) : ta_launch_tc<DP, true, false>(a, grid, k, v, st);
  return a.softcap > 0.0f ? ta_launch_tc<DP, false, true>(a, grid, k, v, st) : ta_launch_tc<DP, false, false>(a, grid, k, v, st);
}

constexpr size_t TA_WS_PREF = 4352;        // pref[TA_MAXR + 1], rounded up to 256 bytes

}  // namespace

// Partial results of 2 slots per block: rs rows x (head_dim sums + maximum and sum). rs * head_dim is at
// most the group's T * cols / heads and at most 256 rows of 256 columns; head_dim >= 8, so the two
// statistics add at most a quarter.
extern "C" size_t dspark_internal_ws_tree_attention(int64_t R, int32_t T, int64_t cols, int32_t heads) {
  if (R <= 0 || T <= 0 || cols <= 0 || heads <= 0) return 0;
  const int64_t vals = std::min<int64_t>(int64_t(T) * (cols / heads), 256 * 256);
  const int64_t slots = 2 * int64_t(ds_num_sms());
  return TA_WS_PREF + size_t(ds_ceil_div(slots * vals * 5, 256) * 256);
}

extern "C" dspark_status dspark_tree_attention(const void* q, int64_t ldq, int64_t R, int32_t T, int32_t Hq,
                                               const dspark_kvcache* cache, const int32_t* ctx_len,
                                               const int32_t* n_nodes, const uint32_t* mask, float scale, float softcap,
                                               void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                                               int32_t* dev_status, dspark_stream_t stream) {
  DS_REQUIRE(ds_cache_ok(cache, false) && R >= 0 && R <= TA_MAXR && T >= 1 && T <= TA_MAXT);
  DS_REQUIRE(Hq >= 1 && Hq <= 1024 && Hq % cache->heads == 0);
  const int64_t D = cache->head_dim;
  DS_REQUIRE(ldq >= Hq * D && ldo >= Hq * D && scale > 0.0f && scale < INFINITY && softcap >= 0.0f && softcap < INFINITY);
  if (R == 0) return DSPARK_OK;
  const size_t e = size_t(ds_dtype_size(cache->dtype));
  DS_REQUIRE(q && ctx_len && out && dev_status && ds_aligned(q, e) && ds_aligned(out, e));
  if (!ws || !ds_aligned(ws, 256) || ws_bytes < dspark_internal_ws_tree_attention(R, T, Hq * D, cache->heads))
    return DSPARK_EWORKSPACE;
  TaArgs a{};
  a.q = q; a.ldq = ldq; a.out = out; a.ldo = ldo; a.lse = lse; a.c = *cache; a.ctx_len = ctx_len; a.n_nodes = n_nodes;
  a.mask = mask; a.R = int32_t(R); a.T = T; a.Hq = Hq; a.G = Hq / cache->heads; a.W = (T + 31) / 32;
  a.rows = T * a.G; a.scale = scale; a.softcap = softcap; a.status = dev_status; a.first_wait = g_ds_first_wait_polls.load();
  int box = 128;
  while (cache->page_size % box) box >>= 1;
  // Tensor cores: rows of bf16 that TMA can copy (16-byte rows; eight places of a page are the smallest box
  // whose swizzle starts on its own pattern) and outputs that 16-byte stores can write.
  const bool tc = cache->dtype == DSPARK_BF16 && D <= 128 && box >= 8 && ds_cache_vec(cache) && ds_aligned(q, 16) &&
                  ds_aligned(out, 16) && ldq % 8 == 0 && ldo % 8 == 0 && cache->page_stride > 0 && cache->token_stride > 0 &&
                  cache->head_stride > 0;
  CUtensorMap mk, mv;
  const bool maps = tc && ta_tensor_map(&mk, cache->k, *cache, box) && ta_tensor_map(&mv, cache->v, *cache, box);
  a.kt = maps ? TA_KT : 64;
  a.box = box;
  a.rpg = maps ? (a.rows > 128 ? 256 : 128) : 64;
  a.mg = int32_t(ds_ceil_div(a.rows, a.rpg));
  a.rs = std::min(a.rows, a.rpg);
  const int nrb = int(ds_ceil_div(a.rs, 8));
  const int64_t jobs = R * cache->heads * int64_t(a.mg) * nrb;
  DS_REQUIRE(jobs <= INT32_MAX);
  const int grid = ds_num_sms();
  const int64_t slots = 2 * int64_t(grid);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  a.pref = reinterpret_cast<int32_t*>(w);
  a.part_o = reinterpret_cast<float4*>(w + TA_WS_PREF);
  a.part_ml = reinterpret_cast<float2*>(w + TA_WS_PREF + size_t(slots) * a.rs * D * 4);
  if (maps) DS_CUDA_TRY(D <= 64 ? ta_dispatch_tc<64>(a, grid, mk, mv, stream) : ta_dispatch_tc<128>(a, grid, mk, mv, stream));
  else DS_CUDA_TRY(ta_launch_float(a, grid, stream));
  if (cache->dtype == DSPARK_BF16)
    DS_CUDA_TRY(ds_launch(tree_attn_join_kernel<__nv_bfloat16>, dim3(unsigned(jobs)), dim3(256), 0, stream, a, grid, nrb));
  else
    DS_CUDA_TRY(ds_launch(tree_attn_join_kernel<float>, dim3(unsigned(jobs)), dim3(256), 0, stream, a, grid, nrb));
  return DSPARK_OK;
}
