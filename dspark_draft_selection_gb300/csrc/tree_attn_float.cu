// tree_attn_float.cu - dspark_tree_attention in float32 arithmetic: float32 caches, and bf16 caches
// that the tensor-core kernel does not take (head_dim above 128, pages that are no multiple of eight
// places, rows off 16-byte boundaries).
//
// One block of eight warps works through its share of the line of tiles (tree_attn.cuh) with up to 64 query
// rows and 64 keys at a time. A warp owns RW rows (2, 4, 6 or 8, the least that covers the rows of a (request,
// key head)); its lanes are keys for the scores (two each) and columns for the result (UC = head_dim / 32
// rounded up), so a warp's weights are its own and need no block-wide barrier. Keys and values stay in their
// own type in shared memory and are copied asynchronously, the values while the scores are computed; the
// weights take the keys' place. Two blocks fit an SM (head_dim <= 128): one computes while the other waits.
// Bound by what shared memory returns to registers - RW + 2 values for 2 RW FMAs of the scores - and, where
// a block has one tile, by the latency of its phases. Six requests of 13 nodes x 3 heads, 80 columns and up
// to 1,500 keys (one tile a block): 27.9 us with the join. Rows: with 8 RW = 64 whatever their number, 4, 32 and
// 64 rows take 133, 137 and 141 us (8 requests of 2,000-4,000 keys), with the least that covers them 62, 86, 141.
#include <type_traits>

#include "tree_attn.cuh"

namespace {

constexpr int TF_KEYS = 64;
constexpr int TF_THREADS = 256;
constexpr int TF_LDP = TF_KEYS + 4;

// Shared memory: 8 RW query rows as float32, four columns of all rows side by side, so that a warp's rows lie at
// constant offsets; the key tile, whose place the weights take; the value tile, its rows a constant 32 UC apart.
template <typename T>
struct TfLayout {
  int ldk;                     // elements of a key row
  size_t q, k, v;              // bytes of each
  __host__ __device__ TfLayout(int D, int rows, int uc) {
    ldk = D + 16 / int(sizeof(T));
    q = size_t(rows) * D * 4;
    const size_t kb = size_t(TF_KEYS) * ldk * sizeof(T), pb = size_t(rows) * TF_LDP * 4;
    k = kb > pb ? kb : pb;
    v = size_t(TF_KEYS) * uc * 32 * sizeof(T);
  }
  __host__ __device__ size_t total() const { return q + k + v; }
};

DS_DEV float4 tf_4(const float* p) { return *reinterpret_cast<const float4*>(p); }
DS_DEV float4 tf_4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
DS_DEV void tf_put(float* p, float x) { *p = x; }
DS_DEV void tf_put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// A tile's rows into shared memory: 16-byte asynchronous copies where rows are aligned, else elements;
// keys without a slot are zero. The caller waits.
template <typename T>
DS_DEV void tf_copy(T* dst, int ld, const T* src, const int64_t* s_at, int D, bool vec) {
  constexpr int E = 16 / int(sizeof(T));
  const int per = D / E;
  for (int u = threadIdx.x; u < TF_KEYS * per; u += TF_THREADS) {
    const int key = u / per, d = (u - key * per) * E;
    const int64_t at = s_at[key];
    T* to = dst + key * ld + d;
    if (at < 0) {
      *reinterpret_cast<uint4*>(to) = make_uint4(0, 0, 0, 0);
    } else if (vec) {
      ds_cp_async16(to, src + at + d);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) to[e] = src[at + d + e];
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// A capped score in units of log2 (out of line: the code of a tile, which short contexts run once, stays small).
__device__ __noinline__ float tf_capped(float s, float scale, float cap) { return cap * tanhf(s * scale / cap) * TA_LOG2E; }

template <typename T, int RW, int UC>
__global__ void __launch_bounds__(TF_THREADS, 2) tree_attn_float_kernel(const TaArgs a, bool vecq, bool veckv) {
  extern __shared__ uint4 smem4[];
  __shared__ TaLens s_len;
  __shared__ int64_t s_at[TF_KEYS];
  const int D = a.c.head_dim, tid = threadIdx.x, lane = tid & 31, row0 = (tid >> 5) * RW;
  constexpr int ROWS = RW * 8, LDV = UC * 32;
  const TfLayout<T> lay(D, ROWS, UC);
  uint8_t* base = reinterpret_cast<uint8_t*>(smem4);
  float4* sQ = reinterpret_cast<float4*>(base);       // [D / 4][ROWS]
  T* sK = reinterpret_cast<T*>(base + lay.q);
  float* sP = reinterpret_cast<float*>(base + lay.q);
  T* sV = reinterpret_cast<T*>(base + lay.q + lay.k);
  ds_pdl_trigger();
  ds_pdl_wait();
  ta_prefix(a, s_len);
  TaWalk walk;
  walk.init(s_len);
  TaPiece p;
  const T* q = reinterpret_cast<const T*>(a.q);
  while (walk.next(s_len, a, p)) {
    const int32_t ctx = s_len.ctx[p.r], n = s_len.n[p.r];
    const int64_t len = int64_t(ctx) + n;
    const T* kc = reinterpret_cast<const T*>(a.c.k) + p.hk * a.c.head_stride;
    const T* vc = reinterpret_cast<const T*>(a.c.v) + p.hk * a.c.head_stride;
    const int m0 = p.g * a.rpg;
    auto slot_of = [&](int t) {
      const int64_t key = int64_t(t) * TF_KEYS + tid;
      return t < p.t1 && key < len ? ta_slot(a, p.r, key) : int64_t(-1);
    };
    int64_t mine = tid < TF_KEYS ? slot_of(p.t0) : -1;
    {                                                // query rows, widened; four columns and row after row a thread
      const int per = D / 4, step = TF_THREADS / per, c = tid % per;
      const T* qr = q + int64_t(p.r) * a.T * a.ldq + int64_t(p.hk) * a.G * D + c * 4;
      int lr = tid / per, i = (m0 + lr) / a.G, h = (m0 + lr) - i * a.G;
#pragma unroll 4
      for (; lr < RW * 8; lr += step) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tid < per * step && m0 + lr < a.rows) {
          const T* at = qr + int64_t(i) * a.ldq + h * D;
          x = vecq ? tf_4(at)
                   : make_float4(ds_load_elem<T>(at), ds_load_elem<T>(at + 1), ds_load_elem<T>(at + 2), ds_load_elem<T>(at + 3));
        }
        if (tid < per * step) sQ[c * ROWS + lr] = x;
        for (h += step; h >= a.G; h -= a.G) ++i;
      }
    }
    float mref[RW], l[RW], o[RW][UC];
    int node[RW];
#pragma unroll
    for (int x = 0; x < RW; ++x) {
      mref[x] = -INFINITY;
      l[x] = 0.0f;
      node[x] = min(m0 + row0 + x, a.rows - 1) / a.G;
#pragma unroll
      for (int c = 0; c < UC; ++c) o[x][c] = 0.0f;
    }
    for (int t = p.t0; t < p.t1; ++t) {
      const int64_t key0 = int64_t(t) * TF_KEYS;
      if (tid < TF_KEYS) s_at[tid] = mine;
      __syncthreads();                               // also: the tile before is used up
      tf_copy(sK, lay.ldk, kc, s_at, D, veckv);
      tf_copy(sV, LDV, vc, s_at, D, veckv);
      mine = tid < TF_KEYS ? slot_of(t + 1) : -1;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      float s[RW][2] = {};
      const float4* qp = sQ + row0;
      const T* kp = sK + lane * lay.ldk;
      const T* kq = kp + 32 * lay.ldk;
#pragma unroll 1
      for (int d = 0; d < D; d += 4, qp += ROWS, kp += 4, kq += 4) {
        const float4 k0 = tf_4(kp), k1 = tf_4(kq);
#pragma unroll
        for (int x = 0; x < RW; ++x) {
          const float4 qx = qp[x];
          s[x][0] = __fmaf_rn(qx.x, k0.x, s[x][0]);
          s[x][1] = __fmaf_rn(qx.x, k1.x, s[x][1]);
          s[x][0] = __fmaf_rn(qx.y, k0.y, s[x][0]);
          s[x][1] = __fmaf_rn(qx.y, k1.y, s[x][1]);
          s[x][0] = __fmaf_rn(qx.z, k0.z, s[x][0]);
          s[x][1] = __fmaf_rn(qx.z, k1.z, s[x][1]);
          s[x][0] = __fmaf_rn(qx.w, k0.w, s[x][0]);
          s[x][1] = __fmaf_rn(qx.w, k1.w, s[x][1]);
        }
      }
      __syncthreads();                               // the keys make room for the weights
      const bool masked = key0 + TF_KEYS > ctx;
#pragma unroll
      for (int x = 0; x < RW; ++x) {
        bool seen[2] = {true, true};
        if (masked) {
#pragma unroll
          for (int b = 0; b < 2; ++b) seen[b] = (ta_mask32(a, p.r, node[x], n, key0 + 32 * b - ctx) >> lane) & 1u;
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {                // scores in units of log2, like the reference maximum
          s[x][b] = a.softcap > 0.0f ? tf_capped(s[x][b], a.scale, a.softcap) : s[x][b] * (a.scale * TA_LOG2E);
          if (!seen[b]) s[x][b] = -INFINITY;
        }
        const float mn = fmaxf(mref[x], ds_warp_max(fmaxf(s[x][0], s[x][1])));
        const float f = mref[x] == -INFINITY ? 0.0f : exp2f(mref[x] - mn), mu = mn == -INFINITY ? 0.0f : mn;
        mref[x] = mn;
        const float w0 = exp2f(s[x][0] - mu), w1 = exp2f(s[x][1] - mu);
        sP[(row0 + x) * TF_LDP + lane] = seen[0] ? w0 : -1.0f;           // -1: not seen
        sP[(row0 + x) * TF_LDP + lane + 32] = seen[1] ? w1 : -1.0f;
        l[x] = __fmaf_rn(l[x], f, ds_warp_sumf((seen[0] ? w0 : 0.0f) + (seen[1] ? w1 : 0.0f)));
#pragma unroll
        for (int c = 0; c < UC; ++c) o[x][c] *= f;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      // What a row does not see has no effect on it, whatever it is: with a value that is not finite in a tile
      // that holds nodes, every weight is looked at; else an unseen key's weight counts as 0.
      bool odd = false;
      if (masked) {
        for (int u = tid; u < TF_KEYS * (LDV / 4); u += TF_THREADS) {
          if (u % (LDV / 4) * 4 >= D) continue;      // columns past head_dim hold anything
          const float4 y = tf_4(sV + u * 4);
          odd = odd || !(fabsf(y.x) + fabsf(y.y) + fabsf(y.z) + fabsf(y.w) < INFINITY);
        }
        odd = __syncthreads_or(odd);
      }
      const int keys = int(min(int64_t(TF_KEYS), (len - key0 + 3) & ~int64_t(3)));   // past them all weights are -1
      auto add = [&](auto mode) {                    // 0: all seen, 1: unseen keys among them, 2: odd values too
        constexpr int MODE = decltype(mode)::value;
        const float* wp = sP + row0 * TF_LDP;
        const T* vp = sV + lane;
#pragma unroll 1
        for (int j = 0; j < keys; j += 4, wp += 4, vp += 4 * LDV) {
          float w[RW][4];
#pragma unroll
          for (int x = 0; x < RW; ++x) {
            const float4 y = tf_4(wp + x * TF_LDP);
            w[x][0] = y.x; w[x][1] = y.y; w[x][2] = y.z; w[x][3] = y.w;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (MODE == 1 && w[x][e] < 0.0f) w[x][e] = 0.0f;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int u = 0; u < UC; ++u) {
              const float y = ds_load_elem<T>(vp + e * LDV + 32 * u);
#pragma unroll
              for (int x = 0; x < RW; ++x) {
                if (MODE == 2 && w[x][e] < 0.0f) continue;
                o[x][u] = __fmaf_rn(w[x][e], y, o[x][u]);
              }
            }
          }
        }
      };
      if (!masked) add(std::integral_constant<int, 0>{});
      else if (!odd) add(std::integral_constant<int, 1>{});
      else add(std::integral_constant<int, 2>{});
    }
    const bool whole = p.whole();
    const int64_t slot = p.slot(blockIdx.x);
#pragma unroll
    for (int x = 0; x < RW; ++x) {
      const int lr = row0 + x, m = m0 + lr;
      if (lr >= a.rpg || m >= a.rows) break;
      const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
      const bool valid = i < n, any = valid && l[x] != 0.0f;
      const int64_t row = int64_t(p.r) * a.T + i;
      const float inv = any ? 1.0f / l[x] : 0.0f;
      if (lane == 0) {
        if (!whole) a.part_ml[slot * a.rs + lr] = valid ? make_float4(mref[x], l[x], l[x], 0.0f) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        else if (a.lse) a.lse[row * a.Hq + h] = any ? (mref[x] + log2f(l[x])) * TA_LN2 : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int d = lane + 32 * u;
        if (d >= D) break;
        if (!whole) a.part_o[(slot * a.rs + lr) * D + d] = o[x][u];
        else tf_put(reinterpret_cast<T*>(a.out) + row * a.ldo + int64_t(h) * D + d, any ? o[x][u] * inv : 0.0f);
      }
    }
  }
}

template <typename T, int RW, int UC>
cudaError_t tf_launch(const TaArgs& a, int grid, cudaStream_t st) {
  const size_t smem = TfLayout<T>(a.c.head_dim, RW * 8, UC).total();
  const cudaError_t e = ds_ensure_smem(reinterpret_cast<const void*>(tree_attn_float_kernel<T, RW, UC>), smem);
  if (e != cudaSuccess) return e;
  return ds_launch(tree_attn_float_kernel<T, RW, UC>, dim3(unsigned(grid)), dim3(TF_THREADS), smem, st, a,
                   ds_aligned(a.q, 16) && (a.ldq * int64_t(sizeof(T))) % 16 == 0, ds_cache_vec(&a.c));
}

template <typename T, int RW>
cudaError_t tf_columns(const TaArgs& a, int grid, cudaStream_t st) {
  const int D = a.c.head_dim;
  return D <= 64 ? tf_launch<T, RW, 2>(a, grid, st) : D <= 96 ? tf_launch<T, RW, 3>(a, grid, st)
       : D <= 128 ? tf_launch<T, RW, 4>(a, grid, st) : tf_launch<T, RW, 8>(a, grid, st);
}

template <typename T>
cudaError_t tf_rows(const TaArgs& a, int grid, cudaStream_t st) {
  switch (ds_ceil_div(a.rpg, 16)) {
    case 1: return tf_columns<T, 2>(a, grid, st);
    case 2: return tf_columns<T, 4>(a, grid, st);
    case 3: return tf_columns<T, 6>(a, grid, st);
    default: return tf_columns<T, 8>(a, grid, st);
  }
}

}  // namespace

cudaError_t ta_launch_float(const TaArgs& a, int grid, cudaStream_t st) {
  return a.c.dtype == DSPARK_BF16 ? tf_rows<__nv_bfloat16>(a, grid, st) : tf_rows<float>(a, grid, st);
}
