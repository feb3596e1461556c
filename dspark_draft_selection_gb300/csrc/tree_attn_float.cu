// tree_attn_float.cu - dspark_tree_attention in float32 arithmetic: float32 caches, and bf16 caches
// that the tensor-core kernel does not take (head_dim above 128, pages that are no multiple of eight
// places, rows off 16-byte boundaries).
//
// One block of 256 threads works through its share of the line of tiles (tree_attn.cuh) with up to 64 query
// rows and 64 keys at a time. A thread holds RPT rows x 4 scores, then RPT rows x 2 UC columns of the result
// (RPT = 1..4, the least that covers the rows of a (request, key head); UC = head_dim / 32 rounded up), the
// row statistics being reduced over the 16 lanes that share a row. Keys and values stay in their own type in
// shared memory and are copied asynchronously, the values while the scores are computed; the weights take the
// keys' place. So two blocks fit an SM (head_dim <= 128) and one computes while the other waits for its
// copies. Bound by the FMA rate: 4 head_dim operations per query row and key, far above what HBM needs.
// Six requests of 13 nodes x 3 heads, 80 columns, up to 1,500 keys: FIGURE.
#include "tree_attn.cuh"

namespace {

constexpr int TF_KEYS = 64;
constexpr int TF_THREADS = 256;
constexpr int TF_LDP = TF_KEYS + 4;

// Shared memory: RPT * 16 query rows as float32; the key tile, whose place the weights take; the value tile.
template <typename T>
struct TfLayout {
  int ldq, ldk, ldv;           // elements of a row
  size_t q, k, v;              // bytes of each
  __host__ __device__ TfLayout(int D, int rows) {
    ldq = D + 4;
    ldk = D + 16 / int(sizeof(T));
    ldv = D;
    q = size_t(rows) * ldq * 4;
    const size_t kb = size_t(TF_KEYS) * ldk * sizeof(T), pb = size_t(rows) * TF_LDP * 4;
    k = kb > pb ? kb : pb;
    v = size_t(TF_KEYS) * ldv * sizeof(T);
  }
  __host__ __device__ size_t total() const { return q + k + v; }
};

DS_DEV float4 tf_4(const float* p) { return *reinterpret_cast<const float4*>(p); }
DS_DEV float4 tf_4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
DS_DEV float2 tf_2(const float* p) { return *reinterpret_cast<const float2*>(p); }
DS_DEV float2 tf_2(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
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

DS_DEV float tf_rowmax(float x) {
#pragma unroll
  for (int d = 8; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
  return x;
}
DS_DEV float tf_rowsum(float x) {
#pragma unroll
  for (int d = 8; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
  return x;
}

template <typename T, int RPT, int UC>
__global__ void __launch_bounds__(TF_THREADS, 2) tree_attn_float_kernel(const TaArgs a, bool veckv) {
  extern __shared__ uint4 smem4[];
  __shared__ TaLens s_len;
  __shared__ int64_t s_at[TF_KEYS];
  const int D = a.c.head_dim, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const TfLayout<T> lay(D, RPT * 16);
  uint8_t* base = reinterpret_cast<uint8_t*>(smem4);
  float* sQ = reinterpret_cast<float*>(base);
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
    for (int u = tid; u < RPT * 16 * D; u += TF_THREADS) {
      const int lr = u / D, d = u - lr * D, m = m0 + lr;
      float x = 0.0f;
      if (m < a.rows) {
        const int i = m / a.G;
        x = ds_load_elem<T>(q + (int64_t(p.r) * a.T + i) * a.ldq + int64_t(p.hk * a.G + m - i * a.G) * D + d);
      }
      sQ[lr * lay.ldq + d] = x;
    }
    float mref[RPT], l[RPT], o[RPT][2 * UC];
    int node[RPT];
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
      mref[x] = -INFINITY;
      l[x] = 0.0f;
      node[x] = min(m0 + ty * RPT + x, a.rows - 1) / a.G;
#pragma unroll
      for (int c = 0; c < 2 * UC; ++c) o[x][c] = 0.0f;
    }
    for (int t = p.t0; t < p.t1; ++t) {
      const int64_t key0 = int64_t(t) * TF_KEYS;
      if (tid < TF_KEYS) s_at[tid] = mine;
      __syncthreads();                               // also: the tile before is used up
      tf_copy(sK, lay.ldk, kc, s_at, D, veckv);
      tf_copy(sV, lay.ldv, vc, s_at, D, veckv);
      mine = tid < TF_KEYS ? slot_of(t + 1) : -1;
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();
      float s[RPT][4] = {};
      for (int d = 0; d < D; d += 4) {
        float4 kx[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) kx[b] = tf_4(sK + (tx + 16 * b) * lay.ldk + d);
#pragma unroll
        for (int x = 0; x < RPT; ++x) {
          const float4 qx = tf_4(sQ + (ty * RPT + x) * lay.ldq + d);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            s[x][b] = __fmaf_rn(qx.x, kx[b].x, s[x][b]);
            s[x][b] = __fmaf_rn(qx.y, kx[b].y, s[x][b]);
            s[x][b] = __fmaf_rn(qx.z, kx[b].z, s[x][b]);
            s[x][b] = __fmaf_rn(qx.w, kx[b].w, s[x][b]);
          }
        }
      }
      __syncthreads();                               // the keys make room for the weights
      const bool masked = key0 + TF_KEYS > ctx;
#pragma unroll
      for (int x = 0; x < RPT; ++x) {
        uint32_t bits[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (masked) {
          bits[0] = ta_mask32(a, p.r, node[x], n, key0 - ctx);
          bits[1] = ta_mask32(a, p.r, node[x], n, key0 + 32 - ctx);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b) {                // scores in units of log2, like the reference maximum
          s[x][b] = a.softcap > 0.0f ? a.softcap * tanhf(s[x][b] * a.scale / a.softcap) * TA_LOG2E : s[x][b] * (a.scale * TA_LOG2E);
          if (!((bits[b >> 1] >> (tx + 16 * (b & 1))) & 1u)) s[x][b] = -INFINITY;
          mx = fmaxf(mx, s[x][b]);
        }
        const float mn = fmaxf(mref[x], tf_rowmax(mx));
        const float f = mref[x] == -INFINITY ? 0.0f : exp2f(mref[x] - mn), mu = mn == -INFINITY ? 0.0f : mn;
        mref[x] = mn;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const bool seen = (bits[b >> 1] >> (tx + 16 * (b & 1))) & 1u;
          const float w = exp2f(s[x][b] - mu);
          sum += seen ? w : 0.0f;
          sP[(ty * RPT + x) * TF_LDP + tx + 16 * b] = seen ? w : -1.0f;   // -1: not seen
        }
        l[x] = __fmaf_rn(l[x], f, tf_rowsum(sum));
#pragma unroll
        for (int c = 0; c < 2 * UC; ++c) o[x][c] *= f;
      }
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
      auto add = [&](bool some) {                    // some: nodes among the keys that a row may not see
        for (int j = 0; j < TF_KEYS; j += 4) {
          float4 w[RPT];
#pragma unroll
          for (int x = 0; x < RPT; ++x) w[x] = tf_4(sP + (ty * RPT + x) * TF_LDP + j);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
#pragma unroll
            for (int u = 0; u < UC; ++u) {
              const int d = tx * 2 + 32 * u;
              if (d >= D) break;
              const float2 y = tf_2(sV + (j + e) * lay.ldv + d);
#pragma unroll
              for (int x = 0; x < RPT; ++x) {
                const float we = e == 0 ? w[x].x : e == 1 ? w[x].y : e == 2 ? w[x].z : w[x].w;
                if (some && we < 0.0f) continue;     // what the row does not see has no effect, whatever it is
                o[x][2 * u] = __fmaf_rn(we, y.x, o[x][2 * u]);
                o[x][2 * u + 1] = __fmaf_rn(we, y.y, o[x][2 * u + 1]);
              }
            }
          }
        }
      };
      if (masked) add(true);
      else add(false);
    }
    const bool whole = p.whole();
    const int64_t slot = p.slot(blockIdx.x);
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
      const int lr = ty * RPT + x, m = m0 + lr;
      if (lr >= a.rpg || m >= a.rows) break;
      const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
      const bool valid = i < n, any = valid && l[x] != 0.0f;
      const int64_t row = int64_t(p.r) * a.T + i;
      const float inv = any ? 1.0f / l[x] : 0.0f;
      if (tx == 0) {
        if (!whole) a.part_ml[slot * a.rs + lr] = valid ? make_float2(mref[x], l[x]) : make_float2(-INFINITY, 0.0f);
        else if (a.lse) a.lse[row * a.Hq + h] = any ? (mref[x] + log2f(l[x])) * TA_LN2 : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int d = tx * 2 + 32 * u;
        if (d >= D) break;
        if (!whole) {
          *reinterpret_cast<float2*>(a.part_o + (slot * a.rs + lr) * D + d) = make_float2(o[x][2 * u], o[x][2 * u + 1]);
        } else {
          T* out = reinterpret_cast<T*>(a.out) + row * a.ldo + int64_t(h) * D + d;
          tf_put(out, any ? o[x][2 * u] * inv : 0.0f);
          tf_put(out + 1, any ? o[x][2 * u + 1] * inv : 0.0f);
        }
      }
    }
  }
}

template <typename T, int RPT, int UC>
cudaError_t tf_launch(const TaArgs& a, int grid, cudaStream_t st) {
  const size_t smem = TfLayout<T>(a.c.head_dim, RPT * 16).total();
  const cudaError_t e = ds_ensure_smem(reinterpret_cast<const void*>(tree_attn_float_kernel<T, RPT, UC>), smem);
  if (e != cudaSuccess) return e;
  return ds_launch(tree_attn_float_kernel<T, RPT, UC>, dim3(unsigned(grid)), dim3(TF_THREADS), smem, st, a, ds_cache_vec(&a.c));
}

template <typename T, int RPT>
cudaError_t tf_columns(const TaArgs& a, int grid, cudaStream_t st) {
  const int D = a.c.head_dim;
  return D <= 64 ? tf_launch<T, RPT, 2>(a, grid, st) : D <= 96 ? tf_launch<T, RPT, 3>(a, grid, st)
       : D <= 128 ? tf_launch<T, RPT, 4>(a, grid, st) : tf_launch<T, RPT, 8>(a, grid, st);
}

template <typename T>
cudaError_t tf_rows(const TaArgs& a, int grid, cudaStream_t st) {
  switch (ds_ceil_div(a.rpg, 16)) {
    case 1: return tf_columns<T, 1>(a, grid, st);
    case 2: return tf_columns<T, 2>(a, grid, st);
    case 3: return tf_columns<T, 3>(a, grid, st);
    default: return tf_columns<T, 4>(a, grid, st);
  }
}

}  // namespace

cudaError_t ta_launch_float(const TaArgs& a, int grid, cudaStream_t st) {
  return a.c.dtype == DSPARK_BF16 ? tf_rows<__nv_bfloat16>(a, grid, st) : tf_rows<float>(a, grid, st);
}
