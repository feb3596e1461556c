// tree_attn_float.cu - dspark_tree_attention in float32 arithmetic: float32 caches, and bf16 caches
// that the tensor-core kernel does not take (head_dim above 128, pages that are no multiple of eight
// places, rows off 16-byte boundaries).
//
// One block of 256 threads works through its share of the line of tiles (tree_attn.cuh) with 64 query
// rows and 64 keys at a time, everything widened to float32 in shared memory. A thread holds 4 x 4
// scores, then 4 rows x 4 U columns of the result (U = head_dim / 64 rounded up), so a 16-byte
// shared-memory read feeds 8 FMAs or more; the row statistics are reduced over the 16 lanes that
// share a row. Bound by the FMA rate.
#include "tree_attn.cuh"

namespace {

constexpr int TF_ROWS = 64;
constexpr int TF_KEYS = 64;
constexpr int TF_THREADS = 256;
constexpr int TF_LDP = TF_KEYS + 4;

size_t tf_smem(int D) { return 4 * (size_t(TF_ROWS + TF_KEYS) * (D + 4) + size_t(TF_KEYS) * D + size_t(TF_ROWS) * TF_LDP); }

template <typename T>
DS_DEV float4 tf_ld4(const T* p, bool vec) {
  if constexpr (sizeof(T) == 4) {
    if (vec) return *reinterpret_cast<const float4*>(p);
    return make_float4(p[0], p[1], p[2], p[3]);
  } else {
    if (vec) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                         __uint_as_float(u.y & 0xFFFF0000u));
    }
    return make_float4(__bfloat162float(p[0]), __bfloat162float(p[1]), __bfloat162float(p[2]), __bfloat162float(p[3]));
  }
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

template <typename T, int U>
__global__ void __launch_bounds__(TF_THREADS) tree_attn_float_kernel(const TaArgs a, bool vecq, bool veckv) {
  extern __shared__ float4 smem4[];
  __shared__ TaLens s_len;
  __shared__ int64_t s_at[TF_KEYS];
  const int D = a.c.head_dim, ld = D + 4, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float* sQ = reinterpret_cast<float*>(smem4);
  float* sK = sQ + TF_ROWS * ld;
  float* sV = sK + TF_KEYS * ld;
  float* sP = sV + TF_KEYS * D;
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
    __syncthreads();
    for (int u = tid; u < TF_ROWS * (D / 4); u += TF_THREADS) {
      const int lr = u / (D / 4), d = (u % (D / 4)) * 4, m = m0 + lr;
      float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (m < a.rows) {
        const int i = m / a.G;
        x = tf_ld4(q + (int64_t(p.r) * a.T + i) * a.ldq + int64_t(p.hk * a.G + m - i * a.G) * D + d, vecq);
      }
      *reinterpret_cast<float4*>(sQ + lr * ld + d) = x;
    }
    float mref[4], l[4], o[4][4 * U];
    int node[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      mref[x] = -INFINITY;
      l[x] = 0.0f;
      node[x] = min(m0 + ty * 4 + x, a.rows - 1) / a.G;
#pragma unroll
      for (int c = 0; c < 4 * U; ++c) o[x][c] = 0.0f;
    }
    for (int t = p.t0; t < p.t1; ++t) {
      const int64_t key0 = int64_t(t) * TF_KEYS;
      __syncthreads();                               // the tile before is used up
      if (tid < TF_KEYS) s_at[tid] = key0 + tid < len ? ta_slot(a, p.r, key0 + tid) : -1;
      __syncthreads();
      for (int u = tid; u < TF_KEYS * (D / 4); u += TF_THREADS) {
        const int key = u / (D / 4), d = (u % (D / 4)) * 4;
        const int64_t at = s_at[key];
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f), y = x;
        if (at >= 0) {
          x = tf_ld4(kc + at + d, veckv);
          y = tf_ld4(vc + at + d, veckv);
        }
        *reinterpret_cast<float4*>(sK + key * ld + d) = x;
        *reinterpret_cast<float4*>(sV + key * D + d) = y;
      }
      __syncthreads();
      float s[4][4] = {};
      for (int d = 0; d < D; d += 4) {
        float4 kx[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) kx[b] = *reinterpret_cast<const float4*>(sK + (tx + 16 * b) * ld + d);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 qx = *reinterpret_cast<const float4*>(sQ + (ty * 4 + x) * ld + d);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            s[x][b] = __fmaf_rn(qx.x, kx[b].x, s[x][b]);
            s[x][b] = __fmaf_rn(qx.y, kx[b].y, s[x][b]);
            s[x][b] = __fmaf_rn(qx.z, kx[b].z, s[x][b]);
            s[x][b] = __fmaf_rn(qx.w, kx[b].w, s[x][b]);
          }
        }
      }
      const bool masked = key0 + TF_KEYS > ctx;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t bits[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (masked) {
          bits[0] = ta_mask32(a, p.r, node[x], n, key0 - ctx);
          bits[1] = ta_mask32(a, p.r, node[x], n, key0 + 32 - ctx);
        }
        float mx = -INFINITY;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          // in units of log2, like the reference maximum; natural exponential arguments keep full accuracy
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
          sP[(ty * 4 + x) * TF_LDP + tx + 16 * b] = seen ? w : -1.0f;   // -1: not seen
        }
        l[x] = __fmaf_rn(l[x], f, tf_rowsum(sum));
#pragma unroll
        for (int c = 0; c < 4 * U; ++c) o[x][c] *= f;
      }
      __syncwarp();                                  // a row's 16 threads are in one warp
      for (int j = 0; j < TF_KEYS; j += 4) {
        float w[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float4 y = *reinterpret_cast<const float4*>(sP + (ty * 4 + x) * TF_LDP + j);
          w[x][0] = y.x; w[x][1] = y.y; w[x][2] = y.z; w[x][3] = y.w;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int d = tx * 4 + 64 * u;
            if (d >= D) break;
            const float4 y = *reinterpret_cast<const float4*>(sV + (j + e) * D + d);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              if (masked && w[x][e] < 0.0f) continue;    // what the row does not see has no effect, whatever it is
              o[x][4 * u + 0] = __fmaf_rn(w[x][e], y.x, o[x][4 * u + 0]);
              o[x][4 * u + 1] = __fmaf_rn(w[x][e], y.y, o[x][4 * u + 1]);
              o[x][4 * u + 2] = __fmaf_rn(w[x][e], y.z, o[x][4 * u + 2]);
              o[x][4 * u + 3] = __fmaf_rn(w[x][e], y.w, o[x][4 * u + 3]);
            }
          }
        }
      }
    }
    const bool whole = p.whole();
    const int64_t slot = p.slot(blockIdx.x);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int lr = ty * 4 + x, m = m0 + lr;
      if (m >= a.rows) break;
      const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
      const bool valid = i < n, any = valid && l[x] != 0.0f;
      const int64_t row = int64_t(p.r) * a.T + i;
      const float inv = any ? 1.0f / l[x] : 0.0f;
      if (tx == 0) {
        if (!whole) a.part_ml[slot * a.rs + lr] = valid ? make_float2(mref[x], l[x]) : make_float2(-INFINITY, 0.0f);
        else if (a.lse) a.lse[row * a.Hq + h] = any ? (mref[x] + log2f(l[x])) * TA_LN2 : -INFINITY;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int d = tx * 4 + 64 * u;
        if (d >= D) break;
        if (!whole) {
          *reinterpret_cast<float4*>(a.part_o + (slot * a.rs + lr) * D + d) =
              make_float4(o[x][4 * u], o[x][4 * u + 1], o[x][4 * u + 2], o[x][4 * u + 3]);
        } else {
          T* out = reinterpret_cast<T*>(a.out) + row * a.ldo + int64_t(h) * D + d;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = any ? o[x][4 * u + e] * inv : 0.0f;
            if constexpr (sizeof(T) == 4) out[e] = y;
            else out[e] = __float2bfloat16_rn(y);
          }
        }
      }
    }
  }
}

template <typename T, int U>
cudaError_t tf_launch(const TaArgs& a, int grid, bool vecq, bool veckv, cudaStream_t st) {
  const size_t smem = tf_smem(a.c.head_dim);
  const cudaError_t e = ds_ensure_smem(reinterpret_cast<const void*>(tree_attn_float_kernel<T, U>), smem);
  if (e != cudaSuccess) return e;
  return ds_launch(tree_attn_float_kernel<T, U>, dim3(unsigned(grid)), dim3(TF_THREADS), smem, st, a, vecq, veckv);
}

template <typename T>
cudaError_t tf_dispatch(const TaArgs& a, int grid, cudaStream_t st) {
  const int64_t e = sizeof(T);
  const bool vecq = ds_aligned(a.q, 16) && (a.ldq * e) % 16 == 0, veckv = ds_cache_vec(&a.c);
  switch ((a.c.head_dim + 63) / 64) {
    case 1: return tf_launch<T, 1>(a, grid, vecq, veckv, st);
    case 2: return tf_launch<T, 2>(a, grid, vecq, veckv, st);
    case 3: return tf_launch<T, 3>(a, grid, vecq, veckv, st);
    default: return tf_launch<T, 4>(a, grid, vecq, veckv, st);
  }
}

}  // namespace

cudaError_t ta_launch_float(const TaArgs& a, int grid, cudaStream_t st) {
  return a.c.dtype == DSPARK_BF16 ? tf_dispatch<__nv_bfloat16>(a, grid, st) : tf_dispatch<float>(a, grid, st);
}
