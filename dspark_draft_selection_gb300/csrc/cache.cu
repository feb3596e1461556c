// cache.cu - the paged key/value cache around a verification step: rotary positions with the append
// of the drafted nodes (dspark_rope_append) and the commit of the accepted ones
// (dspark_cache_commit).
//
// optimum-intel PR #2098 ("Export DFlash v2 and DSpark drafts for PagedAttention and continuous
// batching") and openvino.genai PR #4847 (Fixes > Split validation windows) run the target over a
// paged cache; they leave its layout and these two steps to the runtime.
#include "dspark_common.cuh"
#include "host_common.h"

namespace {

constexpr int RA_THREADS = 128;
constexpr int RA_MAXROWS = 2;
constexpr int CM_THREADS = 128;
constexpr int CM_MAXT = 512;
constexpr int CM_BATCH = 8;

// Element offset of slot `s` of request r (head 0, column 0, layer 0), or -1 for a slot past the
// table's row or a page id out of range.
DS_DEV int64_t kv_slot(const dspark_kvcache& c, int64_t r, int64_t s) {
  const int64_t e = s / c.page_size;
  if (s < 0 || e >= c.table_pages) return -1;
  const int32_t p = c.page_table[r * c.ld_table + e];
  if (p < 0 || p >= c.num_pages) return -1;
  return int64_t(p) * c.page_stride + (s - e * c.page_size) * c.token_stride;
}

struct RaArgs {
  const void *q, *k, *v;
  void* q_out;
  int64_t ldq, ldk, ldv, ldo, rows;
  int32_t T, Hq, A, rot, interleaved;
  const int32_t *pos, *axis, *ctx_len, *n_nodes;
  const float* cos_sin;
  int64_t P;
  dspark_kvcache c;
  int32_t* status;
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) RaVec {
  T e[VEC];
};
DS_DEV float ra_f(float x) { return x; }
DS_DEV float ra_f(__nv_bfloat16 x) { return __bfloat162float(x); }
DS_DEV void ra_set(float& y, float x) { y = x; }
DS_DEV void ra_set(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// Every byte moves once, so the kernel is bound by HBM for many rows and by latency for few. A block of 128
// threads takes one or two node slots: their cosines and sines (gathered over the position axes) are staged in
// shared memory once for all heads, then the threads go over the rows' work items, an item being VEC columns
// of both halves of a rotated head, VEC columns a head passes through unrotated, or VEC columns of a value
// head. VEC * sizeof(T) is 16 bytes where the layout allows, then four elements, else one. With few rows
// grid.y splits the items of a row.
// 12,002 rows of 32 + 2 x 8 heads of 128 bf16 columns, three axes: 45.9 us, 5.6 TB/s of the bytes that have to
// move (float32: 85.7 us, 5.9 TB/s). What carries it is the number of blocks an SM holds (12, at 40 registers), since
// each waits for its page and its table rows before it moves anything: blocks of 256 threads with four rows 49-51 us,
// items two and three at a time (fewer blocks) 55 and 66 us, eight rows a block 58-64 us.
template <typename T, int VEC, int NR>
__global__ void __launch_bounds__(RA_THREADS, NR > 1 ? 12 : 1) rope_append_kernel(const RaArgs a) {
  using V = RaVec<T, VEC>;
  __shared__ __align__(16) float s_cs[NR][256];
  __shared__ int64_t s_slot[NR];                     // >= 0 slot offset; -1 a slot without a place; -2 not a node
  const int tid = threadIdx.x;
  const int64_t row0 = int64_t(blockIdx.x) * NR;
  ds_pdl_trigger();
  ds_pdl_wait();
  if (tid < NR) {
    int64_t at = -2;
    const int64_t row = row0 + tid;
    if (row < a.rows) {
      const int64_t r = row / a.T, i = row - r * a.T;
      int32_t n = a.n_nodes ? a.n_nodes[r] : a.T;
      const int32_t c = a.ctx_len[r];
      if (n < 0 || n > a.T || c < 0) {
        ds_set_error(a.status, DSPARK_EINVAL);
        n = 0;
      }
      if (i < n) {
        at = kv_slot(a.c, r, int64_t(c) + i);
        if (at < 0) ds_set_error(a.status, DSPARK_ERANGE);
      }
    }
    s_slot[tid] = at;
  }
  const int h = a.rot / 2;
  for (int u = tid; u < NR * h; u += RA_THREADS) {
    const int m = u / h, f = u - m * h;
    const int64_t row = row0 + m;
    if (row >= a.rows) break;
    int32_t ax = a.axis ? a.axis[f] : 0;
    bool bad = ax < 0 || ax >= a.A;
    if (bad) ax = 0;
    int64_t p = a.pos[row * a.A + ax];
    if (p < 0 || p >= a.P) {
      const int64_t r = row / a.T;                   // slots past the nodes may hold anything
      bad = bad || (row - r * a.T) < (a.n_nodes ? a.n_nodes[r] : a.T);
      p = 0;
    }
    if (bad) ds_set_error(a.status, DSPARK_ERANGE);
    s_cs[m][f] = a.cos_sin[p * a.rot + f];
    s_cs[m][h + f] = a.cos_sin[p * a.rot + h + f];
  }
  __syncthreads();
  const int D = a.c.head_dim, Hk = a.c.heads, H = a.Hq + Hk;
  const int npair = a.interleaved && VEC > 1 ? a.rot / VEC : h / VEC;    // rotated items of a head
  const T* q = reinterpret_cast<const T*>(a.q);
  const T* k = reinterpret_cast<const T*>(a.k);
  const T* v = reinterpret_cast<const T*>(a.v);
  T* qo = reinterpret_cast<T*>(a.q_out);
  T* kc = reinterpret_cast<T*>(a.c.k);
  T* vc = reinterpret_cast<T*>(a.c.v);
  const int first = blockIdx.y * RA_THREADS + tid, step = gridDim.y * RA_THREADS;
  // walks items (head, x) of `per` a head, `step` apart, without a division each
  struct Item {
    int hd, x, per, shd, sx;
    DS_DEV Item(int at, int per_, int step_) : per(per_) {
      hd = at / per;
      x = at - hd * per;
      shd = step_ / per;
      sx = step_ - shd * per;
    }
    DS_DEV void next() {
      hd += shd;
      x += sx;
      if (x >= per) {
        x -= per;
        ++hd;
      }
    }
  };
  // "head" hv of the block: head hv % H of its row hv / H (one or two rows)
  const int rows = int(min(int64_t(NR), a.rows - row0)), heads = rows * H;
  struct Place {
    const T* src;              // null: a query of a slot that is no node, which becomes zero
    T* dst;                    // null: a key without a place, which is not written
    int m;
  };
  auto place = [&](int hv) {
    Place p;
    p.m = NR > 1 && hv >= H ? 1 : 0;
    const int hd = hv - p.m * H;
    const int64_t row = row0 + p.m, at = s_slot[p.m];
    if (hd < a.Hq) {
      p.src = at == -2 ? nullptr : q + row * a.ldq + int64_t(hd) * D;
      p.dst = qo + row * a.ldo + int64_t(hd) * D;
    } else {
      p.src = at < 0 ? nullptr : k + row * a.ldk + int64_t(hd - a.Hq) * D;
      p.dst = at < 0 ? nullptr : kc + at + (hd - a.Hq) * a.c.head_stride;
    }
    return p;
  };
  // rotated columns: an item is VEC columns of whole pairs, or both halves' VEC
  const bool whole = VEC > 1 && a.interleaved;
  for (Item it(first, npair, step); it.hd < heads; it.next()) {
    const Place p = place(it.hd);
    if (!p.dst) continue;
    const int f = it.x * VEC, d1 = a.interleaved && VEC == 1 ? 2 * f : f, d2 = a.interleaved ? 2 * f + 1 : h + f;
    V y1 = {}, y2 = {};
    if (p.src) {
      y1 = *reinterpret_cast<const V*>(p.src + d1);
      if (!whole) y2 = *reinterpret_cast<const V*>(p.src + d2);
    }
    const float* cs = s_cs[p.m] + (whole ? f / 2 : f);
    if (whole) {
#pragma unroll
      for (int e = 0; e + 1 < VEC; e += 2) {
        const float c = cs[e / 2], s = cs[h + e / 2];
        const float x1 = ra_f(y1.e[e]), x2 = ra_f(y1.e[e + 1]);
        ra_set(y1.e[e], __fmaf_rn(x1, c, -__fmul_rn(x2, s)));
        ra_set(y1.e[e + 1], __fmaf_rn(x2, c, __fmul_rn(x1, s)));
      }
      *reinterpret_cast<V*>(p.dst + d1) = y1;
    } else {
      float c[VEC], s[VEC];
      if constexpr (VEC % 4 == 0) {                    // offsets are multiples of four
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          *reinterpret_cast<float4*>(c + e) = *reinterpret_cast<const float4*>(cs + e);
          *reinterpret_cast<float4*>(s + e) = *reinterpret_cast<const float4*>(cs + h + e);
        }
      } else {
        c[0] = cs[0];
        s[0] = cs[h];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float x1 = ra_f(y1.e[e]), x2 = ra_f(y2.e[e]);
        ra_set(y1.e[e], __fmaf_rn(x1, c[e], -__fmul_rn(x2, s[e])));
        ra_set(y2.e[e], __fmaf_rn(x2, c[e], __fmul_rn(x1, s[e])));
      }
      *reinterpret_cast<V*>(p.dst + d1) = y1;
      *reinterpret_cast<V*>(p.dst + d2) = y2;
    }
  }
  if (a.rot < D) {                                     // columns past the rotated ones
    for (Item pt(first, (D - a.rot) / VEC, step); pt.hd < heads; pt.next()) {
      const Place p = place(pt.hd);
      const int d = a.rot + pt.x * VEC;
      V y = {};
      if (p.src) y = *reinterpret_cast<const V*>(p.src + d);
      if (p.dst) *reinterpret_cast<V*>(p.dst + d) = y;
    }
  }
  for (Item vt(first, D / VEC, step); vt.hd < rows * Hk; vt.next()) {    // values
    const int m = NR > 1 && vt.hd >= Hk ? 1 : 0, hd = vt.hd - m * Hk;
    const int64_t at = s_slot[m];
    if (at >= 0)
      *reinterpret_cast<V*>(vc + at + hd * a.c.head_stride + vt.x * VEC) =
          *reinterpret_cast<const V*>(v + (row0 + m) * a.ldv + int64_t(hd) * D + vt.x * VEC);
  }
}

template <typename T, int VEC>
cudaError_t ra_launch(const RaArgs& a, cudaStream_t st) {
  const int64_t sms = ds_num_sms();
  // Two rows a block from one wave of blocks on: 2,432 rows of 48 heads 14.8 us against 16.1 us with one, 4,864
  // rows 25.1 against 28.7; below it one row a block spreads wider: 1,216 rows 7.5 against 9.2 us, 64 rows 3.6
  // against 5.5.
  if (a.rows >= sms * 12)
    return ds_launch(rope_append_kernel<T, VEC, RA_MAXROWS>, dim3(unsigned(ds_ceil_div(a.rows, RA_MAXROWS))),
                     dim3(RA_THREADS), 0, st, a);
  const int64_t items = int64_t(a.Hq + 2 * a.c.heads) * (a.c.head_dim / VEC);
  const int64_t split = std::min(ds_ceil_div(items, RA_THREADS), std::max<int64_t>(1, sms / a.rows));
  return ds_launch(rope_append_kernel<T, VEC, 1>, dim3(unsigned(a.rows), unsigned(split)), dim3(RA_THREADS), 0, st, a);
}

template <typename T>
cudaError_t ra_dispatch(const RaArgs& a, cudaStream_t st) {
  constexpr int V16 = 16 / int(sizeof(T));
  const int64_t e = sizeof(T);
  const int half = a.interleaved ? a.rot : a.rot / 2;
  const bool vec = ds_cache_vec(&a.c) && ds_aligned(a.q, 16) && ds_aligned(a.k, 16) && ds_aligned(a.v, 16) &&
                   ds_aligned(a.q_out, 16) && (a.ldq * e) % 16 == 0 && (a.ldk * e) % 16 == 0 &&
                   (a.ldv * e) % 16 == 0 && (a.ldo * e) % 16 == 0;
  if (vec && half % V16 == 0) return ra_launch<T, V16>(a, st);
  if (vec && half % 4 == 0) return ra_launch<T, 4>(a, st);
  return ra_launch<T, 1>(a, st);
}

// --- commit ---
// grid (layer x {K, V}, request): a block moves one buffer of one layer of one request, each thread a
// column of VEC elements down the path's rows. Sources lie above their destinations and both rise, so
// a thread that reads CM_BATCH rows before it writes them, batch after batch, never overwrites a row
// that it still has to read; rows that stay where they are are dropped first. Each moved byte is read
// and written once. 64 requests' branches of 1-12 rows in 16 layers (55 MB): 12.6 us, 4.4 TB/s, bound by the
// lookups before a block's first copy; one block for both buffers of a layer, with half the lookups, took the
// same time, and more for one request.
template <typename T, int VEC>
__global__ void __launch_bounds__(CM_THREADS) cache_commit_kernel(const dspark_kvcache c, const int32_t* ctx_len,
                                                                  const int32_t* path, const int32_t* n_accepted,
                                                                  int32_t T_, int32_t* new_len, int32_t* status) {
  using V = RaVec<T, VEC>;
  __shared__ int64_t s_src[CM_MAXT + CM_BATCH], s_dst[CM_MAXT + CM_BATCH];
  __shared__ int s_first;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.y;
  const int layer = blockIdx.x >> 1;
  ds_pdl_trigger();
  ds_pdl_wait();
  const int32_t ctx = ctx_len[r];
  int32_t n = n_accepted[r] + 1;
  bool bad = ctx < 0 || n_accepted[r] >= T_;
  if (n < 0) n = 0;
  if (!bad && path != nullptr) {
    for (int k = tid; k < n; k += CM_THREADS) {
      const int32_t p = path[r * T_ + k], before = k ? path[r * T_ + k - 1] : -1;
      bad = bad || p <= before || p >= T_;
    }
  }
  if (tid == 0) s_first = n;
  if (__syncthreads_or(bad)) {                       // the request stays as it was
    if (tid == 0) ds_set_error(status, DSPARK_EINVAL);
    n = 0;
  }
  if (blockIdx.x == 0 && tid == 0) new_len[r] = ctx + n;
  if (path == nullptr || n == 0) return;
  // rows before the first that moves stay: the path rises, so path[k] = k up to there
  for (int k = tid; k < n; k += CM_THREADS) {
    const int32_t p = path[r * T_ + k];
    int64_t src = -1, dst = -1;
    if (p != k) {
      atomicMin(&s_first, k);
      src = kv_slot(c, r, int64_t(ctx) + p);
      dst = kv_slot(c, r, int64_t(ctx) + k);
      if (src < 0 || dst < 0) {
        ds_set_error(status, DSPARK_ERANGE);
        src = dst = -1;
      }
    }
    s_src[k] = src;
    s_dst[k] = dst;
  }
  for (int k = n + tid; k < n + CM_BATCH; k += CM_THREADS) s_src[k] = s_dst[k] = -1;
  __syncthreads();
  const int per = c.head_dim / VEC, cols = c.heads * per;
  T* buf = reinterpret_cast<T*>((blockIdx.x & 1) ? c.v : c.k) + layer * c.layer_stride;
  for (int x = tid; x < cols; x += CM_THREADS) {
    T* col = buf + int64_t(x / per) * c.head_stride + (x % per) * VEC;
    for (int k = s_first; k < n; k += CM_BATCH) {
      V y[CM_BATCH];
#pragma unroll
      for (int b = 0; b < CM_BATCH; ++b)
        if (s_src[k + b] >= 0) y[b] = *reinterpret_cast<const V*>(col + s_src[k + b]);
#pragma unroll
      for (int b = 0; b < CM_BATCH; ++b)
        if (s_dst[k + b] >= 0) *reinterpret_cast<V*>(col + s_dst[k + b]) = y[b];
    }
  }
}

}  // namespace

extern "C" dspark_status dspark_rope_append(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                                            int64_t ldv, int64_t R, int32_t T, int32_t Hq, const int32_t* pos, int32_t A,
                                            const float* cos_sin, int64_t P, int32_t rot, const int32_t* axis,
                                            int32_t interleaved, const dspark_kvcache* cache, const int32_t* ctx_len,
                                            const int32_t* n_nodes, void* q_out, int64_t ldo, int32_t* dev_status,
                                            dspark_stream_t stream) {
  DS_REQUIRE(ds_cache_ok(cache, false) && R >= 0 && T >= 1 && Hq >= 1 && Hq <= 1024 && Hq % cache->heads == 0);
  const int64_t D = cache->head_dim;
  DS_REQUIRE(rot >= 2 && rot <= D && rot % 2 == 0 && A >= 1 && A <= 8 && P >= 1);
  DS_REQUIRE(ldq >= Hq * D && ldo >= Hq * D && ldk >= cache->heads * D && ldv >= cache->heads * D);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(R <= INT32_MAX / T);
  const size_t e = size_t(ds_dtype_size(cache->dtype));
  DS_REQUIRE(q && k && v && pos && cos_sin && ctx_len && q_out && dev_status);
  DS_REQUIRE(ds_aligned(q, e) && ds_aligned(k, e) && ds_aligned(v, e) && ds_aligned(q_out, e) && (q_out != q || ldo == ldq));
  RaArgs a{q, k, v, q_out, ldq, ldk, ldv, ldo, R * T, T, Hq, A, rot, interleaved != 0, pos, axis, ctx_len, n_nodes, cos_sin, P, *cache, dev_status};
  a.c.layer_stride = 0;
  DS_CUDA_TRY(cache->dtype == DSPARK_BF16 ? ra_dispatch<__nv_bfloat16>(a, stream) : ra_dispatch<float>(a, stream));
  return DSPARK_OK;
}

extern "C" dspark_status dspark_cache_commit(const dspark_kvcache* cache, const int32_t* ctx_len, const int32_t* path,
                                             const int32_t* n_accepted, int64_t R, int32_t T, int32_t* new_len,
                                             int32_t* dev_status, dspark_stream_t stream) {
  DS_REQUIRE(ds_cache_ok(cache, true) && cache->n_layers <= (1 << 20) && R >= 0 && R <= 65535 && T >= 1 && T <= CM_MAXT);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(ctx_len && n_accepted && new_len && dev_status && ds_commit_len_ok(new_len, ctx_len, n_accepted, path, R, T));
  const dim3 grid(path ? 2 * unsigned(cache->n_layers) : 1u, unsigned(R));
  const bool vec = ds_cache_vec(cache) && (cache->head_dim * ds_dtype_size(cache->dtype)) % 16 == 0;
  if (cache->dtype == DSPARK_BF16) {
    if (vec) DS_CUDA_TRY(ds_launch(cache_commit_kernel<__nv_bfloat16, 8>, grid, dim3(CM_THREADS), 0, stream, *cache, ctx_len, path, n_accepted, T, new_len, dev_status));
    else DS_CUDA_TRY(ds_launch(cache_commit_kernel<__nv_bfloat16, 1>, grid, dim3(CM_THREADS), 0, stream, *cache, ctx_len, path, n_accepted, T, new_len, dev_status));
  } else {
    if (vec) DS_CUDA_TRY(ds_launch(cache_commit_kernel<float, 4>, grid, dim3(CM_THREADS), 0, stream, *cache, ctx_len, path, n_accepted, T, new_len, dev_status));
    else DS_CUDA_TRY(ds_launch(cache_commit_kernel<float, 1>, grid, dim3(CM_THREADS), 0, stream, *cache, ctx_len, path, n_accepted, T, new_len, dev_status));
  }
  return DSPARK_OK;
}
