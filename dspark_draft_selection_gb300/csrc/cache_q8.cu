// cache_q8.cu - the paged key/value cache kept in 8 bits: rotary positions with the quantising append
// (dspark_rope_append_q8), the commit of the accepted nodes (dspark_cache_commit_q8) and the read back
// (dspark_cache_read_q8).
//
// optimum-intel PR #2098 ("Export DFlash v2 and DSpark drafts for PagedAttention and continuous batching") and
// openvino.genai PR #4847 (Fixes > Split validation windows) leave the cache and its precision to the runtime; the format and
// the rounding are stated in dspark.h.
#include "cache_q8.cuh"

namespace {

constexpr int QA_THREADS = 128;
constexpr int QA_MAXROWS = 2;
constexpr int QC_THREADS = 128;
constexpr int QC_MAXT = 512;
constexpr int QC_BATCH = 8;
constexpr int QR_THREADS = 128;
constexpr int QR_ROWS = 8;

struct QaArgs {
  const void *q, *k, *v;
  void* q_out;
  int64_t ldq, ldk, ldv, ldo, rows;
  int32_t T, Hq, A, rot, interleaved;
  const int32_t *pos, *axis, *ctx_len, *n_nodes;
  const float* cos_sin;
  int64_t P;
  dspark_qcache c;
  int32_t* status;
};

// Walks items (head, x) of `per` a head, `step` apart, without a division each.
struct QaItem {
  int hd, x, per, shd, sx;
  DS_DEV QaItem(int at, int per_, int step) : per(per_) {
    hd = at / per;
    x = at - hd * per;
    shd = step / per;
    sx = step - shd * per;
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

// VEC consecutive columns as float32.
template <typename T, int VEC>
DS_DEV void qa_load(const T* p, float (&x)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = ds_vec_elem<T>(u, e);
  } else if constexpr (VEC == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    x[0] = ds_load_elem<T>(p);
  }
}
DS_DEV uint32_t qa_pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
template <typename T, int VEC>
DS_DEV void qa_store(T* p, const float (&y)[VEC]) {
  if constexpr (VEC == 8 && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = make_uint4(qa_pack(y[0], y[1]), qa_pack(y[2], y[3]), qa_pack(y[4], y[5]), qa_pack(y[6], y[7]));
  } else if constexpr (VEC == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else if constexpr (sizeof(T) == 2) {
    *p = __float2bfloat16_rn(y[0]);
  } else {
    *p = y[0];
  }
}

// Columns [d, d + VEC) of a head after its rotation, every product and sum rounded to float32 by itself. `x` are the columns themselves;
// the other column of each pair is loaded from the head (it was or will be another thread's own: a hit in L1), or, in adjacent pairs, among
// them. cs: cosines, then sines, of this row's rot / 2 pairs.
template <typename T, int VEC>
DS_DEV void qa_turn(const T* head, int d, int rot, bool interleaved, const float* cs, float (&x)[VEC]) {
  if (d >= rot) return;
  const int h = rot >> 1;
  if (interleaved) {
    if constexpr (VEC == 8) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        if (d + e >= rot) break;
        const float c = cs[(d + e) >> 1], s = cs[h + ((d + e) >> 1)], x1 = x[e], x2 = x[e + 1];
        x[e] = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
        x[e + 1] = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
      }
    } else {
      const float c = cs[d >> 1], s = cs[h + (d >> 1)], y = ds_load_elem<T>(head + (d ^ 1));
      x[0] = d & 1 ? __fadd_rn(__fmul_rn(x[0], c), __fmul_rn(y, s)) : __fsub_rn(__fmul_rn(x[0], c), __fmul_rn(y, s));
    }
  } else {
    const bool second = d >= h;
    const int f = second ? d - h : d;
    float y[VEC];
    qa_load<T, VEC>(head + (second ? f : d + h), y);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float c = cs[f + e], s = cs[h + f + e];
      x[e] = second ? __fadd_rn(__fmul_rn(x[e], c), __fmul_rn(y[e], s)) : __fsub_rn(__fmul_rn(x[e], c), __fmul_rn(y[e], s));
    }
  }
}

// One or two node slots a block: their cosines and sines are staged in shared memory once for all heads, then the threads go over
// the heads' items of VEC columns: queries, keys, values. The 32 / VEC neighbouring threads that hold a block of 32 columns find its largest
// magnitude by shuffles, so a column is loaded once and its code needs no second pass. Every byte moves once. 15,000 rows of 32 + 2 x 8 heads of 128
// in bf16: 68 us, 4.6 TB/s; the queries' part of it runs at the rate of HBM, the keys' and values' part (39 us of them) is bound by the instructions of
// rotation, magnitude and conversion. Few rows are bound by the latency of the lookups: 8 rows 3 us of the GPU. Two rows a block are compiled for 14 blocks
// an SM, 32 registers with 12 bytes of spills (68 us; for 12 blocks, 40 registers and no spills, 73 us, for 10 blocks 76 us; float32 101, 99 and 99 us).
template <typename T, int VEC, int NR>
__global__ void __launch_bounds__(QA_THREADS, NR > 1 ? 14 : 1) rope_append_q8_kernel(const QaArgs a) {
  constexpr int GROUP = Q8_BLOCK / VEC;                // threads of a block of columns
  __shared__ __align__(16) float s_cs[NR][256];
  __shared__ Q8Slot s_slot[NR];                        // at >= 0; -1 a slot without a place; -2 not a node
  const int tid = threadIdx.x;
  const int64_t row0 = int64_t(blockIdx.x) * NR;
  ds_pdl_trigger();
  ds_pdl_wait();
  if (tid < NR) {
    Q8Slot at{-2, -2};
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
        at = q8_slot(a.c, r, int64_t(c) + i);
        if (at.at < 0) ds_set_error(a.status, DSPARK_ERANGE);
      }
    }
    s_slot[tid] = at;
  }
  const int h = a.rot / 2;
  for (int u = tid; u < NR * h; u += QA_THREADS) {
    const int m = u / h, f = u - m * h;
    const int64_t row = row0 + m;
    if (row >= a.rows) break;
    int32_t ax = a.axis ? a.axis[f] : 0;
    bool bad = ax < 0 || ax >= a.A;
    if (bad) ax = 0;
    int64_t p = a.pos[row * a.A + ax];
    if (p < 0 || p >= a.P) {
      const int64_t r = row / a.T;                     // slots past the nodes may hold anything
      bad = bad || (row - r * a.T) < (a.n_nodes ? a.n_nodes[r] : a.T);
      p = 0;
    }
    if (bad) ds_set_error(a.status, DSPARK_ERANGE);
    s_cs[m][f] = a.cos_sin[p * a.rot + f];
    s_cs[m][h + f] = a.cos_sin[p * a.rot + h + f];
  }
  __syncthreads();
  const int D = a.c.head_dim, Hk = a.c.heads, rows = int(min(int64_t(NR), a.rows - row0));
  const int per = q8_blocks(D) * GROUP;                // items of a head, those past its last column among them
  const int first = blockIdx.y * QA_THREADS + tid, step = gridDim.y * QA_THREADS;
  const bool e4m3 = a.c.code == DSPARK_E4M3;
  const T* q = reinterpret_cast<const T*>(a.q);
  T* qo = reinterpret_cast<T*>(a.q_out);
  // queries. In place: a pair's two columns are written by the thread that read both.
  if (VEC > 1 || a.interleaved) {
    // halves: an item is VEC columns of both, or VEC columns past them; adjacent pairs: VEC columns, or (one at a time) a pair
    const int turned = a.interleaved ? (VEC > 1 ? a.rot / VEC : a.rot / 2) : h / VEC, qper = turned + (D - a.rot) / VEC;
    QaItem it(first, qper, step);
    for (; it.hd < rows * a.Hq; it.next()) {
      const int hv = it.hd, m = NR > 1 && hv >= a.Hq ? 1 : 0;
      const int d = it.x < turned ? it.x * (a.interleaved && VEC == 1 ? 2 : VEC) : a.rot + (it.x - turned) * VEC;
      const int64_t row = row0 + m;
      const T* src = q + row * a.ldq + int64_t(hv - m * a.Hq) * D;
      T* dst = qo + row * a.ldo + int64_t(hv - m * a.Hq) * D;
      const float* cs = s_cs[m];
      const bool node = s_slot[m].at != -2;
      float y[VEC] = {};
      if (node) qa_load<T, VEC>(src + d, y);
      if (d < a.rot && (!a.interleaved || VEC == 1)) {
        const int d2 = a.interleaved ? d + 1 : d + h, f = a.interleaved ? d >> 1 : d;
        float z[VEC] = {};
        if (node) {
          qa_load<T, VEC>(src + d2, z);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float c = cs[f + e], s = cs[h + f + e], x1 = y[e], x2 = z[e];
            y[e] = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
            z[e] = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
          }
        }
        qa_store<T, VEC>(dst + d2, z);
      } else if (node) {
        qa_turn<T, VEC>(src, d, a.rot, true, cs, y);
      }
      qa_store<T, VEC>(dst + d, y);
    }
  } else {                                             // single columns, halves: one thread a pair, one a column past them
    QaItem it(first, h + (D - a.rot), step);
    for (; it.hd < rows * a.Hq; it.next()) {
      const int hv = it.hd, x = it.x, m = NR > 1 && hv >= a.Hq ? 1 : 0;
      const int64_t row = row0 + m;
      const T* src = q + row * a.ldq + int64_t(hv - m * a.Hq) * D;
      T* dst = qo + row * a.ldo + int64_t(hv - m * a.Hq) * D;
      const bool node = s_slot[m].at != -2;
      const int d = x < h ? x : a.rot + x - h;
      float y[1] = {0.0f}, z[1] = {0.0f};
      if (node) {
        y[0] = ds_load_elem<T>(src + d);
        if (x < h) {
          const float c = s_cs[m][x], s = s_cs[m][h + x], x1 = y[0], x2 = ds_load_elem<T>(src + h + x);
          y[0] = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
          z[0] = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
        }
      }
      qa_store<T, 1>(dst + d, y);
      if (x < h) qa_store<T, 1>(dst + h + x, z);
    }
  }
  // keys, then values: the block's threads stay together for the shuffles
  bool odd = false;                                    // a number that is not finite was among a block's
  const int heads = rows * 2 * Hk;                     // per row: keys' heads, values' heads
  QaItem it(first, per, step);
  for (int u0 = first - tid; u0 < heads * per; u0 += step, it.next()) {
    const int hv = it.hd, x = it.x, m = NR > 1 && hv >= 2 * Hk ? 1 : 0, kv = hv - m * 2 * Hk;
    const bool value = kv >= Hk;
    const int hd = value ? kv - Hk : kv, d = x * VEC;
    const bool there = hv < heads && d < D;
    const Q8Slot at = s_slot[min(m, NR - 1)];
    float y[VEC] = {};
    if (there && at.at >= 0) {
      const T* src = value ? reinterpret_cast<const T*>(a.v) + (row0 + m) * a.ldv + int64_t(hd) * D
                           : reinterpret_cast<const T*>(a.k) + (row0 + m) * a.ldk + int64_t(hd) * D;
      qa_load<T, VEC>(src + d, y);
      if (!value) qa_turn<T, VEC>(src, d, a.rot, a.interleaved != 0, s_cs[m], y);
    }
    // largest magnitude of the block, as bits, which compare as numbers do; what is not finite lies above all that is
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) top = max(top, __float_as_uint(y[e]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < GROUP; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (__any_sync(0xFFFFFFFFu, top >= 0x7F800000u)) {
      odd = odd || top >= 0x7F800000u;
      top = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (y[e] != y[e]) y[e] = 0.0f;
        if (fabsf(y[e]) < INFINITY) top = max(top, __float_as_uint(fabsf(y[e])));
      }
#pragma unroll
      for (int o = 1; o < GROUP; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    if (!there || at.at < 0) continue;
    const uint32_t byte = q8_choose(__uint_as_float(top), e4m3);
    const float inv = __uint_as_float((254u - byte) << 23);
    uint8_t* dst = reinterpret_cast<uint8_t*>(value ? a.c.v : a.c.k) + at.at + int64_t(hd) * a.c.head_stride + d;
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(q8_codes(y[0], y[1], y[2], y[3], inv, e4m3), q8_codes(y[4], y[5], y[6], y[7], inv, e4m3));
    } else {
      *dst = uint8_t(q8_codes(y[0], 0.0f, 0.0f, 0.0f, inv, e4m3));
    }
    if (x % GROUP == 0) (value ? a.c.v_scale : a.c.k_scale)[at.scale + int64_t(hd) * a.c.scale_head_stride + x / GROUP] = uint8_t(byte);
  }
  if (odd) ds_set_error(a.status, DSPARK_ENONFINITE);
}

template <typename T, int VEC>
cudaError_t qa_launch(const QaArgs& a, cudaStream_t st) {
  // Two rows a block from twelve blocks an SM on: 15,000 rows 68 us, with one row each 95 us; 2,500 rows 22.1 and 23.7 us, but 1,500 rows 17.0 and
  // 15.9 us, 64 rows 16.5 and 14.8 us. With fewer rows than SMs a row's items are split over blocks (8 rows 15.0 us, unsplit 15.8 us, both with the call).
  const int64_t sms = ds_num_sms();
  if (a.rows >= sms * 12)
    return ds_launch(rope_append_q8_kernel<T, VEC, QA_MAXROWS>, dim3(unsigned(ds_ceil_div(a.rows, QA_MAXROWS))), dim3(QA_THREADS), 0, st, a);
  const int64_t items = int64_t(a.Hq + 2 * a.c.heads) * (a.c.head_dim / VEC);
  const int64_t split = std::min(ds_ceil_div(items, QA_THREADS), std::max<int64_t>(1, sms / a.rows));
  return ds_launch(rope_append_q8_kernel<T, VEC, 1>, dim3(unsigned(a.rows), unsigned(split)), dim3(QA_THREADS), 0, st, a);
}

template <typename T>
cudaError_t qa_dispatch(const QaArgs& a, cudaStream_t st) {
  const int64_t e = sizeof(T);
  const bool vec = ds_aligned(a.q, 16) && ds_aligned(a.k, 16) && ds_aligned(a.v, 16) && ds_aligned(a.q_out, 16) &&
                   (a.ldq * e) % 16 == 0 && (a.ldk * e) % 16 == 0 && (a.ldv * e) % 16 == 0 && (a.ldo * e) % 16 == 0 &&
                   q8_codes_aligned(&a.c, 8) && (a.interleaved ? a.rot : a.rot / 2) % 8 == 0;
  return vec ? qa_launch<T, 8>(a, st) : qa_launch<T, 1>(a, st);      // 15,000 rows 68 us, a column at a time 236 us
}

// --- commit ---
// grid (layer x {K, V}, request): a block moves one buffer's codes and scales of one layer of one request. Sources lie above their
// destinations and both rise, so a thread that reads QC_BATCH rows of its column before it writes them, batch after batch, never
// overwrites a row that it still has to read; rows that stay where they are are dropped first. Each moved byte is read and written once. Bound by
// the chain path, page, codes: 64 requests of 16 layers 10.2 us with 16 bytes and 4 scales at a time, 11.2 us with 8 bytes and one scale.
template <int VC, int VS>
__global__ void __launch_bounds__(QC_THREADS) cache_commit_q8_kernel(const dspark_qcache c, const int32_t* ctx_len, const int32_t* path,
                                                                     const int32_t* n_accepted, int32_t T_, int32_t* new_len,
                                                                     int32_t* status) {
  __shared__ Q8Slot s_src[QC_MAXT + QC_BATCH], s_dst[QC_MAXT + QC_BATCH];
  __shared__ int s_first;
  const int tid = threadIdx.x;
  const int64_t r = blockIdx.y;
  const int layer = blockIdx.x >> 1;
  ds_pdl_trigger();
  ds_pdl_wait();
  const int32_t ctx = ctx_len[r];
  int32_t n = n_accepted[r];
  bool bad = ctx < 0 || n >= T_;
  n = n < 0 || bad ? 0 : n + 1;
  if (path != nullptr) {
    for (int k = tid; k < n; k += QC_THREADS) {
      const int32_t p = path[r * T_ + k], before = k ? path[r * T_ + k - 1] : -1;
      bad = bad || p <= before || p >= T_;
    }
  }
  if (tid == 0) s_first = n;
  if (__syncthreads_or(bad)) {                         // the request stays as it was
    if (tid == 0) ds_set_error(status, DSPARK_EINVAL);
    n = 0;
  }
  if (blockIdx.x == 0 && tid == 0) new_len[r] = ctx + n;
  if (path == nullptr || n == 0) return;
  for (int k = tid; k < n; k += QC_THREADS) {
    const int32_t p = path[r * T_ + k];
    Q8Slot src{-1, -1}, dst{-1, -1};
    if (p != k) {                                      // rows before the first that moves stay
      atomicMin(&s_first, k);
      src = q8_slot(c, r, int64_t(ctx) + p);
      dst = q8_slot(c, r, int64_t(ctx) + k);
      if (src.at < 0 || dst.at < 0) {
        ds_set_error(status, DSPARK_ERANGE);
        src.at = dst.at = -1;
      }
    }
    s_src[k] = src;
    s_dst[k] = dst;
  }
  for (int k = n + tid; k < n + QC_BATCH; k += QC_THREADS) s_src[k].at = s_dst[k].at = -1;
  __syncthreads();
  const int per = c.head_dim / VC, cols = c.heads * per;              // columns of codes,
  const int sper = q8_blocks(c.head_dim) / VS, scols = c.heads * sper;   // and of scales behind them
  const bool value = blockIdx.x & 1;
  uint8_t* codes = reinterpret_cast<uint8_t*>(value ? c.v : c.k) + layer * c.layer_stride;
  uint8_t* scales = (value ? c.v_scale : c.k_scale) + layer * c.scale_layer_stride;
  auto move = [&](auto type, uint8_t* col, bool scale) {
    using V = decltype(type);
    for (int k = s_first; k < n; k += QC_BATCH) {
      V y[QC_BATCH];
#pragma unroll
      for (int b = 0; b < QC_BATCH; ++b)
        if (s_src[k + b].at >= 0) y[b] = *reinterpret_cast<const V*>(col + (scale ? s_src[k + b].scale : s_src[k + b].at));
#pragma unroll
      for (int b = 0; b < QC_BATCH; ++b)
        if (s_dst[k + b].at >= 0) *reinterpret_cast<V*>(col + (scale ? s_dst[k + b].scale : s_dst[k + b].at)) = y[b];
    }
  };
  for (int x = tid; x < cols + scols; x += QC_THREADS) {
    if (x < cols) {
      uint8_t* col = codes + int64_t(x / per) * c.head_stride + (x % per) * VC;
      if constexpr (VC == 16) move(uint4{}, col, false);
      else if constexpr (VC == 8) move(uint2{}, col, false);
      else move(uint8_t{}, col, false);
    } else {
      const int y = x - cols;
      uint8_t* col = scales + int64_t(y / sper) * c.scale_head_stride + (y % sper) * VS;
      if constexpr (VS == 4) move(uint32_t{}, col, true);
      else move(uint8_t{}, col, true);
    }
  }
}

// --- read back ---
struct QrArgs {
  dspark_qcache c;
  const int32_t *start, *n;
  int64_t rows, ld;
  int32_t S;
  void *k, *v;
  int32_t* status;
};

// Four E4M3 codes, through f16, which holds them all.
DS_DEV float4 qr_e4m3(uint32_t w) {
  float4 z;
  asm("{\n\t.reg .b16 l, h, a, b, c, d;\n\t.reg .b32 x, y;\n\tmov.b32 {l, h}, %4;\n\t"
      "cvt.rn.f16x2.e4m3x2 x, l;\n\tcvt.rn.f16x2.e4m3x2 y, h;\n\tmov.b32 {a, b}, x;\n\tmov.b32 {c, d}, y;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\tcvt.f32.f16 %2, c;\n\tcvt.f32.f16 %3, d;\n\t}"
      : "=f"(z.x), "=f"(z.y), "=f"(z.z), "=f"(z.w)
      : "r"(w));
  return z;
}

// A block reads QR_ROWS slots: their places are looked up once, then the threads go over the slots' heads (keys, then values) VEC codes at a
// time, side by side. Bound by HBM: 1 + 1/32 bytes read and 2 or 4 written a column. 136,000 slots of 8 heads of 128 to bf16: 141 us, 6.0 TB/s.
// Few loads a thread and small blocks are best, as reads and writes then alternate least far apart: 16 slots and 256 threads a block with four
// loads a thread 167 us, with two 148 us; 8 slots, 128 threads and two loads 141 us; one load 157 us. A number times its scale is exact in
// float32, and in bf16 too (eight bits of fraction hold every code).
template <typename T, int VEC>
__global__ void __launch_bounds__(QR_THREADS) cache_read_q8_kernel(const QrArgs a) {
  __shared__ Q8Slot s_slot[QR_ROWS];                   // at -1: a slot without a place; -2: a row that is left as it is
  const int tid = threadIdx.x;
  const int64_t row0 = int64_t(blockIdx.x) * QR_ROWS;
  ds_pdl_trigger();
  ds_pdl_wait();
  if (tid < QR_ROWS) {
    Q8Slot at{-2, -2};
    if (row0 + tid < a.rows) {
      const int64_t r = (row0 + tid) / a.S, i = row0 + tid - r * a.S;
      int32_t n = a.n[r];
      const int32_t s0 = a.start ? a.start[r] : 0;
      if (n < 0 || n > a.S || s0 < 0) {
        ds_set_error(a.status, DSPARK_EINVAL);
        n = 0;
      }
      if (i < n) {
        at = q8_slot(a.c, r, int64_t(s0) + i);
        if (at.at < 0) ds_set_error(a.status, DSPARK_ERANGE);
      }
    }
    s_slot[tid] = at;
  }
  __syncthreads();
  const int D = a.c.head_dim, per = D / VEC, items = 2 * a.c.heads * per;
  const bool e4m3 = a.c.code == DSPARK_E4M3;
  int m = tid / items, x = tid - m * items;            // slot of the block, item of the slot
  while (m < QR_ROWS) {
    constexpr int AT = 2;                              // items whose codes are on their way together
    uint4 w[AT];
    float f[AT];
    T* to[AT];
#pragma unroll
    for (int c = 0; c < AT; ++c) {
      to[c] = nullptr;
      w[c] = make_uint4(0u, 0u, 0u, 0u);
      f[c] = 0.0f;
      if (m >= QR_ROWS) continue;
      const Q8Slot at = s_slot[m];
      const int hv = x / per, d = (x - hv * per) * VEC;
      const bool value = hv >= a.c.heads;
      const int hd = value ? hv - a.c.heads : hv;
      if (at.at != -2) to[c] = reinterpret_cast<T*>(value ? a.v : a.k) + (row0 + m) * a.ld + int64_t(hd) * D + d;
      if (at.at >= 0) {
        const uint8_t* src = reinterpret_cast<const uint8_t*>(value ? a.c.v : a.c.k) + at.at + int64_t(hd) * a.c.head_stride + d;
        f[c] = q8_power((value ? a.c.v_scale : a.c.k_scale)[at.scale + int64_t(hd) * a.c.scale_head_stride + d / Q8_BLOCK]);
        if constexpr (VEC == 16) {
          w[c] = __ldcs(reinterpret_cast<const uint4*>(src));
        } else if constexpr (VEC == 8) {
          const uint2 y = __ldcs(reinterpret_cast<const uint2*>(src));
          w[c].x = y.x;
          w[c].y = y.y;
        } else {
          w[c].x = *src;
        }
      }
      for (x += QR_THREADS; x >= items && m < QR_ROWS; x -= items) ++m;
    }
#pragma unroll
    for (int c = 0; c < AT; ++c) {
      if (to[c] == nullptr) continue;
      if constexpr (VEC == 1) {
        const float y[1] = {q8_number(w[c].x, e4m3) * f[c]};
        qa_store<T, 1>(to[c], y);
      } else {
#pragma unroll
        for (int u = 0; u < VEC / 8; ++u) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            const uint32_t w4 = u ? (e ? w[c].w : w[c].z) : (e ? w[c].y : w[c].x);
            const float4 z = e4m3 ? qr_e4m3(w4) : make_float4(float(int8_t(w4)), float(int8_t(w4 >> 8)), float(int8_t(w4 >> 16)), float(int8_t(w4 >> 24)));
            y[e] = z.x * f[c];
            y[e + 1] = z.y * f[c];
            y[e + 2] = z.z * f[c];
            y[e + 3] = z.w * f[c];
          }
          qa_store<T, 8>(to[c] + 8 * u, y);
        }
      }
    }
  }
}

}  // namespace

extern "C" dspark_status dspark_rope_append_q8(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                                               dspark_dtype dtype, int64_t R, int32_t T, int32_t Hq, const int32_t* pos, int32_t A,
                                               const float* cos_sin, int64_t P, int32_t rot, const int32_t* axis,
                                               int32_t interleaved, const dspark_qcache* cache, const int32_t* ctx_len,
                                               const int32_t* n_nodes, void* q_out, int64_t ldo, int32_t* dev_status,
                                               dspark_stream_t stream) {
  DS_REQUIRE(ds_dtype_ok(dtype) && q8_cache_ok(cache, false) && R >= 0 && T >= 1 && Hq >= 1 && Hq <= 1024 && Hq % cache->heads == 0);
  const int64_t D = cache->head_dim;
  DS_REQUIRE(rot >= 2 && rot <= D && rot % 2 == 0 && A >= 1 && A <= 8 && P >= 1);
  DS_REQUIRE(ldq >= Hq * D && ldo >= Hq * D && ldk >= cache->heads * D && ldv >= cache->heads * D);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(R <= INT32_MAX / T);
  const size_t e = size_t(ds_dtype_size(dtype));
  DS_REQUIRE(q && k && v && pos && cos_sin && ctx_len && q_out && dev_status);
  DS_REQUIRE(ds_aligned(q, e) && ds_aligned(k, e) && ds_aligned(v, e) && ds_aligned(q_out, e) && (q_out != q || ldo == ldq));
  QaArgs a{q, k, v, q_out, ldq, ldk, ldv, ldo, R * T, T, Hq, A, rot, interleaved != 0, pos, axis, ctx_len, n_nodes, cos_sin, P, *cache, dev_status};
  a.c.layer_stride = a.c.scale_layer_stride = 0;
  DS_CUDA_TRY(dtype == DSPARK_BF16 ? qa_dispatch<__nv_bfloat16>(a, stream) : qa_dispatch<float>(a, stream));
  return DSPARK_OK;
}

extern "C" dspark_status dspark_cache_commit_q8(const dspark_qcache* cache, const int32_t* ctx_len, const int32_t* path,
                                                const int32_t* n_accepted, int64_t R, int32_t T, int32_t* new_len,
                                                int32_t* dev_status, dspark_stream_t stream) {
  DS_REQUIRE(q8_cache_ok(cache, true) && cache->n_layers <= (1 << 20) && R >= 0 && R <= 65535 && T >= 1 && T <= QC_MAXT);
  if (R == 0) return DSPARK_OK;
  DS_REQUIRE(ctx_len && n_accepted && new_len && dev_status && ds_commit_len_ok(new_len, ctx_len, n_accepted, path, R, T));
  const dim3 grid(path ? 2 * unsigned(cache->n_layers) : 1u, unsigned(R));
  const bool v16 = cache->head_dim % 16 == 0 && q8_codes_aligned(cache, 16), v8 = q8_codes_aligned(cache, 8);
  const bool s4 = q8_blocks(cache->head_dim) % 4 == 0 && q8_scales_aligned(cache, 4);
  auto go = [&](auto kern) { return ds_launch(kern, grid, dim3(QC_THREADS), 0, stream, *cache, ctx_len, path, n_accepted, T, new_len, dev_status); };
  if (v16) DS_CUDA_TRY(s4 ? go(cache_commit_q8_kernel<16, 4>) : go(cache_commit_q8_kernel<16, 1>));
  else if (v8) DS_CUDA_TRY(s4 ? go(cache_commit_q8_kernel<8, 4>) : go(cache_commit_q8_kernel<8, 1>));
  else DS_CUDA_TRY(s4 ? go(cache_commit_q8_kernel<1, 4>) : go(cache_commit_q8_kernel<1, 1>));
  return DSPARK_OK;
}

extern "C" dspark_status dspark_cache_read_q8(const dspark_qcache* cache, const int32_t* start, const int32_t* n, int64_t R, int32_t S,
                                              dspark_dtype dtype, void* k_out, void* v_out, int64_t ld, int32_t* dev_status,
                                              dspark_stream_t stream) {
  DS_REQUIRE(q8_cache_ok(cache, false) && ds_dtype_ok(dtype) && R >= 0 && S >= 1 && ld >= int64_t(cache->heads) * cache->head_dim);
  if (R == 0) return DSPARK_OK;
  const size_t e = size_t(ds_dtype_size(dtype));
  DS_REQUIRE(R <= INT32_MAX / S && n && k_out && v_out && k_out != v_out && dev_status && ds_aligned(k_out, e) && ds_aligned(v_out, e));
  QrArgs a{*cache, start, n, R * S, ld, S, k_out, v_out, dev_status};
  a.c.layer_stride = a.c.scale_layer_stride = 0;
  const bool vec = q8_codes_aligned(&a.c, 8) && ds_aligned(k_out, 16) && ds_aligned(v_out, 16) && (ld * int64_t(e)) % 16 == 0;
  const dim3 grid(unsigned(ds_ceil_div(a.rows, QR_ROWS)));
  // Codes a load: 16 for bf16 rows (136,000 slots 141 us; 8 at a time 208 us), 8 for float32 rows (272 us; 16 at a time, whose stores lie 64 bytes
  // apart, 292 us), one where rows are not aligned for that.
  const bool v16 = vec && dtype == DSPARK_BF16 && cache->head_dim % 16 == 0 && q8_codes_aligned(&a.c, 16);
  auto go = [&](auto kern) { return ds_launch(kern, grid, dim3(QR_THREADS), 0, stream, a); };
  if (dtype == DSPARK_BF16) {
    DS_CUDA_TRY((v16 ? go(cache_read_q8_kernel<__nv_bfloat16, 16>) : vec ? go(cache_read_q8_kernel<__nv_bfloat16, 8>) : go(cache_read_q8_kernel<__nv_bfloat16, 1>)));
  } else {
    DS_CUDA_TRY(vec ? go(cache_read_q8_kernel<float, 8>) : go(cache_read_q8_kernel<float, 1>));
  }
  return DSPARK_OK;
}
