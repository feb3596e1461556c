// tree_attn.cuh - what the kernels of dspark_tree_attention share: arguments, the split of the work
// over the blocks and the layout of the partial results.
#pragma once

#include "dspark_common.cuh"
#include "host_common.h"

constexpr int TA_MAXR = 1024;
constexpr int TA_MAXT = 512;

// A cache in 8 bits: what TaArgs::c, whose strides are then bytes and whose dtype is the queries', does not say.
struct TaQ8 {
  const uint8_t *k_scale, *v_scale;
  int64_t page_stride, token_stride, head_stride;   // of the scales
  int32_t e4m3, vec8, vec4;    // rows of codes start on 8-byte boundaries, of scales on 4-byte ones
  int32_t bulk;                // the scale bytes of a box of slots are one run that a bulk copy takes
};

struct TaArgs {
  const void* q;
  int64_t ldq;
  void* out;
  int64_t ldo;
  float* lse;
  dspark_kvcache c;
  const int32_t *ctx_len, *n_nodes;
  const uint32_t* mask;
  int32_t R, T, Hq, G, W;      // G query heads per key head, W mask words per node
  int32_t rows;                // T * G query rows per (request, key head); row m is node m / G, head m % G
  int32_t rpg, mg;             // rows per row group, row groups
  int32_t rs;                  // row stride of a partial result, >= the rows of a group that exist
  int32_t kt;                  // keys per tile
  int32_t box;                 // keys per copy (tensor-core kernel)
  float scale, softcap;
  float wide[7];               // coefficients of the cap's polynomials,
  float2 narrow[4];            // the short one's each twice
  float wide_to, narrow_to;    // and up to which |score| / cap they serve
  int32_t* pref;               // [R + 1] running sum of the requests' tile counts
  float4* part_ml;             // [slots][rs] (reference in log2 units, sum of the weights, sum the result is divided by)
  float* part_o;               // [slots][rs][D] sums of weights times values, relative to the maximum
  float* warp_o;               // [blocks][warps][rs][D] the same of single warps (tree_attn_q8_rows.cu)
  int32_t* status;
  uint32_t first_wait;
  TaQ8 q8;
};

// The work is a line of tiles: requests in order, in each its (key head, row group) items in order,
// in each item its key tiles in order (at least one, so that empty requests get their zeros written).
// Block b of `grid` takes tiles [total b / grid, total (b + 1) / grid): every block has the same
// number of tiles (+-1) whatever the lengths, which only the device knows. An item that a block holds
// whole is finished there; of the others each block leaves a partial result - slot 2 b for one that an
// earlier block began, 2 b + 1 for one that it began itself - and the combine kernel joins them in
// the order of the blocks.
struct TaPiece {
  int32_t r, hk, g;            // request, key head, row group
  int32_t t0, t1, nt;          // tiles [t0, t1) of the item's nt
  DS_DEV bool whole() const { return t0 == 0 && t1 == nt; }
  DS_DEV int64_t slot(int64_t b) const { return 2 * b + (t0 > 0 ? 0 : 1); }
};

// The requests' running tile counts, committed lengths and node counts, and where the block's share
// begins, in shared memory.
struct TaLens {
  int32_t pref[TA_MAXR + 1], ctx[TA_MAXR], n[TA_MAXR];
  int64_t at, end;
  int32_t r;
  TaPiece first;               // the share's first piece, which next() would find
  int32_t any;                 // whether there is one
};

// Quotient of a number that rarely needs more than 32 bits (the long division stays out of line).
static __device__ __noinline__ int64_t ta_div64(int64_t x, int64_t d) { return x / d; }
DS_DEV int64_t ta_div(int64_t x, uint32_t d) {
  return (x >> 32) == 0 ? int64_t(uint32_t(x) / d) : ta_div64(x, d);
}

struct TaWalk {
  int64_t at, end;
  int32_t r;
  bool begun;
  DS_DEV void init(const TaLens& s) {
    at = s.at;
    end = s.end;
    r = s.r;
    begun = false;
  }
  // The next piece of the share; the first one was found once for all warps.
  DS_DEV bool next(const TaLens& s, const TaArgs& a, TaPiece& p) {
    if (begun) return find(s, a, p);
    begun = true;
    p = s.first;
    at += p.t1 - p.t0;
    return s.any != 0;
  }
  DS_DEV bool find(const TaLens& s, const TaArgs& a, TaPiece& p) {
    if (at >= end) return false;
    const int64_t hm = int64_t(a.c.heads) * a.mg;
    while (s.pref[r + 1] * hm <= at) ++r;
    const int64_t off = at - s.pref[r] * hm;
    p.r = r;
    p.nt = s.pref[r + 1] - s.pref[r];
    const int32_t item = int32_t(ta_div(off, uint32_t(p.nt)));
    p.t0 = int32_t(off - int64_t(item) * p.nt);
    p.t1 = int32_t(min(int64_t(p.nt), p.t0 + (end - at)));
    p.hk = int32_t(uint32_t(item) / uint32_t(a.mg));
    p.g = item - p.hk * a.mg;
    at += p.t1 - p.t0;
    return true;
  }
};

// Lengths and running tile counts by all threads of the block. A length or node count out of range is
// reported and cut so that no slot past the page table is read. Block 0 leaves the counts for the
// join.
DS_DEV void ta_prefix(const TaArgs& a, TaLens& s) {
  const int tid = threadIdx.x;
  const int64_t cap = int64_t(a.c.table_pages) * a.c.page_size;
  auto take = [&](int r) -> int32_t {                  // request r's lengths; its tile count
    int32_t ctx = a.ctx_len[r], n = a.n_nodes ? a.n_nodes[r] : a.T;
    if (n < 0 || n > a.T || ctx < 0) {
      ds_set_error(a.status, DSPARK_EINVAL);
      n = 0;
      ctx = max(ctx, 0);
    }
    if (int64_t(ctx) + n > cap) {
      ds_set_error(a.status, DSPARK_ERANGE);
      ctx = int32_t(min(int64_t(ctx), cap));
      n = int32_t(min(int64_t(n), cap - ctx));
    }
    s.ctx[r] = ctx;
    s.n[r] = n;
    return max(1, int32_t(uint32_t(uint32_t(ctx) + uint32_t(n) + uint32_t(a.kt - 1)) / uint32_t(a.kt)));
  };
  const bool few = a.R <= 64;                          // one warp is enough, with one synchronisation less
  if (!few) {
    for (int r = tid; r < a.R; r += blockDim.x) s.pref[r + 1] = take(r);
    __syncthreads();
  }
  if (tid < 32) {
    int32_t run = 0;
    for (int r0 = 0; r0 < a.R; r0 += 32) {
      const int r = r0 + tid;
      int32_t v = r >= a.R ? 0 : few ? take(r) : s.pref[r + 1];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int32_t up = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (tid >= d) v += up;
      }
      v += run;
      if (r < a.R) s.pref[r + 1] = v;
      run = __shfl_sync(0xFFFFFFFFu, v, 31);
    }
    if (tid == 0) s.pref[0] = 0;
    __syncwarp();
    // the block's share and the last request that begins at or before it
    const int64_t hm = int64_t(a.c.heads) * a.mg, total = run * hm, at = ta_div(total * blockIdx.x, gridDim.x);
    int r = 0;
    for (int r0 = 0; r0 < a.R; r0 += 32) {
      const unsigned before = __ballot_sync(0xFFFFFFFFu, r0 + tid < a.R && s.pref[min(r0 + tid, a.R - 1)] * hm <= at);
      if (before) r = r0 + 31 - __clz(int(before));
      if (before != 0xFFFFFFFFu) break;
    }
    TaWalk w;
    w.at = at;
    w.end = ta_div(total * (blockIdx.x + 1), gridDim.x);
    w.r = r;
    TaPiece p = {};
    const bool any = w.find(s, a, p);
    if (tid == 0) {
      s.at = at;
      s.end = w.end;
      s.r = r;
      s.first = p;
      s.any = any;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int r = tid; r <= a.R; r += blockDim.x) a.pref[r] = s.pref[r];
}

// Bits of the 32 keys whose first is node `nd` (negative: committed slots, which every node sees),
// as node i of n sees them.
DS_DEV uint32_t ta_mask32(const TaArgs& a, int r, int i, int n, int64_t nd) {
  if (nd <= -32) return 0xFFFFFFFFu;
  const int lim = a.mask ? n : min(n, i + 1);        // without a mask node i sees nodes j <= i
  if (nd >= lim) return 0u;
  uint32_t bits = 0xFFFFFFFFu;
  if (a.mask) {
    const uint32_t* row = a.mask + (int64_t(r) * a.T + i) * a.W;
    if (nd < 0) {
      bits = (row[0] << uint32_t(-nd)) | ((1u << uint32_t(-nd)) - 1u);
    } else {
      const int w = int(nd >> 5);
      const uint32_t lo = row[w], hi = w + 1 < a.W ? row[w + 1] : 0u;
      bits = __funnelshift_r(lo, hi, uint32_t(nd) & 31u);
    }
  }
  const int64_t left = lim - nd;                     // keys of these 32 that exist
  return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

// Element offset of slot s of request r, or -1.
DS_DEV int64_t ta_slot(const TaArgs& a, int r, int64_t s) {
  const int64_t e = s / a.c.page_size;
  if (e >= a.c.table_pages) return -1;
  const int32_t p = a.c.page_table[int64_t(r) * a.c.ld_table + e];
  if (p < 0 || p >= a.c.num_pages) {
    ds_set_error(a.status, DSPARK_ERANGE);
    return -1;
  }
  return int64_t(p) * a.c.page_stride + (s - e * a.c.page_size) * a.c.token_stride;
}

// The same of a cache in 8 bits; `scale`: the slot's offset among the scales.
DS_DEV int64_t ta_slot_q8(const TaArgs& a, int r, int64_t s, int64_t& scale) {
  const int64_t e = s / a.c.page_size;
  if (e >= a.c.table_pages) return -1;
  const int32_t p = a.c.page_table[int64_t(r) * a.c.ld_table + e];
  if (p < 0 || p >= a.c.num_pages) {
    ds_set_error(a.status, DSPARK_ERANGE);
    return -1;
  }
  const int64_t t = s - e * a.c.page_size;
  scale = int64_t(p) * a.q8.page_stride + t * a.q8.token_stride;
  return int64_t(p) * a.c.page_stride + t * a.c.token_stride;
}

DS_DEV float ta_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// cap * tanh(x) with tanh(x) = 1 - 2 / (1 + e^(2 x)); `x2` is 2 x log2(e). Its error is about 2^-22 of
// the cap whatever x (a tanh instruction leaves about 2^-11).
DS_DEV float ta_tanh(float x2, float cap) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ta_ex2(x2)));
  return __fmaf_rn(-2.0f * cap, r, cap);
}

constexpr float TA_LOG2E = 1.4426950408889634f;
constexpr float TA_LN2 = 0.6931471805599453f;

// The kernels in float32 arithmetic (tree_attn_float.cu, tree_attn_q8_float.cu), the coefficients of the cap's polynomials and the
// join of the partial results (tree_attn.cu; `dtype` of the result).
cudaError_t ta_launch_float(const TaArgs& a, int grid, cudaStream_t st);
cudaError_t ta_launch_float_q8(const TaArgs& a, int grid, cudaStream_t st);
cudaError_t ta_launch_q8_rows(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st);   // tree_attn_q8_rows.cu
cudaError_t ta_launch_q8_tc(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st);     // tree_attn_q8_tc.cu
void ta_tanh_coefficients(TaArgs& a, float scale, float cap);
cudaError_t ta_launch_join(const TaArgs& a, dspark_dtype dtype, int grid, int64_t jobs, cudaStream_t st);
constexpr size_t TA_WS_PREF = 4352;        // pref[TA_MAXR + 1], rounded up to 256 bytes
extern "C" size_t dspark_internal_ws_tree_attention(int64_t R, int32_t T, int64_t cols, int32_t heads);
extern "C" size_t dspark_internal_ws_tree_attention_q8(int64_t R, int32_t T, int64_t cols, int32_t heads);
