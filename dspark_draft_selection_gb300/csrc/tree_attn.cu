// tree_attn.cu - attention of drafted nodes over a paged key/value cache (dspark_tree_attention): the bf16 tensor-core
// kernel (tree_attn_tc.cuh), the join of partial results and the entry point.
//
// openvino.genai PR #4847, Fixes > Split validation windows, and optimum-intel PR #2098 (paged
// attention targets): the target's pass over the drafted candidates of several requests at once.
#include <cmath>

#include "tree_attn_tc.cuh"

namespace {

// Joins the partial results of one row, one warp: 32 parts at a time, a lane takes a part's maximum and sum,
// then the lanes take the columns and add the parts in the order of the blocks that left them, every load of a
// part being independent of the others (U = 128-column pieces of a row). Rows whose item was finished by one block are left at once.
template <typename T, int U>
__global__ void __launch_bounds__(256) tree_attn_join_kernel(const TaArgs a, uint32_t grid, int64_t jobs) {
  ds_pdl_trigger();
  const int64_t job = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t item = ta_div(job, uint32_t(a.rs));
  const int lrow = int(job - item * a.rs);
  const int hm = a.c.heads * a.mg;
  const int r = int(ta_div(item, uint32_t(hm))), sub = int(item - int64_t(r) * hm);
  const int hk = sub / a.mg, g = sub - hk * a.mg, m = g * a.rpg + lrow;
  const int i = m / a.G, h = hk * a.G + m - i * a.G, D = a.c.head_dim;
  const int64_t row = int64_t(r) * a.T + i;
  ds_pdl_wait();
  if (job >= jobs || m >= a.rows) return;
  const int64_t total = int64_t(__ldcg(a.pref + a.R)) * hm, p0 = __ldcg(a.pref + r), nt = __ldcg(a.pref + r + 1) - p0;
  const int64_t g0 = p0 * hm + sub * nt;
  auto start = [&](int64_t b) { return ta_div(total * b, grid); };      // first tile of block b
  auto holder = [&](int64_t tile) {                    // block whose share holds the tile
    const int64_t x = (tile + 1) * grid + total - 1;
    return int((total >> 32 ? ta_div64(x, total) : ta_div(x, uint32_t(total))) - 1);
  };
  const int b0 = holder(g0);
  if (start(b0 + 1) >= g0 + nt) return;                // whole
  const int np = holder(g0 + nt - 1) - b0 + 1;
  float M = -INFINITY, L = 0.0f, Ld = 0.0f;            // Ld: the sum that the result is divided by
  float4 o[U];
#pragma unroll
  for (int u = 0; u < U; ++u) o[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int k0 = 0; k0 < np; k0 += 32) {
    // part k: what block b0 + k left, if its share is not empty
    const int64_t s0 = start(b0 + k0 + lane), s1 = start(b0 + k0 + lane + 1);
    const bool there = k0 + lane < np && s1 > s0;
    const int32_t slot = 2 * (b0 + k0 + lane) + (s0 > g0 ? 0 : 1);
    const float4 ml = there ? __ldcg(a.part_ml + int64_t(slot) * a.rs + lrow) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    const float before = M;
    M = fmaxf(M, ds_warp_max(ml.x));
    const bool seen = ml.y != 0.0f;                    // also a sum that is not a number
    const float w = seen ? ta_ex2(ml.x - M) : 0.0f, f = before == -INFINITY ? 0.0f : ta_ex2(before - M);
    L = __fmaf_rn(w, ml.y, L * f);
    Ld = __fmaf_rn(w, ml.z, Ld * f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      o[u].x *= f;
      o[u].y *= f;
      o[u].z *= f;
      o[u].w *= f;
    }
    const unsigned live = __ballot_sync(0xFFFFFFFFu, seen);
    const int cnt = min(32, np - k0);
    for (int e0 = 0; e0 < cnt; e0 += 8) {
      float4 y[U][8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t se = __shfl_sync(0xFFFFFFFFu, slot, e0 + e);
        const float* x = a.part_o + (se * a.rs + lrow) * D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int d = lane * 4 + 128 * u;
          y[u][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if ((live >> (e0 + e)) & 1u && d < D) y[u][e] = __ldcg(reinterpret_cast<const float4*>(x + d));
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float we = __shfl_sync(0xFFFFFFFFu, w, e0 + e);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          o[u].x = __fmaf_rn(we, y[u][e].x, o[u].x);
          o[u].y = __fmaf_rn(we, y[u][e].y, o[u].y);
          o[u].z = __fmaf_rn(we, y[u][e].z, o[u].z);
          o[u].w = __fmaf_rn(we, y[u][e].w, o[u].w);
        }
      }
    }
  }
  L = ds_warp_sumf(L);
  Ld = ds_warp_sumf(Ld);
  const bool any = L != 0.0f;
  const float inv = any ? 1.0f / Ld : 0.0f;
  T* out = reinterpret_cast<T*>(a.out) + row * a.ldo + int64_t(h) * D;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int d = lane * 4 + 128 * u;
    if (d >= D) continue;
    const float y[4] = {any ? o[u].x * inv : 0.0f, any ? o[u].y * inv : 0.0f, any ? o[u].z * inv : 0.0f, any ? o[u].w * inv : 0.0f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(T) == 2) out[d + e] = __float2bfloat16_rn(y[e]);
      else out[d + e] = y[e];
    }
  }
  if (lane == 0 && a.lse) a.lse[row * a.Hq + h] = any ? (M + log2f(L)) * TA_LN2 : -INFINITY;
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

}  // namespace

void ta_tanh_coefficients(TaArgs& a, float scale, float cap) {
  static const double p[7] = {0x1.fffffep-1, -0x1.55540ap-2, 0x1.10e672p-3, -0x1.b5eb8p-5, 0x1.4c6e4ap-6, -0x1.968b3ap-8, 0x1.10e592p-10};
  static const double q[4] = {0x1.fffffep-1, -0x1.5551c6p-2, 0x1.10110cp-3, -0x1.8b7242p-5};
  if (!(cap > 0.0f)) return;
  const double sy = double(scale) / cap;
  // How far a form serves. A coefficient that is no normal float32 number is 0: one too small belongs to a large cap, and
  // below the limit its term is less than 2^-24 of the sum; one too large belongs to a tiny cap, which the exponential
  // form serves whatever the score.
  const auto scaled = [&](const double* co, int n, float most, auto put) {
    double f = sy * cap * 1.4426950408889634;
    double limit = most;
    for (int k = 0; k < n; ++k, f *= sy * sy) {
      const double x = std::fabs(co[k] * f);
      if (!(x <= 0x1p127)) limit = -1.0;
      else if (x < 0x1p-126) limit = std::min(limit, k ? std::pow(0x1p-24 / std::fabs(co[k]), 0.5 / k) : -1.0);
      put(k, x >= 0x1p-126 && x <= 0x1p127 ? float(co[k] * f) : 0.0f);
    }
    return float(limit);
  };
  a.wide_to = scaled(p, 7, 1.0f, [&](int k, float x) { a.wide[k] = x; });
  a.narrow_to = scaled(q, 4, 0.375f, [&](int k, float x) { a.narrow[k] = make_float2(x, x); });
}

cudaError_t ta_launch_join(const TaArgs& a, dspark_dtype dtype, int grid, int64_t jobs, cudaStream_t st) {
  const dim3 jg{unsigned(ds_ceil_div(jobs, 8))}, jb{256};
  auto go = [&](auto kern) { return ds_launch(kern, jg, jb, 0, st, a, uint32_t(grid), jobs); };
  if (dtype == DSPARK_BF16) return a.c.head_dim <= 128 ? go(tree_attn_join_kernel<__nv_bfloat16, 1>) : go(tree_attn_join_kernel<__nv_bfloat16, 2>);
  return a.c.head_dim <= 128 ? go(tree_attn_join_kernel<float, 1>) : go(tree_attn_join_kernel<float, 2>);
}

// Partial results of 2 slots per block: rs rows x (head_dim sums + reference and sums). rs * head_dim is at
// most the group's T * cols / heads, and at most 256 rows of 256 columns (one block per SM) or 64 rows of
// 256 (the float32 kernel's two blocks); head_dim >= 8, so a row's statistics (16 bytes) add at most a half.
extern "C" size_t dspark_internal_ws_tree_attention(int64_t R, int32_t T, int64_t cols, int32_t heads) {
  if (R <= 0 || T <= 0 || cols <= 0 || heads <= 0) return 0;
  const int64_t item = int64_t(T) * (cols / heads), sms = ds_num_sms();
  const int64_t vals = std::max(2 * sms * std::min<int64_t>(item, 256 * 256), 4 * sms * std::min<int64_t>(item, 64 * 256));
  return TA_WS_PREF + size_t(ds_ceil_div(vals * 6, 256) * 256);
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
  ta_tanh_coefficients(a, scale, softcap);
  a.rows = T * a.G; a.scale = scale; a.softcap = softcap; a.status = dev_status; a.first_wait = g_ds_first_wait_polls.load();
  int box = 128;
  while (cache->page_size % box) box >>= 1;
  // (32 requests of 8 nodes, 300-8,200 keys: 113 us, in float32 arithmetic 681 us; with 256 columns, which only that
  // takes, 2,404 us.)
  // Tensor cores: rows of bf16 that TMA can copy (16-byte rows; eight places of a page are the smallest box
  // whose swizzle starts on its own pattern) and outputs that 16-byte stores can write.
  const bool tc = cache->dtype == DSPARK_BF16 && D <= 128 && box >= 8 && ds_cache_vec(cache) && ds_aligned(q, 16) &&
                  ds_aligned(out, 16) && ldq % 8 == 0 && ldo % 8 == 0 && cache->page_stride > 0 && cache->token_stride > 0 &&
                  cache->head_stride > 0;
  CUtensorMap mk, mv;
  const bool maps = tc && ta_tensor_map(&mk, cache->k, *cache, box) && ta_tensor_map(&mv, cache->v, *cache, box);
  a.kt = maps ? TA_KT : 64;
  // the running tile count of all requests is 32 bits wide (lengths are cut to what the table holds)
  DS_REQUIRE(R * ds_ceil_div(std::min<int64_t>(int64_t(cache->table_pages) * cache->page_size, int64_t(INT32_MAX)) + TA_MAXT, a.kt) <= INT32_MAX);
  a.box = box;
  if (maps) {
    // Two row tiles a block where there are more than 128 rows, so that a key tile is read once for both: 160,
    // 256 and 512 rows (4 requests, 40,000-65,600 keys) 101, 118 and 198 us, with one row tile a block 128, 131
    // and 248 us.
    a.rpg = a.rows > 128 ? 256 : 128;
  } else {                                             // groups of 64 rows or fewer, as even as sixteens allow
    const int64_t groups = ds_ceil_div(a.rows, 64);
    a.rpg = int32_t(ds_ceil_div(a.rows, groups * 16) * 16);
  }
  a.mg = int32_t(ds_ceil_div(a.rows, a.rpg));
  a.rs = std::min(a.rows, a.rpg);
  const int64_t jobs = R * cache->heads * int64_t(a.mg) * a.rs;         // rows of all items
  DS_REQUIRE(jobs <= INT32_MAX);
  const int grid = ds_num_sms() * (maps || D > 128 ? 1 : 2);
  const int64_t slots = 2 * int64_t(grid);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  a.pref = reinterpret_cast<int32_t*>(w);
  a.part_o = reinterpret_cast<float*>(w + TA_WS_PREF);
  a.part_ml = reinterpret_cast<float4*>(a.part_o + slots * a.rs * D);
  // 64 columns have their own form: 64 rows 54.6 us, 512 rows 167 us, padded to 128 columns 60.5 and 183 us.
  if (maps) DS_CUDA_TRY((D <= 64 ? ta_dispatch_tc<64, false>(a, grid, mk, mv, stream) : ta_dispatch_tc<128, false>(a, grid, mk, mv, stream)));
  else DS_CUDA_TRY(ta_launch_float(a, grid, stream));
  DS_CUDA_TRY(ta_launch_join(a, cache->dtype, grid, jobs, stream));
  return DSPARK_OK;
}
