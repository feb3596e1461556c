// tree_attn_q8.cu - attention of drafted nodes, or of one new token, over a paged key/value cache in 8 bits
// (dspark_tree_attention_q8): the entry point.
//
// openvino.genai PR #4847, Fixes > Split validation windows, and optimum-intel PR #2098 (paged attention targets): the target's
// pass over the drafted candidates of several requests at once.
#include "cache_q8.cuh"
#include "tree_attn.cuh"

namespace {

// Tensor map of one buffer of codes: (column, place, head, page), boxes of `cols` columns x `box` places.
bool tq_tensor_map(CUtensorMap* m, void* base, const dspark_qcache& c, int cols, int box) {
  const DsEncodeFn fn = ds_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {cuuint64_t(c.head_dim), cuuint64_t(c.page_size), cuuint64_t(c.heads), cuuint64_t(c.num_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(c.token_stride), cuuint64_t(c.head_stride), cuuint64_t(c.page_stride)};
  const cuuint32_t bx[4] = {cuuint32_t(cols), cuuint32_t(box), 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            cols == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The partial results of dspark_tree_attention, and of each warp of the kernel for few rows one more of at most 32 rows of 128 columns.
extern "C" size_t dspark_internal_ws_tree_attention_q8(int64_t R, int32_t T, int64_t cols, int32_t heads) {
  const size_t base = dspark_internal_ws_tree_attention(R, T, cols, heads);
  if (!base) return 0;
  const int64_t warps = 12 * int64_t(ds_num_sms()) * std::min<int64_t>(int64_t(T) * (cols / heads), 32 * 128);
  return base + size_t(ds_ceil_div(warps * 4, 256) * 256);
}

extern "C" dspark_status dspark_tree_attention_q8(const void* q, int64_t ldq, dspark_dtype dtype, int64_t R, int32_t T, int32_t Hq,
                                                  const dspark_qcache* cache, const int32_t* ctx_len, const int32_t* n_nodes,
                                                  const uint32_t* mask, float scale, float softcap, void* out, int64_t ldo,
                                                  float* lse, void* ws, size_t ws_bytes, int32_t* dev_status,
                                                  dspark_stream_t stream) {
  DS_REQUIRE(ds_dtype_ok(dtype) && q8_cache_ok(cache, false) && R >= 0 && R <= TA_MAXR && T >= 1 && T <= TA_MAXT);
  DS_REQUIRE(Hq >= 1 && Hq <= 1024 && Hq % cache->heads == 0);
  const int64_t D = cache->head_dim;
  DS_REQUIRE(ldq >= Hq * D && ldo >= Hq * D && scale > 0.0f && scale < INFINITY && softcap >= 0.0f && softcap < INFINITY);
  if (R == 0) return DSPARK_OK;
  const size_t e = size_t(ds_dtype_size(dtype));
  DS_REQUIRE(q && ctx_len && out && dev_status && ds_aligned(q, e) && ds_aligned(out, e));
  if (!ws || !ds_aligned(ws, 256) || ws_bytes < dspark_internal_ws_tree_attention_q8(R, T, Hq * D, cache->heads))
    return DSPARK_EWORKSPACE;
  TaArgs a{};
  a.q = q; a.ldq = ldq; a.out = out; a.ldo = ldo; a.lse = lse; a.ctx_len = ctx_len; a.n_nodes = n_nodes; a.mask = mask;
  a.R = int32_t(R); a.T = T; a.Hq = Hq; a.G = Hq / cache->heads; a.W = (T + 31) / 32;
  a.c.k = cache->k; a.c.v = cache->v; a.c.dtype = dtype; a.c.n_layers = 1;
  a.c.page_stride = cache->page_stride; a.c.token_stride = cache->token_stride; a.c.head_stride = cache->head_stride;
  a.c.num_pages = cache->num_pages; a.c.page_size = cache->page_size; a.c.heads = cache->heads; a.c.head_dim = cache->head_dim;
  a.c.page_table = cache->page_table; a.c.ld_table = cache->ld_table; a.c.table_pages = cache->table_pages;
  dspark_qcache one = *cache;
  one.layer_stride = one.scale_layer_stride = 0;
  a.q8 = TaQ8{cache->k_scale, cache->v_scale, cache->scale_page_stride, cache->scale_token_stride, cache->scale_head_stride,
              cache->code == DSPARK_E4M3, q8_codes_aligned(&one, 8), q8_scales_aligned(&one, 4)};
  ta_tanh_coefficients(a, scale, softcap);
  a.rows = T * a.G; a.scale = scale; a.softcap = softcap; a.status = dev_status; a.first_wait = g_ds_first_wait_polls.load();
  // the running tile count of all requests is 32 bits wide (lengths are cut to what the table holds)
  const auto counts = [&](int kt) {
    return R * ds_ceil_div(std::min<int64_t>(int64_t(cache->table_pages) * cache->page_size, int64_t(INT32_MAX)) + TA_MAXT, kt) <= INT32_MAX;
  };
  DS_REQUIRE(counts(64));
  // Few rows a key head: the kernel that widens codes in operand registers; more: the one that stages them for tcgen05, which takes the same
  // time whatever the rows up to 128. 300-8,200 keys: 64 requests with 4 rows 126 and 383 us; 32 requests with 16 rows 105 and 195 us, with 32 rows 187 and
  // 185 us, but 197 and more than 270 us where scales lie by place and not by head.
  const bool few = a.rows <= 32;
  int box = few ? 16 : 128;
  while (cache->page_size % box) box >>= 1;
  // Tensor cores: rows of codes that TMA can copy and bf16 rows that 16-byte accesses can.
  const bool tc = dtype == DSPARK_BF16 && D <= 128 && D % 16 == 0 && box >= 8 && q8_codes_aligned(&one, 16) && ds_aligned(q, 16) &&
                  ds_aligned(out, 16) && ldq % 8 == 0 && ldo % 8 == 0 && cache->page_stride > 0 && cache->token_stride > 0 &&
                  cache->head_stride > 0 && counts(16) && cache->scale_page_stride <= INT32_MAX && cache->scale_token_stride <= INT32_MAX;
  CUtensorMap mk, mv;
  const int cols = D <= 64 ? 64 : 128;
  const bool maps = tc && tq_tensor_map(&mk, cache->k, *cache, cols, box) && tq_tensor_map(&mv, cache->v, *cache, cols, box);
  a.box = box;
  const int nb = q8_blocks(int(D));
  // Scale bytes of a tile by bulk copies where a box's lie side by side: 4 capped trees of 64 nodes 358 us, by plain loads 477 us (before the widening's last change).
  a.q8.bulk = cache->scale_token_stride == nb && (box * nb) % 16 == 0 && q8_scales_box(&one, box * nb);
  if (maps && few) {
    a.kt = 16;
    a.rpg = a.rows <= 8 ? 8 : a.rows <= 16 ? 16 : 32;
  } else if (maps) {
    a.kt = 128;
    a.rpg = a.rows > 128 ? 256 : 128;
  } else {
    a.kt = 64;
    const int64_t groups = ds_ceil_div(a.rows, 64);  // groups of 64 rows or fewer, as even as sixteens allow
    a.rpg = int32_t(ds_ceil_div(a.rows, groups * 16) * 16);
  }
  a.mg = int32_t(ds_ceil_div(a.rows, a.rpg));
  a.rs = std::min(a.rows, a.rpg);
  const int64_t jobs = R * cache->heads * int64_t(a.mg) * a.rs;         // rows of all items
  DS_REQUIRE(jobs <= INT32_MAX);
  const int grid = ds_num_sms() * (maps || D > 128 ? 1 : 2);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  a.pref = reinterpret_cast<int32_t*>(w);
  a.part_o = reinterpret_cast<float*>(w + TA_WS_PREF);
  a.part_ml = reinterpret_cast<float4*>(a.part_o + 2 * int64_t(grid) * a.rs * D);
  a.warp_o = reinterpret_cast<float*>(w + dspark_internal_ws_tree_attention(R, T, Hq * D, cache->heads));
  DS_CUDA_TRY(!maps ? ta_launch_float_q8(a, grid, stream) : few ? ta_launch_q8_rows(a, grid, mk, mv, stream) : ta_launch_q8_tc(a, grid, mk, mv, stream));
  DS_CUDA_TRY(ta_launch_join(a, dtype, grid, jobs, stream));
  return DSPARK_OK;
}
