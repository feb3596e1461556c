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
// even and the odd key tiles of the same rows, joined through tensor memory at the end. The reference m lies
// 8 (in log2) above the maximum that set it, and O is rescaled only when a score passes it: no weight is above
// 1, so no sum is larger than the largest value times the keys, whatever the scores and the cap. (Sums are
// relative to the same reference, so the result is the same softmax; float32 and bf16 hold weights down to 2^-126.)
//
// Roles: warps 0 and 2 copy key and value tiles with TMA, one box per page piece, into a ring of stages;
// warp 1 issues the MMAs; warp 3 copies the query rows; warps 4-7 and 8-11 are the softmax groups.
// Bound: HBM (2 D bytes of keys and of values per cached token and key head) up to about 128 query rows per
// key head, above that the chain P V, Q K^T, softmax of a group: S and P share their tensor memory (S, O of
// both groups take all 512 columns), so a group's next scores wait for its P V. Measured with the join:
//   32 requests of 8 nodes x 4 heads, 300-8,200 keys   113 us   5.1 TB/s, 0.75 of the measured copy rate
//   64 requests of one token x 4 heads, 300-8,200 keys 189 us   6.0 TB/s, 0.88
//   4 trees of 64 nodes x 8 heads, 40,000-65,600 keys  198 us   959 TFLOP/s; with a cap 250 us, 760 TFLOP/s
//   one token x 4 heads, 4,097 keys                     16 us   two tiles a block: latency
#include <cmath>

#include "tree_attn.cuh"

extern "C" size_t dspark_internal_ws_tree_attention(int64_t R, int32_t T, int64_t cols, int32_t heads);

namespace {

constexpr int TA_KT = 128;                 // keys per tile
constexpr int TA_THREADS = 384;
constexpr int TA_QTHREADS = 32;
constexpr uint32_t TA_CHUNK = 128 * 128;   // bytes of 128 rows x 64 bf16 columns
constexpr float TA_ABOVE = 8.0f;           // a new reference lies this far (log2) above the maximum

template <int DP, bool TWO>
__host__ __device__ constexpr int ta_stages() {
  return DP == 128 ? (TWO ? 4 : 5) : 8;
}
template <int DP, bool TWO>
__host__ __device__ constexpr size_t ta_smem() {
  return 1024 + size_t(DP / 64) * TA_CHUNK * ((TWO ? 2 : 1) + ta_stages<DP, TWO>());
}

// 4-D tiled TMA load (column, place in page, head, page), what lies outside the tensor reading as zero,
// by one elected lane of a warp that stays together.
DS_DEV void ta_tma_load(void* dst, const void* tmap, int32_t d, int32_t t, int32_t h, int32_t p, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];\n\t}" ::"r"(ds_smem_addr(dst)),
      "l"(tmap), "r"(d), "r"(t), "r"(h), "r"(p), "r"(ds_smem_addr(bar))
      : "memory");
}

// The MMA warp stays together, so that descriptors and addresses are uniform registers, and one elected
// lane - the same one every time - issues: D[tmem] (+)= A[smem] * B[smem], kind::f16. A descriptor's low word
// holds the address (in 16 bytes: all of shared memory fits its 14 bits, so offsets are plain additions) and
// the leading offset; its high word is a constant of the layout.
template <uint32_t HI>
DS_DEV void ta_umma_ss(uint32_t d_tmem, uint32_t alo, uint32_t blo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(HI)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem],
template <uint32_t HI>
DS_DEV void ta_umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(idesc), "r"(accumulate), "r"(HI)
      : "memory");
}
// and the arrival on an mbarrier once everything issued before is complete.
DS_DEV void ta_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(ds_smem_addr(bar))
      : "memory");
}

// 32 columns of tensor memory on their way into registers; ta_arrived waits for all that are.
DS_DEV void ta_tmem_fetch(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
DS_DEV void ta_arrived(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])::"memory");
}

DS_DEV void ta_tmem_fetch(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
DS_DEV void ta_arrived(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15])::"memory");
}

// cap2 * tanh(sy * s) = s * Q(s^2): tanh(y) = y P(y^2) with the coefficients of P that make the largest
// relative error smallest (fitted by reweighted least squares), scaled by the powers of sy and by cap2; two
// values at a time. Seven coefficients serve |y| <= 1 and four |y| <= 0.375 (wide_to, narrow_to: less where coefficients
// leave float32's range); as evaluated in float32 their errors are 1.6e-7 and 1.5e-7. The scaled coefficients are kernel arguments, made by ta_tanh_coefficients (the narrow
// ones a pair of each).
DS_DEV uint64_t ta_pair(float2 x) { return ds_f2(x.x, x.y); }
DS_DEV uint64_t ta_poly(const float (&co)[7], uint64_t s) {   // a row's own: the wide ones, or the narrow ones and zeros
  const uint64_t u = ds_fma2(s, s, 0);
  uint64_t q = ds_f2(co[6], co[6]);
#pragma unroll
  for (int k = 5; k >= 0; --k) q = ds_fma2(q, u, ds_f2(co[k], co[k]));
  return q;
}
DS_DEV uint64_t ta_poly_narrow(const TaArgs& a, uint64_t s) {
  const uint64_t u = ds_fma2(s, s, 0);
  uint64_t q = ta_pair(a.narrow[3]);
#pragma unroll
  for (int k = 2; k >= 0; --k) q = ds_fma2(q, u, ta_pair(a.narrow[k]));
  return q;
}

// High word of both layouts: groups of eight rows (K-major: query or key rows; N-major: keys) 1024 bytes
// apart, descriptor version 1, 128-byte swizzle. Low words: K-major needs no leading offset; an operand
// whose N index is contiguous (V: 64 columns of D to a 128-byte row) has its 64-column blocks TA_CHUNK apart.
constexpr uint32_t TA_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
DS_DEV uint32_t ta_desc_k(uint32_t saddr) { return (saddr >> 4) | (1u << 16); }
DS_DEV uint32_t ta_desc_n(uint32_t saddr) { return (saddr >> 4) | ((TA_CHUNK >> 4) << 16); }

DS_DEV void ta_tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
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

// Bit 15 and bit 31 are set where the two bf16 numbers of x are infinite or not a number.
DS_DEV uint32_t ta_odd(uint32_t x) { return ((x & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// A value tile with nodes or with the end of the keys, before P multiplies it: 0 times a value that is not finite is
// not 0, and neither need be 0 times what follows the last key in its page. Rows [k0, k1) of the tile, past the last
// key, become 0; rows [f, k0) are nodes, the first of them `node`, whose values that are not finite become 0 too and
// whose bits in `odd` are set before: ta_add_odd gives them to the rows that see such a node. One group's threads;
// two groups on one tile both do this, and each finds what was there or what the other left, which ends the same.
// (In line and before the softmax: as a call behind it 4 trees of 64 took 200 us against 197, capped 248 against 246,
// 32 capped blocks of eight 140 against 133, 64 short requests 60 against 58.)
template <int NC>
DS_DEV void ta_clean(uint8_t* st, int f, int k0, int k1, int node, uint32_t* odd, int thread) {
#pragma unroll 1
  for (int u = thread; u < (k1 - f) * NC * 8; u += 128) {
    const int key = u / (NC * 8), c = u % (NC * 8);
    uint4* at = reinterpret_cast<uint4*>(st + (c >> 3) * TA_CHUNK + (f + key) * 128 + ((c & 7) << 4));
    if (f + key >= k0) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 y = *at;
    if ((ta_odd(y.x) | ta_odd(y.y) | ta_odd(y.z) | ta_odd(y.w)) == 0u) continue;
    atomicOr(odd + ((node + key) >> 5), 1u << ((node + key) & 31));
    __threadfence_block();
    auto finite = [](uint32_t x) { return x & ~((ta_odd(x) >> 15) * 0xFFFFu); };
    *at = make_uint4(finite(y.x), finite(y.y), finite(y.z), finite(y.w));
  }
}

// What nodes whose values are not finite add to a row that sees them: a weight is more than 0, so its product with an
// infinity or with what is not a number is that value itself - unless the score is -inf, whose weight 0 makes it not a
// number. One thread a row; `out` (the result) or `part` (a partial one) holds the row without them, this thread having
// written columns [d0, d1); `q` is its query.
__device__ __noinline__ void ta_add_odd(const TaArgs& a, int r, int32_t ctx, int32_t n, int i, int hk, int d0, int d1,
                                        const uint32_t* odd, const __nv_bfloat16* q, __nv_bfloat16* out, float* part) {
  const __nv_bfloat16* kc = reinterpret_cast<const __nv_bfloat16*>(a.c.k) + hk * a.c.head_stride;
  const __nv_bfloat16* vc = reinterpret_cast<const __nv_bfloat16*>(a.c.v) + hk * a.c.head_stride;
  uint32_t none[TA_MAXT / 32] = {};                    // nodes of weight 0; no capped score is -inf
  for (int w = 0; w < a.W && a.softcap == 0.0f; ++w) {
    if (odd[w] == 0u) continue;
    for (uint32_t bits = odd[w] & ta_mask32(a, r, i, n, 32 * w); bits; bits &= bits - 1) {
      const int64_t at = ta_slot(a, r, int64_t(ctx) + 32 * w + __ffs(int(bits)) - 1);
      if (at < 0) continue;
      float s = 0.0f;
      for (int d = 0; d < a.c.head_dim; d += 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(q + d), y = *reinterpret_cast<const uint4*>(kc + at + d);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __fmaf_rn(ds_vec_elem<__nv_bfloat16>(x, e), ds_vec_elem<__nv_bfloat16>(y, e), s);
      }
      if (s == -INFINITY) none[w] |= bits & (0u - bits);
    }
  }
  for (int d = d0; d < d1; d += 32) {                  // 32 columns for one lookup of a node's slot
    float z[32] = {};
    for (int w = 0; w < a.W; ++w) {
      if (odd[w] == 0u) continue;
      for (uint32_t bits = odd[w] & ta_mask32(a, r, i, n, 32 * w); bits; bits &= bits - 1) {
        const int64_t at = ta_slot(a, r, int64_t(ctx) + 32 * w + __ffs(int(bits)) - 1);
        if (at < 0) continue;
        const float times = none[w] & bits & (0u - bits) ? 0.0f : 1.0f;
        uint32_t x[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 y = d + 8 * e < d1 ? *reinterpret_cast<const uint4*>(vc + at + d + 8 * e) : make_uint4(0, 0, 0, 0);
          x[4 * e] = y.x; x[4 * e + 1] = y.y; x[4 * e + 2] = y.z; x[4 * e + 3] = y.w;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t bad = ta_odd(x[e]);
          z[2 * e] += bad & 0x8000u ? __uint_as_float(x[e] << 16) * times : 0.0f;
          z[2 * e + 1] += bad & 0x80000000u ? __uint_as_float(x[e] & 0xFFFF0000u) * times : 0.0f;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      if (z[e] == 0.0f || d + e >= d1) continue;       // what is not a number is not 0
      if (out) out[d + e] = __float2bfloat16_rn(__bfloat162float(out[d + e]) + z[e]);
      else part[d + e] += z[e];
    }
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
  __shared__ uint32_t s_tmem, s_seq[NS];               // s_seq: sequence number + 1 of a stage's last copy
  __shared__ int s_abort;
  __shared__ TaLens s_len;
  __shared__ float4 s_ml[2][2][128];                   // [piece parity][group][row]
  __shared__ uint4 s_odd[3][TA_MAXT / 128];            // [piece modulo 3]: a bit for every node with a value that is not finite

  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  uint8_t* sQ = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sR = sQ + (TWO ? 2 : 1) * STAGE;            // the ring (a query tile has a stage's size)

  ds_pdl_trigger();
  if (tid == 64) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmK) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmV) : "memory");
  }
  if (tid < 3 * (TA_MAXT / 128)) s_odd[tid / (TA_MAXT / 128)][tid % (TA_MAXT / 128)] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      ds_mbar_init(&s_full[s], 1);
      ds_mbar_init(&s_empty[s], 1);
      s_seq[s] = 0;
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
  ta_prefix(a, s_len);                                // synchronises the block
  ds_tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s_tmem, 0);
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };
  auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t limit) {
    if (ds_mbar_wait_or_abort(bar, parity & 1u, limit, &s_abort)) return true;
    if (!aborted()) ds_set_error(a.status, DSPARK_ETIMEOUT);
    s_abort = 1;
    return false;
  };
  TaWalk walk;
  walk.init(s_len);
  TaPiece p;

  if (warp == 0 || warp == 2) {
    // ---- key tiles (warp 0) and value tiles (warp 2): lane b looks up the page of box b (keys b * box ..),
    // then the boxes go out one after the other. The copy of a box past the last key, or of a page that
    // does not exist, names a page past the last and reads zeros. The tiles lie in the ring in the order in
    // which the MMA warp takes them: K0 V0 K1 V1 .. for two row tiles, else K0 K1 V0 K2 V1 K3 .. ----
    const bool isv = warp == 2;
    const CUtensorMap* tm = isv ? &tmV : &tmK;
    const int box = a.box, nbox = TA_KT / box;
    uint32_t base = 0;                                 // sequence number of the piece's first tile
    bool ok = true;
    while (ok && walk.next(s_len, a, p)) {
      const uint32_t len = uint32_t(s_len.ctx[p.r]) + uint32_t(s_len.n[p.r]), page = uint32_t(a.c.page_size);
      const int32_t* table = a.c.page_table + int64_t(p.r) * a.c.ld_table;
      const int npt = p.t1 - p.t0;
      int32_t place = 0, pg = 0;
      auto look_up = [&](int t) {                      // (page, place) of this lane's box of the piece's tile t
        pg = int32_t(a.c.num_pages);
        const uint32_t key = uint32_t(p.t0 + t) * TA_KT + uint32_t(lane * box);
        if (lane < nbox && t < npt && key < len) {
          const uint32_t e = key / page;
          place = int32_t(key - e * page);
          pg = table[e];
          if (pg < 0 || pg >= a.c.num_pages) {
            ds_set_error(a.status, DSPARK_ERANGE);
            pg = int32_t(a.c.num_pages);
          }
        }
      };
      look_up(0);
      for (int t = 0; t < npt; ++t) {
        const uint32_t sq = base + (TWO ? 2 * t + (isv ? 1 : 0) : isv ? min(npt, t + 2) + t : t < 2 ? t : 2 * t - 1);
        const uint32_t s = sq % NS;
        const int32_t pg_t = pg, place_t = place;
        look_up(t + 1);                                // on its way while this tile waits for its stage
        ok = __all_sync(0xFFFFFFFFu, wait(&s_empty[s], (sq / NS + 1), DS_WAIT_LIMIT));
        if (!ok) break;
        if (lane == 0) {
          s_seq[s] = sq + 1;
          ds_mbar_arrive_expect_tx(&s_full[s], STAGE);
        }
        __syncwarp();
#pragma unroll 1
        for (int b = 0; b < nbox; ++b) {
          const int32_t pb = __shfl_sync(0xFFFFFFFFu, pg_t, b), lb = __shfl_sync(0xFFFFFFFFu, place_t, b);
#pragma unroll
          for (int c = 0; c < NC; ++c)
            ta_tma_load(sR + s * STAGE + c * TA_CHUNK + b * box * 128, tm, c * 64, lb, p.hk, pb, &s_full[s]);
        }
      }
      base += 2 * npt;
    }
  } else if (warp == 1) {
    // ---- one lane issues the MMAs. QK of a group's next tile follows the group's PV: S and P share
    // tensor memory, and the MMAs of one thread run in order ----
    constexpr uint32_t idS = ds_idesc_bf16_f32(128, TA_KT);
    constexpr uint32_t idO = ds_idesc_bf16_f32(128, DP) | (1u << 16);   // B is N-major
    const uint32_t qdesc = ta_desc_k(ds_smem_addr(sQ)), kdesc = ta_desc_k(ds_smem_addr(sR)), vdesc = ta_desc_n(ds_smem_addr(sR));
    uint32_t seq = 0, np = 0, pn[2] = {0, 0};
    bool ok = true;
    auto full = [&](uint32_t sq) {
      ok = ok && wait(&s_full[sq % NS], sq / NS, DS_WAIT_LIMIT);
      ds_tc_fence_after();
      return ok;
    };
    auto release = [&](uint32_t sq) { ta_commit(&s_empty[sq % NS]); };
    auto qk = [&](int g, uint32_t sq) {
      const uint32_t q0 = __shfl_sync(0xFFFFFFFFu, qdesc + (((TWO ? g : 0) * STAGE) >> 4), 0);
      const uint32_t k0 = __shfl_sync(0xFFFFFFFFu, kdesc + (((sq % NS) * STAGE) >> 4), 0);
      const uint32_t d0 = __shfl_sync(0xFFFFFFFFu, tmem + TS + 128 * g, 0);
#pragma unroll
      for (int kb = 0; kb < DP / 16; ++kb) {
        const uint32_t off = ((kb >> 2) * TA_CHUNK + (kb & 3) * 32) >> 4;
        ta_umma_ss<TA_DESC_HI>(d0, q0 + off, k0 + off, idS, kb != 0);
      }
      ta_commit(&s_sfull[g]);
    };
    auto pv = [&](int g, uint32_t sq, bool acc) {
      const uint32_t v0 = __shfl_sync(0xFFFFFFFFu, vdesc + (((sq % NS) * STAGE) >> 4), 0);
      const uint32_t d0 = __shfl_sync(0xFFFFFFFFu, tmem + TO + DP * g, 0), a0 = __shfl_sync(0xFFFFFFFFu, tmem + TS + 128 * g, 0);
      const uint32_t acc0 = __shfl_sync(0xFFFFFFFFu, uint32_t(acc), 0);
#pragma unroll
      for (int kb = 0; kb < TA_KT / 16; ++kb)
        ta_umma_ts<TA_DESC_HI>(d0, a0 + kb * 8, v0 + ((kb * 2048) >> 4), idO, kb ? 1u : acc0);
    };
    auto weights = [&](int g, bool first) {          // P of group g is written; at first O must be free too
      ok = ok && wait(&s_pfull[g], pn[g]++, DS_WAIT_LIMIT);
      if (first && np > 0) ok = ok && wait(&s_ofree, np - 1, DS_WAIT_LIMIT);
      ds_tc_fence_after();
      return ok;
    };
    while (ok && walk.next(s_len, a, p)) {
      const int nt = p.t1 - p.t0;
      ok = wait(&s_qfull, np, DS_WAIT_LIMIT);
      if (!ok) break;
      ds_tc_fence_after();
      if (TWO) {                                     // ring order: K0, then V_t, K_{t+1}
        if (!full(seq)) break;
        qk(0, seq);
        qk(1, seq);
        release(seq++);
        if (nt == 1) ta_commit(&s_qempty);
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
            if (t + 2 == nt) ta_commit(&s_qempty);
          }
        }
      } else {                                       // ring order: K0, K1, then V_t, K_{t+2}
        for (int t = 0; t < min(2, nt); ++t) {
          if (!full(seq)) break;
          qk(t, seq);
          release(seq++);
        }
        if (nt <= 2) ta_commit(&s_qempty);
        for (int t = 0; ok && t < nt; ++t) {
          const int g = t & 1;
          if (!weights(g, t == 0) || !full(seq)) break;
          pv(g, seq, t >= 2);
          release(seq++);
          if (t + 2 < nt) {
            if (!full(seq)) break;
            qk(g, seq);
            release(seq++);
            if (t + 3 == nt) ta_commit(&s_qempty);
          }
        }
      }
      if (!ok) break;
      ta_commit(&s_ofull);
      ++np;
    }
    ta_commit(&s_drain);                        // the MMAs are done before tensor memory goes
    (void)ds_mbar_wait(&s_drain, 0, DS_WAIT_LIMIT);
  } else if (warp < 4) {
    // ---- query rows of each piece into the swizzled layout; columns past head_dim are zero (the key
    // tile's are too), rows past the last warp's keep what was there: a row only reaches its own results ----
    constexpr int CPR = DP / 8, STEP = TA_QTHREADS / CPR;        // 16-byte columns of a row, rows per round
    const int qt = lane, c = qt % CPR, D = a.c.head_dim;
    uint32_t np = 0;
    const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + c * 8;
    uint8_t* dst = sQ + (c >> 3) * TA_CHUNK;
    while (walk.next(s_len, a, p)) {
      if (np > 0 && !wait(&s_qempty, np - 1, DS_WAIT_LIMIT)) break;
      const int m0 = p.g * a.rpg, cnt = min(a.rpg, a.rows - m0);
      int i = (m0 + qt / CPR) / a.G, h = (m0 + qt / CPR) - i * a.G;
      const __nv_bfloat16* qr = q + int64_t(p.r) * a.T * a.ldq + int64_t(p.hk) * a.G * D;
      for (int lr = qt / CPR; lr < cnt; lr += STEP) {
        const int row = lr & 127;
        uint8_t* at = dst + (lr >> 7) * STAGE + row * 128 + (((c & 7) ^ (row & 7)) << 4);
        if (c * 8 < D) ds_cp_async16(at, qr + int64_t(i) * a.ldq + h * D);
        else *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
        for (h += STEP; h >= a.G; h -= a.G) ++i;
      }
      // rows that only fill up a warp: zeros, whose scores disturb no vote
      for (int lr = cnt + qt / CPR; lr < min(a.rpg, (cnt + 31) & ~31); lr += STEP)
        *reinterpret_cast<uint4*>(dst + (lr >> 7) * STAGE + (lr & 127) * 128 + (((c & 7) ^ (lr & 7)) << 4)) = make_uint4(0, 0, 0, 0);
      ds_cp_async_wait_all();
      ds_fence_proxy_async_smem();
      ds_mbar_arrive(&s_qfull);
      ++np;
    }
  } else {
    // ---- softmax: group g, one thread per row ----
    const int g = (warp - 4) >> 2, quarter = warp & 3, lr = quarter * 32 + lane;
    const uint32_t tl = tmem + (uint32_t(quarter * 32) << 16);
    const uint32_t tS = tl + TS + 128 * g, tO = tl + TO + DP * g;
    const float sc = CAP ? fminf(a.scale * 2.0f * TA_LOG2E / a.softcap, 3e38f) : a.scale * TA_LOG2E;   // finite: 0 stays 0
    const float cap2 = a.softcap * TA_LOG2E, sy = CAP ? a.scale / a.softcap : 0.0f;
    const float lin = a.scale * TA_LOG2E;                      // |capped score| <= min(cap, |score|)
    const int D = a.c.head_dim;
    uint32_t np = 0, ns = 0, seq = 0;
    bool first = true, ok = true;
    while (ok && walk.next(s_len, a, p)) {
      const int32_t ctx = s_len.ctx[p.r], n = s_len.n[p.r];
      const int64_t len = int64_t(ctx) + n;
      const int npt = p.t1 - p.t0;
      const int m = p.g * a.rpg + (TWO ? g * 128 : 0) + lr;    // this thread's row
      const bool live = p.g * a.rpg + (TWO ? g * 128 : 0) + quarter * 32 < a.rows;   // any row of this warp
      const int i = min(m, a.rows - 1) / a.G;
      // reference (log2), sum of the weights and, with one row tile, of the weights rounded to bf16: the result
      // is divided by the latter, so that a row whose weight lies on few keys keeps its accuracy (one key: v
      // itself). Two row tiles (many rows) take the first sum for both: there the softmax bounds the kernel.
      float mref = -INFINITY, l = 0.0f, lr16 = 0.0f;
      bool has = false;                                        // O holds an earlier tile
      const int tn = ctx / TA_KT - p.t0;                       // tiles from here on hold nodes or the end of the keys
      for (int t = TWO ? 0 : g; t < npt; t += TWO ? 1 : 2) {
        ok = wait(&s_sfull[g], ns++, first ? a.first_wait : DS_WAIT_LIMIT);
        ok = __all_sync(0xFFFFFFFFu, ok);
        first = false;
        if (!ok) break;
        ds_tc_fence_after();
        const int64_t key0 = int64_t(p.t0 + t) * TA_KT;
        if (t >= tn) {
          const uint32_t sv = seq + (TWO ? 2 * t + 1 : min(npt, t + 2) + t);
          ok = __all_sync(0xFFFFFFFFu, wait(&s_full[sv % NS], sv / NS, DS_WAIT_LIMIT));
          if (!ok) break;
          const int f = int(max(int64_t(ctx) - key0, int64_t(0))), k0 = int(min(len - key0, int64_t(TA_KT)));
          ta_clean<NC>(sR + (sv % NS) * STAGE, f, k0, min(TA_KT, (k0 + a.box - 1) / a.box * a.box), int(key0 + f - ctx),
                       reinterpret_cast<uint32_t*>(s_odd[np % 3]), lr);
          ds_fence_proxy_async_smem();
        }
        if (live) {
          // Masks matter only in tiles that hold nodes or the end of the keys. They are put into S beforehand: -inf, or,
          // under a cap, what is not a number, which neither maximum takes up (there they are looked up again after
          // the cap, and the longer code stays in loops: as straight lines it waits for instructions more than it saves).
          constexpr int FLAT = CAP ? 1 : 8;
          const bool masked = t >= tn;
          const int64_t nd = key0 - ctx;
          if (masked) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float v[16];
              uint32_t w[16];
              ds_tmem_ld_32x32b_x16(tS + 16 * c, v);
              const uint32_t bits = ta_mask32(a, p.r, i, n, nd + 16 * c);
              __syncwarp();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = (bits >> e) & 1u ? __float_as_uint(v[e]) : CAP ? 0x7FFFFFFFu : 0xFF800000u;
              ta_tmem_st_x16(tS + 16 * c, w);
            }
            ta_tmem_wait_st();
          }
          // Under a cap the largest |score| is looked for first, which picks the cap's form below. No row's maximum is
          // above it (and its linear bound), so tiles in which that is below every row's reference need no maximum.
          bool maxima = !CAP || masked || __any_sync(0xFFFFFFFFu, mref == -INFINITY);
          float mx = -INFINITY, mg = 0.0f;
#pragma unroll 1
          for (;;) {
            // chains of four maxima, and below of four sums, side by side: one would wait for itself
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, mg4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float va[32], vb[32];
            auto look = [&](float (&v)[32], int c) {
              if (CAP) {
#pragma unroll
                for (int e = 0; e < 32; e += 2) mg4[(e >> 1) & 3] = fmaxf(mg4[(e >> 1) & 3], fmaxf(fabsf(v[e]), fabsf(v[e + 1])));
                if (!maxima) return;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) mx4[(e >> 1) & 3] = fmaxf(mx4[(e >> 1) & 3], fmaxf(v[e], v[e + 1]));
            };
            ta_tmem_fetch(tS, va);
#pragma unroll FLAT
            for (int c = 0; c < 4; c += 2) {
              ta_arrived(va);
              ta_tmem_fetch(tS + 32 * c + 32, vb);
              look(va, c);
              ta_arrived(vb);
              if (c == 0) ta_tmem_fetch(tS + 64, va);
              look(vb, c + 1);
            }
            mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            mg = fmaxf(fmaxf(mg4[0], mg4[1]), fmaxf(mg4[2], mg4[3]));
            if (maxima || !__any_sync(0xFFFFFFFFu, fminf(cap2, mg * lin) > mref)) break;
            maxima = true;
          }
          float v[16];
          ta_tmem_fetch(tS, v);
          // A row's form of the cap goes by the scores that it sees, so that its result is the same whatever the others
          // are; the warp's votes below only leave out forms that none of its rows needs.
          const bool narrow = CAP && mg * sy <= a.narrow_to, wide = CAP && (narrow || mg * sy <= a.wide_to);
          auto coefficients = [&](float (&co)[7]) {
#pragma unroll
            for (int k = 0; k < 7; ++k) co[k] = narrow ? (k < 4 ? a.narrow[k].x : 0.0f) : a.wide[k];
          };
          float m2 = mx == -INFINITY ? -INFINITY : mx * sc;
          if (CAP && maxima) {
            float co[7];
            coefficients(co);
            m2 = mx == -INFINITY ? -INFINITY : wide ? mx * ds_f2lo(ta_poly(co, ds_f2(mx, mx))) : ta_tanh(mx * sc, cap2);
          }
          // (the bound again, so that a row does the same whoever made its warp look for maxima)
          const bool up = m2 > mref && (!CAP || (maxima && fminf(cap2, mg * lin) > mref));
          if (__any_sync(0xFFFFFFFFu, up)) {
            const float to = m2 + TA_ABOVE, f = up ? ta_ex2(mref - to) : 1.0f;     // 0 from -inf
            if (has) {
#pragma unroll 1
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
            lr16 *= f;
            if (up) mref = to;
          }
          const float mu = mref == -INFINITY ? 0.0f : mref;
          const uint64_t nm2 = ds_f2(-mu, -mu);
          const bool all_narrow = CAP && __all_sync(0xFFFFFFFFu, narrow), all_wide = CAP && __all_sync(0xFFFFFFFFu, wide);
          const bool any_wide = CAP && __any_sync(0xFFFFFFFFu, wide);
          uint64_t sum[4] = {0, 0, 0, 0}, sum16[2] = {0, 0};
          auto put = [&](const uint64_t (&x)[8], int c) {      // weights of 16 keys: exponentials, sums, P
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x0 = ta_ex2(ds_f2lo(x[e])), x1 = ta_ex2(ds_f2hi(x[e]));
              sum[e & 3] = ds_add2(sum[e & 3], ds_f2(x0, x1));
              w[e] = ta_pack(x0, x1);
              if (!TWO) sum16[e & 1] = ds_add2(sum16[e & 1], ds_f2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)));
            }
            ta_tmem_st_x8(tS + 8 * c, w);
          };
          auto exponents = [&](uint64_t (&x)[8]) {             // the common forms, one pair of scores at a time
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint64_t y = ds_f2(v[2 * e], v[2 * e + 1]);
              x[e] = ds_fma2(y, CAP ? ta_poly_narrow(a, y) : ds_f2(sc, sc), nm2);
            }
          };
          if (!CAP || (all_narrow && !masked)) {
            // 16 keys' FMAs beside the 16 keys' exponentials before them: one warp alone keeps both pipes busy
            uint64_t x[2][8];
            ta_arrived(v);
            exponents(x[0]);
            ta_tmem_fetch(tS + 16, v);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (c < 7) {
                ta_arrived(v);
                exponents(x[(c + 1) & 1]);
                if (c < 6) ta_tmem_fetch(tS + 16 * c + 32, v);
              }
              put(x[c & 1], c);
            }
          } else {
            float co[7];
            coefficients(co);
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint64_t x[8] = {};
              ta_arrived(v);
              if (any_wide) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const uint64_t y = ds_f2(v[2 * e], v[2 * e + 1]);
                  x[e] = ds_fma2(y, ta_poly(co, y), nm2);
                }
              }
              if (!all_wide) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const float x0 = ta_tanh(v[2 * e] * sc, cap2) - mu, x1 = ta_tanh(v[2 * e + 1] * sc, cap2) - mu;
                  x[e] = wide ? x[e] : ds_f2(x0, x1);
                }
              }
              if (masked) {
                const uint32_t bits = ta_mask32(a, p.r, i, n, nd + 16 * c);
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  x[e] = ds_f2((bits >> (2 * e)) & 1u ? ds_f2lo(x[e]) : -INFINITY, (bits >> (2 * e + 1)) & 1u ? ds_f2hi(x[e]) : -INFINITY);
              }
              if (c < 7) ta_tmem_fetch(tS + 16 * c + 16, v);
              put(x, c);
            }
          }
          sum[0] = ds_add2(ds_add2(sum[0], sum[1]), ds_add2(sum[2], sum[3]));
          l += ds_f2lo(sum[0]) + ds_f2hi(sum[0]);
          sum16[0] = ds_add2(sum16[0], sum16[1]);
          if (!TWO) lr16 += ds_f2lo(sum16[0]) + ds_f2hi(sum16[0]);
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
        s_ml[np & 1][g][lr] = make_float4(mref, l, lr16, 0.0f);
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
          const float4 x = s_ml[np & 1][0][lr], y = s_ml[np & 1][1][lr];
          mref = fmaxf(x.x, y.x);
          w0 = x.x == -INFINITY ? 0.0f : ta_ex2(x.x - mref);
          w1 = y.x == -INFINITY ? 0.0f : ta_ex2(y.x - mref);
          l = w0 * x.y + w1 * y.y;
          lr16 = w0 * x.z + w1 * y.z;
        } else {
          lr16 = l;
        }
        const bool any = valid && l != 0.0f;                   // also when l is not a number
        const float inv = any ? 1.0f / lr16 : 0.0f;
        const bool whole = p.whole();
        const int d0 = TWO ? 0 : g * (DP / 2), d1 = TWO ? DP : d0 + DP / 2;
        const int64_t slot = p.slot(blockIdx.x);
        const int h = p.hk * a.G + m - i * a.G;
        const int64_t row = int64_t(p.r) * a.T + i;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.ldo + int64_t(h) * D;
        float* part = a.part_o + (slot * a.rs + (m - p.g * a.rpg)) * D;
#pragma unroll 1
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
                if (d + e < D) *reinterpret_cast<float4*>(part + d + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
        }
        __syncwarp();
        if (m < a.rows && (TWO || g == 0)) {
          if (!whole) a.part_ml[slot * a.rs + m - p.g * a.rpg] = valid ? make_float4(mref, l, lr16, 0.0f) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
          else if (a.lse) a.lse[row * a.Hq + h] = any ? (mref + log2f(l)) * TA_LN2 : -INFINITY;
        }
        if (int64_t(p.t1) * TA_KT > ctx) {
          const uint32_t* odd = reinterpret_cast<const uint32_t*>(s_odd[np % 3]);
          uint32_t marks = 0;
#pragma unroll 1
          for (int w = 0; w < a.W; ++w) marks |= odd[w];
          if (marks && valid)
            ta_add_odd(a, p.r, ctx, n, i, p.hk, d0, min(d1, D), odd, reinterpret_cast<const __nv_bfloat16*>(a.q) + row * a.ldq + int64_t(h) * D,
                       whole ? out : nullptr, part);
        }
      }
      // Marks of this piece's nodes. (Those of the piece before are no longer read: O was free for this piece after
      // every warp was done with that one. They are cleared for the piece after the next.)
      if (warp == 4 && lane < TA_MAXT / 128) s_odd[(np + 2) % 3][lane] = make_uint4(0, 0, 0, 0);
      ds_tc_fence_before();
      __syncwarp();
      if (lane == 0) ds_mbar_arrive(&s_ofree);
      seq += 2 * npt;
      ++np;
    }
  }
  __syncthreads();
  // After a wait that ran out, the copies in flight land before the block leaves its shared memory to another
  // (otherwise the MMA warp has waited for every one of them). Only here, past the barrier, has every copy been
  // issued and does every warp know of the wait.
  if (warp == 1) {
    if (aborted())
      for (int k = 0; k < NS; ++k)
        if (s_seq[k]) (void)ds_mbar_wait(&s_full[k], ((s_seq[k] - 1) / NS) & 1u, DS_WAIT_LIMIT);
    __syncwarp();
    ds_tc_fence_after();
    ds_tmem_dealloc(tmem, 512);
  }
}

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

constexpr size_t TA_WS_PREF = 4352;        // pref[TA_MAXR + 1], rounded up to 256 bytes

}  // namespace

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
  if (maps) DS_CUDA_TRY(D <= 64 ? ta_dispatch_tc<64>(a, grid, mk, mv, stream) : ta_dispatch_tc<128>(a, grid, mk, mv, stream));
  else DS_CUDA_TRY(ta_launch_float(a, grid, stream));
  const dim3 jg{unsigned(ds_ceil_div(jobs, 8))}, jb{256};
  if (cache->dtype == DSPARK_BF16) {
    if (D <= 128) DS_CUDA_TRY(ds_launch(tree_attn_join_kernel<__nv_bfloat16, 1>, jg, jb, 0, stream, a, uint32_t(grid), jobs));
    else DS_CUDA_TRY(ds_launch(tree_attn_join_kernel<__nv_bfloat16, 2>, jg, jb, 0, stream, a, uint32_t(grid), jobs));
  } else {
    if (D <= 128) DS_CUDA_TRY(ds_launch(tree_attn_join_kernel<float, 1>, jg, jb, 0, stream, a, uint32_t(grid), jobs));
    else DS_CUDA_TRY(ds_launch(tree_attn_join_kernel<float, 2>, jg, jb, 0, stream, a, uint32_t(grid), jobs));
  }
  return DSPARK_OK;
}
