// tree_attn_q8_rows.cu - attention over a cache in 8 bits for few query rows a key head (dspark_tree_attention_q8): single new
// tokens and short drafted blocks.
//
// openvino.genai PR #4847, Fixes > Split validation windows, and optimum-intel PR #2098 (paged attention targets).
//
// The rows that read one key head (at most 32) make NQ tiles of 8; a warp takes 16 keys (a slice) at a time and turns the products over, keys and
// value columns on the 16-row side of mma.sync:
//   S^T[16 keys, 8 rows] = K Q^T,  P = 2^(x - m) in f16,  O^T[16 columns, 8 rows] += V^T P^T  (P^T by movmatrix)
// with its own running reference m, sum and O, so warps need nothing from each other until their shares end. A contraction may take its
// index in any order and a result its rows, so a thread's operand registers are filled from 16 contiguous codes of a key: codes go from shared
// memory into registers once, become f16 there and are used where they are. tcgen05 would need them staged in 16 bits in shared memory: 2 D
// bytes written and read again a key, which takes longer than HBM needs for the codes.
//
// Numbers. A code times a power of two from 2^-14 to 2^7 is an f16 number exactly. The powers of a slice's keys are taken relative to a
// reference (the largest of the slice, for keys; a running one of each block of columns, for values, which O is relative to), and a slice whose
// powers lie further apart takes bf16 forms with the full range instead. Queries go to f16 under a power of two of each row: what is below
// 2^-38 of the row's largest is lost there, which is less than a float32 sum loses. Weights reach up to 2^15 and are rounded to f16's eleven
// bits (2^-12 of a weight; those below 2^-32 of the row's largest to less).
//
// Every warp copies its own slices with TMA, NS of them in flight, and waits for nothing but its own barriers. The work is the line of
// tiles of tree_attn.cuh with 16 keys a tile: a block's share is cut once more into its warps' shares, what two warps leave of an item is joined
// at the end in shared memory (in the order of the keys), and what two blocks leave by the join kernel.
#include <cuda_fp16.h>

#include <type_traits>

#include "cache_q8.cuh"
#include "tree_attn.cuh"

namespace {

constexpr int TQ_KEYS = 16;                  // keys of a slice
constexpr float TQ_TOP = 15.0f;              // weights reach 2^15;
constexpr float TQ_AT = 7.0f;                // a new reference gives the largest score a weight of 2^7
constexpr float TQ_NONE = -3e38f;            // reference of a row that has seen nothing

template <int DP, int NQ>
struct TqLayout {
  static constexpr int WARPS = NQ == 1 ? 16 : NQ == 2 ? 12 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int NS = NQ <= 2 ? 2 : 4;
  static constexpr int STEPS = DP / 16;                // contraction steps of K Q^T; row tiles of O^T
  static constexpr uint32_t SLICE = 2 * TQ_KEYS * DP;  // bytes of a slice's keys and values
  // dynamic shared memory: rings of slices (where a warp's last partial result goes when they are done with), scale words, queries
  static constexpr uint32_t RING = NS * SLICE;
  static constexpr uint32_t SCALE = WARPS * RING;      // [WARPS][NS][32] words: scale bytes of 16 keys, then of 16 values
  static constexpr uint32_t QF = SCALE + WARPS * NS * 128;
  static constexpr uint32_t QW = NQ * STEPS * 256;     // bytes of a warp's queries
  static constexpr uint32_t TOTAL = QF + WARPS * QW;
  static_assert(8 * NQ * DP * 4 <= RING, "a partial result fits its warp's ring");
};

DS_DEV void tq_tma_load(uint32_t dst, const void* tmap, int32_t d, int32_t t, int32_t h, int32_t p, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(tmap), "r"(d), "r"(t), "r"(h), "r"(p), "r"(bar)
      : "memory");
}

// D += A B, 16 x 8 x 16, with float32 sums.
template <bool BF>
DS_DEV void tq_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DS_DEV uint32_t tq_transpose(uint32_t x) {             // of an 8 x 8 matrix of 16-bit numbers, a warp's
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
DS_DEV uint32_t tq_mul2h(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
DS_DEV uint32_t tq_fma2h(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
DS_DEV uint32_t tq_mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
DS_DEV uint32_t tq_sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF>
DS_DEV uint32_t tq_pack(float lo, float hi) {
  uint32_t r;
  if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes as two pairs of f16 numbers times 2^(byte - 15), `f` being that byte in both halves' exponents (1..22). E4M3: bytes 0, 1 and
// 2, 3 by the conversion. INT8: bytes 0, 2 and 1, 3: 1152 + code is an f16 number (0x6400 + the code's byte with its top bit turned), `c` is
// -1152 times f.
struct TqFactor {
  uint32_t f, c;
};
template <bool E4M3>
DS_DEV TqFactor tq_factor(uint32_t lo, uint32_t hi) {
  TqFactor x;
  x.f = (lo << 10) | (hi << 26);
  x.c = E4M3 ? 0u : tq_mul2h(x.f, 0xE480E480u);
  return x;
}
template <bool E4M3>
DS_DEV void tq_widen(uint32_t w, const TqFactor& f, uint32_t& first, uint32_t& second) {
  if (E4M3) {
    uint32_t a, b;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(a), "=r"(b) : "r"(w));
    first = tq_mul2h(a, f.f);
    second = tq_mul2h(b, f.f);
  } else {
    first = tq_fma2h((w & 0x00FF00FFu) ^ 0x64806480u, f.f, f.c);
    second = tq_fma2h(((w >> 8) & 0x00FF00FFu) ^ 0x64806480u, f.f, f.c);
  }
}

// The same as bf16 numbers over the whole range, in the same order: E4M3's seven bits under the sign go to bits 10..4, the number times 2^-120, so that
// factors above 2^7 take two steps; INT8 is 128 + (low seven bits) - 128 (1 + sign). `e`: the powers' exponents.
template <bool E4M3>
DS_DEV void tq_widen_far(uint32_t w, int elo, int ehi, uint32_t& first, uint32_t& second) {
  auto power = [](int e) { return e < -126 ? 0u : uint32_t(min(e, 127) + 127) << 7; };
  uint32_t x = w, y;
  if (E4M3) x = __byte_perm(w, 0u, 0x3120);            // bytes 0, 2, 1, 3: the pairs are then bytes 0, 2 and 1, 3 in both formats
  if (E4M3) {
    y = (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
    x = ((x << 8) & 0x80008000u) | ((x << 4) & 0x07F007F0u);
    const uint32_t f = power(elo + 120) | (power(ehi + 120) << 16), g = power(max(elo - 7, 0)) | (power(max(ehi - 7, 0)) << 16);
    first = tq_mul2(tq_mul2(x, f), g);
    second = tq_mul2(tq_mul2(y, f), g);
  } else {
    y = x >> 8;
    const uint32_t f = power(elo) | (power(ehi) << 16);
    first = tq_mul2(tq_sub2((x & 0x007F007Fu) | 0x43004300u, (x & 0x00800080u) | 0x43004300u), f);
    second = tq_mul2(tq_sub2((y & 0x007F007Fu) | 0x43004300u, (y & 0x00800080u) | 0x43004300u), f);
  }
}

// Largest of each byte over the warp.
DS_DEV uint32_t tq_max4(uint32_t w) {
  uint32_t r = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) r |= __reduce_max_sync(0xFFFFFFFFu, (w >> (8 * b)) & 0xFFu) << (8 * b);
  return r;
}

// A warp's part of an item that it shares with others.
struct TqPart {
  TaPiece p;
  int valid;
};

template <int DP, int NQ, bool CAP, bool E4M3>
__global__ void __launch_bounds__(TqLayout<DP, NQ>::THREADS, 1)
tree_attn_q8_rows_kernel(const TaArgs a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using L = TqLayout<DP, NQ>;
  constexpr int NS = L::NS, STEPS = L::STEPS, WARPS = L::WARPS, ROWS = 8 * NQ;
  constexpr int VW = DP / 32;                          // words of codes a thread has of a key's values
  constexpr uint32_t HI = E4M3 ? 22u : 20u;            // f16 exponents 1..HI keep code times power exact and finite
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[WARPS][NS];
  __shared__ TaLens s_len;
  __shared__ TaWalk s_walk[WARPS];
  __shared__ TaPiece s_piece[WARPS][3];
  __shared__ int s_there[WARPS][3];                    // whether the piece is one
  __shared__ TqPart s_head[WARPS], s_tail[WARPS];      // the first piece, if an earlier warp began it and it ends here; the last, if it goes on
  __shared__ float2 s_ml[2][WARPS][ROWS];              // their references and sums
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + warp * L::RING;
  uint32_t* scales = reinterpret_cast<uint32_t*>(smem + L::SCALE) + warp * NS * 32;
  uint2* qf = reinterpret_cast<uint2*>(smem + L::QF + warp * L::QW) + lane;
  const int D = a.c.head_dim, nb = q8_blocks(D);
  const bool words = nb == 4 && a.q8.vec4 != 0;        // a slot's scales are one aligned word
  const TaPiece* piece = s_piece[warp];
  const int* there = s_there[warp];
  ds_pdl_trigger();
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) ds_mbar_init(&s_full[warp][s], 1);
    ds_fence_mbar_init_cluster();
    s_head[warp].valid = s_tail[warp].valid = 0;
  }
  if (tid == 0) {
    s_abort = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmK) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmV) : "memory");
  }
  ds_pdl_wait();
  ta_prefix(a, s_len);                                 // synchronises the block
  auto more = [&](int k) {                             // lane 0: finds piece number k of the warp's share
    s_there[warp][k % 3] = s_walk[warp].find(s_len, a, s_piece[warp][k % 3]);
  };
  if (lane == 0) {
    const int64_t share = s_len.end - s_len.at;
    TaWalk w;
    w.init(s_len);
    w.at = s_len.at + share * warp / WARPS;
    w.end = s_len.at + share * (warp + 1) / WARPS;
    s_walk[warp] = w;
    more(0);
    more(1);
  }
  __syncwarp();
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };

  // ---- this warp's slices: the next one to copy, its page known beforehand ----
  int kp = 0;                                          // piece that is worked on
  int np = 0, nt = piece[0].t0;                        // piece (0: that one, 1: the one after it) and tile of the next copy
  bool valid = false;
  int32_t pg = 0, place = 0;                           // page and place of this lane's key of that slice (lane & 15); pg < 0: no key
  uint32_t issued = 0, used = 0, pend = 0;
  int pend_at = -1;
  auto advance = [&]() {                               // finds the next slice and asks for its page
    valid = false;
    for (;; ++np, nt = piece[(kp + 1) % 3].t0) {
      if (!there[(kp + np) % 3]) return;
      if (nt < piece[(kp + np) % 3].t1) break;
      if (np == 1) return;
    }
    const TaPiece& p = piece[(kp + np) % 3];
    const uint32_t key = uint32_t(nt) * TQ_KEYS + (lane & 15), len = uint32_t(s_len.ctx[p.r]) + uint32_t(s_len.n[p.r]);
    pg = -1;
    if (key < len) {
      const uint32_t e = key / uint32_t(a.c.page_size);
      place = int32_t(key - e * uint32_t(a.c.page_size));
      pg = a.c.page_table[int64_t(p.r) * a.c.ld_table + e];
      if (pg < 0 || pg >= a.c.num_pages) {
        ds_set_error(a.status, DSPARK_ERANGE);
        pg = -1;
      }
    }
    valid = true;
  };
  auto flush = [&]() {                                 // the scales asked for last have arrived; no key: 0
    if (pend_at >= 0) scales[pend_at * 32 + lane] = pend;
    pend_at = -1;
  };
  auto issue = [&]() {
    flush();
    const TaPiece& p = piece[(kp + np) % 3];
    const int s = int(issued % NS);
    const uint32_t bar = ds_smem_addr(&s_full[warp][s]), dst = ds_smem_addr(ring + s * L::SLICE);
    if (lane == 0) ds_mbar_arrive_expect_tx(&s_full[warp][s], L::SLICE);
    __syncwarp();
    // boxes of 16 or 8 places: the lane of a box's first key (lanes 16 and above: its values) copies it; past the end, or from a page that
    // does not exist, a box names a page past the last and reads zeros
    if ((lane & (a.box - 1)) == 0)
      tq_tma_load(dst + (lane & 24) * DP, lane < 16 ? &tmK : &tmV, 0, place, p.hk, pg < 0 ? int32_t(a.c.num_pages) : pg, bar);
    pend = 0;
    if (pg >= 0) {
      const uint8_t* at = (lane < 16 ? a.q8.k_scale : a.q8.v_scale) + int64_t(pg) * a.q8.page_stride + int64_t(place) * a.q8.token_stride +
                          int64_t(p.hk) * a.q8.head_stride;
      if (words) {
        pend = *reinterpret_cast<const uint32_t*>(at);
      } else {
        for (int b = 0; b < nb; ++b) pend |= uint32_t(at[b]) << (8 * b);
      }
    }
    pend_at = s;
    ++issued;
    ++nt;
    advance();
  };
  advance();
  const float sc = CAP ? fminf(a.scale * 2.0f * TA_LOG2E / a.softcap, 3e38f) : a.scale * TA_LOG2E;
  const float cap2 = a.softcap * TA_LOG2E, sy = CAP ? a.scale / a.softcap : 0.0f;
  bool ok = true, first = true;
  for (; there[kp % 3]; ++kp) {
    const TaPiece p = piece[kp % 3];
    const int32_t ctx = s_len.ctx[p.r], n = s_len.n[p.r];
    const int m0 = p.g * a.rpg;
    if (ok) {
      while (issued - used < NS) {
        if (!valid) advance();
        if (!valid) break;
        issue();
      }
    }
    // ---- query rows (n index g of each tile) in the order of the operand registers, in f16 under 2^qe of the row ----
    const __nv_bfloat16* qrow[NQ];
    float qfac[NQ][2];                                   // of rows 2 t4, 2 t4 + 1 of each tile: that power back, and the scale
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq) {
      const int m = m0 + 8 * nq + g, i = m / a.G, h = m - i * a.G;
      qrow[nq] = m < a.rows ? reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t(p.r) * a.T + i) * a.ldq + (int64_t(p.hk) * a.G + h) * D : nullptr;
      uint2 x[STEPS];
      float most = 0.0f;
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int d = t4 * (DP / 4) + 4 * st;
        x[st] = make_uint2(0u, 0u);
        if (qrow[nq] && d < D) x[st] = *reinterpret_cast<const uint2*>(qrow[nq] + d);
      }
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = e < 2 ? x[st].x : x[st].y;
          const float v = fabsf(__uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16));
          if (v < INFINITY) most = fmaxf(most, v);
        }
      }
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      const int qe = min(max(int(__float_as_uint(most) >> 23), 27), 254) - 140;     // the largest goes to 2^13 .. 2^14
      const float down = __uint_as_float(uint32_t(127 - qe) << 23);
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        float v[4] = {__uint_as_float(x[st].x << 16), __uint_as_float(x[st].x & 0xFFFF0000u), __uint_as_float(x[st].y << 16), __uint_as_float(x[st].y & 0xFFFF0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] *= down;
        qf[(nq * STEPS + st) * 32] = E4M3 ? make_uint2(tq_pack<false>(v[0], v[1]), tq_pack<false>(v[2], v[3]))
                                          : make_uint2(tq_pack<false>(v[0], v[2]), tq_pack<false>(v[1], v[3]));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int other = __shfl_sync(0xFFFFFFFFu, qe, (2 * t4 + e) * 4);
        qfac[nq][e] = __uint_as_float(uint32_t(other + 127) << 23) * (CAP ? 1.0f : sc);
      }
    }
    float o[NQ][STEPS][4] = {}, mref[NQ][2], l[NQ][2];
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mref[nq][e] = TQ_NONE;
        l[nq][e] = 0.0f;
      }
    uint32_t ev = 0, ek = 0;                           // references: scale bytes of the values' blocks, of keys (all four bytes alike); 0: none
    for (int t = p.t0; ok && t < p.t1; ++t) {
      const int s = int(used % NS);
      flush();
      ok = ds_mbar_wait_or_abort(&s_full[warp][s], (used / NS) & 1u, first ? a.first_wait : DS_WAIT_LIMIT, &s_abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      first = false;
      if (!ok) {
        if (!aborted()) ds_set_error(a.status, DSPARK_ETIMEOUT);
        s_abort = 1;
        break;
      }
      const uint8_t *K = ring + s * L::SLICE, *V = K + TQ_KEYS * DP;
      uint32_t* ws = scales + s * 32;
      const int64_t nd = int64_t(t) * TQ_KEYS - ctx;
      // ---- this slice's powers relative to the references: lane k < 16 has key k's four bytes, lane 16 + k its values' ----
      uint32_t w4 = ws[lane];
      const bool some = w4 != 0u || nd + (lane & 15) < n;      // a key is there (0 may be its bytes, or a page that is not)
#pragma unroll
      for (int b = 0; b < 4; ++b) {                    // bytes 1..245; what is not there is the reference itself
        const uint32_t x = (w4 >> (8 * b)) & 0xFFu;
        if (x == 0u || x > uint32_t(Q8_TOP)) w4 = (w4 & ~(0xFFu << (8 * b))) | ((x == 0u ? 1u : uint32_t(Q8_TOP)) << (8 * b));
      }
      const int cut = nb < 4 ? 8 * (4 - nb) : 0;
      const uint32_t used_bytes = 0xFFFFFFFFu >> cut;
      auto relative = [&](uint32_t& rel) {             // exponents of f16, or false
        const uint32_t ref = lane < 16 ? ek : ev;
        const uint32_t w = some ? (w4 & used_bytes) | (ref & ~used_bytes) : ref;
        const uint32_t de = (w & 0x00FF00FFu) + 0x000F000Fu - (ref & 0x00FF00FFu);
        const uint32_t dq = ((w >> 8) & 0x00FF00FFu) + 0x000F000Fu - ((ref >> 8) & 0x00FF00FFu);
        constexpr uint32_t C = 0x8000u - 1u - HI;      // a half that is 0 or above HI sets a top bit
        constexpr uint32_t CC = C | (C << 16);
        const uint32_t bad = (de | dq | (de + CC) | (dq + CC) | (de - 0x00010001u) | (dq - 0x00010001u)) & 0x80008000u;
        rel = (de & 0x00FF00FFu) | ((dq & 0x00FF00FFu) << 8);
        return bad == 0u && ref != 0u;
      };
      uint32_t rel = 0;
      bool tame = __all_sync(0xFFFFFFFFu, relative(rel));
      if (!tame) {
        // new references: the slice's largest key byte; of each block of values the largest so far, which O changes to
        const uint32_t mk = tq_max4(lane < 16 && some ? w4 & used_bytes : 0u), mv = tq_max4(lane >= 16 && some ? w4 & used_bytes : 0u);
        const uint32_t m1 = max(max(mk & 0xFFu, (mk >> 8) & 0xFFu), max((mk >> 16) & 0xFFu, mk >> 24));
        ek = max(m1, 1u) * 0x01010101u;
        uint32_t to = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t x = (mv >> (8 * b)) & 0xFFu, y = (ev >> (8 * b)) & 0xFFu;
          to |= (y == 0u || x > y + HI - 15u ? max(x, 1u) : y) << (8 * b);
        }
        if (to != ev) {
          const int sh = 8 * (DP == 128 ? g >> 1 : g >> 2);
          const int down = int((ev >> sh) & 0xFFu) - int((to >> sh) & 0xFFu);        // 2^down, in two steps where it is small
          const float f = __uint_as_float(uint32_t(max(down, -126) + 127) << 23), f2 = __uint_as_float(uint32_t(max(down + 126, -126) + 127) << 23);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < STEPS; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nq][j][e] = down < -126 ? o[nq][j][e] * f * f2 : o[nq][j][e] * f;
          ev = to;
        }
        tame = __all_sync(0xFFFFFFFFu, relative(rel));
      }
      ws[lane] = tame ? rel : some ? w4 : 0x01010101u;
      __syncwarp();
      const uint8_t *ks = reinterpret_cast<const uint8_t*>(ws), *vs = ks + 64;
      uint32_t kb[2], vb[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) kb[x] = ks[(8 * x + g) * 4 + (DP == 128 ? t4 : t4 >> 1)];
#pragma unroll
      for (int x = 0; x < 4; ++x) vb[x] = vs[(2 * t4 + (x & 1) + 8 * (x >> 1)) * 4 + (DP == 128 ? g >> 1 : g >> 2)];
      auto slice = [&](auto far) {
        constexpr bool FAR = decltype(far)::value;
        float sco[NQ][4] = {};
        {
          uint32_t w[2][STEPS];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint8_t* row = K + (8 * x + g) * DP;
            if constexpr (DP == 128) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint4 y = *reinterpret_cast<const uint4*>(row + (((2 * t4 + c) ^ g) << 4));
                w[x][4 * c] = y.x; w[x][4 * c + 1] = y.y; w[x][4 * c + 2] = y.z; w[x][4 * c + 3] = y.w;
              }
            } else {
              const uint4 y = *reinterpret_cast<const uint4*>(row + ((t4 ^ (g >> 1)) << 4));
              w[x][0] = y.x; w[x][1] = y.y; w[x][2] = y.z; w[x][3] = y.w;
            }
          }
          const TqFactor f[2] = {tq_factor<E4M3>(kb[0], kb[0]), tq_factor<E4M3>(kb[1], kb[1])};
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            uint32_t k4[4];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (FAR) tq_widen_far<E4M3>(w[x][st], int(kb[x]) - 127, int(kb[x]) - 127, k4[x], k4[2 + x]);
              else tq_widen<E4M3>(w[x][st], f[x], k4[x], k4[2 + x]);
            }
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
              uint2 q = qf[(nq * STEPS + st) * 32];
              if (FAR) {                               // the queries themselves
                const int d = t4 * (DP / 4) + 4 * st;
                q = make_uint2(0u, 0u);
                if (qrow[nq] && d < D) q = *reinterpret_cast<const uint2*>(qrow[nq] + d);
                if (!E4M3) q = make_uint2(__byte_perm(q.x, q.y, 0x5410), __byte_perm(q.x, q.y, 0x7632));
              }
              tq_mma<FAR>(sco[nq], k4, q.x, q.y);
            }
          }
        }
        // ---- scores (keys g, g + 8; rows 2 t4, 2 t4 + 1) in units of log2; what a row does not see becomes -inf ----
        const bool masked = nd + TQ_KEYS > 0;
        const float kfac = FAR ? 1.0f : __uint_as_float((ek & 0xFFu) << 23);
        bool up = false;
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          float c[2] = {qfac[nq][0] * kfac, qfac[nq][1] * kfac};
          if (FAR) c[0] = c[1] = CAP ? 1.0f : sc;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float v = sco[nq][e] * c[e & 1];
            if (CAP) {                                 // the odd polynomial where it serves, else from the exponential
              const float y = v, z = y * y;
              const float poly = y * __fmaf_rn(__fmaf_rn(__fmaf_rn(a.narrow[3].x, z, a.narrow[2].x), z, a.narrow[1].x), z, a.narrow[0].x);
              v = fabsf(y) * sy <= a.narrow_to ? poly : ta_tanh(y * sc, cap2);
            }
            sco[nq][e] = v;
          }
          if (masked) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int i = min(m0 + 8 * nq + 2 * t4 + e, a.rows - 1) / a.G;
              const uint32_t bits = ta_mask32(a, p.r, i, n, nd) >> g;
              if (!(bits & 1u)) sco[nq][e] = -INFINITY;
              if (!(bits & 0x100u)) sco[nq][2 + e] = -INFINITY;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) up = up || fmaxf(sco[nq][e], sco[nq][2 + e]) > mref[nq][e] + TQ_TOP;
        }
        if (__any_sync(0xFFFFFFFFu, up)) {             // the reference of a row whose weights would pass 2^15
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float m = fmaxf(sco[nq][e], sco[nq][2 + e]);
#pragma unroll
              for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
              const bool go = m > mref[nq][e] + TQ_TOP;
              const float to = go ? m - TQ_AT : mref[nq][e], f = go ? ta_ex2(mref[nq][e] - to) : 1.0f;
              l[nq][e] *= f;
              mref[nq][e] = to;
#pragma unroll
              for (int j = 0; j < STEPS; ++j) {
                o[nq][j][e] *= f;
                o[nq][j][2 + e] *= f;
              }
            }
        }
        uint32_t pb[NQ][2];                            // P^T: keys 2 t4, 2 t4 + 1 (and + 8) of row g
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sco[nq][e] = ta_ex2(sco[nq][e] - mref[nq][e & 1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) l[nq][e] += sco[nq][e] + sco[nq][2 + e];
          pb[nq][0] = tq_transpose(tq_pack<FAR>(sco[nq][0], sco[nq][1]));
          pb[nq][1] = tq_transpose(tq_pack<FAR>(sco[nq][2], sco[nq][3]));
        }
        // ---- values: columns DP / 8 g .. of keys 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 ----
        uint32_t w[4][VW];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = 2 * t4 + (x & 1) + 8 * (x >> 1);
          if constexpr (DP == 128) {
            const uint4 y = *reinterpret_cast<const uint4*>(V + key * DP + ((g ^ (key & 7)) << 4));
            w[x][0] = y.x; w[x][1] = y.y; w[x][2] = y.z; w[x][3] = y.w;
          } else {
            const uint2 y = *reinterpret_cast<const uint2*>(V + key * DP + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
            w[x][0] = y.x; w[x][1] = y.y;
          }
        }
        if (E4M3 && masked) {                          // codes that are no numbers, behind the end or in nodes that some rows do not see: 0 times
#pragma unroll                                           // them has to be 0
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int c = 0; c < VW; ++c) w[x][c] &= ~((((w[x][c] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7);
        }
        const TqFactor f0 = tq_factor<E4M3>(vb[0], vb[1]), f1 = tq_factor<E4M3>(vb[2], vb[3]);
        const int e0 = int((ev >> (8 * (DP == 128 ? g >> 1 : g >> 2))) & 0xFFu);
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {              // columns 2 j, 2 j + 1 of the thread's
          // two keys' codes of both columns, in the order that makes a pair of the keys' codes of one column
          const uint32_t sel = E4M3 ? (j & 1 ? 0x7362u : 0x5140u) : (j & 1 ? 0x7632u : 0x5410u);
          const uint32_t x0 = __byte_perm(w[0][j >> 1], w[1][j >> 1], sel), x1 = __byte_perm(w[2][j >> 1], w[3][j >> 1], sel);
          uint32_t v4[4];
          if (FAR) {
            tq_widen_far<E4M3>(x0, int(vb[0]) - e0, int(vb[1]) - e0, v4[0], v4[1]);
            tq_widen_far<E4M3>(x1, int(vb[2]) - e0, int(vb[3]) - e0, v4[2], v4[3]);
          } else {
            tq_widen<E4M3>(x0, f0, v4[0], v4[1]);
            tq_widen<E4M3>(x1, f1, v4[2], v4[3]);
          }
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) tq_mma<FAR>(o[nq][j], v4, pb[nq][0], pb[nq][1]);
        }
      };
      if (tame) slice(std::false_type{});
      else slice(std::true_type{});
      ++used;
      __syncwarp();                                    // every lane has read the slot
      if (valid) issue();
    }
    // ---- the piece's result: rows 2 t4, 2 t4 + 1 of each tile, columns DP / 8 g ..; weights at most 1 from here on ----
    const int rows = min(a.rpg, a.rows - m0), d0 = g * (DP / 8);
    const float unit = __uint_as_float(max(ev >> (8 * (DP == 128 ? g >> 1 : g >> 2)) & 0xFFu, 1u) << 23) * exp2f(-TQ_TOP);
    const bool whole = p.whole(), head = p.t1 == p.nt;
#pragma unroll
    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nq][e];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
        const int lr = 8 * nq + 2 * t4 + e, m = m0 + lr;
        if (lr >= rows || !ok) continue;
        const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
        const bool any = i < n && sum != 0.0f;         // also when the sum is not a number
        if (whole) {
          const float inv = any ? unit / (sum * exp2f(-TQ_TOP)) : 0.0f;
          const int64_t row = int64_t(p.r) * a.T + i;
          if (d0 < D) {
            __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.ldo + int64_t(h) * D + d0;
#pragma unroll
            for (int j = 0; j < STEPS; j += 4) {
              uint32_t y[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) y[c] = any ? tq_pack<true>(o[nq][j + c][e] * inv, o[nq][j + c][2 + e] * inv) : 0u;
              *reinterpret_cast<uint4*>(out + 2 * j) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
          if (g == 0 && a.lse) a.lse[row * a.Hq + h] = any ? (mref[nq][e] + log2f(sum)) * TA_LN2 : -INFINITY;
        } else {
          if (g == 0) s_ml[head ? 0 : 1][warp][lr] = any ? make_float2(mref[nq][e] + TQ_TOP, sum * exp2f(-TQ_TOP)) : make_float2(-INFINITY, 0.0f);
          // a head goes to the workspace, the tail into the ring, which is done with
          float* to = head ? a.warp_o + (int64_t(blockIdx.x * WARPS + warp) * a.rs + lr) * D + d0 : reinterpret_cast<float*>(ring) + lr * DP + d0;
          if (d0 < D) {
#pragma unroll
            for (int j = 0; j < STEPS; j += 2)
              *reinterpret_cast<float4*>(to + 2 * j) = make_float4(o[nq][j][e] * unit, o[nq][j][2 + e] * unit, o[nq][j + 1][e] * unit, o[nq][j + 1][2 + e] * unit);
          }
        }
      }
    __syncwarp();
    if (lane == 0) {
      if (!whole) {
        TqPart& part = head ? s_head[warp] : s_tail[warp];
        part.p = p;
        part.valid = 1;
      }
      more(kp + 2);                                    // the piece after the next, in place of the one before
    }
    __syncwarp();
    if (np == 0) nt = piece[(kp + 1) % 3].t0;
    np = max(np - 1, 0);
  }
  // copies in flight land before the block leaves its shared memory to another
  for (; used != issued; ++used) (void)ds_mbar_wait(&s_full[warp][used % NS], (used / NS) & 1u, DS_WAIT_LIMIT);
  __syncthreads();
  if (aborted()) return;
  // ---- items that several warps of this block share: tails of warps [w0, w1), then the head of warp wh (-1: it goes on behind the block) ----
  auto join = [&](int w0, int w1, int wh, const TaPiece& p, bool began) {
    const int32_t n = s_len.n[p.r];
    const int m0 = p.g * a.rpg, rows = min(a.rpg, a.rows - m0);
    const bool whole = began && wh >= 0;
    const int64_t slot = 2 * int64_t(blockIdx.x) + (began ? 1 : 0);
    for (int u = tid; u < rows * (D / 4); u += L::THREADS) {
      const int lr = u / (D / 4), d = (u - lr * (D / 4)) * 4, m = m0 + lr;
      float M = -INFINITY, sum = 0.0f;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int k = w0; k < w1; ++k)
        if (s_tail[k].valid) M = fmaxf(M, s_ml[1][k][lr].x);
      if (wh >= 0) M = fmaxf(M, s_ml[0][wh][lr].x);
      auto add = [&](const float2& ml, const float4& z) {
        const float f = ml.y == 0.0f ? 0.0f : ta_ex2(ml.x - M);
        sum = __fmaf_rn(f, ml.y, sum);
        if (ml.y == 0.0f) return;
        y.x = __fmaf_rn(f, z.x, y.x);
        y.y = __fmaf_rn(f, z.y, y.y);
        y.z = __fmaf_rn(f, z.z, y.z);
        y.w = __fmaf_rn(f, z.w, y.w);
      };
      for (int k = w0; k < w1; ++k)
        if (s_tail[k].valid) add(s_ml[1][k][lr], *reinterpret_cast<const float4*>(smem + k * L::RING + (lr * DP + d) * 4));
      if (wh >= 0) add(s_ml[0][wh][lr], __ldcg(reinterpret_cast<const float4*>(a.warp_o + (int64_t(blockIdx.x * WARPS + wh) * a.rs + lr) * D + d)));
      const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
      const int64_t row = int64_t(p.r) * a.T + i;
      const bool any = i < n && sum != 0.0f;
      if (whole) {
        const float inv = any ? 1.0f / sum : 0.0f;
        uint2 z;
        z.x = any ? tq_pack<true>(y.x * inv, y.y * inv) : 0u;
        z.y = any ? tq_pack<true>(y.z * inv, y.w * inv) : 0u;
        *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.ldo + int64_t(h) * D + d) = z;
        if (d == 0 && a.lse) a.lse[row * a.Hq + h] = any ? (M + log2f(sum)) * TA_LN2 : -INFINITY;
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * a.rs + lr) * D + d) = y;
        if (d == 0) a.part_ml[slot * a.rs + lr] = any ? make_float4(M, sum, sum, 0.0f) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      }
    }
  };
  int open = -1;                                       // first warp of an item that has not ended yet
  for (int w = 0; w < WARPS; ++w) {
    if (s_head[w].valid) {
      if (open < 0) join(w, w, w, s_head[w].p, false);
      else join(open, w, w, s_tail[open].p, s_tail[open].p.t0 == 0);
      open = -1;
    }
    if (s_tail[w].valid && open < 0) open = w;
  }
  if (open >= 0) join(open, WARPS, -1, s_tail[open].p, s_tail[open].p.t0 == 0);
}

template <int DP, int NQ, bool CAP, bool E4M3>
cudaError_t tq_launch(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  constexpr size_t smem = TqLayout<DP, NQ>::TOTAL + 1024;
  const cudaError_t e = ds_ensure_smem(reinterpret_cast<const void*>(tree_attn_q8_rows_kernel<DP, NQ, CAP, E4M3>), smem);
  if (e != cudaSuccess) return e;
  return ds_launch(tree_attn_q8_rows_kernel<DP, NQ, CAP, E4M3>, dim3(unsigned(grid)), dim3(TqLayout<DP, NQ>::THREADS), smem, st, a, k, v);
}

template <int DP, int NQ>
cudaError_t tq_dispatch(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (a.q8.e4m3) return a.softcap > 0.0f ? tq_launch<DP, NQ, true, true>(a, grid, k, v, st) : tq_launch<DP, NQ, false, true>(a, grid, k, v, st);
  return a.softcap > 0.0f ? tq_launch<DP, NQ, true, false>(a, grid, k, v, st) : tq_launch<DP, NQ, false, false>(a, grid, k, v, st);
}

}  // namespace

cudaError_t ta_launch_q8_rows(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (a.c.head_dim <= 64) {
    if (a.rpg <= 8) return tq_dispatch<64, 1>(a, grid, k, v, st);
    return a.rpg <= 16 ? tq_dispatch<64, 2>(a, grid, k, v, st) : tq_dispatch<64, 4>(a, grid, k, v, st);
  }
  if (a.rpg <= 8) return tq_dispatch<128, 1>(a, grid, k, v, st);
  return a.rpg <= 16 ? tq_dispatch<128, 2>(a, grid, k, v, st) : tq_dispatch<128, 4>(a, grid, k, v, st);
}
