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
// powers lie further apart, blocks of zeros aside, takes bf16 forms with the full range instead. Queries go to f16 under a power of two of each row, the
// largest to 2^13 .. 2^14: each column is off by at most 2^-25, 2^-38 of the largest. Weights are rounded to f16 relative to a reference at which the
// row's largest is 2^7 to 2^15: by at most 2^-11 of a weight down to f16's least normal number (2^-21 to 2^-29 of the largest), below it by at most 2^-25,
// which is 2^-32 of the largest or less (in the bf16 forms by 2^-8 of a weight). The sum that the result is divided by is of the unrounded weights.
//
// Every warp copies its own slices with TMA, NS of them in flight, and waits for nothing but its own barriers. The work is the line of
// tiles of tree_attn.cuh with 16 keys a tile: a block's share is cut once more into its warps' shares; what two warps leave of an item is joined
// at the end in shared memory (in the order of the keys), and what two blocks leave by the join kernel.
//
// Bound by HBM (2 (D + D / 32) bytes a key and key head) for 4 rows a key head, by the latency of a warp's chain of scores, weights and
// products for more (with 17 to 32 rows 255 registers a thread leave 8 warps an SM). Measured with the join, 300-8,200 keys, heads of 128, 8 of them:
//   64 requests of one token x 4 heads    126 us   4.6 TB/s, 0.68 of the measured copy rate (with a bf16 cache 188 us)
//   32 requests of 4 nodes x 4 heads      105 us
//   32 requests of 8 nodes x 4 heads      187 us   (with a bf16 cache 114 us, whose kernel reads tiles as they lie)
//   one token x 4 heads, 5,001 keys      17.6 us   with the host's call: two slices a warp, then the joins
#include <cuda_fp16.h>

#include <type_traits>

#include "cache_q8.cuh"
#include "tree_attn.cuh"

namespace {

constexpr int TQ_KEYS = 16;                  // keys of a slice
constexpr float TQ_TOP = 15.0f;              // weights reach 2^15;
constexpr float TQ_AT = 7.0f;                // a new reference gives the largest score a weight of 2^7
constexpr float TQ_NONE = -3e38f;            // reference of a row that has seen nothing
constexpr uint32_t TQ_FAR = 170;             // largest scale byte that O is relative to: 2^15 * 448 * 2^(245 - 170) times 2^28 keys is a float32
                                             // number, and values whose byte is 53 or more are exact bf16 numbers relative to it

template <int DP, int NQ>
struct TqLayout {
  // 12 warps of 168 registers, or 8 of 255 where four tiles need them. (One tile with 8 or with 16 warps of fewer registers was slower.)
  static constexpr int WARPS = NQ <= 2 ? 12 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int NS = NQ == 1 ? 3 : NQ == 2 ? 2 : 4;
  static constexpr bool QREG = NQ == 1;                // queries stay in registers
  static constexpr int STEPS = DP / 16;                // contraction steps of K Q^T; row tiles of O^T
  static constexpr uint32_t SLICE = 2 * TQ_KEYS * DP;  // bytes of a slice's keys and values
  // dynamic shared memory: rings of slices (where a warp's last partial result goes when they are done with), scale words, queries
  static constexpr uint32_t RING = NS * SLICE;
  static constexpr uint32_t SCALE = WARPS * RING;      // [WARPS][NS][32] words: scale bytes of 16 keys, then of 16 values
  static constexpr uint32_t QF = SCALE + WARPS * NS * 128;
  static constexpr uint32_t QW = QREG ? 0 : NQ * STEPS * 256;   // bytes of a warp's queries
  static constexpr uint32_t TOTAL = QF + WARPS * QW;
  static_assert(8 * NQ * DP * 4 <= RING, "a partial result fits its warp's ring");
};

// A box of keys and the same of values, V bytes behind, by one elected lane of a warp that stays together; BYTES > 0: the arrival that
// the barrier's phase waits for, with that many bytes to come.
template <uint32_t V, uint32_t BYTES>
DS_DEV void tq_tma_pair(uint32_t dst, const void* tk, const void* tv, int32_t t, int32_t h, int32_t p, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e, f;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "setp.ne.and.u32 f, %8, 0, e;\n\t"
      "@f mbarrier.arrive.expect_tx.shared::cta.b64 _, [%6], %8;\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%7, %3, %4, %5}], [%6];\n\t"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%9], [%2, {%7, %3, %4, %5}], [%6];\n\t}" ::"r"(dst),
      "l"(tk), "l"(tv), "r"(t), "r"(h), "r"(p), "r"(bar), "r"(0), "n"(BYTES), "r"(dst + V)
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
    uint32_t x, y;                                     // (one instruction each, which the compiler makes two of)
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(x) : "r"(w), "r"(0x00FF00FFu), "r"(0x64806480u));
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(w >> 8), "r"(0x00FF00FFu), "r"(0x64806480u));
    first = tq_fma2h(x, f.f, f.c);
    second = tq_fma2h(y, f.f, f.c);
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

// Of the line of tiles a block has one share, cut once more into its warps' shares. Of an item's nt tiles the block has [a0, a1) and the warp [t0, t1).
struct TqPiece {
  int32_t r, hk, g;            // request, key head, row group
  int32_t a0, a1, nt, t0, t1;
  DS_DEV bool all() const { return a0 == 0 && a1 == nt; }
  DS_DEV int64_t slot() const { return 2 * int64_t(blockIdx.x) + (a0 > 0 ? 0 : 1); }
};

// Walks a warp's share [at, end) of the line.
struct TqWalk {
  int64_t at, end;
  int32_t r;
  DS_DEV bool find(const TaLens& s, const TaArgs& a, TqPiece& p) {
    if (at >= end) return false;
    const int64_t hm = int64_t(a.c.heads) * a.mg;
    while (s.pref[r + 1] * hm <= at) ++r;
    const int64_t off = at - s.pref[r] * hm;
    const int32_t nt = s.pref[r + 1] - s.pref[r], item = int32_t(ta_div(off, uint32_t(nt)));
    p.r = r;
    p.nt = nt;
    p.hk = int32_t(uint32_t(item) / uint32_t(a.mg));
    p.g = item - p.hk * a.mg;
    p.t0 = int32_t(off - int64_t(item) * nt);
    p.t1 = int32_t(min(int64_t(nt), p.t0 + (end - at)));
    const int64_t i0 = at - p.t0;                      // the item's place on the line
    p.a0 = int32_t(max(s.at - i0, int64_t(0)));
    p.a1 = int32_t(min(int64_t(nt), s.end - i0));
    at += p.t1 - p.t0;
    return true;
  }
};

// A warp's part of an item that it shares with others.
struct TqPart {
  TqPiece p;
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
  __shared__ TqWalk s_walk[WARPS];
  __shared__ TqPiece s_piece[WARPS][3];
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
  const bool narrow = D < DP;                          // some columns are not there
  const bool words = nb == 4 && a.q8.vec4 != 0;        // a slot's scales are one aligned word
  const TqPiece* piece = s_piece[warp];
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
    TqWalk w;
    w.at = s_len.at + ta_div(share * warp, WARPS);
    w.end = s_len.at + ta_div(share * (warp + 1), WARPS);
    w.r = s_len.r;
    s_walk[warp] = w;
    more(0);
    s_there[warp][1] = 0;
  }
  __syncwarp();
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };

  // ---- this warp's slices: the next one to copy, its page known beforehand ----
  int kp = 0;                                          // piece that is worked on
  int np = -1, nt = 0, nt1 = 0;                        // piece (0: that one, 1: the one after it), tile and last tile of the next copy
  bool valid = false;
  const uint32_t psize = uint32_t(a.c.page_size);
  uint32_t key = 0, len = 0, entry = 0, place = 0;     // this lane's key of that slice (lane & 15), the request's keys, the key's page and place
  int32_t pg = -1, next = -1, hk = 0;                  // that page (-1: no key) and the one after it
  const int32_t* table = nullptr;
  const uint8_t* sbase = nullptr;                      // scales of the piece's head: keys' for lanes below 16, else values'
  uint32_t issued = 0, used = 0, pend = 0;
  int pend_at = -1;
  auto advance = [&]() {                               // finds the first slice of the next piece that has one
    valid = false;
    while (np < 1 && there[(kp + np + 1) % 3]) {
      ++np;
      const TqPiece& p = piece[(kp + np) % 3];
      nt = p.t0;
      nt1 = p.t1;
      hk = p.hk;
      key = uint32_t(nt) * TQ_KEYS + (lane & 15);
      len = uint32_t(s_len.ctx[p.r]) + uint32_t(s_len.n[p.r]);
      entry = key / psize;
      place = key - entry * psize;
      table = a.c.page_table + int64_t(p.r) * a.c.ld_table;
      sbase = (lane < 16 ? a.q8.k_scale : a.q8.v_scale) + int64_t(hk) * a.q8.head_stride;
      pg = key < len ? table[entry] : -1;              // looked at when the slice is copied
      next = key - place + psize < len ? table[entry + 1] : -1;
      valid = true;
      return;
    }
  };
  auto flush = [&]() {                                 // the scales asked for last have arrived; no key: 0
    if (pend_at >= 0) scales[pend_at * 32 + lane] = pend;
    pend_at = -1;
  };
  auto issue = [&]() {
    flush();
    const int32_t seen = pg;
    const bool there_ = key < len && uint32_t(pg) < uint32_t(a.c.num_pages);
    if (key < len && !there_) ds_set_error(a.status, DSPARK_ERANGE);
    const int s = int(issued % NS);
    // boxes of 16 or 8 places, keys' and values', by one lane; past the end, or from a page that does not exist, a box names a page past
    // the last and reads zeros
    const int32_t none = int32_t(a.c.num_pages), mine = there_ ? pg : none;
    const uint32_t bar = ds_smem_addr(&s_full[warp][s]), dst = ds_smem_addr(ring + s * L::SLICE);
    tq_tma_pair<16 * DP, L::SLICE>(dst, &tmK, &tmV, __shfl_sync(0xFFFFFFFFu, int32_t(place), 0), hk, __shfl_sync(0xFFFFFFFFu, mine, 0), bar);
    if (a.box == 8)
      tq_tma_pair<16 * DP, 0>(dst + 8 * DP, &tmK, &tmV, __shfl_sync(0xFFFFFFFFu, int32_t(place), 8), hk, __shfl_sync(0xFFFFFFFFu, mine, 8), bar);
    // scale bytes (strides of scales are below 2^31 here); none: 0
    const uint8_t* at = sbase + uint64_t(uint32_t(there_ ? pg : 0)) * uint32_t(a.q8.page_stride) + uint64_t(place) * uint32_t(a.q8.token_stride);
    if (words) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n\tcp.async.commit_group;" ::"r"(ds_smem_addr(scales + s * 32 + lane)), "l"(at),
                   "r"(there_ ? 4 : 0)
                   : "memory");
    } else {
      pend = 0;
      for (int b = 0; b < nb; ++b)
        if (there_) pend |= uint32_t(at[b]) << (8 * b);
      pend_at = s;
    }
    ++issued;
    if (++nt < nt1) {
      key += TQ_KEYS;
      place += TQ_KEYS;
      pg = seen;
      if (place >= psize) {                            // pages of 8 or more places: one or two further
        do {
          place -= psize;
          ++entry;
          pg = next;
          next = key - place + psize < len ? table[entry + 1] : -1;
        } while (place >= psize);
      }
    } else {
      advance();
    }
  };
  advance();
  const float sc = CAP ? fminf(a.scale * 2.0f * TA_LOG2E / a.softcap, 3e38f) : a.scale * TA_LOG2E;
  const float cap2 = a.softcap * TA_LOG2E, sy = CAP ? a.scale / a.softcap : 0.0f;
  bool ok = true, first = true;
  for (; there[kp % 3]; ++kp) {
    const TqPiece p = piece[kp % 3];
    const int32_t ctx = s_len.ctx[p.r], n = s_len.n[p.r];
    const int m0 = p.g * a.rpg, tmask = ctx / TQ_KEYS;   // tiles from tmask on hold nodes or the end of the keys
    if (ok) {
      while (issued - used < NS) {
        if (!valid) advance();
        if (!valid) break;
        issue();
      }
    }
    if (kp == 0) {                                     // the second piece, now that the first's copies are on their way
      if (lane == 0) more(1);
      __syncwarp();
      while (ok && issued - used < NS) {
        if (!valid) advance();
        if (!valid) break;
        issue();
      }
    }
    // ---- query rows (n index g of each tile) in the order of the operand registers, in f16 under 2^qe of the row ----
    const __nv_bfloat16* qrow[NQ];
    uint2 qreg[L::QREG ? STEPS : 1];
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
        (L::QREG ? qreg[L::QREG ? st : 0] : qf[(nq * STEPS + st) * 32]) = E4M3 ? make_uint2(tq_pack<false>(v[0], v[1]), tq_pack<false>(v[2], v[3]))
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
    // references: scale bytes of the thread's block of values and of keys; `near`: there are some, and no byte in their reach is one that is
    // read as another
    uint32_t ev = 0, ek = 0;
    bool near = false;
    for (int t = p.t0; ok && t < p.t1; ++t) {
      const int s = int(used % NS);
      flush();
      ok = ds_mbar_wait_or_abort(&s_full[warp][s], (used / NS) & 1u, first ? a.first_wait : DS_WAIT_LIMIT, &s_abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      first = false;
      if (words) {                                     // a slot's scales: all but the newest NS - 1 copies
        if (issued - used == NS) asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      if (!ok) {
        if (!aborted()) ds_set_error(a.status, DSPARK_ETIMEOUT);
        s_abort = 1;
        break;
      }
      const uint8_t *K = ring + s * L::SLICE, *V = K + TQ_KEYS * DP;
      const uint8_t *ks = reinterpret_cast<const uint8_t*>(scales + s * 32), *vs = ks + 64;
      const bool masked = t >= tmask;
      __syncwarp();                                    // every lane's words are there
      // ---- this slice's powers relative to the references, as exponents of f16: a thread's two keys (of its columns' block), four values ----
      uint32_t kb[2], vb[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) kb[x] = ks[(8 * x + g) * 4 + (DP == 128 ? t4 : t4 >> 1)];
#pragma unroll
      for (int x = 0; x < 4; ++x) vb[x] = vs[(2 * t4 + (x & 1) + 8 * (x >> 1)) * 4 + (DP == 128 ? g >> 1 : g >> 2)];
      uint32_t gone = 0;                               // bits 0, 1: keys, 2..5: values that are not there (columns past head_dim, keys past the end)
      if (narrow) gone = (t4 * (DP / 4) >= D ? 3u : 0u) | (g * (DP / 8) >= D ? 60u : 0u);
      if (masked) {
        const int left = int(min(int64_t(ctx) + n - int64_t(t) * TQ_KEYS, int64_t(TQ_KEYS)));
        gone |= (g >= left ? 1u : 0u) | (8 + g >= left ? 2u : 0u) | (2 * t4 >= left ? 4u : 0u) | (2 * t4 + 1 >= left ? 8u : 0u) |
                (2 * t4 + 8 >= left ? 16u : 0u) | (2 * t4 + 9 >= left ? 32u : 0u);
      }
      uint32_t kr[2], vr[4];                           // 1..HI: code times power is exact in f16
      auto relative = [&]() {
        uint32_t most = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          kr[x] = kb[x] + 15u - ek;
          if (gone) kr[x] = (gone >> x) & 1u ? 15u : kr[x];
          most = max(most, kr[x] - 1u);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          vr[x] = vb[x] + 15u - ev;
          if (gone) vr[x] = (gone >> (2 + x)) & 1u ? 15u : vr[x];
          most = max(most, vr[x] - 1u);
        }
        return most < HI;
      };
      bool tame = __all_sync(0xFFFFFFFFu, relative() && near);
      if (!tame) {
        // New references: the slice's largest key byte; of each block of values (a thread's) the largest so far, which O changes to.
        uint32_t mk = 0, mv = 0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          kb[x] = (gone >> x) & 1u ? 1u : q8_byte(kb[x]);
          mk = max(mk, kb[x]);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          vb[x] = (gone >> (2 + x)) & 1u ? 1u : q8_byte(vb[x]);
          mv = max(mv, vb[x]);
        }
        ek = __reduce_max_sync(0xFFFFFFFFu, mk);
#pragma unroll
        for (int x = 1; x < (DP == 128 ? 8 : 16); x <<= 1) mv = max(mv, __shfl_xor_sync(0xFFFFFFFFu, mv, x));   // the lanes of a block: all four t4, two or four g
        // (No reference lies above TQ_FAR: rows that do not see the largest values keep theirs. Larger ones take the bf16 forms.)
        mv = min(mv, TQ_FAR);
        if (ev == 0u || mv > ev + HI - 15u) {
          const int down = int(ev) - int(mv);          // 2^down, in two steps where it is small
          const float f = __uint_as_float(uint32_t(max(down, -126) + 127) << 23), f2 = __uint_as_float(uint32_t(max(down + 126, -126) + 127) << 23);
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < STEPS; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[nq][j][e] = down < -126 ? o[nq][j][e] * f * f2 : o[nq][j][e] * f;
          ev = mv;
        }
        // references at which no byte in reach of one is read as another
        near = ek >= 16u && ek <= 230u && ((narrow && g * (DP / 8) >= D) || (ev >= 16u && ev <= 230u));
        // A block of zeros, which is written under the least power, has code 0 under any: out of the references' reach it counts as one that is not there
        // instead of sending the slice to the bf16 forms, whose weights have three bits less. (With one in every slice 64 single tokens take 151 us, in
        // those forms 185 us, 32 requests of 8 nodes 206 and 298 us; with none 126 and 187 us.)
        const bool far_k = ek > 15u, far_v = ev > 15u;
        constexpr uint32_t DIGITS = E4M3 ? 0x7F7F7F7Fu : 0xFFFFFFFFu;      // (minus zero)
        if (__any_sync(0xFFFFFFFFu, far_k && min(kb[0], kb[1]) == 1u)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint8_t* row = K + (8 * x + g) * DP;
            uint4 y = *reinterpret_cast<const uint4*>(row + (DP == 128 ? (2 * t4) ^ g : t4 ^ (g >> 1)) * 16);
            uint32_t any = y.x | y.y | y.z | y.w;
            if (DP == 128) {
              y = *reinterpret_cast<const uint4*>(row + ((2 * t4 + 1) ^ g) * 16);
              any |= y.x | y.y | y.z | y.w;
            }
            if (far_k && kb[x] == 1u && (any & DIGITS) == 0u) gone |= 1u << x;
          }
        }
        if (__any_sync(0xFFFFFFFFu, far_v && min(min(vb[0], vb[1]), min(vb[2], vb[3])) == 1u)) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = 2 * t4 + (x & 1) + 8 * (x >> 1);
            uint32_t any;
            if constexpr (DP == 128) {
              const uint4 y = *reinterpret_cast<const uint4*>(V + key * DP + ((g ^ (key & 7)) << 4));
              any = y.x | y.y | y.z | y.w;
            } else {
              const uint2 y = *reinterpret_cast<const uint2*>(V + key * DP + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
              any = y.x | y.y;
            }
            if (far_v && vb[x] == 1u && (any & DIGITS) == 0u) gone |= 4u << x;
          }
        }
        tame = __all_sync(0xFFFFFFFFu, relative());    // with the bytes cut to their range
      }
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
          const TqFactor f[2] = {tq_factor<E4M3>(kr[0], kr[0]), tq_factor<E4M3>(kr[1], kr[1])};
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
              uint2 q = L::QREG ? qreg[L::QREG ? st : 0] : qf[(nq * STEPS + st) * 32];
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
        const float kfac = FAR ? 1.0f : __uint_as_float(ek << 23);
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
              const uint32_t bits = ta_mask32(a, p.r, i, n, int64_t(t) * TQ_KEYS - ctx) >> g;
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
        const TqFactor f0 = tq_factor<E4M3>(vr[0], vr[1]), f1 = tq_factor<E4M3>(vr[2], vr[3]);
        const int e0 = int(ev);
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
    const float unit = __uint_as_float(max(ev, 1u) << 23) * exp2f(-TQ_TOP);
    const bool alone = p.t0 == p.a0 && p.t1 == p.a1, whole = alone && p.all(), head = p.t1 == p.a1;   // no other warp of the block; no other block
    const int64_t slot = p.slot();
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
          const float2 ml = any ? make_float2(mref[nq][e] + TQ_TOP, sum * exp2f(-TQ_TOP)) : make_float2(-INFINITY, 0.0f);
          if (g == 0) {
            if (alone) a.part_ml[slot * a.rs + lr] = make_float4(ml.x, ml.y, ml.y, 0.0f);
            else s_ml[head ? 0 : 1][warp][lr] = ml;
          }
          // the block's part to its slot, a head to the workspace, the tail into the ring, which is done with
          float* to = alone ? a.part_o + (slot * a.rs + lr) * D + d0
                    : head  ? a.warp_o + (int64_t(blockIdx.x * WARPS + warp) * a.rs + lr) * D + d0
                            : reinterpret_cast<float*>(ring) + lr * DP + d0;
          if (d0 < D) {
#pragma unroll
            for (int j = 0; j < STEPS; j += 2)
              *reinterpret_cast<float4*>(to + 2 * j) = make_float4(o[nq][j][e] * unit, o[nq][j][2 + e] * unit, o[nq][j + 1][e] * unit, o[nq][j + 1][2 + e] * unit);
          }
        }
      }
    __syncwarp();
    if (lane == 0) {
      if (!alone) {
        TqPart& part = head ? s_head[warp] : s_tail[warp];
        part.p = p;
        part.valid = 1;
      }
      more(kp + 2);                                    // the piece after the next, in place of the one before
    }
    __syncwarp();
    --np;                                              // (valid: the slice to copy next is of the piece that follows)
  }
  // copies in flight land before the block leaves its shared memory to another
  for (; used != issued; ++used) (void)ds_mbar_wait(&s_full[warp][used % NS], (used / NS) & 1u, DS_WAIT_LIMIT);
  __syncthreads();
  if (aborted()) return;
  // ---- items that several warps of this block share: the end (head) that warp w1 holds and the parts before it (tails of warps from w0 on) ----
  int heads = 0;
  for (int w = 0; w < WARPS; ++w) heads += s_head[w].valid;
  const int per = min(a.rpg, a.rows) * (DP / 4);
#pragma unroll 1
  for (int u = tid; u < heads * per; u += L::THREADS) {
    int q = u / per, w1 = 0;
    const int lr = (u - q * per) / (DP / 4), d = (u % (DP / 4)) * 4;
    for (;; ++w1)
      if (s_head[w1].valid && q-- == 0) break;
    const TqPiece& p = s_head[w1].p;
    const int m = p.g * a.rpg + lr;
    if (m >= a.rows || d >= D) continue;
    const float4 own = __ldcg(reinterpret_cast<const float4*>(a.warp_o + (int64_t(blockIdx.x * WARPS + w1) * a.rs + lr) * D + d));
    int w0 = w1;
    float M = s_ml[0][w1][lr].x, sum = 0.0f;
    while (w0 > 0) {
      --w0;
      if (!s_tail[w0].valid) continue;
      M = fmaxf(M, s_ml[1][w0][lr].x);
      if (s_tail[w0].p.t0 == s_tail[w0].p.a0) break;
    }
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float2& ml, const float4& z) {
      if (ml.y == 0.0f) return;
      const float f = ta_ex2(ml.x - M);
      sum = __fmaf_rn(f, ml.y, sum);
      y.x = __fmaf_rn(f, z.x, y.x);
      y.y = __fmaf_rn(f, z.y, y.y);
      y.z = __fmaf_rn(f, z.z, y.z);
      y.w = __fmaf_rn(f, z.w, y.w);
    };
    for (int k = w0; k < w1; ++k)
      if (s_tail[k].valid) add(s_ml[1][k][lr], *reinterpret_cast<const float4*>(smem + k * L::RING + (lr * DP + d) * 4));
    add(s_ml[0][w1][lr], own);
    const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
    const int64_t row = int64_t(p.r) * a.T + i, slot = p.slot();
    const bool any = i < s_len.n[p.r] && sum != 0.0f;
    if (p.all()) {
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
