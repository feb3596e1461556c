// tree_attn_q8_rows.cu - attention over a cache in 8 bits for few query rows a key head (dspark_tree_attention_q8): single new
// tokens and short drafted blocks.
//
// openvino.genai PR #4847, Fixes > Split validation windows, and optimum-intel PR #2098 (paged attention targets).
//
// The rows that read one key head (at most 32) make one or two 16-row tiles of mma.sync; a warp takes 16 keys at a time:
//   S[16 rows, 16 keys] = Q K^T,  P = 2^(x - m) in bf16,  O[16 rows, D] += P V
// with its own running reference m, sum and O, so warps need nothing from each other until a piece ends. A contraction may take its index in
// any order, so a thread's operand registers are filled from 16 contiguous codes of one key (K: columns 32 t .. of the thread's t in its
// quad; V: columns 16 g .. of its group g): codes go from shared memory into registers once, become bf16 there (exactly: code times power of
// two) and are used where they are. Nothing is staged in 16 bits, which tcgen05 would need: its operands come from shared memory, and 2 D
// bytes written and read again a key cost more shared-memory time than HBM needs for the codes.
//
// Every warp copies its own slices of 16 keys with TMA, NS of them in flight, and waits for nothing but its own barriers. The work is the line
// of tiles of tree_attn.cuh with 16 keys a tile.
#include <type_traits>

#include "cache_q8.cuh"
#include "tree_attn.cuh"

namespace {

constexpr int TQ_KEYS = 16;                  // keys of a slice
constexpr float TQ_ABOVE = 8.0f;             // a new reference lies this far (log2) above the maximum

template <int DP, int MT>
struct TqLayout {
  static constexpr int WARPS = MT == 1 ? 16 : 8;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int NS = MT == 1 ? 2 : 4;
  static constexpr int STEPS = DP / 16;                // contraction steps of Q K^T, and columns of a result lane pair
  static constexpr uint32_t SLICE = 2 * TQ_KEYS * DP;  // bytes of a slice's keys and values
  static constexpr int RB = MT == 1 ? 4 : 8;           // rows joined at a time
  static constexpr uint32_t RING = WARPS * NS * SLICE; // then:
  static constexpr uint32_t SCALE = RING;              // [WARPS][NS][32] words: scale bytes of 16 keys, then of 16 values
  static constexpr uint32_t QF = SCALE + WARPS * NS * 128;
  static constexpr uint32_t JOIN = QF + MT * STEPS * 512;
  static constexpr uint32_t TOTAL = JOIN + WARPS * RB * DP * 4;
};

DS_DEV void tq_tma_load(uint32_t dst, const void* tmap, int32_t d, int32_t t, int32_t h, int32_t p, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst), "l"(tmap), "r"(d), "r"(t), "r"(h), "r"(p), "r"(bar)
      : "memory");
}

// D (+)= A B, 16 x 8 x 16, bf16 with float32 sums.
DS_DEV void tq_mma(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
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
DS_DEV uint32_t tq_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The powers of two by which codes, put into bf16 fields as below, become numbers; as bf16 bits. E4M3's fields are the number times 2^-120,
// so its factor is 2^(120 + e), which above byte 134 (numbers from 2^16 on) takes two factors.
template <bool E4M3>
DS_DEV uint32_t tq_factor(uint32_t byte) {
  const uint32_t b = q8_byte(byte);
  return (E4M3 ? min(b + 120u, 254u) : b) << 7;
}
DS_DEV uint32_t tq_factor_above(uint32_t byte) { return (127u + max(int(q8_byte(byte)) - 134, 0)) << 7; }

// Bytes 0 and 2 of w, and bytes 1 and 3, as pairs of bf16 numbers times their factors. E4M3: sign to bit 15, the seven bits below it to
// bits 10..4 (low exponent bits and high fraction bits). INT8: 128 + (low seven bits) - 128 (1 + sign).
template <bool E4M3, bool BIG>
DS_DEV void tq_widen(uint32_t w, uint32_t f, uint32_t f2, uint32_t& even, uint32_t& odd) {
  if (E4M3) {
    even = ((w << 8) & 0x80008000u) | ((w << 4) & 0x07F007F0u);
    odd = (w & 0x80008000u) | ((w >> 4) & 0x07F007F0u);
    even = tq_mul2(even, f);
    odd = tq_mul2(odd, f);
    if (BIG) {
      even = tq_mul2(even, f2);
      odd = tq_mul2(odd, f2);
    }
  } else {
    const uint32_t v = w >> 8;
    even = tq_mul2(tq_sub2((w & 0x007F007Fu) | 0x43004300u, (w & 0x00800080u) | 0x43004300u), f);
    odd = tq_mul2(tq_sub2((v & 0x007F007Fu) | 0x43004300u, (v & 0x00800080u) | 0x43004300u), f);
  }
}

template <int DP, int MT, bool CAP, bool E4M3>
__global__ void __launch_bounds__(TqLayout<DP, MT>::THREADS, 1)
tree_attn_q8_rows_kernel(const TaArgs a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using L = TqLayout<DP, MT>;
  constexpr int NS = L::NS, STEPS = L::STEPS, WORDS = DP / 16, WARPS = L::WARPS;   // WORDS of codes a thread has of a key (K)
  constexpr int NT = DP / 8;                           // 8-column tiles of the result
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t s_full[WARPS][NS];
  __shared__ TaLens s_len;
  __shared__ TaWalk s_walk;
  __shared__ TaPiece s_piece[3];
  __shared__ int s_there[3];                           // whether the piece is one
  __shared__ int s_abort;
  __shared__ float4 s_ml[WARPS][16 * MT];              // (reference, sum, sum the result is divided by) of each warp
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + warp * NS * L::SLICE;
  uint32_t* scales = reinterpret_cast<uint32_t*>(smem + L::SCALE) + warp * NS * 32;
  const uint4* qf = reinterpret_cast<const uint4*>(smem + L::QF) + lane;
  float* join = reinterpret_cast<float*>(smem + L::JOIN);
  const int D = a.c.head_dim, nb = q8_blocks(D);
  const bool words = nb == 4 && a.q8.vec4 != 0;        // a slot's scales are one aligned word
  ds_pdl_trigger();
  if (lane == 0) {
    for (int s = 0; s < NS; ++s) ds_mbar_init(&s_full[warp][s], 1);
    ds_fence_mbar_init_cluster();
  }
  if (tid == 0) {
    s_abort = 0;
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmK) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tmV) : "memory");
  }
  ds_pdl_wait();
  ta_prefix(a, s_len);                                 // synchronises the block
  auto more = [&](int k) {                             // thread 0: finds piece number k
    s_there[k % 3] = s_walk.next(s_len, a, s_piece[k % 3]);
  };
  if (tid == 0) {
    s_walk.init(s_len);
    more(0);
    more(1);
  }
  __syncthreads();
  auto aborted = [&]() { return *reinterpret_cast<volatile int*>(&s_abort) != 0; };

  // ---- this warp's slices: the next one to copy, its page known beforehand ----
  int kp = 0;                                          // piece that is worked on
  int np = 0, nt = s_piece[0].t0 + warp;               // piece (0: that one, 1: the one after it) and tile of the next copy
  bool valid = false;
  int32_t pg = 0, place = 0;                           // page and place of this lane's key of that slice (lane & 15); pg < 0: no key
  uint32_t issued = 0, used = 0, pend = 0;
  int pend_at = -1;
  auto advance = [&]() {                               // finds the next slice and asks for its page
    valid = false;
    for (;; ++np, nt = s_piece[(kp + 1) % 3].t0 + warp) {
      if (np > 1 || !s_there[(kp + np) % 3]) return;
      if (nt < s_piece[(kp + np) % 3].t1) break;
      if (np == 1) return;
    }
    const TaPiece& p = s_piece[(kp + np) % 3];
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
  auto flush = [&]() {                                 // the scales asked for last have arrived
    if (pend_at >= 0) scales[pend_at * 32 + lane] = pend;
    pend_at = -1;
  };
  auto issue = [&]() {
    flush();
    const TaPiece& p = s_piece[(kp + np) % 3];
    const int s = int(issued % NS);
    const uint32_t bar = ds_smem_addr(&s_full[warp][s]), dst = ds_smem_addr(ring + s * L::SLICE);
    if (lane == 0) ds_mbar_arrive_expect_tx(&s_full[warp][s], L::SLICE);
    __syncwarp();
    // boxes of 16 or 8 places: the lane of a box's first key (lanes 16 and above: its values) copies it; past the end, or from a page that
    // does not exist, a box names a page past the last and reads zeros
    if ((lane & (a.box - 1)) == 0)
      tq_tma_load(dst + (lane & 16) * DP + (lane & 8) * DP, lane < 16 ? &tmK : &tmV, 0, place, p.hk, pg < 0 ? int32_t(a.c.num_pages) : pg, bar);
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
    nt += WARPS;
    advance();
  };
  advance();
  const float sc = CAP ? fminf(a.scale * 2.0f * TA_LOG2E / a.softcap, 3e38f) : a.scale * TA_LOG2E;
  const float cap2 = a.softcap * TA_LOG2E, sy = CAP ? a.scale / a.softcap : 0.0f;
  bool ok = true, first = true;
  for (; s_there[kp % 3]; ++kp) {
    const TaPiece p = s_piece[kp % 3];
    const int32_t ctx = s_len.ctx[p.r], n = s_len.n[p.r];
    const int m0 = p.g * a.rpg;
    // ---- query rows in the order of the first product's operand registers ----
    for (int u = tid; u < MT * STEPS * 32; u += L::THREADS) {
      const int l = u & 31, st = (u >> 5) % STEPS, mt = (u >> 5) / STEPS;
      const int d = (l & 3) * (DP / 4) + 4 * st, row = m0 + mt * 16 + (l >> 2);
      uint2 x[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = row + 8 * e, i = m / a.G, h = m - i * a.G;
        x[e] = make_uint2(0u, 0u);
        if (m < a.rows && d < D)
          x[e] = *reinterpret_cast<const uint2*>(reinterpret_cast<const __nv_bfloat16*>(a.q) + (int64_t(p.r) * a.T + i) * a.ldq +
                                                 (int64_t(p.hk) * a.G + h) * D + d);
      }
      // codes come out of a word as bytes 0 and 2, then 1 and 3
      reinterpret_cast<uint4*>(smem + L::QF)[u] = make_uint4(__byte_perm(x[0].x, x[0].y, 0x5410), __byte_perm(x[1].x, x[1].y, 0x5410),
                                                             __byte_perm(x[0].x, x[0].y, 0x7632), __byte_perm(x[1].x, x[1].y, 0x7632));
    }
    if (ok) {
      while (issued - used < NS) {
        if (!valid) advance();
        if (!valid) break;
        issue();
      }
    }
    __syncthreads();
    float o[MT][NT][4] = {}, mref[2 * MT], l[2 * MT], l16[2 * MT];     // rows g and g + 8 of each tile
    int node[2 * MT];
#pragma unroll
    for (int x = 0; x < 2 * MT; ++x) {
      mref[x] = -INFINITY;
      l[x] = l16[x] = 0.0f;
      node[x] = min(m0 + 8 * x + g, a.rows - 1) / a.G;
    }
    for (int t = p.t0 + warp; ok && t < p.t1; t += WARPS) {
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
      const uint8_t *ks = reinterpret_cast<const uint8_t*>(scales + s * 32), *vs = ks + 64;
      const int64_t nd = int64_t(t) * TQ_KEYS - ctx;
      uint32_t kb[2], vb[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) kb[x] = ks[(8 * x + g) * 4 + (DP == 128 ? t4 : t4 >> 1)];
#pragma unroll
      for (int x = 0; x < 4; ++x) vb[x] = vs[(2 * t4 + (x & 1) + 8 * (x >> 1)) * 4 + (DP == 128 ? g >> 1 : g >> 2)];
      auto slice = [&](auto big) {
        constexpr bool BIG = decltype(big)::value;
        float sco[MT][2][4] = {};
        {
          uint32_t w[2][WORDS], f[2], f2[2];
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
            f[x] = tq_factor<E4M3>(kb[x]) * 0x10001u;
            f2[x] = BIG ? tq_factor_above(kb[x]) * 0x10001u : 0u;
          }
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            uint4 q[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) q[mt] = qf[(mt * STEPS + st) * 32];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t b0, b1;
              tq_widen<E4M3, BIG>(w[x][st], f[x], f2[x], b0, b1);
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) tq_mma(sco[mt][x], q[mt], b0, b1);
            }
          }
        }
        // scores in units of log2; what a row does not see becomes -inf
        const bool masked = nd + TQ_KEYS > 0;
        float mx[2 * MT];
        bool up = false;
#pragma unroll
        for (int x = 0; x < 2 * MT; ++x) {
          float (&s0)[4] = sco[x >> 1][0], (&s1)[4] = sco[x >> 1][1];
          const int c = 2 * (x & 1);
          float v[4] = {s0[c], s0[c + 1], s1[c], s1[c + 1]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (!CAP) {
              v[e] *= sc;
            } else {                                   // the odd polynomial where it serves, else from the exponential
              const float y = v[e], z = y * y;
              const float poly = y * __fmaf_rn(__fmaf_rn(__fmaf_rn(a.narrow[3].x, z, a.narrow[2].x), z, a.narrow[1].x), z, a.narrow[0].x);
              v[e] = fabsf(y) * sy <= a.narrow_to ? poly : ta_tanh(y * sc, cap2);
            }
          }
          if (masked) {
            const uint32_t bits = ta_mask32(a, p.r, node[x], n, nd) >> (2 * t4);
            v[0] = bits & 1u ? v[0] : -INFINITY;
            v[1] = bits & 2u ? v[1] : -INFINITY;
            v[2] = bits & 0x100u ? v[2] : -INFINITY;
            v[3] = bits & 0x200u ? v[3] : -INFINITY;
          }
          s0[c] = v[0]; s0[c + 1] = v[1]; s1[c] = v[2]; s1[c + 1] = v[3];
          mx[x] = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
          up = up || mx[x] > mref[x];
        }
        if (__any_sync(0xFFFFFFFFu, up)) {             // a row's new reference lies above its largest score here
#pragma unroll
          for (int x = 0; x < 2 * MT; ++x) {
            float m = fmaxf(mx[x], __shfl_xor_sync(0xFFFFFFFFu, mx[x], 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const float to = m > mref[x] ? m + TQ_ABOVE : mref[x], f = m > mref[x] ? ta_ex2(mref[x] - to) : 1.0f;
            l[x] *= f;
            l16[x] *= f;
            mref[x] = to;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              o[x >> 1][j][2 * (x & 1)] *= f;
              o[x >> 1][j][2 * (x & 1) + 1] *= f;
            }
          }
        }
        uint4 pa[MT];
#pragma unroll
        for (int x = 0; x < 2 * MT; ++x) {
          const float (&s0)[4] = sco[x >> 1][0], (&s1)[4] = sco[x >> 1][1];
          const int c = 2 * (x & 1);
          const float mu = mref[x] == -INFINITY ? 0.0f : mref[x];
          const float w0 = ta_ex2(s0[c] - mu), w1 = ta_ex2(s0[c + 1] - mu), w2 = ta_ex2(s1[c] - mu), w3 = ta_ex2(s1[c + 1] - mu);
          l[x] += (w0 + w1) + (w2 + w3);
          const uint32_t y0 = tq_pack(w0, w1), y1 = tq_pack(w2, w3);
          l16[x] += (__uint_as_float(y0 << 16) + __uint_as_float(y0 & 0xFFFF0000u)) + (__uint_as_float(y1 << 16) + __uint_as_float(y1 & 0xFFFF0000u));
          if (x & 1) {
            pa[x >> 1].y = y0;
            pa[x >> 1].w = y1;
          } else {
            pa[x >> 1].x = y0;
            pa[x >> 1].z = y1;
          }
        }
        // values: pairs of keys 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of columns DP / 8 g ..
        const uint32_t f0 = tq_factor<E4M3>(vb[0]) | (tq_factor<E4M3>(vb[1]) << 16), f1 = tq_factor<E4M3>(vb[2]) | (tq_factor<E4M3>(vb[3]) << 16);
        const uint32_t h0 = BIG ? tq_factor_above(vb[0]) | (tq_factor_above(vb[1]) << 16) : 0u;
        const uint32_t h1 = BIG ? tq_factor_above(vb[2]) | (tq_factor_above(vb[3]) << 16) : 0u;
        uint32_t w[4][WORDS / 2];
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
#pragma unroll
        for (int j = 0; j < NT; j += 2) {
          const uint32_t sel = j & 2 ? 0x7632u : 0x5410u;
          uint32_t b0[2], b1[2];
          tq_widen<E4M3, BIG>(__byte_perm(w[0][j >> 2], w[1][j >> 2], sel), f0, h0, b0[0], b0[1]);
          tq_widen<E4M3, BIG>(__byte_perm(w[2][j >> 2], w[3][j >> 2], sel), f1, h1, b1[0], b1[1]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            tq_mma(o[mt][j], pa[mt], b0[0], b1[0]);
            tq_mma(o[mt][j + 1], pa[mt], b0[1], b1[1]);
          }
        }
      };
      if (E4M3 && __any_sync(0xFFFFFFFFu, max(max(kb[0], kb[1]), max(max(vb[0], vb[1]), max(vb[2], vb[3]))) > 134u)) slice(std::true_type{});
      else slice(std::false_type{});
      ++used;
      __syncwarp();                                    // every lane has read the slot
      if (valid) issue();
    }
    // ---- the piece's result: the warps' parts, rows RB at a time ----
#pragma unroll
    for (int x = 0; x < 2 * MT; ++x) {
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 1);
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 2);
      l16[x] += __shfl_xor_sync(0xFFFFFFFFu, l16[x], 1);
      l16[x] += __shfl_xor_sync(0xFFFFFFFFu, l16[x], 2);
      if (t4 == 0) s_ml[warp][8 * x + g] = make_float4(mref[x], l[x], l16[x], 0.0f);
    }
    __syncthreads();
    const int parts = min(WARPS, p.t1 - p.t0), rows = min(a.rpg, a.rows - m0);
    float w[2 * MT];
#pragma unroll
    for (int x = 0; x < 2 * MT; ++x) {
      float m = -INFINITY;
      for (int k = 0; k < parts; ++k) m = fmaxf(m, s_ml[k][8 * x + g].x);
      w[x] = mref[x] == -INFINITY ? 0.0f : ta_ex2(mref[x] - m);
    }
    const bool whole = p.whole();
    const int64_t slot = p.slot(blockIdx.x);
    for (int r0 = 0; r0 < rows; r0 += L::RB) {
      if (warp < parts) {
#pragma unroll
        for (int x = 0; x < 2 * MT; ++x) {
          const int row = 8 * x + g - r0;              // each lane pair's columns: DP / 4 t .., in 16-byte pieces that trade places
          if (row < 0 || row >= L::RB) continue;
#pragma unroll
          for (int c = 0; c < DP / 16; ++c) {
            const int hi = c / (NT / 4), j = (c % (NT / 4)) * 4, e = 2 * (x & 1) + hi;
            float* at = join + (warp * L::RB + row) * DP + t4 * (DP / 4) + ((c ^ (lane & (DP / 16 - 1))) << 2);
            *reinterpret_cast<float4*>(at) =
                make_float4(o[x >> 1][j][e] * w[x], o[x >> 1][j + 1][e] * w[x], o[x >> 1][j + 2][e] * w[x], o[x >> 1][j + 3][e] * w[x]);
          }
        }
      }
      __syncthreads();
      for (int u = tid; u < L::RB * (DP / 4); u += L::THREADS) {
        const int lr = r0 + u / (DP / 4), c4 = u % (DP / 4), m = m0 + lr;
        const int t = c4 / (DP / 16), c = c4 % (DP / 16), d = c4 * 4;
        if (lr >= rows || d >= D) continue;
        const int ln = ((lr & 7) << 2) | t;            // the lane that wrote it
        const float* at = join + (u / (DP / 4)) * DP + t * (DP / 4) + ((c ^ (ln & (DP / 16 - 1))) << 2);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float M = -INFINITY, sum = 0.0f, div = 0.0f;
        for (int k = 0; k < parts; ++k) M = fmaxf(M, s_ml[k][lr].x);
        for (int k = 0; k < parts; ++k) {
          const float4 z = *reinterpret_cast<const float4*>(at + k * L::RB * DP);
          y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
          const float4 ml = s_ml[k][lr];
          const float f = ml.x == -INFINITY ? 0.0f : ta_ex2(ml.x - M);
          sum = __fmaf_rn(f, ml.y, sum);
          div = __fmaf_rn(f, ml.z, div);
        }
        const int i = m / a.G, h = p.hk * a.G + m - i * a.G;
        const int64_t row = int64_t(p.r) * a.T + i;
        const bool live = i < n, any = live && sum != 0.0f;    // also when the sum is not a number
        if (aborted()) continue;
        if (whole) {
          const float inv = any ? 1.0f / div : 0.0f;
          uint2 z;
          z.x = any ? tq_pack(y.x * inv, y.y * inv) : 0u;
          z.y = any ? tq_pack(y.z * inv, y.w * inv) : 0u;
          *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.out) + row * a.ldo + int64_t(h) * D + d) = z;
          if (c4 == 0 && a.lse) a.lse[row * a.Hq + h] = any ? (M + log2f(sum)) * TA_LN2 : -INFINITY;
        } else {
          *reinterpret_cast<float4*>(a.part_o + (slot * a.rs + lr) * D + d) = y;
          if (c4 == 0) a.part_ml[slot * a.rs + lr] = live ? make_float4(M, sum, div, 0.0f) : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
        }
      }
      __syncthreads();
    }
    // the piece after the next; every warp has left this one
    if (tid == 0) more(kp + 2);
    if (np == 0) nt = s_piece[(kp + 1) % 3].t0 + warp;
    np = max(np - 1, 0);
    __syncthreads();
  }
  // copies in flight land before the block leaves its shared memory to another
  for (; used != issued; ++used) (void)ds_mbar_wait(&s_full[warp][used % NS], (used / NS) & 1u, DS_WAIT_LIMIT);
}

template <int DP, int MT, bool CAP, bool E4M3>
cudaError_t tq_launch(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  constexpr size_t smem = TqLayout<DP, MT>::TOTAL + 1024;
  const cudaError_t e = ds_ensure_smem(reinterpret_cast<const void*>(tree_attn_q8_rows_kernel<DP, MT, CAP, E4M3>), smem);
  if (e != cudaSuccess) return e;
  return ds_launch(tree_attn_q8_rows_kernel<DP, MT, CAP, E4M3>, dim3(unsigned(grid)), dim3(TqLayout<DP, MT>::THREADS), smem, st, a, k, v);
}

template <int DP, int MT>
cudaError_t tq_dispatch(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (a.q8.e4m3) return a.softcap > 0.0f ? tq_launch<DP, MT, true, true>(a, grid, k, v, st) : tq_launch<DP, MT, false, true>(a, grid, k, v, st);
  return a.softcap > 0.0f ? tq_launch<DP, MT, true, false>(a, grid, k, v, st) : tq_launch<DP, MT, false, false>(a, grid, k, v, st);
}

}  // namespace

cudaError_t ta_launch_q8_rows(const TaArgs& a, int grid, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t st) {
  if (a.c.head_dim <= 64) return a.rpg <= 16 ? tq_dispatch<64, 1>(a, grid, k, v, st) : tq_dispatch<64, 2>(a, grid, k, v, st);
  return a.rpg <= 16 ? tq_dispatch<128, 1>(a, grid, k, v, st) : tq_dispatch<128, 2>(a, grid, k, v, st);
}
