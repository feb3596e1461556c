// cache_q8.cuh - the numbers of a cache in 8 bits: codes, the powers of two that blocks of 32 columns share, slots, and the
// checks that every entry point makes of a dspark_qcache.
#pragma once

#include "dspark_common.cuh"
#include "host_common.h"

constexpr int Q8_BLOCK = 32;                 // columns that share a scale
constexpr int Q8_TOP = 245;                  // largest scale byte: 480 * 2^(245 - 127) is a float32 and a bf16 number

__host__ __device__ constexpr int q8_blocks(int head_dim) { return (head_dim + Q8_BLOCK - 1) / Q8_BLOCK; }

DS_DEV uint32_t q8_byte(uint32_t b) { return min(max(b, 1u), uint32_t(Q8_TOP)); }
// 2^(byte - 127)
DS_DEV float q8_power(uint32_t byte) { return __uint_as_float(q8_byte(byte) << 23); }

// Codes as numbers without their scale. E4M3: the seven bits under the sign, put where a float32's low exponent and high fraction bits
// are, are the number times 2^-120, subnormal ones included; multiplying by 2^120 is exact.
DS_DEV float q8_e4m3(uint32_t c) {
  return __uint_as_float(((c & 0x80u) << 24) | ((c & 0x7Fu) << 20)) * 0x1p120f;
}
DS_DEV float q8_number(uint32_t c, bool e4m3) { return e4m3 ? q8_e4m3(c & 0xFFu) : float(int8_t(c)); }

// The scale byte of a block whose largest |y| is m: the least e with m <= 448 * 2^e = 1.75 * 2^(8 + e), or 127 * 2^e = 1.984375 *
// 2^(6 + e), from m's exponent and whether its fraction is above that of the bound.
DS_DEV uint32_t q8_choose(float m, bool e4m3) {
  const uint32_t u = __float_as_uint(m);
  const int k = int(u >> 23) - 127;
  const bool over = (u & 0x7FFFFFu) > (e4m3 ? 0x600000u : 0x7E0000u);
  const int e = k - (e4m3 ? 8 : 6) + (over ? 1 : 0);
  return uint32_t(min(max(e, -126), 118) + 127);
}

// Codes of four numbers under 2^-e (`inv`), the first in the low byte; infinities become the largest code. E4M3: the
// conversion rounds to nearest, ties to even, and saturates. INT8: adding 1.5 * 2^23 leaves the rounded number in the low bits.
DS_DEV uint32_t q8_codes(float y0, float y1, float y2, float y3, float inv, bool e4m3) {
  const float z[4] = {y0 * inv, y1 * inv, y2 * inv, y3 * inv};
  if (e4m3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(z[1]), "f"(z[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(z[3]), "f"(z[2]));
    return uint32_t(lo) | (uint32_t(hi) << 16);
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(fminf(fmaxf(z[e], -127.0f), 127.0f) + 12582912.0f);
  return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
}

// Where slot s of request r lies: offsets of its codes and of its scales (head 0, column 0, layer 0); at < 0: it has no place.
struct Q8Slot {
  int64_t at, scale;
};
DS_DEV Q8Slot q8_slot(const dspark_qcache& c, int64_t r, int64_t s) {
  const int64_t e = s / c.page_size;
  if (s < 0 || e >= c.table_pages) return Q8Slot{-1, -1};
  const int32_t p = c.page_table[r * c.ld_table + e];
  if (p < 0 || p >= c.num_pages) return Q8Slot{-1, -1};
  const int64_t t = s - e * c.page_size;
  return Q8Slot{int64_t(p) * c.page_stride + t * c.token_stride, int64_t(p) * c.scale_page_stride + t * c.scale_token_stride};
}

// Checks of a dspark_qcache (`layers`: the layer count is used).
static inline bool q8_cache_ok(const dspark_qcache* c, bool layers) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table) return false;
  if (c->code != DSPARK_E4M3 && c->code != DSPARK_INT8) return false;
  return c->page_stride >= 0 && c->token_stride >= 0 && c->head_stride >= 0 && c->scale_page_stride >= 0 &&
         c->scale_token_stride >= 0 && c->scale_head_stride >= 0 && c->num_pages >= 1 && c->num_pages <= INT32_MAX &&
         c->page_size >= 1 && c->page_size <= 65536 && c->heads >= 1 && c->heads <= 1024 && c->head_dim >= 8 &&
         c->head_dim <= 256 && c->head_dim % 8 == 0 && c->table_pages >= 1 && c->ld_table >= c->table_pages &&
         (!layers || (c->n_layers >= 1 && c->layer_stride >= 0 && c->scale_layer_stride >= 0));
}

// Every row of every head's codes starts on a boundary of `a` bytes.
static inline bool q8_codes_aligned(const dspark_qcache* c, int64_t a) {
  return ds_aligned(c->k, size_t(a)) && ds_aligned(c->v, size_t(a)) && c->page_stride % a == 0 && c->token_stride % a == 0 &&
         c->head_stride % a == 0 && c->layer_stride % a == 0;
}
// Every row of every head's scales does.
static inline bool q8_scales_aligned(const dspark_qcache* c, int64_t a) {
  return ds_aligned(c->k_scale, size_t(a)) && ds_aligned(c->v_scale, size_t(a)) && c->scale_page_stride % a == 0 &&
         c->scale_token_stride % a == 0 && c->scale_head_stride % a == 0 && c->scale_layer_stride % a == 0;
}
// The scale bytes of a box of slots (`bytes` of them, a multiple of 16, slots side by side) start on 16-byte boundaries.
static inline bool q8_scales_box(const dspark_qcache* c, int64_t bytes) {
  return bytes % 16 == 0 && ds_aligned(c->k_scale, 16) && ds_aligned(c->v_scale, 16) && c->scale_page_stride % 16 == 0 && c->scale_head_stride % 16 == 0;
}
