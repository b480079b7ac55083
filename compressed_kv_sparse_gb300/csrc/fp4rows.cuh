// Compressed attention rows held in 4 bits (DS4A_FP4_ROWS): where each dim of
// a row lies, and the E2M1 code and 2^k scale arithmetic.
//
// The nope = D - n_rot leading dims are E2M1 codes with one scale 2^k per 16
// dims (k the smallest integer >= -127 with amax <= 6 * 2^k, as in the FP4 round
// trip); the rotated tail keeps the cache's type. The order inside a row is made
// for the attention's tile loader, in which eight lanes read one row: lane j owns
// dims 64 kb + 8 j .. + 7 of every 64-dim block kb, one 32-bit word per block, so
// that its word becomes exactly one 16-byte chunk of the bf16 tile and its whole
// record (words, then the scales it shares with its neighbour) loads as R / 4
// 16-byte vectors, 128 contiguous bytes per row and vector. Inside a word, dim i is
// in half-word i % 2, and pair t = i / 2 has its sign at bit {15, 12, 14, 13}[t] and
// its three magnitude bits at {6, 3, 0, 9}[t] and up: a shift and two masks put
// both dims of a pair where a bf16 pair has sign, lowest exponent and highest
// mantissa bits, which reads as the E2M1 value times 2^-126 (the subnormal 0.5
// included), in 11 integer operations for eight dims.
#pragma once
#include "quant.cuh"

namespace ds4a {

constexpr uint32_t kFp4Block = 16;   // dims per scale

struct Fp4Layout {
  uint32_t nope;       // leading dims held as codes
  uint32_t nb;         // 64-dim blocks = code words per lane
  uint32_t ns;         // scale words per lane
  uint32_t R;          // words per lane record, a multiple of 4
  uint32_t tail;       // byte offset of the rotated dims
  uint32_t row_bytes;
};

__host__ __device__ inline Fp4Layout fp4_layout(uint32_t D, uint32_t n_rot, uint32_t elem_bytes) {
  Fp4Layout L;
  L.nope = D - n_rot;
  L.nb = (L.nope + 63) / 64;
  L.ns = (L.nb + 7) / 8;
  L.R = (L.nb + L.ns + 3) & ~3u;
  L.tail = 32 * L.R;
  L.row_bytes = (L.tail + n_rot * elem_bytes + 31) & ~31u;
  return L;
}

// Byte offset of word w of lane j.
__host__ __device__ inline uint32_t fp4_word_at(uint32_t w, uint32_t j) {
  return 128 * (w / 4) + 16 * j + 4 * (w % 4);
}
// Byte offset of the scale of dims 64 kb + 16 pair .. + 15.
__host__ __device__ inline uint32_t fp4_scale_at(const Fp4Layout &L, uint32_t kb, uint32_t pair) {
  const uint32_t per = 4 * L.ns;
  return fp4_word_at(L.nb + kb % per / 4, 2 * pair + kb / per) + kb % 4;
}
__host__ __device__ inline uint32_t fp4_sign_bit(uint32_t t) { return (0xDECFu >> (4 * t)) & 15; }
__host__ __device__ inline uint32_t fp4_mag_bit(uint32_t t) { return (0x9036u >> (4 * t)) & 15; }

// Scale byte of a block from its largest magnitude: k + 127; 255 when the
// block holds an infinity or a NaN (every dim of it then reads back as NaN).
__device__ __forceinline__ uint32_t fp4_scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax) & 0x7FFFFFFFu;
  if (b >= 0x7F800000u) return 255u;
  return (uint32_t)(block_scale_exp(amax, kE2M1) + 127);
}

// Larger magnitude of two; a NaN stays one (fmaxf would drop it).
__device__ __forceinline__ float fp4_amax(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// Two fp32 values to E2M1 codes (nearest, ties to the even code): lo in bits 0 .. 3
// of the result, hi in bits 4 .. 7.
__device__ __forceinline__ uint32_t fp4_codes2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "cvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// The code word of eight dims under the scale byte sb. x * 2^-k is exact or far
// below the smallest decision point. 6 * 2^126 is beyond fp32: there the largest finite
// value, 3 * 2^126, is taken.
__device__ __forceinline__ uint32_t fp4_encode(const float (&v)[8], uint32_t sb) {
  if (sb == 255u) return 0u;
  const float inv = pow2f(127 - (int)sb);
  uint32_t w = 0;
#pragma unroll
  for (uint32_t t = 0; t < 4; ++t) {
    float lo = __fmul_rn(v[2 * t], inv), hi = __fmul_rn(v[2 * t + 1], inv);
    if (sb == 253u) {
      lo = fminf(fmaxf(lo, -3.f), 3.f);
      hi = fminf(fmaxf(hi, -3.f), 3.f);
    }
    // dim 2 t to bits 0 .. 3, dim 2 t + 1 to bits 16 .. 19, then each part to its place
    // (the places are disjoint: the additions are ors)
    const uint32_t y = (fp4_codes2(lo, hi) * 0x1001u) & 0x000F000Fu;
    w += (y & 0x00070007u) * (1u << fp4_mag_bit(t));
    w += (y & 0x00080008u) * (1u << (fp4_sign_bit(t) - 3));
  }
  return w;
}

// Pair t of a word as two bf16 halves holding the E2M1 values times 2^-126.
template <int T>
__device__ __forceinline__ uint32_t fp4_pair_raw(uint32_t w) {
  if (T == 0) return w & 0x81C081C0u;
  if (T == 1) return (w << 3) & 0x81C081C0u;
  if (T == 2) return ((w << 6) & 0x01C001C0u) | ((w << 1) & 0x80008000u);
  return ((w >> 3) & 0x01C001C0u) | ((w << 2) & 0x80008000u);
}

// The eight fp32 values of a word under the scale byte sb (255: NaN).
__device__ __forceinline__ void fp4_decode(uint32_t w, uint32_t sb, float (&v)[8]) {
  const uint32_t p[4] = {fp4_pair_raw<0>(w), fp4_pair_raw<1>(w), fp4_pair_raw<2>(w),
                         fp4_pair_raw<3>(w)};
  // 2^126 first: the product of a value of at most 6 * 2^-126 is then a small
  // number, and the second product is exact for every scale
  const float s = sb == 255u ? __uint_as_float(0x7FC00000u) : pow2f((int)sb - 127);
#pragma unroll
  for (uint32_t t = 0; t < 4; ++t) {
    v[2 * t] = __fmul_rn(__fmul_rn(__uint_as_float(p[t] << 16), 0x1p126f), s);
    v[2 * t + 1] = __fmul_rn(__fmul_rn(__uint_as_float(p[t] & 0xFFFF0000u), 0x1p126f), s);
  }
}

// A row of fp32 values in shared memory as a 4-bit row, by the first `nt`
// threads of a block (whole warps, all of them here; t: this thread's index).
template <typename T>
__device__ __forceinline__ void fp4_store_row(const float *row, uint8_t *dst, const Fp4Layout &L,
                                              uint32_t n_rot, uint32_t t, uint32_t nt) {
  for (uint32_t base = 0; base < 8 * L.nb; base += nt) {
    const uint32_t kb = (base + t) / 8, j = t & 7, d = 64 * kb + 8 * j;
    const bool in = kb < L.nb && d < L.nope;
    float v[8], am = 0.f;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) {
      v[i] = in ? row[d + i] : 0.f;
      am = fp4_amax(am, v[i]);
    }
    am = fp4_amax(am, __shfl_xor_sync(0xffffffffu, am, 1));
    const uint32_t sb = fp4_scale_byte(am);
    if (kb < L.nb) {
      *reinterpret_cast<uint32_t *>(dst + fp4_word_at(kb, j)) = fp4_encode(v, sb);
      if (!(j & 1)) dst[fp4_scale_at(L, kb, j / 2)] = (uint8_t)sb;
    }
  }
  T *tail = reinterpret_cast<T *>(dst + L.tail);
  for (uint32_t c = t; c < n_rot; c += nt) st_elem(tail, c, row[L.nope + c]);
}

// The same with dims c, c + 1 in this lane and the lanes of a warp in order (c
// = 2 * lane plus a multiple of 64): am is the largest magnitude of the 16 dims
// around c. Every lane of the warp calls it.
template <typename T>
__device__ __forceinline__ void fp4_store_pair(float v0, float v1, uint32_t c, float am,
                                               uint8_t *dst, const Fp4Layout &L, bool store) {
  const uint32_t sb = fp4_scale_byte(am), t = (c % 8) / 2;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i)
    if (i == t) {
      v[2 * i] = v0;
      v[2 * i + 1] = v1;
    }
  uint32_t w = c < L.nope ? fp4_encode(v, sb) : 0u;
  w |= __shfl_xor_sync(0xffffffffu, w, 1);
  w |= __shfl_xor_sync(0xffffffffu, w, 2);
  if (!store) return;
  if (c >= L.nope) {
    T *tail = reinterpret_cast<T *>(dst + L.tail);
    st_elem(tail, c - L.nope, v0);
    st_elem(tail, c - L.nope + 1, v1);
    return;
  }
  const uint32_t kb = c / 64;
  if (c % 8 == 0) *reinterpret_cast<uint32_t *>(dst + fp4_word_at(kb, (c % 64) / 8)) = w;
  if (c % 16 == 0) dst[fp4_scale_at(L, kb, (c % 64) / 16)] = (uint8_t)sb;
}

}  // namespace ds4a
