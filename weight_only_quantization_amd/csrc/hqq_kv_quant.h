// Quantising eight channels of a token and storing their codes: shared by the kernels that write the cache.
#pragma once

#include "hqq_kv.h"

namespace hqq {
namespace kv {

// Bytes of one token's codes, and of the part of them that holds 8 channels.
template <int D, int BITS>
struct Codes {
  static constexpr int kRow = D * BITS / 8;
  static constexpr int kOct = BITS;
  static constexpr int kUnit = D * BITS / 128;  // V: bytes of the D/16 channels of one unit
};

// Byte offset of octet o's codes in the K row of a token.
template <int D, int BITS>
__device__ __forceinline__ int k_place(int o) {
  return ((o & 3) * (D / 32) + (o >> 2)) * Codes<D, BITS>::kOct;
}

// Byte offset of octet o's codes of token t (of the page) in the V codes; an octet spans
// 8 / (D/16) units: two halves 4 units apart for D = 64, one place for D >= 128.
template <int D, int BITS>
__device__ __forceinline__ int v_place(int t, int o) {
  constexpr int U = Codes<D, BITS>::kUnit;
  constexpr int per_unit = D / 16;                     // channels
  const int unit = 8 * o / per_unit, within = (8 * o) % per_unit;
  return (((t >> 2) * 16 + unit) * 4 + (t & 3)) * U + within * BITS / 8;
}

// Eight 4-bit codes to a word: K order (nibble n holds code {0,2,4,6,1,3,5,7}[n]: masks of the word
// then give pairs of neighbouring channels) or plain order.
__device__ __forceinline__ uint32_t nibbles_k(const int (&c)[8]) {
  return c[0] | c[2] << 4 | c[4] << 8 | c[6] << 12 | c[1] << 16 | c[3] << 20 | c[5] << 24 | (uint32_t)c[7] << 28;
}
__device__ __forceinline__ uint32_t nibbles_v(const int (&c)[8]) {
  return c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12 | c[4] << 16 | c[5] << 20 | c[6] << 24 | (uint32_t)c[7] << 28;
}
__device__ __forceinline__ u32x2 bytes8(const int (&c)[8]) {
  u32x2 w;
  w[0] = c[0] | c[1] << 8 | c[2] << 16 | (uint32_t)c[3] << 24;
  w[1] = c[4] | c[5] << 8 | c[6] << 16 | (uint32_t)c[7] << 24;
  return w;
}

template <int BITS, int GS>
__device__ __forceinline__ uint32_t quantise(float (&x)[8], int (&c)[8]) {
  constexpr float qmax = (float)((1 << BITS) - 1);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = x[j] == x[j] ? x[j] : 0.f;
    x[j] = fminf(fmaxf(x[j], -65504.f), 65504.f);
  }
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) lo = fminf(lo, x[j]), hi = fmaxf(hi, x[j]);
#pragma unroll
  for (int d = 1; d < GS / 8; d <<= 1) lo = fminf(lo, __shfl_xor(lo, d)), hi = fmaxf(hi, __shfl_xor(hi, d));
  const _Float16 m = (_Float16)lo;
  // (the floor rounded up past the maximum of a flat group would make the step negative)
  const _Float16 s = (_Float16)fmaxf((hi - (float)m) * (1.0f / qmax), 0.f);
  const float sf = (float)s, mf = (float)m, inv = sf > 0.f ? 1.0f / sf : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float t = fminf(fmaxf(rintf((x[j] - mf) * inv), 0.f), qmax);
    c[j] = (int)t;
    x[j] = mf + t * sf;  // what the code stands for
  }
  const h2 p = {s, m};
  return as_u32(p);
}

// Octet o of token t of the page: its K codes, its V codes.
template <int D, int BITS>
__device__ __forceinline__ void store_k(uint8_t* block, int t, int o, const int (&c)[8]) {
  uint8_t* kp = block + t * Codes<D, BITS>::kRow + k_place<D, BITS>(o);
  if (BITS == 4)
    *reinterpret_cast<uint32_t*>(kp) = nibbles_k(c);
  else
    *reinterpret_cast<u32x2*>(kp) = bytes8(c);
}
template <int D, int BITS>
__device__ __forceinline__ void store_v(uint8_t* block, int page, int t, int o, const int (&c)[8]) {
  uint8_t* vp = block + page * Codes<D, BITS>::kRow + v_place<D, BITS>(t, o);
  if (BITS == 4) {
    const uint32_t w = nibbles_v(c);
    if (D >= 128) {
      *reinterpret_cast<uint32_t*>(vp) = w;
    } else {
      *reinterpret_cast<uint16_t*>(vp) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(vp + 4 * Codes<D, BITS>::kUnit) = (uint16_t)(w >> 16);
    }
  } else {
    const u32x2 w = bytes8(c);
    if (D >= 128) {
      *reinterpret_cast<u32x2*>(vp) = w;
    } else {
      *reinterpret_cast<uint32_t*>(vp) = w[0];
      *reinterpret_cast<uint32_t*>(vp + 4 * Codes<D, BITS>::kUnit) = w[1];
    }
  }
}

// Eight dense values, past the caches: the kernels move more than those hold (read back of 65536 tokens, 8
// bits: 78 us with ordinary stores, 72 so; a prompt batch of 32768 tokens written and echoed 57 and 53).
template <bool BF16>
__device__ __forceinline__ void store_dense(void* to, int64_t at, const float (&x)[8]) {
  __builtin_nontemporal_store(pack8<BF16>(x), reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(to) + at));
}

}  // namespace kv
}  // namespace hqq
