// Writing and reading the quantised key/value cache.
//
// A group of GS channels of one token and head keeps b-bit codes, a step and a floor (fp16):
//   m = fp16(min x),  s = fp16((max x - m) / (2^b - 1)),  c = clamp(rint((x - m) / s), 0, 2^b - 1),
// and stands for m + c s.  The floor (not a zero in code units) keeps a group of small range far
// from 0, as keys with a channel offset have, to fp16 accuracy.  All arithmetic is fp32.
// x is first made finite (NaN to 0, then held to the fp16 range), so no written value is infinite
// or NaN and a masked key can enter the attention's products with weight 0.
//
// Both kernels move bytes: a thread owns 8 channels of one token and head (16 bytes of K and of V),
// D/8 neighbouring lanes a token, and the group's minimum and maximum go over GS/8 lanes by
// shuffles.  Lanes run over four tokens of one head before the next head: V codes of four tokens
// share 16 bytes (the order the attention's wide loads want), so a wave's stores are contiguous.
//
// HBM-bound: 32768 tokens of 8 heads of 128 in 4 bits, with the echo, 306 MB in 53 us, 5.8 TB/s; read back of
// 65536 tokens in 8 bits 411 MB in 72 us, 5.7 TB/s (a large copy: 6.1 TB/s).  64 tokens take 3.4 us, most of it
// the launch.
#include "hqq_kv.h"

namespace hqq {
namespace kv {
namespace {

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

template <int D, int BITS>
__device__ __forceinline__ void store_codes(uint8_t* block, int page, int t, int o, const int (&ck)[8],
                                            const int (&cv)[8]) {
  uint8_t* kp = block + t * Codes<D, BITS>::kRow + k_place<D, BITS>(o);
  uint8_t* vb = block + page * Codes<D, BITS>::kRow;
  uint8_t* vp = vb + v_place<D, BITS>(t, o);
  if (BITS == 4) {
    *reinterpret_cast<uint32_t*>(kp) = nibbles_k(ck);
    const uint32_t w = nibbles_v(cv);
    if (D >= 128) {
      *reinterpret_cast<uint32_t*>(vp) = w;
    } else {
      *reinterpret_cast<uint16_t*>(vp) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(vp + 4 * Codes<D, BITS>::kUnit) = (uint16_t)(w >> 16);
    }
  } else {
    *reinterpret_cast<u32x2*>(kp) = bytes8(ck);
    const u32x2 w = bytes8(cv);
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

// Thread -> (token, head, octet): four tokens of a head, then the next head, then the next four.
template <int D>
__device__ __forceinline__ bool locate(int64_t n, int hkv, int64_t* token, int* head, int* oct) {
  constexpr int OCT = D / 8;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t quad = i / (4 * OCT);
  *oct = (int)(i % OCT);
  *head = (int)(quad % hkv);
  *token = quad / hkv * 4 + (i / OCT) % 4;
  return *token < n;
}

template <int D, int BITS, int GS, bool BF16>
__global__ __launch_bounds__(256) void k_kv_write(WriteArgs a) {
  int64_t token;
  int head, o, t;
  // (a token's D/8 lanes stay or leave together: no shuffle reaches a lane that left)
  if (!locate<D>(a.n, a.f.hkv, &token, &head, &o)) return;
  const int64_t slot = a.slots[token];
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(a.k) + token * a.k_ts + head * a.k_hs + 8 * o;
  const uint16_t* vp = reinterpret_cast<const uint16_t*>(a.v) + token * a.v_ts + head * a.v_hs + 8 * o;
  float xk[8], xv[8];
  int ck[8], cv[8];
  load8<BF16>(kp, xk);
  load8<BF16>(vp, xv);
  const uint32_t mk = quantise<BITS, GS>(xk, ck);
  const uint32_t mv = quantise<BITS, GS>(xv, cv);
  uint8_t* block = slot_block(a.f, slot, head, &t);
  if (block) {
    const int page = 1 << a.f.page_shift;
    store_codes<D, BITS>(block, page, t, o, ck, cv);
    if (o % (GS / 8) == 0) {
      uint32_t* meta = reinterpret_cast<uint32_t*>(block + 2 * page * Codes<D, BITS>::kRow);
      const int g = o / (GS / 8);
      meta[g * page + t] = mk;
      meta[(D / GS + g) * page + t] = mv;
    }
  }
  if (a.k_echo) {
    const int64_t at = (token * a.f.hkv + head) * D + 8 * o;
    store_dense<BF16>(a.k_echo, at, xk);
    store_dense<BF16>(a.v_echo, at, xv);
  }
}

template <int BITS>
__device__ __forceinline__ void values(u32x2 w, uint32_t meta, bool k_order, float (&x)[8]) {
  const h2 p = as_h2(meta);
  const float s = (float)p.x, m = (float)p.y;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t c;
    if (BITS == 8)
      c = (w[j >> 2] >> (8 * (j & 3))) & 255;
    else
      c = (w[0] >> (4 * (k_order ? (j >> 1) + 4 * (j & 1) : j))) & 15;
    x[j] = m + (float)c * s;
  }
}

template <int D, int BITS, int GS, bool BF16>
__global__ __launch_bounds__(256) void k_kv_read(ReadArgs a) {
  int64_t token;
  int head, o, t;
  if (!locate<D>(a.n, a.f.hkv, &token, &head, &o)) return;
  const uint8_t* block = slot_block(a.f, a.slots[token], head, &t);
  float xk[8] = {}, xv[8] = {};
  if (block) {
    const int page = 1 << a.f.page_shift;
    const uint8_t* kp = block + t * Codes<D, BITS>::kRow + k_place<D, BITS>(o);
    const uint8_t* vp = block + page * Codes<D, BITS>::kRow + v_place<D, BITS>(t, o);
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(block + 2 * page * Codes<D, BITS>::kRow);
    const int g = o / (GS / 8);
    u32x2 wk = {}, wv = {};
    if (BITS == 4) {
      wk[0] = *reinterpret_cast<const uint32_t*>(kp);
      if (D >= 128)
        wv[0] = *reinterpret_cast<const uint32_t*>(vp);
      else
        wv[0] = *reinterpret_cast<const uint16_t*>(vp) |
                (uint32_t) * reinterpret_cast<const uint16_t*>(vp + 4 * Codes<D, BITS>::kUnit) << 16;
    } else {
      wk = *reinterpret_cast<const u32x2*>(kp);
      if (D >= 128) {
        wv = *reinterpret_cast<const u32x2*>(vp);
      } else {
        wv[0] = *reinterpret_cast<const uint32_t*>(vp);
        wv[1] = *reinterpret_cast<const uint32_t*>(vp + 4 * Codes<D, BITS>::kUnit);
      }
    }
    values<BITS>(wk, meta[g * page + t], true, xk);
    values<BITS>(wv, meta[(D / GS + g) * page + t], false, xv);
  }
  const int64_t at = (token * a.f.hkv + head) * D + 8 * o;
  store_dense<BF16>(a.k, at, xk);
  store_dense<BF16>(a.v, at, xv);
}

inline dim3 token_grid(int64_t n, int hkv, int D) {
  return dim3((unsigned)(((n + 3) / 4 * 4 * hkv * (D / 8) + 255) / 256));
}

template <int D, int BITS, int GS>
hipError_t write_t(const WriteArgs& a, int dtype, hipStream_t st) {
  const dim3 grid = token_grid(a.n, a.f.hkv, D);
  if (dtype == HQQ_KV_BF16)
    k_kv_write<D, BITS, GS, true><<<grid, 256, 0, st>>>(a);
  else
    k_kv_write<D, BITS, GS, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

template <int D, int BITS, int GS>
hipError_t read_t(const ReadArgs& a, int dtype, hipStream_t st) {
  const dim3 grid = token_grid(a.n, a.f.hkv, D);
  if (dtype == HQQ_KV_BF16)
    k_kv_read<D, BITS, GS, true><<<grid, 256, 0, st>>>(a);
  else
    k_kv_read<D, BITS, GS, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

#define HQQ_KV_FORMATS(X)                                                                                \
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128)       \
  X(128, 8, 32) X(128, 8, 64) X(128, 8, 128)

hipError_t launch_kv_write(const WriteArgs& a, int D, int bits, int gs, int dtype, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return write_t<d, b, g>(a, dtype, st);
  HQQ_KV_FORMATS(X)
#undef X
  return hipErrorInvalidValue;
}

hipError_t launch_kv_read(const ReadArgs& a, int D, int bits, int gs, int dtype, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return read_t<d, b, g>(a, dtype, st);
  HQQ_KV_FORMATS(X)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace hqq
