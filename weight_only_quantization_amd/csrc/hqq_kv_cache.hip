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
#include "hqq_kv_quant.h"

namespace hqq {
namespace kv {
namespace {

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
    store_k<D, BITS>(block, t, o, ck);
    store_v<D, BITS>(block, page, t, o, cv);
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
