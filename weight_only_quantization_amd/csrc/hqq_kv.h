// Internal declarations of the quantised key/value cache: the page format, the launch arguments and
// the device helpers that the cache and attention kernels share.
#pragma once

#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/hqq.h"

namespace hqq {
namespace kv {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// One KV head's block of a page: K codes, V codes, K metadata, V metadata (include/hqq.h).
struct Format {
  uint8_t* pages;
  uint32_t num_pages;
  int hkv, page_shift;
  int64_t block_bytes, page_bytes;
};

struct WriteArgs {
  Format f;
  const void* k;
  const void* v;
  int64_t k_ts, k_hs, v_ts, v_hs;  // token and head strides in elements
  int64_t n;
  const int64_t* slots;
  void* k_echo;  // [n, hkv, D] contiguous, or nullptr
  void* v_echo;
};

struct ReadArgs {
  Format f;
  int64_t n;
  const int64_t* slots;
  void* k;
  void* v;
};

// One pass of attention rows over one list of keys per sequence (lens, table), or over a list that
// all rows share (lens == nullptr: fixed_len keys, one "sequence" of every query token).
struct AttnArgs {
  Format f;
  const void* q;
  int64_t q_ts, q_hs;
  int dtype;
  int hq, per;  // query heads, query heads of one KV head
  int num_seqs, tq, max_q;
  int64_t total_q;
  const int32_t* cu_q;
  const int32_t* table;
  int64_t table_stride;
  int table_cols;
  const int32_t* lens;
  int fixed_len, max_len;
  int causal;
  float scale_log2;  // softmax scale * log2(e)
  int nsplit, chunk;  // key splits and the keys of one
  // nsplit_total == 1: the rows go to out (and lse); else to the partials, from index part0 on
  void* out;
  float* lse;
  float* part_o;    // [parts][total_q * hq][D], not divided by the sum
  float2* part_ml;  // [parts][total_q * hq]: running maximum (log2 units) and sum
  int part0, parts;
};

hipError_t launch_kv_write(const WriteArgs& a, int D, int bits, int gs, int dtype, hipStream_t st);
hipError_t launch_kv_read(const ReadArgs& a, int D, int bits, int gs, int dtype, hipStream_t st);
// Rows of up to 16 * NT per wave, streamed keys; NT 1 or 2.
hipError_t launch_kv_stream(const AttnArgs& a, int D, int bits, int gs, int nt, hipStream_t st);
// Tiles of 256 rows.
hipError_t launch_kv_tile(const AttnArgs& a, int D, int bits, int gs, hipStream_t st);
hipError_t launch_kv_join(const AttnArgs& a, int D, hipStream_t st);

constexpr float kNoKey = -1e30f;  // running maximum before any key (finite: differences of two stay numbers)

// (by value: a bit cast of a vector's element in place takes the vector's first one)
__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }
__device__ __forceinline__ uint32_t as_u32(h2 v) { return __builtin_bit_cast(uint32_t, v); }

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, float (&x)[8]) {
  const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      x[2 * i] = __builtin_bit_cast(float, w[i] << 16);
      x[2 * i + 1] = __builtin_bit_cast(float, w[i] & 0xffff0000u);
    } else {
      const h2 t = as_h2(w[i]);
      x[2 * i] = (float)t.x;
      x[2 * i + 1] = (float)t.y;
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF16) {
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    b2 t = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, t);
  }
  const f32x2 s = {a, b};
  return as_u32(__builtin_convertvector(s, h2));
}

template <bool BF16>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<BF16>(x[2 * i], x[2 * i + 1]);
  return w;
}

// A block's KV head and sequence (grid x), row tile (y) and key split (z).  Blocks go round the eight
// XCDs in order of x, so the pairs are turned by tile and split: the parts of one long sequence
// spread over all XCDs, and so do those of short ones, which end early.  (With the split in x, XCD 0 had every
// sequence's first keys and XCD 7 only the longest ones': 35 us for the ragged lengths of 32 sequences of
// up to 4096 keys, as long as if all had 4096.)
struct BlockPlace {
  int hk, seq, tile, split;
};
__device__ __forceinline__ BlockPlace block_place(int hkv) {
  const uint32_t pair = (blockIdx.x + blockIdx.y + blockIdx.z) % gridDim.x;
  return {(int)(pair % hkv), (int)(pair / hkv), (int)blockIdx.y, (int)blockIdx.z};
}

// Page id and address of a slot; nullptr where the slot is outside the cache.
__device__ __forceinline__ uint8_t* slot_block(const Format& f, int64_t slot, int head, int* off) {
  if (slot < 0) return nullptr;
  const int64_t page = slot >> f.page_shift;
  if (page >= (int64_t)f.num_pages) return nullptr;
  *off = (int)(slot & ((1 << f.page_shift) - 1));
  return f.pages + page * f.page_bytes + head * f.block_bytes;
}

}  // namespace kv
}  // namespace hqq
