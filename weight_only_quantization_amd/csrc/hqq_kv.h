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
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
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

// A list of keys for every sequence: each its own, or one that all query tokens share (lens == nullptr:
// fixed_len keys, a single "sequence" of every query token).
struct KeyList {
  const int32_t* table;
  int64_t table_stride;
  int table_cols;
  const int32_t* lens;
  int fixed_len, max_len;
  const int32_t* cu_q;
  int num_seqs, tq, max_q;
  int causal;
  // where the partial results of its rows begin (in rows of part_o), and their layout: the stream's
  // segments of `cap` rows, or by row
  int64_t part0;
  int tiled;      // split s of row r at s * total_rows + r: of the tiles, or of a stream with a block a pair
  int nsplit, chunk;  // tiles: key splits and the keys of one
  int32_t* segments;  // stream: per pair, its first segment and their number
  int cap;            // stream: rows of a segment, min(16 NT, the widest sequence's rows)
};

struct AttnArgs {
  Format f;
  const void* q;
  int64_t q_ts, q_hs;
  int dtype;
  int hq, per;  // query heads, query heads of one KV head
  int64_t total_q;
  float scale_log2;  // softmax scale * log2(e)
  KeyList list[2];   // the sequences' own keys, the shared prefix
  int joined;        // partial results of both lists meet in the join: no row is finished before it
  int first_list, lists;  // stream: the lists of this launch
  int blocks;             // stream: blocks that share the work of the launch; 0: a block a pair
  void* out;
  float* lse;
  float* part_o;    // [rows][D], not divided by the sum
  float2* part_ml;  // [rows]: running maximum (log2 units) and sum
};

hipError_t launch_kv_write(const WriteArgs& a, int D, int bits, int gs, int dtype, hipStream_t st);
hipError_t launch_kv_read(const ReadArgs& a, int D, int bits, int gs, int dtype, hipStream_t st);
// Rows of up to 16 * nt per block, streamed keys; nt 1 or 2.  stream_blocks: the grid that fills the GPU.
int stream_blocks(int D, int gs, int nt);
hipError_t launch_kv_stream(const AttnArgs& a, int D, int bits, int gs, int nt, hipStream_t st);
// How the stream takes the lists of a launch: shares of the work for each block (loads through the caches, or past them), or a
// block of eight or four waves a pair.
enum StreamMode { kShares, kSharesOnce, kWhole8, kWhole4 };
StreamMode stream_mode(const AttnArgs& a, int nt);
// Tiles of 256 rows of list `which`.
hipError_t launch_kv_tile(const AttnArgs& a, int which, int D, int bits, int gs, hipStream_t st);
// Joins the partial results of every row; nt: of the stream's lists.
hipError_t launch_kv_join(const AttnArgs& a, int D, int nt_own, int nt_prefix, hipStream_t st);

constexpr int kUnitKeys = 128;  // keys of the stream's unit of work: a step of each of a block's four waves
constexpr uint32_t kStartUnits = 3;  // units that beginning a (sequence, row tile, KV head) counts for

// Softmax weights are taken 2^kLift larger than exp(score - running maximum), in the sums too: a score passes the maximum by
// 2^5 at most, so they stay under 2^15 in fp16, which then keeps 11 bits of weights down to 2^-24 of the maximum's and holds
// some down to 2^-35 (without it 2^-14 and 2^-25: a long flat tail under one key counted in the sum but not in the products).
constexpr float kLift = 10.f;
constexpr float kNoKey = -1e30f;  // running maximum before any key (finite: differences of two stay numbers)

// (by value: a bit cast of a vector's element in place takes the vector's first one)
__device__ __forceinline__ h2 as_h2(uint32_t v) { return __builtin_bit_cast(h2, v); }
__device__ __forceinline__ u16x2 as_u16x2(uint32_t v) { return __builtin_bit_cast(u16x2, v); }
__device__ __forceinline__ uint32_t as_u32(h2 v) { return __builtin_bit_cast(uint32_t, v); }

template <bool BF16>
__device__ __forceinline__ void floats8(u32x4 w, float (&x)[8]) {
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
__device__ __forceinline__ void load8(const void* p, float (&x)[8]) {
  floats8<BF16>(*reinterpret_cast<const u32x4*>(p), x);
}
__device__ __forceinline__ void floats8(u32x4 w, int dtype, float (&x)[8]) {
  if (dtype == HQQ_KV_BF16)
    floats8<true>(w, x);
  else
    floats8<false>(w, x);
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

// fp16 outputs: the top code of a group that reaches 65504 may stand for up to 65566 (its step is rounded), so a mean
// of values is held to +-65504; NaN stays.
__device__ __forceinline__ uint32_t pack2_held(float a, float b) {
  a = a > 65504.f ? 65504.f : a < -65504.f ? -65504.f : a;
  b = b > 65504.f ? 65504.f : b < -65504.f ? -65504.f : b;
  return pack2<false>(a, b);
}

template <bool BF16>
__device__ __forceinline__ u32x4 pack8(const float (&x)[8]) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2<BF16>(x[2 * i], x[2 * i + 1]);
  return w;
}

// An entry of an array that no kernel of the call writes, at an index all lanes share: a scalar load.
__device__ __forceinline__ int entry(const int32_t* p, int64_t i) {
  return reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(reinterpret_cast<uintptr_t>(p))[i];
}

// Query tokens and keys of a sequence of a list; nothing of it (tq = 0) where its range of query tokens
// leaves the query tensor.
struct Sequence {
  int q0, tq, len;
};
template <bool SHARED>  // SHARED: all lanes ask for the same sequence
__device__ __forceinline__ Sequence sequence_of(const AttnArgs& a, const KeyList& l, int seq) {
  auto at = [](const int32_t* p, int i) { return SHARED ? entry(p, i) : p[i]; };
  Sequence s{seq * l.tq, l.tq, l.lens ? at(l.lens, seq) : l.fixed_len};
  if (l.cu_q) {
    s.q0 = at(l.cu_q, seq);
    s.tq = at(l.cu_q, seq + 1) - s.q0;
    if (s.q0 < 0 || s.tq < 0 || s.tq > l.max_q || (int64_t)s.q0 + s.tq > a.total_q) s.tq = 0;
  }
  s.len = min(min(max(s.len, 0), l.max_len), l.table_cols << a.f.page_shift);
  return s;
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

// Which kernels a call of hqq_kv_attention(_shared) with these arguments launches, for the tests: per list (own keys, prefix)
// the rows of a block (16, 32 or 256; 0 without the list), the stream's mode (hqq::kv::StreamMode; -1 in tiles) and the tiles' key
// splits; then whether a join follows.  Nothing is read or launched.  Returns the call's status.
extern "C" int hqq_kv_attention_way(const hqq_kv_attention_args* args, int32_t way[7]);
