// Attention of a few query rows over a quantised key/value cache: the launches of the stream (hqq_kv_stream.h), and the join
// of the partial results that streams and tiles leave.
#include "hqq_kv_stream.h"

namespace hqq {
namespace kv {
namespace {

// Where a row's partial results of one list lie: the first, and the k-th at next + k * step.
struct Parts {
  int64_t first, next, step;
  int count;
};

__device__ __forceinline__ Parts parts_of(const AttnArgs& a, const KeyList& l, int nt, int64_t token, int head,
                                          int lane) {
  const int64_t total_rows = a.total_q * a.hq;
  if (l.tiled) {
    const int64_t at = l.part0 + token * a.hq + head;
    return {at, at, total_rows, l.nsplit};
  }
  int seq = 0, t = (int)token;
  if (l.cu_q) {  // the last sequence that begins at or before the token
    seq = -1;
    for (int s0 = 0; s0 < l.num_seqs; s0 += 64) {
      const uint64_t m = __ballot(s0 + lane < l.num_seqs && l.cu_q[s0 + lane] <= token && token < l.cu_q[s0 + lane + 1]);
      if (m) seq = s0 + 63 - __builtin_clzll(m);
    }
    if (seq < 0) return {0, 0, 0, 0};
    const Sequence s = sequence_of<true>(a, l, seq);
    if (s.tq == 0) return {0, 0, 0, 0};
    t = (int)token - s.q0;
  } else if (l.num_seqs > 1) {
    seq = (int)token / l.tq;
    t = (int)token - seq * l.tq;
  }
  const int row = t * a.per + head % a.per, of = 16 * nt;
  const int tiles = (l.max_q * a.per + of - 1) / of;
  const int64_t at = ((int64_t)seq * tiles + row / of) * a.f.hkv + head / a.per;
  const int segment = l.segments[2 * at], count = l.segments[2 * at + 1];
  const int64_t r = l.part0 + row % of;
  if (a.joined) return {r + (int64_t)segment * l.cap, r + (int64_t)segment * l.cap, l.cap, count};
  return {r + (int64_t)segment * l.cap, r + (int64_t)(segment & ~1) * l.cap, 2 * (int64_t)l.cap, count};
}

// Joins the parts of each row: a wave a row.  The parts that hold keys are listed first (their
// weights a lane each), then read 64 / (D / 4) at a time, 16 bytes a lane, four such reads in flight.
template <int D>
__global__ __launch_bounds__(256) void k_kv_join(AttnArgs a, int nt_own, int nt_prefix) {
  constexpr int LP = D / 4, PP = 64 / LP;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (row >= a.total_q * a.hq) return;
  const int lane = threadIdx.x & 63, sub = lane / LP, d = lane % LP * 4;
  const int64_t token = row / a.hq;
  const int head = (int)(row - token * a.hq);
  const Parts own = parts_of(a, a.list[0], nt_own, token, head, lane);
  Parts pre{0, 0, 0, 0};
  if (a.joined) pre = parts_of(a, a.list[1], nt_prefix, token, head, lane);
  const int parts = own.count + pre.count;
  if (parts == 0) return;  // finished by the stream (or a token of no sequence)
  auto place = [&](int p) -> int64_t {
    const bool o = p < own.count;
    const int k = o ? p : p - own.count;
    const Parts& x = o ? own : pre;
    return k == 0 ? x.first : x.next + k * x.step;
  };
  float2 ml = float2{kNoKey, 0.f};
  if (lane < parts) ml = a.part_ml[place(lane)];
  float top = ml.y != 0.f ? ml.x : kNoKey;
  for (int p = lane + 64; p < parts; p += 64) {
    const float2 x = a.part_ml[place(p)];
    if (x.y != 0.f) top = fmaxf(top, x.x);
  }
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) top = fmaxf(top, __shfl_xor(top, i));
  float sum = 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int p0 = 0; p0 < parts; p0 += 64) {
    if (p0) {
      ml = float2{kNoKey, 0.f};
      if (p0 + lane < parts) ml = a.part_ml[place(p0 + lane)];
    }
    const bool on = ml.y != 0.f;
    const float w = on ? exp2_(ml.x - top) : 0.f;
    sum += on ? w * ml.y : 0.f;
    const uint64_t mask = __ballot(on), below = (1ull << lane) - 1;
    const int count = __popcll(mask);
    const int to = on ? __popcll(mask & below) : count + __popcll(~mask & below);
    const int listed = __builtin_amdgcn_ds_permute(4 * to, lane);  // lane i: the i-th part with keys
    for (int k = 0; k < count; k += 4 * PP) {
      f32x4 x[4];
      float wx[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = k + u * PP + sub;
        const int part = __shfl(listed, i < count ? i : 0);
        wx[u] = __shfl(w, part);
        if (i >= count) wx[u] = 0.f;
        x[u] = *reinterpret_cast<const f32x4*>(a.part_o + place(p0 + part) * D + d);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) o += x[u] * wx[u];
    }
  }
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) sum += __shfl_xor(sum, i);
#pragma unroll
  for (int i = LP; i < 64; i <<= 1)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] += __shfl_xor(o[c], i);
  if (sub == 0) {
    const float inv = sum != 0.f ? 1.0f / sum : 0.f;
    u32x2 w;
    if (a.dtype == HQQ_KV_BF16)
      w = u32x2{pack2<true>(o[0] * inv, o[1] * inv), pack2<true>(o[2] * inv, o[3] * inv)};
    else
      w = u32x2{pack2_held(o[0] * inv, o[1] * inv), pack2_held(o[2] * inv, o[3] * inv)};
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + row * D + d) = w;
    if (a.lse && lane == 0) a.lse[row] = sum != 0.f ? (top + __log2f(sum)) * 0.69314718056f : -INFINITY;
  }
}

// Joins the parts of the own keys of a call without a prefix, by (sequence, row tile, KV head): a block takes 16 rows of one, 16
// threads a row, and ends at once where the pair was finished by one block (a wave a row, which looks for
// its pair itself, took 12 us for 32768 rows with nothing to join).
template <int D>
__global__ __launch_bounds__(256) void k_kv_join_pairs(AttnArgs a, int tile_rows) {
  constexpr int CH = D / 16, U = 4;
  const KeyList& l = a.list[0];
  const uint32_t tiles = (uint32_t)(((int64_t)l.max_q * a.per + tile_rows - 1) / tile_rows);
  const uint32_t pair = blockIdx.x, hk = pair % a.f.hkv, seq = pair / a.f.hkv / tiles, tile = pair / a.f.hkv - seq * tiles;
  const Sequence s = sequence_of<true>(a, l, seq);
  const int in_tile = 16 * blockIdx.y + threadIdx.x / 16, row = tile * tile_rows + in_tile, d = threadIdx.x % 16 * CH;
  // (the segments of a tile without rows were never written)
  if ((int)(tile * tile_rows + 16 * blockIdx.y) >= s.tq * a.per) return;
  const int segment = l.segments[2 * (int64_t)pair], count = l.segments[2 * (int64_t)pair + 1];
  if (count == 0 || row >= s.tq * a.per) return;
  float m = kNoKey, sum = 0.f;
  f32x4 o[CH / 4];
#pragma unroll
  for (int j = 0; j < CH / 4; ++j) o[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int p0 = 0; p0 < count; p0 += U) {
    float2 ml[U];
    f32x4 x[U][CH / 4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = min(p0 + u, count - 1);
      const int64_t part = l.part0 + (int64_t)(p == 0 ? segment : (segment & ~1) + 2 * p) * l.cap + in_tile;
      ml[u] = a.part_ml[part];
#pragma unroll
      for (int j = 0; j < CH / 4; ++j) x[u][j] = *reinterpret_cast<const f32x4*>(a.part_o + part * D + d + 4 * j);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = p0 + u < count && ml[u].y != 0.f;  // (the sums of a part without keys were never written)
      const float next = on ? fmaxf(m, ml[u].x) : m;
      const float f = exp2_(m - next), w = on ? exp2_(ml[u].x - next) : 0.f;
      m = next;
      sum = sum * f + (on ? ml[u].y * w : 0.f);
#pragma unroll
      for (int j = 0; j < CH / 4; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][c] = o[j][c] * f + (on ? x[u][j][c] * w : 0.f);
    }
  }
  const int64_t at = (int64_t)(s.q0 + row / a.per) * a.hq + hk * a.per + row % a.per;
  const float inv = sum != 0.f ? 1.0f / sum : 0.f;
  uint16_t* to = reinterpret_cast<uint16_t*>(a.out) + at * D + d;
#pragma unroll
  for (int j = 0; j < CH / 4; ++j) {
    u32x2 w;
    if (a.dtype == HQQ_KV_BF16)
      w = u32x2{pack2<true>(o[j][0] * inv, o[j][1] * inv), pack2<true>(o[j][2] * inv, o[j][3] * inv)};
    else
      w = u32x2{pack2_held(o[j][0] * inv, o[j][1] * inv), pack2_held(o[j][2] * inv, o[j][3] * inv)};
    *reinterpret_cast<u32x2*>(to + 4 * j) = w;
  }
  if (a.lse && d == 0) a.lse[at] = sum != 0.f ? (m + __log2f(sum)) * 0.69314718056f : -INFINITY;
}

}  // namespace

StreamMode stream_mode(const AttnArgs& a, int nt) {
  const KeyList& l = a.list[a.first_list];
  const int tiles = tiles_in(a, l, nt);
  if (a.blocks) return tiles == 1 && (a.lists == 1 || tiles_in(a, a.list[1], nt) == 1) ? kSharesOnce : kShares;
  // A CU holds one block of eight waves; more blocks than CUs would take it in turns, blocks of four run side by side
  // (64 sequences of 1000 keys, 64 heads on 8: 23.5 us with eight waves, 18.9 with four).
  return (int64_t)a.f.hkv * l.num_seqs * tiles <= 256 ? kWhole8 : kWhole4;
}

int stream_blocks(int D, int gs, int nt) { return 256 * stream_waves(D, gs, nt); }

hipError_t launch_kv_stream(const AttnArgs& a, int D, int bits, int gs, int nt, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return stream_t<d, b, g, false>(a, nt, st);
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128) X(128, 8, 32)
  X(128, 8, 64) X(128, 8, 128)
#undef X
  return hipErrorInvalidValue;
}

hipError_t launch_kv_join(const AttnArgs& a, int D, int nt_own, int nt_prefix, hipStream_t st) {
  const dim3 grid((unsigned)((a.total_q * a.hq + 3) / 4));
  if (D == 128)
    k_kv_join<128><<<grid, 256, 0, st>>>(a, nt_own, nt_prefix);
  else
    k_kv_join<64><<<grid, 256, 0, st>>>(a, nt_own, nt_prefix);
  return hipGetLastError();
}

hipError_t launch_kv_join_pairs(const AttnArgs& a, int D, int tile_rows, hipStream_t st) {
  const KeyList& l = a.list[0];
  const int64_t rows = (int64_t)l.max_q * a.per, pairs = (rows + tile_rows - 1) / tile_rows * a.f.hkv * l.num_seqs;
  const dim3 grid((unsigned)pairs, (unsigned)((l.cap + 15) / 16));
  if (D == 128)
    k_kv_join_pairs<128><<<grid, 256, 0, st>>>(a, tile_rows);
  else
    k_kv_join_pairs<64><<<grid, 256, 0, st>>>(a, tile_rows);
  return hipGetLastError();
}

}  // namespace kv
}  // namespace hqq
