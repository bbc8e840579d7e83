// Rotary positions: by themselves, and on the way into the quantised cache.
//
// Of each head the first rot channels are pairs (a, b), turned by theta = position * freq of the pair:
//   a' = a c - b s,  b' = b c + a s,  c = m cos theta, s = m sin theta;   the gradient is the transposed one, s = -m sin theta.
// Angles and the rotation are 64 bits, the result is rounded once: at position 10^6 a 32-bit angle is 0.03 off, and a key
// that is rounded like the separate calls' (and like a reference's) takes the same code where it lies next to a border.
//
// Both kernels move bytes: a wave takes a head of some tokens, 16 bytes of it a lane and load; the cosines and sines of a
// block's tokens are worked out once, a pair or two a thread, and serve all heads that the block's waves walk over.
#include "hqq_draft.h"
#include "hqq_kv_quant.h"

namespace hqq {
namespace kv {
namespace {

constexpr int kTab = 512;  // pairs of all tokens of a block

// Place of a token's pair i in the table: pairs 8 apart are neighbours, as lanes of a wave ask for them.
__device__ __forceinline__ int pair_at(int rot, int i) { return (i & 7) * (rot / 16) + (i >> 3); }

// c and s of the block's tokens: tab[t * rot / 2 + pair_at(i)].
__device__ __forceinline__ void make_table(const Turn& turn, int64_t token0, int tokens, int64_t n, double2* tab) {
  const int half = turn.rot / 2;
  for (int e = threadIdx.x; e < tokens * half; e += blockDim.x) {
    const int t = e / half, i = e - t * half;
    const int64_t token = token0 + t;
    double2 cs = {0.0, 0.0};
    if (token < n) {
      double s, c;
      sincos((double)turn.positions[token] * turn.freqs[i], &s, &c);
      cs = {c * turn.c_scale, s * turn.s_scale};
    }
    tab[t * half + pair_at(turn.rot, i)] = cs;
  }
}

// (a c - b s, b c + a s)
__device__ __forceinline__ void turn_pair(float& a, float& b, double2 cs) {
  const double x = a, y = b;
  a = (float)fma(-y, cs.y, x * cs.x);
  b = (float)fma(x, cs.y, y * cs.x);
}

// A lane owns 16 channels of a head: two runs of 8, which are whole pairs: channels 8 u .. and rot / 2 + 8 u .. (halves), or
// 16 u .. 16 u + 15 (interleaved, and the channels that are only copied).
template <bool BF16, bool INTER>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a) {
  __shared__ double2 tab[kTab];
  const int units = a.head_dim / 16, tokens = 64 / units;
  const int64_t token0 = (int64_t)blockIdx.x * tokens;
  make_table(a.turn, token0, tokens, a.n, tab);
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = lane / units, u = lane - t * units;
  const int64_t token = token0 + t;
  if (t >= tokens || token >= a.n) return;
  const int rot = a.turn.rot, half = rot / 2;
  const bool turned = 16 * u < rot;
  const int at0 = !INTER && turned ? 8 * u : 16 * u, at1 = !INTER && turned ? half + 8 * u : 16 * u + 8;
  double2 cs[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) cs[j] = tab[turned ? t * half + pair_at(rot, 8 * u + j) : 0];

  const int heads = a.q.count + a.k.count, step = 4 * gridDim.y;
  auto from = [&](int h) {
    const bool is_q = h < a.q.count;
    const Heads& x = is_q ? a.q : a.k;
    return reinterpret_cast<const uint16_t*>(x.in) + token * x.in_ts + (is_q ? h : h - a.q.count) * x.in_hs;
  };
  int h = blockIdx.y * 4 + wave;
  if (h >= heads) return;
  u32x4 w0 = *reinterpret_cast<const u32x4*>(from(h) + at0), w1 = *reinterpret_cast<const u32x4*>(from(h) + at1);
  while (true) {
    // (the next head's are asked for before this one's are stored)
    const int next = h + step;
    u32x4 n0 = {}, n1 = {};
    if (next < heads) {
      n0 = *reinterpret_cast<const u32x4*>(from(next) + at0);
      n1 = *reinterpret_cast<const u32x4*>(from(next) + at1);
    }
    if (turned) {
      float x[8], y[8];
      floats8<BF16>(w0, x);
      floats8<BF16>(w1, y);
      if (INTER) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          turn_pair(x[2 * j], x[2 * j + 1], cs[j]);
          turn_pair(y[2 * j], y[2 * j + 1], cs[4 + j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn_pair(x[j], y[j], cs[j]);
      }
      w0 = pack8<BF16>(x);
      w1 = pack8<BF16>(y);
    }
    const bool is_q = h < a.q.count;
    const Heads& o = is_q ? a.q : a.k;
    uint16_t* to = reinterpret_cast<uint16_t*>(o.out) + token * o.out_ts + (is_q ? h : h - a.q.count) * o.out_hs;
    *reinterpret_cast<u32x4*>(to + at0) = w0;
    *reinterpret_cast<u32x4*>(to + at1) = w1;
    if (next >= heads) break;
    h = next, w0 = n0, w1 = n1;
  }
}

// Into the cache: a lane owns 8 channels, as in the cache's own write, whose quantisation takes a group's
// lanes side by side; the other channels of its pairs come from the lane that has them.  The waves of a block walk over the query heads
// (turned), the key heads (turned, rounded to the type, quantised) and the value heads (quantised).
template <int D, int BITS, int GS, bool BF16, bool INTER>
__global__ __launch_bounds__(256) void k_write_rope(WriteRopeArgs a) {
  constexpr int OCT = D / 8, TOKENS = 64 / OCT, NG = D / GS;
  __shared__ double2 tab[kTab];
  const int64_t n = a.w.n, token0 = (int64_t)blockIdx.x * TOKENS;
  make_table(a.turn, token0, TOKENS, n, tab);
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = lane / OCT, o = lane % OCT;
  const bool there = token0 + t < n;
  // (lanes behind the last token go along on it, and store nothing)
  const int64_t token = there ? token0 + t : n - 1;
  const int rot = a.turn.rot, half = rot / 2;
  const bool turned = 8 * o < rot, first = 8 * o < half;
  const int partner = t * OCT + (INTER || !turned ? o : first ? o + rot / 16 : o - rot / 16);
  // halves: own c + other s, the sine with the sign that the half's formula gives it
  double2 cs[INTER ? 4 : 8];
#pragma unroll
  for (int j = 0; j < (INTER ? 4 : 8); ++j) {
    cs[j] = tab[!turned ? 0 : t * half + pair_at(rot, (INTER ? 4 * o : first ? 8 * o : 8 * o - half) + j)];
    if (!INTER && first) cs[j].y = -cs[j].y;
  }
  const int64_t slot = a.w.slots[token];

  const int hkv = a.w.f.hkv, hq = a.q.count, items = hq + 2 * hkv, step = 4 * gridDim.y;
  auto load = [&](int i) {
    const bool is_q = i < hq, is_k = i < hq + hkv;
    const int head = is_q ? i : is_k ? i - hq : i - hq - hkv;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(is_q ? a.q.in : is_k ? a.w.k : a.w.v);
    p += token * (is_q ? a.q.in_ts : is_k ? a.w.k_ts : a.w.v_ts) + head * (is_q ? a.q.in_hs : is_k ? a.w.k_hs : a.w.v_hs);
    return *reinterpret_cast<const u32x4*>(p + 8 * o);
  };
  int i = blockIdx.y * 4 + wave;
  if (i >= items) return;
  u32x4 w = load(i);
  while (true) {
    const int next = i + step;
    u32x4 ahead = {};
    if (next < items) ahead = load(next);
    if (i < hq + hkv) {
      float x[8];
      floats8<BF16>(w, x);
      if (INTER) {
#pragma unroll
        for (int j = 0; j < 4; ++j) turn_pair(x[2 * j], x[2 * j + 1], cs[j]);
      } else {
        u32x4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __shfl((int)w[j], partner);
        float y[8];
        floats8<BF16>(v, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = (float)fma((double)y[j], cs[j].y, (double)x[j] * cs[j].x);
      }
      const u32x4 r = pack8<BF16>(x);
      if (turned) w = r;
    }
    if (i < hq) {
      uint16_t* to = reinterpret_cast<uint16_t*>(a.q.out) + token * a.q.out_ts + i * a.q.out_hs + 8 * o;
      if (there) *reinterpret_cast<u32x4*>(to) = w;
    } else {
      const bool is_k = i < hq + hkv;
      const int head = is_k ? i - hq : i - hq - hkv;
      float x[8];
      int c[8], at;
      floats8<BF16>(w, x);
      const uint32_t m = quantise<BITS, GS>(x, c);
      uint8_t* block = there ? slot_block(a.w.f, slot, head, &at) : nullptr;
      if (block) {
        const int page = 1 << a.w.f.page_shift;
        if (is_k)
          store_k<D, BITS>(block, at, o, c);
        else
          store_v<D, BITS>(block, page, at, o, c);
        if (o % (GS / 8) == 0) {
          uint32_t* meta = reinterpret_cast<uint32_t*>(block + 2 * page * Codes<D, BITS>::kRow);
          meta[((is_k ? 0 : NG) + o / (GS / 8)) * page + at] = m;
        }
      }
      if (a.w.k_echo && there) store_dense<BF16>(is_k ? a.w.k_echo : a.w.v_echo, (token * hkv + head) * D + 8 * o, x);
    }
    if (next >= items) break;
    i = next, w = ahead;
  }
}

// Blocks over the tokens, and how many share a block's heads: four waves walk over them, and the more the fewer tokens there are.
dim3 rope_grid(int64_t n, int tokens, int heads) {
  const int64_t x = (n + tokens - 1) / tokens, most = (heads + 3) / 4;
  int64_t y = (1024 + x - 1) / x;
  y = y > most ? most : y;
  return dim3((unsigned)x, (unsigned)(y < 1 ? 1 : y));
}

template <int D, int BITS, int GS>
hipError_t write_rope_t(const WriteRopeArgs& a, int dtype, bool inter, hipStream_t st) {
  const dim3 grid = rope_grid(a.w.n, write_rope_tokens(D), a.q.count + 2 * a.w.f.hkv);
  if (dtype == HQQ_KV_BF16) {
    inter ? k_write_rope<D, BITS, GS, true, true><<<grid, 256, 0, st>>>(a)
          : k_write_rope<D, BITS, GS, true, false><<<grid, 256, 0, st>>>(a);
  } else {
    inter ? k_write_rope<D, BITS, GS, false, true><<<grid, 256, 0, st>>>(a)
          : k_write_rope<D, BITS, GS, false, false><<<grid, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int dtype, bool inter, hipStream_t st) {
  const dim3 grid = rope_grid(a.n, rope_tokens(a.head_dim), a.q.count + a.k.count);
  if (dtype == HQQ_KV_BF16)
    inter ? k_rope<true, true><<<grid, 256, 0, st>>>(a) : k_rope<true, false><<<grid, 256, 0, st>>>(a);
  else
    inter ? k_rope<false, true><<<grid, 256, 0, st>>>(a) : k_rope<false, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_write_rope(const WriteRopeArgs& a, int D, int bits, int gs, int dtype, bool inter, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return write_rope_t<d, b, g>(a, dtype, inter, st);
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128) X(128, 8, 32)
  X(128, 8, 64) X(128, 8, 128)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace hqq
