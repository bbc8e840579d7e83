// Rotary positions: by themselves, and on the way into the quantised cache.
//
// Of each head the first rot channels are pairs (a, b), turned by theta = position * freq of the pair:
//   a' = a c - b s,  b' = b c + a s,  c = m cos theta, s = m sin theta;   the gradient is the transposed one, s = -m sin theta.
// Angles and the rotation are 64 bits, the result is rounded once: at position 10^6 a 32-bit angle is 0.03 off, and a key
// that is rounded like the separate calls' (and like a reference's) takes the same code where it lies next to a border.
//
// Both kernels move bytes; the cosines and sines of a block's tokens are worked out once, a pair or two a thread, and serve
// all heads that the block's waves walk over.  16411 tokens of 64 heads of 128 channels (538 MB): 95 us, 5.7 TB/s, where a large copy has
// 5.8-6.1; 64 bits cost nothing there (105 and 107 us at an earlier step).  16387 prompt tokens of 64 query heads on 8 into a cache of
// 8 bits with their echo (707 MB): 129 us, 5.5 TB/s.  A step of 64 tokens of 40 heads takes 4.3 us, the chain position -> angle ->
// pair -> store, and the host's call three times that.
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

// How a wave takes the heads of a token: a lane owns two runs of 8 channels of a head (at0, at1) that make whole pairs, `per` heads
// side by side are a wave's step, and `lane_head` is the lane's among them (per where the lane has none).  So a wave walks through a
// token's heads as they lie in memory.
struct Lane {
  int at0, at1, per, lane_head;
  bool t0, t1;  // whether the runs are turned (else copied)
};
template <bool INTER>
__device__ __forceinline__ Lane lane_of(int head_dim, int rot, int lane) {
  const int units = head_dim / 16, u = lane % units;
  Lane l;
  l.per = 64 / units;
  l.lane_head = lane / units;
  if (INTER) {
    l.at0 = 8 * u, l.at1 = 8 * (u + units);
    l.t0 = l.at0 < rot, l.t1 = l.at1 < rot;
  } else {
    l.t0 = l.t1 = 16 * u < rot;
    l.at0 = l.t0 ? 8 * u : 16 * u, l.at1 = l.t0 ? rot / 2 + 8 * u : 16 * u + 8;
  }
  return l;
}
// The lane's pairs of a token, whose table this is: of run 0 (halves: of both runs), and of run 1.
template <bool INTER>
__device__ __forceinline__ void lane_pairs(const double2* tab, int rot, const Lane& l, double2 (&cs)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool on = INTER && j >= 4 ? l.t1 : l.t0;
    const int i = !INTER ? l.at0 + j : j < 4 ? l.at0 / 2 + j : l.at1 / 2 + j - 4;
    cs[j] = tab[on ? pair_at(rot, i) : 0];
  }
}

template <bool BF16, bool INTER>
__device__ __forceinline__ void turn_runs(const Lane& l, const double2 (&cs)[8], u32x4& w0, u32x4& w1) {
  float x[8], y[8];
  floats8<BF16>(w0, x);
  floats8<BF16>(w1, y);
  if (INTER) {
    if (l.t0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn_pair(x[2 * j], x[2 * j + 1], cs[j]);
      w0 = pack8<BF16>(x);
    }
    if (l.t1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) turn_pair(y[2 * j], y[2 * j + 1], cs[4 + j]);
      w1 = pack8<BF16>(y);
    }
  } else if (l.t0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) turn_pair(x[j], y[j], cs[j]);
    w0 = pack8<BF16>(x);
    w1 = pack8<BF16>(y);
  }
}

// Heads first + lane_head, then every `step` further, two steps' loads in flight.  Loads past the caches (16411 tokens, 538 MB into
// ever new outputs: 103 us for 108), and stores where there is much (Heads::past: 95 for 103; calls that reuse one output, half of
// which the last cache then holds, lose by it: 94 for 85).
template <bool BF16, bool INTER, bool PAST>
__device__ __forceinline__ void turn_heads_to(const Heads& x, int64_t token, int first, int step, const Lane& l, const double2 (&cs)[8]) {
  const uint16_t* from = reinterpret_cast<const uint16_t*>(x.in) + token * x.in_ts;
  uint16_t* to = reinterpret_cast<uint16_t*>(x.out) + token * x.out_ts;
  for (int h0 = first; h0 < x.count; h0 += 2 * step) {
    u32x4 w[2][2];
    bool on[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = h0 + k * step + l.lane_head;
      on[k] = l.lane_head < l.per && h < x.count;
      if (on[k]) {
        w[k][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + h * x.in_hs + l.at0));
        w[k][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + h * x.in_hs + l.at1));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!on[k]) continue;
      const int h = h0 + k * step + l.lane_head;
      turn_runs<BF16, INTER>(l, cs, w[k][0], w[k][1]);
      u32x4 *to0 = reinterpret_cast<u32x4*>(to + h * x.out_hs + l.at0), *to1 = reinterpret_cast<u32x4*>(to + h * x.out_hs + l.at1);
      if (PAST) {
        __builtin_nontemporal_store(w[k][0], to0);
        __builtin_nontemporal_store(w[k][1], to1);
      } else {
        *to0 = w[k][0];
        *to1 = w[k][1];
      }
    }
  }
}

template <bool BF16, bool INTER>
__device__ __forceinline__ void turn_heads(const Heads& x, int64_t token, int first, int step, const Lane& l, const double2 (&cs)[8]) {
  if (x.past)
    turn_heads_to<BF16, INTER, true>(x, token, first, step, l, cs);
  else
    turn_heads_to<BF16, INTER, false>(x, token, first, step, l, cs);
}

// A wave a token, or every fourth of the block's.
template <bool BF16, bool INTER>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a, int tokens) {
  __shared__ double2 tab[kTab];
  const int64_t token0 = (int64_t)blockIdx.x * tokens;
  make_table(a.turn, token0, tokens, a.n, tab);
  __syncthreads();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Lane l = lane_of<INTER>(a.head_dim, a.turn.rot, threadIdx.x & 63);
  for (int t = wave; t < tokens && token0 + t < a.n; t += 4) {
    double2 cs[8];
    lane_pairs<INTER>(tab + t * (a.turn.rot / 2), a.turn.rot, l, cs);
    turn_heads<BF16, INTER>(a.q, token0 + t, blockIdx.y * l.per, gridDim.y * l.per, l, cs);
    turn_heads<BF16, INTER>(a.k, token0 + t, blockIdx.y * l.per, gridDim.y * l.per, l, cs);
  }
}

// Into the cache.  The queries as above; keys (turned, rounded to the type, quantised) and values (quantised) in the order of the
// cache's own write, a lane 8 channels, so that a group's lanes are side by side and four tokens' value codes
// meet in one store: the other channels of a key's pairs come from the lane that has them.
template <int D, int BITS, int GS, bool BF16, bool INTER>
__global__ __launch_bounds__(256) void k_write_rope(WriteRopeArgs a) {
  constexpr int OCT = D / 8, TOKENS = 64 / OCT, NG = D / GS;
  __shared__ double2 tab[TOKENS * D / 2];
  const int64_t n = a.w.n, token0 = (int64_t)blockIdx.x * TOKENS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = lane / OCT, o = lane % OCT;
  const bool there = token0 + t < n;
  // (lanes behind the last token go along on it, and store nothing)
  const int64_t token = there ? token0 + t : n - 1;
  const int64_t slot = a.w.slots[token];
  const int hkv = a.w.f.hkv;
  auto load = [&](int i) {
    const bool is_k = i < hkv;
    const uint16_t* p = reinterpret_cast<const uint16_t*>(is_k ? a.w.k : a.w.v);
    p += token * (is_k ? a.w.k_ts : a.w.v_ts) + (is_k ? i : i - hkv) * (is_k ? a.w.k_hs : a.w.v_hs);
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p + 8 * o));
  };
  const int step = 4 * gridDim.y;
  int i = blockIdx.y * 4 + wave;
  u32x4 w = {};
  if (i < 2 * hkv) w = load(i);
  make_table(a.turn, token0, TOKENS, n, tab);
  __syncthreads();
  const int rot = a.turn.rot, half = rot / 2;
  {
  const bool turned = 8 * o < rot, first = 8 * o < half;
  const int partner = t * OCT + (INTER || !turned ? o : first ? o + rot / 16 : o - rot / 16);
  // halves: own c + other s, the sine with the sign that the half's formula gives it
  double2 cs[INTER ? 4 : 8];
#pragma unroll
  for (int j = 0; j < (INTER ? 4 : 8); ++j) {
    cs[j] = tab[!turned ? 0 : t * half + pair_at(rot, (INTER ? 4 * o : first ? 8 * o : 8 * o - half) + j)];
    if (!INTER && first) cs[j].y = -cs[j].y;
  }
  auto take = [&](int i, u32x4 w) {
    const bool is_k = i < hkv;
    const int head = is_k ? i : i - hkv;
    float x[8];
    floats8<BF16>(w, x);
    if (is_k) {
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
      floats8<BF16>(turned ? r : w, x);
    }
    int c[8], at;
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
  };
  for (; i < 2 * hkv; i += step) {
    u32x4 next = {};
    if (i + step < 2 * hkv) next = load(i + step);
    take(i, w);
    w = next;
  }
  }
  {
    const Lane l = lane_of<INTER>(D, rot, lane);
    for (int i = wave; i < TOKENS && token0 + i < n; i += 4) {
      double2 cs[8];
      lane_pairs<INTER>(tab + i * half, rot, l, cs);
      turn_heads<BF16, INTER>(a.q, token0 + i, blockIdx.y * l.per, gridDim.y * l.per, l, cs);
    }
  }
}

// Blocks over the tokens, and how many share a block's heads (`most` at most): the more the fewer tokens there are.
dim3 rope_grid(int64_t n, int tokens, int most) {
  const int64_t x = (n + tokens - 1) / tokens;
  int64_t y = (1024 + x - 1) / x;
  y = y > most ? most : y;
  return dim3((unsigned)x, (unsigned)(y < 1 ? 1 : y));
}

template <int D, int BITS, int GS>
hipError_t write_rope_t(const WriteRopeArgs& a, int dtype, bool inter, hipStream_t st) {
  const int per = 64 / (D / 16), q = (a.q.count + per - 1) / per, kv = (2 * a.w.f.hkv + 3) / 4;
  const dim3 grid = rope_grid(a.w.n, write_rope_tokens(D), q > kv ? q : kv);
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
  const int tokens = rope_tokens(a.head_dim), per = 64 / (a.head_dim / 16);
  const dim3 grid = rope_grid(a.n, tokens, ((a.q.count > a.k.count ? a.q.count : a.k.count) + per - 1) / per);
  if (dtype == HQQ_KV_BF16)
    inter ? k_rope<true, true><<<grid, 256, 0, st>>>(a, tokens) : k_rope<true, false><<<grid, 256, 0, st>>>(a, tokens);
  else
    inter ? k_rope<false, true><<<grid, 256, 0, st>>>(a, tokens) : k_rope<false, false><<<grid, 256, 0, st>>>(a, tokens);
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
