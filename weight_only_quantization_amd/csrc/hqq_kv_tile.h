// Attention of many query rows over a quantised key/value cache: tiles of 256 rows by 128 keys.
//
// Prompts' chunks, and a prefix under all the rows of a batch: the keys of a tile are dequantised once
// for 256 rows, k = fp16(m + c s) with one rounding, into LDS, and both products run on the matrix unit:
//   S^T[key][row] = K Q^T,  o^T[channel][row] += V^T P^T,
// so a lane's scores (16 of one row to 32 keys) are its operand of the second product as they are: V^T is
// kept in LDS with its keys in that order.  p is rounded to fp16 (kLift); all sums are fp32.
// Eight waves, 32 rows each; all of them unpack 1/8 of the next tile next to this one's products (two
// buffers of K and V, one barrier a tile).  Codes, step and floor become values in packed fp16:
// (1024 + c) - 1024 is exact, fma(c, s, m) rounds once.
// Softmax as in the stream kernel: one pass, fp32, the maximum raised only when a score passes it by 2^5.
//
// 2048 tokens on 8192 keys, 32 heads on 8, 4 bits: 240 Gflop in 270-287 us among such calls, by the card (304 in a trace), 0.84-0.89 Pflop/s; a
// library product of two 8192 x 8192 fp16 matrices reaches 1.18-1.32.  Keys, values and weights in fp16 cost 6.9e-4 of the output (2-norm)
// with the fp16 output's own 2.1e-4.  Per 32 x 32 scores a wave needs 512 cycles of
// the matrix unit and about 600 of the vector unit (16 exponentials take 256); with K and V from LDS and
// their unpacking it takes about 1500 of its SIMD, without either 920: the two waves of a SIMD overlap only in part.
// Of a tile of 128 keys and 256 rows a wave's products and weights take 3.55 us of 4.5, unpacking 0.6, loads 0.24, the barrier 0.3; the
// counters have the matrix unit busy for 43 % of the time and the vector unit for 56 %.
// Padded rows against swizzled ones (an address a read less) 330 -> 312 us, the tile's two halves
// unrolled and each half's values multiplied while the next half's weights are worked out -> 285-310, nothing loaded looked at
// before its tile is unpacked 286 -> 272.  Tried without
// gain: operands read from LDS a phase ahead or 2 to 6 reads ahead (259 against 263, 272 against 277 us: within the runs' spread), 64 rows
// a wave with one wave a SIMD (480 us), wave priorities around the products, a prescribed alternation of matrix and vector
// instructions, one half's weights between the other half's products (274-288 against 266), blocks of four waves on tiles of 64 keys. Two waves that alternate
// such instructions by themselves take 619-678 ns a turn against 499 for the matrix part alone: little overlaps.
#pragma once

#include "hqq_kv.h"

namespace hqq {
namespace kv {
namespace {


constexpr int kWaves = 8, kRows = 32 * kWaves, kKeys = 128;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = reinterpret_cast<const u32x4*>(p)[i];
      w[4 * i] = t[0], w[4 * i + 1] = t[1], w[4 * i + 2] = t[2], w[4 * i + 3] = t[3];
    }
  } else {
    const u32x2 t = *reinterpret_cast<const u32x2*>(p);
    w[0] = t[0], w[1] = t[1];
  }
}

template <int U>
constexpr uint32_t pair_sel(int t, int b) {
  const int x = t * U + b, y = (t + 1) * U + b;
  const uint32_t sx = x % 4, sy = y / 4 == x / 4 ? y % 4 : 4 + y % 4;
  return 0x0c000c00u | sy << 16 | sx;
}

// LDS: rows of K (a key's D halves) and of V^T (a channel's 128 keys), 16 bytes of padding each, so that 16
// lanes reading one 16-byte column, and the unpacking writes, spread over all banks, and every read of a phase is
// one lane address with a constant offset.  V^T's row x is channel (D/16) (x % 16) + x / 16: the 16 units written at
// once are neighbours, and a lane of the output holds whole units.
template <int D>
constexpr int kRowK = 2 * D + 16;
constexpr int kRowV = 2 * kKeys + 16;

template <int D, int BITS, int NG>
struct Raw {
  uint32_t k[D * BITS / 128];  // a quarter of a key's codes
  uint32_t v[D * BITS / 128];  // a unit's codes of four tokens
  uint32_t km[NG];
  u32x4 vm;
  bool has_k;   // whether the key is on a page of the cache
  int tokens;   // of the four how many are there
};

template <int D>
using TilesK = uint8_t[2][kKeys * kRowK<D>];
template <int D>
using TilesV = uint8_t[2][D * kRowV];
template <int N>
struct Lanes {
  static constexpr int value = N;
};

// Rows row0 .. of a pair over its keys kb .. ke - 1: all there is for the block to do.  partial: the sums are left as partial
// result part0 + (its place by row of the call, or TREE: by row of the tile), else the output is finished.
// TREE: the last tq keys are drafted tokens, and a row sees those of them that its mask names.  KG: 2 where the pair has up to 128
// rows, a wave's 32 rows being two waves', one for either half of a tile's keys: no wave is without rows, and the tiles
// are read from LDS once for the two.
template <int D, int BITS, int GS, bool TREE, int KG>
__device__ __forceinline__ void tile_pair(const AttnArgs& a, const KeyList& list, const Sequence& sequence, int seq, int hk, int row0,
                                          int kb, int ke, bool partial, int64_t part0, TilesK<D>& sh_k, TilesV<D>& sh_v,
                                          float2 (&sh_ml)[8][64], int (&sh_holes)[4]) {
  constexpr int NG = D / GS, U = D * BITS / 128;
  constexpr int kRow = D * BITS / 8;
  constexpr int KS = D / 16, DT = D / 32;  // MFMA steps of a score, channel tiles of the output
  int tid = threadIdx.x;
  // (opaque, where a block takes several pairs: else what follows from it is worked out in front of them, and kept in scratch)
  if (TREE) asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 31, h = lane >> 5;
  const int q0 = sequence.q0, tq = sequence.tq, len = sequence.len;
  const int rows = tq * a.per;
  const int page = 1 << a.f.page_shift;
  // the wave's own rows
  const int w_row0 = row0 + 32 * (KG == 2 ? wave & 3 : wave);
  const bool w_on = w_row0 < rows;
  const int w_first = w_on ? w_row0 / a.per : 0, w_last = w_on ? (min(w_row0 + 32, rows) - 1) / a.per : 0;
  const int w_end = !w_on ? 0 : list.causal ? min(ke, len - tq + w_last + 1) : ke;   // keys that some row sees
  const int w_min = list.causal ? len - tq + w_first + 1 : TREE ? len - tq : len;  // keys that all rows see

  // ---- a tile's codes: a quarter of one key and one unit of four tokens a thread.  Nothing that is loaded is looked at before the
  // tile it belongs to is unpacked (of a page's id, before the codes it leads to are asked for), a tile later, so that no load is waited for
  // (with every load's answer tested at once a tile of 256 rows took 5.3 us for 4.5).
  const int32_t* table = list.table + (int64_t)seq * list.table_stride;
  const int last_page = max(list.table_cols - 1, 0);  // (a table without columns: any readable entry)
  const int ik = tid >> 2, iv = (tid >> 4) * 4;
  const uint32_t k_off = (tid & 3) * (kRow / 4);
  const int unit = tid & 15;
  Raw<D, BITS, NG> raw;
  uint32_t id_k, id_v;  // pages of the next tile to load
  auto ask_pages = [&](int key0) {
    id_k = (uint32_t)table[min((key0 + ik) >> a.f.page_shift, last_page)];
    id_v = (uint32_t)table[min((key0 + iv) >> a.f.page_shift, last_page)];
  };
  auto load = [&](int key0, int slot) {  // the codes of the tile at key0, and the page ids of the one after it
    if (key0 >= ke) return;
    const bool on_k = key0 + ik < ke && id_k < a.f.num_pages, on_v = key0 + iv < ke && id_v < a.f.num_pages;
    raw.has_k = on_k;
    raw.tokens = on_v ? len - key0 - iv : 0;
    if (!on_k && key0 + ik < ke) sh_holes[slot] = 1;
    {
      const int off = (key0 + ik) & (page - 1);
      const uint8_t* base = a.f.pages + (int64_t)(on_k ? id_k : 0) * a.f.page_bytes + hk * a.f.block_bytes;
      load_words(base + off * kRow + k_off, raw.k);
      const uint32_t* m = reinterpret_cast<const uint32_t*>(base + 2 * page * kRow) + off;
#pragma unroll
      for (int g = 0; g < NG; ++g) raw.km[g] = m[g * page];
    }
    {
      const int off = (key0 + iv) & (page - 1);
      const uint8_t* base = a.f.pages + (int64_t)(on_v ? id_v : 0) * a.f.page_bytes + hk * a.f.block_bytes;
      load_words(base + page * kRow + off * kRow + unit * 4 * U, raw.v);
      raw.vm = *reinterpret_cast<const u32x4*>(base + 2 * page * kRow + 4 * (page * (NG + unit * (D / 16) / GS) + off));
    }
    ask_pages(key0 + kKeys);
  };
  ask_pages(kb);

  // ---- queries
  h8 qf[KS];
  float cs, odd = 0.f;  // odd: NaN where the row's query is not finite
  int lim;
  const int r = w_row0 + n;
  const bool there = r < rows;
  const int rt = (there ? r : 0) / a.per, rg = (there ? r : 0) % a.per;
  {
    const int64_t at = (int64_t)(q0 + rt) * a.q_ts + (int64_t)(hk * a.per + rg) * a.q_hs;
    u32x4 w[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      w[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.q) + at + 16 * i + 8 * h);
    }
    // the first tile's codes behind the queries
    if (tid < 4) sh_holes[tid] = 0;
    __syncthreads();
    load(kb, 0);
    // the row's largest value, as bits without a sign (infinities and NaN are past all others)
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) most = __builtin_elementwise_max(most, as_u16x2(w[i][j] & 0x7fff7fffu));
    uint32_t top = max((uint32_t)most.x, (uint32_t)most.y);
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    const bool bf16 = a.dtype == HQQ_KV_BF16;
    if (!there) top = 0;
    if (top >= (bf16 ? 0x7f80u : 0x7c00u)) odd = NAN, top = 0;
    if (top == 0) {
#pragma unroll
      for (int i = 0; i < KS; ++i) w[i] = u32x4{0, 0, 0, 0};
    }
    // it goes to [2^14, 2^15): bfloat16 rows of any size keep their bits in fp16
    const float f = bf16 ? __builtin_bit_cast(float, top << 16) : (float)__builtin_bit_cast(_Float16, (uint16_t)top);
    const int e = top ? min(14 - (int)(__builtin_bit_cast(uint32_t, f) >> 23) + 127, 100) : 0;
    cs = ldexpf(a.scale_log2, -e);
    if (bf16 || __any(e > 15)) {
      const float up = ldexpf(1.f, e);
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        float x[8];
        floats8(w[i], a.dtype, x);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const h2 y = __builtin_convertvector((f32x2{x[j] * up, x[j + 1] * up}), h2);
          qf[i][j] = y.x, qf[i][j + 1] = y.y;
        }
      }
    } else {
      const _Float16 up = (_Float16)ldexpf(1.f, e);
#pragma unroll
      for (int i = 0; i < KS; ++i) qf[i] = __builtin_bit_cast(h8, w[i]) * up;
    }
    lim = there ? (list.causal ? min(len - 1, len - tq + rt) : len - 1) : -1;
  }

  // ---- unpacking
  uint32_t m_lo, m_hi, or1024, or64;
  asm("s_mov_b32 %0, 0x000f000f" : "=s"(m_lo));
  asm("s_mov_b32 %0, 0x00f000f0" : "=s"(m_hi));
  asm("v_mov_b32 %0, 0x64006400" : "=v"(or1024));
  asm("v_mov_b32 %0, 0x54005400" : "=v"(or64));
  const h2 n1024 = {(_Float16)-1024.f, (_Float16)-1024.f}, n64 = {(_Float16)-64.f, (_Float16)-64.f};
  auto unpack = [&](Raw<D, BITS, NG>& s, uint8_t* to_k, uint8_t* to_v) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t mm = s.has_k ? s.km[i * 32 / GS] : 0u;  // (a key that is not there: any finite value; its scores are masked)
      const h2 st = as_h2(__builtin_amdgcn_perm(mm, mm, 0x01000100)), fm = as_h2(__builtin_amdgcn_perm(mm, mm, 0x03020302));
      u32x4 w;
      if (BITS == 4) {
        const uint32_t c = s.k[i], d = c >> 8;
        w[0] = as_u32(__builtin_elementwise_fma(as_h2((c & m_lo) | or1024) + n1024, st, fm));
        w[1] = as_u32(__builtin_elementwise_fma(as_h2((c & m_hi) | or64) + n64, st, fm));
        w[2] = as_u32(__builtin_elementwise_fma(as_h2((d & m_lo) | or1024) + n1024, st, fm));
        w[3] = as_u32(__builtin_elementwise_fma(as_h2((d & m_hi) | or64) + n64, st, fm));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t c = __builtin_amdgcn_perm(0, s.k[2 * i + j / 2], j & 1 ? 0x0c030c02 : 0x0c010c00) | or1024;
          w[j] = as_u32(__builtin_elementwise_fma(as_h2(c) + n1024, st, fm));
        }
      }
      *reinterpret_cast<u32x4*>(to_k + ik * kRowK<D> + (4 * i + (tid & 3)) * 16) = w;
    }
    h2 st[2], fm[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = 2 * i < s.tokens ? (uint32_t)s.vm[2 * i] : 0u, y = 2 * i + 1 < s.tokens ? (uint32_t)s.vm[2 * i + 1] : 0u;
      st[i] = as_h2(__builtin_amdgcn_perm(y, x, 0x05040100));
      fm[i] = as_h2(__builtin_amdgcn_perm(y, x, 0x07060302));
    }
    // a 16-key group's chunks: keys 0-3 8-11, keys 4-7 12-15
    const int q = tid >> 4, chunk = 2 * (q >> 2) + (q & 1), half = (q >> 1) & 1;
#pragma unroll
    for (int b = 0; b < U; ++b) {
      u32x2 lo, hi;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t c = __builtin_amdgcn_perm(s.v[((2 * i + 1) * U + b) / 4], s.v[(2 * i * U + b) / 4], pair_sel<U>(2 * i, b));
        lo[i] = as_u32(__builtin_elementwise_fma(as_h2(BITS == 4 ? (c & m_lo) | or1024 : c | or1024) + n1024, st[i], fm[i]));
        if (BITS == 4) hi[i] = as_u32(__builtin_elementwise_fma(as_h2((c & m_hi) | or64) + n64, st[i], fm[i]));
      }
      const int j = BITS == 4 ? 2 * b : b;  // channel of the unit
      uint8_t* at = to_v + (16 * j + unit) * kRowV + chunk * 16 + half * 8;
      *reinterpret_cast<u32x2*>(at) = lo;
      if (BITS == 4) *reinterpret_cast<u32x2*>(at + 16 * kRowV) = hi;
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float mref = kNoKey / fmaxf(cs, 1.f), l = 0.f;  // running maximum (of the scores before cs) and sum

  // 64 keys at a time: two chains of products and of weights side by side
  auto attend = [&](int key0, const uint8_t* kt, const uint8_t* vt, bool holes) {
    const uint8_t* kl = kt + n * kRowK<D> + h * 16;
    const uint8_t* vl = vt + n * kRowV + h * 16;
#pragma unroll
    for (int s2 = 0; s2 < 2 / KG; ++s2) {
      const int sub = KG == 2 ? 2 * (wave >> 2) : 2 * s2;
      const int first = key0 + 32 * sub;
      if (first >= w_end) return;
      f32x16 s[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[c][i] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const h8 kf = *reinterpret_cast<const h8*>(kl + 32 * (sub + c) * kRowK<D> + 32 * i);
          s[c] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[i], s[c], 0, 0, 0);
        }
      if (holes | (first + 64 > w_min) | (first + 64 > ke)) {
        // the drafts among these keys that the lane's row sees
        uint32_t sees[2] = {~0u, ~0u};
        if (TREE) {
          drafts_seen(a.mask + (int64_t)(q0 + rt) * a.mask_words, a.mask_words, first - (len - tq), sees);
          sees[0] >>= 4 * h, sees[1] >>= 4 * h;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = first + 32 * c + 8 * (i >> 2) + 4 * h + (i & 3);
            bool on = key <= lim && key < ke;
            if (TREE) on = on && (sees[c] >> (8 * (i >> 2) + (i & 3)) & 1);
            if (holes) {
              const int id = table[min(key >> a.f.page_shift, max(list.table_cols - 1, 0))];
              on = on && (uint32_t)id < a.f.num_pages;
            }
            s[c][i] = on ? s[c][i] : -INFINITY;
          }
        }
      }
      float top = s[0][0];
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(fmaxf(top, s[0][i]), s[1][i]);
      if (__any((top - mref) * cs > 5.f)) {
        top = fmaxf(top, __shfl_xor(top, 32));
        const float next = (top - mref) * cs > 5.f ? top : mref;  // (each row by its own scores alone)
        const float f = exp2_((mref - next) * cs);
        mref = next;
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] *= f;
      }
      // (exponents as in the stream kernel)
      const float c0 = fmaf(-mref, cs, kLift);
      const bool far = fabsf(c0) > 0x1p20f && mref > kNoKey / 1e17f;
      if (__builtin_expect(__any(far), 0)) {
        const float less = far ? mref : 0.f, plus = far ? kLift : c0;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[c][i] = fmaf(s[c][i] - less, cs, plus);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[c][i] = fmaf(s[c][i], cs, c0);
      }
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        h8 pf[2];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const f32x2 e = {exp2_(s[c][i]), exp2_(s[c][i + 1])};
          sum += e[0] + e[1];
          const h2 p = __builtin_convertvector(e, h2);
          pf[i >> 3][i & 7] = p.x, pf[i >> 3][(i & 7) + 1] = p.y;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const h8 vf = *reinterpret_cast<const h8*>(vl + 32 * d * kRowV + (4 * (sub + c) + 2 * t) * 16);
            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[t], o[d], 0, 0, 0);
          }
      }
      l += sum;
    }
  };

  if (kb < ke) {
    unpack(raw, sh_k[0], sh_v[0]);
    load(kb + kKeys, 1);
    // The second wave of each SIMD unpacks before its products and the first one after them, so that one's matrix
    // instructions meet the other's vector instructions.
    const bool early = wave >= kWaves / 2;
    int i = 0;  // tiles so far; sh_holes[i % 4]: whether tile i has keys that are on no page
    for (int key0 = kb; key0 < ke; key0 += kKeys, ++i) {
      const bool more = key0 + kKeys < ke;
      uint8_t *next_k = sh_k[(i + 1) & 1], *next_v = sh_v[(i + 1) & 1];
      __syncthreads();  // this tile is written; the other buffer is free
      const bool holes = sh_holes[i & 3];
      if (tid == 0) sh_holes[(i + 3) & 3] = 0;
      if (more && early) {
        unpack(raw, next_k, next_v);
        load(key0 + 2 * kKeys, (i + 2) & 3);
      }
      attend(key0, sh_k[i & 1], sh_v[i & 1], holes);
      if (more && !early) {
        unpack(raw, next_k, next_v);
        load(key0 + 2 * kKeys, (i + 2) & 3);
      }
    }
  }

  // ---- output: row x = 32 d + 8 a + 4 h + c of the tile's channels is element 4 a + c of o[d]; the lane holds the
  // units 8 (a % 2) + 4 h + c whole, channel 2 d + a / 2 of each
  mref = fmaf(mref, cs, -kLift);  // what the weights are over, in units of the exponent, from here on
  l += __shfl_xor(l, 32);
  // Half the channels at a time: those of the units 8 p .., elements 4 a + c of even and of odd a.
  const int p0 = KG == 2 ? wave >> 2 : 0;  // the half that the wave finishes, or the first of both
  if (KG == 2) {
    // the two waves of a row tile have half of its keys each, and finish half of its channels each: the other half's sums go over,
    // 16 bytes a lane and store, through the tiles' memory
    float* sh_o = reinterpret_cast<float*>(sh_k[0]);
    static_assert(sizeof(sh_k) >= 8 * 64 * DT * 8 * sizeof(float), "");
    __syncthreads();  // the last tile has been read
    sh_ml[wave][lane] = float2{mref, l};
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) {
      f32x4 x;
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = p0 ? o[i >> 1][8 * (i & 1) + c] : o[i >> 1][8 * (i & 1) + 4 + c];
      *reinterpret_cast<f32x4*>(sh_o + ((wave * 2 * DT + i) * 64 + lane) * 4) = x;
    }
    __syncthreads();
    const float2 other = sh_ml[wave ^ 4][lane];
    const float mm = fmaxf(mref, other.x), f0 = exp2_(mref - mm), f1 = exp2_(other.x - mm);
    mref = mm;
    l = l * f0 + other.y * f1;
#pragma unroll
    for (int i = 0; i < 2 * DT; ++i) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(sh_o + (((wave ^ 4) * 2 * DT + i) * 64 + lane) * 4);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // (kept where the half's first elements are, whichever half it is)
        const float own = p0 ? o[i >> 1][8 * (i & 1) + 4 + c] : o[i >> 1][8 * (i & 1) + c];
        o[i >> 1][8 * (i & 1) + c] = fmaf(own, f0, x[c] * f1);
      }
    }
  }
  // a query with an infinity or NaN gives NaN wherever it sees a key (it entered the products as 0: the fp16 mode above
  // does not hand a NaN on)
  if (l != 0.f) l += odd;
  // Rows are stored whole, 16 bytes a lane, through a part of the tiles' memory: a lane's own pieces are 8 bytes of 32 rows, and
  // as many requests (8 us at the end of every block).
  const int64_t at = (int64_t)(q0 + rt) * a.hq + hk * a.per + rg, part = part0 + (TREE ? r - row0 : at);
  constexpr bool kOver = KG == 1 || sizeof(sh_v) < sizeof(sh_k);  // over the keys, or what has gone from wave to wave
  uint8_t* stage = (kOver ? sh_k[0] : sh_v[0]) + wave * 32 * kRowK<D>;
  static_assert(sizeof(sh_k) == 8 * 32 * kRowK<D>, "");
  if (kOver) __syncthreads();  // all of it has been read
  if (!w_on) return;
  const int live = min(rows - w_row0, 32);  // rows of the wave
  int from = lane;  // (opaque, so that the rows' places are not worked out in front of the tiles)
  asm volatile("" : "+v"(from));
  // rows of `row_lanes` pieces of 16 bytes to to[place of the row by the lane that holds it]
  auto store_rows = [&](uint8_t* to, int64_t row_at, int64_t row_bytes, auto row_lanes) {
    constexpr int PR = decltype(row_lanes)::value, STEP = 16 * PR + 16;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < PR / 2; ++i) {
      const int x = 64 * i + from, row = x / PR, c = x % PR;
      const int64_t to_row = __shfl((long long)row_at, row);
      if (row < live) *reinterpret_cast<u32x4*>(to + to_row * row_bytes + 16 * c) = *reinterpret_cast<const u32x4*>(stage + row * STEP + 16 * c);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
  };
  if (partial) {
    if (h == 0 && there && p0 == 0) a.part_ml[part] = float2{mref, l};
#pragma unroll
    for (int p = 0; p < 2 / KG; ++p) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = 4 * p + u;
#pragma unroll
        for (int d = 0; d < DT; d += 2)
          *reinterpret_cast<f32x4*>(stage + n * kRowK<D> + ((4 * h + u) * (D / 16) + 2 * d) * 4) =
              f32x4{o[d][e], o[d][e + 8], o[d + 1][e], o[d + 1][e + 8]};
      }
      store_rows(reinterpret_cast<uint8_t*>(a.part_o) + (p0 + p) * 2 * D, part, 4 * D, Lanes<D / 8>());
    }
  } else {
    const float inv = l != 0.f ? 1.0f / l : 0.f;
#pragma unroll
    for (int p = 0; p < 2 / KG; ++p)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = 4 * p + u;
#pragma unroll
        for (int d = 0; d < DT; d += 2) {
          const float y0 = o[d][e] * inv, y1 = o[d][e + 8] * inv, y2 = o[d + 1][e] * inv, y3 = o[d + 1][e + 8] * inv;
          u32x2 w = a.dtype == HQQ_KV_BF16 ? u32x2{pack2<true>(y0, y1), pack2<true>(y2, y3)}
                                           : u32x2{pack2<false>(y0, y1), pack2<false>(y2, y3)};
          if (l != l) w = u32x2{0x7fff7fffu, 0x7fff7fffu};
          *reinterpret_cast<u32x2*>(stage + n * (KG == 2 ? D + 16 : kRowK<D>) + ((8 * p + 4 * h + u) * (D / 16) + 2 * d) * 2) = w;
        }
      }
    store_rows(reinterpret_cast<uint8_t*>(a.out) + p0 * D, at, 2 * D, Lanes<D / 8 / KG>());
    if (a.lse && h == 0 && there && p0 == 0) a.lse[at] = l != 0.f ? (mref + __log2f(l)) * 0.69314718056f : -INFINITY;
  }
}

template <int D, int BITS, int GS>
__global__ __launch_bounds__(512, 2) void k_kv_tile(AttnArgs a, int which) {
  const KeyList list = which ? a.list[1] : a.list[0];
  __shared__ __attribute__((aligned(16))) TilesK<D> sh_k;
  __shared__ __attribute__((aligned(16))) TilesV<D> sh_v;

  const int tid = threadIdx.x;
  // fp16 results past the largest number stay there (MODE.FP16_OVFL): a group that reaches +-65504 may stand for
  // a little more than fp16 holds
  __builtin_amdgcn_s_setreg(1 | 23 << 6, 1);

  // Grid: KV head and sequence (x), row tile (y), key split (z).  Blocks go round the eight XCDs in order
  // of x, so the pairs are turned by tile and split: the parts of one long sequence spread over
  // all XCDs.  The tiles with the most keys under a causal rule start first.
  const uint32_t pair = (blockIdx.x + blockIdx.y + blockIdx.z) % gridDim.x;
  const int hk = pair % a.f.hkv, seq = pair / a.f.hkv, split = blockIdx.z, tile = gridDim.y - 1 - blockIdx.y;

  const Sequence sequence = sequence_of<true>(a, list, seq);
  const int q0 = sequence.q0, tq = sequence.tq, len = sequence.len;
  const int rows = tq * a.per;
  const int row0 = tile * kRows;
  if (row0 >= rows) return;
  const int64_t total_rows = a.total_q * a.hq;
  const int last_t = (min(row0 + kRows, rows) - 1) / a.per;
  const int end_all = list.causal ? min(len, max(0, len - tq + last_t + 1)) : len;
  const int kb = split * list.chunk;
  const int ke = min(kb + list.chunk, end_all);
  const bool partial = list.nsplit > 1 || a.joined;
  if (kb >= end_all && partial) {  // no key of this split
    const int row = row0 + tid;
    if (tid < kRows && row < rows)
      a.part_ml[list.part0 + split * total_rows + (int64_t)(q0 + row / a.per) * a.hq + hk * a.per + row % a.per] =
          float2{kNoKey, 0.f};
    return;
  }
  __shared__ int sh_holes[4];
  float2 none[8][64];
  tile_pair<D, BITS, GS, false, 1>(a, list, sequence, seq, hk, row0, kb, ke, partial, list.part0 + split * total_rows, sh_k, sh_v, none, sh_holes);
}

template <int D, int BITS, int GS>
hipError_t tile_t(const AttnArgs& a, int which, hipStream_t st) {
  const KeyList& l = a.list[which];
  const int tiles = (int)(((int64_t)l.max_q * a.per + kRows - 1) / kRows);
  k_kv_tile<D, BITS, GS><<<dim3(a.f.hkv * l.num_seqs, tiles, l.nsplit), 512, 0, st>>>(a, which);
  return hipGetLastError();
}

}  // namespace
}  // namespace kv
}  // namespace hqq
