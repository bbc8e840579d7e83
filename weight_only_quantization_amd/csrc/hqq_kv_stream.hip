// Attention of a few query rows over a quantised key/value cache: one stream over the keys.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  k = m + c s,  v = m + c s per group.
//
// A wave owns 16 * NT rows (the query tokens and heads that share a KV head) and walks its keys in
// steps of 32, registers only: the cache is stored so that each lane's wide loads are operands of the
// matrix unit.
//   scores  S^T[key][row] = sum_g s_jg (sum_{d in g} c_jd q_d) + m_jg (sum_{d in g} q_d): the codes go
//           in exactly, as fp16 subnormals c 2^-24 (a mask of the word is the operand; the other
//           nibble of a byte is 16 c, its q carries 1/16), step and floor apply to the fp32 sums.
//   softmax one pass, running maximum and sum in fp32; a lane holds 8 keys of one row.  A row's maximum is
//           raised (and its sums rescaled) only when a score passes it by 2^5, so the cross-lane
//           reduction is rare; the weights stay within fp16.
//   values  O^T[channel][row] += (c s)[channel][key] p[key][row]: a lane's 8 scores are its operand as
//           they are (keys keep their order inside the step).  c s is one fp16 rounding,
//           fma(1024 + c, s, -1024 s), 2^-8 smaller for steps of 32 and more; the floors enter as one more product, sum_j p_j m_j.
//           p is rounded to fp16 (2^-11 relative at most, from 2^-24 of the maximum's weight down 2^-35 of that; kLift).
//           These two roundings are what the matrix unit's fp16 operands cost: 5.2e-4 to 5.8e-4 of the output (2-norm) with the fp16
//           output's own 2.1e-4 (fp32 products run at a sixteenth of the rate).
// Next keys are loaded as soon as this step's scores are done, the next values after this
// step's product, each into the registers just read: few registers, so three waves a SIMD cover the
// memory's latency (two with both steps' registers held: 3.2 TB/s at 16 sequences of 16384-32768 keys,
// 64 heads on 8; so 5.9, of 455.6 MB by the counters, 1.004 of the bytes it cannot do without).  The four or eight waves of a block
// take every fourth or eighth step of its keys and are joined through LDS; pairs that several blocks share, and both lists of
// a shared call, are joined by k_kv_join.
#include "hqq_kv.h"

namespace hqq {
namespace kv {
namespace {

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// mask and or in one instruction (its constants in registers)
struct Masks {
  uint32_t lo, hi;        // 0x000f000f, 0x00f000f0
  uint32_t or1024, or64;  // fp16 pairs (1024, 1024), (64, 64)
};

template <int D, int BITS>
struct Geo {
  static constexpr int kRow = D * BITS / 8;     // bytes of a token's codes
  static constexpr int kUnit = D * BITS / 128;  // V: bytes of a token in one lane's unit
  static constexpr int kKW = kRow / 16;         // dwords of K codes per lane and 16-key tile
  static constexpr int kVW = kUnit;             // dwords of V codes per lane and 16-key tile (4 tokens)
  static constexpr int kMf = D / 32;            // MFMAs of a K tile
  static constexpr int kVm = D / 16;            // MFMAs of the values (= channels of a unit)
};

// One step's keys or values as loaded: two tiles of 16 keys.
template <int D, int BITS, int NG>
struct StepK {
  uint32_t c[2][Geo<D, BITS>::kKW];
  u32x4 m[2][NG];
};
template <int D, int BITS>
struct StepV {
  uint32_t c[2][Geo<D, BITS>::kVW];
  u32x4 m[2];
};

// Where a step's two tiles lie: their pages' blocks, and bit t set where tile t has no keys (past the end, or no such
// page; some tokens of page 0 are loaded then, unused).
struct Place {
  const uint8_t* base[2];
  uint32_t bad;
};
// A step's registers, and the places of the step they hold and of the next one they will hold.
template <int D, int BITS, int NG>
struct Stage {
  StepK<D, BITS, NG> k;
  StepV<D, BITS> v;
  Place now, then;
};

// ONCE: past the caches, for keys that one block alone reads (the mode kSharesOnce below).
template <bool ONCE, typename T>
__device__ __forceinline__ T load(const uint8_t* p) {
  const T* from = reinterpret_cast<const T*>(p);
  return ONCE ? __builtin_nontemporal_load(from) : *from;
}
template <bool ONCE, int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const u32x4 t = load<ONCE, u32x4>(p + 16 * i);
      w[4 * i] = t[0], w[4 * i + 1] = t[1], w[4 * i + 2] = t[2], w[4 * i + 3] = t[3];
    }
  } else {
    const u32x2 t = load<ONCE, u32x2>(p);
    w[0] = t[0], w[1] = t[1];
  }
}

// Selector that takes byte `b` of token `t` and of token `t + 1` (bytes t * U + b of the lane's dwords)
// to bytes 0 and 2, zeros between; of v_perm_b32(second word, first word).
template <int U>
constexpr uint32_t pair_sel(int t, int b) {
  const int x = t * U + b, y = (t + 1) * U + b;
  const uint32_t sx = x % 4, sy = y / 4 == x / 4 ? y % 4 : 4 + y % 4;
  return 0x0c000c00u | sy << 16 | sx;
}

// Waves per SIMD (blocks per CU) that the registers are held to: the most that does not spill.
constexpr int stream_waves(int D, int GS, int NT) {
  if (NT == 1) return D == 64 ? (GS == 64 ? 4 : 3) : D / GS <= 2 ? 3 : 2;
  return D == 64 || D / GS <= 2 ? 2 : 1;
}

// Steps whose registers a wave of an eight-wave block holds (256 registers a lane there).
constexpr int whole_sets(int D, int BITS, int GS, int NT) {
  return D == 64 || (BITS == 4 ? NT == 1 || D / GS <= 2 : NT == 1 && D / GS <= 2) ? 2 : 1;
}

// The work of a launch: units of 128 keys of every (sequence, row tile, KV head), in one order, cut into
// equal shares, one a block.  A block walks the pieces ("segments") of its share; a pair that several
// blocks share leaves a partial result per segment, a pair within one share is finished there.
// Lengths live on the device, so every wave works the cut out for itself.
struct Share {
  uint32_t per, more;  // units of a block; the first `more` blocks have one more
  __device__ uint32_t begin(uint32_t i) const { return i * per + min(i, more); }
  __device__ uint32_t block_of(uint32_t u) const {
    const uint32_t wide = more * (per + 1);
    return u < wide ? u / (per + 1) : more + (u - wide) / per;
  }
};

template <int NT>
__device__ __forceinline__ uint32_t tiles_of(const AttnArgs& a, int tq) {
  return (uint32_t)(tq * a.per + 16 * NT - 1) / (16 * NT);
}
// A pair's units: kStartUnits without keys for what it costs to begin one (queries, page table, first
// loads, joining the waves: about as long as three units), then those of its keys.
__device__ __forceinline__ uint32_t units_of(int len) { return kStartUnits + (uint32_t)(len + kUnitKeys - 1) / kUnitKeys; }

// PAIR: pages of at least 32 tokens, so a step's two tiles share a page (one lookup, one address).
// MODE (StreamMode): shares as above, four waves a block; or a block takes a whole pair with eight waves or with four: what short
// sequences want, with no schedule to work out and nothing to join.
// kSharesOnce: shares of pairs whose rows are one tile each, so that no other block reads the keys: their loads pass the
// caches by (16 sequences of 16384-32768 keys, 64 heads on 8: 88 us, 95 with ordinary loads; where several tiles of rows read the
// keys the caches serve the later ones: 104 rows on 5834 keys in 8 bits 27 us, 34 past the caches).
template <int D, int BITS, int GS, int NT, bool PAIR, int MODE>
__global__ __launch_bounds__(MODE == kWhole8 ? 512 : 256, MODE == kWhole8 ? 2 : stream_waves(D, GS, NT)) void k_kv_stream(
    AttnArgs a) {
  constexpr bool ONCE = MODE == kSharesOnce, SPLIT = ONCE || MODE == kShares;
  using G = Geo<D, BITS>;
  constexpr int NG = D / GS;
  constexpr int kLdsRow = D + 4;
  constexpr int W = MODE == kWhole8 ? 8 : 4;  // waves
  constexpr int SETS = MODE == kWhole8 ? whole_sets(D, BITS, GS, NT) : 1, kStride = 32 * W;  // steps whose registers are held; keys of a block's step
  __shared__ __attribute__((aligned(16))) float sh_o[W][16][kLdsRow];
  __shared__ float sh_m[W][16 * NT], sh_l[W][16 * NT];

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, h = lane >> 4;
  const int page = 1 << a.f.page_shift;

  // ---- the block's share, and where it begins
  KeyList list = SPLIT && a.first_list ? a.list[1] : a.list[0];
  Share share{0, 0};
  uint32_t u = 0, u_end = 0, u_begin = 0, pair = 0, x0 = 0, pairs = 0;  // pairs: in front of this one
  int seq = 0;
  if (SPLIT) {
  // units and pairs up to and with each lane's sequence, 64 sequences at a time
  struct Scan {
    uint32_t units, pairs, own_units, own_pairs;
  };
  auto scan = [&](const KeyList& l, int s0) {
    Scan x{0, 0, 0, 0};
    if (s0 + lane < l.num_seqs) {
      const Sequence s = sequence_of<false>(a, l, s0 + lane);
      x.own_pairs = tiles_of<NT>(a, s.tq) * a.f.hkv;
      x.own_units = units_of(s.len) * x.own_pairs;
    }
    x.units = x.own_units, x.pairs = x.own_pairs;
    if (l.num_seqs > 1) {
#pragma unroll
      for (int i = 1; i < 64; i <<= 1) {
        const uint32_t y = __shfl_up(x.units, i), z = __shfl_up(x.pairs, i);
        if (lane >= i) x.units += y, x.pairs += z;
      }
    } else {
      x.units = __shfl(x.units, 0), x.pairs = __shfl(x.pairs, 0);
    }
    return x;
  };
  const int last = a.first_list + a.lists - 1;
  const Scan first_scan = scan(list, 0);
  uint32_t total = __shfl(first_scan.units, 63);
  if (list.num_seqs > 64 || a.lists > 1) {
    for (int li = a.first_list; li <= last; ++li) {
      const KeyList l = li ? a.list[1] : a.list[0];
      for (int s0 = li == a.first_list ? 64 : 0; s0 < l.num_seqs; s0 += 64) total += __shfl(scan(l, s0).units, 63);
    }
  }
  total = __builtin_amdgcn_readfirstlane(total);
  const uint32_t blocks = min((uint32_t)a.blocks, total);
  if (blockIdx.x >= blocks) return;
  const uint32_t per_block = __builtin_amdgcn_readfirstlane(total / blocks);
  share = Share{per_block, total - per_block * blocks};
  u = u_begin = share.begin(blockIdx.x);
  u_end = share.begin(blockIdx.x + 1);
  int li = a.first_list;
  uint32_t before = 0;  // units in front of the sequence
  Scan x = first_scan;
  for (int s0 = 0;;) {
    const uint64_t past = __ballot(before + x.units > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      seq = s0 + at;
      before += __shfl(x.units - x.own_units, at);
      pairs += __shfl(x.pairs - x.own_pairs, at);
      break;
    }
    before += __shfl(x.units, 63);
    pairs += __shfl(x.pairs, 63);
    s0 += 64;
    if (s0 >= (li ? a.list[1].num_seqs : a.list[0].num_seqs)) ++li, s0 = 0;
    x = scan(li ? a.list[1] : a.list[0], s0);
  }
  seq = __builtin_amdgcn_readfirstlane(seq);
  before = __builtin_amdgcn_readfirstlane(before);
  pairs = __builtin_amdgcn_readfirstlane(pairs);
  list = li ? a.list[1] : a.list[0];
  // within the sequence: tile * hkv + KV head, and the first unit of the segment
  const uint32_t each = units_of(sequence_of<true>(a, list, seq).len);
  pair = __builtin_amdgcn_readfirstlane((u - before) / each);
  x0 = (u - before) - pair * each;
  pairs += pair;
  } else {
    // (pairs of one sequence go round the XCDs, whatever its tile)
    const uint32_t x = (blockIdx.x + blockIdx.y) % gridDim.x;
    seq = x / a.f.hkv;
    pair = blockIdx.y * a.f.hkv + x % a.f.hkv;
    u_end = 0x7fffffff;
  }
  Sequence sq_ = sequence_of<true>(a, list, seq);
  if (!SPLIT && pair >= tiles_of<NT>(a, sq_.tq) * a.f.hkv) return;
  uint32_t units = units_of(sq_.len);

  while (true) {
  const int q0 = sq_.q0, tq = sq_.tq, len = sq_.len;
  const int tile = __builtin_amdgcn_readfirstlane(pair / a.f.hkv), hk = pair - tile * a.f.hkv;
  const uint32_t x1 = min(units, x0 + (u_end - u));
  const int rows = tq * a.per;
  const int row0 = tile * 16 * NT;
  const int last_t = __builtin_amdgcn_readfirstlane((min(row0 + 16 * NT, rows) - 1) / a.per);
  const int end_all = list.causal ? min(len, max(0, len - tq + last_t + 1)) : len;
  const int kb = max((int)x0 - (int)kStartUnits, 0) * kUnitKeys;
  const int ke = min(max((int)x1 - (int)kStartUnits, 0) * kUnitKeys, end_all);
  const int first_t = __builtin_amdgcn_readfirstlane(row0 / a.per);
  const int end_min = list.causal ? len - tq + first_t + 1 : len;  // keys below it are seen by every row

  // ---- queries, page ids and the wave's first keys are on their way before any of them is waited for
  u32x4 qw[NT][G::kMf];
  int rt[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = row0 + 16 * t + n;
    rt[t] = r < rows ? r / a.per : -1;
    const int token = max(rt[t], 0), head = r < rows ? r - token * a.per : 0;
    const uint16_t* p =
        reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(q0 + token) * a.q_ts + (int64_t)(hk * a.per + head) * a.q_hs + 8 * h;
#pragma unroll
    for (int i = 0; i < G::kMf; ++i) qw[t][i] = *reinterpret_cast<const u32x4*>(p + 32 * i);
  }
  uint32_t k_off = n * G::kRow + h * (G::kRow / 4);
  uint32_t v_off = page * G::kRow + (h * 16 + n) * (4 * G::kUnit);
  uint32_t km_off = 2 * page * G::kRow + 16 * h;
  uint32_t vm_off = km_off + 4 * page * (NG + (n * (D / 16)) / GS);
  const int32_t* table = list.table + (int64_t)seq * list.table_stride;

  const int last_page = max(list.table_cols - 1, 0);  // (a table without columns: any readable entry)
  auto place_of = [&](int key0) {
    Place x;
    x.bad = 0;
#pragma unroll
    for (int t = 0; t < (PAIR ? 1 : 2); ++t) {
      // (the entry is loaded before the length that says whether it counts has arrived)
      const int key = key0 + 16 * t;
      const uint32_t id = entry(table, min(key >> a.f.page_shift, last_page));
      const bool ok = key < ke && id < a.f.num_pages;
      x.bad |= ok ? 0u : (PAIR ? 3u : 1u << t);
      x.base[t] = a.f.pages + (uint64_t)(ok ? id : 0) * (uint64_t)a.f.page_bytes + hk * a.f.block_bytes;
    }
    if (PAIR) x.base[1] = x.base[0], x.bad |= key0 + 16 < ke ? 0u : 2u;
    return x;
  };
  auto fetch_k = [&](int key0, const Place& x, StepK<D, BITS, NG>& s) {
    // (opaque per step, so that the lane's 32-bit offset stays one next to the wave's 64-bit address)
    asm volatile("" : "+v"(k_off), "+v"(km_off));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* base = x.base[t];
      const int off = (PAIR ? key0 : key0 + 16 * t) & (page - 1), more = PAIR ? 16 * t : 0;
      load_words<ONCE>(base + off * G::kRow + k_off + more * G::kRow, s.c[t]);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        s.m[t][g] = load<ONCE, u32x4>(base + (off + g * page) * 4 + km_off + more * 4);
    }
  };
  auto fetch_v = [&](int key0, const Place& x, StepV<D, BITS>& s) {
    asm volatile("" : "+v"(v_off), "+v"(vm_off));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* base = x.base[t];
      const int off = (PAIR ? key0 : key0 + 16 * t) & (page - 1), more = PAIR ? 16 * t : 0;
      load_words<ONCE>(base + off * G::kRow + v_off + more * G::kRow, s.c[t]);
      s.m[t] = load<ONCE, u32x4>(base + off * 4 + vm_off + more * 4);
    }
  };
  const int first = kb + 32 * wave;
  Stage<D, BITS, NG> stage[SETS];
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    stage[i].now = place_of(first + i * kStride);
    stage[i].then = place_of(first + (SETS + i) * kStride);
  }
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    // (without keys here: some tokens of page 0, unused)
    const int key0 = first + i * kStride;
    fetch_k(key0, stage[i].now, stage[i].k);
    fetch_v(key0, stage[i].now, stage[i].v);
  }

  // ---- queries: rows in fp16 with a power of two of their own, sums per group
  h8 qf[NT][G::kMf];
  float sq[NT][NG], cs[NT];
  int lim[NT];  // last key the lane's row sees
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const bool there = rt[t] >= 0;
    u32x4(&w)[G::kMf] = qw[t];
    // the row's largest value by its bits (their order is that of the magnitudes, in either type)
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < G::kMf; ++i) {
      if (!there) w[i] = u32x4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) most = __builtin_elementwise_max(most, as_u16x2(w[i][j] & 0x7fff7fffu));
    }
    uint32_t top = max((uint32_t)most.x, (uint32_t)most.y);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    // a row with an infinity gives NaN wherever it sees a key, as one with NaN does (infinite products of one sign alone
    // would look like a row without keys)
    if (top >= (a.dtype == HQQ_KV_BF16 ? 0x7f80u : 0x7c00u)) w[0][0] = 0x7fff7fffu;
    // 2^e takes it to [2^14, 2^15) (fp16 rows: e up to 15): q / 16 then keeps fp16's precision for 2^13
    // below it, and a bfloat16 row of any size keeps its bits
    int e = 0;
    if (a.dtype == HQQ_KV_BF16) {
      const int x = top >> 7;
      if (x != 0 && x != 255) e = min(14 + 127 - x, 100);
#pragma unroll
      for (int i = 0; i < G::kMf; ++i) {
        float x8[8];
        floats8<true>(w[i], x8);
#pragma unroll
        for (int j = 0; j < 8; ++j) qf[t][i][j] = (_Float16)ldexpf(x8[j], BITS == 4 && (j & 2) ? e - 4 : e);
      }
    } else {
      const int x = top >> 10;
      if (top != 0 && x != 31) e = min(14 + 15 - x, 15);
      const _Float16 up = (_Float16)ldexpf(1.f, e), up4 = (_Float16)ldexpf(1.f, BITS == 4 ? e - 4 : e);
#pragma unroll
      for (int i = 0; i < G::kMf; ++i) {
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = as_u32(as_h2(w[i][j]) * (j & 1 ? h2{up4, up4} : h2{up, up}));
        qf[t][i] = __builtin_bit_cast(h8, y);
      }
    }
    cs[t] = ldexpf(a.scale_log2, 24 - e);
    const h2 one = {(_Float16)1.f, (_Float16)1.f}, back = {(_Float16)16.f, (_Float16)16.f};
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int i = g * GS / 32; i < (g + 1) * GS / 32; ++i) {
        const u32x4 y = __builtin_bit_cast(u32x4, qf[t][i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = __builtin_amdgcn_fdot2(as_h2(y[j]), BITS == 4 && (j & 1) ? back : one, sum, false);
      }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      sq[t][g] = sum * 0x1p-24f;  // the scale of the codes' products
    }
    lim[t] = there ? (list.causal ? min(len - 1, len - tq + rt[t]) : len - 1) : -1;
  }

  // ---- the stream
  Masks mk;
  asm("s_mov_b32 %0, 0x000f000f" : "=s"(mk.lo));
  asm("s_mov_b32 %0, 0x00f000f0" : "=s"(mk.hi));
  asm("v_mov_b32 %0, 0x64006400" : "=v"(mk.or1024));
  asm("v_mov_b32 %0, 0x54005400" : "=v"(mk.or64));
  float zero;  // (opaque: a fused step and floor instead of a conversion and a product)
  asm("v_mov_b32 %0, 0" : "=v"(zero));
  f32x4 o[NT][G::kVm], fl[NT];  // channels (4h + i) * (D/16) + j; floors' sums of those units
  float mref[NT], l[NT];  // running maximum (of the scores before cs) and sum
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    mref[t] = kNoKey / fmaxf(cs[t], 1.f), l[t] = 0.f;
    fl[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < G::kVm; ++j) o[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  auto step = [&](int key0, Stage<D, BITS, NG>& g) {
    StepK<D, BITS, NG>& sk = g.k;
    StepV<D, BITS>& sv = g.v;
    const uint32_t bad = g.now.bad;
    // scores
    float p[NT][8];
#pragma unroll
    for (int t2 = 0; t2 < 2; ++t2) {
      f32x4 acc[NT][NG];
#pragma unroll
      for (int i = 0; i < G::kMf; ++i) {
        u32x4 w;
        if (BITS == 4) {
          const uint32_t c = sk.c[t2][i], d = c >> 8;
          w = u32x4{c & mk.lo, c & mk.hi, d & mk.lo, d & mk.hi};
        } else {
          const uint32_t c = sk.c[t2][2 * i], d = sk.c[t2][2 * i + 1];
          w = u32x4{__builtin_amdgcn_perm(0, c, 0x0c010c00), __builtin_amdgcn_perm(0, c, 0x0c030c02),
                    __builtin_amdgcn_perm(0, d, 0x0c010c00), __builtin_amdgcn_perm(0, d, 0x0c030c02)};
        }
        const h8 kf = __builtin_bit_cast(h8, w);
        const int g = i * 32 / GS;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 from = i * 32 % GS == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[t][g];
          acc[t][g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[t][i], from, 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float x = zero;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const h2 m = as_h2((uint32_t)sk.m[t2][g][c]);
            x = fmaf((float)m.y, sq[t][g], x);
            x = fmaf(acc[t][g][c], (float)m.x, x);
          }
          p[t][4 * t2 + c] = x;
        }
      }
    }
    // the next keys take the registers of these, the next values those of this step's further down
    // (the scores are done before: else these registers are copied)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 8; ++c) asm volatile("" : "+v"(p[t][c]));
    const bool more = key0 + SETS * kStride < ke;
    if (more) fetch_k(key0 + SETS * kStride, g.then, sk);
    if (bad | (uint32_t)(key0 + 32 > end_min) | (uint32_t)(key0 + 32 > len)) {
      // keys that a row does not see (by selection: whatever their memory holds), and floors and
      // steps of keys that are not there
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2) {
        const bool gone = bad >> t2 & 1;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int key = key0 + 16 * t2 + 4 * h + c;
#pragma unroll
          for (int t = 0; t < NT; ++t)
            p[t][4 * t2 + c] = gone || key > lim[t] ? -INFINITY : p[t][4 * t2 + c];
          sv.m[t2][c] = gone || key >= len ? 0u : (uint32_t)sv.m[t2][c];
        }
      }
    }
    // values: steps and floors of the lane's unit as pairs of keys
    h2 st[4], fm[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = sv.m[i >> 1][2 * (i & 1)], y = sv.m[i >> 1][2 * (i & 1) + 1];
      st[i] = as_h2(__builtin_amdgcn_perm(y, x, 0x05040100));
      fm[i] = as_h2(__builtin_amdgcn_perm(y, x, 0x07060302));
    }
    h8 pf[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top = p[t][0];
#pragma unroll
      for (int c = 1; c < 8; ++c) top = fmaxf(top, p[t][c]);
      if (__any((top - mref[t]) * cs[t] > 5.f)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float next = (top - mref[t]) * cs[t] > 5.f ? top : mref[t];  // (each row by its own scores alone)
        const float f = exp2_((mref[t] - next) * cs[t]);
        mref[t] = next;
        l[t] *= f;
#pragma unroll
        for (int j = 0; j < G::kVm; ++j) o[t][j] *= f;
        fl[t] *= f;
      }
      // exponents: one fused operation, whose constant's rounding is nothing until scores of 2^20; from there on the
      // difference first, so that the largest score's is 0 and none passes the largest number (a row without a key so
      // far, or of NaN, does not count)
      const float c0 = fmaf(-mref[t], cs[t], kLift);
      const bool far = fabsf(c0) > 0x1p20f && mref[t] > kNoKey / 1e17f;
      if (__builtin_expect(__any(far), 0)) {
#pragma unroll
        for (int c = 0; c < 8; ++c) p[t][c] = far ? fmaf(p[t][c] - mref[t], cs[t], kLift) : fmaf(p[t][c], cs[t], c0);
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) p[t][c] = fmaf(p[t][c], cs[t], c0);
      }
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        p[t][c] = exp2_(p[t][c]);
        sum += p[t][c];
      }
      l[t] += sum;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const f32x2 e = {p[t][2 * c], p[t][2 * c + 1]};
        const h2 r = __builtin_convertvector(e, h2);
        pf[t][2 * c] = r.x, pf[t][2 * c + 1] = r.y;
      }
    }
    u32x4 flw;
#pragma unroll
    for (int i = 0; i < 4; ++i) flw[i] = as_u32(fm[i]);
    const h8 ff = __builtin_bit_cast(h8, flw);
#pragma unroll
    for (int t = 0; t < NT; ++t) fl[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(ff, pf[t], fl[t], 0, 0, 0);
    // values: dword i of operand b of the lane's units, from two tokens' words of codes, steps, and -1024 and -64 steps
    auto value = [&](uint32_t wx, uint32_t wy, int b, int i, h2 s, h2 s1024, h2 s64, u32x4& lo, u32x4& hi) {
      const uint32_t c = __builtin_amdgcn_perm(wy, wx, pair_sel<G::kUnit>(2 * (i & 1), b));
      const h2 x = as_h2(BITS == 4 ? (c & mk.lo) | mk.or1024 : c | mk.or1024);
      lo[i] = as_u32(__builtin_elementwise_fma(x, s, s1024));
      if (BITS == 4) {
        const h2 y = as_h2((c & mk.hi) | mk.or64);
        hi[i] = as_u32(__builtin_elementwise_fma(y, s, s64));
      }
    };
    auto word = [&](int b, int i, int t) { return sv.c[i >> 1][((2 * (i & 1) + t) * G::kUnit + b) / 4]; };
    const h2 n1024 = {(_Float16)-1024.f, (_Float16)-1024.f}, n64 = {(_Float16)-64.f, (_Float16)-64.f};
    // 1024 s passes fp16 for steps of 64 and more, and c s where a group is wider than it: entries whose step is 32 or
    // more (its half plus 0x3000 reaches the sign) are taken by themselves, 2^-8 smaller, and then the others without them, so that
    // these keep their bits.  Groups that wide, 480 and more in 4 bits, are rare, and so is the way (where all are: 36 us for 25 at 32
    // sequences of 65-4096 keys, 32 heads on 8); it holds no registers (opaque operands: else the compiler works out in front
    // what both ways share).
    auto past = [](uint32_t s) { return (s + 0x30003000u) >> 15 & 0x00010001u; };
    const u16x2 s01 = __builtin_elementwise_max(as_u16x2(as_u32(st[0])), as_u16x2(as_u32(st[1])));
    const u16x2 s23 = __builtin_elementwise_max(as_u16x2(as_u32(st[2])), as_u16x2(as_u32(st[3])));
    if (__any(past(__builtin_bit_cast(uint32_t, __builtin_elementwise_max(s01, s23))))) {
#pragma unroll
      for (int b = 0; b < G::kUnit; ++b) {
        u32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t wx = word(b, i, 0), wy = word(b, i, 1), s = as_u32(st[i]);
          asm volatile("" : "+v"(wx), "+v"(wy), "+v"(s));
          const h2 large = as_h2(past(s) * 0xffffu & s) * h2{(_Float16)0x1p-8f, (_Float16)0x1p-8f};
          value(wx, wy, b, i, large, large * n1024, large * n64, lo, hi);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const f32x4 none = {0.f, 0.f, 0.f, 0.f};
          const int j = BITS == 4 ? 2 * b : b;
          o[t][j] += 256.f * __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, lo), pf[t], none, 0, 0, 0);
          if (BITS == 4) o[t][j + 1] += 256.f * __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, hi), pf[t], none, 0, 0, 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) st[i] = as_h2(as_u32(st[i]) & ~(past(as_u32(st[i])) * 0xffffu));
    }
    h2 s1024[4], s64[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s1024[i] = st[i] * n1024;
      if (BITS == 4) s64[i] = st[i] * n64;
    }
#pragma unroll
    for (int b = 0; b < G::kUnit; ++b) {
      u32x4 lo, hi;
#pragma unroll
      for (int i = 0; i < 4; ++i) value(word(b, i, 0), word(b, i, 1), b, i, st[i], s1024[i], s64[i], lo, hi);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (BITS == 4) {
          o[t][2 * b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, lo), pf[t], o[t][2 * b], 0, 0, 0);
          o[t][2 * b + 1] =
              __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, hi), pf[t], o[t][2 * b + 1], 0, 0, 0);
        } else {
          o[t][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, lo), pf[t], o[t][b], 0, 0, 0);
        }
      }
    }
    if (more) fetch_v(key0 + SETS * kStride, g.then, sv);
    g.now = g.then;
    g.then = place_of(key0 + 2 * SETS * kStride);
  };
  for (int key0 = first; key0 < ke; key0 += SETS * kStride) {
#pragma unroll
    for (int i = 0; i < SETS; ++i)
      if (i == 0 || key0 + i * kStride < ke) step(key0 + i * kStride, stage[i]);
  }

  // ---- the block's waves joined, then written
  const bool whole = x0 == 0 && x1 == units;
  // a pair's segment: of the block's share the first one or the last one; with a join of both lists every
  // pair leaves one (blocks and pairs in front: each further segment adds one to the sum)
  const uint32_t segment = a.joined ? blockIdx.x + pairs : 2 * blockIdx.x + (u == u_begin ? 0 : 1);
  if (SPLIT && x0 == 0 && threadIdx.x == 0 && list.segments) {
    const int64_t at = ((int64_t)seq * tiles_of<NT>(a, list.max_q) + tile) * a.f.hkv + hk;
    list.segments[2 * at] = segment;
    list.segments[2 * at + 1] = whole && !a.joined ? 0 : (int)(share.block_of(u + units - 1) - blockIdx.x + 1);
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    mref[t] = fmaf(mref[t], cs[t], -kLift);  // what the weights are over, in units of the exponent, from here on
    l[t] += __shfl_xor(l[t], 16);
    l[t] += __shfl_xor(l[t], 32);
    if (h == 0) sh_m[wave][16 * t + n] = mref[t], sh_l[wave][16 * t + n] = l[t];
  }
  __syncthreads();
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float mm = sh_m[0][16 * t + n];
#pragma unroll
    for (int w = 1; w < W; ++w) mm = fmaxf(mm, sh_m[w][16 * t + n]);
    const float f = exp2_(mref[t] - mm);
    if (t) __syncthreads();  // the tile before has been read
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < G::kVm; j += 4) {
        f32x4 x;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) x[jj] = (o[t][j + jj][i] + fl[t][i]) * f;
        *reinterpret_cast<f32x4*>(&sh_o[wave][n][(4 * h + i) * (D / 16) + j]) = x;
      }
    __syncthreads();
    // 16 rows, CH channels a thread
    constexpr int CH = D / (4 * W), VEC = CH < 4 ? 2 : 4;
    typedef float vec __attribute__((ext_vector_type(VEC)));
    const int r = threadIdx.x / (4 * W), d0 = threadIdx.x % (4 * W) * CH;
    const int row = row0 + 16 * t + r;
    if (row < rows) {
      float rm = sh_m[0][16 * t + r];
#pragma unroll
      for (int w = 1; w < W; ++w) rm = fmaxf(rm, sh_m[w][16 * t + r]);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) sum += sh_l[w][16 * t + r] * exp2_(sh_m[w][16 * t + r] - rm);
      const int64_t at = (int64_t)(q0 + row / a.per) * a.hq + hk * a.per + row % a.per;
      vec x[CH / VEC];
#pragma unroll
      for (int j = 0; j < CH / VEC; ++j) {
        x[j] = *reinterpret_cast<const vec*>(&sh_o[0][r][d0 + j * VEC]);
#pragma unroll
        for (int w = 1; w < W; ++w) x[j] += *reinterpret_cast<const vec*>(&sh_o[w][r][d0 + j * VEC]);
      }
      if (!whole || a.joined) {
        const int64_t part = list.part0 + (SPLIT ? (int64_t)segment * list.cap + 16 * t + r : at);
        if (d0 == 0) a.part_ml[part] = float2{rm, sum};
        float* to = a.part_o + part * D + d0;
        if (sum != 0.f)  // (an empty part's sums are never read)
#pragma unroll
          for (int j = 0; j < CH / VEC; ++j) *reinterpret_cast<vec*>(to + j * VEC) = x[j];
      } else {
        const float inv = sum != 0.f ? 1.0f / sum : 0.f;
        uint16_t* to = reinterpret_cast<uint16_t*>(a.out) + at * D + d0;
#pragma unroll
        for (int j = 0; j < CH / VEC; ++j) {
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            const float y0 = x[j][i] * inv, y1 = x[j][i + 1] * inv;
            *reinterpret_cast<uint32_t*>(to + j * VEC + i) = a.dtype == HQQ_KV_BF16 ? pack2<true>(y0, y1) : pack2_held(y0, y1);
          }
        }
        if (a.lse && d0 == 0) a.lse[at] = sum != 0.f ? (rm + __log2f(sum)) * 0.69314718056f : -INFINITY;
      }
    }
  }

  // ---- the next pair
  if (!SPLIT) break;
  u += x1 - x0;
  if (u >= u_end) break;
  ++pair, ++pairs;
  x0 = 0;
  if (pair >= tiles_of<NT>(a, tq) * a.f.hkv) {
    pair = 0;
    do {
      if (++seq >= list.num_seqs) list = a.list[1], seq = 0;
      sq_ = sequence_of<true>(a, list, seq);
    } while (sq_.tq == 0);
    units = units_of(sq_.len);
  }
  __syncthreads();  // the joined rows have been read
  }
}

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

int tiles_in(const AttnArgs& a, const KeyList& l, int nt) {
  return (int)(((int64_t)l.max_q * a.per + 16 * nt - 1) / (16 * nt));
}

template <int D, int BITS, int GS, int NT, bool PAIR>
void stream_nt(const AttnArgs& a, hipStream_t st) {
  const KeyList& l = a.list[a.first_list];
  const dim3 grid(a.f.hkv * l.num_seqs, tiles_in(a, l, NT));
  switch (stream_mode(a, NT)) {
    case kSharesOnce: k_kv_stream<D, BITS, GS, NT, PAIR, kSharesOnce><<<a.blocks, 256, 0, st>>>(a); break;
    case kShares: k_kv_stream<D, BITS, GS, NT, PAIR, kShares><<<a.blocks, 256, 0, st>>>(a); break;
    case kWhole8: k_kv_stream<D, BITS, GS, NT, PAIR, kWhole8><<<grid, 512, 0, st>>>(a); break;
    case kWhole4: k_kv_stream<D, BITS, GS, NT, PAIR, kWhole4><<<grid, 256, 0, st>>>(a); break;
  }
}

template <int D, int BITS, int GS>
hipError_t stream_t(const AttnArgs& a, int nt, hipStream_t st) {
  const bool pair = a.f.page_shift >= 5;
  if (nt == 2)
    pair ? stream_nt<D, BITS, GS, 2, true>(a, st) : stream_nt<D, BITS, GS, 2, false>(a, st);
  else
    pair ? stream_nt<D, BITS, GS, 1, true>(a, st) : stream_nt<D, BITS, GS, 1, false>(a, st);
  return hipGetLastError();
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
  if (D == d && bits == b && gs == g) return stream_t<d, b, g>(a, nt, st);
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

}  // namespace kv
}  // namespace hqq
