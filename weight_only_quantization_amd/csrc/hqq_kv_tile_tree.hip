// Tiles over a sequence's keys that end in drafted tokens (hqq_kv_tile.h).
//
// The batch's lengths differ, and a draft has few tiles of rows, so fixed key splits would leave the longest sequence's
// blocks to run alone: the tiles of all (sequence, row tile, KV head) are cut into equal shares, one a block, as the stream's
// units are (hqq_kv_stream.h), and pairs that several blocks share leave partial results for the join.
//
// 16 sequences of 200-4096 keys, 16-32 drafts, 32 heads on 8, 8 bits: 44 us, and 6 for the join; a block has 1.4 pieces, each of 7.5 us
// beside 2.6 us a tile, and 2.2 us go by before it knows its first.  8 sequences of 9000-16384 keys, 64 drafts, 64 heads on 8, 4 bits:
// 213 Gflop in 240-250 us between the calls of a row (0.87 Pflop/s, as the prompts' tiles), and 12 for the join.
#include "hqq_kv_tile.h"

namespace hqq {
namespace kv {
namespace {

template <int R>
__device__ __forceinline__ uint32_t row_tiles_of(const AttnArgs& a, int tq) {
  return (uint32_t)(tq * a.per + R - 1) / R;
}
// Tiles that beginning and ending a (sequence, row tile, KV head) counts for: 7.5 us (queries and the first codes 3.4, its
// unpacking 0.6, sums and stores 3.5), at 2.6 us a tile of 128 rows and 4.5 of 256 (ragged drafts of 16 sequences, 128 rows: 57 us with 2,
// 54.5 with 3, 55.5 with 4).  Shares may end within them: the pair then begins with the block that has its first tile (60.5 us where
// both blocks began it).
constexpr uint32_t tile_start(int kg) { return kg == 2 ? 3 : 2; }

template <int D, int BITS, int GS, int KG>
__global__ __launch_bounds__(512, 2) void k_kv_tile_shares(AttnArgs a) {
  constexpr int R = kRows / KG;
  constexpr uint32_t kStart = tile_start(KG);
  auto units_of = [](int len) { return kStart + (uint32_t)(len + kKeys - 1) / kKeys; };
  static_assert(kKeys == kUnitKeys, "");
  const KeyList list = a.list[0];
  __shared__ __attribute__((aligned(16))) TilesK<D> sh_k;
  __shared__ __attribute__((aligned(16))) TilesV<D> sh_v;
  __shared__ float2 sh_ml[8][64];
  __shared__ int sh_holes[4];
  // (as in k_kv_tile)
  __builtin_amdgcn_s_setreg(1 | 23 << 6, 1);

  // ---- the block's share, and where it begins: units and pairs up to and with each lane's sequence, 64 at a time
  const int lane = threadIdx.x & 63;
  struct Scan {
    Sequence s;
    uint32_t units, pairs, own_units, own_pairs;
  };
  auto scan = [&](int s0) {
    Scan x{};
    if (s0 + lane < list.num_seqs) {
      x.s = sequence_of<false>(a, list, s0 + lane);
      x.own_pairs = row_tiles_of<R>(a, x.s.tq) * a.f.hkv;
      x.own_units = units_of(x.s.len) * x.own_pairs;
    }
    x.units = x.own_units, x.pairs = x.own_pairs;
#pragma unroll
    for (int i = 1; i < 64; i <<= 1) {
      const uint32_t y = __shfl_up(x.units, i), z = __shfl_up(x.pairs, i);
      if (lane >= i) x.units += y, x.pairs += z;
    }
    return x;
  };
  Scan x = scan(0);
  uint32_t total = __shfl(x.units, 63);
  for (int s0 = 64; s0 < list.num_seqs; s0 += 64) total += __shfl(scan(s0).units, 63);
  total = __builtin_amdgcn_readfirstlane(total);
  const uint32_t blocks = min((uint32_t)a.blocks, total);
  if (blockIdx.x >= blocks) return;
  const uint32_t per_block = __builtin_amdgcn_readfirstlane(total / blocks);
  const Share share{per_block, total - per_block * blocks};
  const uint32_t u_begin = share.begin(blockIdx.x), u_end = share.begin(blockIdx.x + 1);
  uint32_t u = u_begin, before = 0, pairs = 0;  // units and pairs in front of the sequence
  int seq = 0;
  Sequence s;
  for (int s0 = 0;; s0 += 64, x = scan(s0)) {
    const uint64_t past = __ballot(before + x.units > u);
    if (past) {
      const int at = __builtin_ctzll(past);
      seq = s0 + at;
      before += __shfl(x.units - x.own_units, at);
      pairs += __shfl(x.pairs - x.own_pairs, at);
      s = {__builtin_amdgcn_readlane(x.s.q0, at), __builtin_amdgcn_readlane(x.s.tq, at), __builtin_amdgcn_readlane(x.s.len, at)};
      break;
    }
    before += __shfl(x.units, 63);
    pairs += __shfl(x.pairs, 63);
  }
  seq = __builtin_amdgcn_readfirstlane(seq);
  before = __builtin_amdgcn_readfirstlane(before);
  pairs = __builtin_amdgcn_readfirstlane(pairs);
  uint32_t units = units_of(s.len);
  uint32_t pair = __builtin_amdgcn_readfirstlane((u - before) / units), x0 = (u - before) - pair * units;  // tile * hkv + KV head
  pairs += pair;

  while (true) {
    const int tile = __builtin_amdgcn_readfirstlane(pair / a.f.hkv), hk = pair - tile * a.f.hkv;
    const uint32_t x1 = min(units, x0 + (u_end - u));
    const int kb = max((int)x0 - (int)kStart, 0) * kKeys;
    const int ke = min(max((int)x1 - (int)kStart, 0) * kKeys, s.len);
    // A pair begins with the block that has its first tile (a block whose share ends before it leaves the pair to the next).
    const bool begins = x0 <= kStart, whole = begins && x1 == units;
    if (x1 > kStart || x1 == units) {
      // (segments are numbered as the stream's are)
      const uint32_t segment = a.joined ? blockIdx.x + pairs : 2 * blockIdx.x + (u == u_begin ? 0 : 1);
      if (begins && threadIdx.x == 0) {
        const int64_t at = ((int64_t)seq * row_tiles_of<R>(a, list.max_q) + tile) * a.f.hkv + hk;
        list.segments[2 * at] = segment;
        list.segments[2 * at + 1] = whole && !a.joined ? 0 : (int)(share.block_of(u - x0 + units - 1) - blockIdx.x + 1);
      }
      tile_pair<D, BITS, GS, true, KG>(a, list, s, seq, hk, tile * R, kb, ke, !whole || a.joined, list.part0 + (int64_t)segment * list.cap,
                                       sh_k, sh_v, sh_ml, sh_holes);
    }
    u += x1 - x0;
    if (u >= u_end) break;
    ++pair, ++pairs;
    x0 = 0;
    if (pair >= row_tiles_of<R>(a, s.tq) * a.f.hkv) {
      pair = 0;
      do s = sequence_of<true>(a, list, ++seq);
      while (s.tq == 0);
      units = units_of(s.len);
    }
    __syncthreads();  // the tiles and the halves' sums have been read
  }
}

template <int D, int BITS, int GS>
hipError_t shares_t(const AttnArgs& a, int rows, hipStream_t st) {
  if (rows == kRows)
    k_kv_tile_shares<D, BITS, GS, 1><<<a.blocks, 512, 0, st>>>(a);
  else
    k_kv_tile_shares<D, BITS, GS, 2><<<a.blocks, 512, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_tile_tree(const AttnArgs& a, int rows, int D, int bits, int gs, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return shares_t<d, b, g>(a, rows, st);
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128) X(128, 8, 32)
  X(128, 8, 64) X(128, 8, 128)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace hqq
