// The tiles with a mask over a sequence's last keys, as hqq_kv_stream_tree.hip.
#include "hqq_kv_tile.h"

namespace hqq {
namespace kv {

hipError_t launch_kv_tile_tree(const AttnArgs& a, int which, int D, int bits, int gs, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return tile_t<d, b, g, true>(a, which, st);
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128) X(128, 8, 32)
  X(128, 8, 64) X(128, 8, 128)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace hqq
