// Attention of many query rows over a quantised key/value cache: the launches of the tiles (hqq_kv_tile.h).
#include "hqq_kv_tile.h"

namespace hqq {
namespace kv {

hipError_t launch_kv_tile(const AttnArgs& a, int which, int D, int bits, int gs, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return tile_t<d, b, g>(a, which, st);
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128) X(128, 8, 32)
  X(128, 8, 64) X(128, 8, 128)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace hqq
