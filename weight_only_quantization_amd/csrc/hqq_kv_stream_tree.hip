// Attention of a tree of drafted tokens over a quantised key/value cache: the stream with a mask over a sequence's last
// keys (hqq_kv_stream.h; in a file of its own, which compiles beside hqq_kv_stream.hip).  The mask is read where a step reaches the drafts, so
// the others cost what they cost without: 26 drafts on 1049 keys, 32 heads, take 12 us, five steps of a block of eight waves.
#include "hqq_kv_stream.h"

namespace hqq {
namespace kv {

hipError_t launch_kv_stream_tree(const AttnArgs& a, int D, int bits, int gs, int nt, hipStream_t st) {
#define X(d, b, g) \
  if (D == d && bits == b && gs == g) return stream_t<d, b, g, true>(a, nt, st);
  X(64, 4, 32) X(64, 4, 64) X(64, 8, 32) X(64, 8, 64) X(128, 4, 32) X(128, 4, 64) X(128, 4, 128) X(128, 8, 32)
  X(128, 8, 64) X(128, 8, 128)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace kv
}  // namespace hqq
