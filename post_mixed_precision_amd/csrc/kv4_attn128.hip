// Attention over the 4-bit cache, heads of 128 channels (a file of its own: the
// kernels are compiled beside each other).
#include "kv4_attn.hpp"

namespace slim {
namespace kv4 {

hipError_t launch_dim128(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st) {
  if (a.group == 128) return launch_group<128, 128>(a, cut, p, st);
  return a.group == 64 ? launch_group<128, 64>(a, cut, p, st) : launch_group<128, 32>(a, cut, p, st);
}

}  // namespace kv4
}  // namespace slim
