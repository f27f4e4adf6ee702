// Attention over the 4-bit cache, heads of 256 channels (a file of its own: the
// kernels are compiled beside each other).
#include "kv4_attn.hpp"

namespace slim {
namespace kv4 {

hipError_t launch_dim256(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st) {
  if (a.group == 128) return launch_group<256, 128>(a, cut, p, st);
  return a.group == 64 ? launch_group<256, 64>(a, cut, p, st) : launch_group<256, 32>(a, cut, p, st);
}

}  // namespace kv4
}  // namespace slim
