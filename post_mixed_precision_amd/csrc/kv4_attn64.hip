// Attention over the 4-bit cache, heads of 64 channels (a file of its own: the
// kernels are compiled beside each other).
#include "kv4_attn.hpp"

namespace slim {
namespace kv4 {

hipError_t launch_dim64(const Kv4Args &a, const Kv4Cut &cut, const Kv4Plan &p, hipStream_t st) {
  return a.group == 64 ? launch_group<64, 64>(a, cut, p, st) : launch_group<64, 32>(a, cut, p, st);
}

}  // namespace kv4

hipError_t launch_kv4_attention(const Kv4Args &a, void *ws, const Kv4Plan &p, hipStream_t st) {
  const Kv4Cut cut = {(float *)ws, p.tm, __builtin_ctz(p.tm), p.tiles, p.slots, p.extra, p.least};
  return a.dim == 64    ? kv4::launch_dim64(a, cut, p, st)
         : a.dim == 128 ? kv4::launch_dim128(a, cut, p, st)
                        : kv4::launch_dim256(a, cut, p, st);
}

}  // namespace slim
