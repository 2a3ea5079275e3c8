// Paged attention of long chunks of new tokens over a cache in 8 bits (kda_attn_tiles.hpp).
#include "kda_attn_tiles.hpp"

namespace kda {
namespace {

template <typename E, int DIM, int NW, int CODE> hipError_t tiles_go(const AttnQ8Launch& L) {
  const int64_t tiles = (int64_t)L.total * L.group / (32 * NW) + L.n;
  hipLaunchKernelGGL((tiles_kernel<AttnQ8Launch, E, DIM, NW, CODE>),
                     dim3((unsigned)(tiles * L.hkv), (unsigned)L.splits), dim3(64 * NW), 0,
                     (hipStream_t)L.stream, L);
  return hipGetLastError();
}
template <typename E, int DIM, int NW> hipError_t tiles_code(const AttnQ8Launch& L) {
  return L.code == E4M3 ? tiles_go<E, DIM, NW, E4M3>(L) : tiles_go<E, DIM, NW, INT8>(L);
}
template <typename E, int DIM> hipError_t tiles_nw(const AttnQ8Launch& L) {
  return L.tile_waves == 8 ? tiles_code<E, DIM, 8>(L) : tiles_code<E, DIM, 4>(L);
}
template <typename E> hipError_t tiles_dim(const AttnQ8Launch& L) {
  return L.dim == 64 ? tiles_nw<E, 64>(L) : tiles_nw<E, 128>(L);
}

}  // namespace

hipError_t launch_attn_q8_tiles(const AttnQ8Launch& L) {
  return L.dtype == 1 ? tiles_dim<bf16>(L) : tiles_dim<_Float16>(L);
}

}  // namespace kda
