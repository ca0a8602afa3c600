// cache4_tile.cu -- the tile kernel over a cache in 4 bits.
#include "cache_tile.cuh"

namespace swa {

cudaError_t launch_cache4_fwd_tiles(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    const cudaError_t e = launch_tiles_typed<true>(a, dtype, s);
    return e != cudaSuccess ? e : launch_cache_fwd_join(a.f, dtype, 256, s);
}

}  // namespace swa
