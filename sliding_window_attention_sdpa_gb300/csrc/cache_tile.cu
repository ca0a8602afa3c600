// cache_tile.cu -- the tile kernel over a cache in its tensors' dtype.
#include "cache_tile.cuh"

namespace swa {

cudaError_t launch_cache_fwd_tiles(const CacheTileArgs& a, int dtype, cudaStream_t s)
{
    return launch_tiles_typed<false>(a, dtype, s);
}

}  // namespace swa
