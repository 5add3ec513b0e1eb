// pa_paged_attention_scored for many rows: head dim 128.
#include "pa_scored_tiles.cuh"

namespace pa {

template cudaError_t launch_tiles<128, 2>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
template cudaError_t tiles_attributes<128, 2>();
template cudaError_t launch_tiles<128, 1>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
template cudaError_t tiles_attributes<128, 1>();

}  // namespace pa
