// pa_paged_attention_scored for many rows: head dim 512.
#include "pa_scored_tiles.cuh"

namespace pa {

template cudaError_t launch_tiles<512, 1>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
template cudaError_t tiles_attributes<512, 1>();

}  // namespace pa
