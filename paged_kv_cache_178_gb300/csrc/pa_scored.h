// Between the parts of pa_paged_attention_scored: the choice of a kernel
// (pa_scored.cu), few rows (pa_scored_rows.cu).
#pragma once
#include "pa_score.cuh"

namespace pa {

constexpr int kScoredSms = 152;              // CTAs of a wave are counted by it, on the host alone
constexpr int kScoredMaxTilesHost = 8192;    // requests times tiles of rows that a CTA sums over

// Tensor maps of K and V: boxes of 64 columns by the 16 tokens of one page and head.
bool scored_pool_maps(const ScoreParams &p, int32_t head_dim, CUtensorMap (&tm)[2]);

bool scored_rows_fits(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len,
                      int32_t max_seq_len);
size_t scored_rows_bytes(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len,
                         int32_t max_seq_len);
cudaError_t launch_scored_rows(const ScoreParams &p, int32_t head_dim, void *workspace, cudaStream_t stream, char *info,
                               size_t info_len);
cudaError_t init_scored_rows_attributes();

}  // namespace pa
