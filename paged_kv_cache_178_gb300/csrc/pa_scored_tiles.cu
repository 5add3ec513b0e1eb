// pa_paged_attention_scored for many rows: the host's part.
#include <cstdio>

#include "pa_scored_tiles.cuh"

namespace pa {

extern template cudaError_t launch_tiles<128, 2>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
extern template cudaError_t launch_tiles<128, 1>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
extern template cudaError_t launch_tiles<256, 1>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
extern template cudaError_t launch_tiles<512, 1>(const ScoreParams &, const CUtensorMap (&)[3], const TileWork &, int, cudaStream_t);
extern template cudaError_t tiles_attributes<128, 2>();
extern template cudaError_t tiles_attributes<128, 1>();
extern template cudaError_t tiles_attributes<256, 1>();
extern template cudaError_t tiles_attributes<512, 1>();

// Two row tiles of 128 share their keys where a request can fill them (head
// dim 128: tensor memory has room for both outputs).
static int row_tiles(int group, int32_t head_dim, int32_t max_query_len)
{
    return head_dim == 128 && (int64_t)max_query_len * group > 128 ? 2 : 1;
}

int64_t scored_tiles_bound(int32_t num_seqs, int group, int32_t head_dim, int32_t max_query_len, int64_t num_q_tokens)
{
    const int rows = 128 * row_tiles(group, head_dim, max_query_len);
    const int64_t by_len = num_seqs * (((int64_t)max_query_len * group + rows - 1) / rows);
    const int64_t by_tokens = num_q_tokens * group / rows + num_seqs;
    return by_len < by_tokens ? by_len : by_tokens;
}

bool scored_tiles_fits(int32_t num_seqs, int32_t hkv, int group, int32_t head_dim, int32_t max_query_len,
                       int32_t max_seq_len, int64_t num_q_tokens)
{
    if (num_q_tokens < 0)
        return true;  // (a workspace's size: the call itself is refused)
    const int64_t tiles = scored_tiles_bound(num_seqs, group, head_dim, max_query_len, num_q_tokens);
    return num_seqs + tiles + 2 <= kScoredMaxEntriesHost &&
           tiles * hkv * 2 * (((int64_t)max_seq_len + kTileKeys - 1) / kTileKeys + 1 + kGroupSetup<2>) <= INT32_MAX;
}

static size_t align256(size_t n) { return (n + 255) / 256 * 256; }

struct TileSizes {
    int nt;
    int64_t record_floats;
    size_t records, bytes;  // offset, and the whole
};

static TileSizes tile_sizes(int group, int32_t head_dim, int32_t max_query_len)
{
    TileSizes s{};
    s.nt = row_tiles(group, head_dim, max_query_len);
    s.record_floats = s.nt * tile_record(head_dim == 512 ? 256 : head_dim);
    s.records = align256((size_t)kScoredSms * sizeof(int4));
    s.bytes = s.records + (size_t)2 * kScoredSms * s.record_floats * 4;
    return s;
}

size_t scored_tiles_bytes(int group, int32_t head_dim, int32_t max_query_len)
{
    return tile_sizes(group, head_dim, max_query_len).bytes;
}

cudaError_t launch_scored_tiles(const ScoreParams &p, int32_t head_dim, void *workspace, cudaStream_t stream, char *info,
                                size_t info_len)
{
    CUtensorMap pool[2], tm[3] = {};
    if (!scored_pool_maps(p, head_dim, pool))
        return cudaErrorInvalidValue;
    tm[0] = pool[0], tm[1] = pool[1];
    const bool q_boxes = 128 % p.group == 0;
    if (q_boxes) {
        const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)p.hq, (cuuint64_t)p.num_q_tokens};
        const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)p.q_tok_stride * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(128 / p.group)};
        if (encode_tiled(&tm[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(p.q), dims, strides, box,
                         CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const TileSizes s = tile_sizes(p.group, head_dim, p.max_query_len);
    const int64_t tiles = scored_tiles_bound(p.num_seqs, p.group, head_dim, p.max_query_len, p.num_q_tokens);
    TileWork w{};
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    w.tails = reinterpret_cast<int4 *>(ws);
    w.records = reinterpret_cast<float *>(ws + s.records);
    w.record_floats = s.record_floats;
    w.q_boxes = q_boxes;
    const int64_t items = tiles * p.hkv * (head_dim == 512 ? 2 : 1) * (((int64_t)p.max_seq_len + kTileKeys - 1) / kTileKeys + 1 + kGroupSetup<2>);
    w.ctas = (int32_t)(items < kScoredSms ? items : kScoredSms);
    w.max_tiles = (int32_t)tiles;
    // Without a maximum the exponents stay within the cap: 2^80 times any number
    // of keys and values up to 2^20 is far from overflow (and a row that overflows
    // all the same is computed again key by key).  Where all scores lie at the negative
    // cap, values below 2^-46 lose bits: their products pass fp32's smallest normal.
    const int mode = p.cap_log2 > kCapNarrow          ? kModeWide
                     : p.slopes                       ? kModeAny
                     : p.cap_log2 > 0.f               ? kModeCapped
                                                      : kModePlain;
    snprintf(info, info_len, "scored attention dh=%d kernel=tiles-m%d mode=%d grid=%d tiles=%lld", head_dim, 128 * s.nt, mode,
             w.ctas, (long long)tiles);
    switch (head_dim) {
    case 128: return s.nt == 2 ? launch_tiles<128, 2>(p, tm, w, mode, stream) : launch_tiles<128, 1>(p, tm, w, mode, stream);
    case 256: return launch_tiles<256, 1>(p, tm, w, mode, stream);
    default: return launch_tiles<512, 1>(p, tm, w, mode, stream);
    }
}

cudaError_t init_scored_tiles_attributes()
{
    cudaError_t e;
    if ((e = tiles_attributes<128, 2>()) != cudaSuccess || (e = tiles_attributes<128, 1>()) != cudaSuccess ||
        (e = tiles_attributes<256, 1>()) != cudaSuccess)
        return e;
    return tiles_attributes<512, 1>();
}

}  // namespace pa
