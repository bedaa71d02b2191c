// Internal declarations of the group norm (group_norm.cu; entry points in group_norm_api.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace gla {

// Forward and backward (passed by value): x [N, S, C], groups of W = C / G channels.
struct GroupNormArgs {
    const void *x, *dy;
    const float *w, *b, *mean_in, *rstd_in;
    void *y, *dx;
    float *mean, *rstd, *dw, *db;
    float4 *part;                      // maps: [N][slices][entries] moments or sums of a slice's groups
    float *part_dw, *part_db;          // rows of C of partial sums
    int64_t N, S;
    int C, G, W;
    float eps;
    bool silu;
};

// How the maps' kernels cut a tensor.
struct GroupNormSplit {
    int rows, slices, chunk, chunks;   // positions of a slice, slices of a sample, channels of a chunk, chunks
    int tx, ty;                        // threads of a row, rows at a time
    int64_t entries;                   // partial results of a slice: its groups, and one more for each further chunk
};

bool group_norm_tokens(int64_t S, int W);   // whether the tokens' kernel takes it
int64_t group_norm_token_ctas(const GroupNormArgs &a, int dtype, bool back);
int64_t group_norm_token_parts(const GroupNormArgs &a, int dtype);
GroupNormSplit group_norm_split(const GroupNormArgs &a, int dtype);
cudaError_t launch_group_norm_tokens(const GroupNormArgs &a, int dtype, bool back, cudaStream_t s);
cudaError_t launch_group_norm_maps(const GroupNormArgs &a, const GroupNormSplit &sp, int dtype, bool back, int pass, cudaStream_t s);
cudaError_t launch_group_norm_dw(const GroupNormArgs &a, int64_t many, cudaStream_t s);

}  // namespace gla
