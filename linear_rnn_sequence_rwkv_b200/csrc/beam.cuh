// Arguments of the beam-search entries after validation.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "wkv7.h"

namespace wkv7 {

struct BeamArgs {
    int B, K, V, M;
    wkv7_dtype dt;
    const void *logits;
    long long row_stride;           // elements
    const float *scores;
    const unsigned char *finished;  // nullable
    int eos;
    float *out_scores;
    int *parents, *tokens;
    void *ws;
    cudaStream_t stream;
};

size_t beam_select_workspace(int B, int K, int V, int M);
cudaError_t launch_beam_select(const BeamArgs &p);
// dst[l][b][j] = src[l][b][parents[b][j]], rows of row_bytes (a multiple of 16)
cudaError_t launch_beam_reorder(int L, int B, int K, size_t row_bytes, const int *parents, const void *src, void *dst,
                                cudaStream_t stream);

}  // namespace wkv7
