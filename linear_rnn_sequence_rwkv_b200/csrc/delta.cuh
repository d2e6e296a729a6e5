// Arguments of the gated delta rule's kernels after validation, and what they share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "wkv7.h"

namespace wkv7 {

struct DeltaArgs {
    int B, T;               // sequences; tokens per sequence, or rows in all when packed
    int H, Hk, N;
    wkv7_dtype dt;
    const void *q, *k, *v, *g, *beta;
    const float *S0;        // nullable: zero initial state
    void *y;
    float *S_T;             // nullable
    const int *cu;          // nullable: B sequences of T tokens
    long long qs, ks, vs;   // row strides of q, k, v in elements
    float scale;
    int qk_norm;
    float norm_eps;
    // step: the pool
    float *S;
    int n_slots;
    const int *slots;       // nullable: row b takes slot b
    // backward
    const void *dy;
    const float *dS_T;      // nullable
    void *dq, *dk, *dv, *dg, *dbeta;
    float *dS0;             // nullable
    void *keep_E;           // workspace: the errors, [rows][H][N] (bf16: two terms, keep_lo elements apart)
    long long keep_lo;
    void *keep_dlo;         // workspace, bf16: the second term of dv
    void *keep_S, *keep_dS; // workspace: the state a chunk of 64 tokens starts from and its last state's gradient
    long long keep_second;  // bf16: elements from their first terms to the second
    float *keep_parts;      // workspace: dq, then dk, of each part of the value heads, parts_step elements each
    long long parts_step;
    int group;              // value heads of a key head
    cudaStream_t stream;
};

cudaError_t launch_delta_forward(const DeltaArgs &p);
cudaError_t launch_delta_step(const DeltaArgs &p);
cudaError_t launch_delta_backward(const DeltaArgs &p);      // two to four launches: the sweeps, the gradients, their sum
size_t delta_backward_workspace(size_t rows, int B, int H, int Hk, int N, wkv7_dtype dt);

// Chunks of 64 tokens are numbered over all sequences so that each has a place of its own without a pass over
// the lengths: sequence s starts at number (first row) / 64 + s, and there are at most rows / 64 + B.
__host__ __device__ __forceinline__ long long delta_slot(long long first_row, int s) { return first_row / 64 + s; }

// Rows [first, last) of sequence s. Packed bounds outside 0..T or decreasing are clamped, so that no
// row outside the buffers is reached.
__device__ __forceinline__ void delta_rows(const int *cu, int T, int s, long long &first, long long &last) {
    if (!cu) {
        first = (long long)s * T;
        last = first + T;
        return;
    }
    const int a = min(max(cu[s], 0), T), b = min(max(cu[s + 1], a), T);
    first = a;
    last = b;
}

// exp(g) of a log decay. Values below -120 (exp is 0 in fp32, denormals included), -inf among them,
// count as -120, so that differences of sums of decays stay finite; a NaN stays one.
__device__ __forceinline__ float delta_clamp(float g) { return g < -120.f ? -120.f : g; }

// What brings a vector of this sum of squares to unit length; NaN where the sum is not finite (it would be 0, and the
// vector silently the zero vector, where finite elements have squares beyond fp32).
__device__ __forceinline__ float delta_unit(float squares, float eps) { return rsqrtf(squares + eps) + 0.f * squares; }

}  // namespace wkv7
