// The gated delta rule, token by token:
//     e = v_t - exp(g_t) S k_t,  S <- exp(g_t) S + beta_t e k_t^T,  y_t = S q_t.
// The rows of S (value channels) do not see one another, so a CTA owns 16 rows of one (sequence,
// head): eight lanes share a row, each with N / 8 of its columns in registers for the whole sequence.
// The row products reduce over the eight lanes. Bound by the latency of one token (two dependent
// reductions); every type and length takes it.
#include "common.cuh"
#include "delta.cuh"

namespace wkv7 {
namespace {

constexpr int kScanRows = 16, kLanes = 8;

__device__ __forceinline__ float sum8(float x) {
#pragma unroll
    for (int o = 4; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16(x); }

template <class Tin, int NN>
__global__ void __launch_bounds__(kScanRows *kLanes) delta_scan_kernel(const DeltaArgs p) {
    constexpr int G = NN / (4 * kLanes);        // float4 groups per lane: columns 4 * (lane + 8 m)
    const int slices = NN / kScanRows;
    const unsigned unit = blockIdx.x / slices;  // (sequence, head)
    const int s = unit / p.H, h = unit % p.H, hk = h / (p.H / p.Hk);
    const int lane = threadIdx.x % kLanes, row = (blockIdx.x % slices) * kScanRows + threadIdx.x / kLanes;
    long long t0, t1;
    delta_rows(p.cu, p.T, s, t0, t1);
    const Tin *q = static_cast<const Tin *>(p.q) + hk * NN, *k = static_cast<const Tin *>(p.k) + hk * NN;
    const Tin *v = static_cast<const Tin *>(p.v) + h * NN + row;
    const Tin *g = static_cast<const Tin *>(p.g) + h, *beta = static_cast<const Tin *>(p.beta) + h;
    Tin *y = static_cast<Tin *>(p.y) + h * NN + row;
    const size_t so = (size_t(unit) * NN + row) * NN;
    float4 S[G];
#pragma unroll
    for (int m = 0; m < G; ++m)
        S[m] = p.S0 ? __ldg(reinterpret_cast<const float4 *>(p.S0 + so + 4 * (lane + kLanes * m))) : make_float4(0, 0, 0, 0);
    for (long long t = t0; t < t1; ++t) {
        float4 k4[G], q4[G];
        float kn = 0.f, qn = 0.f, sk = 0.f;
#pragma unroll
        for (int m = 0; m < G; ++m) {
            k4[m] = load4(k + t * p.ks + 4 * (lane + kLanes * m));
            q4[m] = load4(q + t * p.qs + 4 * (lane + kLanes * m));
            kn += dot4(k4[m], k4[m]);
            qn += dot4(q4[m], q4[m]);
            sk += dot4(S[m], k4[m]);
        }
        sk = sum8(sk);
        float rk = 1.f, rq = p.scale;
        if (p.qk_norm) {
            rk = rsqrtf(sum8(kn) + p.norm_eps);
            rq *= rsqrtf(sum8(qn) + p.norm_eps);
        }
        const float a = expf(delta_clamp(load1(g + t * p.H))), b = load1(beta + t * p.H);
        const float u = b * (load1(v + t * p.vs) - a * rk * sk) * rk;
        float yv = 0.f;
#pragma unroll
        for (int m = 0; m < G; ++m) {
            S[m].x = fmaf(u, k4[m].x, a * S[m].x);
            S[m].y = fmaf(u, k4[m].y, a * S[m].y);
            S[m].z = fmaf(u, k4[m].z, a * S[m].z);
            S[m].w = fmaf(u, k4[m].w, a * S[m].w);
            yv += dot4(S[m], q4[m]);
        }
        yv = sum8(yv) * rq;
        if (lane == 0) store1(y + t * p.H * NN, yv);
    }
    if (p.S_T) {
#pragma unroll
        for (int m = 0; m < G; ++m) *reinterpret_cast<float4 *>(p.S_T + so + 4 * (lane + kLanes * m)) = S[m];
    }
}

template <class Tin>
cudaError_t launch_t(const DeltaArgs &p) {
    const unsigned grid = unsigned(p.B) * p.H * (p.N / kScanRows);
    if (p.N == 128) delta_scan_kernel<Tin, 128><<<grid, kScanRows * kLanes, 0, p.stream>>>(p);
    else delta_scan_kernel<Tin, 64><<<grid, kScanRows * kLanes, 0, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

// ---- host side ---------------------------------------------------------------------------------------

cudaError_t launch_delta_forward(const DeltaArgs &p) {
    return p.dt == WKV7_BF16 ? launch_t<__nv_bfloat16>(p) : launch_t<float>(p);
}

}  // namespace wkv7
