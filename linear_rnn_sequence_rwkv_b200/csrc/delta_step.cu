// One token of the gated delta rule for every row of a batch, against a pool of fp32 states:
//     e = v - exp(g) S k,  S <- exp(g) S + beta e k^T,  y = S q.
// 16 KB of state in and 16 KB out per head (N = 64) for 28 kflop: bound by HBM bandwidth. One CTA
// owns 16 KB, a (row, head) at N = 64 and a quarter of one at N = 128; a half-warp (N = 64) or a warp (N = 128) covers one
// row of the state with a float4 per lane, and all of a thread's four rows are loaded before any arithmetic. (32 rows of 40
// heads of N = 128, 168 MB: 28 us against 34 with half a state per CTA and 39 with a whole one, whose 16 rows per thread
// leave two CTAs to an SM.) 250 rows of 40 heads scattered over a
// pool of 320 slots (333 MB): 58 to 60 us, 5.7 TB/s, of 50.7 us at the rate of a plain copy; CTAs of 128 threads, 6 to 12
// to an SM, took 61 to 94 us against 61 on the same card.
// Rows that share a slot: the first of them carries the state through all of the others, in
// order; the others leave at once. Finding them costs one pass over the slots, which runs under the
// state's loads.
#include "common.cuh"
#include "delta.cuh"

namespace wkv7 {
namespace {

__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16(x); }

template <class Tin, int NN, int THREADS, int PARTS>
__global__ void __launch_bounds__(THREADS) delta_step_kernel(const DeltaArgs p) {
    constexpr int CL = NN / 4, RS = THREADS / CL, ROWS = NN / PARTS, RPT = ROWS / RS;
    const int part = blockIdx.x % PARTS;                   // of the state's rows, which never meet
    const int h = blockIdx.x / PARTS % unsigned(p.H), hk = h / (p.H / p.Hk);
    int b = blockIdx.x / PARTS / unsigned(p.H);
    const int c4 = threadIdx.x % CL, rbase = part * ROWS + threadIdx.x / CL;
    const Tin *q = static_cast<const Tin *>(p.q) + hk * NN + 4 * c4, *k = static_cast<const Tin *>(p.k) + hk * NN + 4 * c4;
    const Tin *v = static_cast<const Tin *>(p.v) + h * NN;
    const Tin *g = static_cast<const Tin *>(p.g) + h, *beta = static_cast<const Tin *>(p.beta) + h;
    Tin *y = static_cast<Tin *>(p.y) + h * NN;
    auto lanes_sum = [](float x) {
#pragma unroll
        for (int off = CL / 2; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        return x;
    };
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.n_slots) {        // padding: uniform over the CTA
        for (int i = threadIdx.x; i < ROWS; i += THREADS) store1(y + size_t(b) * p.H * NN + part * ROWS + i, 0.f);
        return;
    }
    float *S = p.S + (size_t(slot) * p.H + h) * NN * NN;
    float4 s[RPT];
#pragma unroll
    for (int m = 0; m < RPT; ++m) s[m] = __ldcs(reinterpret_cast<const float4 *>(S + (rbase + RS * m) * NN + 4 * c4));
    __shared__ int s_next;
    bool shared_slot = false;
    if (p.slots) {
        bool before = false, after = false;
        for (int i = threadIdx.x; i < p.B; i += THREADS) {
            const bool same = __ldg(p.slots + i) == slot;
            before |= same && i < b;
            after |= same && i > b;
        }
        if (__syncthreads_or(before)) return;
        shared_slot = __syncthreads_or(after);
    }
    while (true) {
        const float4 k4 = load4(k + b * p.ks), q4 = load4(q + b * p.qs);
        const float a = expf(delta_clamp(load1(g + size_t(b) * p.H))), bt = load1(beta + size_t(b) * p.H);
        float vi[RPT];
#pragma unroll
        for (int m = 0; m < RPT; ++m) vi[m] = load1(v + b * p.vs + rbase + RS * m);
        float rk = 1.f, rq = p.scale;
        if (p.qk_norm) {
            rk = delta_unit(lanes_sum(dot4(k4, k4)), p.norm_eps);
            rq *= delta_unit(lanes_sum(dot4(q4, q4)), p.norm_eps);
        }
#pragma unroll
        for (int m = 0; m < RPT; ++m) {
            const float sk = lanes_sum(dot4(s[m], k4));
            const float u = bt * rk * (vi[m] - a * rk * sk);
            s[m].x = fmaf(u, k4.x, a * s[m].x);
            s[m].y = fmaf(u, k4.y, a * s[m].y);
            s[m].z = fmaf(u, k4.z, a * s[m].z);
            s[m].w = fmaf(u, k4.w, a * s[m].w);
            const float yv = lanes_sum(dot4(s[m], q4)) * rq;
            if (c4 == 0) store1(y + size_t(b) * p.H * NN + rbase + RS * m, yv);
        }
        if (!shared_slot) break;
        // the next row with this slot
        if (threadIdx.x == 0) s_next = p.B;
        __syncthreads();
        for (int i = b + 1 + threadIdx.x; i < p.B; i += THREADS)
            if (__ldg(p.slots + i) == slot) {
                atomicMin(&s_next, i);
                break;
            }
        __syncthreads();
        const int nb = s_next;
        __syncthreads();
        if (nb >= p.B) break;
        b = nb;
    }
#pragma unroll
    for (int m = 0; m < RPT; ++m) __stcs(reinterpret_cast<float4 *>(S + (rbase + RS * m) * NN + 4 * c4), s[m]);
}

template <class Tin>
cudaError_t launch_t(const DeltaArgs &p) {
    const unsigned grid = unsigned(p.B) * unsigned(p.H);
    if (p.N == 128) delta_step_kernel<Tin, 128, 256, 4><<<4 * grid, 256, 0, p.stream>>>(p);
    else delta_step_kernel<Tin, 64, 256, 1><<<grid, 256, 0, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

// ---- host side ---------------------------------------------------------------------------------------

cudaError_t launch_delta_step(const DeltaArgs &p) {
    return p.dt == WKV7_BF16 ? launch_t<__nv_bfloat16>(p) : launch_t<float>(p);
}

}  // namespace wkv7
