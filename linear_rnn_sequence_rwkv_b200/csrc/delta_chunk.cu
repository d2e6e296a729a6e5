// The gated delta rule's forward: the sweep of delta_sweep.cuh over every sequence and head.
#include "delta_sweep.cuh"

namespace wkv7 {

using namespace dm;

namespace {

template <int NN, int RW, bool F32, int GROUPS>
__global__ void __launch_bounds__(RW * 32 + GROUPS * kGroup, (!F32 && NN == 64 && GROUPS == 2) ? 2 : 1) delta_chunk_kernel(const DeltaArgs p) {
    forward_sweep<NN, RW, F32, false, GROUPS>(p, blockIdx.x);
}

}  // namespace

// ---- host side ---------------------------------------------------------------------------------------

cudaError_t allow_dynamic_smem(const void *kernel, int bytes);

namespace {

template <int NN, int RW, bool F32, int GROUPS>
cudaError_t launch_t(const DeltaArgs &p) {
    using L = Layout<NN, RW, F32, false, GROUPS>;
    const void *kernel = reinterpret_cast<const void *>(delta_chunk_kernel<NN, RW, F32, GROUPS>);
    const cudaError_t e = allow_dynamic_smem(kernel, L::total);
    if (e != cudaSuccess) return e;
    delta_chunk_kernel<NN, RW, F32, GROUPS><<<unsigned(p.B) * p.H * (NN / (16 * RW)), L::threads, L::total, p.stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_forward(const DeltaArgs &p) {
    if (p.dt == WKV7_F32) return p.N == 64 ? launch_t<64, 4, true, 2>(p) : launch_t<128, 4, true, 2>(p);
    // Rows per CTA: 64 (four warps, one per scheduler). N = 128 took 2.74 us per chunk so against 5.09 with all 128
    // rows in a CTA for 40 and 72 heads, and as long for 144. N = 64 with 32 rows and a third group that prepares
    // took 1.63 us against 1.90 for 40 heads, but 1.8 times as long for 512: taken while two CTAs per head fit the SMs.
    if (p.N == 128) return launch_t<128, 4, false, 2>(p);
    return (long long)p.B * p.H <= 74 ? launch_t<64, 2, false, 3>(p) : launch_t<64, 4, false, 2>(p);
}

}  // namespace wkv7
