// Beam search over recurrent states: the selection of the best continuations over beams and
// vocabulary, and the reordering of the states' rows.
//
// Selection reads the logits once. beam_part_kernel: a CTA takes a segment of one row into registers,
// sums its exponentials against its own maximum, and finds its M best elements as 64-bit keys
// (order-preserving bits of the value above the complement of the index, so that keys never tie and
// equal values go to the lowest index). The M-th largest of the 256 threads' own maxima is a floor
// for the M-th best element, and only the M threads at or above it can hold more, so the elements that
// pass the floor fit a buffer of M times a thread's elements whatever the input. beam_pick_kernel: one
// CTA per request joins the segments' sums in fp64, merges the sorted lists of a row and then those
// of the rows. An element's place in a merged list is its place in its own plus, for every other list,
// how many there precede it (a binary search), so nothing is sorted twice. Bound by the logits' bytes
// where the batch is large, by two launches where it is small.
#include "beam.cuh"

#include <cuda_bf16.h>

namespace wkv7 {
namespace {

constexpr int kT = 256;                 // threads of beam_part_kernel
constexpr int kPickT = 512;
constexpr unsigned long long kOne = 1;

struct Part {
    float top;      // largest logit of the segment (-inf: none)
    float pad;
    double sum;     // sum of exp(logit - top)
};

// Order-preserving bits of a float; 0 for -inf and NaN, which are never chosen.
__device__ __forceinline__ uint32_t order_bits(float x) {
    if (!(x > -INFINITY)) return 0u;
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ unsigned long long make_key(float x, uint32_t index) {
    const uint32_t o = order_bits(x == 0.f ? 0.f : x);   // -0 and +0 are the same score
    return o ? ((unsigned long long)o << 32) | (0xffffffffu - index) : 0ull;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes from p, which lies `shift` elements behind a 16-byte boundary: the two aligned vectors
// around it, shifted together. Rows of an odd vocabulary start anywhere; equal rows must be cut into
// the same vectors all the same, so that their sums, and with them ties between beams, come out equal.
template <class Tin>
__device__ __forceinline__ uint4 load_shifted(const Tin *p, int shift) {
    const uint4 *a = reinterpret_cast<const uint4 *>(p - shift);
    if (shift == 0) return __ldg(a);
    const uint4 u = __ldg(a), v = __ldg(a + 1);
    uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    const int bytes = shift * int(sizeof(Tin));
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (bytes & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack(const uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Sorts one key per lane over the warp, largest in lane 0.
__device__ __forceinline__ unsigned long long warp_sort_desc(unsigned long long k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride; stride >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, k, stride);
            const bool keep_max = ((lane & stride) == 0) == ((lane & size) == 0);
            k = (keep_max == (o > k)) ? o : k;
        }
    return k;
}

// How many of the n keys, sorted from the largest down, are above x.
__device__ __forceinline__ int count_above(const unsigned long long *list, int n, unsigned long long x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[mid] > x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

template <class Tin, int EPT>
__global__ void __launch_bounds__(kT) beam_part_kernel(const BeamArgs p, int splits) {
    constexpr int VW = 16 / sizeof(Tin), NV = EPT / VW, SEG = kT * EPT;
    extern __shared__ unsigned long long cand[];          // [M * EPT]
    __shared__ unsigned long long s_sort[kT / 32][32], s_floor;
    __shared__ float s_top[kT / 32];
    __shared__ double s_sum[kT / 32];
    __shared__ int s_n;
    const int row = blockIdx.x / unsigned(splits), split = blockIdx.x % unsigned(splits);
    if (p.finished && p.finished[row]) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Tin *base = static_cast<const Tin *>(p.logits) + (long long)row * p.row_stride;
    const int shift = int((reinterpret_cast<uintptr_t>(base) / sizeof(Tin)) % VW);
    const int beyond = shift ? VW - shift : 0;            // elements that a shifted load reads behind its own
    const long long at = (long long)split * SEG + (long long)tid * VW;
    float x[EPT];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const long long i = at + (long long)j * kT * VW;
        float t[VW];
        if (i + VW + beyond <= p.V) {
            unpack(load_shifted(base + i, shift), t);
        } else {
#pragma unroll
            for (int e = 0; e < VW; ++e) t[e] = i + e < p.V ? to_f(base[i + e]) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < VW; ++e) x[j * VW + e] = t[e];
    }
    if (tid == 0) {
        s_floor = 1;
        s_n = 0;
    }
    // the thread's largest element, first of equals (NaN fails every comparison)
    float top = -INFINITY;
    int arg = 0;
#pragma unroll
    for (int e = 0; e < EPT; ++e)
        if (x[e] > top) {
            top = x[e];
            arg = e;
        }
    const uint32_t first = uint32_t(at + (long long)(arg / VW) * kT * VW + arg % VW);
    const unsigned long long mine = make_key(top, first);
    const unsigned long long sorted = warp_sort_desc(mine);
    s_sort[warp][lane] = sorted;
    float wtop = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) wtop = fmaxf(wtop, __shfl_xor_sync(0xffffffffu, wtop, o));
    if (lane == 0) s_top[warp] = wtop;
    __syncthreads();
    float ctop = s_top[0];
#pragma unroll
    for (int w = 1; w < kT / 32; ++w) ctop = fmaxf(ctop, s_top[w]);
    // the M-th largest of the threads' maxima
    if (lane < p.M && sorted) {
        int rank = lane;
#pragma unroll
        for (int w = 0; w < kT / 32; ++w)
            if (w != warp) rank += count_above(s_sort[w], 32, sorted);
        if (rank == p.M - 1) s_floor = sorted;
    }
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < EPT; ++e) sum += x[e] > -INFINITY ? __expf(x[e] - ctop) : 0.f;
    double ds = sum;
#pragma unroll
    for (int o = 16; o; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
    if (lane == 0) s_sum[warp] = ds;
    __syncthreads();
    const unsigned long long low = s_floor;
    if (mine >= low) {
#pragma unroll
        for (int e = 0; e < EPT; ++e) {
            const unsigned long long key = make_key(x[e], uint32_t(at + (long long)(e / VW) * kT * VW + e % VW));
            if (key >= low) cand[atomicAdd(&s_n, 1)] = key;
        }
    }
    __syncthreads();
    const int n = s_n;
    Part *part = static_cast<Part *>(p.ws);
    unsigned long long *list = reinterpret_cast<unsigned long long *>(part + size_t(p.B) * p.K * splits) +
                               size_t(blockIdx.x) * p.M;
    for (int i = tid; i < n; i += kT) {
        const unsigned long long c = cand[i];
        int rank = 0;
        for (int j = 0; j < n; ++j) rank += cand[j] > c;
        if (rank < p.M) list[rank] = c;
    }
    for (int i = n + tid; i < p.M; i += kT) list[i] = 0;
    if (tid == 0) {
        double t = 0.;
#pragma unroll
        for (int w = 0; w < kT / 32; ++w) t += s_sum[w];
        part[blockIdx.x] = Part{ctop, 0.f, t};
    }
}

__global__ void __launch_bounds__(kPickT) beam_pick_kernel(const BeamArgs p, int splits) {
    extern __shared__ unsigned long long dyn[];
    __shared__ double s_norm[WKV7_BEAM_MAX];
    __shared__ int s_have[WKV7_BEAM_MAX];
    const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int K = p.K, M = p.M;
    unsigned long long *best = dyn;                                  // [K][M] keys of each row
    double *score = reinterpret_cast<double *>(dyn + size_t(K) * M);   // [K][M]
    const Part *part = static_cast<const Part *>(p.ws) + size_t(b) * K * splits;
    const unsigned long long *lists = reinterpret_cast<const unsigned long long *>(
                                          static_cast<const Part *>(p.ws) + size_t(p.B) * K * splits) +
                                      size_t(b) * K * splits * M;
    for (int i = tid; i < K * M; i += kPickT) best[i] = 0;
    // the rows' normalisers
    for (int j = warp; j < K; j += kPickT / 32) {
        if (p.finished && p.finished[size_t(b) * K + j]) continue;
        float top = -INFINITY;
        for (int s = lane; s < splits; s += 32) top = fmaxf(top, part[j * splits + s].top);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        double sum = 0.;
        if (top > -INFINITY)
            for (int s = lane; s < splits; s += 32)
                if (part[j * splits + s].top > -INFINITY)
                    sum += part[j * splits + s].sum * exp(double(part[j * splits + s].top) - double(top));
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_norm[j] = double(top) + log(sum);      // NaN where the row has +inf or nothing
    }
    __syncthreads();
    // each row's M best of its segments' lists
    const int per_row = splits * M;
    for (int i = tid; i < K * per_row; i += kPickT) {
        const int j = i / per_row, r = i % per_row, s = r / M, pos = r % M;
        if (p.finished && p.finished[size_t(b) * K + j]) continue;
        const unsigned long long *row = lists + size_t(j) * per_row;
        const unsigned long long key = row[r];
        if (!key) continue;
        int rank = pos;
        for (int o = 0; o < splits && rank < M; ++o)
            if (o != s) rank += count_above(row + o * M, M, key);
        if (rank < M) best[j * M + rank] = key;
    }
    __syncthreads();
    for (int i = tid; i < K * M; i += kPickT) {
        const int j = i / M;
        const double own = p.scores[size_t(b) * K + j];
        double x = -INFINITY;
        if (p.finished && p.finished[size_t(b) * K + j]) {
            if (i % M == 0) {
                x = own;
                best[i] = 0xffffffffu - uint32_t(p.eos);
            }
        } else if (best[i]) {
            x = own + (double(order_value(uint32_t(best[i] >> 32))) - s_norm[j]);
        }
        score[i] = x > -INFINITY ? x : -INFINITY;          // NaN offers nothing
    }
    if (tid < K) s_have[tid] = 0;
    __syncthreads();
    for (int i = tid; i < K * M; i += kPickT)              // the valid ones are a prefix of the row
        if (score[i] > -INFINITY && (i % M == M - 1 || !(score[i + 1] > -INFINITY))) s_have[i / M] = i % M + 1;
    __syncthreads();
    for (int i = tid; i < K * M; i += kPickT) {
        const double x = score[i];
        if (!(x > -INFINITY)) continue;
        const int j = i / M;
        int rank = i % M;
        for (int o = 0; o < K && rank < M; ++o) {
            if (o == j) continue;
            int lo = 0, hi = s_have[o];
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                const double y = score[o * M + mid];
                if (y > x || (y == x && o < j)) lo = mid + 1;
                else hi = mid;
            }
            rank += lo;
        }
        if (rank < M) {
            const size_t at = size_t(b) * M + rank;
            p.out_scores[at] = float(x);
            p.parents[at] = j;
            p.tokens[at] = int(0xffffffffu - uint32_t(best[i] & 0xffffffffu));
        }
    }
    int have = 0;
    for (int o = 0; o < K; ++o) have += s_have[o];
    for (int i = have + tid; i < M; i += kPickT) {
        const size_t at = size_t(b) * M + i;
        p.out_scores[at] = -INFINITY;
        p.parents[at] = -1;
        p.tokens[at] = -1;
    }
}

// One thread per 16-byte (or 8-byte) column of a request's K rows: every row that changes is loaded
// from its source before any is stored, so the move is safe in place whatever the chains and cycles,
// and rows that stay cost nothing in place. KM bounds K for the registers that hold the column.
template <int KM, class Vec>
__global__ void __launch_bounds__(256) beam_reorder_kernel(int B, int K, size_t row_vecs, const int *__restrict__ parents,
                                                           const Vec *src, Vec *dst, unsigned cols) {
    const unsigned group = blockIdx.x / cols;                    // l * B + b
    const size_t c = size_t(blockIdx.x % cols) * blockDim.x + threadIdx.x;
    const int b = group % unsigned(B);
    const size_t at = size_t(group) * K * row_vecs + c;
    if (c >= row_vecs) return;
    const bool in_place = src == dst;
    Vec r[KM];
    unsigned long long moved = 0;
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (j < K) {
            int o = __ldg(parents + size_t(b) * K + j);
            if (unsigned(o) >= unsigned(K)) o = j;
            if (o != j || !in_place) {
                moved |= kOne << j;
                r[j] = src[at + size_t(o) * row_vecs];
            }
        }
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (moved >> j & 1) dst[at + size_t(j) * row_vecs] = r[j];
}

template <int KM, class Vec>
cudaError_t reorder_t(int L, int B, int K, size_t row_bytes, const int *parents, const void *src, void *dst,
                      cudaStream_t stream) {
    const size_t vecs = row_bytes / sizeof(Vec);
    const unsigned cols = unsigned((vecs + 255) / 256);
    beam_reorder_kernel<KM, Vec><<<unsigned(L) * unsigned(B) * cols, 256, 0, stream>>>(
        B, K, vecs, parents, static_cast<const Vec *>(src), static_cast<Vec *>(dst), cols);
    return cudaGetLastError();
}

// ---- host side ---------------------------------------------------------------------------------------

// Elements per thread of beam_part_kernel: 32, or 8 where 32 would leave SMs without a segment.
int elements_per_thread(int B, int K, int V) {
    return (long long)B * K * ((V - 1) / (kT * 32) + 1) < 2 * 148 ? 8 : 32;
}
int segments(int B, int K, int V) {
    const int seg = kT * elements_per_thread(B, K, V);
    return (V - 1) / seg + 1;
}

template <class Tin>
cudaError_t select_t(const BeamArgs &p) {
    const int splits = segments(p.B, p.K, p.V), ept = elements_per_thread(p.B, p.K, p.V);
    const unsigned grid = unsigned(p.B) * unsigned(p.K) * unsigned(splits);
    const size_t smem = size_t(p.M) * ept * 8;            // at most 16 KB
    if (ept == 8) beam_part_kernel<Tin, 8><<<grid, kT, smem, p.stream>>>(p, splits);
    else beam_part_kernel<Tin, 32><<<grid, kT, smem, p.stream>>>(p, splits);
    return cudaGetLastError();
}

}  // namespace

cudaError_t allow_dynamic_smem(const void *kernel, int bytes);

size_t beam_select_workspace(int B, int K, int V, int M) {
    return size_t(B) * K * segments(B, K, V) * (sizeof(Part) + size_t(M) * 8);
}

cudaError_t launch_beam_select(const BeamArgs &p) {
    const int smem = p.K * p.M * 16;                      // at most 64 KB
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(beam_pick_kernel), WKV7_BEAM_MAX * WKV7_BEAM_MAX * 16);
    if (e != cudaSuccess) return e;
    e = p.dt == WKV7_BF16 ? select_t<__nv_bfloat16>(p) : select_t<float>(p);
    if (e != cudaSuccess) return e;
    beam_pick_kernel<<<p.B, kPickT, smem, p.stream>>>(p, segments(p.B, p.K, p.V));
    return cudaGetLastError();
}

cudaError_t launch_beam_reorder(int L, int B, int K, size_t row_bytes, const int *parents, const void *src, void *dst,
                                cudaStream_t stream) {
    if (K <= 4) return reorder_t<4, float4>(L, B, K, row_bytes, parents, src, dst, stream);
    if (K <= 8) return reorder_t<8, float4>(L, B, K, row_bytes, parents, src, dst, stream);
    if (K <= 16) return reorder_t<16, float4>(L, B, K, row_bytes, parents, src, dst, stream);
    if (K <= 32) return reorder_t<32, float4>(L, B, K, row_bytes, parents, src, dst, stream);
    return reorder_t<64, float2>(L, B, K, row_bytes, parents, src, dst, stream);
}

}  // namespace wkv7
