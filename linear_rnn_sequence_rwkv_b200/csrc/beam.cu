// Beam search over recurrent states: the selection of the best continuations over beams and
// vocabulary, and the reordering of the states' rows.
//
// Selection reads the logits once. beam_part_kernel: a CTA takes a segment of one row into registers (packed, as
// loaded), sums its exponentials against its own maximum, and finds its M best elements. Each of the 8 warps finds
// the M/8-th largest of its threads' own maxima; the least of these is a floor for the M-th best element, and what
// reaches it (on logits without order about 5 M/2 elements) is gathered and placed by counting. Where the
// elements lie so that more than 2 M + 64 reach it, the M-th largest of all threads' maxima is the floor: what is
// above that lies in fewer than M threads. Only where more elements equal that floor than there is room for are they
// taken in the order of their index instead. The lists hold 64-bit keys, order-preserving bits of the value above the
// complement of the index, so that keys never tie and equal values go to the lowest index.
// beam_pick_kernel: one CTA per request joins the segments' sums in fp64, merges the sorted lists of a row and
// then those of the rows.
// 64 requests of 8 beams over 50277 bf16 logits (51.5 MB): 28 us, of which the segments 24 (2.1 TB/s; issue 62 %, 715
// instructions per warp of 1280 logits, 140 of them for the exponentials); 27 us where rows are aligned to 16 bytes.
// One request of 4 beams over 65536 fp32 logits: 8.4 us.
#include "beam.cuh"

#include <cuda_bf16.h>

#include <limits.h>

#include <algorithm>

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

// A thread's vectors from a row that starts SHIFT elements behind a 16-byte boundary: each is two aligned ones, shifted
// together. Rows of an odd vocabulary start anywhere; equal rows must be cut into the same vectors all the same, so that
// their sums, and with them ties between beams, come out equal. Vectors from behind `most` are left out, and so is the
// first where it `opens` a buffer that starts anywhere.
template <class Tin, int NV, int STEP, int SHIFT>
__device__ __forceinline__ void load_shifted(uint4 (&v)[NV], const Tin *row, int at, int most, bool opens) {
    constexpr int q = SHIFT * int(sizeof(Tin)) / 4, half = SHIFT * int(sizeof(Tin)) % 4;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = at + j * STEP;
        if (i > most || (j == 0 && opens)) continue;
        const uint4 *a = reinterpret_cast<const uint4 *>(row + i - SHIFT);
        if constexpr (SHIFT == 0) {
            v[j] = __ldg(a);
        } else {
            const uint4 x = __ldg(a), y = __ldg(a + 1);
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = half ? __funnelshift_r(w[k + q], w[min(k + q + 1, 7)], 16) : w[k + q];
            v[j] = make_uint4(r[0], r[1], r[2], r[3]);
        }
    }
}
template <int NV, int STEP>
__device__ __forceinline__ void load_row(uint4 (&v)[NV], const float *row, int shift, int at, int most, bool opens) {
    switch (shift) {
        case 0: return load_shifted<float, NV, STEP, 0>(v, row, at, most, opens);
        case 1: return load_shifted<float, NV, STEP, 1>(v, row, at, most, opens);
        case 2: return load_shifted<float, NV, STEP, 2>(v, row, at, most, opens);
        default: return load_shifted<float, NV, STEP, 3>(v, row, at, most, opens);
    }
}
template <int NV, int STEP>
__device__ __forceinline__ void load_row(uint4 (&v)[NV], const __nv_bfloat16 *row, int shift, int at, int most, bool opens) {
    switch (shift) {
        case 0: return load_shifted<__nv_bfloat16, NV, STEP, 0>(v, row, at, most, opens);
        case 1: return load_shifted<__nv_bfloat16, NV, STEP, 1>(v, row, at, most, opens);
        case 2: return load_shifted<__nv_bfloat16, NV, STEP, 2>(v, row, at, most, opens);
        case 3: return load_shifted<__nv_bfloat16, NV, STEP, 3>(v, row, at, most, opens);
        case 4: return load_shifted<__nv_bfloat16, NV, STEP, 4>(v, row, at, most, opens);
        case 5: return load_shifted<__nv_bfloat16, NV, STEP, 5>(v, row, at, most, opens);
        case 6: return load_shifted<__nv_bfloat16, NV, STEP, 6>(v, row, at, most, opens);
        default: return load_shifted<__nv_bfloat16, NV, STEP, 7>(v, row, at, most, opens);
    }
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

// The elements from i on of a row that ends before a whole vector does; -inf behind its end.
__device__ __forceinline__ uint4 load_edge(const float *p, int i, int n) {
    float t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = i + e < n ? p[i + e] : -INFINITY;
    return make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]), __float_as_uint(t[3]));
}
__device__ __forceinline__ uint4 load_edge(const __nv_bfloat16 *p, int i, int n) {
    const unsigned short *u = reinterpret_cast<const unsigned short *>(p);
    uint32_t t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = i + e < n ? u[i + e] : 0xff80u;
    return make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16);
}

// The thread's largest element (NaN only if all are).
template <int NV>
__device__ __forceinline__ float largest(const uint4 (&v)[NV], const float *) {
    float m = __uint_as_float(v[0].x);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float x[4];
        unpack(v[j], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, x[e]);
    }
    return m;
}
template <int NV>
__device__ __forceinline__ float largest(const uint4 (&v)[NV], const __nv_bfloat16 *) {
    auto b2 = [](const uint32_t &u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); };
    __nv_bfloat162 m = b2(v[0].x);
#pragma unroll
    for (int j = 0; j < NV; ++j) m = __hmax2(__hmax2(__hmax2(m, b2(v[j].x)), b2(v[j].y)), __hmax2(b2(v[j].z), b2(v[j].w)));
    return fmaxf(__low2float(m), __high2float(m));
}
// Which elements are at least `least`, a bit each: bf16 word 4 j + i of the first four vectors in bits 4 j + i (its first
// element) and 16 more (its second) of the first mask, of the others in the second; fp32 element 4 j + e in bit
// 4 j + e of the first. place(mask, bit): element of its vector + 8 or 4 times the vector's number.
template <int NV>
__device__ __forceinline__ void at_least(const uint4 (&v)[NV], float least, uint32_t (&mask)[2], const float *) {
    mask[0] = mask[1] = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float x[4];
        unpack(v[j], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) mask[0] |= x[e] >= least ? 1u << (4 * j + e) : 0u;
    }
}
template <int NV>
__device__ __forceinline__ void at_least(const uint4 (&v)[NV], float least, uint32_t (&mask)[2], const __nv_bfloat16 *) {
    const __nv_bfloat162 l = __float2bfloat162_rn(least);      // a logit: exact
    mask[0] = mask[1] = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mask[j >> 2] |= __hge2_mask(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), l) & (0x00010001u << (4 * (j & 3) + i));
    }
}
__device__ __forceinline__ int place(int, int bit, const float *) { return bit; }
__device__ __forceinline__ int place(int mask, int bit, const __nv_bfloat16 *) { return 32 * mask + 2 * (bit & 15) + (bit >> 4); }

__device__ __forceinline__ float value(const float *p) { return __ldg(p); }
__device__ __forceinline__ float value(const __nv_bfloat16 *p) {
    return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const unsigned short *>(p))) << 16);
}
// The least value that is above -inf.
__device__ __forceinline__ float lowest(const float *) { return __uint_as_float(0xff7fffffu); }
__device__ __forceinline__ float lowest(const __nv_bfloat16 *) { return __uint_as_float(0xff7f0000u); }

// Sorts one value per lane over the warp, largest in lane 0.
__device__ __forceinline__ uint32_t warp_sort_desc(uint32_t k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride; stride >>= 1) {
            const uint32_t o = __shfl_xor_sync(0xffffffffu, k, stride);
            k = ((lane & stride) == 0) == ((lane & size) == 0) ? max(k, o) : min(k, o);
        }
    return k;
}

// exp in three instructions, relative error about 1e-7 + 6e-8 |x| (a tiny result may become 0).
__device__ __forceinline__ float quick_exp(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// The same of x + c and y + c, and a sum of pairs: two numbers to an instruction.
__device__ __forceinline__ unsigned long long pair(float x, float y) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 halves(unsigned long long r) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ float2 quick_exp2(float x, float y, float c) {
    unsigned long long r;
    asm("{\n\t.reg .b64 t;\n\tadd.rn.f32x2 t, %1, %2;\n\tmul.rn.f32x2 %0, t, %3;\n\t}"
        : "=l"(r) : "l"(pair(x, y)), "l"(pair(c, c)), "l"(pair(1.4426950408889634f, 1.4426950408889634f)));
    float2 v = halves(r);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(v.y));
    return v;
}
__device__ __forceinline__ void add2(float2 &a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a.x, a.y)), "l"(pair(b.x, b.y)));
    a = halves(r);
}

// How many of the n keys, sorted from the largest down, are above x.
template <class U>
__device__ __forceinline__ int count_above(const U *list, int n, U x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (list[mid] > x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// What beam_part_kernel ranks without a second look, and what it has room for in all.
__host__ __device__ __forceinline__ int few_of(int M) { return 2 * M + 64; }
__host__ __device__ __forceinline__ int room_of(int M, int elements) {
    const int all = M * (elements + 1), few = few_of(M);
    return all > few ? all : few;
}

template <class Tin, int NV>
__global__ void __launch_bounds__(kT, NV > 4 ? 5 : 6) beam_part_kernel(const BeamArgs p, int splits) {
    constexpr int VW = 16 / sizeof(Tin), EPT = NV * VW, SEG = kT * EPT, W = kT / 32;
    extern __shared__ unsigned long long cand[];          // [room_of(M, EPT)]
    __shared__ uint32_t s_sort[W][32], s_floor, s_top[W], s_low[W];
    __shared__ double s_sum[W];
    __shared__ int s_n, s_ties[W];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");     // the picking kernel may take its place
    const int row = blockIdx.x / unsigned(splits), split = blockIdx.x % unsigned(splits);
    if (p.finished && p.finished[row]) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Tin *base = static_cast<const Tin *>(p.logits) + (long long)row * p.row_stride;
    const int shift = int((reinterpret_cast<uintptr_t>(base) / sizeof(Tin)) % VW);
    const int most = p.V - VW - (shift ? VW - shift : 0);  // last place from which a whole (shifted) vector may be read
    const int at = split * SEG + tid * VW;                 // V + 65536 fits an int
    uint4 v[NV] = {};
    const bool opens = shift != 0 && row == 0 && at == 0;
    load_row<NV, kT * VW>(v, base, shift, at, most, opens);
    if (opens) v[0] = load_edge(base, 0, p.V);
    if (at + (NV - 1) * kT * VW > most) {                  // the row ends here
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (at + j * kT * VW > most) v[j] = load_edge(base, at + j * kT * VW, p.V);
    }
    if (tid == 0) {
        s_floor = 0;
        s_n = 0;
    }
    const float top = largest<NV>(v, static_cast<const Tin *>(nullptr));
    const uint32_t own_top = order_bits(top == 0.f ? 0.f : top);
    // the warp's largest, and the last of as many as it has to hold for W warps to hold M
    uint32_t first = 0, last = 0, left = own_top;
    for (int i = 0; i < (p.M + W - 1) / W; ++i) {
        last = __reduce_max_sync(0xffffffffu, left);
        if (i == 0) first = last;
        if (__ffs(__ballot_sync(0xffffffffu, left == last)) - 1 == lane) left = 0;
    }
    if (lane == 0) {
        s_top[warp] = first;
        s_low[warp] = last;
    }
    __syncthreads();
    const uint32_t peak = __reduce_max_sync(0xffffffffu, s_top[lane % W]);
    uint32_t low = __reduce_min_sync(0xffffffffu, s_low[lane % W]);
    const float ctop = peak ? order_value(peak) : -INFINITY, ref = peak ? ctop : 0.f;
    float2 sums = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        float x[VW];
        unpack(v[j], x);
#pragma unroll
        for (int e = 0; e < VW; e += 2) add2(sums, quick_exp2(x[e], x[e + 1], -ref));
    }
    float sum = sums.x + sums.y;
    if (sum != sum) {                                      // a NaN among them counts as -inf
        sum = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float x[VW];
            unpack(v[j], x);
#pragma unroll
            for (int e = 0; e < VW; ++e) sum += quick_exp(fmaxf(x[e], -INFINITY) - ref);
        }
    }
    double ds = sum;
#pragma unroll
    for (int o = 16; o; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
    if (lane == 0) s_sum[warp] = ds;
    constexpr const Tin *type = nullptr;
    float least = low ? order_value(low) : lowest(type);
    // Calls f(value, index) for this thread's elements that reach the floor. They are few: their values are read again, so
    // that there is one copy of what is done with them and not one per element.
    auto each = [&](auto f) {
        if (!(top >= least)) return;
        uint32_t mask[2];
        at_least<NV>(v, least, mask, type);
#pragma unroll 1
        for (int m = 0; m < (NV * VW > 32 ? 2 : 1); ++m)
            for (uint32_t left = m ? mask[1] : mask[0]; left; left &= left - 1) {
                const int e = place(m, __ffs(left) - 1, type), i = at + e / VW * (kT * VW) + e % VW;
                f(value(base + i), i);
            }
    };
    auto gather = [&](int most) {
        each([&](float x, int i) {
            const int to = atomicAdd(&s_n, 1);
            if (to < most) cand[to] = make_key(x, uint32_t(i));
        });
        __syncthreads();
    };
    const int few = few_of(p.M), room = max(few, p.M * EPT);
    gather(few);
    int n = s_n;
    if (n > few) {              // the same with the best floor that the threads' maxima give
        __syncthreads();
        if (tid == 0) s_n = 0;
        // the M-th largest of the threads' maxima (0: fewer than M threads hold anything): up to 32, by merging the
        // sorted warps pairwise; above, by counting in the other warps' lists
        uint32_t sorted = warp_sort_desc(own_top);
        s_sort[warp][lane] = sorted;
        __syncthreads();
        if (p.M <= 32) {
#pragma unroll
            for (int step = 1; step < W; step *= 2) {
                __syncthreads();
                if (warp % (2 * step) == 0) {
                    sorted = max(sorted, s_sort[warp + step][31 - lane]);      // the 32 largest of both, rising then falling
#pragma unroll
                    for (int stride = 16; stride; stride >>= 1) {
                        const uint32_t o = __shfl_xor_sync(0xffffffffu, sorted, stride);
                        sorted = (lane & stride) == 0 ? max(sorted, o) : min(sorted, o);
                    }
                    s_sort[warp][lane] = sorted;
                }
            }
            if (warp == 0 && lane == p.M - 1) s_floor = sorted;
        } else if (sorted) {
            int above = lane, same = 0;                        // equal values: those of lower warps come first
            for (int w = 0; w < W; ++w)
                if (w != warp) {
                    const int a = count_above(s_sort[w], 32, sorted);
                    above += a;
                    if (w < warp) same += count_above(s_sort[w], 32, sorted - 1) - a;
                }
            if (above + same == p.M - 1) s_floor = sorted;
        }
        __syncthreads();
        low = s_floor;
        least = low ? order_value(low) : lowest(type);
        gather(room);
        n = s_n;
    }
    if (n > room) {             // more elements equal that floor than there is room for: the lowest indices of them
        __syncthreads();
        if (tid == 0) s_n = 0;
        __syncthreads();
        each([&](float x, int i) {
            if (x > least) cand[atomicAdd(&s_n, 1)] = make_key(x, uint32_t(i));
        });
        __syncthreads();
        n = s_n;                                           // in fewer than M threads
        const int need = p.M - min(n, p.M);
        int got = 0;
#pragma unroll 1
        for (int j = 0; j < NV && got < need; ++j) {
            const int i0 = at + j * kT * VW, ends = min(VW, p.V - i0);
            int mine = 0;
            for (int e = 0; e < ends; ++e) mine += value(base + i0 + e) == least;
            int before = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += x;
            }
            if (lane == 31) s_ties[warp] = before;
            __syncthreads();
            int all = 0;
            for (int w = 0; w < W; ++w) {
                if (w < warp) before += s_ties[w];
                all += s_ties[w];
            }
            int to = got + before - mine;
            for (int e = 0; e < ends; ++e)
                if (value(base + i0 + e) == least) {
                    if (to < need) cand[n + to] = make_key(least, uint32_t(i0 + e));
                    ++to;
                }
            got += all;
            __syncthreads();
        }
        n += min(got, need);
    }
    Part *part = static_cast<Part *>(p.ws);
    unsigned long long *list = reinterpret_cast<unsigned long long *>(part + size_t(p.B) * p.K * splits) +
                               size_t(blockIdx.x) * p.M;
    for (int i = tid >> 2; i < ((n + 7) & ~7); i += kT / 4) {       // four threads to a candidate, whole warps
        const unsigned long long c = i < n ? cand[i] : 0;
        int rank = 0;
        for (int j = tid & 3; j < n; j += 4) rank += cand[j] > c;
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        if (i < n && (tid & 3) == 0 && rank < p.M) list[rank] = c;
    }
    for (int i = n + tid; i < p.M; i += kT) list[i] = 0;
    if (tid == 0) {
        double t = 0.;
#pragma unroll
        for (int w = 0; w < W; ++w) t += s_sum[w];
        part[blockIdx.x] = Part{ctop, 0.f, peak ? t : 0.};
    }
}

// Order-preserving bits of a score; 0 for -inf and NaN, which are never chosen. -0 is 0.
__device__ __forceinline__ unsigned long long score_bits(double x) {
    if (!(x > -INFINITY)) return 0ull;
    const long long u = __double_as_longlong(x + 0.);
    return u < 0 ? ~(unsigned long long)u : (unsigned long long)u | (kOne << 63);
}
__device__ __forceinline__ double score_value(unsigned long long o) {
    return __longlong_as_double((long long)(o >> 63 ? o & ~(kOne << 63) : ~o));
}
// The largest key over the warp (0: none left).
__device__ __forceinline__ unsigned long long warp_max(unsigned long long key) {
    const uint32_t hi = uint32_t(key >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t low = __reduce_max_sync(0xffffffffu, hi == top ? uint32_t(key) : 0u);
    return (unsigned long long)top << 32 | low;
}

// One CTA per request. A warp merges a row's sorted lists, a lane to each: M times, the largest of the lanes' first
// elements is taken and its lane moves on. The first warp then does the same with the rows.
// staged: the segments' lists fit shared memory behind the rows' results.
__global__ void __launch_bounds__(kPickT) beam_pick_kernel(const BeamArgs p, int splits, bool staged) {
    extern __shared__ unsigned long long dyn[];
    const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int K = p.K, M = p.M;
    unsigned long long *best = dyn, *score = dyn + size_t(K) * M;    // [K][M] each: a row's keys, and their scores' bits
    const Part *part = static_cast<const Part *>(p.ws) + size_t(b) * K * splits;
    const unsigned long long *lists = reinterpret_cast<const unsigned long long *>(
                                          static_cast<const Part *>(p.ws) + size_t(p.B) * K * splits) +
                                      size_t(b) * K * splits * M;
    asm volatile("griddepcontrol.wait;" ::: "memory");               // the segments are there
    if (staged) {
        unsigned long long *to = score + size_t(K) * M;
        for (int i = tid; i < K * splits * M; i += kPickT) to[i] = lists[i];
        lists = to;
        __syncthreads();
    }
    for (int j = warp; j < K; j += kPickT / 32) {
        const double own = p.scores[size_t(b) * K + j];
        unsigned long long *to = best + size_t(j) * M, *bits = score + size_t(j) * M;
        if (p.finished && p.finished[size_t(b) * K + j]) {
            for (int i = lane; i < M; i += 32) {
                to[i] = 0xffffffffu - uint32_t(p.eos);
                bits[i] = i == 0 ? score_bits(own) : 0;
            }
            continue;
        }
        // the normaliser
        const Part *mine = part + size_t(j) * splits;
        float top = -INFINITY;
        for (int s = lane; s < splits; s += 32) top = fmaxf(top, mine[s].top);
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        double sum = 0.;
        if (top > -INFINITY)
            for (int s = lane; s < splits; s += 32)
                if (mine[s].top > -INFINITY) sum += mine[s].sum * double(expf(mine[s].top - top));
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const double norm = double(top) + log(sum);        // NaN where the row has +inf or nothing
        // the lists: 32 of them, then what came of those (lane 0) and 31 more at a time, from one buffer to the other
        const int rounds = splits <= 32 ? 1 : 1 + (splits - 2) / 31;
        for (int r = 0; r < rounds; ++r) {
            const bool odd = (rounds - 1 - r) & 1;
            unsigned long long *out = odd ? bits : to;
            const int s = r == 0 ? lane : 31 * r + lane;
            const unsigned long long *list = r > 0 && lane == 0 ? (odd ? to : bits) : lists + (size_t(j) * splits + s) * M;
            const int n = (r > 0 && lane == 0) || s < splits ? M : 0;
            int at = 0;
            unsigned long long head = n ? list[0] : 0;
            for (int m = 0; m < M; ++m) {
                const unsigned long long key = warp_max(head);
                if (lane == 0) out[m] = key;
                if (key && head == key) head = ++at < n ? list[at] : 0;
            }
            __syncwarp();
        }
        for (int i = lane; i < M; i += 32) {
            const unsigned long long key = to[i];
            bits[i] = key ? score_bits(own + (double(order_value(uint32_t(key >> 32))) - norm)) : 0;
        }
    }
    __syncthreads();
    if (warp) return;
    // the rows: two to a lane; equal scores go to the lowest
    int at[2] = {};
    unsigned long long head[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) head[i] = lane + 32 * i < K ? score[(lane + 32 * i) * M] : 0;
    for (int m = 0; m < M; ++m) {
        const int second = head[1] > head[0];
        const unsigned long long mine = second ? head[1] : head[0], key = warp_max(mine);
        const unsigned row = __reduce_min_sync(0xffffffffu, mine == key ? unsigned(lane + 32 * second) : ~0u);
        const size_t o = size_t(b) * M + m;
        if (key == 0) {
            if (lane == 0) {
                p.out_scores[o] = -INFINITY;
                p.parents[o] = -1;
                p.tokens[o] = -1;
            }
        } else if (row % 32 == unsigned(lane)) {
            const int i = int(row >> 5), x = i ? at[1] : at[0];
            p.out_scores[o] = float(score_value(key));
            p.parents[o] = int(row);
            p.tokens[o] = int(0xffffffffu - uint32_t(best[row * M + x]));
            const unsigned long long next = x + 1 < M ? score[row * M + x + 1] : 0;
            if (i) {
                at[1] = x + 1;
                head[1] = next;
            } else {
                at[0] = x + 1;
                head[0] = next;
            }
        }
    }
}

// One thread per 16-byte (or 8-byte) column of a request's K rows: every row that changes is loaded
// from its source before any is stored, so the move is safe in place whatever the chains and cycles,
// and rows that stay cost nothing in place. KM bounds K for the registers that hold the column. 24 layers of 16 requests
// of 8 beams, five of which survive (604 MB moved): 94 us, 6.4 TB/s.
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

// Vectors of 16 bytes per thread of beam_part_kernel. A segment costs about as much as three vectors on top of its
// own, so that four to six are taken by where the segments end: a row of 50277 bf16 makes five segments of five
// instead of six and a seventh of four. One or two (8 elements) where more would leave SMs without a segment.
int vectors_of(int B, int K, int V, int vw) {
    int best = 4;
    long long least = LLONG_MAX;
    for (int n = 4; n <= 6; ++n) {
        const long long cost = ((V - 1) / (kT * vw * n) + 1) * (n + 3ll);
        if (cost < least) {
            least = cost;
            best = n;
        }
    }
    return (long long)B * K * ((V - 1) / (kT * vw * best) + 1) < 2 * 148 ? 8 / vw : best;
}
int segments(int B, int K, int V, int vw) { return (V - 1) / (kT * vw * vectors_of(B, K, V, vw)) + 1; }
int width_of(wkv7_dtype dt) { return dt == WKV7_BF16 ? 8 : 4; }

template <class Tin, int NV>
cudaError_t part_t(const BeamArgs &p, int splits) {
    const unsigned grid = unsigned(p.B) * unsigned(p.K) * unsigned(splits);
    const size_t smem = size_t(room_of(p.M, NV * (16 / int(sizeof(Tin))))) * 8;         // at most 25 KB
    beam_part_kernel<Tin, NV><<<grid, kT, smem, p.stream>>>(p, splits);
    return cudaGetLastError();
}
template <class Tin>
cudaError_t select_t(const BeamArgs &p) {
    constexpr int vw = 16 / int(sizeof(Tin));
    const int splits = segments(p.B, p.K, p.V, vw);
    switch (vectors_of(p.B, p.K, p.V, vw)) {
        case 4: return part_t<Tin, 4>(p, splits);
        case 5: return part_t<Tin, 5>(p, splits);
        case 6: return part_t<Tin, 6>(p, splits);
        default: return part_t<Tin, 8 / vw>(p, splits);
    }
}

}  // namespace

cudaError_t allow_dynamic_smem(const void *kernel, int bytes);

size_t beam_select_workspace(int B, int K, int V, int M) {
    const int n = std::max(segments(B, K, V, 4), segments(B, K, V, 8));       // either type's
    return size_t(B) * K * size_t(n) * (sizeof(Part) + size_t(M) * 8);
}

cudaError_t launch_beam_select(const BeamArgs &p) {
    constexpr int most = 160 * 1024;
    const int splits = segments(p.B, p.K, p.V, width_of(p.dt));
    const size_t rows = size_t(p.K) * p.M * 16, lists = size_t(p.K) * splits * p.M * 8;     // rows: at most 64 KB
    const bool staged = rows + lists <= most;
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(beam_pick_kernel), most);
    if (e != cudaSuccess) return e;
    e = p.dt == WKV7_BF16 ? select_t<__nv_bfloat16>(p) : select_t<float>(p);
    if (e != cudaSuccess) return e;
    // launched while the segments still run: its blocks start as theirs end, and wait for the last of them
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(unsigned(p.B));
    c.blockDim = dim3(kPickT);
    c.dynamicSmemBytes = rows + (staged ? lists : 0);
    c.stream = p.stream;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, beam_pick_kernel, p, splits, staged);
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
