// Building blocks of the gated delta rule's chunked kernels: warp-level bf16 matrix instructions on
// operands split into bf16 terms, and the part of a chunk that does not depend on the state.
//
// Why warp-level instructions and not tcgen05: a chunk is a chain of small products (a warp's 16 value
// rows by 32 tokens) whose operands are rescaled, split and masked between every two of them. The
// accumulator fragment of one product is, split, the left operand of the next, so the chain runs in a
// warp's registers with no barrier; through tensor memory each link would be a round trip of store, fence,
// issue, commit, wait and load, which is longer than the product itself. Measured on B200:
// 555 TFLOP/s at 8 warps per scheduler, 516 with a single warp and 8 accumulators, 12.8 ns from one
// product to the next that needs it.
//
// Precision: x = x0 + x1 + x2 in bf16 terms holds 24 bits of x, a product of two split operands keeps
// the pairs (a, b) with a + b < the larger count, and sums are fp32. bf16 inputs are one exact term.
#pragma once

#include <type_traits>

#include "delta.cuh"

namespace wkv7 {
namespace dm {

constexpr int C = 32;               // tokens per chunk
constexpr int kGroup = 64;          // threads that prepare one chunk: a warp for the keys, one for the queries
constexpr int kTri = 3 * 512;       // bytes of one term of a lower triangular [32][32]: blocks (0,0), (1,0), (1,1)
constexpr int kAs = 20;             // row of a 16 x 16 fp32 scratch block, two of which lie where W goes
constexpr int kAb = 16 * kAs + 16;  // from one block to the next, in other banks
static_assert(2 * kAb * 4 <= 3 * kTri, "the scratch blocks fit W's place");

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t a, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t a, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// d += a b: a 16 x 16 (rows g, g + 8; columns 2t, 2t + 1, + 8), b 16 x 8, d 16 x 8 with g = lane / 4, t = lane % 4
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory"); }

__device__ __forceinline__ void st_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ void ld_v4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void st_b32(uint32_t a, uint32_t x) { asm volatile("st.shared.b32 [%0], %1;" :: "r"(a), "r"(x) : "memory"); }

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float x, float y) {      // x in the low half
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(y), "f"(x));
    return u;
}
// Two values as T bf16 terms each: r[0] the values rounded, r[1] what that left, rounded, and so on. The
// remainder is one mixed-precision multiply-add per value (x - hi), without unpacking hi first: 13.6
// against 16.3 issue slots for a split with its surroundings, same bits.
template <int T>
__device__ __forceinline__ void split2(float x, float y, uint32_t *r) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
        r[i] = pack(x, y);
        if (i + 1 < T)
            asm("{\n\t.reg .b16 l, h, m;\n\tmov.b16 m, 0xBF80;\n\tmov.b32 {l, h}, %2;\n\t"
                "fma.rn.f32.bf16 %0, l, m, %0;\n\tfma.rn.f32.bf16 %1, h, m, %1;\n\t}"
                : "+f"(x), "+f"(y) : "r"(r[i]));
    }
}
// The accumulators of two neighbouring 16 x 8 tiles as the left operand of a 16-deep product, T terms.
template <int T>
__device__ __forceinline__ void split_a(const float (&u)[4], const float (&v)[4], uint32_t (&a)[T][4]) {
    uint32_t r[4][T];
    split2<T>(u[0], u[1], r[0]);
    split2<T>(u[2], u[3], r[1]);
    split2<T>(v[0], v[1], r[2]);
    split2<T>(v[2], v[3], r[3]);
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) a[i][j] = r[j][i];
}

// The tensor cores cut, not round, as they add to an accumulator (half a unit in the last place each time, always
// towards zero). Where fp32's accuracy is wanted the products of leading terms therefore get an
// accumulator of their own, so that it sees few additions, and the small products another.
template <bool TWO, int N>
struct Acc {
    float d[N][4], small[TWO ? N : 1][4];
    __device__ __forceinline__ Acc() {
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                d[n][e] = 0.f;
                if (TWO) small[n % (TWO ? N : 1)][e] = 0.f;
            }
    }
    __device__ __forceinline__ void add(int n, bool leading, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        if (TWO && !leading) mma(small[TWO ? n : 0], a, b0, b1);
        else mma(d[n], a, b0, b1);
    }
    __device__ __forceinline__ void join() {
        if constexpr (TWO) {
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[n][e] += small[n][e];
                    small[n][e] = 0.f;
                }
        }
    }
};

// Byte offset of 16-byte chunk c of row r in a tile of rows of NB bytes (64 or a multiple of 128): eight rows
// of one chunk column lie in eight different bank groups.
template <int NB> __device__ __forceinline__ uint32_t tile(int r, int c) {
    return uint32_t(r * NB + ((NB == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7)) << 4));
}
// The same inside a 16 x 16 block of bf16 (rows of 32 bytes).
__device__ __forceinline__ uint32_t block(int r, int c) { return uint32_t(r * 32 + ((c ^ ((r >> 2) & 1)) << 4)); }

// The addresses below step through a row's chunks by an exclusive or on the whole address: tiles start at
// multiples of 256 bytes, and a lane's first chunk differs from the next ones in the chunk's bits alone.
// Right operand from a tile that holds it by columns (rows n0 .. n0 + 15 are columns of the operand),
// depth 16 ks ..: r[0], r[1] for the first eight columns, r[2], r[3] for the next.
template <int NB> __device__ __forceinline__ uint32_t addr_b(uint32_t base, int n0, int ks) {
    const int l = threadIdx.x & 31;
    return (base + n0 * NB + tile<NB>((l & 7) + ((l >> 4) << 3), (l >> 3) & 1)) ^ (ks << 5);
}
// Right operand from a tile that holds it by rows (depth k0 ..), columns 8 c .. (c even); for ldsm4t.
template <int NB> __device__ __forceinline__ uint32_t addr_bt(uint32_t base, int k0, int c) {
    const int l = threadIdx.x & 31;
    return (base + k0 * NB + tile<NB>((l & 7) + (((l >> 3) & 1) << 3), l >> 4)) ^ (c << 4);
}
// Left operand from a tile by rows m0 .., depth 16 ks ..
template <int NB> __device__ __forceinline__ uint32_t addr_a(uint32_t base, int m0, int ks) {
    const int l = threadIdx.x & 31;
    return (base + m0 * NB + tile<NB>((l & 7) + (((l >> 3) & 1) << 3), l >> 4)) ^ (ks << 5);
}
__device__ __forceinline__ uint32_t addr_block(uint32_t base) {      // by columns, as addr_b
    const int l = threadIdx.x & 31;
    return base + block((l & 7) + ((l >> 4) << 3), (l >> 3) & 1);
}
__device__ __forceinline__ uint32_t addr_block_t(uint32_t base) {    // by rows, as addr_bt
    const int l = threadIdx.x & 31;
    return base + block((l & 7) + (((l >> 3) & 1) << 3), l >> 4);
}

// What the kernels read of one chunk besides the matrices.
struct Scalars {
    float kin[C];    // exp(G_i) / |k_i|: applied to S k_i
    float qin[C];    // scale exp(G_i) / |q_i|: applied to S q_i
    float out[C];    // exp(G_C - G_j) beta_j / |k_j|: applied to e_j in the state's update
    float whole;     // exp(G_C)
    int odd;         // a key or gate of the chunk is not finite, or the state may grow beyond fp32
    float pad[2];
};

// What the two warps of a preparing group exchange.
struct PrepScratch {
    float rk[C], rq[C];
};

// One strided tensor's rows on their way to the tiles of a stage, by one preparing group: a thread keeps
// one 16-byte column (fp32: 32 bytes) of every STEP-th row.
template <int W, bool F32>
struct RowLoader {
    static constexpr int CH = W / 8, STEP = kGroup / CH, N = C / STEP;   // STEP rows at a time
    using Tin = std::conditional_t<F32, float, __nv_bfloat16>;
    const Tin *at, *safe;            // safe: an address inside the tensor for copies of no bytes
    long long stride;
    int r, c;
    __device__ __forceinline__ RowLoader(const void *base, long long first, long long offset, long long row_stride, int tid) {
        r = tid / CH;
        c = tid % CH;
        stride = row_stride;
        safe = static_cast<const Tin *>(base);
        at = static_cast<const Tin *>(base) + offset + (first + r) * row_stride + 8 * c;
    }
    // Moves on by so many chunks of C rows (or back).
    __device__ __forceinline__ void advance(int chunks) { at += chunks * (C * stride); }
    // C rows from the current ones on; rows from n on become zeros. bf16: asynchronous (the caller commits).
    __device__ __forceinline__ void load(uint32_t dst, int n) const {
        const Tin *p = at;
#pragma unroll
        for (int i = 0; i < N; ++i, p += STEP * stride) {
            const bool there = r + i * STEP < n;
            const uint32_t to = dst + tile<W * 2>(r + i * STEP, c);
            if constexpr (!F32) {
                cp16(to, there ? p : safe, there);
            } else {
                float4 x = make_float4(0, 0, 0, 0), y = x;
                if (there) {
                    x = __ldg(reinterpret_cast<const float4 *>(p));
                    y = __ldg(reinterpret_cast<const float4 *>(p) + 1);
                }
                uint32_t w[4][3];
                split2<3>(x.x, x.y, w[0]);
                split2<3>(x.z, x.w, w[1]);
                split2<3>(y.x, y.y, w[2]);
                split2<3>(y.z, y.w, w[3]);
#pragma unroll
                for (int k = 0; k < 3; ++k) st_v4(to + k * (C * W * 2), w[0][k], w[1][k], w[2][k], w[3][k]);
            }
        }
    }
};

// A token's gates as loaded; turned into numbers only when the chunk is prepared, so that nothing waits.
template <bool F32> struct Gate {
    using T = std::conditional_t<F32, float, unsigned short>;
    T g, beta;
    __device__ __forceinline__ void load(const void *gp, const void *bp, long long at, bool there) {
        g = beta = T(0);
        if (there) {
            g = __ldg(static_cast<const T *>(gp) + at);
            beta = __ldg(static_cast<const T *>(bp) + at);
        }
    }
    static __device__ __forceinline__ float num(T x) {
        if constexpr (F32) return x;
        else return __uint_as_float(uint32_t(x) << 16);
    }
};

// exp for decays between tokens: two instructions, relative error about 1e-7 + 6e-8 |x|, so the decays
// that weigh anything keep fp32's accuracy (denormal results become 0).
__device__ __forceinline__ float fast_exp(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// The state-free part of one chunk, by a group of two warps (`queries`: this warp's role; named barrier
// `bar`). With D_ij = exp(G_i - G_j) and unit or given q, k:
//     P_ij = scale D_ij beta_j q_i.k_j  (j <= i)         -> TP terms       (the warp of the queries)
//     W = (I + A)^-1, A_ij = D_ij beta_j k_i.k_j (j < i)  -> 3 terms        (the warp of the keys)
// k, q: TI tiles of bf16 terms; g, beta: lane's token, 0 behind the end. The warps exchange the keys'
// lengths and are otherwise on their own.
// The sums G are exact in 64-bit fixed point (steps of 2^-32) and kept as two floats (the first a multiple
// of 2^-10), so that differences of large sums keep their low bits.
// W in blocks of 16: the diagonal ones by forward substitution in fp32, a half-warp per block and a
// column per lane (as soon as t_j is known it is taken from all later rows, so that one product and one
// selection lie between t_j and t_j+1), the one below them as -W_11 (A_10 W_00) on the tensor cores.
// Substitution over all 32 rows took 496 products in a row of straight-line code, and the
// warps of both kinds then waited for instructions: code size is what this routine is written for, and
// why its loop over the depth stays a loop.
// TP = 0: neither P nor anything of the queries is wanted (the warp of the queries writes the scalars).
template <int NN, int TI, int TP>
__device__ __forceinline__ void prepare_chunk(uint32_t k, uint32_t q, unsigned char *w_at, uint32_t p_out, Scalars *sc, PrepScratch *ps,
                                              const DeltaArgs &p, float g, float beta, bool queries, int bar) {
    constexpr int NB = NN * 2, TB = C * NB;
    const int lane = threadIdx.x & 31, gr = lane >> 2, tc = lane & 3;
    const uint32_t left = queries ? q : k, w_out = smem_addr(w_at);
    float *scratch = reinterpret_cast<float *>(w_at);
    // products with the keys, tiles (m, n): (0, 0), (0, 1), (1, 0), (1, 1), (1, 2), (1, 3)
    Acc<(TI > 1), 6> prod;
    float (&acc)[6][4] = prod.d;
    float len[4] = {};
    if (TP > 0 || !queries) {
#pragma unroll 1
        for (int ks = 0; ks < NN / 16; ++ks) {
            uint32_t a0[TI][4], a1[TI][4], b0[TI][4], b1[TI][4];
#pragma unroll
            for (int i = 0; i < TI; ++i) {
                ldsm4(a0[i], addr_a<NB>(left + i * TB, 0, ks));
                ldsm4(a1[i], addr_a<NB>(left + i * TB, 16, ks));
                ldsm4(b0[i], addr_b<NB>(k + i * TB, 0, ks));
                ldsm4(b1[i], addr_b<NB>(k + i * TB, 16, ks));
            }
#pragma unroll
            for (int x = TI - 1; x >= 0; --x)
#pragma unroll
                for (int y = TI - 1 - x; y >= 0; --y) {
                    const bool top = x + y == 0;
                    prod.add(0, top, a0[x], b0[y][0], b0[y][1]);
                    prod.add(1, top, a0[x], b0[y][2], b0[y][3]);
                    prod.add(2, top, a1[x], b0[y][0], b0[y][1]);
                    prod.add(3, top, a1[x], b0[y][2], b0[y][3]);
                    prod.add(4, top, a1[x], b1[y][0], b1[y][1]);
                    prod.add(5, top, a1[x], b1[y][2], b1[y][3]);
                }
            if (!queries) continue;     // the keys' squares are the products' diagonal
            // the queries' from the same fragments: rows gr, gr + 8, 16 + gr, 24 + gr
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = 0.f, y = 0.f;
#pragma unroll
                    for (int i = TI - 1; i >= 0; --i) {
                        const uint32_t u = (r < 2 ? a0[i] : a1[i])[(r & 1) + 2 * c];
                        x += lo_f(u);
                        y += hi_f(u);
                    }
                    len[r] = fmaf(x, x, fmaf(y, y, len[r]));
                }
        }
    }
    prod.join();
    bool fine = true;               // what this lane's rows and token add to `odd`
    if (queries) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            len[r] += __shfl_xor_sync(0xffffffffu, len[r], 1);
            len[r] += __shfl_xor_sync(0xffffffffu, len[r], 2);
        }
    } else {                        // row gr of a diagonal tile is its column 2 tc + e where tc = gr / 2, e = gr % 2
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float (&d)[4] = acc[r < 2 ? r : r + 2];
            const float x = d[2 * (r & 1)], y = d[2 * (r & 1) + 1];
            len[r] = __shfl_sync(0xffffffffu, gr & 1 ? y : x, 4 * gr + (gr >> 1));
        }
        fine = len[0] + len[1] + len[2] + len[3] < INFINITY && fabsf(beta) < INFINITY;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) len[r] = (p.qk_norm ? delta_unit(len[r], p.norm_eps) : 1.f) * (queries ? p.scale : 1.f);
    if (tc == 0 && (TP > 0 || !queries)) {
#pragma unroll
        for (int r = 0; r < 4; ++r) (queries ? ps->rq : ps->rk)[gr + 8 * r] = len[r];
    }
    // running sums of the log decays
    unsigned nan = __ballot_sync(0xffffffffu, g != g);
    long long G = llrintf(fminf(g, 120.f) * 4294967296.f);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, G, o);
        if (lane >= o) G += x;
    }
    // A state that grows by more than e^80 from some token of the chunk (or its start) to a later one leaves what exp(G)
    // and D can hold: that token counts as one with a NaN gate. From e^40 on the chunk is watched for overflow. (In steps
    // of 2^-10: the code's size is what this costs, 0.1 to 0.8 % of the sweeps' time; sums of 64 bits took 1 to 3 %.)
    if (__any_sync(0xffffffffu, g > 0.f)) {
        const int at = int(G >> 22);
        int low = min(at, 0);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) low = min(low, __shfl_up_sync(0xffffffffu, low, o));
        nan |= __ballot_sync(0xffffffffu, at - low > (80 << 10));
        fine = fine && at - low < (40 << 10);
    }
    const float bad = __int_as_float(0x7fffffff);
    const bool seen = (nan & (0xffffffffu >> (31 - lane))) != 0;          // a NaN at or before this token
    const float ghi = seen ? bad : float(int(G >> 22)) * 9.765625e-4f;
    const float glo = float(int(G & 0x3fffff)) * 2.3283064365386963e-10f;
    bar_sync(bar, kGroup);
    const float rk = ps->rk[lane], kb = rk * beta;
    if (queries) {
        const long long rest = __shfl_sync(0xffffffffu, G, 31) - G;
        const float in = seen ? bad : expf(float(G) * 2.3283064365386963e-10f);
        const float out = (nan ? bad : expf(float(rest) * 2.3283064365386963e-10f)) * rk;
        sc->kin[lane] = in * rk;
        if constexpr (TP > 0) sc->qin[lane] = in * ps->rq[lane];
        sc->out[lane] = out * beta;
        if (lane == 31) sc->whole = nan ? bad : in;
        if constexpr (TP == 0) return;
    }
    // D and the factors of rows and columns. Where the chunk's sums stay within 30 of the middle one, D is a
    // product of a row's and a column's factor, two exponentials per token; elsewhere one per element.
    const int last = queries ? 0 : -1;          // column j of row i stays if j <= i + last
    const long long off = G - __shfl_sync(0xffffffffu, G, C / 2 - 1);
    const bool near = __all_sync(0xffffffffu, off < (30ll << 32) && off > -(30ll << 32));
    if (near) {
        const float hi = float(int(off >> 22)) * 9.765625e-4f, lo = float(int(off & 0x3fffff)) * 2.3283064365386963e-10f;
        const float up = expf(hi), down = expf(-hi);
        const float l2 = 0.5f * lo * lo;        // exp(lo) = 1 + lo + lo^2 / 2: lo is below 2^-10
        const float row = (seen ? bad : fmaf(up, lo + l2, up)) * (queries ? ps->rq : ps->rk)[lane];
        const float col = (seen ? bad : fmaf(down, l2 - lo, down)) * kb;
        float rf[4], cf[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) rf[i] = __shfl_sync(0xffffffffu, row, gr + 8 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) cf[j] = __shfl_sync(0xffffffffu, col, 8 * (j >> 1) + 2 * tc + (j & 1));
#pragma unroll
        for (int x = 0; x < 6; ++x) {
            const int m = x < 2 ? 0 : 1, n = x < 2 ? x : x - 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ri = 2 * m + (e >> 1), ci = 2 * n + (e & 1);
                const float w = acc[x][e] * cf[ci] * rf[ri];
                acc[x][e] = 8 * n + 2 * tc + (e & 1) <= gr + 8 * ri + last ? w : 0.f;
            }
        }
    } else {
        float rh[4], rl[4], ch[8], cl[8], cb[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            rh[i] = __shfl_sync(0xffffffffu, ghi, gr + 8 * i);
            rl[i] = __shfl_sync(0xffffffffu, glo, gr + 8 * i);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int from = 8 * (j >> 1) + 2 * tc + (j & 1);
            ch[j] = __shfl_sync(0xffffffffu, ghi, from);
            cl[j] = __shfl_sync(0xffffffffu, glo, from);
            cb[j] = __shfl_sync(0xffffffffu, kb, from);
        }
#pragma unroll
        for (int x = 0; x < 6; ++x) {
            const int m = x < 2 ? 0 : 1, n = x < 2 ? x : x - 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ri = 2 * m + (e >> 1), ci = 2 * n + (e & 1);
                const float w = acc[x][e] * fast_exp((rh[ri] - ch[ci]) + (rl[ri] - cl[ci])) * (cb[ci] * len[ri]);
                acc[x][e] = 8 * n + 2 * tc + (e & 1) <= gr + 8 * ri + last ? w : 0.f;
            }
        }
    }
    if (queries) {
#pragma unroll
        for (int x = 0; x < 6; ++x) {
            const int m = x < 2 ? 0 : 1, n = x < 2 ? x : x - 2;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                uint32_t r[TP > 0 ? TP : 1];
                split2<TP>(acc[x][e], acc[x][e + 1], r);
#pragma unroll
                for (int z = 0; z < TP; ++z) st_b32(p_out + z * kTri + (m + (n >> 1)) * 512 + block(gr + 4 * e, n & 1) + 4 * tc, r[z]);
            }
        }
        return;
    }
    fine = !__any_sync(0xffffffffu, !fine);
    if (lane == 0) sc->odd = !fine || nan;
    // the diagonal blocks, by columns
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) scratch[b * kAb + (8 * n + 2 * tc + (e & 1)) * kAs + gr + 8 * (e >> 1)] = acc[4 * b + n][e];
    __syncwarp();
    const int col = lane & 15;
    float *D = scratch + (lane >> 4) * kAb;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = i == col ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < 15; ++j) {
        t[j] = j < col ? 0.f : t[j];
#pragma unroll
        for (int i = (j + 1) >> 2; i < 4; ++i) {
            const float4 a = *reinterpret_cast<const float4 *>(&D[j * kAs + 4 * i]);
            const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * i + e > j) t[4 * i + e] = fmaf(-v[e], t[j], t[4 * i + e]);
        }
    }
    t[15] = 15 < col ? 0.f : t[15];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) D[i * kAs + col] = t[i];
    __syncwarp();
    float4 own[4];                  // row `col` of this half-warp's block
#pragma unroll
    for (int c = 0; c < 4; ++c) own[c] = *reinterpret_cast<const float4 *>(&D[col * kAs + 4 * c]);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        uint32_t w[4][3];
        split2<3>(own[2 * c].x, own[2 * c].y, w[0]);
        split2<3>(own[2 * c].z, own[2 * c].w, w[1]);
        split2<3>(own[2 * c + 1].x, own[2 * c + 1].y, w[2]);
        split2<3>(own[2 * c + 1].z, own[2 * c + 1].w, w[3]);
#pragma unroll
        for (int z = 0; z < 3; ++z)
            st_v4(w_out + z * kTri + (lane >> 4) * 1024 + block(col, c), w[0][z], w[1][z], w[2][z], w[3][z]);
    }
    __syncwarp();
    // the block below: -W_11 (A_10 W_00)
    float v[2][4] = {}, r[2][4] = {};
    {
        uint32_t a[3][4], w[3][4];
        split_a<3>(acc[2], acc[3], a);
#pragma unroll
        for (int z = 0; z < 3; ++z) ldsm4t(w[z], addr_block_t(w_out + z * kTri));
#pragma unroll
        for (int x = 2; x >= 0; --x)
#pragma unroll
            for (int z = 2 - x; z >= 0; --z) {
                mma(v[0], a[x], w[z][0], w[z][1]);
                mma(v[1], a[x], w[z][2], w[z][3]);
            }
    }
    // A row that is not finite would reach the rows above it through the zeros of W_11; it needs no
    // place here, since its own token is already marked where the values are.
    auto put = [&](const float (&x)[2][4], bool neg) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                uint32_t u[3];
                split2<3>(neg ? -x[n][e] : x[n][e], neg ? -x[n][e + 1] : x[n][e + 1], u);
#pragma unroll
                for (int z = 0; z < 3; ++z) st_b32(w_out + z * kTri + 512 + block(gr + 4 * e, n) + 4 * tc, u[z]);
            }
    };
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[n][e] = fabsf(v[n][e]) < INFINITY ? v[n][e] : 0.f;
    put(v, false);
    __syncwarp();
    {
        uint32_t a[3][4], w[3][4];
#pragma unroll
        for (int z = 0; z < 3; ++z) {
            ldsm4(a[z], addr_block_t(w_out + z * kTri + 1024));     // by rows, as a left operand
            ldsm4t(w[z], addr_block_t(w_out + z * kTri + 512));
        }
#pragma unroll
        for (int x = 2; x >= 0; --x)
#pragma unroll
            for (int z = 2 - x; z >= 0; --z) {
                mma(r[0], a[x], w[z][0], w[z][1]);
                mma(r[1], a[x], w[z][2], w[z][3]);
            }
    }
    __syncwarp();
    put(r, true);
}

// A warp's 16 rows of a state to a workspace's [unit][N][N]: as fp32, or for bf16 inputs as two bf16 terms in arrays
// `second` elements apart, in whole 16-byte pieces through `at`, 64 N bytes of shared memory of the warp's own. Four bytes
// per lane straight to memory took 8 x 1024 tokens of 12 heads 258 us for the whole backward against 246 (N = 64), and
// seven packed sequences of 8 heads 525 against 532 (N = 128).
template <bool F32, int NN>
__device__ __forceinline__ void keep_state(void *ws, long long second, long long unit, int row, const float (&S)[NN / 8][4], uint32_t at) {
    const int lane = threadIdx.x & 31;
    if constexpr (F32) {
        float *to = static_cast<float *>(ws) + (size_t(unit) * NN + row + (lane >> 2)) * NN + 2 * (lane & 3);
#pragma unroll
        for (int n = 0; n < NN / 8; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) *reinterpret_cast<float2 *>(to + 8 * e * NN + 8 * n) = make_float2(S[n][2 * e], S[n][2 * e + 1]);
        return;
    }
    constexpr int TERM = 16 * NN * 2, PER_ROW = NN / 8;
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NN / 8; n += 2) {
        uint32_t r[2][4];           // [term][rows g, g + 8 of one tile, of the next]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t t[2];
            split2<2>(S[n + (i >> 1)][2 * (i & 1)], S[n + (i >> 1)][2 * (i & 1) + 1], t);
            r[0][i] = t[0];
            r[1][i] = t[1];
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) stsm4(at + z * TERM + tile<NN * 2>(lane & 15, n + (lane >> 4)), r[z]);
    }
    __syncwarp();
    __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(ws) + (size_t(unit) * NN + row) * NN;
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < NN / 16; ++i) {
            const int r = (32 * i + lane) / PER_ROW, c = lane % PER_ROW;
            uint32_t u[4];
            ld_v4(u, at + z * TERM + tile<NN * 2>(r, c));
            *reinterpret_cast<uint4 *>(to + z * second + r * NN + 8 * c) = make_uint4(u[0], u[1], u[2], u[3]);
        }
}
// X^T of a warp (16 value channels, 32 tokens) as two bf16 terms, to rows of tokens `stride` elements apart; through
// `at` as above.
__device__ __forceinline__ void put_terms(__nv_bfloat16 *first, __nv_bfloat16 *second, size_t stride, int n_tok, float (&X)[4][4], uint32_t at) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float *x = &X[2 * m + (i >> 1)][2 * (i & 1)];
                o[i] = pack(x[0], x[1]);
                x[0] -= lo_f(o[i]);             // what the rounding leaves
                x[1] -= hi_f(o[i]);
            }
            stsm4t(at + z * 1024 + block(16 * m + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1), o);
        }
    __syncwarp();
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int tok = 16 * m + (lane >> 1);
            uint32_t u[4];
            ld_v4(u, at + z * 1024 + block(tok, lane & 1));
            if (tok < n_tok) *reinterpret_cast<uint4 *>((z ? second : first) + tok * stride + 8 * (lane & 1)) = make_uint4(u[0], u[1], u[2], u[3]);
        }
}

}  // namespace dm
}  // namespace wkv7
