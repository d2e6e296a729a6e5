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

#include "delta.cuh"

namespace wkv7 {
namespace dm {

constexpr int C = 32;               // tokens per chunk
constexpr int kPrep = 128;          // threads that prepare chunks
constexpr int kTri = 3 * 512;       // bytes of one term of a lower triangular [32][32]: blocks (0,0), (1,0), (1,1)
constexpr int kAs = 36;             // row of the fp32 scratch matrix

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
// d += a b: a 16 x 16 (rows g, g + 8; columns 2t, 2t + 1, + 8), b 16 x 8, d 16 x 8 with g = lane / 4, t = lane % 4
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" :: "r"(id), "r"(threads) : "memory"); }

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float x, float y) {      // x in the low half
    uint32_t u;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u) : "f"(y), "f"(x));
    return u;
}
// Two values as T bf16 terms each: r[0] the values rounded, r[1] what that left, rounded, and so on.
template <int T>
__device__ __forceinline__ void split2(float x, float y, uint32_t *r, int step = 1) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
        r[i * step] = pack(x, y);
        if (i + 1 < T) {
            x -= lo_f(r[i * step]);
            y -= hi_f(r[i * step]);
        }
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

// Byte offset of 16-byte chunk c of row r in a tile of rows of NB bytes (a multiple of 128): eight rows
// of one chunk column lie in eight different bank groups.
template <int NB> __device__ __forceinline__ uint32_t tile(int r, int c) { return uint32_t(r * NB + ((c ^ (r & 7)) << 4)); }
// The same inside a 16 x 16 block of bf16 (rows of 32 bytes).
__device__ __forceinline__ uint32_t block(int r, int c) { return uint32_t(r * 32 + ((c ^ ((r >> 2) & 1)) << 4)); }

// Right operand from a tile that holds it by columns (rows n0 .. n0 + 15 are columns of the operand),
// depth 16 ks ..: r[0], r[1] for the first eight columns, r[2], r[3] for the next.
template <int NB> __device__ __forceinline__ uint32_t addr_b(uint32_t base, int n0, int ks) {
    const int l = threadIdx.x & 31;
    return base + tile<NB>(n0 + (l & 7) + ((l >> 4) << 3), 2 * ks + ((l >> 3) & 1));
}
// Right operand from a tile that holds it by rows (depth k0 ..), columns 8 c ..; for ldsm4t.
template <int NB> __device__ __forceinline__ uint32_t addr_bt(uint32_t base, int k0, int c) {
    const int l = threadIdx.x & 31;
    return base + tile<NB>(k0 + (l & 7) + (((l >> 3) & 1) << 3), c + (l >> 4));
}
// Left operand from a tile by rows m0 .., depth 16 ks ..
template <int NB> __device__ __forceinline__ uint32_t addr_a(uint32_t base, int m0, int ks) {
    const int l = threadIdx.x & 31;
    return base + tile<NB>(m0 + (l & 7) + (((l >> 3) & 1) << 3), 2 * ks + (l >> 4));
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
    float kout[C];   // exp(G_C - G_j) / |k_j| (backward)
    float beta[C];
    float whole;     // exp(G_C)
    float pad[3];
};

// Scratch of the preparing threads.
struct PrepScratch {
    float A[C * kAs];
    float T[C * kAs];
    float ghi[C], glo[C], rk[C], rq[C];
};

// Rows [t0, t0 + C) of a strided tensor into TI tiles of bf16 terms; rows from `n` on are zero.
// bf16: asynchronous copies (the caller commits and waits). fp32: loaded, split and stored.
template <int NN, bool F32>
__device__ __forceinline__ void load_tile(uint32_t dst, const void *src, long long t0, int n, long long stride, int tid, int threads) {
    if constexpr (!F32) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(src);
        for (int i = tid; i < C * NN / 8; i += threads) {
            const int r = i / (NN / 8), c = i % (NN / 8);
            cp16(dst + tile<NN * 2>(r, c), p + (t0 + (r < n ? r : 0)) * stride + 8 * c, r < n);
        }
    } else {
        const float *p = static_cast<const float *>(src);
        for (int i = tid; i < C * NN / 8; i += threads) {
            const int r = i / (NN / 8), c = i % (NN / 8);
            float4 x = make_float4(0, 0, 0, 0), y = x;
            if (r < n) {
                const float4 *q = reinterpret_cast<const float4 *>(p + (t0 + r) * stride + 8 * c);
                x = __ldg(q);
                y = __ldg(q + 1);
            }
            uint32_t w[4][3];
            split2<3>(x.x, x.y, w[0]);
            split2<3>(x.z, x.w, w[1]);
            split2<3>(y.x, y.y, w[2]);
            split2<3>(y.z, y.w, w[3]);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint32_t at = dst + k * (C * NN * 2) + tile<NN * 2>(r, c);
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(at), "r"(w[0][k]), "r"(w[1][k]), "r"(w[2][k]), "r"(w[3][k]) : "memory");
            }
        }
    }
}

// The state-free part of one chunk, by the kPrep preparing threads (thread index tid, named barrier
// `bar`). With D_ij = exp(G_i - G_j) and unit or given q, k:
//     P_ij = scale D_ij beta_j q_i.k_j  (j <= i)         -> TP terms
//     W = (I + A)^-1, A_ij = D_ij beta_j k_i.k_j (j < i)  -> 3 terms
// k, q: TI tiles of bf16 terms; g, beta: this thread's token (lanes of the last warp), 0 behind the end.
// The sums G are taken in fp64 and kept as two floats (the first a multiple of 2^-10), so that differences
// of large sums keep their low bits. W comes from forward substitution by one warp, a column per lane, in
// fp32 (496 products); the warp changes with the chunk so that no scheduler gets all of it.
template <int NN, int TI, int TP>
__device__ __forceinline__ void prepare_chunk(uint32_t k, uint32_t q, uint32_t w_out, uint32_t p_out, Scalars *sc, PrepScratch *ps,
                                              const DeltaArgs &p, float g, float beta, int chunk, int tid, int bar) {
    constexpr int NB = NN * 2, TB = C * NB;
    const int warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tc = lane & 3;
    // products: warps 0, 1 keys by keys, warps 2, 3 queries by keys; each the tiles (m 0, n h), (m 1, n h), (m 1, n 2 + h)
    const int h = warp & 1;
    const uint32_t left = warp < 2 ? k : q;
    float acc[3][4] = {};
#pragma unroll
    for (int ks = 0; ks < NN / 16; ++ks) {
        uint32_t a0[TI][4], a1[TI][4], b[TI][4];
#pragma unroll
        for (int i = 0; i < TI; ++i) {
            ldsm4(a0[i], addr_a<NB>(left + i * TB, 0, ks));
            ldsm4(a1[i], addr_a<NB>(left + i * TB, 16, ks));
            // rows 8 h .. + 7 and 16 + 8 h .. + 7
            ldsm4(b[i], k + i * TB + tile<NB>(8 * h + (lane & 7) + ((lane >> 4) << 4), 2 * ks + ((lane >> 3) & 1)));
        }
#pragma unroll
        for (int x = TI - 1; x >= 0; --x)
#pragma unroll
            for (int y = TI - 1 - x; y >= 0; --y) {
                mma(acc[0], a0[x], b[y][0], b[y][1]);
                mma(acc[1], a1[x], b[y][0], b[y][1]);
                mma(acc[2], a1[x], b[y][2], b[y][3]);
            }
    }
    {   // lengths: two threads per row, keys then queries
        const int row = (tid >> 1) & 31, half = tid & 1;
        const uint32_t base = tid < 64 ? k : q;
        float s = 0.f;
        if (p.qk_norm) {
#pragma unroll
            for (int c = 0; c < NN / 16; ++c) {
                float x[8] = {};
#pragma unroll
                for (int i = TI - 1; i >= 0; --i) {
                    uint32_t u[4];
                    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                                 : "r"(base + i * TB + tile<NB>(row, half * (NN / 16) + c)));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[2 * e] += lo_f(u[e]);
                        x[2 * e + 1] += hi_f(u[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
            }
            s += __shfl_xor_sync(0xffffffffu, s, 1);
        }
        const float r = p.qk_norm ? rsqrtf(s + p.norm_eps) : 1.f;
        if (half == 0) (tid < 64 ? ps->rk : ps->rq)[row] = tid < 64 ? r : r * p.scale;
    }
    if (warp == 3) {
        double G = g;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double x = __shfl_up_sync(0xffffffffu, G, o);
            if (lane >= o) G += x;
        }
        const double last = __shfl_sync(0xffffffffu, G, 31);
        const float hi = float(rint(G * 1024.) * (1. / 1024.));
        ps->ghi[lane] = hi;
        ps->glo[lane] = float(G - double(hi));
        sc->beta[lane] = beta;
        sc->kin[lane] = expf(float(G));
        sc->kout[lane] = expf(float(last - G));
        if (lane == 31) sc->whole = expf(float(last));
    }
    bar_sync(bar, kPrep);
    if (warp == 0) {
        const float in = sc->kin[lane], out = sc->kout[lane] * ps->rk[lane];
        sc->kin[lane] = in * ps->rk[lane];
        sc->qin[lane] = in * ps->rq[lane];
        sc->kout[lane] = out;
        sc->out[lane] = out * sc->beta[lane];
    }
#pragma unroll
    for (int x = 0; x < 3; ++x) {
        const int m = x ? 16 : 0, n0 = (x == 2 ? 16 : 0) + 8 * h;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const int i = m + gr + 4 * e;                   // e = 0: row gr, e = 2: row gr + 8
            float v[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int j = n0 + 2 * tc + f;
                const float d = expf((ps->ghi[i] - ps->ghi[j]) + (ps->glo[i] - ps->glo[j]));
                const float s = acc[x][e + f] * d * (ps->rk[j] * sc->beta[j]);
                v[f] = warp < 2 ? (j < i ? s * ps->rk[i] : 0.f) : (j <= i ? s * ps->rq[i] : 0.f);
            }
            const int j = n0 + 2 * tc;
            if (warp < 2) {
                *reinterpret_cast<float2 *>(&ps->A[i * kAs + j]) = make_float2(v[0], v[1]);
            } else {
                uint32_t r[TP];
                split2<TP>(v[0], v[1], r);
#pragma unroll
                for (int k2 = 0; k2 < TP; ++k2)
                    asm volatile("st.shared.b32 [%0], %1;" :: "r"(p_out + k2 * kTri + x * 512 + block(i & 15, (j >> 3) & 1) + ((j & 7) << 1)), "r"(r[k2]) : "memory");
            }
        }
    }
    bar_sync(bar, kPrep);
    if (warp == (chunk & 3)) {
        float t[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            float s[4] = {};
#pragma unroll
            for (int kk = 0; kk < i; kk += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(&ps->A[i * kAs + kk]);
                s[0] = fmaf(a.x, t[kk], s[0]);
                if (kk + 1 < i) s[1] = fmaf(a.y, t[kk + 1], s[1]);
                if (kk + 2 < i) s[2] = fmaf(a.z, t[kk + 2], s[2]);
                if (kk + 3 < i) s[3] = fmaf(a.w, t[kk + 3], s[3]);
            }
            t[i] = i < lane ? 0.f : (i == lane ? 1.f : -((s[0] + s[1]) + (s[2] + s[3])));
            ps->T[i * kAs + lane] = t[i];
        }
    }
    bar_sync(bar, kPrep);
    {
        const int i = tid >> 2, c = tid & 3;                // row, eight columns 8 c ..
        if (i >= 16 || c < 2) {
            const float4 x = *reinterpret_cast<const float4 *>(&ps->T[i * kAs + 8 * c]);
            const float4 y = *reinterpret_cast<const float4 *>(&ps->T[i * kAs + 8 * c + 4]);
            uint32_t w[4][3];
            split2<3>(x.x, x.y, w[0]);
            split2<3>(x.z, x.w, w[1]);
            split2<3>(y.x, y.y, w[2]);
            split2<3>(y.z, y.w, w[3]);
            const int bl = (i >> 4) + (c >> 1);             // 0, 1 or 2
#pragma unroll
            for (int k2 = 0; k2 < 3; ++k2)
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(w_out + k2 * kTri + bl * 512 + block(i & 15, c & 1)),
                             "r"(w[0][k2]), "r"(w[1][k2]), "r"(w[2][k2]), "r"(w[3][k2]) : "memory");
        }
    }
}

}  // namespace dm
}  // namespace wkv7
