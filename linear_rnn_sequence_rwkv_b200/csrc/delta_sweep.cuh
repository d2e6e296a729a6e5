// The gated delta rule over whole sequences, 32 tokens at a time. Within a chunk that starts from S,
// with G the running sums of the log decays, D_ij = exp(G_i - G_j) and unit (or given) q, k:
//     X = V - exp(G) (K S^T),  E = W X,  W = (I + A)^-1,  A_ij = D_ij beta_j k_i.k_j (j < i)
//     Y = exp(G) (Q S^T) + P E,  P_ij = scale D_ij beta_j q_i.k_j (j <= i)
//     S <- exp(G_C) S + (exp(G_C - G) beta E)^T K
// The rows of S (value channels) never meet, so a warp owns 16 of them and walks the sequence with
// everything transposed: S [16][N], X^T, E^T and Y^T [16][32] are accumulator fragments, and each is the
// next product's left operand after a split into bf16 terms. Only K, Q, W and P come from shared memory.
// Four more warps load the chunks ahead and prepare W and P (delta_mma.cuh), two to a chunk; they meet the
// others at named barriers, `full` and `empty` per stage.
// The state keeps fp32's accuracy (three terms wherever it is read or written). A bf16 y is summed from S, P
// and E in two terms: one would do for gates and keys as they usually are, but where keys repeat the
// errors e_j alternate in sign and cancel in y, and a P of one term then missed y by four roundings.
#pragma once

#include "delta_mma.cuh"

namespace wkv7 {
namespace dm {

// STATES: the backward's forward sweep, which keeps the errors E and every second chunk's first state and
// has no use for the queries.
template <int NN, int RW, bool F32, bool STATES, int GROUPS>
struct Layout {
    static constexpr int TI = F32 ? 3 : 1, TP = STATES ? 0 : F32 ? 3 : 2;
    static constexpr int KB = TI * C * NN * 2;              // keys (and as much for queries)
    static constexpr int VB = F32 ? 0 : C * RW * 32;        // values of the CTA's rows; y on its way out
    static constexpr int kK = 0, kQ = KB, kV = STATES ? KB : 2 * KB, kW = kV + VB, kP = kW + 3 * kTri, kS = kP + TP * kTri;
    static constexpr int stage = (kS + int(sizeof(Scalars)) + 255) / 256 * 256;
    // GROUPS chunks being prepared, one at work, and the rest loading: what two CTAs of N = 64 bf16 with two
    // groups, or one of the others, have room (and named barriers) for
    static constexpr int stages = F32 ? (NN == 64 ? 6 : 3) : (NN == 64 && GROUPS == 2 ? 5 : 6);
    static constexpr int own = STATES && !F32 ? 64 * NN : 0;           // bytes of each state warp's own
    static constexpr int kOwn = stages * stage, kPrep = kOwn + RW * own;
    static constexpr int total = kPrep + GROUPS * int(sizeof(PrepScratch));
    static constexpr int threads = RW * 32 + GROUPS * kGroup, meet = RW * 32 + kGroup;
};

// Below it a number's first bf16 term is finite; from it on, up to fp32's own largest, the terms would be infinite.
constexpr float kTermMost = 0x1.ffp127f;

// Values that are not finite (or as good as that: kTermMost) leave the products (0) and their places the mask: bit 4 n + e.
__device__ __forceinline__ void take_out(float (&x)[4][4], uint32_t &mask) {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool ok = fabsf(x[n][e]) < kTermMost;
            mask |= ok ? 0u : 1u << (4 * n + e);
            x[n][e] = ok ? x[n][e] : 0.f;
        }
}
// Index (0 .. C) of the first such token of the row that holds elements r, r + 1 of this lane's tiles
// (tokens 8 n + 2 t, + 1), over the four lanes of the row.
__device__ __forceinline__ int first_bad(uint32_t mask, int r) {
    int at = C;
#pragma unroll
    for (int n = 3; n >= 0; --n)
#pragma unroll
        for (int f = 1; f >= 0; --f)
            if (mask >> (4 * n + r + f) & 1) at = 8 * n + 2 * (threadIdx.x & 3) + f;
    at = min(at, __shfl_xor_sync(0xffffffffu, at, 1));
    return min(at, __shfl_xor_sync(0xffffffffu, at, 2));
}

// A row's outputs from its first bad token on.
__device__ __forceinline__ void poison(float (&y)[4][4], uint32_t mask) {
    const int from[2] = {first_bad(mask, 0), first_bad(mask, 2)};
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (8 * n + 2 * int(threadIdx.x & 3) + (e & 1) >= from[e >> 1]) y[n][e] = __int_as_float(0x7fffffff);
}

template <int NN, int RW, bool F32, bool STATES, int GROUPS>
__device__ __forceinline__ void forward_sweep(const DeltaArgs &p, unsigned block) {
    using L = Layout<NN, RW, F32, STATES, GROUPS>;
    using Tin = std::conditional_t<F32, float, __nv_bfloat16>;
    constexpr int TI = L::TI, TP = L::TP, TS = F32 ? 3 : 2, NB = NN * 2, TB = C * NB, VNB = RW * 32;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_addr(sm);
    constexpr int slices = NN / (16 * RW);
    const unsigned unit = block / slices;
    const int row0 = (block % slices) * 16 * RW;           // first value row of the CTA
    const int s = unit / unsigned(p.H), h = unit % unsigned(p.H), hk = h / (p.H / p.Hk);
    long long t0, t1;
    delta_rows(p.cu, p.T, s, t0, t1);
    const int chunks = int((t1 - t0 + C - 1) / C);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int full = GROUPS, empty = full + L::stages;       // named barriers; 0 .. GROUPS - 1: the groups' own
    static_assert(empty + L::stages <= 16 && L::stages > GROUPS, "sixteen named barriers; a stage for what is at work");

    if (threadIdx.x >= RW * 32) {           // ---- preparing warps: group g takes chunks g, g + GROUPS, ... ----
        const int group = (threadIdx.x - RW * 32) / kGroup, tid = (threadIdx.x - RW * 32) % kGroup;
        PrepScratch *ps = reinterpret_cast<PrepScratch *>(sm + L::kPrep) + group;
        RowLoader<NN, F32> k(p.k, t0 + group * C, (long long)hk * NN, p.ks, tid), q(p.q, t0 + group * C, (long long)hk * NN, p.qs, tid);
        RowLoader<RW * 16, F32> v(p.v, t0 + group * C, (long long)h * NN + row0, p.vs, tid);
        Gate<F32> gate, next{};
        auto load = [&](int c) {
            const uint32_t st = base + (c % L::stages) * L::stage;
            const int n = int(min((long long)C, t1 - t0 - (long long)c * C));
            next.load(p.g, p.beta, (t0 + (long long)c * C + lane) * p.H + h, lane < n);
            k.load(st + L::kK, n);
            if constexpr (!STATES) q.load(st + L::kQ, n);
            if constexpr (!F32) v.load(st + L::kV, n);
            k.advance(GROUPS);
            q.advance(GROUPS);
            v.advance(GROUPS);
            cp_commit();
        };
        if (group < chunks) load(group);
        for (int c = group; c < chunks; c += GROUPS) {
            gate = next;
            if (c + GROUPS < chunks) {
                if (c + GROUPS >= L::stages) bar_sync(empty + (c + GROUPS) % L::stages, L::meet);
                load(c + GROUPS);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            bar_sync(group, kGroup);
            unsigned char *st = sm + (c % L::stages) * L::stage;
            const uint32_t sa = base + (c % L::stages) * L::stage;
            // the longer of the two roles changes between the warps, and with them the schedulers
            const bool queries = ((warp ^ (c / GROUPS)) & 1) != 0;
            Scalars *sc = reinterpret_cast<Scalars *>(st + L::kS);
            const float g = delta_clamp(gate.num(gate.g)), bt = gate.num(gate.beta);
            prepare_chunk<NN, TI, TP>(sa + L::kK, sa + L::kQ, st + L::kW, sa + L::kP, sc, ps, p, g, bt, queries, group);
            bar_arrive(full + c % L::stages, L::meet);
        }
        return;
    }

    // ---- one warp per 16 value rows ----
    const int gr = lane >> 2, tc = lane & 3;
    const int row = row0 + 16 * warp;
    const size_t ys = size_t(p.H) * NN;
    Tin *y = static_cast<Tin *>(STATES ? p.keep_E : p.y) + size_t(h) * NN + row;
    [[maybe_unused]] const long long slot0 = delta_slot(t0, s);
    // y (bf16, tokens t ..) from its fragments through the values' place (this warp's own columns) to whole
    // 32-byte pieces
    auto put = [&](Tin *to, uint32_t st, int n_tok, const uint32_t (&r)[2][4]) {
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int tok = 16 * m + (lane & 7) + ((lane >> 4) << 3);
            stsm4t(st + L::kV + tile<VNB>(tok, 2 * warp + ((lane >> 3) & 1)), r[m]);
        }
        __syncwarp();
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const int tok = 16 * m + (lane >> 1);
            uint4 u;
            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "r"(st + L::kV + tile<VNB>(tok, 2 * warp + (lane & 1))) : "memory");
            if (tok < n_tok) *reinterpret_cast<uint4 *>(to + tok * ys + 8 * (lane & 1)) = u;
        }
    };
    const size_t so = (size_t(unit) * NN + row) * NN;
    float S[NN / 8][4];
#pragma unroll
    for (int n = 0; n < NN / 8; ++n) {
        float2 a = make_float2(0, 0), b = a;
        if (p.S0) {
            a = __ldg(reinterpret_cast<const float2 *>(p.S0 + so + gr * NN + 8 * n + 2 * tc));
            b = __ldg(reinterpret_cast<const float2 *>(p.S0 + so + (gr + 8) * NN + 8 * n + 2 * tc));
        }
        S[n][0] = a.x; S[n][1] = a.y; S[n][2] = b.x; S[n][3] = b.y;
    }
    const Tin *vrow = static_cast<const Tin *>(p.v) + size_t(h) * NN + row;
    int stage = -1;
    for (int c = 0; c < chunks; ++c) {
        stage = stage + 1 == L::stages ? 0 : stage + 1;
        const uint32_t st = base + stage * L::stage;
        const Scalars *sc = reinterpret_cast<const Scalars *>(sm + stage * L::stage + L::kS);
        [[maybe_unused]] const long long t = t0 + (long long)c * C;
        [[maybe_unused]] const int n_tok = int(min((long long)C, t1 - t));
        Acc<F32, 4> xa, ya, ea;
        float (&X)[4][4] = xa.d, (&Y)[4][4] = ya.d, (&E)[4][4] = ea.d;
        [[maybe_unused]] float V[4][4];
        [[maybe_unused]] uint32_t vraw[2][4];
        if constexpr (F32) {    // loaded under the products
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 8 * n + 2 * tc + (e & 1);
                    V[n][e] = i < n_tok ? __ldg(vrow + (t + i) * p.vs + gr + 8 * (e >> 1)) : 0.f;
                }
        }
        if constexpr (STATES) {         // what the grads' chunks of 64 tokens start from
            if (c % 2 == 0) keep_state<F32, NN>(p.keep_S, p.keep_second, (slot0 + c / 2) * p.H + h, row, S, base + L::kOwn + warp * L::own);
        }
        bar_sync(full + stage, L::meet);
        // X^T = S K^T, Y^T = S Q^T
#pragma unroll
        for (int ks = 0; ks < NN / 16; ++ks) {
            uint32_t a[3][4], b[TI][2][4];
            split_a<3>(S[2 * ks], S[2 * ks + 1], a);
#pragma unroll
            for (int i = 0; i < TI; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n) ldsm4(b[i][n], addr_b<NB>(st + L::kK + i * TB, 16 * n, ks));
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int z = TI - 1; z >= 0; --z) {
                    if (x + z > 2) continue;
#pragma unroll
                    for (int n = 0; n < 4; ++n) xa.add(n, x + z == 0, a[x], b[z][n >> 1][2 * (n & 1)], b[z][n >> 1][2 * (n & 1) + 1]);
                }
            if constexpr (!STATES) {
#pragma unroll
                for (int i = 0; i < TI; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n) ldsm4(b[i][n], addr_b<NB>(st + L::kQ + i * TB, 16 * n, ks));
#pragma unroll
                for (int x = TS - 1; x >= 0; --x)
#pragma unroll
                    for (int z = TI - 1; z >= 0; --z) {
                        if (x + z > TS - 1) continue;
#pragma unroll
                        for (int n = 0; n < 4; ++n) ya.add(n, x + z == 0, a[x], b[z][n >> 1][2 * (n & 1)], b[z][n >> 1][2 * (n & 1) + 1]);
                    }
            }
        }
        float z = 0.f;
        if constexpr (!F32) {   // the values, transposed on the way: tokens 2 t, 2 t + 1 of rows g and g + 8
            __nv_bfloat162 zz = __float2bfloat162_rn(0.f);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int tok = 16 * m + (lane & 7) + ((lane >> 4) << 3);
                ldsm4t(vraw[m], st + L::kV + tile<VNB>(tok, 2 * warp + ((lane >> 3) & 1)));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    zz = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&vraw[m][i]), __float2bfloat162_rn(0.f), zz);
            }
            z = __low2float(zz) + __high2float(zz);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) z += fabsf(V[n][e]) < kTermMost ? 0.f : 1.f;
        }
        // A value that is not finite makes its row so from its token on and no earlier, which products with
        // the zeros of W and P would not keep. In a chunk with such inputs (NaN or infinite v, k, g or beta)
        // such values are taken out of the products, and what follows them is set at the end.
        const bool careful = sc->odd || __any_sync(0xffffffffu, z != 0.f);       // the same in every lane
        if constexpr (!F32) {
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                V[n][0] = lo_f(vraw[n >> 1][2 * (n & 1)]);
                V[n][1] = hi_f(vraw[n >> 1][2 * (n & 1)]);
                V[n][2] = lo_f(vraw[n >> 1][2 * (n & 1) + 1]);
                V[n][3] = hi_f(vraw[n >> 1][2 * (n & 1) + 1]);
            }
        }
        xa.join();
        ya.join();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 in = *reinterpret_cast<const float2 *>(&sc->kin[8 * n + 2 * tc]);
            float2 qn;
            if constexpr (!STATES) qn = *reinterpret_cast<const float2 *>(&sc->qin[8 * n + 2 * tc]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                X[n][e] = fmaf(-(e & 1 ? in.y : in.x), X[n][e], V[n][e]);
                if constexpr (!STATES) Y[n][e] *= e & 1 ? qn.y : qn.x;
            }
        }
        uint32_t bad = 0;
        if (careful) take_out(X, bad);
        // E^T = X^T W^T; four accumulators at a time, so that none waits for its own last product
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint32_t a[3][4], w[2][3][4];
            split_a<3>(X[2 * kb], X[2 * kb + 1], a);
#pragma unroll
            for (int ib = kb; ib < 2; ++ib)
#pragma unroll
                for (int z = 0; z < 3; ++z) ldsm4(w[ib][z], addr_block(st + L::kW + z * kTri + (ib + kb) * 512));
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int z = 2 - x; z >= 0; --z)
#pragma unroll
                    for (int ib = kb; ib < 2; ++ib) {
                        ea.add(2 * ib, x + z == 0, a[x], w[ib][z][0], w[ib][z][1]);
                        ea.add(2 * ib + 1, x + z == 0, a[x], w[ib][z][2], w[ib][z][3]);
                    }
        }
        ea.join();
        if (careful) take_out(E, bad);
        if constexpr (STATES) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) Y[n][e] = E[n][e];
        }
        // Y^T += E^T P^T
#pragma unroll
        for (int kb = 0; kb < (STATES ? 0 : 2); ++kb) {
            uint32_t a[TS][4];
            split_a<TS>(E[2 * kb], E[2 * kb + 1], a);
#pragma unroll
            for (int ib = kb; ib < 2; ++ib) {
                uint32_t w[TP > 0 ? TP : 1][4];
#pragma unroll
                for (int z = 0; z < TP; ++z) ldsm4(w[z], addr_block(st + L::kP + z * kTri + (ib + kb) * 512));
#pragma unroll
                for (int x = TS - 1; x >= 0; --x)
#pragma unroll
                    for (int z = TP - 1; z >= 0; --z) {
                        if (x + z > TS - 1) continue;
                        ya.add(2 * ib, x + z == 0, a[x], w[z][0], w[z][1]);
                        ya.add(2 * ib + 1, x + z == 0, a[x], w[z][2], w[z][3]);
                    }
            }
        }
        ya.join();
        // S <- exp(G_C) S + U^T K, U = out E: what is added is summed on its own, small products first
        const float whole = sc->whole;
        uint32_t u[2][3][4];
        {
            float U[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const float2 o = *reinterpret_cast<const float2 *>(&sc->out[8 * n + 2 * tc]);
#pragma unroll
                for (int e = 0; e < 4; ++e) U[n][e] = E[n][e] * (e & 1 ? o.y : o.x);
            }
            split_a<3>(U[0], U[1], u[0]);
            split_a<3>(U[2], U[3], u[1]);
        }
        constexpr int NP = TI == 1 ? 2 : 1;     // 16 or 32 key channels at a time: four accumulators
#pragma unroll
        for (int n = 0; n < NN / 16; n += NP) {
            uint32_t b[NP][2][TI][4];
            float d[NP][2][4];
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                    for (int z = 0; z < TI; ++z) ldsm4t(b[m][kb][z], addr_bt<NB>(st + L::kK + z * TB, 16 * kb, 2 * (n + m)));
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int z = TI - 1; z >= 0; --z) {
                    if (x + z > 2) continue;
#pragma unroll
                    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
                        for (int m = 0; m < NP; ++m) {
                            if (x == 2 && z == 0 && kb == 0) {
                                mma0(d[m][0], u[kb][x], b[m][kb][z][0], b[m][kb][z][1]);
                                mma0(d[m][1], u[kb][x], b[m][kb][z][2], b[m][kb][z][3]);
                            } else {
                                mma(d[m][0], u[kb][x], b[m][kb][z][0], b[m][kb][z][1]);
                                mma(d[m][1], u[kb][x], b[m][kb][z][2], b[m][kb][z][3]);
                            }
                        }
                }
#pragma unroll
            for (int m = 0; m < NP; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    S[2 * (n + m)][e] = fmaf(whole, S[2 * (n + m)][e], d[m][0][e]);
                    S[2 * (n + m) + 1][e] = fmaf(whole, S[2 * (n + m) + 1][e], d[m][1][e]);
                }
        }
        if (careful) {
            poison(Y, bad);
            const int from[2] = {first_bad(bad, 0), first_bad(bad, 2)};
#pragma unroll
            for (int n = 0; n < NN / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (from[e >> 1] < C) S[n][e] = __int_as_float(0x7fffffff);
        }
        if constexpr (F32) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 8 * n + 2 * tc + (e & 1);
                    if (i < n_tok) y[(t + i) * ys + gr + 8 * (e >> 1)] = Y[n][e];
                }
        } else if constexpr (STATES) {
            put_terms(y + t * ys, y + t * ys + p.keep_lo, ys, n_tok, Y, base + L::kOwn + warp * L::own);
        } else {
            uint32_t o[2][4];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[m][i] = pack(Y[2 * m + (i >> 1)][2 * (i & 1)], Y[2 * m + (i >> 1)][2 * (i & 1) + 1]);
            put(y + t * ys, st, n_tok, o);
        }
        if (c + L::stages < chunks) bar_arrive(empty + stage, L::meet);
    }
    if (p.S_T) {
#pragma unroll
        for (int n = 0; n < NN / 8; ++n) {
            *reinterpret_cast<float2 *>(p.S_T + so + gr * NN + 8 * n + 2 * tc) = make_float2(S[n][0], S[n][1]);
            *reinterpret_cast<float2 *>(p.S_T + so + (gr + 8) * NN + 8 * n + 2 * tc) = make_float2(S[n][2], S[n][3]);
        }
    }
}

}  // namespace dm
}  // namespace wkv7
