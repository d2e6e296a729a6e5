// The gated delta rule's backward: two sweeps, in one launch or two, then the gradients, and where a key head's value
// heads are divided the sum of the parts. With the chunk quantities of delta_sweep.cuh and
// dS' the gradient of a chunk's last state:
//   1. the forward sweep (delta_sweep.cuh, STATES): the errors E, and the state every 64 tokens start from;
//   2. the reverse sweep: the chain back through the chunks of 32,
//          dE = P^T dY + out (K dS'^T),   dX = W^T dE,   dV = dX,
//          dS = exp(G_C) dS' + (qin dY)^T Q - (kin dX)^T K
//      (out, qin, kin: the scalars of delta_mma.cuh). As forward, the rows of dS never meet: a warp owns 16 of
//      them, in accumulators, and the chain runs through its registers. Neither sweep needs anything of the other, so
//      that one launch may run both (delta_sweeps_kernel);
//   3. delta_grad_kernel: everything that contracts over the value channels, for all chunks of 64 at once:
//          A = dY E^T (j <= i), B = dX E^T (j < i), n = sq_i rk_j D beta_j A, o = rk_i rk_j D beta_j B
//          sq dQ = n K + qin (dY S),    rk dK = n^T Q - o K - o^T K + out (E dS') - kin (dX S)
//          z = (n (Q K^T) - o (K K^T)) / beta_j,   tail_j = kout_j k_j.(E dS')_j
//          dbeta_j = sum_i z_ij + tail_j
//          dG_i = sum_{j<i} beta_j z_ij - beta_i sum_{j>i} z_ji + q_i.(qin dY S)_i - k_i.(kin dX S)_i
//          dg_t = sum_{i >= t} dG_i + sum_{j < t} beta_j tail_j + exp(G_C) <S, dS'>
//      (rk, sq: 1 / |k| and scale / |q|; with unit keys dk = rk dK - k^ (k^.rk dK), and q alike).
//      The value heads of one key head are summed in the same accumulators, in order; where that would leave SMs idle
//      they go to several CTAs, whose sums delta_grad_sum_kernel adds up in order.
// Precision: the chain of dS keeps three bf16 terms wherever a state or its gradient is read or written. For
// outputs in bf16, everything computed (E, dX, S, dS', n, o) enters the sums in two terms, 16 bits: dg is a
// difference of large sums and would show a single term's rounding several times over.
#include "delta_sweep.cuh"

#include <algorithm>

namespace wkv7 {

using namespace dm;

namespace {

template <int NN, int RW, bool F32, int GROUPS>
struct RevLayout {
    static constexpr int TI = F32 ? 3 : 1, TP = 3;
    static constexpr int KB = TI * C * NN * 2, YB = TI * C * RW * 32;
    static constexpr int kK = 0, kQ = KB, kY = 2 * KB, kW = kY + YB, kP = kW + 3 * kTri, kS = kP + TP * kTri;
    static constexpr int stage = (kS + int(sizeof(Scalars)) + 255) / 256 * 256;
    static constexpr int stages = F32 ? (NN == 64 ? 4 : 3) : (GROUPS == 2 ? 4 : 6);
    static constexpr int own = F32 ? 0 : 64 * NN;
    static constexpr int kOwn = stages * stage, kPrep = kOwn + RW * own;
    static constexpr int total = kPrep + GROUPS * int(sizeof(PrepScratch));
    static constexpr int meet = RW * 32 + kGroup;
};

template <int NN, int RW, bool F32, int GROUPS>
__device__ __forceinline__ void reverse_sweep(const DeltaArgs &p, unsigned block) {
    using L = RevLayout<NN, RW, F32, GROUPS>;
    using Tin = std::conditional_t<F32, float, __nv_bfloat16>;
    constexpr int TI = L::TI, NB = NN * 2, TB = C * NB, YNB = RW * 32, YTB = C * YNB;
    extern __shared__ __align__(1024) unsigned char sm[];
    const uint32_t base = smem_addr(sm);
    constexpr int slices = NN / (16 * RW);
    const unsigned unit = block / slices;
    const int row0 = (block % slices) * 16 * RW;
    const int s = unit / unsigned(p.H), h = unit % unsigned(p.H), hk = h / (p.H / p.Hk);
    long long t0, t1;
    delta_rows(p.cu, p.T, s, t0, t1);
    const int chunks = int((t1 - t0 + C - 1) / C);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int full = GROUPS, empty = full + L::stages;       // named barriers; 0 .. GROUPS - 1: the groups' own

    // step r takes chunk chunks - 1 - r
    if (warp >= RW) {
        const int group = (warp - RW) >> 1, tid = (threadIdx.x - RW * 32) % kGroup;
        PrepScratch *ps = reinterpret_cast<PrepScratch *>(sm + L::kPrep) + group;
        const long long first = t0 + (long long)(chunks - 1 - group) * C;
        RowLoader<NN, F32> k(p.k, first, (long long)hk * NN, p.ks, tid), q(p.q, first, (long long)hk * NN, p.qs, tid);
        RowLoader<RW * 16, F32> dy(p.dy, first, (long long)h * NN + row0, (long long)p.H * NN, tid);
        Gate<F32> gate, next{};
        auto load = [&](int r) {
            const uint32_t st = base + (r % L::stages) * L::stage;
            const long long at = (long long)(chunks - 1 - r) * C;
            const int n = int(min((long long)C, t1 - t0 - at));
            next.load(p.g, p.beta, (t0 + at + lane) * p.H + h, lane < n);
            k.load(st + L::kK, n);
            q.load(st + L::kQ, n);
            dy.load(st + L::kY, n);
            k.advance(-GROUPS);
            q.advance(-GROUPS);
            dy.advance(-GROUPS);
            cp_commit();
        };
        if (group < chunks) load(group);
        for (int r = group; r < chunks; r += GROUPS) {
            gate = next;
            if (r + GROUPS < chunks) {
                if (r + GROUPS >= L::stages) bar_sync(empty + (r + GROUPS) % L::stages, L::meet);
                load(r + GROUPS);
                cp_wait<1>();
            } else {
                cp_wait<0>();
            }
            bar_sync(group, kGroup);
            unsigned char *st = sm + (r % L::stages) * L::stage;
            const uint32_t sa = base + (r % L::stages) * L::stage;
            const bool queries = ((warp ^ (r / GROUPS)) & 1) != 0;
            prepare_chunk<NN, TI, 3>(sa + L::kK, sa + L::kQ, st + L::kW, sa + L::kP, reinterpret_cast<Scalars *>(st + L::kS), ps, p,
                                     delta_clamp(gate.num(gate.g)), gate.num(gate.beta), queries, group);
            bar_arrive(full + r % L::stages, L::meet);
        }
        return;
    }

    const int gr = lane >> 2, tc = lane & 3, row = row0 + 16 * warp;
    const size_t so = (size_t(unit) * NN + row) * NN;
    float S[NN / 8][4];             // dS
#pragma unroll
    for (int n = 0; n < NN / 8; ++n) {
        float2 a = make_float2(0, 0), b = a;
        if (p.dS_T) {
            a = *reinterpret_cast<const float2 *>(p.dS_T + so + gr * NN + 8 * n + 2 * tc);
            b = *reinterpret_cast<const float2 *>(p.dS_T + so + (gr + 8) * NN + 8 * n + 2 * tc);
        }
        S[n][0] = a.x; S[n][1] = a.y; S[n][2] = b.x; S[n][3] = b.y;
    }
    Tin *dv = static_cast<Tin *>(p.dv) + size_t(h) * NN + row;
    [[maybe_unused]] Tin *dlo = static_cast<Tin *>(p.keep_dlo) + size_t(h) * NN + row;
    const size_t ys = size_t(p.H) * NN;
    const long long slot0 = delta_slot(t0, s);
    const int tok_l = (lane & 7) + ((lane >> 4) << 3), col_l = 2 * warp + ((lane >> 3) & 1);
    for (int r = 0; r < chunks; ++r) {
        const int c = chunks - 1 - r;
        const uint32_t st = base + (r % L::stages) * L::stage;
        const Scalars *sc = reinterpret_cast<const Scalars *>(sm + (r % L::stages) * L::stage + L::kS);
        const long long t = t0 + (long long)c * C;
        const int n_tok = int(min((long long)C, t1 - t));
        if (r == 0 || c % 2 == 1) keep_state<F32, NN>(p.keep_dS, p.keep_second, (slot0 + c / 2) * p.H + h, row, S, base + L::kOwn + warp * L::own);
        bar_sync(full + r % L::stages, L::meet);
        // dE^T = out (dS K^T) + dY^T P
        Acc<F32, 4> ea, xa;
        float (&E)[4][4] = ea.d, (&X)[4][4] = xa.d;
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
                    for (int n = 0; n < 4; ++n) ea.add(n, x + z == 0, a[x], b[z][n >> 1][2 * (n & 1)], b[z][n >> 1][2 * (n & 1) + 1]);
                }
        }
        ea.join();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 o = *reinterpret_cast<const float2 *>(&sc->out[8 * n + 2 * tc]);
#pragma unroll
            for (int e = 0; e < 4; ++e) E[n][e] *= e & 1 ? o.y : o.x;
        }
        uint32_t y[2][TI][4];       // dY^T: rows are value channels, depth tokens
#pragma unroll
        for (int ib = 0; ib < 2; ++ib) {
#pragma unroll
            for (int i = 0; i < TI; ++i) ldsm4t(y[ib][i], st + L::kY + i * YTB + tile<YNB>(16 * ib + tok_l, col_l));
            uint32_t w[2][3][4];
#pragma unroll
            for (int jb = 0; jb <= ib; ++jb)
#pragma unroll
                for (int z = 0; z < 3; ++z) ldsm4t(w[jb][z], addr_block_t(st + L::kP + z * kTri + (ib + jb) * 512));
#pragma unroll
            for (int x = TI - 1; x >= 0; --x)
#pragma unroll
                for (int z = 2 - x; z >= 0; --z)
#pragma unroll
                    for (int jb = 0; jb <= ib; ++jb) {
                        ea.add(2 * jb, x + z == 0, y[ib][x], w[jb][z][0], w[jb][z][1]);
                        ea.add(2 * jb + 1, x + z == 0, y[ib][x], w[jb][z][2], w[jb][z][3]);
                    }
        }
        ea.join();
        // dX^T = dE^T W
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
            uint32_t a[3][4];
            split_a<3>(E[2 * kb], E[2 * kb + 1], a);
            uint32_t w[2][3][4];
#pragma unroll
            for (int jb = 0; jb <= kb; ++jb)
#pragma unroll
                for (int z = 0; z < 3; ++z) ldsm4t(w[jb][z], addr_block_t(st + L::kW + z * kTri + (kb + jb) * 512));
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int z = 2 - x; z >= 0; --z)
#pragma unroll
                    for (int jb = 0; jb <= kb; ++jb) {
                        xa.add(2 * jb, x + z == 0, a[x], w[jb][z][0], w[jb][z][1]);
                        xa.add(2 * jb + 1, x + z == 0, a[x], w[jb][z][2], w[jb][z][3]);
                    }
        }
        xa.join();
        // dS <- exp(G_C) dS + (qin dY)^T Q - (kin dX)^T K: each sum on its own, small products first
        const float whole = sc->whole;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
            uint32_t u[2][3][4];
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
                float w[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float2 f = *reinterpret_cast<const float2 *>(&(part ? sc->kin : sc->qin)[16 * kb + 8 * n + 2 * tc]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = part ? -X[2 * kb + n][e] : 0.f;
                        if (part == 0)
#pragma unroll
                            for (int i = TI - 1; i >= 0; --i) {
                                const uint32_t v = y[kb][i][2 * n + (e >> 1)];
                                x += e & 1 ? hi_f(v) : lo_f(v);
                            }
                        w[n][e] = x * (e & 1 ? f.y : f.x);
                    }
                }
                split_a<3>(w[0], w[1], u[kb]);
            }
            const uint32_t right = st + (part ? L::kK : L::kQ);
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
                        for (int z = 0; z < TI; ++z) ldsm4t(b[m][kb][z], addr_bt<NB>(right + z * TB, 16 * kb, 2 * (n + m)));
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
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float &x = S[2 * (n + m) + i][e];
                            x = part ? x + d[m][i][e] : fmaf(whole, x, d[m][i][e]);
                        }
            }
        }
        if constexpr (F32) {
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 8 * n + 2 * tc + (e & 1);
                    if (i < n_tok) dv[(t + i) * ys + gr + 8 * (e >> 1)] = X[n][e];
                }
        } else {
            put_terms(dv + t * ys, dlo + t * ys, ys, n_tok, X, base + L::kOwn + warp * L::own);
        }
        if (r + L::stages < chunks) bar_arrive(empty + r % L::stages, L::meet);
    }
    if (p.dS0) {
#pragma unroll
        for (int n = 0; n < NN / 8; ++n) {
            *reinterpret_cast<float2 *>(p.dS0 + so + gr * NN + 8 * n + 2 * tc) = make_float2(S[n][0], S[n][1]);
            *reinterpret_cast<float2 *>(p.dS0 + so + (gr + 8) * NN + 8 * n + 2 * tc) = make_float2(S[n][2], S[n][3]);
        }
    }
}

template <int NN, int RW, bool F32, int GROUPS>
__global__ void __launch_bounds__(RW * 32 + GROUPS * kGroup, (!F32 && NN == 64 && GROUPS == 2) ? 2 : 1) delta_sweeps_kernel(const DeltaArgs p, int which) {
    const bool both = which == 2;                       // else 0: the reverse sweep, 1: the forward one
    const unsigned block = both ? blockIdx.x >> 1 : blockIdx.x;
    if (both ? blockIdx.x & 1 : which) forward_sweep<NN, RW, F32, true, GROUPS>(p, block);
    else reverse_sweep<NN, RW, F32, GROUPS>(p, block);
}

// ---- the gradients of a chunk of 64 tokens ------------------------------------------------------------

constexpr int GC = 64, GT = 512;        // tokens, threads (16 warps: 4 row blocks of 16 by 4 column groups)

// Tokens t0 .. t0 + n - 1 of a sequence, number `slot` of all chunks; a key head, and `heads` of its value heads from
// `first` on. n = 0: none left. opens: the sequence starts here.
struct GradChunk {
    long long t0, slot;
    int n, hk, first, heads, part, opens;
};
struct GradScalars {
    float ghi[GC], glo[GC], rk[GC], sq[GC], beta[GC], kin[GC], qin[GC], kout[GC], out[GC];
    float up[GC], down[GC];         // near: D_ij = up_i down_j
    float open[GC];                 // 0 where nothing is left of the state before a token, 1 elsewhere
    float row[4][GC], tail[4][GC], col[4][GC], diag[GC], dq[4][GC], dk[4][GC];
    float ss[GT / 32];
    float whole;
    int near;                       // the chunk's sums of log decays stay within 30 of the middle one
    GradChunk chunk[2];             // at work and next, in turn
};

template <int NN, bool F32>
struct GradLayout {
    static constexpr int TI = F32 ? 3 : 1, TE = F32 ? 3 : 2, DW = F32 ? 32 : 64;   // DW: value channels at a time
    static constexpr int KB = GC * NN * 2, YB = GC * DW * 2, SB = DW * NN * 2, MB = GC * GC * 2;   // one term each
    // Two sets of tiles fit: a CTA per SM stays and loads the next chunk under the products of this one (8 x 1024 tokens
    // of 12 heads, the whole backward: 258 us against 270 with a CTA per chunk).
    static constexpr bool AHEAD = NN == 64 && !F32;
    static constexpr int kK = 0, kQ = TI * KB, kSlice = 2 * TI * KB;
    static constexpr int kY = kSlice, kE = kY + TI * YB, kX = kE + TE * YB, kS = kX + TE * YB, kD = kS + TE * SB;
    static constexpr int kN = kSlice, kO = kN + TE * MB;                 // n and -o, where the slice was
    static constexpr int slice_end = kD + TE * SB, mats_end = kO + TE * MB;
    static constexpr int kF = slice_end > mats_end ? slice_end : mats_end;
    static constexpr int total = (AHEAD ? 2 : 1) * kF + int(sizeof(GradScalars));
};

// Where a thread's pieces of a tile of ROWS rows of W elements lie: piece i is row r + i STEP, column chunk c.
template <int W, int ROWS>
struct Pieces {
    static constexpr int STEP = GT / (W / 8), N = (ROWS + STEP - 1) / STEP;
    int r;
    uint32_t to;            // of the first piece in the tile
    long long from, step;   // elements, of rows `stride` apart
    __device__ __forceinline__ Pieces(long long stride) {
        r = threadIdx.x / (W / 8);
        to = tile<W * 2>(r, threadIdx.x % (W / 8));
        from = r * stride + 8 * (threadIdx.x % (W / 8));
        step = STEP * stride;
    }
    // From an array of the inputs' type into a tile (rows from n on as zeros): bf16 asynchronously; fp32 as three
    // terms `term` bytes apart.
    template <bool F32>
    __device__ __forceinline__ void load(uint32_t dst, const void *src, int n, int term) const {
        const char *p = static_cast<const char *>(src) + from * (F32 ? 4 : 2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (ROWS % STEP && r + i * STEP >= ROWS) break;
            const bool there = r + i * STEP < n;
            const uint32_t at = dst + to + i * STEP * W * 2;        // eight rows or more on: the same place in the swizzle
            if constexpr (!F32) {
                cp16(at, there ? p + i * step * 2 : static_cast<const char *>(src), there);
            } else {
                float4 x = make_float4(0, 0, 0, 0), y = x;
                if (there) {
                    x = *reinterpret_cast<const float4 *>(p + i * step * 4);
                    y = *reinterpret_cast<const float4 *>(p + i * step * 4 + 16);
                }
                uint32_t w[4][3];
                split2<3>(x.x, x.y, w[0]);
                split2<3>(x.z, x.w, w[1]);
                split2<3>(y.x, y.y, w[2]);
                split2<3>(y.z, y.w, w[3]);
#pragma unroll
                for (int k = 0; k < 3; ++k) st_v4(at + k * term, w[0][k], w[1][k], w[2][k], w[3][k]);
            }
        }
    }
};

// d[0 .. CT) += a b over the pairs of terms that count: a TA terms of a left operand, b TB terms of right operands
// of 16 columns each. top: 1 only the leading pair, 0 only the others, -1 all.
template <int TA, int TB, int CT>
__device__ __forceinline__ void mma_terms(float (&d)[CT][4], const uint32_t (&a)[TA][4], const uint32_t (&b)[TB][CT / 2][4], int top = -1) {
    constexpr int most = (TA > TB ? TA : TB) - 1;
#pragma unroll
    for (int x = TA - 1; x >= 0; --x)
#pragma unroll
        for (int z = TB - 1; z >= 0; --z) {
            if (x + z > most || (top >= 0 && top != (x + z == 0))) continue;
#pragma unroll
            for (int n = 0; n < CT; ++n) mma(d[n], a[x], b[z][n >> 1][2 * (n & 1)], b[z][n >> 1][2 * (n & 1) + 1]);
        }
}

template <int N>
__device__ __forceinline__ void add_to(float (&x)[N][4], const float (&y)[N][4]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] += y[n][e];
}

__device__ __forceinline__ float quad_sum(float x) {        // over the lanes of one row
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
__device__ __forceinline__ float col_sum(float x) {         // over the eight rows of a tile
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// Two tiles' worth (16 columns from 16 ks on) of elements at the accumulators' places, rows m0 + gr and + 8:
// v[tile][row half], summed over the terms.
template <int NB, int TI>
__device__ __forceinline__ void pairs_at(float2 (&v)[2][2], uint32_t base, int term, int m0, int ks) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) v[t][r] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = TI - 1; i >= 0; --i) {
        uint32_t u[4];
        ldsm4(u, addr_a<NB>(base + i * term, m0, ks));
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                v[t][r].x += lo_f(u[2 * t + r]);
                v[t][r].y += hi_f(u[2 * t + r]);
            }
    }
}
// Eight elements of T terms, `term` bytes apart, from 16 bytes of each.
template <int T>
__device__ __forceinline__ void eight_at(float (&x)[8], uint32_t at, int term) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
    for (int i = T - 1; i >= 0; --i) {
        uint32_t u[4];
        ld_v4(u, at + i * term);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] += lo_f(u[e]);
            x[2 * e + 1] += hi_f(u[e]);
        }
    }
}

// The first task from `task` on that has tokens: task = ((chunk number) * Hk + key head) * parts + part, where a key head's
// value heads go to `parts` tasks.
__device__ __forceinline__ GradChunk grad_chunk(const DeltaArgs &p, unsigned &task, unsigned tasks, int parts) {
    for (; task < tasks; task += gridDim.x) {
        const unsigned whole = parts == 1 ? task : task / unsigned(parts), number = p.Hk == 1 ? whole : whole / unsigned(p.Hk);
        const long long slot = number;
        // the sequence of this chunk: the last one that starts at or before it
        int s = 0;
        for (int lo = 0, hi = p.B; lo < hi;) {
            const int mid = (lo + hi) >> 1;
            const long long first = p.cu ? min(max(p.cu[mid], 0), p.T) : (long long)mid * p.T;
            if (delta_slot(first, mid) <= slot) {
                s = mid;
                lo = mid + 1;
            } else {
                hi = mid;
            }
        }
        long long t0, t1;
        delta_rows(p.cu, p.T, s, t0, t1);
        const long long chunk = slot - delta_slot(t0, s);
        t0 += chunk * GC;
        if (chunk >= 0 && t0 < t1) {
            const int hk = whole - number * p.Hk, part = task - whole * parts, n = int(min((long long)GC, t1 - t0));
            if (parts == 1) return {t0, slot, n, hk, hk * p.group, p.group, 0, chunk == 0};
            const int from = p.group * part / parts;
            return {t0, slot, n, hk, hk * p.group + from, p.group * (part + 1) / parts - from, part, chunk == 0};
        }
    }
    return {};
}

// A, B, dY S, dX S and E dS' are independent contractions; unlike the sweeps' chain nothing ties them to warp-level
// instructions, which are what this kernel was built from. 8 x 1024 tokens of 12 heads: 97 us, 29 % of the tensor pipe. Its
// 16 warps of 128 registers fill the SM; N = 128 and fp32 spill (396 bytes of stores; 476 at N = 64 fp32, 1080 at
// N = 128 fp32).
// SPLIT: a key head's value heads are divided into n_parts (one otherwise).
template <int NN, bool F32, bool SPLIT>
__global__ void __launch_bounds__(GT, 1) delta_grad_kernel(const DeltaArgs p, unsigned tasks, int n_parts) {
    using L = GradLayout<NN, F32>;
    using Tin = std::conditional_t<F32, float, __nv_bfloat16>;
    constexpr int TI = L::TI, TE = L::TE, DW = L::DW, NB = NN * 2, YNB = DW * 2, CT = NN / 32, CW = NN / 4;
    const int parts = SPLIT ? n_parts : 1;
    extern __shared__ __align__(1024) unsigned char sm[];
    GradScalars *sc = reinterpret_cast<GradScalars *>(sm + L::total - sizeof(GradScalars));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, tc = lane & 3;
    constexpr int scalar_warp = 12;     // the one with the fewest products (wr = 0, wc = 3) sees to the gates
    const int wr = warp & 3, wc = warp >> 2, c0 = wc * CW, j0 = wc * 16;   // rows 16 wr; key channels c0; tokens j0 ..
    const Pieces<DW, GC> tok((long long)p.H * NN);
    const Pieces<NN, DW> sta(NN);
    auto load_keys = [&](uint32_t to, const GradChunk &c) {
        Pieces<NN, GC>(p.ks).template load<F32>(to + L::kK, static_cast<const Tin *>(p.k) + c.t0 * p.ks + c.hk * NN, c.n, L::KB);
        Pieces<NN, GC>(p.qs).template load<F32>(to + L::kQ, static_cast<const Tin *>(p.q) + c.t0 * p.qs + c.hk * NN, c.n, L::KB);
    };
    auto load_slice = [&](uint32_t to, const GradChunk &c, int h, int sl) {
        const long long ye = c.t0 * p.H * NN + (long long)h * NN + sl * DW, se = ((c.slot * p.H + h) * NN + sl * DW) * NN;
        tok.template load<F32>(to + L::kY, static_cast<const Tin *>(p.dy) + ye, c.n, L::YB);
        tok.template load<F32>(to + L::kE, static_cast<const Tin *>(p.keep_E) + ye, c.n, L::YB);
        tok.template load<F32>(to + L::kX, static_cast<const Tin *>(p.dv) + ye, c.n, L::YB);
        sta.template load<F32>(to + L::kS, static_cast<const Tin *>(p.keep_S) + se, DW, L::SB);
        sta.template load<F32>(to + L::kD, static_cast<const Tin *>(p.keep_dS) + se, DW, L::SB);
        if constexpr (!F32) {           // the second terms
            tok.template load<F32>(to + L::kE + L::YB, static_cast<const Tin *>(p.keep_E) + p.keep_lo + ye, c.n, L::YB);
            tok.template load<F32>(to + L::kX + L::YB, static_cast<const Tin *>(p.keep_dlo) + ye, c.n, L::YB);
            sta.template load<F32>(to + L::kS + L::SB, static_cast<const Tin *>(p.keep_S) + p.keep_second + se, DW, L::SB);
            sta.template load<F32>(to + L::kD + L::SB, static_cast<const Tin *>(p.keep_dS) + p.keep_second + se, DW, L::SB);
        }
    };
    unsigned at_task = blockIdx.x;
    GradChunk *cur = &sc->chunk[0];         // in shared memory: the registers are full
    {
        const GradChunk c = grad_chunk(p, at_task, tasks, parts);
        if (c.n == 0) return;
        if (tid == 0) *cur = c;
        __syncthreads();
    }
    // of the keys and queries, and of the slice: each moves to the other set and back
    const uint32_t both = 2 * smem_addr(sm) + L::kF;
    uint32_t keys = smem_addr(sm), base = keys;
    load_keys(keys, *cur);
    if constexpr (L::AHEAD) load_slice(base, *cur, cur->first, 0);
    cp_commit();
    while (true) {
        const long long t0 = cur->t0;
        const int n = cur->n;
        float DQ[CT][4] = {}, DK[CT][4] = {};
        for (int hg = 0; hg < (SPLIT ? cur->heads : p.group); ++hg) {
            const int h = cur->first + hg;
            float A[2][4] = {}, B[2][4] = {}, QK[2][4] = {}, KK[2][4] = {}, aq[CT][4] = {}, ak[CT][4] = {}, ao[CT][4] = {};
            float ss = 0.f;
            for (int sl = 0; sl < NN / DW; ++sl) {
                [[maybe_unused]] Gate<F32> gates[2];
                if constexpr (L::AHEAD) cp_wait<0>();
                __syncthreads();            // the last readers of what lies there
                if constexpr (L::AHEAD) {
                    if (warp == scalar_warp) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) gates[e].load(p.g, p.beta, (t0 + 2 * lane + e) * p.H + h, 2 * lane + e < n);
                    }
                    if (hg + 1 < (SPLIT ? cur->heads : p.group)) {
                        // the keys and queries stay where they are
                        load_slice(both - base, *cur, h + 1, 0);
                    } else {
                        const GradChunk next = grad_chunk(p, at_task += gridDim.x, tasks, parts);
                        if (tid == 0) (cur == &sc->chunk[0] ? sc->chunk[1] : sc->chunk[0]) = next;
                        if (next.n) {
                            load_keys(both - keys, next);
                            load_slice(both - base, next, next.first, 0);
                        }
                    }
                } else {
                    load_slice(base, *cur, h, sl);
                }
                cp_commit();
                if (sl == 0) {              // what needs only keys, queries and gates, while the slice is on its way
                    if (hg == 0) {          // lengths: four threads per row, keys then queries
                        if constexpr (!L::AHEAD) {
                            cp_wait<1>();
                            __syncthreads();
                        }
                        const int row = (tid >> 2) & 63, part = tid & 3;
                        const uint32_t at = keys + (tid < 256 ? L::kK : L::kQ);
                        float l = 0.f;
#pragma unroll
                        for (int c = 0; c < NN / 32; ++c) {
                            float x[8];
                            eight_at<TI>(x, at + tile<NB>(row, part * (NN / 32) + c), L::KB);
#pragma unroll
                            for (int e = 0; e < 8; ++e) l = fmaf(x[e], x[e], l);
                        }
                        l = quad_sum(l);
                        l = p.qk_norm ? delta_unit(l, p.norm_eps) : 1.f;
                        if (part == 0) (tid < 256 ? sc->rk : sc->sq)[row] = tid < 256 ? l : l * p.scale;
                        __syncthreads();
                    }
                    // the keys' and queries' products
                    if (wc <= wr) {
#pragma unroll
                        for (int pass = 0; pass < (F32 ? 2 : 1); ++pass)
#pragma unroll 1
                            for (int ks = 0; ks < NN / 16; ++ks) {
                                uint32_t a[TI][4], d[TI][4], b[TI][1][4];
#pragma unroll
                                for (int i = 0; i < TI; ++i) {
                                    ldsm4(a[i], addr_a<NB>(keys + L::kQ + i * L::KB, 16 * wr, ks));
                                    ldsm4(d[i], addr_a<NB>(keys + L::kK + i * L::KB, 16 * wr, ks));
                                    ldsm4(b[i][0], addr_b<NB>(keys + L::kK + i * L::KB, j0, ks));
                                }
                                mma_terms<TI, TI, 2>(QK, a, b, F32 ? pass : -1);
                                mma_terms<TI, TI, 2>(KK, d, b, F32 ? pass : -1);
                            }
                    }
                    if (warp == scalar_warp) {        // the decays: two tokens per lane
                        float g[2], b[2];
                        long long G[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = 2 * lane + e;
                            if constexpr (!L::AHEAD) gates[e].load(p.g, p.beta, (t0 + i) * p.H + h, i < n);
                            g[e] = delta_clamp(gates[e].num(gates[e].g));
                            b[e] = gates[e].num(gates[e].beta);
                            G[e] = llrintf(fminf(g[e], 120.f) * 4294967296.f);
                        }
                        const bool nan = __any_sync(0xffffffffu, g[0] != g[0] || g[1] != g[1]);
                        const long long second = G[1];
                        G[1] += G[0];
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const long long x = __shfl_up_sync(0xffffffffu, G[1], o);
                            if (lane >= o) G[1] += x;
                        }
                        G[0] = G[1] - second;
                        const long long last = __shfl_sync(0xffffffffu, G[1], 31), mid = __shfl_sync(0xffffffffu, G[1], 15);
                        const bool near = !nan && __all_sync(0xffffffffu, llabs(G[0] - mid) < (30ll << 32) && llabs(G[1] - mid) < (30ll << 32));
                        if (lane == 0) sc->near = near;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = 2 * lane + e;
                            const float bad = nan ? __int_as_float(0x7fffffff) : 0.f;
                            const float in = expf(float(G[e]) * 2.3283064365386963e-10f) + bad;
                            const float to = expf(float(last - G[e]) * 2.3283064365386963e-10f);
                            sc->ghi[i] = float(int(G[e] >> 22)) * 9.765625e-4f + bad;
                            sc->glo[i] = float(int(G[e] & 0x3fffff)) * 2.3283064365386963e-10f;
                            sc->beta[i] = b[e];
                            sc->open[i] = g[e] <= -104.f || (i == 0 && cur->opens && !p.S0) ? 0.f : 1.f;    // exp(g) is 0
                            sc->kin[i] = in * sc->rk[i];
                            sc->qin[i] = in * sc->sq[i];
                            sc->kout[i] = to * sc->rk[i];
                            sc->out[i] = to * sc->rk[i] * b[e];
                            if (i == GC - 1) sc->whole = in;
                            // exp(G_i - mid) and its inverse: the high part's exponential, the low part's to second order
                            const long long off = near ? G[e] - mid : 0;
                            const float hi = float(int(off >> 22)) * 9.765625e-4f, lo = float(int(off & 0x3fffff)) * 2.3283064365386963e-10f;
                            const float up = expf(hi), down = expf(-hi), l2 = 0.5f * lo * lo;
                            sc->up[i] = fmaf(up, lo + l2, up);
                            sc->down[i] = fmaf(down, l2 - lo, down);
                        }
                    }
                }
                if constexpr (!L::AHEAD) {
                    cp_wait<0>();
                    __syncthreads();
                }
                // A, B over the value channels; dY S, dX S, E dS'. fp32: the slice's sums on their own, small products
                // first (the tensor cores cut as they add, see Acc), then added to the others.
                float tA[2][4] = {}, tB[2][4] = {}, tq[CT][4] = {}, tk[CT][4] = {}, to[CT][4] = {};
                float (&A_)[2][4] = F32 ? tA : A, (&B_)[2][4] = F32 ? tB : B;
                float (&q_)[CT][4] = F32 ? tq : aq, (&k_)[CT][4] = F32 ? tk : ak, (&o_)[CT][4] = F32 ? to : ao;
#pragma unroll
                for (int pass = 0; pass < (F32 ? 2 : 1); ++pass) {
                    const int top = F32 ? pass : -1;
#pragma unroll 1
                    for (int ks = 0; ks < DW / 16; ++ks) {
                        uint32_t y[TI][4], x[TE][4], e[TE][4];
#pragma unroll
                        for (int i = 0; i < TI; ++i) ldsm4(y[i], addr_a<YNB>(base + L::kY + i * L::YB, 16 * wr, ks));
#pragma unroll
                        for (int i = 0; i < TE; ++i) {
                            ldsm4(x[i], addr_a<YNB>(base + L::kX + i * L::YB, 16 * wr, ks));
                            ldsm4(e[i], addr_a<YNB>(base + L::kE + i * L::YB, 16 * wr, ks));
                        }
                        if (wc <= wr) {         // tokens j of this warp's column group are not all behind its rows
                            uint32_t b[TE][1][4];
#pragma unroll
                            for (int i = 0; i < TE; ++i) ldsm4(b[i][0], addr_b<YNB>(base + L::kE + i * L::YB, j0, ks));
                            mma_terms<TI, TE, 2>(A_, y, b, top);
                            mma_terms<TE, TE, 2>(B_, x, b, top);
                        }
                        uint32_t b[TE][CT / 2][4];
#pragma unroll
                        for (int i = 0; i < TE; ++i)
#pragma unroll
                            for (int m = 0; m < CT / 2; ++m) ldsm4t(b[i][m], addr_bt<NB>(base + L::kS + i * L::SB, 16 * ks, c0 / 8 + 2 * m));
                        mma_terms<TI, TE, CT>(q_, y, b, top);
                        mma_terms<TE, TE, CT>(k_, x, b, top);
#pragma unroll
                        for (int i = 0; i < TE; ++i)
#pragma unroll
                            for (int m = 0; m < CT / 2; ++m) ldsm4t(b[i][m], addr_bt<NB>(base + L::kD + i * L::SB, 16 * ks, c0 / 8 + 2 * m));
                        mma_terms<TE, TE, CT>(o_, e, b, top);
                    }
                }
                if constexpr (F32) {
                    add_to(A, tA);
                    add_to(B, tB);
                    add_to(aq, tq);
                    add_to(ak, tk);
                    add_to(ao, to);
                }
#pragma unroll
                for (int i = tid; i < DW * NN / 8; i += GT) {       // <S, dS'>: both tiles have one layout
                    float a[8], b[8];
                    eight_at<TE>(a, base + L::kS + i * 16, L::SB);
                    eight_at<TE>(b, base + L::kD + i * 16, L::SB);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(a[e], b[e], ss);
                }
            }
            __syncthreads();                // the slice has been read, the scalars are there
            // rows i = 16 wr + gr (+ 8), columns j = j0 + 8 m + 2 tc (+ 1)
            float rows[2] = {}, tails[2] = {};
            const bool near = sc->near != 0;
            float rn[2], ro[2], rh[2], rl[2];           // rows: factors of n and o, the sums of log decays
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 16 * wr + gr + 8 * e;
                const float f = near ? sc->up[i] : 1.f;
                rn[e] = f * sc->sq[i];
                ro[e] = f * sc->rk[i];
                rh[e] = sc->ghi[i];
                rl[e] = sc->glo[i];
            }
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int j = j0 + 8 * m + 2 * tc;
                float cols[2] = {}, cf[2], ch[2], cl[2], bt[2];
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    cf[f] = (near ? sc->down[j + f] : 1.f) * sc->rk[j + f];
                    ch[f] = sc->ghi[j + f];
                    cl[f] = sc->glo[j + f];
                    bt[f] = sc->beta[j + f];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 16 * wr + gr + 8 * e;
                    float vn[2], vo[2];
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const float d = near ? cf[f] : cf[f] * fast_exp((rh[e] - ch[f]) + (rl[e] - cl[f]));
                        const float nn = j + f <= i ? A[m][2 * e + f] * d * rn[e] : 0.f, oo = j + f < i ? B[m][2 * e + f] * d * ro[e] : 0.f;
                        const float z = nn * QK[m][2 * e + f] - oo * KK[m][2 * e + f];
                        if (j + f == i) {       // z_ii belongs to beta alone: g_i changes neither side of it
                            sc->diag[i] = z;
                        } else {
                            cols[f] += z;
                            rows[e] = fmaf(bt[f], z, rows[e]);
                        }
                        vn[f] = nn * bt[f];
                        vo[f] = -oo * bt[f];
                    }
                    uint32_t a[TE], b[TE];
                    split2<TE>(vn[0], vn[1], a);
                    split2<TE>(vo[0], vo[1], b);
                    const uint32_t to = base + tile<GC * 2>(i, j >> 3) + ((j & 7) << 1);
#pragma unroll
                    for (int z = 0; z < TE; ++z) {
                        st_b32(to + z * L::MB + L::kN, a[z]);
                        st_b32(to + z * L::MB + L::kO, b[z]);
                    }
                }
#pragma unroll
                for (int f = 0; f < 2; ++f) {
                    const float x = col_sum(cols[f]);
                    if (gr == 0) sc->col[wr][j + f] = x;
                }
            }
            // what came through the states, over this warp's key channels
            float fq[2], fk[2], fo[2], fb[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 16 * wr + gr + 8 * e;
                fq[e] = sc->qin[i];
                fk[e] = sc->kin[i];
                fo[e] = sc->kout[i];
                fb[e] = sc->out[i];
            }
#pragma unroll
            for (int t = 0; t < CT / 2; ++t) {
                float2 qv[2][2], kv[2][2];
                pairs_at<NB, TI>(qv, keys + L::kQ, L::KB, 16 * wr, c0 / 16 + t);
                pairs_at<NB, TI>(kv, keys + L::kK, L::KB, 16 * wr, c0 / 16 + t);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int m = 2 * t + u;
                        const float q0 = fq[e] * aq[m][2 * e], q1 = fq[e] * aq[m][2 * e + 1];
                        const float k0 = fk[e] * ak[m][2 * e], k1 = fk[e] * ak[m][2 * e + 1], o0 = ao[m][2 * e], o1 = ao[m][2 * e + 1];
                        rows[e] += fmaf(qv[u][e].x, q0, qv[u][e].y * q1) - fmaf(kv[u][e].x, k0, kv[u][e].y * k1);
                        tails[e] += fo[e] * fmaf(kv[u][e].x, o0, kv[u][e].y * o1);
                        DQ[m][2 * e] += q0;
                        DQ[m][2 * e + 1] += q1;
                        DK[m][2 * e] += fmaf(fb[e], o0, -k0);
                        DK[m][2 * e + 1] += fmaf(fb[e], o1, -k1);
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = quad_sum(rows[e]), y = quad_sum(tails[e]);
                if (tc == 0) {
                    sc->row[wc][16 * wr + gr + 8 * e] = x;
                    sc->tail[wc][16 * wr + gr + 8 * e] = y;
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (lane == 0) sc->ss[warp] = ss;
            __syncthreads();
            float tQ[CT][4] = {}, tK[CT][4] = {};
            float (&Q_)[CT][4] = F32 ? tQ : DQ, (&K_)[CT][4] = F32 ? tK : DK;
#pragma unroll
            for (int pass = 0; pass < (F32 ? 2 : 1); ++pass) {
                const int top = F32 ? pass : -1;
                // sq dQ += n K, rk dK -= o K: depth j up to this row block
#pragma unroll 1
                for (int kb = 0; kb <= wr; ++kb) {
                    uint32_t a[TE][4], d[TE][4], b[TI][CT / 2][4];
#pragma unroll
                    for (int i = 0; i < TE; ++i) {
                        ldsm4(a[i], addr_a<GC * 2>(base + L::kN + i * L::MB, 16 * wr, kb));
                        ldsm4(d[i], addr_a<GC * 2>(base + L::kO + i * L::MB, 16 * wr, kb));
                    }
#pragma unroll
                    for (int i = 0; i < TI; ++i)
#pragma unroll
                        for (int m = 0; m < CT / 2; ++m) ldsm4t(b[i][m], addr_bt<NB>(keys + L::kK + i * L::KB, 16 * kb, c0 / 8 + 2 * m));
                    mma_terms<TE, TI, CT>(Q_, a, b, top);
                    mma_terms<TE, TI, CT>(K_, d, b, top);
                }
                // rk dK += n^T Q - o^T K: depth i from this row block on
#pragma unroll 1
                for (int ib = wr; ib < 4; ++ib) {
                    uint32_t a[TE][4], d[TE][4], b[TI][CT / 2][4];
                    const uint32_t at = tile<GC * 2>(16 * ib + (lane & 7) + ((lane >> 4) << 3), 2 * wr + ((lane >> 3) & 1));
#pragma unroll
                    for (int i = 0; i < TE; ++i) {
                        ldsm4t(a[i], base + L::kN + i * L::MB + at);
                        ldsm4t(d[i], base + L::kO + i * L::MB + at);
                    }
#pragma unroll
                    for (int i = 0; i < TI; ++i)
#pragma unroll
                        for (int m = 0; m < CT / 2; ++m) ldsm4t(b[i][m], addr_bt<NB>(keys + L::kQ + i * L::KB, 16 * ib, c0 / 8 + 2 * m));
                    mma_terms<TE, TI, CT>(K_, a, b, top);
#pragma unroll
                    for (int i = 0; i < TI; ++i)
#pragma unroll
                        for (int m = 0; m < CT / 2; ++m) ldsm4t(b[i][m], addr_bt<NB>(keys + L::kK + i * L::KB, 16 * ib, c0 / 8 + 2 * m));
                    mma_terms<TE, TI, CT>(K_, d, b, top);
                }
            }
            if constexpr (F32) {
                add_to(DQ, tQ);
                add_to(DK, tK);
            }
            if (warp == scalar_warp) {                // dbeta and dg: two tokens per lane, sums in a fixed order
                float db[2], dG[2], bt[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = 2 * lane + e;
                    const float t = (sc->tail[0][i] + sc->tail[1][i]) + (sc->tail[2][i] + sc->tail[3][i]);
                    const float c = (sc->col[0][i] + sc->col[1][i]) + (sc->col[2][i] + sc->col[3][i]);
                    db[e] = t + sc->diag[i] + c;
                    dG[e] = ((sc->row[0][i] + sc->row[1][i]) + (sc->row[2][i] + sc->row[3][i])) - sc->beta[i] * c;
                    bt[e] = sc->beta[i] * t;
                }
                float x = lane < GT / 32 ? sc->ss[lane] : 0.f;
#pragma unroll
                for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                // from a token on: what depends on G_i there; before it: what reaches the chunk's end from there
                float later = dG[0] + dG[1], before = bt[0] + bt[1];
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float z = __shfl_down_sync(0xffffffffu, later, o), w = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane + o < 32) later += z;
                    if (lane >= o) before += w;
                }
                float up = __shfl_up_sync(0xffffffffu, before, 1), down = __shfl_down_sync(0xffffffffu, later, 1);
                if (lane == 0) up = 0.f;
                if (lane == 31) down = 0.f;
                const float last = sc->whole * x;
                // where nothing is left of the state before a token, the sums cancel but for their roundings (a NaN stays one)
                const float dg[2] = {(((dG[0] + dG[1]) + down) + (up + last)) * sc->open[2 * lane],
                                     ((dG[1] + down) + ((up + bt[0]) + last)) * sc->open[2 * lane + 1]};
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (2 * lane + e < n) {
                        const long long at = (t0 + 2 * lane + e) * p.H + h;
                        if constexpr (F32) {
                            static_cast<float *>(p.dg)[at] = dg[e];
                            static_cast<float *>(p.dbeta)[at] = db[e];
                        } else {
                            static_cast<__nv_bfloat16 *>(p.dg)[at] = __float2bfloat16(dg[e]);
                            static_cast<__nv_bfloat16 *>(p.dbeta)[at] = __float2bfloat16(db[e]);
                        }
                    }
            }
            if constexpr (L::AHEAD) base = both - base;
        }
        // back through the lengths, and out
        if (p.qk_norm) {
            float dq[2] = {}, dk[2] = {};
#pragma unroll
            for (int t = 0; t < CT / 2; ++t) {
                float2 qv[2][2], kv[2][2];
                pairs_at<NB, TI>(qv, keys + L::kQ, L::KB, 16 * wr, c0 / 16 + t);
                pairs_at<NB, TI>(kv, keys + L::kK, L::KB, 16 * wr, c0 / 16 + t);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        dq[e] += fmaf(qv[u][e].x, DQ[2 * t + u][2 * e], qv[u][e].y * DQ[2 * t + u][2 * e + 1]);
                        dk[e] += fmaf(kv[u][e].x, DK[2 * t + u][2 * e], kv[u][e].y * DK[2 * t + u][2 * e + 1]);
                    }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = quad_sum(dq[e]), y = quad_sum(dk[e]);
                if (tc == 0) {
                    sc->dq[wc][16 * wr + gr + 8 * e] = x;
                    sc->dk[wc][16 * wr + gr + 8 * e] = y;
                }
            }
            __syncthreads();
            float fq[2], fk[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 16 * wr + gr + 8 * e;
                const float rq = sc->sq[i] / p.scale, rk = sc->rk[i];
                fq[e] = rq * rq * ((sc->dq[0][i] + sc->dq[1][i]) + (sc->dq[2][i] + sc->dq[3][i]));
                fk[e] = rk * rk * ((sc->dk[0][i] + sc->dk[1][i]) + (sc->dk[2][i] + sc->dk[3][i]));
            }
#pragma unroll
            for (int t = 0; t < CT / 2; ++t) {
                float2 qv[2][2], kv[2][2];
                pairs_at<NB, TI>(qv, keys + L::kQ, L::KB, 16 * wr, c0 / 16 + t);
                pairs_at<NB, TI>(kv, keys + L::kK, L::KB, 16 * wr, c0 / 16 + t);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int m = 2 * t + u;
                        DQ[m][2 * e] = fmaf(-fq[e], qv[u][e].x, DQ[m][2 * e]);
                        DQ[m][2 * e + 1] = fmaf(-fq[e], qv[u][e].y, DQ[m][2 * e + 1]);
                        DK[m][2 * e] = fmaf(-fk[e], kv[u][e].x, DK[m][2 * e]);
                        DK[m][2 * e + 1] = fmaf(-fk[e], kv[u][e].y, DK[m][2 * e + 1]);
                    }
            }
        }
#pragma unroll
        for (int m = 0; m < CT; ++m)
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const int i = 16 * wr + gr + 4 * e;
                if (i >= n) continue;
                const long long at = ((t0 + i) * p.Hk + cur->hk) * NN + c0 + 8 * m + 2 * tc;
                if constexpr (SPLIT) {
                    float *to = p.keep_parts + cur->part * 2 * p.parts_step + at;
                    *reinterpret_cast<float2 *>(to) = make_float2(DQ[m][e], DQ[m][e + 1]);
                    *reinterpret_cast<float2 *>(to + p.parts_step) = make_float2(DK[m][e], DK[m][e + 1]);
                } else if constexpr (F32) {
                    *reinterpret_cast<float2 *>(static_cast<float *>(p.dq) + at) = make_float2(DQ[m][e], DQ[m][e + 1]);
                    *reinterpret_cast<float2 *>(static_cast<float *>(p.dk) + at) = make_float2(DK[m][e], DK[m][e + 1]);
                } else {
                    *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.dq) + at) = pack(DQ[m][e], DQ[m][e + 1]);
                    *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.dk) + at) = pack(DK[m][e], DK[m][e + 1]);
                }
            }
        if constexpr (!L::AHEAD) return;
        cur = cur == &sc->chunk[0] ? &sc->chunk[1] : &sc->chunk[0];
        if (cur->n == 0) return;
        keys = both - keys;
    }
}

// The sum of the parts of dq and dk, in order.
template <int NN, bool F32>
__global__ void __launch_bounds__(256) delta_grad_sum_kernel(const DeltaArgs p, unsigned tasks, int parts) {
    unsigned task = blockIdx.x;
    const GradChunk c = grad_chunk(p, task, tasks, 1);
    for (int i = threadIdx.x; i < c.n * (NN / 2); i += 256) {
        const int which = i / (c.n * (NN / 4)), j = i % (c.n * (NN / 4));
        const long long at = ((c.t0 + j / (NN / 4)) * p.Hk + c.hk) * NN + 4 * (j % (NN / 4));
        const float *from = p.keep_parts + which * p.parts_step + at;
        float4 x = *reinterpret_cast<const float4 *>(from);
        for (int k = 1; k < parts; ++k) {
            const float4 y = *reinterpret_cast<const float4 *>(from + k * 2 * p.parts_step);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        void *to = which ? p.dk : p.dq;
        if constexpr (F32) *reinterpret_cast<float4 *>(static_cast<float *>(to) + at) = x;
        else *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(to) + at) = make_uint2(pack(x.x, x.y), pack(x.z, x.w));
    }
}

}  // namespace

// ---- host side ---------------------------------------------------------------------------------------

cudaError_t allow_dynamic_smem(const void *kernel, int bytes);

namespace {

// Into how many parts the value heads of a key head go: one, in the same accumulators, where the chunks and key heads fill
// the SMs; else as many as do. One sequence of 173 tokens with 36 heads on 4 key heads (fp32, N = 128)
// takes 188 us for the whole backward so and 573 in one part; 14 sequences of 3 tokens, 27 heads on one: 159 and 544.
int parts_of(long long slots, int H, int Hk) {
    const long long whole = slots * Hk;
    return whole >= 148 ? 1 : int(std::max(1ll, std::min<long long>(H / Hk, 148 / whole)));
}

template <int NN, int RW, bool F32, int GROUPS>
cudaError_t launch_t(const DeltaArgs &p, long long slots) {
    constexpr int fwd_bytes = Layout<NN, RW, F32, true, GROUPS>::total, rev_bytes = RevLayout<NN, RW, F32, GROUPS>::total;
    constexpr int sweep_bytes = fwd_bytes > rev_bytes ? fwd_bytes : rev_bytes;
    using G = GradLayout<NN, F32>;
    const void *sweeps = reinterpret_cast<const void *>(delta_sweeps_kernel<NN, RW, F32, GROUPS>);
    cudaError_t e = allow_dynamic_smem(sweeps, sweep_bytes);
    if (e != cudaSuccess) return e;
    // Together where that fills SMs that one sweep leaves idle (and at N = 128, where a CTA has an SM to itself:
    // 541 us against 584 for seven packed sequences of 8 heads); in turn otherwise, since blocks of the two kinds
    // on one SM crowd each other's instructions out (96 heads of N = 64: 320 us against 267).
    const unsigned blocks = unsigned(p.B) * p.H * (NN / (16 * RW));
    const bool both = NN == 128 || blocks <= 74;
    for (int which = both ? 2 : 1; which >= (both ? 2 : 0); --which) {
        delta_sweeps_kernel<NN, RW, F32, GROUPS><<<both ? 2 * blocks : blocks, RW * 32 + GROUPS * kGroup, sweep_bytes, p.stream>>>(p, which);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const int parts = parts_of(slots, p.H, p.Hk);
    const long long whole = slots * p.Hk, tasks = whole * parts;
    const auto grad = parts > 1 ? delta_grad_kernel<NN, F32, true> : delta_grad_kernel<NN, F32, false>;
    e = allow_dynamic_smem(reinterpret_cast<const void *>(grad), G::total);
    if (e != cudaSuccess) return e;
    grad<<<unsigned(G::AHEAD ? std::min(tasks, 148ll) : tasks), GT, G::total, p.stream>>>(p, unsigned(tasks), parts);
    e = cudaGetLastError();
    if (e != cudaSuccess || parts == 1) return e;
    delta_grad_sum_kernel<NN, F32><<<unsigned(whole), 256, 0, p.stream>>>(p, unsigned(whole), parts);
    return cudaGetLastError();
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Per row E (bf16: in two terms) and the second term of dv, per chunk of 64 S and dS (bf16: in two terms); dq and dk of
// each part in fp32 where there are several.
size_t delta_backward_workspace(size_t rows, int B, int H, int Hk, int N, wkv7_dtype dt) {
    const size_t row = rows * H * N, state = (rows / 64 + B) * H * N * N;
    const int parts = parts_of((long long)(rows / 64 + B), H, Hk);
    const size_t summed = parts > 1 ? size_t(parts) * 2 * rows * Hk * N * 4 : 0;
    return summed + (dt == WKV7_BF16 ? 3 * up(row * 2) + 4 * up(state * 2) : up(row * 4) + 2 * up(state * 4));
}

cudaError_t launch_delta_backward(const DeltaArgs &p0) {
    DeltaArgs p = p0;
    const size_t rows = p.cu ? size_t(p.T) : size_t(p.B) * p.T, el = p.dt == WKV7_BF16 ? 2 : 4;
    const size_t row = up(rows * p.H * p.N * el), slots = rows / 64 + p.B, state = up(slots * p.H * p.N * p.N * el);
    char *ws = static_cast<char *>(p.keep_E);
    p.keep_lo = (long long)(row / el);
    p.keep_dlo = ws + 2 * row;
    ws += p.dt == WKV7_BF16 ? 3 * row : row;
    p.keep_S = ws;
    p.keep_dS = ws + (p.dt == WKV7_BF16 ? 2 : 1) * state;
    p.keep_second = (long long)(state / el);
    p.keep_parts = reinterpret_cast<float *>(ws + (p.dt == WKV7_BF16 ? 4 : 2) * state);
    p.parts_step = (long long)rows * p.Hk * p.N;
    p.group = p.H / p.Hk;
    if (p.dt == WKV7_F32) return p.N == 64 ? launch_t<64, 4, true, 2>(p, slots) : launch_t<128, 4, true, 2>(p, slots);
    if (p.N == 128) return launch_t<128, 4, false, 2>(p, slots);
    return (long long)p.B * p.H <= 37 ? launch_t<64, 2, false, 3>(p, slots) : launch_t<64, 4, false, 2>(p, slots);     // as forward, twice the blocks
}

}  // namespace wkv7
