// gated_delta_pack_bwd: gradients of gated_delta_pack_fwd, chunk by chunk
// backwards. With dO' = scale dOut, dS' the gradient of the state that leaves
// the chunk, and the forward's L, P, G, U = diag(beta) E and entering state S,
//   Y = P^T dO' + diag(e^{G_last - G}) K dS',  dU = (I + diag(beta) L)^-T Y,  dE = diag(beta) dU,
//   dS = e^{G_last} dS' + (diag(e^G) Q)^T dO' - (diag(e^G) K)^T dE,
//   dv = dE,  dbeta = rows of dU . E.
// A token reads the state twice, as q (gradient dO') and as k (gradient -dE),
// and writes it once, as k. With a = D . dO' U^T and b = D . dE U^T (below the
// diagonal for b),
//   dq       =  diag(e^G) dO' S^T + a K
//   dk read  = -diag(e^G) dE S^T - b K
//   dk write =  diag(e^{G_last - G}) U dS'^T + a^T Q - b^T K
// and, since e^{G_i} scales what token i reads and e^{-G_i} what it writes,
//   dG_i = q_i.dq_i + k_i.dkread_i - k_i.dkwrite_i,  the last token's also + <dS', S'>,
//   <dS', S'> = e^{G_last} <dS', S> + sum_j e^{G_last - G_j} k_j.(dS' U_j),
//   dg_t = sum of dG_i, i >= t in the chunk.
// k_delta_prepare makes what no gradient enters, k_delta_chain_bwd walks each
// sequence's chunks back with dS in registers, and k_delta_grads forms the
// chunks' gradients, all at once, from S, E, dS' and dU.
#include "delta_prepare.h"

namespace ssmp {

// As k_delta_chain, from the last chunk to the first.
template <typename T, int DKP, int NW>
__global__ __launch_bounds__(NW * 64) void k_delta_chain_bwd(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    constexpr int MT = DKP / 16;
    using Loads = ChainLoads<T, DKP, 3, NW * 64>;
    __shared__ alignas(16) typename Loads::Tiles lds;
    constexpr int kCols = NW * kWaveCols;
    const int ncb = (a.Dv + kCols - 1) / kCols, group = a.Hv / a.Hk;
    const Spread sp = spread(blockIdx.x, ncb * group);
    if (sp.group >= (int64_t)a.nseq * a.Hk) return;
    const int seq = (int)(sp.group / a.Hk), hk = (int)(sp.group % a.Hk);
    const int hv = hk * group + sp.member / ncb, cb = sp.member % ncb;
    const int wave = wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    const int col = cb * kCols + wave * 16 + l16;
    const bool busy = cb * kCols + wave * 16 < a.Dv;
    const Seq q = seq_at(a.cu, seq, a.T);
    const int chunks = (q.len + kC - 1) / kC;
    const Column cs = column_of<float>(1, a.Dv, col), cv = column_of<T>(a.Hv, a.Dv, col);
    const size_t state = ((size_t)seq * a.Hv + hv) * a.Dk * a.Dv;
    f32x4 S[MT];
    load_matrix(a.dhT ? a.dhT + state : nullptr, a.Dk, a.Dv, cs, S);
    Loads next;
    uint32_t onext[16];
    if (chunks > 0) {
        const int64_t start = q.start + (int64_t)(chunks - 1) * kC;
        const int n = q.len - (chunks - 1) * kC;
        next.load(a, q.slot0 + chunks - 1, start, n, hk, hv);
        load_column<T>(a.dout, start, n, a.Hv, hv, a.Dv, cv, onext);
    }
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const int64_t slot = q.slot0 + ch, start = q.start + (int64_t)ch * kC;
        const size_t sh = (size_t)slot * a.Hv + hv;
        __syncthreads();  // the last chunk's operands have been read
        next.put(lds);
        f32x4 o[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i >> 2][i & 3] = Elt<T>::cvt(onext[i]);
        __syncthreads();
        if (ch > 0) {
            next.load(a, slot - 1, start - kC, kC, hk, hv);
            load_column<T>(a.dout, start - kC, kC, a.Hv, hv, a.Dv, cv, onext);
        }
        if (!busy) continue;
        store_matrix(a.dS1 + sh * a.Dk * a.Dv, a.Dk, a.Dv, cs, S);
        f32x4 x[4] = {}, y[4] = {};  // K dS', scale P^T dOut
#pragma unroll
        for (int s = 0; s < DKP / 32; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            const auto sb = split_tiles<3>(S[2 * s], S[2 * s + 1]);
#pragma unroll
            for (int m = 0; m < 4; ++m) mma<3>(x[m], lds.k.frag(m * 16 + l16, s * 4 + l4), sb);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            const auto ob = split_tiles<NX>(o[2 * s], o[2 * s + 1]);
#pragma unroll
            for (int m = 0; m < 2 + 2 * s; ++m)
                mma<3>(y[m], tri_frag<3>(lds.att, (s ? 0 : 64) + m * 16 + l16, l4), ob);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 el = *reinterpret_cast<const f32x4*>(lds.el + m * 16 + l4 * 4);
            y[m] += el * x[m];
        }
        f32x4 u[4] = {};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            const auto yb = split_tiles<3>(y[2 * s], y[2 * s + 1]);
#pragma unroll
            for (int m = 0; m < 2 + 2 * s; ++m)
                mma<3>(u[m], tri_frag<3>(lds.inv, (s ? 0 : 64) + m * 16 + l16, l4), yb);
        }
        store_matrix(a.dU + sh * kC * a.Dv, kC, a.Dv, cs, u);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 be = *reinterpret_cast<const f32x4*>(lds.beta + m * 16 + l4 * 4);
            const f32x4 eg = *reinterpret_cast<const f32x4*>(lds.eg + m * 16 + l4 * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                u[m][r] *= -eg[r] * be[r];         // -e^G dE
                o[m][r] *= eg[r] * a.scale;        // e^G scale dOut
            }
        }
        const float ec = lds.eg[kC - 1];
#pragma unroll
        for (int m = 0; m < MT; ++m) S[m] *= ec;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            const auto ob = split_tiles<3>(o[2 * s], o[2 * s + 1]);
            const auto ub = split_tiles<3>(u[2 * s], u[2 * s + 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                mma<3>(S[m], lds.q.token_frag(s, m), ob);
                mma<3>(S[m], lds.k.token_frag(s, m), ub);
            }
        }
    }
    if (a.dh0 && busy) store_matrix(a.dh0 + state, a.Dk, a.Dv, cs, S);
}

// One workgroup per (slot, key head), over the value heads of its group, whose
// dq and dk it adds in registers (GROUP; a head that has its keys to itself
// needs no second set). Wave w of DKP / 16 holds columns 16 w .. of dq and dk
// for all 64 tokens, so its rows of S and dS' come straight from memory, and
// some of the tiles of a^T and b^T. The next 64 columns of dOut, E and dU are
// under way in registers while the present ones are multiplied.
template <typename T, int DKP, bool GROUP>
__global__ __launch_bounds__(DKP * 4) void k_delta_grads(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    constexpr int kThreads = DKP * 4, kWaves = DKP / 16;
    constexpr int SG = 512 / kThreads;    // 8-column units a thread stages
    constexpr int TT = 16 / kWaves;       // tiles of a^T a wave holds: row tile w / (4 / TT)
    constexpr int LT = kC + 8, PT = kC * LT;
    // planes of dOut, dE and U (64 columns at a time, [token][column]), then of
    // a or -b and its transpose
    __shared__ alignas(16) __bf16 lds[(NX + 6) * PT];
    __shared__ alignas(16) RowTile<T, DKP> kt, qt;
    __shared__ double G[kC];
    __shared__ alignas(16) float decay[2][kC];
    __shared__ float red[kWaves][kC], ends[kWaves];
    const int64_t slot = blockIdx.x;
    const int hk = blockIdx.y, group = a.Hv / a.Hk;
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, slot, c)) return;
    const int tid = threadIdx.x, wave = wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    __bf16* const Op = lds;
    __bf16* const Ep = lds + NX * PT;
    __bf16* const Up = Ep + 3 * PT;
    __bf16* const M = lds;
    __bf16* const Mt = lds + 3 * PT;
    for (int u = tid; u < kC * DKP / 8; u += kThreads) {
        const int i = u / (DKP / 8), k8 = u % (DKP / 8);
        const size_t first = ((size_t)c.start * a.Hk + hk) * a.Dk;
        const uint32_t o = k8 * 8 < a.Dk ? (uint32_t)(i * a.Hk * a.Dk + k8 * 8) * (uint32_t)sizeof(T) : kNowhere;
        Unit<T> x, y;
        x.load(rows_rsrc(static_cast<const T*>(a.k) + first, c.n, a.Hk * a.Dk, a.Dk), o);
        y.load(rows_rsrc(static_cast<const T*>(a.q) + first, c.n, a.Hk * a.Dk, a.Dk), o);
        kt.put(i, k8, x);
        qt.put(i, k8, y);
    }
    const int d = wave * 16 + l16;                       // this lane's column of dq and dk
    const int tj = wave / (4 / TT), ti0 = (wave % (4 / TT)) * TT;  // tiles (tj, ti0 + x) of a^T: rows j, columns i
    f32x4 tq[4] = {}, tk[4] = {};
    for (int hv = hk * group; hv < (hk + 1) * group; ++hv) {
        const size_t sh = (size_t)slot * a.Hv + hv;
        Unit<T> fo[SG];
        Unit<float> fE[SG], fU[SG];
        float beta[SG], db[SG];
        const auto stage_load = [&](int v0) {
#pragma unroll
            for (int x = 0; x < SG; ++x) {
                const int u = tid + x * kThreads, t = u >> 3, e = (u & 7) * 8;
                const bool on = v0 + e < a.Dv;
                const size_t ws = (sh * kC + t) * a.Dv + v0 + e;
                fo[x].load(static_cast<const T*>(a.dout) + ((size_t)(c.start + t) * a.Hv + hv) * a.Dv + v0 + e,
                           on && t < c.n);
                fE[x].load(a.E + ws, on);
                fU[x].load(a.dU + ws, on);
            }
        };
        stage_load(0);
#pragma unroll
        for (int x = 0; x < SG; ++x) {
            const int t = (tid + x * kThreads) >> 3;
            beta[x] = t < c.n ? a.beta[(size_t)(c.start + t) * a.Hv + hv] : 0.0f;
            db[x] = 0.0f;
        }
        __syncthreads();  // the last head's sums have been read
        if (wave == 0) {
            G[l] = chunk_decay_sum(a.g, c.start, c.n, a.Hv, hv);
            decay[0][l] = a.dec[sh * 2 * kC + l];
            decay[1][l] = a.dec[sh * 2 * kC + kC + l];
        }
        f32x4 dq[4] = {}, dr[4] = {}, dw[4] = {};  // dq, dk read, dk write
        f32x4 at[TT] = {}, bt[TT] = {};
        float sd = 0.0f;                           // <dS', S>
        for (int v0 = 0; v0 < a.Dv; v0 += 64) {
            Unit<float> s0[2], s1[2];              // this lane's row of S and dS'
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k0 = s * 32 + l4 * 8;
                const bool on = d < a.Dk && v0 + k0 < a.Dv;
                const size_t o = (sh * a.Dk + d) * a.Dv + v0 + k0;
                s0[s].load(a.S0 + o, on);
                s1[s].load(a.dS1 + o, on);
            }
#pragma unroll
            for (int x = 0; x < SG; ++x) {
                const int u = tid + x * kThreads, t = u >> 3, e = (u & 7) * 8;
                float E[8], dU[8];
                T dv[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    E[p] = fE[x].w[p >> 2][p & 3];
                    dU[p] = fU[x].w[p >> 2][p & 3];
                    db[x] = fmaf(dU[p], E[p], db[x]);
                    E[p] *= beta[x];
                    dU[p] *= beta[x];
                    Elt<T>::st(dv, p, dU[p]);
                }
                if (v0 + e < a.Dv && t < c.n)
                    put8(static_cast<T*>(a.dv) + ((size_t)(c.start + t) * a.Hv + hv) * a.Dv + v0 + e, dv);
                const auto po = unit_planes(fo[x]);
                const auto pe = split8<3>(dU), pu = split8<3>(E);
                const int o = t * LT + e;
#pragma unroll
                for (int p = 0; p < NX; ++p) *reinterpret_cast<bf16x8*>(Op + p * PT + o) = po.p[p];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    *reinterpret_cast<bf16x8*>(Ep + p * PT + o) = pe.p[p];
                    *reinterpret_cast<bf16x8*>(Up + p * PT + o) = pu.p[p];
                }
            }
            __syncthreads();
            if (v0 + 64 < a.Dv) stage_load(v0 + 64);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k0 = s * 32 + l4 * 8;
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int e = 0; e < 8; ++e) sd = fmaf(s0[s].w[e >> 2][e & 3], s1[s].w[e >> 2][e & 3], sd);
                const auto sb = unit_planes(s0[s]), db1 = unit_planes(s1[s]);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    __builtin_amdgcn_sched_barrier(0);
                    mma<3>(dq[m], plane_frag<NX>(Op, PT, LT, m * 16 + l16, k0), sb);
                    mma<3>(dr[m], plane_frag<3>(Ep, PT, LT, m * 16 + l16, k0), sb);
                    mma<3>(dw[m], plane_frag<3>(Up, PT, LT, m * 16 + l16, k0), db1);
                }
                __builtin_amdgcn_sched_barrier(0);
                const auto uw = plane_frag<3>(Up, PT, LT, tj * 16 + l16, k0);
#pragma unroll
                for (int x = 0; x < TT; ++x) {
                    const int i = ti0 + x;
                    if (i >= tj) {  // below the diagonal of a and b
                        mma<3>(at[x], uw, plane_frag<NX>(Op, PT, LT, i * 16 + l16, k0));
                        mma<3>(bt[x], uw, plane_frag<3>(Ep, PT, LT, i * 16 + l16, k0));
                    }
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int x = 0; x < SG; ++x) {
            const int u = tid + x * kThreads, t = u >> 3;
            float s = db[x];
            s += __shfl_xor(s, 1);
            s += __shfl_xor(s, 2);
            s += __shfl_xor(s, 4);
            if ((u & 7) == 0 && t < c.n) a.dbeta[(size_t)(c.start + t) * a.Hv + hv] = s;
        }
        __builtin_amdgcn_sched_barrier(0);
        float end = decay[0][kC - 1] * sd;
        float kv[4][4], qv[4][4];  // this lane's column of K and Q: tokens 16 m + 4 l4 + r
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = m * 16 + l4 * 4;
            kt.values4(m, wave, kv[m]);
            qt.values4(m, wave, qv[m]);
            const f32x4 eg = *reinterpret_cast<const f32x4*>(&decay[0][i]);
            const f32x4 el = *reinterpret_cast<const f32x4*>(&decay[1][i]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dq[m][r] *= eg[r] * a.scale;
                dr[m][r] *= -eg[r];
                dw[m][r] *= el[r];
                end = fmaf(kv[m][r], dw[m][r], end);
            }
        }
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {  // a, then -b
#pragma unroll
            for (int x = 0; x < TT; ++x) {
                const int i = (ti0 + x) * 16 + l16, j = tj * 16 + l4 * 4;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool on = pass ? i > j + r : i >= j + r;
                    const float w = on ? decay_of(G[i] - G[j + r]) : 0.0f;
                    v[r] = on ? (pass ? -w * bt[x][r] : w * a.scale * at[x][r]) : 0.0f;
                }
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    uint32_t p[3];
                    split2<3>(v[r], v[r + 1], p);
#pragma unroll
                    for (int y = 0; y < 3; ++y) {
                        uint16_t* const to = reinterpret_cast<uint16_t*>(Mt) + y * PT + (j + r) * LT + kplace(i);
                        to[0] = (uint16_t)p[y];
                        to[LT] = (uint16_t)(p[y] >> 16);
                    }
                }
                lds_put4<3>(M, PT, LT, i, kplace(j), v);
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k0 = s * 32 + l4 * 8;
                __builtin_amdgcn_sched_barrier(0);
                const auto kb = kt.token_frag(s, wave), qb = qt.token_frag(s, wave);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if (m >= 2 * s) mma<3>(pass ? dr[m] : dq[m], plane_frag<3>(M, PT, LT, m * 16 + l16, k0), kb);
                    if (m < 2 + 2 * s) mma<3>(dw[m], plane_frag<3>(Mt, PT, LT, m * 16 + l16, k0), pass ? kb : qb);
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = m * 16 + l4 * 4;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float s = fmaf(qv[m][r], dq[m][r], kv[m][r] * (dr[m][r] - dw[m][r]));
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) s += __shfl_xor(s, x);
                if (l16 == 0) red[wave][i + r] = s;
            }
            if constexpr (GROUP) {
                tq[m] += dq[m];
                tk[m] += dr[m] + dw[m];
            }
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) end += __shfl_xor(end, x);
        if (l == 0) ends[wave] = end;
        __syncthreads();
        if (wave == 0) {
            double s = 0.0, e = 0.0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                s += (double)red[w][l];
                e += (double)ends[w];
            }
            if (l == kC - 1) s += e;
#pragma unroll
            for (int x = 1; x < kC; x <<= 1) {
                const double o = __shfl_down(s, x);
                if (l + x < kC) s += o;
            }
            if (l < c.n) a.dg[(size_t)(c.start + l) * a.Hv + hv] = (float)s;
        }
        if constexpr (!GROUP) {
#pragma unroll
            for (int m = 0; m < 4; ++m) dr[m] += dw[m];
            store_column<T>(a.dq, c.start, c.n, a.Hk, hk, a.Dk, column_of<T>(a.Hk, a.Dk, d), dq, 1.0f);
            store_column<T>(a.dk, c.start, c.n, a.Hk, hk, a.Dk, column_of<T>(a.Hk, a.Dk, d), dr, 1.0f);
        }
    }
    if constexpr (GROUP) {
        store_column<T>(a.dq, c.start, c.n, a.Hk, hk, a.Dk, column_of<T>(a.Hk, a.Dk, d), tq, 1.0f);
        store_column<T>(a.dk, c.start, c.n, a.Hk, hk, a.Dk, column_of<T>(a.Hk, a.Dk, d), tk, 1.0f);
    }
}

template <typename T, int DKP>
int launch_delta_bwd(const DeltaArgs& a, hipStream_t s) {
    if (a.T > 0)
        if (const int st = launch_delta_prepare<T, DKP, true>(a, s)) return st;
    if (a.T > 0 || a.dh0) {
        if (const int nw = chain_waves(a); nw == 8)
            k_delta_chain_bwd<T, DKP, 8><<<chain_blocks(a, nw), nw * 64, 0, s>>>(a);
        else
            k_delta_chain_bwd<T, DKP, 4><<<chain_blocks(a, nw), nw * 64, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    if (a.T > 0) {
        const dim3 grid((unsigned)delta_slots(a.T, a.nseq), a.Hk);
        if (a.Hv > a.Hk) k_delta_grads<T, DKP, true><<<grid, DKP * 4, 0, s>>>(a);
        else k_delta_grads<T, DKP, false><<<grid, DKP * 4, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}

struct DeltaBwdLayout {
    size_t dec, inv, att, dS1, dU, total;
};
inline DeltaBwdLayout delta_bwd_layout(int64_t T, int32_t nseq, int32_t Hv, int32_t Dk, int32_t Dv) {
    const size_t n = (size_t)delta_slots(T, nseq);
    DeltaBwdLayout L;
    L.dec = 0;
    L.inv = L.dec + round256(n * Hv * 2 * kC * 4);
    L.att = L.inv + round256(n * Hv * kTri * 4);
    L.dS1 = L.att + round256(n * Hv * kTri * 4);
    L.dU = L.dS1 + round256(n * Hv * Dk * Dv * 4);
    L.total = L.dU + round256(n * Hv * kC * Dv * 4);
    return L;
}

}  // namespace ssmp

extern "C" size_t gated_delta_pack_bwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                     int32_t Dv, int32_t dtype) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype) || T == 0) return 0;
    return delta_bwd_layout(T, nseq, Hv, Dk, Dv).total;
}

extern "C" int gated_delta_pack_bwd(const void* q, const void* k, const float* g, const float* beta,
                                    const int32_t* cu_seqlens, int32_t nseq, const void* dout, int64_t T, int32_t Hk,
                                    int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, float scale,
                                    const float* dfinal_state, float* dinitial_state, void* dq, void* dk, void* dv,
                                    float* dg, float* dbeta, const void* saved, size_t saved_bytes, void* scratch,
                                    size_t scratch_bytes, void* stream) {
    using namespace ssmp;
    if (const int st = delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    if (!cu_seqlens) return SSMP_ERR_NULL;
    if (T > 0 && (!q || !k || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta)) return SSMP_ERR_NULL;
    if (!aligned16(q, k, dout, dq, dk, dv, dfinal_state, dinitial_state, saved, scratch)) return SSMP_ERR_ALIGN;
    if (T > 0 && (!saved || saved_bytes < gated_delta_pack_saved_bytes(T, nseq, Hk, Hv, Dk, Dv)))
        return SSMP_ERR_WORKSPACE;
    if (T > 0 && (!scratch || scratch_bytes < gated_delta_pack_bwd_scratch_bytes(T, nseq, Hk, Hv, Dk, Dv, dtype)))
        return SSMP_ERR_WORKSPACE;
    if (T == 0 && !dinitial_state) return SSMP_OK;
    const DeltaBwdLayout L = delta_bwd_layout(T, nseq, Hv, Dk, Dv);
    char* const ws = static_cast<char*>(scratch);
    DeltaArgs a = {};
    a.q = q;
    a.k = k;
    a.dout = dout;
    a.g = g;
    a.beta = beta;
    a.cu = cu_seqlens;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    a.dhT = dfinal_state;
    a.dh0 = dinitial_state;
    a.T = T;
    a.nseq = nseq;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dk = Dk;
    a.Dv = Dv;
    a.scale = scale;
    if (T > 0) {
        char* const kept = static_cast<char*>(const_cast<void*>(saved));
        a.S0 = reinterpret_cast<float*>(kept);
        a.E = reinterpret_cast<float*>(kept + round256((size_t)delta_slots(T, nseq) * Hv * Dk * Dv * 4));
        a.dec = reinterpret_cast<float*>(ws + L.dec);
        a.inv = reinterpret_cast<float*>(ws + L.inv);
        a.att = reinterpret_cast<float*>(ws + L.att);
        a.dS1 = reinterpret_cast<float*>(ws + L.dS1);
        a.dU = reinterpret_cast<float*>(ws + L.dU);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wide = Dk > 64;
    if (dtype == SSMP_F32) return wide ? launch_delta_bwd<float, 128>(a, s) : launch_delta_bwd<float, 64>(a, s);
    return wide ? launch_delta_bwd<uint16_t, 128>(a, s) : launch_delta_bwd<uint16_t, 64>(a, s);
}
