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
template <typename T, int DKP>
__global__ __launch_bounds__(256) void k_delta_chain_bwd(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    constexpr int MT = DKP / 64;
    constexpr int LS = DKP + 8, LT = kC + 8;
    constexpr int PS = kCols * LS, PT = kCols * LT;
    __shared__ alignas(16) __bf16 St[3 * PS];   // dS', [column][row]
    __shared__ alignas(16) __bf16 Ot[NX * PT];  // dOut, [column][token]
    __shared__ alignas(16) __bf16 Gt[3 * PT];   // e^G scale dOut
    __shared__ alignas(16) __bf16 Yt[3 * PT];   // Y
    __shared__ alignas(16) __bf16 Wt[3 * PT];   // -e^G dE
    const int ncb = (a.Dv + kCols - 1) / kCols;
    const int cb = blockIdx.x % ncb, hv = (blockIdx.x / ncb) % a.Hv, seq = blockIdx.x / (ncb * a.Hv);
    const int hk = hv / (a.Hv / a.Hk);
    const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, l16 = l & 15, l4 = l >> 4;
    const Seq q = seq_at(a.cu, seq, a.T);
    const int chunks = (q.len + kC - 1) / kC;
    f32x4 S[MT][2];
    const auto state_row = [&](int m, int r) { return wave * (DKP / 4) + m * 16 + l4 * 4 + r; };
    const auto state_col = [&](int n) { return cb * kCols + n * 16 + l16; };
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int d = state_row(m, r), e = state_col(n);
                S[m][n][r] = a.dhT && d < a.Dk && e < a.Dv
                                 ? a.dhT[(((size_t)seq * a.Hv + hv) * a.Dk + d) * a.Dv + e] : 0.0f;
            }
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const int64_t slot = q.slot0 + ch, start = q.start + (int64_t)ch * kC;
        const int cn = q.len - ch * kC < kC ? q.len - ch * kC : kC;
        const size_t sh = (size_t)slot * a.Hv + hv;
        const float* const dec = a.dec + sh * 2 * kC;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    v[r] = S[m][n][r];
                    const int d = state_row(m, r), e = state_col(n);
                    if (d < a.Dk && e < a.Dv) a.dS1[(sh * a.Dk + d) * a.Dv + e] = v[r];
                }
                lds_put4<3>(St, PS, LS, n * 16 + l16, state_row(m, 0), v);
            }
        {  // the chunk's dOut: token tid / 4, 8 columns
            const int i = tid >> 2, e = cb * kCols + (tid & 3) * 8;
            const bool on = i < cn && e < a.Dv;
            const auto f = load_frag(static_cast<const T*>(a.dout) + ((size_t)(start + i) * a.Hv + hv) * a.Dv + e, on);
            const float w = dec[i] * a.scale;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int at = ((tid & 3) * 8 + x) * LT + i;
                float v = 0.0f;
#pragma unroll
                for (int p = NX - 1; p >= 0; --p) v += (float)f.p[p][x];
                __bf16 g[3];
                split<3>(v * w, g);
#pragma unroll
                for (int p = 0; p < NX; ++p) Ot[p * PT + at] = f.p[p][x];
#pragma unroll
                for (int p = 0; p < 3; ++p) Gt[p * PT + at] = g[p];
            }
        }
        __syncthreads();
        f32x4 y[2] = {}, x[2] = {};
        const int i0 = wave * 16 + l16;
        const size_t row = ((size_t)(start + i0) * a.Hk + hk) * a.Dk;
#pragma unroll
        for (int s = 0; s < DKP / 32; ++s) {
            const int k0 = s * 32 + l4 * 8;
            const auto ka = load_frag(static_cast<const T*>(a.k) + row + k0, i0 < cn && k0 < a.Dk);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma<3>(x[n], ka, plane_frag<3>(St, PS, LS, n * 16 + l16, k0));
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k0 = s * 32 + l4 * 8;
            const auto pa = plane_frag<3>(a.att + sh * 3 * kC * kC, kC * kC, kC, i0, k0);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma<3>(y[n], pa, plane_frag<NX>(Ot, PT, LT, n * 16 + l16, k0));
        }
        float eg[4], el[4], bt[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = wave * 16 + l4 * 4 + r;
            eg[r] = dec[i];
            el[r] = dec[kC + i];
            bt[r] = i < cn ? a.beta[(size_t)(start + i) * a.Hv + hv] : 0.0f;
        }
        const float ec = dec[kC - 1];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float v[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = fmaf(el[r], x[n][r], y[n][r]);
            lds_put4<3>(Yt, PT, LT, n * 16 + l16, wave * 16 + l4 * 4, v);
        }
        __syncthreads();
        f32x4 u[2] = {};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k0 = s * 32 + l4 * 8;
            const auto ia = plane_frag<3>(a.inv + sh * 3 * kC * kC, kC * kC, kC, i0, k0);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma<3>(u[n], ia, plane_frag<3>(Yt, PT, LT, n * 16 + l16, k0));
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                w[r] = -eg[r] * (bt[r] * u[n][r]);
                const int i = wave * 16 + l4 * 4 + r, e = state_col(n);
                if (e < a.Dv) a.dU[(sh * kC + i) * a.Dv + e] = u[n][r];
            }
            lds_put4<3>(Wt, PT, LT, n * 16 + l16, wave * 16 + l4 * 4, w);
        }
        __syncthreads();
        const size_t tr = ((size_t)slot * a.Hk + hk) * DKP * kC;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n) S[m][n] *= ec;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k0 = s * 32 + l4 * 8;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const size_t at = tr + (wave * (DKP / 4) + m * 16 + l16) * kC + k0;
                const auto ka = load_frag(static_cast<const T*>(a.kt) + at, true);
                const auto qa = load_frag(static_cast<const T*>(a.qt) + at, true);
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    mma<3>(S[m][n], qa, plane_frag<3>(Gt, PT, LT, n * 16 + l16, k0));
                    mma<3>(S[m][n], ka, plane_frag<3>(Wt, PT, LT, n * 16 + l16, k0));
                }
            }
        }
        __syncthreads();  // Gt and Wt have been read
    }
    if (a.dh0) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int d = state_row(m, r), e = state_col(n);
                    if (d < a.Dk && e < a.Dv) a.dh0[(((size_t)seq * a.Hv + hv) * a.Dk + d) * a.Dv + e] = S[m][n][r];
                }
    }
}

// One workgroup per (slot, key head), over the value heads of its group, whose
// dq and dk it adds in registers. Wave w holds columns w DKP / 4 .. of dq and
// dk for all 64 tokens, so its rows of S and dS' come straight from memory,
// and rows 16 w .. of a^T and b^T.
template <typename T, int DKP>
__global__ __launch_bounds__(256, 1) void k_delta_grads(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    constexpr int NT = DKP / 64;  // 16-column tiles of dq and dk a wave holds
    constexpr int LT = kC + 8, PT = kC * LT;
    // planes of dOut, dE and U (64 columns at a time, [token][column]), then of
    // a or -b and its transpose
    __shared__ alignas(16) __bf16 lds[(NX + 6) * PT];
    __shared__ double G[kC];
    __shared__ float decay[2][kC], red[4][kC], ends[4];
    const int64_t slot = blockIdx.x;
    const int hk = blockIdx.y;
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, slot, c)) return;
    const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, l16 = l & 15, l4 = l >> 4;
    __bf16* const Op = lds;
    __bf16* const Ep = lds + NX * PT;
    __bf16* const Up = Ep + 3 * PT;
    __bf16* const M = lds;
    __bf16* const Mt = lds + 3 * PT;
    const size_t tr = ((size_t)slot * a.Hk + hk) * DKP * kC;
    f32x4 tq[4][NT] = {}, tk[4][NT] = {};
    for (int hv = hk * (a.Hv / a.Hk); hv < (hk + 1) * (a.Hv / a.Hk); ++hv) {
        const size_t sh = (size_t)slot * a.Hv + hv;
        __syncthreads();
        if (wave == 0) {
            G[l] = chunk_decay_sum(a.g, c.start, c.n, a.Hv, hv);
            decay[0][l] = a.dec[sh * 2 * kC + l];
            decay[1][l] = a.dec[sh * 2 * kC + kC + l];
        }
        f32x4 dq[4][NT] = {}, dr[4][NT] = {}, dw[4][NT] = {};  // dq, dk read, dk write
        f32x4 at[4] = {}, bt[4] = {};                          // rows j of tile `wave`, columns i of tile n
        float sd = 0.0f;                                       // <dS', S>
        const int ti = tid >> 2;
        const float beta = ti < c.n ? a.beta[(size_t)(c.start + ti) * a.Hv + hv] : 0.0f;
        float db = 0.0f;
        for (int v0 = 0; v0 < a.Dv; v0 += 64) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {  // token tid / 4, 16 columns
                const int e = (tid & 3) * 16 + x * 8;
                const bool on = v0 + e < a.Dv;
                const size_t io = ((size_t)(c.start + ti) * a.Hv + hv) * a.Dv + v0 + e;
                const size_t ws = (sh * kC + ti) * a.Dv + v0 + e;
                const auto fo = load_frag(static_cast<const T*>(a.dout) + io, on && ti < c.n);
                float E[8], dU[8];
                load8(a.E + ws, on, E);
                load8(a.dU + ws, on, dU);
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    db = fmaf(dU[p], E[p], db);
                    E[p] *= beta;
                    dU[p] *= beta;
                    if (on && ti < c.n) Elt<T>::st(static_cast<T*>(a.dv), io + p, dU[p]);
                }
                const auto fe = split8<3>(dU), fu = split8<3>(E);
                const int o = ti * LT + e;
#pragma unroll
                for (int p = 0; p < NX; ++p) *reinterpret_cast<bf16x8*>(Op + p * PT + o) = fo.p[p];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    *reinterpret_cast<bf16x8*>(Ep + p * PT + o) = fe.p[p];
                    *reinterpret_cast<bf16x8*>(Up + p * PT + o) = fu.p[p];
                }
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k0 = s * 32 + l4 * 8;
                Frag<3> sb[NT], db1[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int d = wave * (DKP / 4) + n * 16 + l16;
                    const bool on = d < a.Dk && v0 + k0 < a.Dv;
                    const size_t o = (sh * a.Dk + d) * a.Dv + v0 + k0;
                    float s0[8], s1[8];
                    load8(a.S0 + o, on, s0);
                    load8(a.dS1 + o, on, s1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) sd = fmaf(s0[e], s1[e], sd);
                    sb[n] = split8<3>(s0);
                    db1[n] = split8<3>(s1);
                }
                const auto uw = plane_frag<3>(Up, PT, LT, wave * 16 + l16, k0);
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const auto fo = plane_frag<NX>(Op, PT, LT, m * 16 + l16, k0);
                    const auto fe = plane_frag<3>(Ep, PT, LT, m * 16 + l16, k0);
                    const auto fu = plane_frag<3>(Up, PT, LT, m * 16 + l16, k0);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma<3>(dq[m][n], fo, sb[n]);
                        mma<3>(dr[m][n], fe, sb[n]);
                        mma<3>(dw[m][n], fu, db1[n]);
                    }
                    mma<3>(at[m], uw, fo);
                    mma<3>(bt[m], uw, fe);
                }
            }
            __syncthreads();
        }
        db += __shfl_xor(db, 1);
        db += __shfl_xor(db, 2);
        if ((tid & 3) == 0 && ti < c.n) a.dbeta[(size_t)(c.start + ti) * a.Hv + hv] = db;
        float end = decay[0][kC - 1] * sd;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int i = m * 16 + l4 * 4, d = wave * (DKP / 4) + n * 16 + l16;
                float kv[4];
                load4(static_cast<const T*>(a.kt) + tr + d * kC + i, kv);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    dq[m][n][r] *= decay[0][i + r] * a.scale;
                    dr[m][n][r] *= -decay[0][i + r];
                    dw[m][n][r] *= decay[1][i + r];
                    end = fmaf(kv[r], dw[m][n][r], end);
                }
            }
        for (int x = 0; x < 2; ++x) {  // a, then -b
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int i = n * 16 + l16, j = wave * 16 + l4 * 4;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const bool on = x ? i > j + r : i >= j + r;
                    const float w = on ? expf((float)(G[i] - G[j + r])) : 0.0f;
                    v[r] = on ? (x ? -w * bt[n][r] : w * a.scale * at[n][r]) : 0.0f;
                    __bf16 p[3];
                    split<3>(v[r], p);
#pragma unroll
                    for (int y = 0; y < 3; ++y) Mt[y * PT + (j + r) * LT + i] = p[y];
                }
                lds_put4<3>(M, PT, LT, i, j, v);
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k0 = s * 32 + l4 * 8;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const size_t o = tr + (wave * (DKP / 4) + n * 16 + l16) * kC + k0;
                    const auto kb = load_frag(static_cast<const T*>(a.kt) + o, true);
                    const auto qb = load_frag(static_cast<const T*>(a.qt) + o, true);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const auto fm = plane_frag<3>(M, PT, LT, m * 16 + l16, k0);
                        const auto ft = plane_frag<3>(Mt, PT, LT, m * 16 + l16, k0);
                        if (x == 0) {
                            mma<3>(dq[m][n], fm, kb);
                            mma<3>(dw[m][n], ft, qb);
                        } else {
                            mma<3>(dr[m][n], fm, kb);
                            mma<3>(dw[m][n], ft, kb);
                        }
                    }
                }
            }
            __syncthreads();
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float s[4] = {};
            const int i = m * 16 + l4 * 4;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int d = wave * (DKP / 4) + n * 16 + l16;
                float kv[4], qv[4];
                load4(static_cast<const T*>(a.kt) + tr + d * kC + i, kv);
                load4(static_cast<const T*>(a.qt) + tr + d * kC + i, qv);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    s[r] = fmaf(qv[r], dq[m][n][r], s[r]);
                    s[r] = fmaf(kv[r], dr[m][n][r] - dw[m][n][r], s[r]);
                }
                tq[m][n] += dq[m][n];
                tk[m][n] += dr[m][n] + dw[m][n];
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
#pragma unroll
                for (int x = 1; x < 16; x <<= 1) s[r] += __shfl_xor(s[r], x);
                if (l16 == 0) red[wave][i + r] = s[r];
            }
        }
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) end += __shfl_xor(end, x);
        if (l == 0) ends[wave] = end;
        __syncthreads();
        if (wave == 0) {
            double s = (double)red[0][l] + red[1][l] + red[2][l] + red[3][l];
            if (l == kC - 1) s += (double)ends[0] + ends[1] + ends[2] + ends[3];
#pragma unroll
            for (int x = 1; x < kC; x <<= 1) {
                const double o = __shfl_down(s, x);
                if (l + x < kC) s += o;
            }
            if (l < c.n) a.dg[(size_t)(c.start + l) * a.Hv + hv] = (float)s;
        }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = m * 16 + l4 * 4 + r, d = wave * (DKP / 4) + n * 16 + l16;
                if (i < c.n && d < a.Dk) {
                    const size_t o = ((size_t)(c.start + i) * a.Hk + hk) * a.Dk + d;
                    Elt<T>::st(static_cast<T*>(a.dq), o, tq[m][n][r]);
                    Elt<T>::st(static_cast<T*>(a.dk), o, tk[m][n][r]);
                }
            }
}

template <typename T, int DKP>
int launch_delta_bwd(const DeltaArgs& a, hipStream_t s) {
    const int64_t slots = delta_slots(a.T, a.nseq);
    if (a.T > 0) {
        k_delta_prepare<T, DKP, true><<<dim3((unsigned)slots, a.Hk), 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    if (a.T > 0 || a.dh0) {
        const unsigned blocks = (unsigned)((int64_t)a.nseq * a.Hv * ((a.Dv + kCols - 1) / kCols));
        k_delta_chain_bwd<T, DKP><<<blocks, 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    if (a.T > 0) {
        k_delta_grads<T, DKP><<<dim3((unsigned)slots, a.Hk), 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}

struct DeltaBwdLayout {
    size_t dec, inv, att, kt, qt, dS1, dU, total;
};
inline DeltaBwdLayout delta_bwd_layout(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv,
                                       int32_t dtype) {
    const size_t n = (size_t)delta_slots(T, nseq), elt = dtype == SSMP_F32 ? 4 : 2;
    DeltaBwdLayout L;
    L.dec = 0;
    L.inv = L.dec + round256(n * Hv * 2 * kC * 4);
    L.att = L.inv + round256(n * Hv * 3 * kC * kC * 2);
    L.kt = L.att + round256(n * Hv * 3 * kC * kC * 2);
    L.qt = L.kt + round256(n * Hk * delta_dkp(Dk) * kC * elt);
    L.dS1 = L.qt + round256(n * Hk * delta_dkp(Dk) * kC * elt);
    L.dU = L.dS1 + round256(n * Hv * Dk * Dv * 4);
    L.total = L.dU + round256(n * Hv * kC * Dv * 4);
    return L;
}

}  // namespace ssmp

extern "C" size_t gated_delta_pack_bwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                     int32_t Dv, int32_t dtype) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype) || T == 0) return 0;
    return delta_bwd_layout(T, nseq, Hk, Hv, Dk, Dv, dtype).total;
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
    const DeltaBwdLayout L = delta_bwd_layout(T, nseq, Hk, Hv, Dk, Dv, dtype);
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
        a.inv = reinterpret_cast<__bf16*>(ws + L.inv);
        a.att = reinterpret_cast<__bf16*>(ws + L.att);
        a.kt = ws + L.kt;
        a.qt = ws + L.qt;
        a.dS1 = reinterpret_cast<float*>(ws + L.dS1);
        a.dU = reinterpret_cast<float*>(ws + L.dU);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wide = Dk > 64;
    if (dtype == SSMP_F32) return wide ? launch_delta_bwd<float, 128>(a, s) : launch_delta_bwd<float, 64>(a, s);
    return wide ? launch_delta_bwd<uint16_t, 128>(a, s) : launch_delta_bwd<uint16_t, 64>(a, s);
}
