// gated_delta_pack_fwd: the gated delta rule over packed sequences. Per value
// head with its key head, and a_t = exp(g_t),
//   E_t = v_t - (a_t S_{t-1})^T k_t,  U_t = beta_t E_t,
//   S_t = a_t S_{t-1} + k_t U_t^T,    out_t = scale S_t^T q_t.
// In chunks of 64 tokens, with G the running sum of g in the chunk, S the
// state that enters it and D_ij = e^{G_i - G_j},
//   (I + L diag(beta)) E = X,  X = V - diag(e^G) K S,  L = D . K K^T below the diagonal,
//   out = scale (diag(e^G) Q S + P U),                 P = D . Q K^T on and below it,
//   S'  = e^{G_last} S + (diag(e^{G_last - G}) K)^T U.
// What does not depend on the state (the inverse, P, K^T, the decays) is made
// for all chunks at once by k_delta_prepare; k_delta_chain then goes along
// each sequence's chunks with the state in registers.
#include "delta_prepare.h"

namespace ssmp {

// One workgroup per (sequence, value head, 32 columns of the state). Wave w
// holds the state's rows w DKP / 4 .. and the chunk's tokens 16 w .. in its
// results; left operands come from global memory in operand order, each read
// by one wave alone, right operands pass through LDS as bf16 planes.
template <typename T, int DKP>
__global__ __launch_bounds__(256) void k_delta_chain(DeltaArgs a) {
    constexpr int NX = kExact<T>, NO = kOutP<T>;
    constexpr int MT = DKP / 64;  // 16-row tiles of the state a wave holds
    constexpr int LS = DKP + 8, LT = kC + 8;
    constexpr int PS = kCols * LS, PT = kCols * LT;
    __shared__ alignas(16) __bf16 St[3 * PS];   // the state, [column][row]
    __shared__ alignas(16) __bf16 Xt[3 * PT];   // X, [column][token]
    __shared__ alignas(16) __bf16 Ut[NO * PT];  // U
    __shared__ alignas(16) __bf16 Wt[3 * PT];   // e^{G_last - G} U
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
                S[m][n][r] = a.h0 && d < a.Dk && e < a.Dv
                                 ? a.h0[(((size_t)seq * a.Hv + hv) * a.Dk + d) * a.Dv + e] : 0.0f;
            }
    for (int ch = 0; ch < chunks; ++ch) {
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
                for (int r = 0; r < 4; ++r) v[r] = S[m][n][r];
                lds_put4<3>(St, PS, LS, n * 16 + l16, state_row(m, 0), v);
                if (a.S0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int d = state_row(m, r), e = state_col(n);
                        if (d < a.Dk && e < a.Dv) a.S0[(sh * a.Dk + d) * a.Dv + e] = v[r];
                    }
                }
            }
        __syncthreads();
        // K S and Q S for this wave's 16 tokens
        f32x4 x[2] = {}, o[2] = {};
        const int i0 = wave * 16 + l16;
        const size_t row = ((size_t)(start + i0) * a.Hk + hk) * a.Dk;
#pragma unroll
        for (int s = 0; s < DKP / 32; ++s) {
            const int k0 = s * 32 + l4 * 8;
            const bool on = i0 < cn && k0 < a.Dk;
            const auto ka = load_frag(static_cast<const T*>(a.k) + row + k0, on);
            const auto qa = load_frag(static_cast<const T*>(a.q) + row + k0, on);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const auto sb = plane_frag<3>(St, PS, LS, n * 16 + l16, k0);
                mma<3>(x[n], ka, sb);
                mma<NO>(o[n], qa, sb);
            }
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
            for (int r = 0; r < 4; ++r) {
                const int i = wave * 16 + l4 * 4 + r, e = state_col(n);
                const float vv = i < cn && e < a.Dv
                                     ? Elt<T>::ld(static_cast<const T*>(a.v), ((size_t)(start + i) * a.Hv + hv) * a.Dv + e)
                                     : 0.0f;
                v[r] = fmaf(-eg[r], x[n][r], vv);
                o[n][r] *= eg[r];
            }
            lds_put4<3>(Xt, PT, LT, n * 16 + l16, wave * 16 + l4 * 4, v);
        }
        __syncthreads();
        // E = inverse X
        f32x4 E[2] = {};
        const __bf16* const inv = a.inv + sh * 3 * kC * kC;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k0 = s * 32 + l4 * 8;
            const auto ia = plane_frag<3>(inv, kC * kC, kC, i0, k0);
#pragma unroll
            for (int n = 0; n < 2; ++n) mma<3>(E[n], ia, plane_frag<3>(Xt, PT, LT, n * 16 + l16, k0));
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float u[4], w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                u[r] = bt[r] * E[n][r];
                w[r] = el[r] * u[r];
                const int i = wave * 16 + l4 * 4 + r, e = state_col(n);
                if (a.E && e < a.Dv) a.E[(sh * kC + i) * a.Dv + e] = E[n][r];
            }
            lds_put4<NO>(Ut, PT, LT, n * 16 + l16, wave * 16 + l4 * 4, u);
            lds_put4<3>(Wt, PT, LT, n * 16 + l16, wave * 16 + l4 * 4, w);
        }
        __syncthreads();
        // S = e^{G_last} S + K^T W
        const T* const kt = static_cast<const T*>(a.kt) + ((size_t)slot * a.Hk + hk) * DKP * kC;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n) S[m][n] *= ec;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k0 = s * 32 + l4 * 8;
            const auto pa = plane_frag<NO>(a.att + sh * NO * kC * kC, kC * kC, kC, i0, k0);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const auto wb = plane_frag<3>(Wt, PT, LT, n * 16 + l16, k0);
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    mma<3>(S[m][n], load_frag(kt + (wave * (DKP / 4) + m * 16 + l16) * kC + k0, true), wb);
                mma<NO>(o[n], pa, plane_frag<NO>(Ut, PT, LT, n * 16 + l16, k0));
            }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = wave * 16 + l4 * 4 + r, e = state_col(n);
                if (i < cn && e < a.Dv)
                    Elt<T>::st(static_cast<T*>(a.out), ((size_t)(start + i) * a.Hv + hv) * a.Dv + e, a.scale * o[n][r]);
            }
    }
    if (a.hT) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int d = state_row(m, r), e = state_col(n);
                    if (d < a.Dk && e < a.Dv) a.hT[(((size_t)seq * a.Hv + hv) * a.Dk + d) * a.Dv + e] = S[m][n][r];
                }
    }
}

template <typename T, int DKP>
int launch_delta_fwd(const DeltaArgs& a, hipStream_t s) {
    const int64_t slots = delta_slots(a.T, a.nseq);
    if (a.T > 0) {
        k_delta_prepare<T, DKP, false><<<dim3((unsigned)slots, a.Hk), 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    const unsigned blocks = (unsigned)((int64_t)a.nseq * a.Hv * ((a.Dv + kCols - 1) / kCols));
    k_delta_chain<T, DKP><<<blocks, 256, 0, s>>>(a);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

struct DeltaFwdLayout {
    size_t dec, inv, att, kt, total;
};
inline DeltaFwdLayout delta_fwd_layout(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk, int32_t dtype) {
    const size_t n = (size_t)delta_slots(T, nseq), elt = dtype == SSMP_F32 ? 4 : 2;
    const size_t np = dtype == SSMP_F32 ? kOutP<float> : kOutP<uint16_t>;
    DeltaFwdLayout L;
    L.dec = 0;
    L.inv = L.dec + round256(n * Hv * 2 * kC * 4);
    L.att = L.inv + round256(n * Hv * 3 * kC * kC * 2);
    L.kt = L.att + round256(n * Hv * np * kC * kC * 2);
    L.total = L.kt + round256(n * Hk * delta_dkp(Dk) * kC * elt);
    return L;
}

}  // namespace ssmp

extern "C" size_t gated_delta_pack_saved_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                               int32_t Dv) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, SSMP_F32) || T == 0) return 0;
    const size_t n = (size_t)delta_slots(T, nseq) * Hv;
    return round256(n * Dk * Dv * 4) + round256(n * kC * Dv * 4);
}

extern "C" size_t gated_delta_pack_fwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                     int32_t Dv, int32_t dtype) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype) || T == 0) return 0;
    return delta_fwd_layout(T, nseq, Hk, Hv, Dk, dtype).total;
}

extern "C" int gated_delta_pack_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                    const int32_t* cu_seqlens, int32_t nseq, void* out, int64_t T, int32_t Hk,
                                    int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, float scale,
                                    const float* initial_state, float* final_state, void* saved, size_t saved_bytes,
                                    void* scratch, size_t scratch_bytes, void* stream) {
    using namespace ssmp;
    if (const int st = delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    if (!cu_seqlens) return SSMP_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !out)) return SSMP_ERR_NULL;
    if (!aligned16(q, k, v, out, initial_state, final_state, saved, scratch)) return SSMP_ERR_ALIGN;
    if (T > 0 && (!scratch || scratch_bytes < gated_delta_pack_fwd_scratch_bytes(T, nseq, Hk, Hv, Dk, Dv, dtype)))
        return SSMP_ERR_WORKSPACE;
    if (T > 0 && saved && saved_bytes < gated_delta_pack_saved_bytes(T, nseq, Hk, Hv, Dk, Dv))
        return SSMP_ERR_WORKSPACE;
    if (T == 0 && !final_state) return SSMP_OK;
    const DeltaFwdLayout L = delta_fwd_layout(T, nseq, Hk, Hv, Dk, dtype);
    char* const ws = static_cast<char*>(scratch);
    DeltaArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.cu = cu_seqlens;
    a.out = out;
    a.h0 = initial_state;
    a.hT = final_state;
    a.T = T;
    a.nseq = nseq;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dk = Dk;
    a.Dv = Dv;
    a.scale = scale;
    if (T > 0) {
        a.dec = reinterpret_cast<float*>(ws + L.dec);
        a.inv = reinterpret_cast<__bf16*>(ws + L.inv);
        a.att = reinterpret_cast<__bf16*>(ws + L.att);
        a.kt = ws + L.kt;
        if (saved) {
            a.S0 = static_cast<float*>(saved);
            a.E = reinterpret_cast<float*>(static_cast<char*>(saved) +
                                           round256((size_t)delta_slots(T, nseq) * Hv * Dk * Dv * 4));
        }
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wide = Dk > 64;
    if (dtype == SSMP_F32) return wide ? launch_delta_fwd<float, 128>(a, s) : launch_delta_fwd<float, 64>(a, s);
    return wide ? launch_delta_fwd<uint16_t, 128>(a, s) : launch_delta_fwd<uint16_t, 64>(a, s);
}
