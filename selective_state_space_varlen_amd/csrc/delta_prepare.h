// What the forward and the backward of the gated delta rule make of every chunk
// before they go along the sequences: nothing here depends on the states.
#pragma once

#include "delta_common.h"

namespace ssmp {

// planes of P and of U where they form the output: its own rounding to bf16
// hides what two planes (16 bits) leave out
template <typename T>
constexpr int kOutP = std::is_same<T, float>::value ? 3 : 2;

// One workgroup per (slot, key head): its products K K^T and Q K^T serve all
// value heads of the group.
template <typename T, int DKP, bool BWD>
__global__ __launch_bounds__(256) void k_delta_prepare(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    const int64_t slot = blockIdx.x;
    const int hk = blockIdx.y;
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, slot, c)) return;
    const int tid = threadIdx.x, wave = tid >> 6, l = tid & 63, l16 = l & 15, l4 = l >> 4;
    __shared__ alignas(16) float A[kC * kLdA], X[kC * kLdA];
    __shared__ double G[kC];
    __shared__ float beta[kC];
    const T* const kp = static_cast<const T*>(a.k);
    const T* const qp = static_cast<const T*>(a.q);
    const auto row = [&](int i) { return ((size_t)(c.start + i) * a.Hk + hk) * a.Dk; };
    // kk[n]: rows (4 l4 ..) of tile `wave`, columns of tile n, of K K^T. qk[n]:
    // forward: K Q^T (rows j, columns i), so that a lane holds four j of one i;
    // backward: Q K^T, four i of one j.
    f32x4 kk[4] = {}, qk[4] = {};
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
        const int k0 = s * 32 + l4 * 8;
        const int i = wave * 16 + l16;
        const auto ka = load_frag(kp + row(i) + k0, i < c.n && k0 < a.Dk);
        const auto qa = load_frag(qp + row(i) + k0, i < c.n && k0 < a.Dk);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int j = n * 16 + l16;
            const auto kb = load_frag(kp + row(j) + k0, j < c.n && k0 < a.Dk);
            mma<NX>(kk[n], ka, kb);
            if constexpr (BWD) mma<NX>(qk[n], qa, kb);
            else mma<NX>(qk[n], ka, load_frag(qp + row(j) + k0, j < c.n && k0 < a.Dk));
        }
    }
    // keys (and for the backward queries) transposed to [d][token]
    for (int w = 0; w < (BWD ? 2 : 1); ++w) {
        const T* const src = w ? qp : kp;
        T* const dst = static_cast<T*>(w ? a.qt : a.kt) + ((size_t)slot * a.Hk + hk) * DKP * kC;
        for (int e = tid; e < DKP * kC; e += 256) {
            const int i = e & 63, d = e >> 6;
            dst[e] = i < c.n && d < a.Dk ? src[row(i) + d] : T(0);
        }
    }
    for (int hv = hk * (a.Hv / a.Hk); hv < (hk + 1) * (a.Hv / a.Hk); ++hv) {
        const size_t sh = (size_t)slot * a.Hv + hv;
        __syncthreads();  // the last head's A, G and beta have been read
        if (wave == 0) {
            const double s = chunk_decay_sum(a.g, c.start, c.n, a.Hv, hv);
            G[l] = s;
            beta[l] = l < c.n ? a.beta[(size_t)(c.start + l) * a.Hv + hv] : 0.0f;
            const double last = __shfl(s, kC - 1);
            a.dec[sh * 2 * kC + l] = expf((float)s);
            a.dec[sh * 2 * kC + kC + l] = expf((float)(last - s));
        }
        __syncthreads();
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            float p[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = wave * 16 + l4 * 4 + r, j = n * 16 + l16;  // row and column of the tiles
                const float d = i > j ? expf((float)(G[i] - G[j])) : 0.0f;
                A[i * kLdA + j] = i > j ? (BWD ? beta[i] : beta[j]) * d * kk[n][r] : 0.0f;
                if constexpr (BWD) {
                    p[r] = i >= j ? (i == j ? 1.0f : d) * qk[n][r] * a.scale : 0.0f;
                } else {  // rows are j here, columns i
                    const float e = j >= i ? expf((float)(G[j] - G[i])) : 0.0f;
                    p[r] = j >= i ? e * qk[n][r] : 0.0f;
                }
            }
            // forward: att[i][j], lane's i = its column, four j. Backward: att[j][i], transposed.
            constexpr int NPA = BWD ? 3 : kOutP<T>;
            __bf16* const att = a.att + sh * NPA * kC * kC;
            lds_put4<NPA>(att, kC * kC, kC, n * 16 + l16, wave * 16 + l4 * 4, p);
        }
        __syncthreads();
        chunk_inverse(A, X);
        __bf16* const inv = a.inv + sh * 3 * kC * kC;
        for (int e = tid; e < kC * kC / 4; e += 256) {
            const int r = e >> 4, k4 = (e & 15) * 4;
            float v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) v[x] = BWD ? X[(k4 + x) * kLdA + r] : X[r * kLdA + k4 + x];
            lds_put4<3>(inv, kC * kC, kC, r, k4, v);
        }
    }
}

}  // namespace ssmp
