// What the forward and the backward of the gated delta rule make of every chunk
// before they go along the sequences: nothing here depends on the states.
#pragma once

#include "delta_common.h"

namespace ssmp {

// One workgroup per (slot, value head); the heads of a group run on one XCD,
// whose L2 then holds their keys and queries, and the first of them also
// writes these transposed.
//   forward:  (I + L diag(beta))^-1 and P,           both lower triangular
//   backward: (I + diag(beta) L)^-T and scale P^T,   both upper triangular
template <typename T, int DKP, bool BWD>
__global__ __launch_bounds__(256) void k_delta_prepare(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    using Rows = Tile<T, DKP>;
    constexpr int kKeys = kC * DKP * (int)sizeof(T), kMats = kC * kLdA * 4;
    // keys and queries; then, once they are multiplied, the matrix and its inverse
    __shared__ alignas(16) char lds[2 * (kKeys > kMats ? kKeys : kMats)];
    __shared__ double G[kC];
    __shared__ float beta[kC];
    T* const Kl = reinterpret_cast<T*>(lds);
    T* const Ql = Kl + kC * DKP;
    float* const A = reinterpret_cast<float*>(lds);
    float* const X = A + kC * kLdA;
    const int members = a.Hv / a.Hk;
    const Spread sp = spread(blockIdx.x, members);
    const int64_t slots = delta_slots(a.T, a.nseq);
    if (sp.group >= slots * a.Hk) return;
    const int64_t slot = sp.group / a.Hk;
    const int hk = (int)(sp.group % a.Hk), hv = hk * members + sp.member;
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, slot, c)) return;
    const int tid = threadIdx.x, wave = wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    constexpr int kUnits = DKP / 8;
#pragma unroll
    for (int u = tid; u < kC * kUnits; u += 256) {
        const int i = u / kUnits, k8 = u % kUnits;
        const bool on = i < c.n && k8 * 8 < a.Dk;
        const size_t o = ((size_t)(c.start + i) * a.Hk + hk) * a.Dk + k8 * 8;
        copy8(Kl + Rows::at(i, k8), static_cast<const T*>(a.k) + o, on);
        copy8(Ql + Rows::at(i, k8), static_cast<const T*>(a.q) + o, on);
    }
    const size_t sh = (size_t)slot * a.Hv + hv;
    if (wave == 0) {
        const double s = chunk_decay_sum(a.g, c.start, c.n, a.Hv, hv);
        G[l] = s;
        beta[l] = l < c.n ? a.beta[(size_t)(c.start + l) * a.Hv + hv] : 0.0f;
        const double last = __shfl(s, kC - 1);
        a.dec[sh * 2 * kC + l] = expf((float)s);
        a.dec[sh * 2 * kC + kC + l] = expf((float)(last - s));
    }
    __syncthreads();
    // Wave w has rows 16 w .. of both products. kk: K K^T. qk: forward K Q^T
    // (rows j, columns i), backward Q K^T (rows i, columns j): a lane then
    // holds four contiguous k of one row of what is stored.
    f32x4 kk[4] = {}, qk[4] = {};
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
        const int i = wave * 16 + l16, u = s * 4 + l4;
        const auto ka = tile_frag(Kl + Rows::at(i, u));
        const auto qa = tile_frag(Ql + Rows::at(i, u));
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int j = n * 16 + l16;
            const bool below = n <= wave;  // tiles with some i >= j, rows i
            if (below || !BWD) {
                const auto kb = tile_frag(Kl + Rows::at(j, u));
                if (below) mma<NX>(kk[n], ka, kb);
                if constexpr (BWD) mma<NX>(qk[n], qa, kb);
            }
            if constexpr (!BWD)
                if (n >= wave) mma<NX>(qk[n], ka, tile_frag(Ql + Rows::at(j, u)));
        }
    }
    if (sp.member == 0) {
        // keys (and for the backward queries) as [d][token], 8 places a lane
        for (int w = 0; w < (BWD ? 2 : 1); ++w) {
            const T* const src = w ? Ql : Kl;
            T* const dst = static_cast<T*>(w ? a.qt : a.kt) + ((size_t)slot * a.Hk + hk) * DKP * kC;
            for (int u = tid; u < DKP * 8; u += 256) {
                const int d = u >> 3, p = u & 7, i = (p >> 2) * 32 + (p & 3) * 4;
                T v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = i + (e < 4 ? e : 12 + e);
                    v[e] = src[Rows::at(t, d >> 3) + (d & 7)];
                }
                put8(dst + d * kC + p * 8, v);
            }
        }
    }
    __syncthreads();
    float* const att = a.att + sh * kTri;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        f32x4 p;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = wave * 16 + l4 * 4 + r, j = n * 16 + l16;  // row and column of the tiles
            const float d = expf((float)(i > j ? G[i] - G[j] : G[j] - G[i]));
            A[i * kLdA + j] = i > j ? (BWD ? beta[i] : beta[j]) * d * kk[n][r] : 0.0f;
            if constexpr (BWD) p[r] = i >= j ? d * qk[n][r] * a.scale : 0.0f;
            else p[r] = j >= i ? d * qk[n][r] : 0.0f;
        }
        const int row = n * 16 + l16, k = wave * 16 + l4 * 4;
        // what lies in neither block of the other triangle is not stored
        if (BWD ? (k >= 32 || row < 32) : (k < 32 || row >= 32))
            *reinterpret_cast<f32x4*>(att + tri_row<BWD>(row, k) * 32 + (kplace(k) & 31)) = p;
    }
    __syncthreads();
    chunk_inverse(A, X);
    float* const inv = a.inv + sh * kTri;
    for (int e = tid; e < kTri / 4; e += 256) {
        const int t = e >> 3, q = e & 7;
        const bool second = t >= 64;  // place q of block: k = 4 g, g = q / 2 + 4 (q % 2)
        const int row = BWD ? (second ? t - 64 : t) : (second ? t - 32 : t);
        const int k = (BWD != second ? 32 : 0) + ((q >> 1) + (q & 1) * 4) * 4;
        f32x4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = BWD ? X[(k + x) * kLdA + row] : X[row * kLdA + k + x];
        *reinterpret_cast<f32x4*>(inv + t * 32 + q * 4) = v;
    }
}

template <typename T, int DKP, bool BWD>
int launch_delta_prepare(const DeltaArgs& a, hipStream_t s) {
    const int64_t blocks = spread_blocks(delta_slots(a.T, a.nseq) * a.Hk, a.Hv / a.Hk);
    k_delta_prepare<T, DKP, BWD><<<(unsigned)blocks, 256, 0, s>>>(a);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

// ---------------------------------------------------------------------------
// The operands of one chunk that a chain holds in LDS, for its four waves, and
// the registers in which the next chunk's are under way meanwhile.
//   rows:  keys (forward: and queries), [token][d in places]
//   cols:  keys (backward: and queries) transposed, [d][token in places]
//   tris:  the inverse (3 planes) and the products (NP planes)
// 78 KB for bf16 heads of 128, so that two workgroups share a CU.
template <typename T, int DKP, int NROWS, int NCOLS, int NP>
struct ChainTiles {
    static constexpr int kRow = kC * DKP, kCol = DKP * kC;
    using Rows = Tile<T, DKP>;
    using Cols = Tile<T, kC>;
    T rows[NROWS][kRow];
    T cols[NCOLS][kCol];
    __bf16 inv[3 * kTri];
    __bf16 att[NP * kTri];
    float eg[kC], el[kC], beta[kC];

    __device__ __forceinline__ Frag<kExact<T>> row_frag(int w, int row, int unit) const {
        return tile_frag(rows[w] + Rows::at(row, unit));
    }
    __device__ __forceinline__ Frag<kExact<T>> col_frag(int w, int row, int unit) const {
        return tile_frag(cols[w] + Cols::at(row, unit));
    }
};

template <typename T, int DKP, int NROWS, int NCOLS, int NP>
struct ChainLoads {
    using Tiles = ChainTiles<T, DKP, NROWS, NCOLS, NP>;
    static constexpr int kN = DKP * kC / 8 / 256;  // units of 8 elements a thread
    Unit<T> rows[NROWS][kN], cols[NCOLS][kN];
    f32x4 inv[kTri / 4 / 256], att[kTri / 4 / 256];
    float dec;

    __device__ __forceinline__ void load(const DeltaArgs& a, int64_t slot, int64_t start, int n, int hk, int hv) {
        const int tid = threadIdx.x;
        const size_t sh = (size_t)slot * a.Hv + hv;
        const size_t first = ((size_t)start * a.Hk + hk) * a.Dk, tr = ((size_t)slot * a.Hk + hk) * DKP * kC;
        const int stride = a.Hk * a.Dk;
        const auto k = rows_rsrc(static_cast<const T*>(a.k) + first, n, stride, a.Dk);
        const auto q = rows_rsrc(static_cast<const T*>(a.q) + first, n, stride, a.Dk);
        const auto kt = bytes_rsrc(static_cast<const T*>(a.kt) + tr, DKP * kC * sizeof(T));
        const auto qt = bytes_rsrc(static_cast<const T*>(a.qt) + tr, DKP * kC * sizeof(T));
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int u = tid + x * 256, i = u / (DKP / 8), k8 = u % (DKP / 8);
            const uint32_t o = k8 * 8 < a.Dk ? (uint32_t)(i * stride + k8 * 8) * (uint32_t)sizeof(T) : kNowhere;
            rows[0][x].load(k, o);
            if constexpr (NROWS > 1) rows[1][x].load(q, o);
            cols[0][x].load(kt, (uint32_t)u * 8u * (uint32_t)sizeof(T));
            if constexpr (NCOLS > 1) cols[1][x].load(qt, (uint32_t)u * 8u * (uint32_t)sizeof(T));
        }
#pragma unroll
        for (int x = 0; x < kTri / 4 / 256; ++x) {
            inv[x] = *reinterpret_cast<const f32x4*>(at_bytes(a.inv + sh * kTri, (uint32_t)(tid + x * 256) * 16u));
            att[x] = *reinterpret_cast<const f32x4*>(at_bytes(a.att + sh * kTri, (uint32_t)(tid + x * 256) * 16u));
        }
        dec = 0.0f;
        if (tid < 2 * kC) dec = a.dec[sh * 2 * kC + tid];
        else if (tid < 2 * kC + n) dec = a.beta[(size_t)(start + tid - 2 * kC) * a.Hv + hv];
    }
    __device__ __forceinline__ void put(Tiles& t) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int u = tid + x * 256, i = u / (DKP / 8), k8 = u % (DKP / 8);
            // d = 8 k8 .. + 3 and + 4 .. + 7 go to two places
            const int p0 = kplace(k8 * 8), p1 = kplace(k8 * 8 + 4);
#pragma unroll
            for (int w = 0; w < NROWS; ++w) {
                rows[w][x].put_half(t.rows[w] + Tiles::Rows::at(i, p0 >> 3) + (p0 & 4), 0);
                rows[w][x].put_half(t.rows[w] + Tiles::Rows::at(i, p1 >> 3) + (p1 & 4), 1);
            }
#pragma unroll
            for (int w = 0; w < NCOLS; ++w) {
                T* const p = t.cols[w] + Tiles::Cols::at(u >> 3, u & 7);
                cols[w][x].put_half(p, 0);
                cols[w][x].put_half(p + 4, 1);
            }
        }
#pragma unroll
        for (int x = 0; x < kTri / 4 / 256; ++x) {
            tri_put4<3>(t.inv, tid + x * 256, inv[x]);
            tri_put4<NP>(t.att, tid + x * 256, att[x]);
        }
        if (tid < kC) t.eg[tid] = dec;
        else if (tid < 2 * kC) t.el[tid - kC] = dec;
        else if (tid < 3 * kC) t.beta[tid - 2 * kC] = dec;
    }
};

// workgroups of a chain that share a CU (as waves per SIMD, for the register budget)
template <typename T>
constexpr int NWG = std::is_same<T, float>::value ? 1 : 2;

// A lane's elements of a (tokens, Dv) tensor of one head, as a result of 4
// tiles holds them: tokens 16 m + 4 (l / 16) + r of its column (kNowhere where
// the column is none).
struct Column {
    uint32_t o;  // byte offset of its first element
    int stride;  // bytes between tokens
};
template <typename T>
__device__ __forceinline__ Column column_of(int H, int Dv, int col) {
    const int stride = H * Dv * (int)sizeof(T), l4 = lane_id() >> 4;
    return {col < Dv ? (uint32_t)(l4 * 4 * stride + col * (int)sizeof(T)) : kNowhere, stride};
}
// The offset again, in a way that the compiler does not see through: it would
// else form the offsets of all rows ahead of the loop over the chunks and keep
// them, 64 registers that the chain does not have.
__device__ __forceinline__ uint32_t fresh(uint32_t o) {
    asm volatile("" : "+v"(o));
    return o;
}
template <typename T>
__device__ __forceinline__ void load_column(const void* p, int64_t start, int n, int H, int h, int Dv, const Column& c,
                                            uint32_t (&v)[16]) {
    const auto r = rows_rsrc(static_cast<const T*>(p) + ((size_t)start * H + h) * Dv, n, H * Dv, Dv);
    const uint32_t o = fresh(c.o);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = Elt<T>::raw_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride);
}
template <typename T>
__device__ __forceinline__ void store_column(void* p, int64_t start, int n, int H, int h, int Dv, const Column& c,
                                             const f32x4 (&v)[4], float scale) {
    const auto r = rows_rsrc(static_cast<T*>(p) + ((size_t)start * H + h) * Dv, n, H * Dv, Dv);
    const uint32_t o = fresh(c.o);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        Elt<T>::st_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride, scale * v[i >> 2][i & 3]);
}
// the same of a dense fp32 matrix of `rows` rows (a state; E or dU of a chunk)
template <int MT>
__device__ __forceinline__ void store_matrix(float* p, int rows, int Dv, const Column& c, const f32x4 (&v)[MT]) {
    const auto r = rows_rsrc(p, rows, Dv, Dv);
    const uint32_t o = fresh(c.o);
#pragma unroll
    for (int i = 0; i < MT * 4; ++i)
        Elt<float>::st_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride, v[i >> 2][i & 3]);
}
template <int MT>
__device__ __forceinline__ void load_matrix(const float* p, int rows, int Dv, const Column& c, f32x4 (&v)[MT]) {
    const auto r = rows_rsrc(p, p ? rows : 0, Dv, Dv);
#pragma unroll
    for (int i = 0; i < MT * 4; ++i)
        v[i >> 2][i & 3] = Elt<float>::cvt(
            Elt<float>::raw_rsrc(r, c.o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride));
}

}  // namespace ssmp
