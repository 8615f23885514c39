// layer_norm_pack: the layer norm of rows or heads, with the residual sum and
// dropout before it in the same pass, and its gradients. Over a row's D
// components,
//   h = residual + drop(x),  n = (h - mean) r,  r = (var + eps)^(-1/2),  y = n w + b;
// with c = dy w the gradients are
//   dh' = r (c - mean(c) - n mean(c n)) + dh,  dresidual = dh',  dx = drop(dh'),
//   dw = sum_rows dy n,  db = sum_rows dy.
// Bound by HBM: each row is read and written once, and lies in registers
// between (32768 rows of 4096 in bf16 with residual and dropout: forward 205 us
// or 5.2 TB/s, backward with the weights' gradients 341 and 9, 3.9 TB/s, which
// is short of memory's by what two barriers and the generator take in a row).
// That holds for pieces of 8 elements up to 8192 components, and a few registers
// over for fp32 from 4096 on with the weights' gradients. Backward, rows of over
// 8192 do not fit the 128 registers a lane of 1024 has, but for bf16 without the
// weights' gradients, and pass through scratch memory: 4096 rows of 16384 take,
// forward, backward, and backward with dw and db, 79, 96 and 396 us in bf16 (at
// a copy's rate 55, 82, 82), 120, 273 and 478 in fp32 (110, 164, 164). Rows that
// pieces of 8 do not divide are read by the element, of which each has ten rounds
// of the generator to itself: 32768 x 4097 in bf16 takes 304, 451 and 467 us
// (110, 164, 164), with residual and dropout 801 forward and 1130 backward (219,
// 274); over 4096 they spill as well (4096 x 16383 with both: 483 and 1140).
// The variance is formed from the differences from the mean, so that
// no difference of large sums loses it.
#pragma once

#include "dropout.h"

namespace ssmp {

constexpr int kLnMaxD = 16384;
// threads of a workgroup whose rows lie across so many lanes
constexpr int ln_threads(int lanes) { return lanes > 256 ? lanes : 256; }
constexpr int kLnWaves = 16;  // of the largest workgroup

struct LnArgs {
    const void *x, *residual, *dy, *dh;  // backward: x is h
    const float *w, *b;
    void *y, *h;                         // backward: dx, dresidual
    float *dw, *db;
    void* part;                          // backward: [group][2][D] sums
    Drop drop;
    int64_t rows;
    int32_t H, D;
    float eps;
    int32_t wide;                        // the sums in `part` are doubles
};

// sum over the LANES lanes that share a row; a whole workgroup's through LDS
template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
    if constexpr (LANES >= 2) v = dpp_add<0xB1>(v);
    if constexpr (LANES >= 4) v = dpp_add<0x4E>(v);
    if constexpr (LANES >= 8) v = dpp_add<0x141>(v);
    if constexpr (LANES >= 16) v = dpp_add<0x140>(v);
    if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
    if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
    return v;
}
template <int WAVES>
__device__ __forceinline__ float waves_sum(const float* lds) {
    float t[WAVES];
#pragma unroll
    for (int i = 0; i < WAVES; ++i) t[i] = lds[i];
#pragma unroll
    for (int d = 1; d < WAVES; d *= 2)
#pragma unroll
        for (int i = 0; i < WAVES; i += 2 * d) t[i] += t[i + d];
    return t[0];
}
// several sums at one barrier
template <int LANES, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*lds)[kLnWaves]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_sum<LANES>(v[i]);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) lds[i][threadIdx.x >> 6] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = waves_sum<LANES / 64>(lds[i]);
    }
}

// A row of NV pieces of V in each of LANES lanes: piece j of lane i at column (j LANES + i) V
template <typename T, int V, int LANES, int NV>
struct LnRow {
    Piece<T, V> u[NV];
    __device__ __forceinline__ void load(const void* base, int64_t row, int D, int lane, bool on) {
        const T* const p = static_cast<const T*>(base) + row * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LANES + lane) * V;
            if (on && c < D) u[j].load(p + c);
            else u[j].zero();
        }
    }
    __device__ __forceinline__ void add(float (&v)[NV][V]) const {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            float t[V];
            u[j].get(t);
#pragma unroll
            for (int e = 0; e < V; ++e) v[j][e] += t[e];
        }
    }
    static __device__ __forceinline__ void store(void* base, int64_t row, int D, int lane, const float (&v)[NV][V]) {
        T* const p = static_cast<T*>(base) + row * D;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int c = (j * LANES + lane) * V;
            if (c < D) Piece<T, V>::store(p + c, v[j]);
        }
    }
};
template <int V, int LANES, int NV>
__device__ __forceinline__ void drop_row(const Philox& ph, const Drop& d, int64_t row, int D, int lane, float (&v)[NV][V]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint64_t e = (uint64_t)row * D + (j * LANES + lane) * V;
        if constexpr (V == 8) drop8(ph, d, e >> 3, v[j]);
        else v[j][0] = drop1(ph, d, e, v[j][0]);
    }
}
// weights of a lane's columns, fill where there are none
template <int V, int LANES, int NV>
__device__ __forceinline__ void ln_weights(const float* w, int D, int lane, float fill, float (&v)[NV][V]) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int c = (j * LANES + lane) * V + e;
            v[j][e] = w && c < D ? w[c] : fill;
        }
}
// The reciprocal root of a row's variance from the sums of its differences
// from a mean and of their squares. The first sum is what that mean was off by,
// a rounding of its size, which may be far over the row's spread: `more`, to be
// taken off the differences too.
__device__ __forceinline__ float ln_root(const LnArgs& a, float sum, float squares, float& more) {
    more = sum / (float)a.D;
    const float var = squares / (float)a.D - more * more;
    return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
}

// How a row lies: pieces of 8 elements where every row starts at a multiple of
// 16 bytes, single ones otherwise; up to 512 (256) components in one wave or a
// part of it, longer rows across a workgroup of as many lanes as leave each one
// piece, or two: more of them in a lane leave a backward that adds up the
// weights' gradients too few waves a CU to hide the loads (32768 rows of 4096 in
// bf16: 351 us with 512 lanes of one piece, 365 with 256 of two).
struct LnForm {
    int vec, lanes, nv;
};
// The most lanes of a row in two pieces a lane, which waits at barriers with
// half as many waves. bf16, in us, with one piece a lane and with two:
//   rows x columns                32768 x 4096  32768 x 2560  16384 x 8192  4096 x 4096  1024 x 8192
//   forward, residual, dropout    242, 227      175, 159      214, 204      32.4, 33.2   24.3, 24.5
//   forward                       125, 115      110, 85       164, 115      26.5, 24.8   24.3, 20.6
//   backward without dw, db       229, 207      200, 148      238, 281      29.2, 25.0   20.0, 20.2
//   rows x columns                2048 x 4096   1024 x 4096   512 x 4096    256 x 4096   512 x 2560
//   forward, residual, dropout    23.9, 25.1    20.0, 20.3    12.5, 12.7    9.7, 9.7     9.8, 9.9
//   forward                       20.7, 20.5    18.8, 18.7    11.1, 11.0    8.5, 8.6     8.4, 8.4
//   backward without dw, db       18.4, 17.0    11.9, 12.1    11.3, 11.4    11.2, 11.1   10.3, 10.2
//   the same, residual, dropout   23.1, 23.4    15.5, 16.4    14.3, 15.2    13.8, 14.7   12.9, 13.5
// So a few rows lose up to 7 % by it, 1 us, where the call waits for latency; the
// rule looks at columns alone. With the weights' gradients it loses (above), and
// so do rows of fp32 (16384 x 4096: forward 202 and 208, backward 196 and 212).
constexpr int ln_two(bool bf16, bool backward, bool dw) { return !bf16 || dw ? 0 : backward ? 256 : 512; }
inline LnForm ln_form(int32_t D, int two) {
    if (D % 8 == 0) {
        for (int lanes = 4; lanes <= 64; lanes *= 2)
            if (D <= lanes * 8) return {8, lanes, 1};
        for (int lanes = 256; lanes <= 1024; lanes *= 2)
            for (int nv = 1; nv <= (lanes <= two ? 2 : 1); ++nv)
                if (D <= lanes * 8 * nv) return {8, lanes, nv};
        return {8, 1024, 2};
    }
    if (D <= 64) return {1, 64, 1};
    if (D <= 256) return {1, 64, 4};
    if (D <= 1024) return {1, 256, 4};
    return {1, 1024, D <= 4096 ? 4 : D <= 8192 ? 8 : 16};
}
inline int ln_groups(int32_t D, int two) { return ln_threads(ln_form(D, two).lanes) / ln_form(D, two).lanes; }  // of a workgroup
// Workgroups: as many as have room at a time (`most` of 256 threads), a
// multiple of what gives each group one head; at least `least` rows a group
inline int64_t ln_blocks(int64_t rows, int32_t H, int32_t D, int two, int64_t most, int64_t least = 1) {
    const LnForm m = ln_form(D, two);
    const int sg = ln_groups(D, two);
    most = most * 256 / ln_threads(m.lanes);
    int64_t a = H, b = sg;
    while (b) {
        const int64_t t = a % b;
        a = b;
        b = t;
    }
    const int64_t unit = H / a;  // groups = blocks * sg is then a multiple of H
    int64_t n = (rows + sg * least - 1) / (sg * least);
    n = n < most ? n : most;
    return (n + unit - 1) / unit * unit;
}
// Forward half as many workgroups where a lane has two pieces, which are all that
// a CU has room for: more of them start late (4096 x 4096: 35 us, 45 with as many).
// Backward four rows a group at least, or the groups' sums take longer than the
// rows (1237 tokens x 6 heads of 72: rows 10.2 and sums 7.2 us, 11.2 and 16.8
// with a row a group).
constexpr int64_t kLnFwdBlocks = 2048, kLnBwdBlocks = 1024, kLnBwdRows = 4;

// f(vector length, lanes, pieces) of a row's form, as constants
template <int V, int L, int N>
struct LnShape {
    static constexpr int vec = V, lanes = L, nv = N;
};
template <int TWO, typename F>
void ln_dispatch(int32_t D, F f) {
    const LnForm m = ln_form(D, TWO);
    if constexpr (TWO >= 256)
        if (m.vec == 8 && m.lanes == 256 && m.nv == 2) return f(LnShape<8, 256, 2>{});
    if constexpr (TWO >= 512)
        if (m.vec == 8 && m.lanes == 512 && m.nv == 2) return f(LnShape<8, 512, 2>{});
    if (m.vec == 8) {
        switch (m.lanes) {
            case 4: return f(LnShape<8, 4, 1>{});
            case 8: return f(LnShape<8, 8, 1>{});
            case 16: return f(LnShape<8, 16, 1>{});
            case 32: return f(LnShape<8, 32, 1>{});
            case 64: return f(LnShape<8, 64, 1>{});
            case 256: return f(LnShape<8, 256, 1>{});
            case 512: return f(LnShape<8, 512, 1>{});
        }
        return m.nv == 1 ? f(LnShape<8, 1024, 1>{}) : f(LnShape<8, 1024, 2>{});
    }
    if (m.lanes == 64) return m.nv == 1 ? f(LnShape<1, 64, 1>{}) : f(LnShape<1, 64, 4>{});
    if (m.lanes == 256) return f(LnShape<1, 256, 4>{});
    if (m.nv == 4) return f(LnShape<1, 1024, 4>{});
    return m.nv == 8 ? f(LnShape<1, 1024, 8>{}) : f(LnShape<1, 1024, 16>{});
}

inline int ln_check(int64_t T, int32_t H, int32_t D, int32_t dtype) {
    constexpr int64_t most = int64_t(1) << 40;
    if (T < 0 || H < 1 || D < 1 || H > 65536 || T >= (int64_t(1) << 31) || T * H > (most - 1) / D) return SSMP_ERR_SHAPE;
    if (D > kLnMaxD) return SSMP_ERR_UNSUPPORTED;
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    return SSMP_OK;
}
}  // namespace ssmp
