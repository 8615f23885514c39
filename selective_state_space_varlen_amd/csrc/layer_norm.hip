// layer_norm_pack: the layer norm of rows or heads, with the residual sum and
// dropout before it in the same pass, and its gradients. Over a row's D
// components,
//   h = residual + drop(x),  n = (h - mean) r,  r = (var + eps)^(-1/2),  y = n w + b;
// with c = dy w the gradients are
//   dh' = r (c - mean(c) - n mean(c n)) + dh,  dresidual = dh',  dx = drop(dh'),
//   dw = sum_rows dy n,  db = sum_rows dy.
// Bound by HBM: each row is read and written once, and lies in registers
// between. The variance is formed from the differences from the mean, so that
// no difference of large sums loses it.
#include "dropout.h"

namespace ssmp {

constexpr int kLnThreads = 256;
constexpr int kLnMaxD = 16384;

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
__device__ __forceinline__ float row_sum(float v, float* lds) {
    if constexpr (LANES >= 2) v = dpp_add<0xB1>(v);
    if constexpr (LANES >= 4) v = dpp_add<0x4E>(v);
    if constexpr (LANES >= 8) v = dpp_add<0x141>(v);
    if constexpr (LANES >= 16) v = dpp_add<0x140>(v);
    if constexpr (LANES >= 32) v += __shfl_xor(v, 16);
    if constexpr (LANES >= 64) v += __shfl_xor(v, 32);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        v = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    }
    return v;
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
// Both sums over the lanes that share a row, at one barrier
template <int LANES>
__device__ __forceinline__ void row_sums(float& v, float& w, float (*lds)[4]) {
    constexpr int L = LANES > 64 ? 64 : LANES;
    v = row_sum<L>(v, nullptr);
    w = row_sum<L>(w, nullptr);
    if constexpr (LANES > 64) {
        if ((threadIdx.x & 63) == 0) {
            lds[0][threadIdx.x >> 6] = v;
            lds[1][threadIdx.x >> 6] = w;
        }
        __syncthreads();
        v = (lds[0][0] + lds[0][1]) + (lds[0][2] + lds[0][3]);
        w = (lds[1][0] + lds[1][1]) + (lds[1][2] + lds[1][3]);
    }
}
// v becomes (v - mean) r; returns r. The differences from the mean are added
// up once more beside their squares: what the first mean was off by, a
// rounding of its size, which may be far over the row's spread. lds: 3 rows
template <int V, int LANES, int NV>
__device__ __forceinline__ float normalise(const LnArgs& a, int lane, float (&v)[NV][V], float (*lds)[4]) {
    const float n = (float)a.D;
    float s = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) s += v[j][e];
    const float mean = row_sum<LANES>(s, lds[0]) / n;
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[j][e] = (j * LANES + lane) * V + e < a.D ? v[j][e] - mean : 0.0f;
            s += v[j][e];
            s2 = fmaf(v[j][e], v[j][e], s2);
        }
    row_sums<LANES>(s, s2, lds + 1);
    const float more = s / n;
    const float var = s2 / n - more * more;
    const float r = 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) v[j][e] = (j * LANES + lane) * V + e < a.D ? (v[j][e] - more) * r : 0.0f;
    return r;
}

// Groups of LANES lanes take rows group, group + groups, ...: their number is a
// multiple of H, so that a group stays with one head and keeps its weights.
template <typename T, int V, int LANES, int NV, bool DROP>
__global__ __launch_bounds__(kLnThreads) void k_layer_norm_fwd(LnArgs a) {
    constexpr int SG = kLnThreads / LANES;
    constexpr bool KEEP = NV * V <= 16;  // weights in registers
    __shared__ float lds[2][3][4];
    const int lane = threadIdx.x % LANES;
    const int64_t group = (int64_t)blockIdx.x * SG + threadIdx.x / LANES, groups = (int64_t)gridDim.x * SG;
    const int head = (int)(group % a.H);
    const float* const w = a.w ? a.w + (size_t)head * a.D : nullptr;
    const float* const b = a.b ? a.b + (size_t)head * a.D : nullptr;
    float wv[NV][V], bv[NV][V];
    if constexpr (KEEP) {
        ln_weights<V, LANES, NV>(w, a.D, lane, 1.0f, wv);
        ln_weights<V, LANES, NV>(b, a.D, lane, 0.0f, bv);
    }
    LnRow<T, V, LANES, NV> x, res;
    int turn = 0;
    const auto load = [&](int64_t row) {
        x.load(a.x, row, a.D, lane, row < a.rows);
        if (a.residual) res.load(a.residual, row, a.D, lane, row < a.rows);
    };
    load(group);
    const int64_t first = (int64_t)blockIdx.x * SG;  // the same number of turns for every group of a workgroup
    for (int64_t i = 0; first + i * groups < a.rows; ++i) {
        const int64_t row = group + i * groups;
        float v[NV][V] = {};
        x.add(v);
        if constexpr (DROP) drop_row<V, LANES, NV>(Philox(a.drop), a.drop, row, a.D, lane, v);
        if (a.residual) res.add(v);
        load(row + groups);
        if (a.h && row < a.rows) LnRow<T, V, LANES, NV>::store(a.h, row, a.D, lane, v);
        normalise<V, LANES, NV>(a, lane, v, lds[turn]);
        turn ^= 1;
        if constexpr (!KEEP) {
            ln_weights<V, LANES, NV>(w, a.D, lane, 1.0f, wv);
            ln_weights<V, LANES, NV>(b, a.D, lane, 0.0f, bv);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) v[j][e] = fmaf(v[j][e], wv[j][e], bv[j][e]);
        if (row < a.rows) LnRow<T, V, LANES, NV>::store(a.y, row, a.D, lane, v);
    }
}

// Weights' gradients: a lane adds up its columns over its group's rows in 32
// bits for at most kLnFlush rows, then in `part`, in 64 bits where there are
// more; k_layer_norm_dw adds the groups' sums in 64 bits.
constexpr int kLnFlush = 64;

template <typename T, int V, int LANES, int NV, bool DROP, bool DW>
__global__ __launch_bounds__(kLnThreads) void k_layer_norm_bwd(LnArgs a) {
    constexpr int SG = kLnThreads / LANES;
    constexpr bool KEEP = NV * V <= 16;
    __shared__ float lds[2][5][4];
    const int lane = threadIdx.x % LANES;
    const int64_t group = (int64_t)blockIdx.x * SG + threadIdx.x / LANES, groups = (int64_t)gridDim.x * SG;
    const int head = (int)(group % a.H);
    const float* const w = a.w ? a.w + (size_t)head * a.D : nullptr;
    float wv[NV][V], dw[NV][V] = {}, db[NV][V] = {};
    if constexpr (KEEP) ln_weights<V, LANES, NV>(w, a.D, lane, 1.0f, wv);
    LnRow<T, V, LANES, NV> x, dy, dh;
    int turn = 0, added = 0;
    bool again = false;
    const auto load = [&](int64_t row) {
        const bool on = row < a.rows;
        x.load(a.x, row, a.D, lane, on);
        dy.load(a.dy, row, a.D, lane, on);
        if (a.dh) dh.load(a.dh, row, a.D, lane, on);
    };
    const auto flush = [&]() {
        const size_t at = (size_t)group * 2 * a.D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int c = (j * LANES + lane) * V + e;
                if (c >= a.D) continue;
                if (a.wide) {
                    double* const p = static_cast<double*>(a.part) + at + c;
                    p[0] = (again ? p[0] : 0.0) + (double)dw[j][e];
                    p[a.D] = (again ? p[a.D] : 0.0) + (double)db[j][e];
                } else {
                    float* const p = static_cast<float*>(a.part) + at + c;
                    p[0] = dw[j][e];
                    p[a.D] = db[j][e];
                }
                dw[j][e] = db[j][e] = 0.0f;
            }
        again = true;
        added = 0;
    };
    load(group);
    const int64_t first = (int64_t)blockIdx.x * SG;
    for (int64_t i = 0; first + i * groups < a.rows; ++i) {
        const int64_t row = group + i * groups;
        float n[NV][V] = {}, c[NV][V] = {}, d[NV][V] = {};
        x.add(n);
        dy.add(c);
        if (a.dh) dh.add(d);
        load(row + groups);
        const float r = normalise<V, LANES, NV>(a, lane, n, lds[turn]);
        if constexpr (!KEEP) ln_weights<V, LANES, NV>(w, a.D, lane, 1.0f, wv);
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if constexpr (DW) {
                    if (row < a.rows) {
                        dw[j][e] = fmaf(c[j][e], n[j][e], dw[j][e]);
                        db[j][e] += c[j][e];
                    }
                }
                c[j][e] *= wv[j][e];
                s0 += c[j][e];
                s1 = fmaf(c[j][e], n[j][e], s1);
            }
        row_sums<LANES>(s0, s1, lds[turn] + 3);
        turn ^= 1;
        s0 /= (float)a.D;
        s1 /= (float)a.D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) d[j][e] += r * (c[j][e] - s0 - n[j][e] * s1);
        if (a.h && row < a.rows) LnRow<T, V, LANES, NV>::store(a.h, row, a.D, lane, d);
        if constexpr (DROP) drop_row<V, LANES, NV>(Philox(a.drop), a.drop, row, a.D, lane, d);
        if (row < a.rows) LnRow<T, V, LANES, NV>::store(a.y, row, a.D, lane, d);
        if constexpr (DW)
            if (++added == kLnFlush && a.wide) flush();
    }
    if constexpr (DW)
        if (!again || added) flush();
}

// The groups' sums of one head, 32 columns a workgroup, every 32nd group a lane
constexpr int kLnDwThreads = 1024, kLnDwLanes = kLnDwThreads / 32;
template <typename S>
__global__ __launch_bounds__(kLnDwThreads) void k_layer_norm_dw(LnArgs a, int64_t groups) {
    const int cols = 2 * a.D, nb = (cols + 31) / 32, head = blockIdx.x / nb, c = blockIdx.x % nb * 32 + threadIdx.x % 32;
    const int lane = threadIdx.x / 32;
    const S* const part = static_cast<const S*>(a.part);
    double s = 0.0;
    if (c < cols) {
        constexpr int kBatch = 16;  // loads under way
        const int64_t step = (int64_t)kLnDwLanes * a.H;
        for (int64_t g = head + (int64_t)lane * a.H; g < groups; g += kBatch * step) {
            S v[kBatch];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) v[x] = g + x * step < groups ? part[(size_t)(g + x * step) * cols + c] : S(0);
#pragma unroll
            for (int x = 0; x < kBatch; ++x) s += (double)v[x];
        }
    }
    __shared__ double lds[kLnDwLanes][32];
    lds[lane][threadIdx.x % 32] = s;
    __syncthreads();
    if (lane == 0 && c < cols) {
        for (int i = 1; i < kLnDwLanes; ++i) s += lds[i][threadIdx.x];
        float* const to = c < a.D ? a.dw : a.db;
        if (to) to[(size_t)head * a.D + (c < a.D ? c : c - a.D)] = (float)s;
    }
}

// How a row lies: pieces of 8 elements where every row starts at a multiple of
// 16 bytes, single ones otherwise; up to 512 components in one wave or a part
// of it, longer rows in a workgroup.
struct LnForm {
    int vec, lanes, nv;
};
inline LnForm ln_form(int32_t D) {
    if (D % 8 == 0) {
        for (int lanes = 4; lanes <= 64; lanes *= 2)
            if (D <= lanes * 8) return {8, lanes, 1};
        return {8, 256, D <= 2048 ? 1 : D <= 4096 ? 2 : D <= 8192 ? 4 : 8};
    }
    if (D <= 64) return {1, 64, 1};
    if (D <= 256) return {1, 64, 4};
    return {1, 256, D <= 1024 ? 4 : D <= 4096 ? 16 : 64};
}
// Workgroups: enough to fill the GPU, a multiple of what gives each group one head
inline int64_t ln_blocks(int64_t rows, int32_t H, int32_t D, int64_t most) {
    const int sg = kLnThreads / ln_form(D).lanes;
    int64_t a = H, b = sg;
    while (b) {
        const int64_t t = a % b;
        a = b;
        b = t;
    }
    const int64_t unit = H / a;  // groups = blocks * sg is then a multiple of H
    int64_t n = (rows + sg - 1) / sg;
    n = n < most ? n : most;
    n = (n + unit - 1) / unit * unit;
    return n;
}
constexpr int64_t kLnFwdBlocks = 2048, kLnBwdBlocks = 1024;

template <typename T, int V, int LANES, int NV>
void launch_ln_form(const LnArgs& a, bool bwd, bool dw, int64_t blocks, hipStream_t s) {
    const dim3 g((unsigned)blocks), b(kLnThreads);
    const bool drop = a.drop.cut > 0;
    if (!bwd) {
        if (drop) k_layer_norm_fwd<T, V, LANES, NV, true><<<g, b, 0, s>>>(a);
        else k_layer_norm_fwd<T, V, LANES, NV, false><<<g, b, 0, s>>>(a);
    } else if (dw) {
        if (drop) k_layer_norm_bwd<T, V, LANES, NV, true, true><<<g, b, 0, s>>>(a);
        else k_layer_norm_bwd<T, V, LANES, NV, false, true><<<g, b, 0, s>>>(a);
    } else {
        if (drop) k_layer_norm_bwd<T, V, LANES, NV, true, false><<<g, b, 0, s>>>(a);
        else k_layer_norm_bwd<T, V, LANES, NV, false, false><<<g, b, 0, s>>>(a);
    }
}
template <typename T>
void launch_ln(const LnArgs& a, bool bwd, bool dw, int64_t n, hipStream_t s) {
    const LnForm f = ln_form(a.D);
    if (f.vec == 8) {
        switch (f.lanes) {
            case 4: return launch_ln_form<T, 8, 4, 1>(a, bwd, dw, n, s);
            case 8: return launch_ln_form<T, 8, 8, 1>(a, bwd, dw, n, s);
            case 16: return launch_ln_form<T, 8, 16, 1>(a, bwd, dw, n, s);
            case 32: return launch_ln_form<T, 8, 32, 1>(a, bwd, dw, n, s);
            case 64: return launch_ln_form<T, 8, 64, 1>(a, bwd, dw, n, s);
        }
        switch (f.nv) {
            case 1: return launch_ln_form<T, 8, 256, 1>(a, bwd, dw, n, s);
            case 2: return launch_ln_form<T, 8, 256, 2>(a, bwd, dw, n, s);
            case 4: return launch_ln_form<T, 8, 256, 4>(a, bwd, dw, n, s);
            default: return launch_ln_form<T, 8, 256, 8>(a, bwd, dw, n, s);
        }
    }
    if (f.lanes == 64) {
        if (f.nv == 1) return launch_ln_form<T, 1, 64, 1>(a, bwd, dw, n, s);
        return launch_ln_form<T, 1, 64, 4>(a, bwd, dw, n, s);
    }
    switch (f.nv) {
        case 4: return launch_ln_form<T, 1, 256, 4>(a, bwd, dw, n, s);
        case 16: return launch_ln_form<T, 1, 256, 16>(a, bwd, dw, n, s);
        default: return launch_ln_form<T, 1, 256, 64>(a, bwd, dw, n, s);
    }
}

inline int ln_check(int64_t T, int32_t H, int32_t D, int32_t dtype) {
    if (T < 0 || H < 1 || D < 1 || H > 65536 || T >= (int64_t(1) << 31) || T * H >= (int64_t(1) << 40) ||
        T * H * D >= (int64_t(1) << 40))
        return SSMP_ERR_SHAPE;
    if (D > kLnMaxD) return SSMP_ERR_UNSUPPORTED;
    if ((int64_t)H * ((2 * D + 31) / 32) >= kMaxBlocks / 4) return SSMP_ERR_SHAPE;  // k_layer_norm_dw's workgroups of 1024
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    return SSMP_OK;
}
// The backward's sums for any number of rows up to T H: a group adds at most
// kLnFlush rows in 32 bits, and keeps doubles where it has more.
inline bool ln_wide(int64_t rows, int64_t blocks, int32_t D) {
    const int64_t groups = blocks * (kLnThreads / ln_form(D).lanes);
    return (rows + groups - 1) / groups > kLnFlush;
}
inline size_t ln_part_bytes(int64_t rows, int32_t H, int32_t D) {
    const int64_t blocks = ln_blocks(rows, H, D, kLnBwdBlocks);
    return (size_t)blocks * (kLnThreads / ln_form(D).lanes) * 2 * D * (ln_wide(rows, blocks, D) ? 8 : 4);
}

}  // namespace ssmp

extern "C" int layer_norm_pack_fwd(const void* x, const void* residual, const float* w, const float* b,
                                   const uint64_t* rng, void* y, void* h, int64_t T, int32_t H, int32_t D,
                                   int32_t dtype, double p, float eps, void* stream) {
    using namespace ssmp;
    if (const int st = ln_check(T, H, D, dtype)) return st;
    LnArgs a = {};
    if (!make_drop(p, rng, a.drop)) return SSMP_ERR_SHAPE;
    if (T == 0) return SSMP_OK;
    if (!x || !y || (a.drop.cut && !rng)) return SSMP_ERR_NULL;
    if (!aligned16(x, residual, y, h)) return SSMP_ERR_ALIGN;
    a.x = x;
    a.residual = residual;
    a.w = w;
    a.b = b;
    a.y = y;
    a.h = h;
    a.rows = T * H;
    a.H = H;
    a.D = D;
    a.eps = eps;
    const int64_t blocks = ln_blocks(a.rows, H, D, kLnFwdBlocks);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SSMP_F32) launch_ln<float>(a, false, false, blocks, s);
    else launch_ln<uint16_t>(a, false, false, blocks, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

extern "C" size_t layer_norm_pack_bwd_workspace_bytes(int64_t T, int32_t H, int32_t D) {
    using namespace ssmp;
    if (ln_check(T, H, D, SSMP_F32) || T == 0) return 0;
    return ln_part_bytes(T * H, H, D);
}

extern "C" int layer_norm_pack_bwd(const void* dy, const void* h, const float* w, const void* dh, const uint64_t* rng,
                                   void* dx, void* dresidual, float* dw, float* db, void* workspace,
                                   size_t workspace_bytes, int64_t T, int32_t H, int32_t D, int32_t dtype, double p,
                                   float eps, void* stream) {
    using namespace ssmp;
    if (const int st = ln_check(T, H, D, dtype)) return st;
    LnArgs a = {};
    if (!make_drop(p, rng, a.drop)) return SSMP_ERR_SHAPE;
    if (dw && !w) return SSMP_ERR_NULL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        if (const int st = zero_f32(dw, (int64_t)H * D, s)) return st;
        return zero_f32(db, (int64_t)H * D, s);
    }
    if (!dy || !h || !dx || (a.drop.cut && !rng)) return SSMP_ERR_NULL;
    if (!aligned16(dy, h, dh, dx, dresidual)) return SSMP_ERR_ALIGN;
    const bool sums = dw || db;
    if (sums && (!workspace || workspace_bytes < layer_norm_pack_bwd_workspace_bytes(T, H, D)))
        return SSMP_ERR_WORKSPACE;
    if (sums && !aligned16(workspace)) return SSMP_ERR_ALIGN;
    a.x = h;
    a.dy = dy;
    a.dh = dh;
    a.w = w;
    a.y = dx;
    a.h = dresidual;
    a.dw = dw;
    a.db = db;
    a.part = workspace;
    a.rows = T * H;
    a.H = H;
    a.D = D;
    a.eps = eps;
    const int64_t blocks = ln_blocks(a.rows, H, D, kLnBwdBlocks);
    a.wide = ln_wide(a.rows, blocks, D);
    if (dtype == SSMP_F32) launch_ln<float>(a, true, sums, blocks, s);
    else launch_ln<uint16_t>(a, true, sums, blocks, s);
    SSMP_LAUNCH_CHECK();
    if (sums) {
        const unsigned n = (unsigned)((int64_t)H * ((2 * D + 31) / 32));
        const int64_t groups = blocks * (kLnThreads / ln_form(D).lanes);
        if (a.wide) k_layer_norm_dw<double><<<n, kLnDwThreads, 0, s>>>(a, groups);
        else k_layer_norm_dw<float><<<n, kLnDwThreads, 0, s>>>(a, groups);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}
