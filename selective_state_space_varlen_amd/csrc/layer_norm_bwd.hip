// layer_norm_pack_bwd: the gradients of layer_norm_pack_fwd.
#include "layer_norm.h"

namespace ssmp {

// Weights' gradients: a lane adds up its columns over its group's rows in 32
// bits for at most kLnFlush rows, then in `part`, in 64 bits where there are
// more; k_layer_norm_dw adds the groups' sums in 64 bits.
constexpr int kLnFlush = 64;

template <typename T, int V, int LANES, int NV, bool DROP, bool DW>
__global__ __launch_bounds__(ln_threads(LANES)) void k_layer_norm_bwd(LnArgs a) {
    constexpr int SG = ln_threads(LANES) / LANES;
    __shared__ float lds[2][5][kLnWaves];
    const int lane = threadIdx.x % LANES;
    const int64_t group = (int64_t)blockIdx.x * SG + threadIdx.x / LANES, groups = (int64_t)gridDim.x * SG;
    const int head = (int)(group % a.H);
    const float* const w = a.w ? a.w + (size_t)head * a.D : nullptr;
    float wv[NV][V], dw[NV][V] = {}, db[NV][V] = {};
    ln_weights<V, LANES, NV>(w, a.D, lane, 1.0f, wv);
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
        // mean(c n) = r (mean(c (h - m)) - (mean - m) mean(c)) for a mean m that is nearly right
        float one[2] = {}, two[3] = {}, more;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                one[0] += n[j][e];
                one[1] = fmaf(c[j][e], wv[j][e], one[1]);
            }
        row_sums<LANES>(one, lds[turn]);
        const float mean = one[0] / (float)a.D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                n[j][e] = (j * LANES + lane) * V + e < a.D ? n[j][e] - mean : 0.0f;
                two[0] += n[j][e];
                two[1] = fmaf(n[j][e], n[j][e], two[1]);
                two[2] = fmaf(c[j][e] * wv[j][e], n[j][e], two[2]);
            }
        row_sums<LANES>(two, lds[turn] + 2);
        turn ^= 1;
        const float r = ln_root(a, two[0], two[1], more);
        const float s0 = one[1] / (float)a.D, s1 = r * (two[2] / (float)a.D - more * s0);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = (n[j][e] - more) * r;
                if constexpr (DW) {
                    if (row < a.rows) {
                        dw[j][e] = fmaf(c[j][e], x, dw[j][e]);
                        db[j][e] += c[j][e];
                    }
                }
                d[j][e] += r * (c[j][e] * wv[j][e] - s0 - x * s1);
            }
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

template <typename T, bool DW>
void launch_ln_bwd(const LnArgs& a, int64_t blocks, hipStream_t s) {
    ln_dispatch<ln_two(sizeof(T) == 2, true, DW)>(a.D, [&](auto f) {
        constexpr int V = decltype(f)::vec, L = decltype(f)::lanes, N = decltype(f)::nv;
        const dim3 g((unsigned)blocks), b(ln_threads(L));
        if (a.drop.cut) k_layer_norm_bwd<T, V, L, N, true, DW><<<g, b, 0, s>>>(a);
        else k_layer_norm_bwd<T, V, L, N, false, DW><<<g, b, 0, s>>>(a);
    });
}

// The backward's sums for any number of rows up to T H: a group adds at most
// kLnFlush rows in 32 bits, and keeps doubles where it has more.
inline bool ln_wide(int64_t rows, int64_t blocks, int32_t D) {
    const int64_t groups = blocks * ln_groups(D, 0);
    return (rows + groups - 1) / groups > kLnFlush;
}
// k_layer_norm_dw's workgroups are more than a launch takes
inline bool ln_dw_over(int32_t H, int32_t D) { return (int64_t)H * ((2 * D + 31) / 32) >= kMaxBlocks * 256 / kLnDwThreads; }
inline size_t ln_part_bytes(int64_t rows, int32_t H, int32_t D) {
    const int64_t blocks = ln_blocks(rows, H, D, 0, kLnBwdBlocks, kLnBwdRows);
    return (size_t)blocks * ln_groups(D, 0) * 2 * D * (ln_wide(rows, blocks, D) ? 8 : 4);
}

}  // namespace ssmp

extern "C" size_t layer_norm_pack_bwd_workspace_bytes(int64_t T, int32_t H, int32_t D) {
    using namespace ssmp;
    if (ln_check(T, H, D, SSMP_F32) || ln_dw_over(H, D) || T == 0) return 0;
    return ln_part_bytes(T * H, H, D);
}

extern "C" int layer_norm_pack_bwd(const void* dy, const void* h, const float* w, const void* dh, const uint64_t* rng,
                                   void* dx, void* dresidual, float* dw, float* db, void* workspace,
                                   size_t workspace_bytes, int64_t T, int32_t H, int32_t D, int32_t dtype, double p,
                                   float eps, void* stream) {
    using namespace ssmp;
    if (const int st = ln_check(T, H, D, dtype)) return st;
    if ((dw || db) && ln_dw_over(H, D)) return SSMP_ERR_SHAPE;
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
    const int64_t blocks = ln_blocks(a.rows, H, D, ln_two(dtype == SSMP_BF16, true, sums), kLnBwdBlocks, kLnBwdRows);
    a.wide = ln_wide(a.rows, blocks, D);
    const auto launch = [&](auto dw) {
        constexpr bool DW = decltype(dw)::value;
        if (dtype == SSMP_F32) launch_ln_bwd<float, DW>(a, blocks, s);
        else launch_ln_bwd<uint16_t, DW>(a, blocks, s);
    };
    if (sums) launch(std::true_type{});
    else launch(std::false_type{});
    SSMP_LAUNCH_CHECK();
    if (sums) {
        const unsigned n = (unsigned)((int64_t)H * ((2 * D + 31) / 32));
        const int64_t groups = blocks * ln_groups(D, 0);
        if (a.wide) k_layer_norm_dw<double><<<n, kLnDwThreads, 0, s>>>(a, groups);
        else k_layer_norm_dw<float><<<n, kLnDwThreads, 0, s>>>(a, groups);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}
