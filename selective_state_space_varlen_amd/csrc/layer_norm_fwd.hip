// layer_norm_pack_fwd: h = residual + drop(x) and its layer norm.
#include "layer_norm.h"

namespace ssmp {

// Groups of LANES lanes take rows group, group + groups, ...: their number is a
// multiple of H, so that a group stays with one head and keeps its weights.
template <typename T, int V, int LANES, int NV, bool DROP>
__global__ __launch_bounds__(ln_threads(LANES)) void k_layer_norm_fwd(LnArgs a) {
    constexpr int SG = ln_threads(LANES) / LANES;
    __shared__ float lds[2][3][kLnWaves];
    const int lane = threadIdx.x % LANES;
    const int64_t group = (int64_t)blockIdx.x * SG + threadIdx.x / LANES, groups = (int64_t)gridDim.x * SG;
    const int head = (int)(group % a.H);
    const float* const w = a.w ? a.w + (size_t)head * a.D : nullptr;
    const float* const b = a.b ? a.b + (size_t)head * a.D : nullptr;
    float wv[NV][V], bv[NV][V];
    ln_weights<V, LANES, NV>(w, a.D, lane, 1.0f, wv);
    ln_weights<V, LANES, NV>(b, a.D, lane, 0.0f, bv);
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
        float sum[1] = {}, two[2] = {}, more;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) sum[0] += v[j][e];
        row_sums<LANES>(sum, lds[turn]);
        const float mean = sum[0] / (float)a.D;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                v[j][e] = (j * LANES + lane) * V + e < a.D ? v[j][e] - mean : 0.0f;
                two[0] += v[j][e];
                two[1] = fmaf(v[j][e], v[j][e], two[1]);
            }
        row_sums<LANES>(two, lds[turn] + 1);
        const float r = ln_root(a, two[0], two[1], more);
        turn ^= 1;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < V; ++e) v[j][e] = fmaf((v[j][e] - more) * r, wv[j][e], bv[j][e]);
        if (row < a.rows) LnRow<T, V, LANES, NV>::store(a.y, row, a.D, lane, v);
    }
}

template <typename T>
void launch_ln_fwd(const LnArgs& a, int64_t blocks, hipStream_t s) {
    ln_dispatch<ln_two(sizeof(T) == 2, false, false)>(a.D, [&](auto f) {
        constexpr int V = decltype(f)::vec, L = decltype(f)::lanes, N = decltype(f)::nv;
        const dim3 g((unsigned)blocks), b(ln_threads(L));
        if (a.drop.cut) k_layer_norm_fwd<T, V, L, N, true><<<g, b, 0, s>>>(a);
        else k_layer_norm_fwd<T, V, L, N, false><<<g, b, 0, s>>>(a);
    });
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
    const int two = ln_two(dtype == SSMP_BF16, false, false);
    const LnForm m = ln_form(D, two);
    const int64_t blocks = ln_blocks(a.rows, H, D, two, m.vec == 8 && m.lanes <= two ? kLnFwdBlocks / m.nv : kLnFwdBlocks);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SSMP_F32) launch_ln_fwd<float>(a, blocks, s);
    else launch_ln_fwd<uint16_t>(a, blocks, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
