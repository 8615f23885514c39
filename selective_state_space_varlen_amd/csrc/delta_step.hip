// gated_delta_pack_step: one token of the gated delta rule for each row of a
// serving batch, on states held in a pool. Per value head, a = exp(g):
//   e = v - (a S)^T k;  S' = a S + beta k e^T;  out = scale S'^T q
//                                                   = scale (a S^T q + beta (q.k) e)
// so one pass over S gives S^T k and S^T q, one barrier joins them, and the
// state is written back from registers.
//
// Bound by HBM: the state (fp32, Dk x Dv per head) is read and written once.
// A workgroup takes 32 columns of one head's state, eight lanes of 16 bytes to
// a row (one 128-byte line): 4 workgroups a head at Dv = 128, so that a single
// sequence of 32 heads already has 128 of them.
#include "delta_common.h"

namespace ssmp {

constexpr int kStepCols = 32;
constexpr int kStepThreads = 256;
constexpr int kStepRowGroups = kStepThreads / (kStepCols / 4);  // 32
constexpr int kStepMaxDk = 128;

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float* state;
    const int32_t* slots;
    void* out;
    int32_t B, Hk, Hv, Dk, Dv, nslots;
    float scale;
};

// The state passes once each way and would push everything else out of the
// caches: without temporal hint 246 us for 256 sequences of 32 heads of
// 128 x 128, with it 211 (5.1 TB/s); the same 4.7 us for one sequence.
__device__ __forceinline__ float4 state_load(const float* p) {
    const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    return make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void state_store(float* p, float4 v) {
    __builtin_nontemporal_store(f32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<f32x4*>(p));
}

// RPG: rows of the state a thread holds (Dk <= 32 RPG). Rows of the batch that
// name the same slot are applied in their order, by the workgroups of the
// first of them (the others end at once), so a slot may be named twice.
template <typename T, int RPG>
__global__ __launch_bounds__(kStepThreads) void k_delta_step(StepArgs a) {
    const int ncb = (a.Dv + kStepCols - 1) / kStepCols;
    const int cb = blockIdx.x % ncb, hv = (blockIdx.x / ncb) % a.Hv;
    int b = blockIdx.x / (ncb * a.Hv);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int cg = tid & 7, rg = tid >> 3;
    const int col = cb * kStepCols + cg * 4;
    const bool in = col < a.Dv;
    const int hk = hv / (a.Hv / a.Hk);
    const int slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.nslots) return;
    float* const S = a.state + ((size_t)slot * a.Hv + hv) * a.Dk * a.Dv;
    float4 s[RPG];
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
        const int d = rg + j * kStepRowGroups;
        s[j] = in && d < a.Dk ? state_load(S + (size_t)d * a.Dv + col) : make_float4(0, 0, 0, 0);
    }
    if (a.slots) {
        int earlier = 0;
        for (int i = tid; i < b; i += kStepThreads) earlier |= a.slots[i] == slot;
        if (__syncthreads_or(earlier)) return;
    }
    __shared__ float part[4][8][9];
    __shared__ int next;
    while (true) {
        const float decay = expf(a.g[(size_t)b * a.Hv + hv]), beta = a.beta[(size_t)b * a.Hv + hv];
        const T* const kp = static_cast<const T*>(a.k) + ((size_t)b * a.Hk + hk) * a.Dk;
        const T* const qp = static_cast<const T*>(a.q) + ((size_t)b * a.Hk + hk) * a.Dk;
        float k[RPG], r[9] = {};  // S^T k and S^T q of the four columns, q.k
#pragma unroll
        for (int j = 0; j < RPG; ++j) {
            const int d = rg + j * kStepRowGroups;
            k[j] = d < a.Dk ? Elt<T>::ld(kp, d) : 0.0f;
            const float q = d < a.Dk ? Elt<T>::ld(qp, d) : 0.0f;
            const float sv[4] = {s[j].x, s[j].y, s[j].z, s[j].w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                r[c] = fmaf(sv[c], k[j], r[c]);
                r[4 + c] = fmaf(sv[c], q, r[4 + c]);
            }
            r[8] = fmaf(q, k[j], r[8]);
        }
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            r[i] += __shfl_xor(r[i], 8);
            r[i] += __shfl_xor(r[i], 16);
            r[i] += __shfl_xor(r[i], 32);
        }
        if (lane < 8)
#pragma unroll
            for (int i = 0; i < 9; ++i) part[wave][lane][i] = r[i];
        if (tid == 0) next = a.B;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 9; ++i) r[i] = (part[0][cg][i] + part[1][cg][i]) + (part[2][cg][i] + part[3][cg][i]);
        const size_t at = ((size_t)b * a.Hv + hv) * a.Dv + col;
        float u[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float v = in ? Elt<T>::ld(static_cast<const T*>(a.v), at + c) : 0.0f;
            u[c] = beta * fmaf(-decay, r[c], v);
        }
        if (rg == 0 && in)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                Elt<T>::st(static_cast<T*>(a.out), at + c, a.scale * fmaf(decay, r[4 + c], r[8] * u[c]));
#pragma unroll
        for (int j = 0; j < RPG; ++j) {
            s[j].x = fmaf(k[j], u[0], decay * s[j].x);
            s[j].y = fmaf(k[j], u[1], decay * s[j].y);
            s[j].z = fmaf(k[j], u[2], decay * s[j].z);
            s[j].w = fmaf(k[j], u[3], decay * s[j].w);
        }
        if (!a.slots) break;
        int mine = a.B;
        for (int i = b + 1 + tid; i < a.B && mine == a.B; i += kStepThreads)
            if (a.slots[i] == slot) mine = i;
        if (mine < a.B) atomicMin(&next, mine);
        __syncthreads();
        b = next;
        if (b >= a.B) break;
        __syncthreads();  // everyone has read `next` and `part` before they are written again
    }
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
        const int d = rg + j * kStepRowGroups;
        if (in && d < a.Dk) state_store(S + (size_t)d * a.Dv + col, s[j]);
    }
}

template <typename T>
void launch_step(const StepArgs& a, hipStream_t s) {
    const unsigned blocks = (unsigned)((int64_t)a.B * a.Hv * ((a.Dv + kStepCols - 1) / kStepCols));
    switch ((a.Dk + kStepRowGroups - 1) / kStepRowGroups) {
        case 1: k_delta_step<T, 1><<<blocks, kStepThreads, 0, s>>>(a); break;
        case 2: k_delta_step<T, 2><<<blocks, kStepThreads, 0, s>>>(a); break;
        case 3: k_delta_step<T, 3><<<blocks, kStepThreads, 0, s>>>(a); break;
        default: k_delta_step<T, 4><<<blocks, kStepThreads, 0, s>>>(a); break;
    }
}

}  // namespace ssmp

extern "C" int gated_delta_pack_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                     float* state, const int32_t* slots, void* out, int32_t B, int32_t nslots,
                                     int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, float scale,
                                     void* stream) {
    using namespace ssmp;
    if (B < 0 || nslots < 0 || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1 || Hv % Hk) return SSMP_ERR_SHAPE;
    if (!slots && B > nslots) return SSMP_ERR_SHAPE;
    if (Hv > 65536 || Dv > 65536 || (int64_t)B * Hv * ((Dv + kStepCols - 1) / kStepCols) >= kMaxBlocks)
        return SSMP_ERR_SHAPE;
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    if (Dk % 8 || Dv % 8 || Dk > kStepMaxDk) return SSMP_ERR_UNSUPPORTED;
    if (B == 0) return SSMP_OK;
    if (!q || !k || !v || !g || !beta || !state || !out) return SSMP_ERR_NULL;
    if (!aligned16(q, k, v, state, out)) return SSMP_ERR_ALIGN;
    const StepArgs a = {q, k, v, g, beta, state, slots, out, B, Hk, Hv, Dk, Dv, nslots, scale};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SSMP_F32) launch_step<float>(a, s);
    else launch_step<uint16_t>(a, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
