// decay_attn_pack_step: one token of linear attention with a decay for each
// row of a serving batch, on states held in a pool. Per value head, a = exp(g):
//   S' = a S + k v^T;  out = scale S'^T q
// Bound by HBM: the state (fp32, Dk x Dv per head) is read and written once
// (256 rows x 32 heads of 128 x 128: 217 us, 5.0 TB/s).
#include "state_step.h"

namespace ssmp {

struct DecayStepArgs {
    const void *q, *k, *v;
    const float* g;
    float* state;
    const int32_t* slots;
    void* out;
    int32_t B, Hk, Hv, Dk, Dv, nslots;
    int32_t gstride;  // Hv, or 0: one decay for a head
    float scale;
};

// RPG: rows of the state a thread holds (Dk <= 32 RPG). Rows of the batch that
// name the same slot are applied in their order, by the workgroups of the
// first of them (the others end at once), so a slot may be named twice.
template <typename T, int RPG>
__global__ __launch_bounds__(kStepThreads) void k_decay_step(DecayStepArgs a) {
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
    __shared__ float part[4][8][4];
    __shared__ int next;
    while (true) {
        const float decay = expf(a.g[(size_t)b * a.gstride + hv]);
        const T* const kp = static_cast<const T*>(a.k) + ((size_t)b * a.Hk + hk) * a.Dk;
        const T* const qp = static_cast<const T*>(a.q) + ((size_t)b * a.Hk + hk) * a.Dk;
        const size_t at = ((size_t)b * a.Hv + hv) * a.Dv + col;
        float v[4], r[4] = {};  // S'^T q of the four columns
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = in ? Elt<T>::ld(static_cast<const T*>(a.v), at + c) : 0.0f;
#pragma unroll
        for (int j = 0; j < RPG; ++j) {
            const int d = rg + j * kStepRowGroups;
            const float k = d < a.Dk ? Elt<T>::ld(kp, d) : 0.0f, q = d < a.Dk ? Elt<T>::ld(qp, d) : 0.0f;
            s[j].x = fmaf(k, v[0], decay * s[j].x);
            s[j].y = fmaf(k, v[1], decay * s[j].y);
            s[j].z = fmaf(k, v[2], decay * s[j].z);
            s[j].w = fmaf(k, v[3], decay * s[j].w);
            r[0] = fmaf(s[j].x, q, r[0]);
            r[1] = fmaf(s[j].y, q, r[1]);
            r[2] = fmaf(s[j].z, q, r[2]);
            r[3] = fmaf(s[j].w, q, r[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] += __shfl_xor(r[i], 8);
            r[i] += __shfl_xor(r[i], 16);
            r[i] += __shfl_xor(r[i], 32);
        }
        if (lane < 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) part[wave][lane][i] = r[i];
        if (tid == 0) next = a.B;
        __syncthreads();
        if (rg == 0 && in)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                Elt<T>::st(static_cast<T*>(a.out), at + c,
                           a.scale * ((part[0][cg][c] + part[1][cg][c]) + (part[2][cg][c] + part[3][cg][c])));
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
void launch_decay_step(const DecayStepArgs& a, hipStream_t s) {
    const unsigned blocks = (unsigned)((int64_t)a.B * a.Hv * ((a.Dv + kStepCols - 1) / kStepCols));
    switch ((a.Dk + kStepRowGroups - 1) / kStepRowGroups) {
        case 1: k_decay_step<T, 1><<<blocks, kStepThreads, 0, s>>>(a); break;
        case 2: k_decay_step<T, 2><<<blocks, kStepThreads, 0, s>>>(a); break;
        case 3: k_decay_step<T, 3><<<blocks, kStepThreads, 0, s>>>(a); break;
        default: k_decay_step<T, 4><<<blocks, kStepThreads, 0, s>>>(a); break;
    }
}

}  // namespace ssmp

extern "C" int decay_attn_pack_step(const void* q, const void* k, const void* v, const float* g, float* state,
                                    const int32_t* slots, void* out, int32_t B, int32_t nslots, int32_t Hk,
                                    int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, int32_t per_token, float scale,
                                    void* stream) {
    using namespace ssmp;
    if (B < 0 || nslots < 0 || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1 || Hv % Hk) return SSMP_ERR_SHAPE;
    if (!slots && B > nslots) return SSMP_ERR_SHAPE;
    if (Hv > 65536 || Dv > 65536 || (int64_t)B * Hv * ((Dv + kStepCols - 1) / kStepCols) >= kMaxBlocks)
        return SSMP_ERR_SHAPE;
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    if (Dk % 8 || Dv % 8 || Dk > kStepMaxDk) return SSMP_ERR_UNSUPPORTED;
    if (B == 0) return SSMP_OK;
    if (!q || !k || !v || !g || !state || !out) return SSMP_ERR_NULL;
    if (!aligned16(q, k, v, state, out)) return SSMP_ERR_ALIGN;
    const DecayStepArgs a = {q, k, v, g, state, slots, out, B, Hk, Hv, Dk, Dv, nslots, per_token ? Hv : 0, scale};
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SSMP_F32) launch_decay_step<float>(a, s);
    else launch_decay_step<uint16_t>(a, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
