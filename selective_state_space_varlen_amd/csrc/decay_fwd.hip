// decay_attn_pack_fwd: linear attention with a decay for each head over packed
// sequences.
#include "decay_walk.h"

extern "C" size_t decay_attn_pack_fwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                    int32_t Dv) {
    using namespace ssmp;
    if (decay_check(T, nseq, Hk, Hv, Dk, Dv, SSMP_F32)) return 0;
    return decay_joint(T, Hv, Dk, Dv, (int64_t)Hv * decay_col_blocks(Dv)).total;
}

extern "C" int decay_attn_pack_fwd(const void* q, const void* k, const void* v, const float* g,
                                   const int32_t* cu_seqlens, int32_t nseq, void* out, int64_t T, int32_t Hk,
                                   int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, int32_t per_token, float scale,
                                   const float* initial_state, float* final_state, void* scratch,
                                   size_t scratch_bytes, void* stream) {
    using namespace ssmp;
    if (const int st = decay_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    if (initial_state && initial_state == final_state) return SSMP_ERR_UNSUPPORTED;  // segments of a sequence start from the one while the last writes the other
    if (!cu_seqlens) return SSMP_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !out)) return SSMP_ERR_NULL;
    if (!aligned16(q, k, v, out, initial_state, final_state, scratch)) return SSMP_ERR_ALIGN;
    const size_t need = decay_attn_pack_fwd_scratch_bytes(T, nseq, Hk, Hv, Dk, Dv);
    if (need && (!scratch || scratch_bytes < need)) return SSMP_ERR_WORKSPACE;
    if (T == 0 && !final_state) return SSMP_OK;
    const int64_t work = (int64_t)Hv * decay_col_blocks(Dv);
    const DecayJoint L = decay_joint(T, Hv, Dk, Dv, work);
    DecayArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
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
    a.gstride = per_token ? Hv : 0;
    a.scale = scale;
    a.slices = 1;
    a.seg = decay_segment(T, nseq, work);
    a.few = T / a.seg <= kFewStates;
    if (need) {
        a.joint[0] = reinterpret_cast<float*>(static_cast<char*>(scratch) + L.joint);
        a.seg_decay[0] = reinterpret_cast<float*>(static_cast<char*>(scratch) + L.decay);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T > a.seg) {
        if (const int st = launch_decay_walk<kSumS, false>(a, dtype, s)) return st;
        if (const int st = launch_decay_join(a, 1, s)) return st;
    }
    return launch_decay_walk<kOut, false>(a, dtype, s);
}
