// decay_attn_pack_bwd: gradients of linear attention with a decay for each
// head. Nothing is kept from the forward: dq's walk forms the states again as
// it goes, and those between segments are summed again.
#include "decay_walk.h"

namespace ssmp {

// exp(g) in 32 bits without its smallest numbers, as the walks form it
__device__ __forceinline__ bool decay_is_zero(float g) { return g * kLog2e < -126.0f; }

// dg of one piece of kPiece tokens, a wave for 64 / kDgChunks heads, a lane
// for one chunk of a head: back from the anchor at the chunk's end, d g_t =
// d g_{t+1} + q_t.dq_t - k_t.dk_t, in 64 bits. Where a token's decay is zero,
// so is its gradient, and the sum starts again.
constexpr int kDgChunks = kPiece / kC, kDgHeads = 64 / kDgChunks;
__global__ __launch_bounds__(64) void k_decay_dg(DecayArgs p, int parts) {
    const int hb = (p.Hv + kDgHeads - 1) / kDgHeads;
    const int64_t slot = blockIdx.x / hb;
    const int hv = blockIdx.x % hb * kDgHeads + threadIdx.x % kDgHeads, ch = threadIdx.x / kDgHeads;
    Chunk c;
    const bool any = chunk_at(p.cu, p.nseq, p.T, slot, c, kPiece) && hv < p.Hv;
    const int n = any ? min(c.n - ch * kC, kC) : 0;  // tokens of this lane's chunk
    const int64_t t0 = c.start + ch * kC;
    double acc = 0.0, sum = 0.0, cross = 0.0;  // cross: what goes through the chunk's states
    if (n > 0) {
        if (!c.last || p.dhT)
            for (int i = 0; i < parts; ++i) acc += p.meet[((size_t)slot * p.Hv + hv) * parts + i];
        const int64_t first = c.start - c.index * kPiece, chunk = first / kC + c.seq + c.index * kDgChunks + ch;
        for (int i = 0; i < parts; ++i) {
            const size_t at = ((size_t)chunk * p.Hv + hv) * parts + i;
            cross += p.chunk[0][at] - p.chunk[1][at];
        }
    }
    // the anchor at this chunk's end: that of the piece's, and what crosses the chunks between
    double behind = cross;
#pragma unroll
    for (int d = kDgHeads; d < 64; d *= 2) {
        const double v = __shfl_down(behind, d);
        behind += threadIdx.x + d < 64 ? v : 0.0;
    }
    acc += behind - cross;
    constexpr int kBatch = 32;  // tokens' loads under way
    for (int t1 = n; t1 > 0; t1 -= kBatch) {
        double r[kBatch];
        float g[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int t = t1 - 1 - x;
            const size_t at = (size_t)(t0 + (t < 0 ? 0 : t)) * p.Hv + hv;
            r[x] = (double)p.rows[0][at] - (double)p.rows[1][at];
            g[x] = p.g[p.gstride ? at : hv];
        }
        for (int i = 1; i < parts; ++i)
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                const int t = t1 - 1 - x;
                const size_t at = ((size_t)i * p.T + t0 + (t < 0 ? 0 : t)) * p.Hv + hv;
                r[x] += (double)p.rows[0][at] - (double)p.rows[1][at];
            }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
            const int t = t1 - 1 - x;
            if (t < 0) continue;
            acc += r[x];
            if (decay_is_zero(g[x])) acc = 0.0;
            if (p.gstride) p.dg[(size_t)(t0 + t) * p.Hv + hv] = (float)acc;
            sum += acc;
        }
    }
    if (!p.gstride) {
        for (int d = kDgHeads; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        if (threadIdx.x < kDgHeads && hv < p.Hv) p.dgsum[(size_t)slot * p.Hv + hv] = sum;
    }
}

// one decay for a head: its gradient, in a fixed order
__global__ __launch_bounds__(64) void k_decay_dg_sum(DecayArgs p, int64_t slots) {
    const int hv = blockIdx.x, lane = threadIdx.x;
    double s = 0.0;
    for (int64_t i = lane; i < slots; i += 64) s += p.dgsum[(size_t)i * p.Hv + hv];
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
    if (lane == 0) p.dg[hv] = (float)s;
}

// dq and dk: the sums of their parts by value head and slice, up to the last sequence's end
template <typename T>
__global__ __launch_bounds__(256) void k_decay_add(DecayArgs p, int members) {
    const float* __restrict__ const part = p.part[blockIdx.y];
    T* const out = static_cast<T*>(blockIdx.y ? p.dk : p.dq);
    int64_t end = p.cu[p.nseq];
    end = end < 0 ? 0 : end > p.T ? p.T : end;
    const int per = p.Dk / 4;
    const int64_t n = end * p.Hk * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const float* at = part + (i / per) * members * (int64_t)p.Dk + i % per * 4;
        f32x4 s = {0, 0, 0, 0};
        for (int m = 0; m < members; ++m) s += *reinterpret_cast<const f32x4*>(at + (int64_t)m * p.Dk);
#pragma unroll
        for (int x = 0; x < 4; ++x) Elt<T>::st(out, (size_t)i * 4 + x, s[x]);
    }
}

struct DecayBwdLayout {
    size_t joint[2], decay[2], part[2], rows[2], chunk[2], snap, meet, dgsum, total;
};
inline DecayBwdLayout decay_bwd_layout(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv) {
    DecayBwdLayout L;
    const size_t slices = (Dv + kDecayMaxDb - 1) / kDecayMaxDb, parts = slices * (Dk > 64 ? 2 : 1);
    const DecayJoint j = decay_joint(T, Hv, Dk, Dv, Hv);
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        const size_t here = take(j.total);
        L.joint[i] = here + j.joint;
        L.decay[i] = here + j.decay;
    }
    const bool partial = (size_t)(Hv / Hk) * slices > 1;
    for (int i = 0; i < 2; ++i) L.part[i] = take(partial ? (size_t)T * Hv * slices * Dk * sizeof(float) : 0);
    for (int i = 0; i < 2; ++i) L.rows[i] = take(parts * T * Hv * sizeof(float));
    for (int i = 0; i < 2; ++i) L.chunk[i] = take((size_t)delta_slots(T, nseq) * Hv * parts * sizeof(double));
    const size_t db = Dv > 64 ? 128 : 64, dc = Dk > 64 ? 128 : 64;
    L.snap = take((size_t)(T / kPiece) * Hv * slices * db * dc * sizeof(float));
    L.meet = take((size_t)(T / kPiece + nseq) * Hv * parts * sizeof(double));
    L.dgsum = take((size_t)(T / kPiece + nseq) * Hv * sizeof(double));
    L.total = at;
    return L;
}

}  // namespace ssmp

extern "C" size_t decay_attn_pack_bwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                    int32_t Dv) {
    using namespace ssmp;
    if (decay_check(T, nseq, Hk, Hv, Dk, Dv, SSMP_F32) || T == 0) return 0;
    return decay_bwd_layout(T, nseq, Hk, Hv, Dk, Dv).total;
}

extern "C" int decay_attn_pack_bwd(const void* q, const void* k, const void* v, const float* g,
                                   const int32_t* cu_seqlens, int32_t nseq, const void* dout, int64_t T, int32_t Hk,
                                   int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, int32_t per_token, float scale,
                                   const float* initial_state, const float* dfinal_state, float* dinitial_state,
                                   void* dq, void* dk, void* dv, float* dg, void* scratch, size_t scratch_bytes,
                                   void* stream) {
    using namespace ssmp;
    if (const int st = decay_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    if (dinitial_state && (dinitial_state == initial_state || dinitial_state == dfinal_state)) return SSMP_ERR_UNSUPPORTED;  // segments of a sequence start from the one while the first writes the other
    if (!cu_seqlens) return SSMP_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !dout || !dq || !dk || !dv)) return SSMP_ERR_NULL;
    if (!aligned16(q, k, v, dout, dq, dk, dv, initial_state, dfinal_state, dinitial_state, scratch))
        return SSMP_ERR_ALIGN;
    if (T > 0 && (!scratch || scratch_bytes < decay_attn_pack_bwd_scratch_bytes(T, nseq, Hk, Hv, Dk, Dv)))
        return SSMP_ERR_WORKSPACE;
    hipStream_t s = static_cast<hipStream_t>(stream);
    DecayArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.dout = dout;
    a.g = g;
    a.cu = cu_seqlens;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dg = dg;
    a.h0 = initial_state;
    a.dhT = dfinal_state;
    a.dh0 = dinitial_state;
    a.T = T;
    a.nseq = nseq;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dk = Dk;
    a.Dv = Dv;
    a.gstride = per_token ? Hv : 0;
    a.scale = scale;
    a.slices = (Dv + kDecayMaxDb - 1) / kDecayMaxDb;
    a.seg = decay_segment(T, nseq, Hv);
    a.few = T / a.seg <= kFewStates;
    a.heads = decay_heads_of(a, dtype);
    if (T == 0) {
        if (!per_token)
            if (const int st = zero_f32(dg, Hv, s)) return st;
        a.dg = nullptr;
        return dinitial_state ? launch_decay_dkv(a, dtype, s) : SSMP_OK;  // hands on dfinal_state
    }
    const DecayBwdLayout L = decay_bwd_layout(T, nseq, Hk, Hv, Dk, Dv);
    char* const ws = static_cast<char*>(scratch);
    for (int i = 0; i < 2; ++i) {
        a.joint[i] = reinterpret_cast<float*>(ws + L.joint[i]);
        a.seg_decay[i] = reinterpret_cast<float*>(ws + L.decay[i]);
        a.part[i] = reinterpret_cast<float*>(ws + L.part[i]);
        a.rows[i] = reinterpret_cast<float*>(ws + L.rows[i]);
        a.chunk[i] = reinterpret_cast<double*>(ws + L.chunk[i]);
    }
    a.snap = reinterpret_cast<float*>(ws + L.snap);
    a.meet = reinterpret_cast<double*>(ws + L.meet);
    a.dgsum = reinterpret_cast<double*>(ws + L.dgsum);
    if (T > a.seg) {
        if (const int st = launch_decay_pair<kSumS, false, kSumD>(a, dtype, s)) return st;
        if (const int st = launch_decay_join(a, 2, s)) return st;
    }
    if (const int st = launch_decay_dq(a, dtype, s)) return st;
    if (const int st = launch_decay_dkv(a, dtype, s)) return st;
    if (dg) {
        const int64_t slots = T / kPiece + nseq;
        k_decay_dg<<<(unsigned)(slots * ((Hv + kDgHeads - 1) / kDgHeads)), 64, 0, s>>>(a, a.slices * decay_blocks_of(Dv, Dk, dtype));
        SSMP_LAUNCH_CHECK();
        if (!per_token) {
            k_decay_dg_sum<<<(unsigned)Hv, 64, 0, s>>>(a, slots);
            SSMP_LAUNCH_CHECK();
        }
    }
    const int members = Hv / Hk / a.heads * a.slices;
    if (members > 1) {
        const int64_t want = (T * Hk * (Dk / 4) + 255) / 256;
        const dim3 blocks((unsigned)(want < 8192 ? want : 8192), 2);
        if (dtype == SSMP_F32) k_decay_add<float><<<blocks, 256, 0, s>>>(a, members);
        else k_decay_add<uint16_t><<<blocks, 256, 0, s>>>(a, members);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}
