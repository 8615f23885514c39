// gated_delta_pack_fwd: the gated delta rule over packed sequences. Per value
// head with its key head, and a_t = exp(g_t),
//   E_t = v_t - (a_t S_{t-1})^T k_t,  U_t = beta_t E_t,
//   S_t = a_t S_{t-1} + k_t U_t^T,    out_t = scale S_t^T q_t.
// In chunks of 64 tokens, with G the running sum of g in the chunk, S the
// state that enters it and D_ij = e^{G_i - G_j},
//   (I + L diag(beta)) E = X,  X = V - diag(e^G) K S,  L = D . K K^T below the diagonal,
//   out = scale (diag(e^G) Q S + P U),                 P = D . Q K^T on and below it,
//   S'  = e^{G_last} S + (diag(e^{G_last - G}) K)^T U.
// What does not depend on the state (the inverse, P, the decays) is made
// for all chunks at once by k_delta_prepare; k_delta_chain then goes along
// each sequence's chunks with the state in registers.
#include "delta_prepare.h"

namespace ssmp {

// One workgroup per (sequence, value head, 64 or 128 columns of the state), 16
// columns a wave. Columns do not meet in the chain, and a wave's results are
// its next right operands in the registers they are in (kplace), so the waves
// share nothing but the left operands: of one chunk in LDS, the next one's on
// their way there, and those of the one after it under way in registers.
// kKeep: keep S and E for the backward. kSum: the first walk over the parts of
// split sequences (split_chunks), whose last columns are A's.
// Bound by what a SIMD can issue: a wave's chunk (heads of 128, bf16) is 216
// matrix instructions of 16 cycles, and the rest of its 10000 cycles in
// splitting fp32 values into planes, reading LDS, storing, and the latency of
// each upon the last. One prompt of 513 tokens x 32 heads takes 46 us; a long
// chain 4.4 a chunk, 4.7 keeping S and E (with every CU at work, eight waves on
// each and the clock lower, 7.4 and 10.5); 32768 tokens x 32 heads 480 to 500 us,
// 670 to 690 keeping.
enum ChainMode { kPlain, kKeep, kSum };
template <typename T, int DKP, int NW, ChainMode MODE>
__global__ __launch_bounds__(NW * 64) void k_delta_chain(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    constexpr bool SAVE = MODE == kKeep, SUM = MODE == kSum;
    constexpr int MT = DKP / 16;  // 16-row tiles of the state
    using Loads = ChainLoads<T, DKP, NW * 64>;
    constexpr int SETS = kSets<typename Loads::Tiles, DKP, NW>;
    __shared__ alignas(16) typename Loads::Tiles sets[SETS];
    constexpr int kCols = NW * kWaveCols;
    const int ncb = SUM ? (joint_b(a.Dv) + DKP) / kCols : (a.Dv + kCols - 1) / kCols, group = a.Hv / a.Hk;
    const Spread sp = spread(blockIdx.x, ncb * group);
    const bool split = SUM || (NW == 4 && a.split);
    if (sp.group >= (split ? split_parts(a) : (int64_t)a.nseq) * a.Hk) return;
    const int hk = (int)(sp.group % a.Hk);
    Walk q;
    if (!walk_at<NW == 4>(a, sp.group / a.Hk, q) || (SUM && q.last)) return;
    const int hv = hk * group + sp.member / ncb, cb = sp.member % ncb;
    const int wave = wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    const int col = cb * kCols + wave * 16 + l16;
    const int chunks = (q.len + kC - 1) / kC;
    const Column cs = column_of<float>(1, a.Dv, col), cv = column_of<T>(a.Hv, a.Dv, col);
    const size_t state = ((size_t)q.seq * a.Hv + hv) * a.Dk * a.Dv;
    const int width = joint_b(a.Dv) + DKP;
    float* const joint = a.joint + ((size_t)q.part * a.Hv + hv) * DKP * width;
    f32x4 S[MT];
    if constexpr (SUM) unit_state<DKP>(S, col - joint_b(a.Dv));
    else if (split) load_state(joint, DKP, width, column_of<float>(1, width, col), S);
    else load_state(a.h0 ? a.h0 + state : nullptr, a.Dk, a.Dv, cs, S);
    Loads next;
    uint32_t v[16];
    ChainAt<T> at(a, q.slot0, q.start, hk, hv);
    const size_t vrow = ((size_t)q.start * a.Hv + hv) * a.Dv;
    const T* vp = static_cast<const T*>(a.v) + vrow;
    T* op = static_cast<T*>(a.out) + vrow;
    const int64_t vstep = (int64_t)kC * a.Hv * a.Dv;
    // tokens of the i-th chunk from here on, none behind the last
    const auto tokens = [&](int ch) { return min(q.len - ch * kC, kC); };
    next.load_rows(a, at, tokens(0));
    next.load_rest(a, at, tokens(0));
    load_column<T>(vp, tokens(0), a.Hv, a.Dv, cv, v);
    next.put_rows(sets[0]);
    next.put_rest(sets[0]);
    at.step(a, 1);
    next.load_rows(a, at, tokens(1));
    next.load_rest(a, at, tokens(1));
    __syncthreads();
    for (int ch = 0; ch < chunks; ++ch) {
        const size_t sh = (size_t)(q.slot0 + ch) * a.Hv + hv;
        const typename Loads::Tiles& lds = sets[SETS == 2 ? ch & 1 : 0];
        typename Loads::Tiles& other = sets[SETS == 2 ? (ch & 1) ^ 1 : 0];
        if constexpr (SAVE) store_kept(a.S0 + sh * DKP * kept_cols(a.Dv), a.Dv, col, S);
        f32x4 x[4] = {}, o[4] = {};  // K S and Q S
        Frag<3> sb = split_tiles<3>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < DKP / 32; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            Frag<NX> ka[4], qa[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                ka[m] = lds.k.frag(m * 16 + l16, s * 4 + l4);
                qa[m] = lds.q.frag(m * 16 + l16, s * 4 + l4);
            }
            Frag<3> nb;
            if (s + 1 < DKP / 32) nb = split_tiles<3>(S[2 * s + 2], S[2 * s + 3]);
            mma_tiles<3, 0, 4>(x, ka, sb);
            if constexpr (!SUM) mma_tiles<3, 0, 4>(o, qa, sb);
            if constexpr (NX == 1 && !SUM) step_order<8, 24, 3>();
            sb = nb;
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 eg = *reinterpret_cast<const f32x4*>(lds.eg + m * 16 + l4 * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[m][r] = fmaf(-eg[r], x[m][r], Elt<T>::cvt(v[m * 4 + r]));
                o[m][r] *= eg[r];
            }
        }
        vp += vstep;
        load_column<T>(vp, tokens(ch + 1), a.Hv, a.Dv, cv, v);
        // E = inverse X; in its shadow the state decays
        f32x4 E[4] = {};
        const float ec = lds.eg[kC - 1];
        {
            Frag<3> ia[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) ia[m] = tri_frag<3>(lds.inv, m * 16 + l16, l4);
            const auto xb = split_tiles<3>(x[0], x[1]);
            __builtin_amdgcn_sched_barrier(0);
            const auto xc = split_tiles<3>(x[2], x[3]);
            mma_tiles<3, 0, 4>(E, ia, xb);
            step_order<0, 24, 2>();
            __builtin_amdgcn_sched_barrier(0);
            Frag<3> ib[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) ib[m] = tri_frag<3>(lds.inv, 64 + m * 16 + l16, l4);
            mma_tiles<3, 2, 4>(E, ib, xc);
#pragma unroll
            for (int m = 0; m < MT; ++m) S[m] *= ec;
            step_order<6, 12, 3>();
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (SAVE) store_kept(a.E + sh * kC * kept_cols(a.Dv), a.Dv, col, E);
        f32x4 w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 be = *reinterpret_cast<const f32x4*>(lds.beta + m * 16 + l4 * 4);
            const f32x4 el = *reinterpret_cast<const f32x4*>(lds.el + m * 16 + l4 * 4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                E[m][r] *= be[r];  // U
                w[m][r] = el[r] * E[m][r];
            }
        }
        // S += K^T W, out += P U
        Frag<3> wb = split_tiles<3>(w[0], w[1]);
        Frag<3> ub = split_tiles<3>(E[0], E[1]);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            Frag<NX> ka[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) ka[m] = lds.k.token_frag(l, s, m);
            Frag<3> wn;
            Frag<3> un;
            if (s == 0) {
                wn = split_tiles<3>(w[2], w[3]);
                un = split_tiles<3>(E[2], E[3]);
            }
            if constexpr (SETS == 2) {  // the next chunk's operands
                if (s == 0) next.put_rows(other);
                else next.put_rest(other);
            }
            mma_tiles<3, 0, MT>(S, ka, wb);
            if constexpr (NX == 1) step_order<2 * MT, 3 * MT, 3>();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!SUM) {
                Frag<3> pa[4];
#pragma unroll
                for (int m = 2 * s; m < 4; ++m) pa[m - 2 * s] = tri_frag<3>(lds.att, s * 32 + m * 16 + l16, l4);
                if (s == 0) mma_tiles<3, 0, 4>(o, pa, ub);
                else mma_tiles<3, 2, 4>(o, pa, ub);
            }
            wb = wn;
            ub = un;
        }
        if constexpr (SETS == 1) {
            __syncthreads();  // this chunk's operands have been read
            next.put_rows(other);
            next.put_rest(other);
        }
        at.step(a, 1);
        next.load_rows(a, at, tokens(ch + 2));
        if constexpr (!SUM) store_column<T>(op, tokens(ch), a.Hv, a.Dv, cv, o, a.scale);
        op += vstep;
        next.load_rest(a, at, tokens(ch + 2));
        __syncthreads();
    }
    if constexpr (SUM) store_state(joint, DKP, width, column_of<float>(1, width, col), S);
    else if (a.hT && q.last) store_state(a.hT + state, a.Dk, a.Dv, cs, S);
}

template <typename T, int DKP, ChainMode MODE>
void launch_delta_chain(const DeltaArgs& a, int waves, hipStream_t s) {
    if constexpr (kWide<T, DKP>)
        if (waves == 8) {
            k_delta_chain<T, DKP, 8, MODE><<<chain_blocks(a, 8), 512, 0, s>>>(a);
            return;
        }
    k_delta_chain<T, DKP, 4, MODE><<<chain_blocks(a, 4), 256, 0, s>>>(a);
}

template <typename T, int DKP>
int launch_delta_fwd(DeltaArgs a, hipStream_t s) {
    const int waves = chain_waves<T, DKP>(a);
    if (!chain_ordered(a, waves)) a.order = nullptr;
    if (a.T > 0)
        if (const int st = launch_delta_prepare<T, DKP, false>(a, s)) return st;
    if (a.split) {
        k_delta_chain<T, DKP, 4, kSum><<<split_blocks(a, DKP), 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
        launch_delta_join<DKP, false>(a, a.h0, a.hT, s);
        SSMP_LAUNCH_CHECK();
    }
    if (a.S0) launch_delta_chain<T, DKP, kKeep>(a, waves, s);
    else launch_delta_chain<T, DKP, kPlain>(a, waves, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

struct DeltaFwdLayout {
    size_t dec, inv, att, order, joint, total;
};
inline DeltaFwdLayout delta_fwd_layout(int64_t T, int32_t nseq, int32_t Hv, int32_t Dk, int32_t Dv) {
    const size_t n = (size_t)delta_slots(T, nseq);
    DeltaFwdLayout L;
    L.dec = 0;
    L.inv = L.dec + round256(n * Hv * kDec * 4);
    L.att = L.inv + round256(n * Hv * kTri * 4);
    L.order = L.att + round256(n * Hv * kTri * 4);
    L.joint = L.order + round256((size_t)nseq * 4);
    L.total = L.joint + joint_bytes(T, nseq, Hv, delta_dkp(Dk), Dv);
    return L;
}

}  // namespace ssmp

extern "C" size_t gated_delta_pack_saved_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                               int32_t Dv) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, SSMP_F32) || T == 0) return 0;
    return kept_bytes(T, nseq, Hv, delta_dkp(Dk), Dv) + kept_bytes(T, nseq, Hv, kC, Dv);
}

extern "C" size_t gated_delta_pack_fwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                     int32_t Dv, int32_t dtype) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype) || T == 0) return 0;
    return delta_fwd_layout(T, nseq, Hv, Dk, Dv).total;
}

extern "C" int gated_delta_pack_fwd(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                    const int32_t* cu_seqlens, int32_t nseq, void* out, int64_t T, int32_t Hk,
                                    int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, float scale,
                                    const float* initial_state, float* final_state, void* saved, size_t saved_bytes,
                                    void* scratch, size_t scratch_bytes, void* stream) {
    using namespace ssmp;
    if (const int st = delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    if (!cu_seqlens) return SSMP_ERR_NULL;
    if (T > 0 && (!q || !k || !v || !g || !beta || !out)) return SSMP_ERR_NULL;
    if (!aligned16(q, k, v, out, initial_state, final_state, saved, scratch)) return SSMP_ERR_ALIGN;
    if (T > 0 && (!scratch || scratch_bytes < gated_delta_pack_fwd_scratch_bytes(T, nseq, Hk, Hv, Dk, Dv, dtype)))
        return SSMP_ERR_WORKSPACE;
    if (T > 0 && saved && saved_bytes < gated_delta_pack_saved_bytes(T, nseq, Hk, Hv, Dk, Dv))
        return SSMP_ERR_WORKSPACE;
    if (T == 0 && !final_state) return SSMP_OK;
    const DeltaFwdLayout L = delta_fwd_layout(T, nseq, Hv, Dk, Dv);
    char* const ws = static_cast<char*>(scratch);
    DeltaArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
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
    a.scale = scale;
    if (T > 0) {
        a.dec = reinterpret_cast<float*>(ws + L.dec);
        a.inv = reinterpret_cast<float*>(ws + L.inv);
        a.att = reinterpret_cast<float*>(ws + L.att);
        a.order = reinterpret_cast<int32_t*>(ws + L.order);
        a.joint = reinterpret_cast<float*>(ws + L.joint);
        a.split = split_chunks(T, nseq, Hv, Dv);
        if (saved) {
            a.S0 = static_cast<float*>(saved);
            a.E = reinterpret_cast<float*>(static_cast<char*>(saved) +
                                           kept_bytes(T, nseq, Hv, delta_dkp(Dk), Dv));
        }
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wide = Dk > 64;
    if (dtype == SSMP_F32) return wide ? launch_delta_fwd<float, 128>(a, s) : launch_delta_fwd<float, 64>(a, s);
    return wide ? launch_delta_fwd<uint16_t, 128>(a, s) : launch_delta_fwd<uint16_t, 64>(a, s);
}
