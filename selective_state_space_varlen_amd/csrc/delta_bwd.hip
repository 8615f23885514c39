// gated_delta_pack_bwd: gradients of gated_delta_pack_fwd, chunk by chunk
// backwards. With dO' = scale dOut, dS' the gradient of the state that leaves
// the chunk, and the forward's L, P, G, U = diag(beta) E and entering state S,
//   Y = P^T dO' + diag(e^{G_last - G}) K dS',  dU = (I + diag(beta) L)^-T Y,  dE = diag(beta) dU,
//   dS = e^{G_last} dS' + (diag(e^G) Q)^T dO' - (diag(e^G) K)^T dE,
//   dv = dE,  dbeta = rows of dU . E.
// A token reads the state twice, as q (gradient dO') and as k (gradient -dE),
// and writes it once, as k. With a = D . dO' U^T and b = D . dE U^T (below the
// diagonal for b),
//   dq       =  diag(e^G) dO' S^T + a K
//   dk read  = -diag(e^G) dE S^T - b K
//   dk write =  diag(e^{G_last - G}) U dS'^T + a^T Q - b^T K
// and, since e^{G_i} scales what token i reads and e^{-G_i} what it writes,
//   dG_i = q_i.dq_i + k_i.dkread_i - k_i.dkwrite_i,  the last token's also + <dS', S'>,
//   dg_t = sum of dG_i, i >= t in the chunk.
// U_i is written through k_i alone, so k_i.dkwrite_i = U_i.dU_i = beta_i dbeta_i;
// and the sum of U_i.Y_i, taken from Y's two forms, gives
//   <dS', S'> = e^{G_last} <dS', S> + sum_i beta_i dbeta_i - (q.dq + k.dkread of a K and -b K, summed),
// so that dkwrite enters nothing but dk.
// k_delta_prepare makes what no gradient enters, k_delta_chain_bwd walks each
// sequence's chunks back with dS in registers, and k_delta_grads forms the
// chunks' gradients, all at once, from S, E, dS' and dU (k_delta_dg the last
// sums of dg).
#include "delta_prepare.h"

namespace ssmp {

// As k_delta_chain, from the last chunk to the first, with the same bound: 635
// to 655 us for 32768 tokens x 32 heads of 128 x 128 in bf16.
// SUM: the first walk over the parts of split sequences.
template <typename T, int DKP, int NW, bool SUM>
__global__ __launch_bounds__(NW * 64) void k_delta_chain_bwd(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    constexpr int MT = DKP / 16;
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
    if (!walk_at<NW == 4>(a, sp.group / a.Hk, q) || (SUM && q.first)) return;
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
    else load_state(a.dhT ? a.dhT + state : nullptr, a.Dk, a.Dv, cs, S);
    Loads next;
    uint32_t onext[16];
    // an empty sequence has no last chunk
    const int last = chunks > 0 ? chunks - 1 : 0;
    const auto tokens = [&](int ch) { return ch < 0 ? 0 : min(q.len - ch * kC, kC); };
    ChainAt<T> at(a, q.slot0 + last, q.start + (int64_t)last * kC, hk, hv);
    const T* dp = static_cast<const T*>(a.dout) + (((size_t)q.start + (size_t)last * kC) * a.Hv + hv) * a.Dv;
    const int64_t dstep = (int64_t)kC * a.Hv * a.Dv;
    next.load_rows(a, at, tokens(last));
    next.load_rest(a, at, tokens(last));
    load_column<T>(dp, tokens(last), a.Hv, a.Dv, cv, onext);
    next.put_rows(sets[0]);
    next.put_rest(sets[0]);
    at.step(a, -1);
    next.load_rows(a, at, tokens(last - 1));
    next.load_rest(a, at, tokens(last - 1));
    __syncthreads();
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const size_t sh = (size_t)(q.slot0 + ch) * a.Hv + hv;
        const int set = SETS == 2 ? (last - ch) & 1 : 0;
        const typename Loads::Tiles& lds = sets[set];
        typename Loads::Tiles& other = sets[SETS == 2 ? set ^ 1 : 0];
        f32x4 o[4];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i >> 2][i & 3] = Elt<T>::cvt(onext[i]);
        dp -= dstep;
        load_column<T>(dp, tokens(ch - 1), a.Hv, a.Dv, cv, onext);
        if constexpr (!SUM) store_kept(a.dS1 + sh * DKP * kept_cols(a.Dv), a.Dv, col, S);
        f32x4 x[4] = {}, y[4] = {};  // K dS', scale P^T dOut
        Frag<3> sb = split_tiles<3>(S[0], S[1]);
#pragma unroll
        for (int s = 0; s < DKP / 32; ++s) {
            __builtin_amdgcn_sched_barrier(0);
            Frag<NX> ka[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) ka[m] = lds.k.frag(m * 16 + l16, s * 4 + l4);
            Frag<3> nb;
            if (s + 1 < DKP / 32) nb = split_tiles<3>(S[2 * s + 2], S[2 * s + 3]);
            mma_tiles<3, 0, 4>(x, ka, sb);
            if constexpr (NX == 1) step_order<4, 12, 4>();
            sb = nb;
        }
        const float ec = lds.eg[kC - 1];
#pragma unroll
        for (int s = 0; s < 2; ++s) {  // in its shadow the state's gradient decays
            __builtin_amdgcn_sched_barrier(0);
            const auto ob = split_tiles<NX>(o[2 * s], o[2 * s + 1]);
            Frag<3> pa[4];
#pragma unroll
            for (int m = 0; m < 2 + 2 * s; ++m) pa[m] = tri_frag<3>(lds.att, (s ? 0 : 64) + m * 16 + l16, l4);
            if (s == 0) mma_tiles<3, 0, 2>(y, pa, ob);
            else mma_tiles<3, 0, 4>(y, pa, ob);
#pragma unroll
            for (int m = s * MT / 2; m < (s + 1) * MT / 2; ++m) S[m] *= ec;
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 el = *reinterpret_cast<const f32x4*>(lds.el + m * 16 + l4 * 4);
            y[m] += el * x[m];
        }
        f32x4 u[4] = {};
        {
            Frag<3> ia[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) ia[m] = tri_frag<3>(lds.inv, m * 16 + l16, l4);
            const auto yb = split_tiles<3>(y[2], y[3]);
            __builtin_amdgcn_sched_barrier(0);
            const auto yc = split_tiles<3>(y[0], y[1]);
            mma_tiles<3, 0, 4>(u, ia, yb);
            step_order<0, 24, 2>();
            __builtin_amdgcn_sched_barrier(0);
            Frag<3> ib[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) ib[m] = tri_frag<3>(lds.inv, 64 + m * 16 + l16, l4);
            mma_tiles<3, 0, 2>(u, ib, yc);
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const f32x4 eg = *reinterpret_cast<const f32x4*>(lds.eg + m * 16 + l4 * 4);
                o[m] *= eg * a.scale;  // e^G scale dOut
            }
            step_order<10, 12, 3>();
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (!SUM) store_kept(a.dU + sh * kC * kept_cols(a.Dv), a.Dv, col, u);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const f32x4 be = *reinterpret_cast<const f32x4*>(lds.beta + m * 16 + l4 * 4);
            const f32x4 eg = *reinterpret_cast<const f32x4*>(lds.eg + m * 16 + l4 * 4);
            u[m] *= -eg * be;  // -e^G dE
        }
        // dS += (e^G Q)^T scale dOut - (e^G K)^T dE
        Frag<3> rb = split_tiles<3>(o[0], o[1]);
#pragma unroll
        for (int t = 0; t < 4; ++t) {  // queries, keys of the first 32 tokens, then of the others
            const int s = t >> 1;
            __builtin_amdgcn_sched_barrier(0);
            Frag<NX> ra[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) ra[m] = t & 1 ? lds.k.token_frag(l, s, m) : lds.q.token_frag(l, s, m);
            Frag<3> rn;
            if (t == 0) rn = split_tiles<3>(u[0], u[1]);
            if (t == 1) rn = split_tiles<3>(o[2], o[3]);
            if (t == 2) rn = split_tiles<3>(u[2], u[3]);
            if constexpr (SETS == 2) {  // the next chunk's operands
                if (t == 1) next.put_rows(other);
                if (t == 2) next.put_rest(other);
            }
            mma_tiles<3, 0, MT>(S, ra, rb);
            if constexpr (NX == 1) step_order<2 * MT, 3 * MT, 2>();
            rb = rn;
        }
        if constexpr (SETS == 1) {
            __syncthreads();  // this chunk's operands have been read
            next.put_rows(other);
            next.put_rest(other);
        }
        at.step(a, -1);
        next.load_rows(a, at, tokens(ch - 2));
        next.load_rest(a, at, tokens(ch - 2));
        __syncthreads();
    }
    if constexpr (SUM) store_state(joint, DKP, width, column_of<float>(1, width, col), S);
    else if (a.dh0 && q.first) store_state(a.dh0 + state, a.Dk, a.Dv, cs, S);
}

// One workgroup per (slot, key head, 64 columns of dq and dk), over the value
// heads of the group, whose dq and dk it adds in registers. Wave w holds
// columns 16 w .. for all 64 tokens, so its rows of S and dS' come straight
// from memory, and its share of the ten tiles of a^T and b^T. It goes over
// dOut, dE, U, S and dS' 32 columns at a time, the next ones (of the next head
// too) under way in registers meanwhile. Two workgroups share a CU and fill
// each other's waits at barriers: one of eight waves with all columns of a
// head, which stages each chunk once instead of twice, took 1660 us where these
// took 1415 (32768 tokens, 32 heads of 128 x 128 on 16 key heads; 1390 now).
// That is 4.5 GB of memory's traffic at 3.2 TB/s, 60 % of what a copy reaches,
// beside the matrix instructions and the splitting, which a workgroup cannot
// put wholly in the other's waits.
// The rows of q.dq + k.dkread over these columns go to a.rows, with what the
// columns give of <dS', S'> on the last, for k_delta_dg to add up.
constexpr int kDh = 64;

// what a thread has under way of KC columns of one head
template <typename T, int KC>
struct GradLoads {
    Unit<T> o;                         // token tid / (KC / 8), 8 columns: dOut,
    Unit<float> E, dU;                 // E and dU
    Unit<float> s0[KC / 32], s1[KC / 32];  // row of S and dS' of this lane, 8 columns of each 32
    uint32_t beta, dec;                // of its token; and place tid of the chunk's decays

    // (the same loads whether there is such a head or not: n = 0 makes zeros)
    __device__ __forceinline__ void load(const DeltaArgs& a, int64_t slot, const Chunk& c, int hv, int v0, int d0, int n) {
        const int tid = fresh(threadIdx.x), l = tid & 63, t = tid / (KC / 8);
        const size_t sh = (size_t)slot * a.Hv + (n > 0 ? hv : 0);
        const size_t at = (size_t)c.start * a.Hv + (n > 0 ? hv : 0);
        const int e = v0 + (tid % (KC / 8)) * 8;
        const int dkp = delta_dkp(a.Dk), kept = kept_cols(a.Dv);
        o.load(rows_rsrc(static_cast<const T*>(a.dout) + at * a.Dv, n, a.Hv * a.Dv, a.Dv),
               e < a.Dv ? (uint32_t)(t * a.Hv * a.Dv + e) * (uint32_t)sizeof(T) : kNowhere);
        const auto rows = [&](const float* p, int r) {
            return bytes_rsrc(p + sh * r * kept, n > 0 ? (uint32_t)(r * kept) * 4u : 0u);
        };
        const uint32_t oe = e < a.Dv ? (uint32_t)kept_at(kC, t, e) * 4u : kNowhere;
        E.load(rows(a.E, kC), oe);
        dU.load(rows(a.dU, kC), oe);
#pragma unroll
        for (int s = 0; s < KC / 32; ++s) {
            const int es = v0 + s * 32 + (l >> 4) * 8;
            const uint32_t os = es < a.Dv ? (uint32_t)kept_at(dkp, d0 + (l & 15), es) * 4u : kNowhere;
            s0[s].load(rows(a.S0, dkp), os);
            s1[s].load(rows(a.dS1, dkp), os);
        }
        beta = Elt<float>::raw_rsrc(rows_rsrc(a.beta + at, n, a.Hv, 1), (uint32_t)(t * a.Hv) * 4u);
        dec = Elt<float>::raw_rsrc(bytes_rsrc(a.dec + sh * kDec, n > 0 ? kDec * 4 : 0), (uint32_t)tid * 4u);
    }
};

template <typename T>
__global__ __launch_bounds__(256, kExact<T> == 1 ? 2 : 1) void k_delta_grads(DeltaArgs a) {
    constexpr int NW = 4;
    constexpr int NX = kExact<T>;
    constexpr int KC = NW * 8;    // columns at a time
    constexpr int TT = (10 + NW - 1) / NW;  // tiles of a^T a wave has: w, w + NW, ...
    using Plane = Tile<uint16_t, KC>;
    using Square = Tile<uint16_t, kC>;
    constexpr int PT = kC * KC, MT = kC * kC;
    constexpr int kPlanes = (NX + 6) * PT, kSquares = 6 * MT;
    // planes of dOut, dE and U ([token][column]); after a head's columns, of a
    // or -b ([i][j]) and its transpose
    __shared__ alignas(16) __bf16 lds[kPlanes > kSquares ? kPlanes : kSquares];
    __shared__ alignas(16) RowTile<T, NW * 16> kt, qt;
    __shared__ alignas(16) double G[kC];
    __shared__ alignas(16) float decay[2][kC];
    __shared__ float red[NW][kC], ends[NW * 4];
    const int halves = (a.Dk + kDh - 1) / kDh;
    const Spread sp = spread(blockIdx.x, halves);
    if (sp.group >= delta_slots(a.T, a.nseq) * a.Hk) return;
    const int64_t slot = sp.group / a.Hk;
    const int hk = (int)(sp.group % a.Hk), half = sp.member, group = a.Hv / a.Hk;
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, slot, c)) return;
    const int wave = wave_id();
    __bf16* const Op = lds;
    __bf16* const Ep = lds + NX * PT;
    __bf16* const Up = Ep + 3 * PT;
    __bf16* const M = lds;
    __bf16* const Mt = lds + 3 * MT;
    const int d0 = half * kDh + wave * 16;  // this wave's first column of dq and dk
    // tile x of this wave: rows j of tile tj, columns i of tile ti >= tj, in the
    // order (0,0) (0,1) (0,2) (0,3) (1,1) ... (3,3); four bits each. The two
    // waves that have two make the last one again rather than branch.
    const auto tj = [&](int x) { return (int)((0x333221110000ull >> (4 * (wave + x * NW))) & 15); };
    const auto ti = [&](int x) { return (int)((0x333323213210ull >> (4 * (wave + x * NW))) & 15); };
    GradLoads<T, KC> next;
    next.load(a, slot, c, hk * group, 0, d0, c.n);
    {
        const int stride = a.Hk * a.Dk, dh = half * kDh;
        const size_t first = ((size_t)c.start * a.Hk + hk) * a.Dk;
        const auto kr = rows_rsrc(static_cast<const T*>(a.k) + first, c.n, stride, a.Dk);
        const auto qr = rows_rsrc(static_cast<const T*>(a.q) + first, c.n, stride, a.Dk);
        Unit<T> ku[2], qu[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int u = threadIdx.x + x * NW * 64, i = u / (NW * 2), k8 = u % (NW * 2);
            const uint32_t o =
                dh + k8 * 8 < a.Dk ? (uint32_t)(i * stride + dh + k8 * 8) * (uint32_t)sizeof(T) : kNowhere;
            ku[x].load(kr, o);
            qu[x].load(qr, o);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int u = threadIdx.x + x * NW * 64;
            kt.put(u / (NW * 2), u % (NW * 2), ku[x]);
            qt.put(u / (NW * 2), u % (NW * 2), qu[x]);
        }
    }
    f32x4 tq[4] = {}, tk[4] = {};
    for (int hv = hk * group; hv < (hk + 1) * group; ++hv) {
        f32x4 dq[4] = {}, dr[4] = {}, dw[4] = {};  // dq, dk read, dk write
        f32x4 at[TT] = {}, bt[TT] = {};
        float sd = 0.0f, db = 0.0f;                // <dS', S>; this thread's part of dbeta
        for (int v0 = 0; v0 < a.Dv; v0 += KC) {
            __syncthreads();  // what lies in lds, and the last head's decays, have been read
            const int tid = fresh(threadIdx.x), l = tid & 63, l16 = l & 15, l4 = l >> 4;
            {
                if (wave < 2) reinterpret_cast<uint32_t*>(G)[tid] = next.dec;
                else reinterpret_cast<uint32_t*>(&decay[0][0])[tid - 2 * kC] = next.dec;
                const int t = tid / (KC / 8), u = tid % (KC / 8), e = v0 + u * 8;
                const float beta = Elt<float>::cvt(next.beta);
                float E[8], dU[8];
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    E[p] = next.E.w[p >> 2][p & 3];
                    dU[p] = next.dU.w[p >> 2][p & 3];
                    db = fmaf(dU[p], E[p], db);
                    E[p] *= beta;
                    dU[p] *= beta;
                }
                Unit<T> dv;
                dv.pack(dU);
                dv.store(rows_rsrc(static_cast<const T*>(a.dv) + ((size_t)c.start * a.Hv + hv) * a.Dv,
                                   half == 0 ? c.n : 0, a.Hv * a.Dv, a.Dv),
                         e < a.Dv ? (uint32_t)(t * a.Hv * a.Dv + e) * (uint32_t)sizeof(T) : kNowhere);
                const auto po = unit_planes(next.o);
                const auto pe = split8<3>(dU), pu = split8<3>(E);
                const int o = Plane::at(t, u);
#pragma unroll
                for (int p = 0; p < NX; ++p) *reinterpret_cast<bf16x8*>(Op + p * PT + o) = po.p[p];
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    *reinterpret_cast<bf16x8*>(Ep + p * PT + o) = pe.p[p];
                    *reinterpret_cast<bf16x8*>(Up + p * PT + o) = pu.p[p];
                }
            }
            Frag<3> sb[KC / 32];
            Frag<3> gb[KC / 32];
#pragma unroll
            for (int s = 0; s < KC / 32; ++s) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sd = fmaf(next.s0[s].w[e >> 2][e & 3], next.s1[s].w[e >> 2][e & 3], sd);
                sb[s] = unit_planes(next.s0[s]);
                gb[s] = split_tiles<3>(next.s1[s].w[0], next.s1[s].w[1]);
            }
            {
                const bool more = v0 + KC < a.Dv;
                next.load(a, slot, c, more ? hv : hv + 1, more ? v0 + KC : 0, d0,
                          more || hv + 1 < (hk + 1) * group ? c.n : 0);
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < KC / 32; ++s) {
                const int u = s * 4 + l4;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int o = Plane::at(m * 16 + l16, u);
                    const auto po = tile_planes<NX>(Op, PT, o);
                    const auto pe = tile_planes<3>(Ep, PT, o);
                    const auto pu = tile_planes<3>(Up, PT, o);
                    static_for<6>([&](auto t) {
                        mma_term<3, t>(dr[m], pe, sb[s]);
                        mma_term<3, t>(dq[m], po, sb[s]);
                        mma_term<3, t>(dw[m], pu, gb[s]);
                    });
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int x = 0; x < TT; ++x) {
                    const auto uj = tile_planes<3>(Up, PT, Plane::at(tj(x) * 16 + l16, u));
                    const int o = Plane::at(ti(x) * 16 + l16, u);
                    const auto po = tile_planes<NX>(Op, PT, o);
                    const auto pe = tile_planes<3>(Ep, PT, o);
                    static_for<6>([&](auto t) {
                        mma_term<3, t>(bt[x], uj, pe);
                        mma_term<3, t>(at[x], uj, po);
                    });
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        __syncthreads();
        const int tid = fresh(threadIdx.x), l = tid & 63, l16 = l & 15, l4 = l >> 4;
        {
            const int t = tid / (KC / 8);
            const float s = dpp_add<0x4E>(dpp_add<0xB1>(db));
            const bool first = tid % (KC / 8) == 0;
            Elt<float>::st_rsrc(rows_rsrc(a.dbeta + (size_t)c.start * a.Hv + hv, half == 0 ? c.n : 0, a.Hv, 1),
                                first ? (uint32_t)(t * a.Hv) * 4u : kNowhere, s);
        }
        // the empty tiles (0, 1), (2, 3) of a and (1, 0), (3, 2) of its transpose
        for (int x = tid; x < 4 * 16 * 4; x += NW * 64) {
            const int w = x >> 6, r = (x >> 2) & 15, k4 = (x & 3) * 4;
            const int row = (w & 1) * 32 + (w >> 1) * 16 + r, k = kplace((w & 1) * 32 + (1 - (w >> 1)) * 16 + k4);
            const float zero[4] = {};
            if (w < 2) lds_put4<3>(M, MT, Square::at(row, k >> 3) + (k & 7), zero);
            else lds_put4<3>(Mt, MT, Square::at(row, k >> 3) + (k & 7), zero);
        }
        float end = decay[0][kC - 1] * sd;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            __builtin_amdgcn_sched_barrier(0);
            float kv[4], qv[4];
            kt.values4(l, m, wave, kv);
            qt.values4(l, m, wave, qv);
            const f32x4 eg = *reinterpret_cast<const f32x4*>(&decay[0][m * 16 + l4 * 4]);
            const f32x4 el = *reinterpret_cast<const f32x4*>(&decay[1][m * 16 + l4 * 4]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dq[m][r] *= eg[r] * a.scale;
                dr[m][r] *= -eg[r];
                end += fmaf(qv[r], dq[m][r], kv[r] * dr[m][r]);
            }
            tk[m] += el * dw[m];
        }
        float dx[TT][4];  // the decays of this wave's tiles
#pragma unroll
        for (int x = 0; x < TT; ++x) {
            const double gi = G[ti(x) * 16 + l16];
#pragma unroll
            for (int r = 0; r < 4; ++r) dx[x][r] = decay_of(gi - G[tj(x) * 16 + l4 * 4 + r]);
        }
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {  // a, then -b
#pragma unroll
            for (int x = 0; x < TT; ++x) {
                const int i = ti(x) * 16 + (int)fresh(l16), j = tj(x) * 16 + (int)fresh(l4) * 4;
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // (where it is not wanted the decay may be infinite: chosen, not multiplied, away)
                    const float w = dx[x][r] * (pass ? -bt[x][r] : a.scale * at[x][r]);
                    v[r] = (pass ? i > j + r : i >= j + r) ? w : 0.0f;
                }
                const int pj = kplace(j), pi = kplace(i);
                lds_put4<3>(M, MT, Square::at(i, pj >> 3) + (pj & 7), v);
#pragma unroll
                for (int r = 0; r < 4; r += 2) {
                    uint32_t p[3];
                    split2<3>(v[r], v[r + 1], p);
#pragma unroll
                    for (int y = 0; y < 3; ++y) {
                        uint16_t* const to = reinterpret_cast<uint16_t*>(Mt) + y * MT;
                        to[Square::at(j + r, pi >> 3) + (pi & 7)] = (uint16_t)p[y];
                        to[Square::at(j + r + 1, pi >> 3) + (pi & 7)] = (uint16_t)(p[y] >> 16);
                    }
                }
            }
            __syncthreads();
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int u = s * 4 + l4;
                __builtin_amdgcn_sched_barrier(0);
                const auto kb = kt.token_frag(l, s, wave), qb = qt.token_frag(l, s, wave);
                // rows 32 s .. of a, rows .. 32 s + 31 of its transpose
                Frag<3> fm[4];
                Frag<3> ft[4];
#pragma unroll
                for (int m = 2 * s; m < 4; ++m) fm[m - 2 * s] = tile_planes<3>(M, MT, Square::at(m * 16 + l16, u));
                if (s == 0) mma_tiles<3, 0, 4>(pass ? dr : dq, fm, kb);
                else mma_tiles<3, 2, 4>(pass ? dr : dq, fm, kb);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int m = 0; m < 2 + 2 * s; ++m) ft[m] = tile_planes<3>(Mt, MT, Square::at(m * 16 + l16, u));
                if (s == 0) mma_tiles<3, 0, 2>(tk, ft, pass ? kb : qb);
                else mma_tiles<3, 0, 4>(tk, ft, pass ? kb : qb);
            }
            if (pass == 0) __syncthreads();
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const int i = m * 16 + l4 * 4;
            __builtin_amdgcn_sched_barrier(0);
            float kv[4], qv[4];
            kt.values4(l, m, wave, kv);
            qt.values4(l, m, wave, qv);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float s = fmaf(qv[r], dq[m][r], kv[r] * dr[m][r]);
                end -= s;
                const float row = sum16(s);
                if (l16 == 0) red[wave][i + r] = row;
            }
            tq[m] += dq[m];
            tk[m] += dr[m];
        }
        end = sum16(end);
        if (l16 == 0) ends[wave * 4 + l4] = end;
        __syncthreads();
        if (wave == 0) {
            float s = (red[0][l] + red[1][l]) + (red[2][l] + red[3][l]);
            const float e = sum16(ends[l16]);
            if (l == kC - 1) s += e;
            *at_bytes(a.rows + ((size_t)(slot * a.Hv + hv) * halves + half) * kC, (uint32_t)l * 4u) = s;
        }
    }
    const Column cd = column_of<T>(a.Hk, a.Dk, d0 + (lane_id() & 15));
    const size_t first = ((size_t)c.start * a.Hk + hk) * a.Dk;
    store_column<T>(static_cast<T*>(a.dq) + first, c.n, a.Hk, a.Dk, cd, tq, 1.0f);
    store_column<T>(static_cast<T*>(a.dk) + first, c.n, a.Hk, a.Dk, cd, tk, 1.0f);
}

// dg of a chunk: the sums of a.rows from each token to the chunk's end, in 64
// bits. One wave per (slot, value head).
template <int kUnused = 0>
__global__ __launch_bounds__(256) void k_delta_dg(DeltaArgs a) {
    const int64_t sh = (int64_t)blockIdx.x * 4 + wave_id();
    if (sh >= delta_slots(a.T, a.nseq) * a.Hv) return;
    const int hv = (int)(sh % a.Hv), halves = (a.Dk + kDh - 1) / kDh, l = lane_id();
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, sh / a.Hv, c)) return;
    double s = 0.0;
    for (int h = 0; h < halves; ++h) s += (double)a.rows[(sh * halves + h) * kC + l];
    // what token i writes counts against it, and once for the whole chunk
    const size_t at = (size_t)(c.start + l) * a.Hv + hv;
    const double w = l < c.n ? (double)a.beta[at] * (double)a.dbeta[at] : 0.0;
    double all = w;
#pragma unroll
    for (int x = 1; x < kC; x <<= 1) all += __shfl_xor(all, x);
    s += (l == kC - 1 ? all : 0.0) - w;
#pragma unroll
    for (int x = 1; x < kC; x <<= 1) {
        const double o = __shfl_down(s, x);
        if (l + x < kC) s += o;
    }
    if (l < c.n) a.dg[at] = (float)s;
}

template <typename T, int DKP>
void launch_delta_chain_bwd(const DeltaArgs& a, int waves, hipStream_t s) {
    if constexpr (kWide<T, DKP>)
        if (waves == 8) {
            k_delta_chain_bwd<T, DKP, 8, false><<<chain_blocks(a, 8), 512, 0, s>>>(a);
            return;
        }
    k_delta_chain_bwd<T, DKP, 4, false><<<chain_blocks(a, 4), 256, 0, s>>>(a);
}

template <typename T, int DKP>
int launch_delta_bwd(DeltaArgs a, hipStream_t s) {
    const int waves = chain_waves<T, DKP>(a);
    if (!chain_ordered(a, waves)) a.order = nullptr;
    if (a.T > 0)
        if (const int st = launch_delta_prepare<T, DKP, true>(a, s)) return st;
    if (a.T > 0 || a.dh0) {
        if (a.split) {
            k_delta_chain_bwd<T, DKP, 4, true><<<split_blocks(a, DKP), 256, 0, s>>>(a);
            SSMP_LAUNCH_CHECK();
            launch_delta_join<DKP, true>(a, a.dhT, a.dh0, s);
            SSMP_LAUNCH_CHECK();
        }
        launch_delta_chain_bwd<T, DKP>(a, waves, s);
        SSMP_LAUNCH_CHECK();
    }
    if (a.T > 0) {
        const int64_t slots = delta_slots(a.T, a.nseq);
        const unsigned blocks = (unsigned)spread_blocks(slots * a.Hk, (a.Dk + kDh - 1) / kDh);
        k_delta_grads<T><<<blocks, 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
        k_delta_dg<><<<(unsigned)((slots * a.Hv + 3) / 4), 256, 0, s>>>(a);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}

struct DeltaBwdLayout {
    size_t dec, inv, att, order, dS1, dU, rows, joint, total;
};
inline DeltaBwdLayout delta_bwd_layout(int64_t T, int32_t nseq, int32_t Hv, int32_t Dk, int32_t Dv) {
    const size_t n = (size_t)delta_slots(T, nseq);
    DeltaBwdLayout L;
    L.dec = 0;
    L.inv = L.dec + round256(n * Hv * kDec * 4);
    L.att = L.inv + round256(n * Hv * kTri * 4);
    L.order = L.att + round256(n * Hv * kTri * 4);
    L.dS1 = L.order + round256((size_t)nseq * 4);
    L.dU = L.dS1 + kept_bytes(T, nseq, Hv, delta_dkp(Dk), Dv);
    L.rows = L.dU + kept_bytes(T, nseq, Hv, kC, Dv);
    L.joint = L.rows + round256(n * Hv * ((Dk + kDh - 1) / kDh) * kC * 4);
    L.total = L.joint + joint_bytes(T, nseq, Hv, delta_dkp(Dk), Dv);
    return L;
}

}  // namespace ssmp

extern "C" size_t gated_delta_pack_bwd_scratch_bytes(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk,
                                                     int32_t Dv, int32_t dtype) {
    using namespace ssmp;
    if (delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype) || T == 0) return 0;
    return delta_bwd_layout(T, nseq, Hv, Dk, Dv).total;
}

extern "C" int gated_delta_pack_bwd(const void* q, const void* k, const float* g, const float* beta,
                                    const int32_t* cu_seqlens, int32_t nseq, const void* dout, int64_t T, int32_t Hk,
                                    int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype, float scale,
                                    const float* dfinal_state, float* dinitial_state, void* dq, void* dk, void* dv,
                                    float* dg, float* dbeta, const void* saved, size_t saved_bytes, void* scratch,
                                    size_t scratch_bytes, void* stream) {
    using namespace ssmp;
    if (const int st = delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    if (!cu_seqlens) return SSMP_ERR_NULL;
    if (T > 0 && (!q || !k || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta)) return SSMP_ERR_NULL;
    if (!aligned16(q, k, dout, dq, dk, dv, dfinal_state, dinitial_state, saved, scratch)) return SSMP_ERR_ALIGN;
    if (T > 0 && (!saved || saved_bytes < gated_delta_pack_saved_bytes(T, nseq, Hk, Hv, Dk, Dv)))
        return SSMP_ERR_WORKSPACE;
    if (T > 0 && (!scratch || scratch_bytes < gated_delta_pack_bwd_scratch_bytes(T, nseq, Hk, Hv, Dk, Dv, dtype)))
        return SSMP_ERR_WORKSPACE;
    if (T == 0 && !dinitial_state) return SSMP_OK;
    const DeltaBwdLayout L = delta_bwd_layout(T, nseq, Hv, Dk, Dv);
    char* const ws = static_cast<char*>(scratch);
    DeltaArgs a = {};
    a.q = q;
    a.k = k;
    a.dout = dout;
    a.g = g;
    a.beta = beta;
    a.cu = cu_seqlens;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dg = dg;
    a.dbeta = dbeta;
    a.dhT = dfinal_state;
    a.dh0 = dinitial_state;
    a.T = T;
    a.nseq = nseq;
    a.Hk = Hk;
    a.Hv = Hv;
    a.Dk = Dk;
    a.Dv = Dv;
    a.scale = scale;
    if (T > 0) {
        char* const kept = static_cast<char*>(const_cast<void*>(saved));
        a.S0 = reinterpret_cast<float*>(kept);
        a.E = reinterpret_cast<float*>(kept + kept_bytes(T, nseq, Hv, delta_dkp(Dk), Dv));
        a.dec = reinterpret_cast<float*>(ws + L.dec);
        a.inv = reinterpret_cast<float*>(ws + L.inv);
        a.att = reinterpret_cast<float*>(ws + L.att);
        a.dS1 = reinterpret_cast<float*>(ws + L.dS1);
        a.dU = reinterpret_cast<float*>(ws + L.dU);
        a.rows = reinterpret_cast<float*>(ws + L.rows);
        a.order = reinterpret_cast<int32_t*>(ws + L.order);
        a.joint = reinterpret_cast<float*>(ws + L.joint);
        a.split = split_chunks(T, nseq, Hv, Dv);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wide = Dk > 64;
    if (dtype == SSMP_F32) return wide ? launch_delta_bwd<float, 128>(a, s) : launch_delta_bwd<float, 64>(a, s);
    return wide ? launch_delta_bwd<uint16_t, 128>(a, s) : launch_delta_bwd<uint16_t, 64>(a, s);
}
