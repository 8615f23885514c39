// Linear attention with a decay for each head, over packed sequences. Per
// value head with its key head, and a_t = exp(g_t),
//   S_t = a_t S_{t-1} + k_t v_t^T,   out_t = scale S_t^T q_t.
// Written out, out_i = scale sum_{j <= i} e^{G_i - G_j} (q_i.k_j) v_j with G
// the running sum of g, and every gradient is a sum of the same form:
//   dq_i = scale sum_{j <= i} e^{G_i - G_j} (dout_i.v_j) k_j
//   dk_j = scale sum_{i >= j} e^{G_i - G_j} (v_j.dout_i) q_i
//   dv_j = scale sum_{i >= j} e^{G_i - G_j} (k_j.q_i) dout_i
// so one kernel, k_decay_walk, serves all four: rows of `a` meet rows of `b`,
// and rows of `c` are added up, forwards in time or backwards. Its state is
// X = sum of decayed b c^T: S, S^T, and their gradients dS^T, dS.
//   d g_t = (dS_t . a_t S_{t-1}), and since (dS_t . S_t) is d g_t + k_t.dk_t as
// well as d g_{t+1} + q_t.dq_t:  d g_t = d g_{t+1} + q_t.dq_t - k_t.dk_t.
#pragma once

#include "delta_common.h"

namespace ssmp {

// ---------------------------------------------------------------------------
// Segments: pieces of seg tokens of a sequence, each walked by workgroups of
// its own, in slots by the rule of chunk_at. The states between the segments
// of a sequence come from a first walk over all that have one behind them
// (kSumS; kSumD: before them) and k_decay_join. The state between segments i
// and i + 1 of a sequence lies at cu[s] / seg + i, which meets no other
// sequence's, since segment i is whole: T / seg + 1 in all.
constexpr int kDecayCols = 128;     // columns of c a workgroup takes at most
constexpr int kDecayMaxDb = 128;    // rows of the state a workgroup takes
constexpr int kPiece = 256;         // tokens between the points where dg is anchored
constexpr int kSegMin = 256, kSegMax = 2048;
constexpr int kSegWork = 512;       // workgroups that a launch should have

inline int decay_cols(int32_t Dc) { return Dc <= 64 ? 64 : kDecayCols; }
inline int decay_col_blocks(int32_t Dc) { return (Dc + kDecayCols - 1) / kDecayCols; }
// heads * column blocks: the workgroups that a segment has
inline int32_t decay_segment(int64_t T, int64_t work) {
    const int64_t n = T * work / kSegWork / kSegMin * kSegMin;
    return (int32_t)(n < kSegMin ? kSegMin : n > kSegMax ? kSegMax : n);
}
// The most T' / decay_segment(T') for T' <= T, plus one: below kSegMax a
// segment is at least half of T' work / kSegWork long.
inline int64_t decay_states(int64_t T, int64_t work) {
    const int64_t few = T / kSegMin, many = 2 * kSegWork / work, least = T / kSegMax;
    const int64_t n = few < many ? few : many;
    return (n > least ? n : least) + 1;
}

// kOut, kSumS: decay_fwd.hip; kDq: decay_dq.hip; kDk: decay_dk.hip; kDv, kSumD: decay_bwd.hip
enum DecayKind { kOut, kDq, kDk, kDv, kSumS, kSumD };

struct DecayArgs {
    const void *q, *k, *v, *dout;
    const float* g;
    const int32_t* cu;
    void *out, *dq, *dk, *dv;
    float* dg;
    const float *h0, *dhT;
    float *hT, *dh0;
    int64_t T;
    int32_t nseq, Hk, Hv, Dk, Dv;
    int32_t gstride;      // Hv, or 0: one decay for a head
    float scale;
    int32_t seg;
    float *joint[2];      // states S, dS between segments: [state][Hv][Dk][Dv]
    float* seg_decay[2];  // [state][Hv]: e^(sum of g over the segment)
    // backward
    int32_t slices;       // of 128 rows that Dv has in dq and dk
    float* part[2];       // dq, dk by value head and slice: [T][Hk][members][Dk]; null where there is one
    float* rows[2];       // q.dq and k.dk: [parts][T][Hv]; null without dg
    float* snap;          // S^T after every kPiece-th token, in the walk's layout
    float* meet;          // (dS . S) at the ends of the pieces: [T / kPiece + nseq][Hv][parts]
    double* dgsum;        // one decay for a head: dg by piece, [T / kPiece + nseq][Hv]
};

constexpr bool decay_reverse(int kind) { return kind == kDk || kind == kDv || kind == kSumD; }
constexpr bool decay_by_key(int kind) { return kind == kDq || kind == kDk; }  // c and the result have key heads

// One side's rows: those of head h of H, columns off .. off + width - 1 of D
template <typename T>
struct Side {
    const T* p;
    int stride, width;
    __device__ __forceinline__ Side(const void* base, int64_t start, int H, int h, int D, int off, int w)
        : p(static_cast<const T*>(base) + ((size_t)start * H + h) * D + off), stride(H * D), width(w) {}
};

// 64 rows of a side on their way to LDS, W columns of it
template <typename T, int W, int THREADS>
struct SideLoads {
    static constexpr int kN = kC * W / 8 / THREADS;
    Unit<T> u[kN];
    __device__ __forceinline__ void load(const Side<T>& s, int64_t row, int n) {
        const auto r = rows_rsrc(s.p + row * s.stride, n, s.stride, s.width);
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int i = (threadIdx.x + x * THREADS) / (W / 8), c = (threadIdx.x + x * THREADS) % (W / 8);
            u[x].load(r, c * 8 < s.width ? (uint32_t)(i * s.stride + c * 8) * (uint32_t)sizeof(T) : kNowhere);
        }
    }
    // columns in places (they are a product's k), or as they come
    __device__ __forceinline__ void put_places(RowTile<T, W>& t) const {
#pragma unroll
        for (int x = 0; x < kN; ++x)
            t.put((threadIdx.x + x * THREADS) / (W / 8), (threadIdx.x + x * THREADS) % (W / 8), u[x]);
    }
    __device__ __forceinline__ void put_plain(RowTile<T, W>& t) const {
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            T* const p = t.x + RowTile<T, W>::L::at((threadIdx.x + x * THREADS) / (W / 8), (threadIdx.x + x * THREADS) % (W / 8));
            u[x].put_half(p, 0);
            u[x].put_half(p + 4, 1);
        }
    }
};

// Columns of c: in a tile that is stored plain, the reading that gives columns
// 16 m + n of one in places gives 32 (m / 2) + 8 (n / 4) + 4 (m % 2) + n % 4.
// A result whose rows are those of tiles m = 2 i and 2 i + 1 then leaves in
// each lane eight columns that lie together, 32 i + 8 (l / 16) .. + 7.
__device__ __forceinline__ int decay_col(int m, int n) { return (m >> 1) * 32 + (n >> 2) * 8 + (m & 1) * 4 + (n & 3); }

__device__ __forceinline__ float wave_sum(float v) {
    v = sum16(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

template <typename T, int DBP, int CT, int NP>
struct DecayTiles {
    RowTile<T, DBP> a, b;
    RowTile<T, 64 * CT> c;
    u32x4 P[8 * NP][64];          // [row tile][block of 32 columns][plane]: as one lane reads them
    double G[kC];
    float into[kC], onto[kC];     // decay from the state to a row, and from a row to the state
    float whole;                  // of the chunk
    float red[4][kC];
};

// One workgroup of four waves per (segment, value head, slice of the state's
// rows, column block), 16 CT columns a wave. In chunks of 64 rows:
//   out = into . (A X) + (D . A B^T) C,   X' = whole X + B^T (onto . C)
// The state's columns do not meet, so a wave keeps its own in registers; the
// decayed products P = D . A B^T are shared through LDS, a row tile from each
// wave. The products leave rows of the state as rows of a register, which is
// how the next product takes them (kplace), and rows of out along the lanes.
// kDots: rows of out times rows of q or k, for dg.
template <typename T, int KIND, int DBP, int CT, bool DOTS>
__global__ __launch_bounds__(256) void k_decay_walk(DecayArgs p) {
    constexpr int NX = kExact<T>;
    // Planes of P and of the state where out is formed: two hold 16 bits, of
    // which a bf16 result keeps 8; dg and fp32 results see all three. What is
    // added to the state has three always.
    constexpr int NP = NX == 3 || DOTS ? 3 : 2;
    constexpr bool REV = decay_reverse(KIND), SUM = KIND == kSumS || KIND == kSumD, KEYS = decay_by_key(KIND);
    constexpr int MT = DBP / 16, KS = DBP / 32, COLS = 64 * CT;
    __shared__ alignas(16) DecayTiles<T, DBP, CT, NP> lds;
    const int Dc = KEYS ? p.Dk : p.Dv, Db = KEYS ? p.Dv : p.Dk;
    const int ncb = (Dc + COLS - 1) / COLS, slices = KEYS ? p.slices : 1, group = p.Hv / p.Hk;
    const Spread sp = spread(blockIdx.x, group * slices * ncb);
    if (sp.group >= (p.T / p.seg + p.nseq) * (int64_t)p.Hk) return;
    Chunk sg;
    if (!chunk_at(p.cu, p.nseq, p.T, sp.group / p.Hk, sg, p.seg, true)) return;
    if (SUM && (REV ? sg.index == 0 : sg.last)) return;
    const int hk = (int)(sp.group % p.Hk), cb = sp.member % ncb, slice = sp.member / ncb % slices;
    const int hv = hk * group + sp.member / (ncb * slices);
    const int wave = wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    const int col0 = cb * COLS, off = slice * kDecayMaxDb, db = min(Db - off, DBP), parts = slices * ncb;
    const int64_t state0 = (sg.start - sg.index * p.seg) / p.seg + sg.index;  // of the state behind this segment
    // a and b by the heads that have them
    const void* const ta = KIND == kOut ? p.q : KIND == kDq ? p.dout : KIND == kDk ? p.v : p.k;
    const void* const tb = KIND == kOut || KIND == kSumS ? p.k : KIND == kDq ? p.v : KIND == kDk ? p.dout : p.q;
    const void* const tc = KIND == kOut || KIND == kSumS ? p.v : KIND == kDq ? p.k : KIND == kDk ? p.q : p.dout;
    const int Hb = KEYS ? p.Hv : p.Hk, hb = KEYS ? hv : hk, Hc = KEYS ? p.Hk : p.Hv, hc = KEYS ? hk : hv;
    const Side<T> sa(ta, sg.start, Hb, hb, Db, off, db), sb(tb, sg.start, Hb, hb, Db, off, db);
    const Side<T> sc(tc, sg.start, Hc, hc, Dc, col0, min(Dc - col0, COLS));
    // the state's element (row of b, column of c) in tensors of [Dk][Dv]
    const auto element = [&](int row, int col) { return KEYS ? (size_t)col * p.Dv + row : (size_t)row * p.Dv + col; };
    const auto state_ptr = [&](const float* base, int64_t n) { return base + ((size_t)n * p.Hv + hv) * p.Dk * p.Dv; };
    const auto each = [&](auto f) {  // of the lane's elements
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = m * 16 + l4 * 4 + r, col = col0 + decay_col(wave * CT + ct, l16);
                    if (row < db && col < Dc) f(m, ct, r, element(off + row, col));
                }
    };
    f32x4 S[MT][CT] = {};
    if constexpr (!SUM) {
        const float* from = nullptr;
        if (!REV) from = sg.index > 0 ? state_ptr(p.joint[0], state0 - 1) : p.h0 ? state_ptr(p.h0, sg.seq) : nullptr;
        else from = !sg.last ? state_ptr(p.joint[1], state0) : p.dhT ? state_ptr(p.dhT, sg.seq) : nullptr;
        if (from) each([&](int m, int ct, int r, size_t e) { S[m][ct][r] = from[e]; });
    }
    const int chunks = (sg.n + kC - 1) / kC;
    SideLoads<T, DBP, 256> la, lb;
    SideLoads<T, COLS, 256> lc;
    uint32_t lg;
    const auto load = [&](int i) {  // the i-th chunk of the walk
        const int ch = REV ? chunks - 1 - i : i;
        const int n = i < chunks ? min(sg.n - ch * kC, kC) : 0;
        if constexpr (!SUM) la.load(sa, (int64_t)ch * kC, n);
        lb.load(sb, (int64_t)ch * kC, n);
        lc.load(sc, (int64_t)ch * kC, n);
        const int64_t t = sg.start + ch * kC;
        lg = Elt<float>::raw_rsrc(rows_rsrc(p.g + (p.gstride ? t * p.gstride : 0) + hv, n, p.gstride, 1),
                                  l < n ? (uint32_t)(l * p.gstride) * 4u : kNowhere);
    };
    double total = 0.0;
    load(0);
    for (int i = 0; i < chunks; ++i) {
        const int ch = REV ? chunks - 1 - i : i, n = min(sg.n - ch * kC, kC);
        const int64_t t0 = sg.start + ch * kC;
        // dg's anchors: the state S^T of dq's walk behind every piece meets dS^T of dk's
        const int64_t from_seq = sg.index * p.seg + ch * kC;
        const bool piece_end = (from_seq + kC) % kPiece == 0 && !(sg.last && ch == chunks - 1);
        const int64_t pieces = (sg.start - sg.index * p.seg) / kPiece + from_seq / kPiece;
        float* snap = nullptr;
        if constexpr (DOTS)
            snap = p.snap + (((size_t)pieces * p.Hv + hv) * parts + slice * ncb + cb) * (DBP * COLS) +
                   (size_t)wave * (MT * CT * 256) + l * 4;
        if constexpr (!SUM) la.put_places(lds.a);
        lb.put_places(lds.b);
        lc.put_plain(lds.c);
        if (wave == 0) {
            const double G = chunk_decay_sum(l < n ? Elt<float>::cvt(lg) : 0.0f), last = read_lane(G, kC - 1);
            lds.G[l] = G;
            const float head = decay_of(G), tail = decay_of(last - G);
            lds.into[l] = REV ? tail : head * p.scale;
            lds.onto[l] = REV ? head * p.scale : tail;
            if (l == 0) lds.whole = decay_of(last);
            total += last;
        }
        if constexpr (DOTS && KIND == kDk) {
            if (piece_end) {
                float e = 0.0f;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        const f32x4 w = *reinterpret_cast<const f32x4*>(snap + (m * CT + ct) * 256);
#pragma unroll
                        for (int r = 0; r < 4; ++r) e = fmaf(S[m][ct][r], w[r], e);
                    }
                e = wave_sum(e);
                if (l == 0) lds.red[wave][0] = e;
            }
        }
        __syncthreads();
        if constexpr (DOTS && KIND == kDk) {
            if (piece_end && threadIdx.x == 0)
                p.meet[((size_t)(pieces + sg.seq) * p.Hv + hv) * parts + slice * ncb + cb] =
                    (lds.red[0][0] + lds.red[1][0]) + (lds.red[2][0] + lds.red[3][0]);
        }
        load(i + 1);
        f32x4 o[CT][4] = {};
        if constexpr (!SUM) {
            // P: wave w has rows 16 w .. + 15 along its lanes
            f32x4 x[4] = {};
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const Frag<NX> fa = lds.a.frag(wave * 16 + l16, s * 4 + l4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (REV ? j >= wave : j <= wave) mma<NX>(x[j], lds.b.frag(j * 16 + l16, s * 4 + l4), fa);
            }
            const int row = wave * 16 + l16;
            const double Gi = lds.G[row];
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int col = j * 16 + l4 * 4 + r;
                    const float d = decay_of(REV ? lds.G[col] - Gi : Gi - lds.G[col]) * p.scale;
                    x[j][r] = (REV ? col >= row : col <= row) ? d * x[j][r] : 0.0f;
                }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (REV ? s == 0 && wave >= 2 : s == 1 && wave < 2) continue;
                const Frag<NP> f = split_tiles<NP>(x[2 * s], x[2 * s + 1]);
#pragma unroll
                for (int i = 0; i < NP; ++i) lds.P[(wave * 2 + s) * NP + i][l] = __builtin_bit_cast(u32x4, f.p[i]);
            }
            // A X, rows of out along the lanes
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                Frag<NP> fs[CT];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) fs[ct] = split_tiles<NP>(S[2 * s][ct], S[2 * s + 1][ct]);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const Frag<NX> fa = lds.a.frag(t * 16 + l16, s * 4 + l4);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma<NP>(o[ct][t], fs[ct], fa);
                }
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float d = lds.into[t * 16 + l16];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[ct][t] *= d;
            }
            __syncthreads();
        }
        const float whole = lds.whole;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) S[m][ct] *= whole;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const f32x4 w0 = *reinterpret_cast<const f32x4*>(lds.onto + s * 32 + l4 * 4);
            const f32x4 w1 = *reinterpret_cast<const f32x4*>(lds.onto + s * 32 + 16 + l4 * 4);
            Frag<NX> fc[CT];
            Frag<3> fw[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int m = wave * CT + ct;
                fc[ct] = lds.c.token_frag(l, s, m);
                float c0[4], c1[4];
                lds.c.values4(l, 2 * s, m, c0);
                lds.c.values4(l, 2 * s + 1, m, c1);
                fw[ct] = split8<3>({c0[0] * w0[0], c0[1] * w0[1], c0[2] * w0[2], c0[3] * w0[3], c1[0] * w1[0],
                                    c1[1] * w1[1], c1[2] * w1[2], c1[3] * w1[3]});
            }
            if constexpr (!SUM) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (REV ? s == 0 && t >= 2 : s == 1 && t < 2) continue;
                    Frag<NP> f;
#pragma unroll
                    for (int i = 0; i < NP; ++i) f.p[i] = __builtin_bit_cast(bf16x8, lds.P[(t * 2 + s) * NP + i][l]);
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) mma<NP>(o[ct][t], fc[ct], f);
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const Frag<NX> fb = lds.b.token_frag(l, s, m);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) mma<3>(S[m][ct], fb, fw[ct]);
            }
        }
        if constexpr (!SUM) {
            // out: a lane has 4 CT columns of the rows 16 t + l16
            const int D = Dc, H = KEYS ? p.Hk : p.Hv, h = KEYS ? hk : hv;
            const int col = col0 + (CT == 2 ? wave * 32 + l4 * 8 : (wave >> 1) * 32 + l4 * 8 + (wave & 1) * 4);
            const int members = group * slices;
            const bool partial = KEYS && members > 1;
            if (partial) {
                const int member = sp.member / ncb;
                float* const base = p.part[REV] + (((size_t)t0 * H + h) * members + member) * D;
                const auto r = rows_rsrc(base, n, H * members * D, D);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, o[ct][t]), r,
                            (int)(col < D ? (uint32_t)((t * 16 + l16) * (H * members * D) + col + ct * 4) * 4u : kNowhere), 0, 0);
            } else {
                T* const base = static_cast<T*>(KIND == kOut ? p.out : KIND == kDq ? p.dq : KIND == kDk ? p.dk : p.dv) +
                                ((size_t)t0 * H + h) * D;
                const auto r = rows_rsrc(base, n, H * D, D);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t at = col < D ? (uint32_t)((t * 16 + l16) * H * D + col) * (uint32_t)sizeof(T) : kNowhere;
                    if constexpr (CT == 2) {
                        Unit<T> u;
                        const f32x4 y = o[0][t], z = o[CT - 1][t];
                        u.pack({y[0], y[1], y[2], y[3], z[0], z[1], z[2], z[3]});
                        u.store(r, at);
                    } else if constexpr (NX == 3) {
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[0][t]), r, (int)at, 0, 0);
                    } else {
                        const f32x4 y = o[0][t];
                        const u32x2 w = {(uint32_t)f32_to_bf16(y[0]) | ((uint32_t)f32_to_bf16(y[1]) << 16),
                                         (uint32_t)f32_to_bf16(y[2]) | ((uint32_t)f32_to_bf16(y[3]) << 16)};
                        __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)at, 0, 0);
                    }
                }
            }
            if constexpr (DOTS) {
                const Side<T> sd(KIND == kDq ? p.q : p.k, t0, p.Hk, hk, p.Dk, 0, p.Dk);
                const auto r = rows_rsrc(sd.p, n, sd.stride, sd.width);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float e = 0.0f;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint32_t at = col < D ? (uint32_t)((t * 16 + l16) * sd.stride + col + ct * 4 + x) * (uint32_t)sizeof(T) : kNowhere;
                            e = fmaf(o[ct][t][x], Elt<T>::cvt(Elt<T>::raw_rsrc(r, at)), e);
                        }
                    e += __shfl_xor(e, 16);
                    e += __shfl_xor(e, 32);
                    if (l4 == 0) lds.red[wave][t * 16 + l16] = e;
                }
                if constexpr (KIND == kDq) {
                    if (piece_end) {
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct)
                                *reinterpret_cast<f32x4*>(snap + (m * CT + ct) * 256) = S[m][ct];
                    }
                }
            }
        }
        __syncthreads();
        if constexpr (DOTS) {
            if (threadIdx.x < n) {
                const int x = threadIdx.x;
                p.rows[REV][((size_t)(slice * ncb + cb) * p.T + t0 + x) * p.Hv + hv] =
                    (lds.red[0][x] + lds.red[1][x]) + (lds.red[2][x] + lds.red[3][x]);
            }
            __syncthreads();
        }
    }
    if constexpr (SUM) {
        float* const to = const_cast<float*>(state_ptr(p.joint[REV], state0 - REV));
        each([&](int m, int ct, int r, size_t e) { to[e] = S[m][ct][r]; });
        if (threadIdx.x == 0 && cb == 0) p.seg_decay[REV][(size_t)(state0 - REV) * p.Hv + hv] = decay_of(total);
    } else if constexpr (KIND == kOut) {
        if (p.hT && sg.last) {
            float* const to = const_cast<float*>(state_ptr(p.hT, sg.seq));
            each([&](int m, int ct, int r, size_t e) { to[e] = S[m][ct][r]; });
        }
    } else if constexpr (KIND == kDv) {
        if (p.dh0 && sg.index == 0) {
            float* const to = const_cast<float*>(state_ptr(p.dh0, sg.seq));
            each([&](int m, int ct, int r, size_t e) { to[e] = S[m][ct][r]; });
        }
    } else if constexpr (DOTS && KIND == kDq) {
        if (p.dhT && sg.last) {  // the last piece's anchor
            const float* const w = state_ptr(p.dhT, sg.seq);
            float e = 0.0f;
            each([&](int m, int ct, int r, size_t at) { e = fmaf(S[m][ct][r], w[at], e); });
            e = wave_sum(e);
            if (l == 0) lds.red[wave][0] = e;
            __syncthreads();
            const int64_t first = sg.start - sg.index * p.seg, len = sg.index * p.seg + sg.n;
            if (threadIdx.x == 0 && len > 0)
                p.meet[((size_t)(first / kPiece + sg.seq + (len - 1) / kPiece) * p.Hv + hv) * parts + slice * ncb + cb] =
                    (lds.red[0][0] + lds.red[1][0]) + (lds.red[2][0] + lds.red[3][0]);
        }
    }
}

// Along the segments of each sequence that has several, in place: what a
// segment adds becomes the state on its far side, X' = decay X + U. One
// workgroup per (segment slot that is a sequence's first, head, block of
// elements): each element is read and written once.
template <bool REV>
__global__ __launch_bounds__(256) void k_decay_join(DecayArgs p, int blocks) {
    const int64_t slot = blockIdx.x / ((int64_t)p.Hv * blocks);
    const int hv = blockIdx.x / blocks % p.Hv, block = blockIdx.x % blocks;
    Chunk c;
    if (!chunk_at(p.cu, p.nseq, p.T, slot, c, p.seg) || c.index != 0 || c.last) return;
    const int64_t end = p.cu[c.seq + 1] < p.T ? p.cu[c.seq + 1] : p.T;
    const int n = (int)((end - c.start + p.seg - 1) / p.seg) - 1;  // states between its segments
    const int64_t state0 = c.start / p.seg;
    const size_t size = (size_t)p.Dk * p.Dv, step = size * p.Hv;
    float* const x = p.joint[REV] + (size_t)state0 * step + hv * size;
    const float* const d = p.seg_decay[REV] + state0 * p.Hv + hv;
    const float* const first = REV ? (p.dhT ? p.dhT + ((size_t)c.seq * p.Hv + hv) * size : nullptr)
                                   : (p.h0 ? p.h0 + ((size_t)c.seq * p.Hv + hv) * size : nullptr);
    for (size_t e = ((size_t)block * 256 + threadIdx.x) * 4; e < size; e += (size_t)blocks * 1024) {
        f32x4 s = first ? *reinterpret_cast<const f32x4*>(first + e) : f32x4{0, 0, 0, 0};
        for (int i = 0; i < n; ++i) {
            float* const at = x + (REV ? n - 1 - i : i) * step + e;
            s = s * d[(REV ? n - 1 - i : i) * p.Hv] + *reinterpret_cast<const f32x4*>(at);
            *reinterpret_cast<f32x4*>(at) = s;
        }
    }
}

// The walks' workgroups, by kind: those of heads that share a and b, or c, on
// one XCD.
inline int64_t decay_walk_blocks(const DecayArgs& a, int kind) {
    const int32_t Dc = decay_by_key(kind) ? a.Dk : a.Dv;
    const int members = a.Hv / a.Hk * (decay_by_key(kind) ? a.slices : 1) * ((Dc + decay_cols(Dc) - 1) / decay_cols(Dc));
    return spread_blocks((a.T / a.seg + a.nseq) * a.Hk, members);
}
template <typename T, int KIND, bool DOTS>
void launch_decay_walk_t(const DecayArgs& a, hipStream_t s) {
    const unsigned n = (unsigned)decay_walk_blocks(a, KIND);
    const int32_t Dc = decay_by_key(KIND) ? a.Dk : a.Dv, Db = decay_by_key(KIND) ? a.Dv : a.Dk;
    if (Db > 64) {
        if (Dc > 64) k_decay_walk<T, KIND, 128, 2, DOTS><<<n, 256, 0, s>>>(a);
        else k_decay_walk<T, KIND, 128, 1, DOTS><<<n, 256, 0, s>>>(a);
    } else {
        if (Dc > 64) k_decay_walk<T, KIND, 64, 2, DOTS><<<n, 256, 0, s>>>(a);
        else k_decay_walk<T, KIND, 64, 1, DOTS><<<n, 256, 0, s>>>(a);
    }
}
template <int KIND, bool DOTS>
int launch_decay_walk_of(const DecayArgs& a, int32_t dtype, hipStream_t s) {
    if (dtype == SSMP_F32) launch_decay_walk_t<float, KIND, DOTS>(a, s);
    else launch_decay_walk_t<uint16_t, KIND, DOTS>(a, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
// each kind is compiled in the source that DecayKind's comment names
template <int KIND>
int launch_decay_walk(const DecayArgs& a, int32_t dtype, hipStream_t s);

template <bool REV>
int launch_decay_join(const DecayArgs& a, hipStream_t s) {
    const int64_t slots = a.T / a.seg + a.nseq, per = (int64_t)a.Dk * a.Dv / 1024 + 1;
    int64_t blocks = 2048 / (slots * a.Hv);
    blocks = blocks < 1 ? 1 : blocks > per ? per : blocks;
    k_decay_join<REV><<<(unsigned)(slots * a.Hv * blocks), 256, 0, s>>>(a, (int)blocks);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

inline int decay_check(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype) {
    if (const int st = delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    const int64_t slices = (Dv + kDecayMaxDb - 1) / kDecayMaxDb;
    if (Hv * slices * Dk > kMaxRow) return SSMP_ERR_SHAPE;  // a row of dq's parts
    if ((T / kPiece + nseq + 7) * (int64_t)Hv * slices >= kMaxBlocks) return SSMP_ERR_SHAPE;
    return SSMP_OK;
}

// States between segments, and the segments' decays
struct DecayJoint {
    size_t joint, decay, total;
};
inline DecayJoint decay_joint(int64_t T, int32_t Hv, int32_t Dk, int32_t Dv, int64_t work) {
    const size_t n = T > kSegMin ? (size_t)decay_states(T, work) : 0;
    DecayJoint j;
    j.joint = 0;
    j.decay = round256(n * Hv * Dk * Dv * sizeof(float));
    j.total = j.decay + round256(n * Hv * sizeof(float));
    return j;
}

}  // namespace ssmp
