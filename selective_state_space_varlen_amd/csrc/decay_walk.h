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
// well as d g_{t+1} + q_t.dq_t:  d g_t = d g_{t+1} + q_t.dq_t - k_t.dk_t,
// from (dS . S) at a sequence's end. The terms nearly cancel where decays are
// strong, so roundings must not add up along the sequence: (dS . S) is formed
// anew after every kPiece tokens, where dq's walk leaves S for dk's, and goes
// from chunk to chunk by what crosses between chunks alone: (dS . S) before a
// chunk is that behind it + sum q.dq' - sum k.dk', dq' and dk' being the parts
// that come through the states. Both are the start of many tokens' dg, so they
// are summed in 64 bits (in 32: dg of 16384 tokens in long sequences errs by
// 3.7e-7 of its norm, now by 3.0e-7, the sum over the tokens of short ones by
// up to 8.3e-7, now 6.4e-7; the backward takes as long).
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
constexpr int kSegMin = 128, kSegMax = 2048;
constexpr int kSegWork = 768;       // workgroups that a launch should have

inline int decay_col_blocks(int32_t Dc) { return (Dc + kDecayCols - 1) / kDecayCols; }
// work: heads * column blocks, the workgroups that a segment has. Enough
// sequences are walked whole, as the first walk costs a third of the forward;
// a longest segment bounds what one long sequence among them takes. 16384
// tokens in 6 sequences x 24 heads of 128 x 64, segments of 768, 512, 384 and
// 256 tokens: forward 177, 144, 158 and 153 us, backward 725, 583, 646 and 618.
inline int32_t decay_segment(int64_t T, int32_t nseq, int64_t work) {
    if (nseq * work >= kSegWork) return kSegMax;
    const int64_t n = T * work / kSegWork / kSegMin * kSegMin;
    return (int32_t)(n < kSegMin ? kSegMin : n > kSegMax ? kSegMax : n);
}
// The most T' / decay_segment(T', any nseq) for T' <= T, plus one: below kSegMax
// a segment is at least half of T' work / kSegWork long.
inline int64_t decay_states(int64_t T, int64_t work) {
    const int64_t few = T / kSegMin, many = 2 * kSegWork / work, least = T / kSegMax;
    const int64_t n = few < many ? few : many;
    return (n > least ? n : least) + 1;
}

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
    int32_t few;          // few segments: each walk adds up what the others left (no k_decay_join)
    // backward
    int32_t slices;       // of 128 rows that Dv has in dq and dk
    int32_t heads;        // of a key head that a workgroup of dq's and dk's walks has
    float* part[2];       // dq, dk by value head and slice: [T][Hk][members][Dk]; null where there is one
    float* rows[2];       // q.dq and k.dk: [parts][T][Hv]
    double* chunk[2];     // what a chunk's rows of them get from and give to other chunks: [T / 64 + nseq][Hv][parts]
    float* snap;          // S^T after every kPiece-th token, in the walk's layout
    double* meet;         // (dS . S) at the ends of the pieces: [T / kPiece + nseq][Hv][parts]
    double* dgsum;        // one decay for a head: dg by piece, [T / kPiece + nseq][Hv]
};

constexpr bool decay_reverse(int kind) { return kind == kDk || kind == kDv || kind == kSumD; }
constexpr bool decay_by_key(int kind) { return kind == kDq || kind == kDk; }  // c and the result have key heads

// The r-th segment of a walk, longest first, where there are at most 64
// sequences: a launch takes as long as the workgroup that ends last, and a
// long segment that starts last is waited for alone. Whole segments come
// first, then what remains of each sequence by its length (and sequences
// without tokens). Lane s looks at sequence s.
__device__ __forceinline__ bool segment_at(const DecayArgs& p, int64_t r, Chunk& c) {
    if (p.nseq > 64) return chunk_at(p.cu, p.nseq, p.T, r, c, p.seg, true);
    const int l = lane_id();
    const Seq q = l < p.nseq ? seq_at(p.cu, l, p.T) : Seq{0, 0, 0};
    const int whole = q.len / p.seg, rest = l < p.nseq && (q.len == 0 || q.len % p.seg) ? q.len % p.seg : -1;
    int before = whole;  // running sum of the whole ones
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(before, d);
        before += l >= d ? v : 0;
    }
    const int all = __builtin_amdgcn_readlane(before, 63);
    int at, index;
    if (r < all) {
        at = __popcll(__ballot(before <= r));
        index = (int)r - __builtin_amdgcn_readlane(before - whole, at);
    } else {
        int rank = 0;
        for (int s = 0; s < p.nseq; ++s) {
            const int v = __builtin_amdgcn_readlane(rest, s);
            rank += v > rest || (v == rest && s < l);
        }
        const uint64_t hit = __ballot(rest >= 0 && rank == (int)r - all);
        if (!hit) return false;
        at = __ffsll((unsigned long long)hit) - 1;
        index = __builtin_amdgcn_readlane(whole, at);
    }
    const int len = __builtin_amdgcn_readlane(q.len, at);
    const int start = __builtin_amdgcn_readlane((int)q.start, at);
    c.start = (int64_t)start + (int64_t)index * p.seg;
    c.n = min(len - index * p.seg, p.seg);
    c.seq = at;
    c.index = index;
    c.last = len - index * p.seg <= p.seg;
    return true;
}

// fresh(), of a scalar
__device__ __forceinline__ int fresh_scalar(int v) {
    asm volatile("" : "+s"(v));
    return v;
}

// One side's rows: those of head h of H, columns off .. off + width - 1 of D
template <typename T>
struct Side {
    const T* p;
    int stride, width;
    __device__ __forceinline__ Side(const void* base, int64_t start, int H, int h, int D, int off, int w)
        : p(static_cast<const T*>(base) + ((size_t)start * H + h) * D + off), stride(H * D), width(w) {}
    // byte offset of column c of row i, which a multiple of rows may be added to
    __device__ __forceinline__ uint32_t at(int i, int c) const {
        return c < width ? (uint32_t)(i * stride + c) * (uint32_t)sizeof(T) : kNowhere;
    }
    __device__ __forceinline__ uint32_t rows(int n) const { return (uint32_t)(n * stride) * (uint32_t)sizeof(T); }
};

// The same in every lane, as a scalar: buffer resources are to be made of it
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int32_t)(v >> 32)) << 32) | (uint32_t)uniform((int32_t)v));
}

// 64 rows in LDS as bf16 planes, for fp32 three: splitting at every read, in
// every wave, took more time than the products (1237 tokens x 6 heads of 40 x
// 72 in fp32: the forward's walk 25.5 us, now 23.5). The two readings are RowTile's.
template <typename T, int W>
struct DecayTile {
    static constexpr int NX = kExact<T>;
    RowTile<uint16_t, W> p[NX];
    __device__ __forceinline__ void put(int i, int unit, const Unit<T>& u) {
        const Frag<NX> f = unit_planes(u);
#pragma unroll
        for (int x = 0; x < NX; ++x)
            *reinterpret_cast<u32x4*>(p[x].x + RowTile<uint16_t, W>::L::at(i, unit)) = __builtin_bit_cast(u32x4, f.p[x]);
    }
    __device__ __forceinline__ Frag<NX> frag(int token, int unit) const {
        Frag<NX> f;
#pragma unroll
        for (int x = 0; x < NX; ++x) f.p[x] = p[x].frag(token, unit).p[0];
        return f;
    }
    __device__ __forceinline__ Frag<NX> token_frag(int l, int s, int m) const {
        Frag<NX> f;
#pragma unroll
        for (int x = 0; x < NX; ++x) f.p[x] = p[x].token_frag(l, s, m).p[0];
        return f;
    }
};

// 64 rows of a side on their way to LDS, W columns of it
template <typename T, int W, int THREADS>
struct SideLoads {
    static constexpr int kN = kC * W / 8 / THREADS, kRows = THREADS / (W / 8);  // rows between a thread's units
    Unit<T> u[kN];
    __device__ __forceinline__ void load(const Side<T>& s, int64_t row, int n, int tid) {
        const auto r = rows_rsrc(s.p + row * s.stride, n, s.stride, s.width);
        const uint32_t at = s.at(tid / (W / 8), tid % (W / 8) * 8);
#pragma unroll
        for (int x = 0; x < kN; ++x) u[x].load(r, at + s.rows(x * kRows));
    }
    __device__ __forceinline__ void put(DecayTile<T, W>& t) const {
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int at = (int)(threadIdx.x % THREADS) + x * THREADS;
            t.put(at / (W / 8), at % (W / 8), u[x]);
        }
    }
};

// Tiles hold their columns as they come. Their reading of columns 16 m + n
// then gives columns 32 (m / 2) + 8 (n / 4) + 4 (m % 2) + n % 4, so that what
// tiles m = 2 i and 2 i + 1 of a result leave in a lane are eight rows that lie
// together, 32 i + 8 (l / 16) .. + 7: the order in which the next product takes
// its k, and columns of out that are stored together.
__device__ __forceinline__ int decay_col(int m, int n) { return (m >> 1) * 32 + (n >> 2) * 8 + (m & 1) * 4 + (n & 3); }

__device__ __forceinline__ void unit_values(const Unit<uint16_t>& u, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = bf16_to_f32(u.w[e]);
        v[2 * e + 1] = bf16_hi_to_f32(u.w[e]);
    }
}
__device__ __forceinline__ void unit_values(const Unit<float>& u, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = u.w[e >> 2][e & 3];
}
// the values that an operand's planes hold
__device__ __forceinline__ void frag_values(const Frag<1>& f, float (&v)[8]) {
    const u32x4 w = __builtin_bit_cast(u32x4, f.p[0]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[2 * e] = bf16_to_f32(w[e]);
        v[2 * e + 1] = bf16_hi_to_f32(w[e]);
    }
}
__device__ __forceinline__ void frag_values(const Frag<3>& f, float (&v)[8]) {
    float a[8], b[8];
    frag_values(Frag<1>{{f.p[2]}}, v);
    frag_values(Frag<1>{{f.p[1]}}, a);
    frag_values(Frag<1>{{f.p[0]}}, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (v[e] + a[e]) + b[e];
}

// d[ct][t] += x[ct] a[t], one plane product after the other over all tiles
template <int LIM, int NA, int NB, int CT>
__device__ __forceinline__ void decay_mma(f32x4 (&d)[CT][4], const Frag<NA> (&x)[CT], const Frag<NB> (&a)[4]) {
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        d[ct][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[ct].p[i], a[t].p[s - i], d[ct][t], 0, 0, 0);
}

__device__ __forceinline__ double wave_sum(double v) {
    v = dpp_add_f64<0xB1>(v);
    v = dpp_add_f64<0x4E>(v);
    v = dpp_add_f64<0x141>(v);
    v = dpp_add_f64<0x140>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// Of one chunk: G and its exponentials
struct DecayRows {
    double G[kC];
    float into[kC], onto[kC];     // decay from the state to a row, and from a row to the state
    float whole;                  // of the chunk
};
// Planes of P, of the state and of what is added to it: all 24 bits. (With two,
// cut off, 5 bf16 results in 1000 are not the nearest to the exact value, 2.1e-4
// of a tensor's norm; with three 0.12, 2.3e-5, as of any sums in 32 bits.)
constexpr int kPlanes = 3;
template <typename T, int DBP, int CT>
struct DecayTiles {
    DecayTile<T, DBP> a, b;
    DecayTile<T, 64 * CT> c;
    u32x4 P[8 * kPlanes][64];     // [row tile][block of 32 columns][plane]: as one lane reads them
    DecayRows rows[2];            // this chunk's and the next one's
    float dot[4][kC];             // by wave: dg's row sums
    double sum[2][4];             // the anchor and the chunk's sum
};

// One workgroup of four waves per (segment, value head, slice of the state's
// rows, column block), 16 CT columns a wave. In chunks of 64 rows:
//   out = into . (A X) + (D . A B^T) C,   X' = whole X + B^T (onto . C)
// The state's columns do not meet, so a wave keeps its own in registers; the
// decayed products P = D . A B^T are shared through LDS, a row tile from each
// wave. The products leave rows of the state as rows of a register, which is
// how the next product takes them (decay_col), and rows of out along the lanes.
// The next chunk's rows are under way in registers meanwhile, those of a in
// the first half of a chunk and those of b and c in the second, so that two
// workgroups share a CU. DOTS: rows of out times rows of q or k, for dg.
// What bounds it: 32768 tokens x 32 heads of 128 x 128 in bf16 take 296 to 325
// us forward, 220 at a copy's rate; copies of the walk that only compute take
// 292 to 303, that only load and store 252. With 16 key heads 296 to 311, 284 to
// 292 and 187 (164 at a copy's rate): its arithmetic bounds it. (Eight waves a
// workgroup of 16 columns each took no less.) In training dq 390 to 455, dk 440
// to 510, dv 305 to 365 (a launch takes longer as the clock falls under load).
// HEADS = 2 (dq, dk): both value heads of a key head in a workgroup of eight
// waves, which add up what they have formed, so that there are no parts: each
// four waves hand those rows to the others that the others store. (dk of 128 x
// 128 with dg spills 4 registers a lane in this form, none in the other.)
template <typename T, int KIND, int DBP, int CT, bool DOTS, int HEADS = 1>
__device__ __forceinline__ void decay_walk(const DecayArgs& p, int64_t block,
                                           DecayTiles<T, DBP, CT>* tiles) {
    constexpr int NX = kExact<T>, NP = kPlanes;
    constexpr bool REV = decay_reverse(KIND), SUM = KIND == kSumS || KIND == kSumD, KEYS = decay_by_key(KIND);
    constexpr int MT = DBP / 16, KS = DBP / 32, COLS = 64 * CT;
    // Vector operations of the next product in the shadow of one's matrix
    // instructions; dg's rows, or three planes of an input, leave no registers
    // for it.
    constexpr bool kAhead = !DOTS && NX == 1;
    constexpr int kFew = REV ? 3 : 0;  // the wave with the fewest tiles of P has G to do
    const int Dc = KEYS ? p.Dk : p.Dv, Db = KEYS ? p.Dv : p.Dk;
    const int ncb = (Dc + COLS - 1) / COLS, slices = KEYS ? p.slices : 1, group = p.Hv / p.Hk;
    const Spread sp = spread(block, group / HEADS * slices * ncb);  // (HEADS = 2: one group, one slice)
    const int mine = HEADS == 2 ? wave_id() >> 2 : 0;  // of the workgroup's heads
    DecayTiles<T, DBP, CT>& lds = tiles[mine];
    if (sp.group >= (p.T / p.seg + p.nseq) * (int64_t)p.Hk) return;
    Chunk sg;
    if (SUM ? !chunk_at(p.cu, p.nseq, p.T, sp.group / p.Hk, sg, p.seg) : !segment_at(p, sp.group / p.Hk, sg)) return;
    sg = {uniform(sg.start), uniform(sg.n), uniform(sg.seq), uniform(sg.index), uniform((int32_t)sg.last) != 0};
    if (SUM && (REV ? sg.index == 0 : sg.last)) return;
    const int hk = (int)(sp.group % p.Hk), cb = sp.member % ncb, slice = sp.member / ncb % slices;
    const int hv = hk * group + sp.member / (ncb * slices) * HEADS + mine;
    const int wave = HEADS == 2 ? wave_id() & 3 : wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    const int col0 = cb * COLS, off = slice * kDecayMaxDb, db = min(Db - off, DBP), parts = slices * ncb;
    const int64_t first = sg.start - sg.index * p.seg;    // of the sequence
    const int64_t state0 = first / p.seg + sg.index;      // of the state behind this segment
    // a and b by the heads that have them
    const void* const ta = KIND == kOut ? p.q : KIND == kDq ? p.dout : KIND == kDk ? p.v : p.k;
    const void* const tb = KIND == kOut || KIND == kSumS ? p.k : KIND == kDq ? p.v : KIND == kDk ? p.dout : p.q;
    const void* const tc = KIND == kOut || KIND == kSumS ? p.v : KIND == kDq ? p.k : KIND == kDk ? p.q : p.dout;
    const int Hb = KEYS ? p.Hv : p.Hk, hb = KEYS ? hv : hk, Hc = KEYS ? p.Hk : p.Hv, hc = KEYS ? hk : hv;
    const Side<T> sa(ta, sg.start, Hb, hb, Db, off, db), sb(tb, sg.start, Hb, hb, Db, off, db);
    const Side<T> sc(tc, sg.start, Hc, hc, Dc, col0, min(Dc - col0, COLS));
    // a lane's columns of out: 4 CT from here on
    const auto column = [&]() {
        const int quarter = (int)(fresh(l) >> 4);
        return col0 + (CT == 2 ? wave * 32 + quarter * 8 : (wave >> 1) * 32 + quarter * 8 + (wave & 1) * 4);
    };
    // The state in a tensor of [Dk][Dv], of which this workgroup has rows off ..
    // of b and columns col0 .. of c: a lane's elements at(m, ct, r), four rows
    // r of b together where b is v's or dout's
    f32x4 S[MT][CT] = {};
    const auto state_rsrc = [&](const float* base, int64_t n) {
        return bytes_rsrc(base + ((size_t)n * p.Hv + hv) * p.Dk * p.Dv, (uint32_t)(p.Dk * p.Dv) * 4u);
    };
    const auto at = [&](int m, int ct, int r) {
        const int row = decay_col(m, l4 * 4 + r), c = col0 + decay_col(wave * CT + ct, l16);
        return row < db && c < Dc ? (uint32_t)(KEYS ? c * p.Dv + off + row : (off + row) * p.Dv + c) * 4u : kNowhere;
    };
    const auto state_at = [&](__amdgpu_buffer_rsrc_t r, int m, int ct) {
        if constexpr (KEYS) return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at(m, ct, 0), 0, 0));
        f32x4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = Elt<float>::cvt(Elt<float>::raw_rsrc(r, at(m, ct, x)));
        return v;
    };
    const auto store_state = [&](const float* base, int64_t n) {
        const auto r = state_rsrc(base, n);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int x = 0; x < 4; ++x) Elt<float>::st_rsrc<0>(r, at(m, ct, x), S[m][ct][x]);
    };
    if constexpr (!SUM) {
        const auto from = [&](const float* base, int64_t n) {
            const auto r = state_rsrc(base, n);
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[m][ct] = state_at(r, m, ct);
        };
        const float* const given = REV ? p.dhT : p.h0;
        const bool inner = REV ? !sg.last : sg.index > 0;  // the state is another segment's
        if (inner && !p.few) from(p.joint[REV], REV ? state0 : state0 - 1);
        else if (given) from(given, sg.seq);
        if (inner && p.few) {  // what each segment on the way has added to the given one
            const int64_t all = first / p.seg;
            const int ends = uniform((int32_t)((seq_at(p.cu, sg.seq, p.T).len - 1) / p.seg));  // states between segments
            const int n = REV ? ends - (int)sg.index : (int)sg.index;
            for (int j = 0; j < n; ++j) {
                const int64_t at_j = all + (REV ? ends - 1 - j : j);
                const auto r = state_rsrc(p.joint[REV], at_j);
                const float d = p.seg_decay[REV][at_j * p.Hv + hv];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) S[m][ct] = S[m][ct] * d + state_at(r, m, ct);
            }
        }
    }
    const int chunks = (sg.n + kC - 1) / kC;
    SideLoads<T, DBP, 256> la, lb;
    SideLoads<T, COLS, 256> lc;
    uint32_t lg;
    const auto chunk = [&](int i) { return REV ? chunks - 1 - i : i; };  // the walk's i-th
    const auto tokens = [&](int i) { return i < chunks ? min(sg.n - chunk(i) * kC, kC) : 0; };
    const auto load_a = [&](int i) {
        const int n = tokens(i);
        if constexpr (!SUM) la.load(sa, (int64_t)chunk(i) * kC, n, wave * 64 + (int)fresh(l));
        const int64_t t = sg.start + chunk(i) * kC;
        lg = Elt<float>::raw_rsrc(rows_rsrc(p.g + (p.gstride ? t * p.gstride : 0) + hv, n, p.gstride, 1),
                                  l < n ? fresh(l) * (uint32_t)p.gstride * 4u : kNowhere);
    };
    const auto load_bc = [&](int i) {
        const int n = tokens(i);
        const int tid = wave * 64 + (int)fresh(l);
        lb.load(sb, (int64_t)chunk(i) * kC, n, tid);
        lc.load(sc, (int64_t)chunk(i) * kC, n, tid);
    };
    double total = 0.0;
    const auto put_rows = [&](int i) {
        if (wave != kFew || i >= chunks) return;
        DecayRows& to = lds.rows[i & 1];
        const double G = chunk_decay_sum(l < tokens(i) ? Elt<float>::cvt(lg) : 0.0f), last = read_lane(G, kC - 1);
        const int row = (int)fresh(l);
        to.G[row] = G;
        const float head = decay_of(G), tail = decay_of(last - G);
        to.into[row] = REV ? tail : head * p.scale;
        to.onto[row] = REV ? head * p.scale : tail;
        if (row == 0) to.whole = decay_of(last);
        total += last;
    };
    load_a(0);
    load_bc(0);
    if constexpr (!SUM) la.put(lds.a);
    lb.put(lds.b);
    lc.put(lds.c);
    put_rows(0);
    __syncthreads();
    for (int i = 0; i < chunks; ++i) {
        const int n = tokens(i), wv = fresh_scalar(wave), tid = wv * 64 + (int)fresh(l);  // or what follows from them fills registers

        const int64_t t0 = sg.start + chunk(i) * kC;
        const DecayRows& rows = lds.rows[i & 1];
        // dg's anchors: the state S^T of dq's walk behind every piece meets dS^T of dk's
        const int64_t from_seq = t0 - first, piece = first / kPiece + from_seq / kPiece;
        const bool piece_end = DOTS && (from_seq + kC) % kPiece == 0 && !(sg.last && chunk(i) == chunks - 1);
        const auto snap = [&]() {  // the wave's part of it; tile i lies 1024 i bytes on
            return bytes_rsrc(p.snap + (((size_t)piece * p.Hv + hv) * parts + slice * ncb + cb) * (DBP * COLS) +
                                  (size_t)wv * (MT * CT * 256), MT * CT * 1024);
        };
        Unit<T> dots[DOTS ? 4 : 1];
        if constexpr (DOTS) {
            const Side<T> sd(KIND == kDq ? p.q : p.k, t0, p.Hk, hk, p.Dk, 0, p.Dk);
            const auto r = rows_rsrc(sd.p, n, sd.stride, sd.width);
            const uint32_t at = sd.at(fresh(l16), column() & ~7);
#pragma unroll
            for (int t = 0; t < 4; ++t) dots[t].load(r, at + sd.rows(t * 16));
        }
        load_a(i + 1);
        if constexpr (DOTS && KIND == kDk) {
            if (piece_end) {
                double e = 0.0;
                const auto sr = snap();
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) {
                        const f32x4 w = __builtin_bit_cast(
                            f32x4, __builtin_amdgcn_raw_buffer_load_b128(sr, l * 16, (m * CT + ct) * 1024, 0));
#pragma unroll
                        for (int r = 0; r < 4; ++r) e = fma((double)S[m][ct][r], (double)w[r], e);
                    }
                e = wave_sum(e);
                if ((tid & 63) == 0) lds.sum[0][wv] = e;
            }
        }
        f32x4 o[CT][4] = {};
        // the lane's share of rows of out times rows of q or k, rows 16 t + l16
        const auto dot_of = [&](int t) {
            float v[8], e = 0.0f;
            unit_values(dots[DOTS ? t : 0], v);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if constexpr (CT == 2) e = fmaf(o[CT - 1][t][x], v[4 + x], fmaf(o[0][t][x], v[x], e));
                else {
                    const float lo = v[x], hi = v[4 + x];
                    e = fmaf(o[0][t][x], wv & 1 ? hi : lo, e);
                }
            }
            return e;
        };
        if constexpr (!SUM) {
            const int ml = (int)fresh((uint32_t)l), m16 = ml & 15, m4 = ml >> 4;  // addresses are this half's own
            // P: wave w has rows 16 w .. + 15 along its lanes
            f32x4 x[4] = {};
            const auto has = [&](int j) { return REV ? j >= wv : j <= wv; };  // row tile w meets rows of tile j of b
            {
                Frag<NX> fa[KS];
#pragma unroll
                for (int s = 0; s < KS; ++s) fa[s] = lds.a.frag(wv * 16 + m16, s * 4 + m4);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (has(j))
#pragma unroll
                        for (int s = 0; s < KS; ++s) mma<NX>(x[j], lds.b.frag(j * 16 + m16, s * 4 + m4), fa[s]);
            }
            const double Gi = rows.G[wv * 16 + m16];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (has(j)) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const double Gj = rows.G[j * 16 + m4 * 4 + r];
                        x[j][r] *= decay_of(REV ? Gj - Gi : Gi - Gj) * p.scale;
                    }
                    if (j == wv)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (REV ? m4 * 4 + r < m16 : m4 * 4 + r > m16) x[j][r] = 0.0f;
                }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (REV ? s == 0 && wv >= 2 : s == 1 && wv < 2) continue;
                const Frag<NP> f = split_tiles<NP>(x[2 * s], x[2 * s + 1]);
#pragma unroll
                for (int i = 0; i < NP; ++i) lds.P[(wv * 2 + s) * NP + i][ml] = __builtin_bit_cast(u32x4, f.p[i]);
            }
            // A X, rows of out along the lanes; in its shadow the state decays
            const float whole = rows.whole;
            Frag<NP> fs[CT], next[CT];
            const auto planes = [&](int s, Frag<NP> (&f)[CT]) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) f[ct] = split_tiles<NP>(S[2 * s][ct], S[2 * s + 1][ct]);
            };
            if constexpr (kAhead) planes(0, next);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                __builtin_amdgcn_sched_barrier(0);
                Frag<NX> fa[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) fa[t] = lds.a.frag(t * 16 + m16, s * 4 + m4);
                if constexpr (kAhead) {
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) fs[ct] = next[ct];
                    if (s + 1 < KS) planes(s + 1, next);
                } else {
                    planes(s, fs);
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    S[2 * s][ct] *= whole;
                    S[2 * s + 1][ct] *= whole;
                }
                decay_mma<NP>(o, fs, fa);
                if constexpr (kAhead) step_order<4, 4 * CT * NP, 4>();
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const float d = rows.into[t * 16 + m16];
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) o[ct][t] *= d;
            }
            if constexpr (DOTS) {
                double e = 0.0;
#pragma unroll
                for (int t = 0; t < 4; ++t) e += (double)dot_of(t);
                e = wave_sum(e);
                if ((tid & 63) == 0) lds.sum[1][wv] = e;
            }
            __syncthreads();
            if constexpr (DOTS) {
                const double* const w = lds.sum[tid & 1];
                const double e = (w[0] + w[1]) + (w[2] + w[3]);
                if (tid == 1)
                    p.chunk[REV][((size_t)(first / kC + sg.seq + from_seq / kC) * p.Hv + hv) * parts + slice * ncb + cb] = e;
                if (KIND == kDk && tid == 0 && piece_end)
                    p.meet[((size_t)(piece + sg.seq) * p.Hv + hv) * parts + slice * ncb + cb] = e;
            }
            la.put(lds.a);
        }
        load_bc(i + 1);
        put_rows(i + 1);
        if constexpr (SUM) {
            const float whole = rows.whole;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) S[m][ct] *= whole;
        }
        // P C and B^T (onto . C), 32 tokens at a time
        const int ml = (int)fresh((uint32_t)l);
        Frag<NX> fc[CT];
        Frag<3> fw[CT];
        const auto weigh = [&](int s) {
            const f32x4 w0 = *reinterpret_cast<const f32x4*>(rows.onto + s * 32 + (ml >> 4) * 4);
            const f32x4 w1 = *reinterpret_cast<const f32x4*>(rows.onto + s * 32 + 16 + (ml >> 4) * 4);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                float x[8];
                frag_values(fc[ct], x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] *= w0[e];
                    x[4 + e] *= w1[e];
                }
                fw[ct] = split8<3>(x);
            }
        };
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) fc[ct] = lds.c.token_frag(ml, s, wv * CT + ct);
            if constexpr (kAhead) weigh(s);
            if constexpr (!SUM) {
                constexpr int kFrom[2] = {0, REV ? 0 : 2}, kTo[2] = {REV ? 2 : 4, 4};  // row tiles that meet this block
                constexpr int kStep = kAhead ? 4 : 1;  // of them at a time
#pragma unroll
                for (int t0 = kFrom[s]; t0 < kTo[s]; t0 += kStep) {
                    Frag<NP> f[kStep];
#pragma unroll
                    for (int t = t0; t < t0 + kStep && t < kTo[s]; ++t)
#pragma unroll
                        for (int i = 0; i < NP; ++i)
                            f[t - t0].p[i] = __builtin_bit_cast(bf16x8, lds.P[(t * 2 + s) * NP + i][ml]);
#pragma unroll
                    for (int i = NP - 1; i >= 0; --i)
#pragma unroll
                        for (int j = 0; j < NX; ++j)
                            if (i + j < NP)
#pragma unroll
                                for (int t = t0; t < t0 + kStep && t < kTo[s]; ++t)
#pragma unroll
                                    for (int ct = 0; ct < CT; ++ct)
                                        o[ct][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fc[ct].p[j], f[t - t0].p[i],
                                                                                           o[ct][t], 0, 0, 0);
                }
            }
            if constexpr (!kAhead) {
                __builtin_amdgcn_sched_barrier(0);
                weigh(s);
            }
            __builtin_amdgcn_sched_barrier(0);
            Frag<NX> fb[2] = {lds.b.token_frag(ml, s, 0), lds.b.token_frag(ml, s, 1)};
#pragma unroll
            for (int m = 0; m < MT; m += 2) {
                Frag<NX> now[2] = {fb[0], fb[1]};
                if (m + 2 < MT) {
                    fb[0] = lds.b.token_frag(ml, s, m + 2);
                    fb[1] = lds.b.token_frag(ml, s, m + 3);
                }
#pragma unroll
                for (int i = 2; i >= 0; --i)
#pragma unroll
                    for (int j = 0; j < NX; ++j)
                        if (i + j < 3)
#pragma unroll
                            for (int y = 0; y < 2; ++y)
#pragma unroll
                                for (int ct = 0; ct < CT; ++ct)
                                    S[m + y][ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now[y].p[j], fw[ct].p[i], S[m + y][ct], 0, 0, 0);
                if constexpr (!kAhead) __builtin_amdgcn_sched_barrier(0);  // or reads pile up in registers
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        // rows from .. from + 16 N - 1 of the result
        const auto store = [&](const auto& y, int from) {
            constexpr int N = 4 / HEADS;
            const int H = KEYS ? p.Hk : p.Hv, h = KEYS ? hk : hv, members = HEADS == 2 ? 1 : group * slices;
            if (KEYS && members > 1) {
                const Side<float> to(p.part[REV], t0, H * members, h * members + sp.member / ncb, Dc, 0, Dc);
                const auto r = rows_rsrc(to.p, n, to.stride, Dc);
                const uint32_t at = to.at(fresh(l16), column()) + to.rows(from);
#pragma unroll
                for (int t = 0; t < N; ++t)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y[ct][t]), r,
                                                               (int)(at + to.rows(t * 16) + ct * 16), 0, 0);
                return;
            }
            const Side<T> to(KIND == kOut ? p.out : KIND == kDq ? p.dq : KIND == kDk ? p.dk : p.dv, t0, H, h, Dc, 0, Dc);
            const auto r = rows_rsrc(to.p, n, to.stride, Dc);
            const uint32_t at = to.at(fresh(l16), column()) + to.rows(from);
#pragma unroll
            for (int t = 0; t < N; ++t) {
                const f32x4 x = y[0][t], z = y[CT - 1][t];
                if constexpr (CT == 2) {
                    Unit<T> u;
                    u.pack({x[0], x[1], x[2], x[3], z[0], z[1], z[2], z[3]});
                    u.store(r, at + to.rows(t * 16));
                } else if constexpr (NX == 3) {
                    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, (int)(at + to.rows(t * 16)), 0, 0);
                } else {
                    const u32x2 w = {(uint32_t)f32_to_bf16(x[0]) | ((uint32_t)f32_to_bf16(x[1]) << 16),
                                     (uint32_t)f32_to_bf16(x[2]) | ((uint32_t)f32_to_bf16(x[3]) << 16)};
                    __builtin_amdgcn_raw_buffer_store_b64(w, r, (int)(at + to.rows(t * 16)), 0, 0);
                }
            }
        };
        if constexpr (!SUM) {
            if constexpr (HEADS == 1) store(o, 0);
            if constexpr (DOTS) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    float e = dot_of(t);
                    e += __shfl_xor(e, 16);
                    e += __shfl_xor(e, 32);
                    if ((tid & 48) == 0) lds.dot[wv][t * 16 + l16] = e;
                }
                if constexpr (KIND == kDq) {
                    if (piece_end) {
                        const auto sr = snap();
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int ct = 0; ct < CT; ++ct)
                                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[m][ct]), sr, l * 16,
                                                                       (m * CT + ct) * 1024, 0);
                    }
                }
            }
        }
        __syncthreads();
        if constexpr (HEADS == 2) {  // P has been read: row tiles that the other head's waves store, at their places
            u32x4* const give = &lds.P[0][0] + tid;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    give[(t * CT + ct) * 256] = __builtin_bit_cast(u32x4, mine ? o[ct][t] : o[ct][2 + t]);
        }
        lb.put(lds.b);
        lc.put(lds.c);
        if constexpr (DOTS) {
            if (wv == 0) {
                const auto r = rows_rsrc(p.rows[REV] + ((size_t)(slice * ncb + cb) * p.T + t0) * p.Hv + hv, n, p.Hv, 1);
                Elt<float>::st_rsrc<0>(r, (uint32_t)(tid * p.Hv) * 4u,
                                       (lds.dot[0][tid] + lds.dot[1][tid]) + (lds.dot[2][tid] + lds.dot[3][tid]));
            }
        }
        __syncthreads();
        if constexpr (HEADS == 2) {
            const u32x4* const take = &tiles[mine ^ 1].P[0][0] + tid;
            f32x4 y[CT][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
                    y[ct][t] = __builtin_bit_cast(f32x4, take[(t * CT + ct) * 256]) + (mine ? o[ct][2 + t] : o[ct][t]);
            __syncthreads();  // before the next P
            store(y, mine * 32);
        }
    }
    if constexpr (SUM) {
        store_state(p.joint[REV], state0 - REV);
        if (wave == kFew && l == 0 && cb == 0) p.seg_decay[REV][(size_t)(state0 - REV) * p.Hv + hv] = decay_of(total);
    } else if constexpr (KIND == kOut) {
        if (p.hT && sg.last) store_state(p.hT, sg.seq);
    } else if constexpr (KIND == kDv) {
        if (p.dh0 && sg.index == 0) store_state(p.dh0, sg.seq);
    } else if constexpr (DOTS && KIND == kDq) {
        if (p.dhT && sg.last) {  // the last piece's anchor
            const auto r = state_rsrc(p.dhT, sg.seq);
            double e = 0.0;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    const f32x4 w = state_at(r, m, ct);
#pragma unroll
                    for (int x = 0; x < 4; ++x) e = fma((double)S[m][ct][x], (double)w[x], e);
                }
            e = wave_sum(e);
            if (l == 0) lds.sum[0][wave] = e;
            __syncthreads();
            const int64_t len = sg.start - first + sg.n;
            if (threadIdx.x % 256 == 0 && len > 0)
                p.meet[((size_t)(first / kPiece + sg.seq + (len - 1) / kPiece) * p.Hv + hv) * parts + slice * ncb + cb] =
                    (lds.sum[0][0] + lds.sum[0][1]) + (lds.sum[0][2] + lds.sum[0][3]);
        }
    }
}

template <typename T, int KIND, int DBP, int CT, bool DOTS>
__global__ __launch_bounds__(256, kExact<T> == 1 ? 2 : 1) void k_decay_walk(DecayArgs p) {
    __shared__ alignas(16) DecayTiles<T, DBP, CT> lds;
    decay_walk<T, KIND, DBP, CT, DOTS>(p, blockIdx.x, &lds);
}
template <int KIND, int DBP, int CT, bool DOTS>
__global__ __launch_bounds__(512, 2) void k_decay_heads(DecayArgs p) {
    __shared__ alignas(16) DecayTiles<uint16_t, DBP, CT> lds[2];
    decay_walk<uint16_t, KIND, DBP, CT, DOTS, 2>(p, blockIdx.x, lds);
}
// Two walks that do not wait for each other in one launch, the first in the
// first `blocks` workgroups, where all of them have a CU of their own: small
// ones then run beside each other. (Compiled together they need more registers
// than two workgroups a CU have: a backward of 32768 tokens x 32 heads of 128 x
// 128 takes 1487 us with dk and dv in one launch, 1306 one after the other.)
constexpr int kPairBlocks = 512;  // half of them, or more, without a segment
template <typename T, int KIND, int DBP, int CT, bool DOTS, int KIND2, int DBP2, int CT2>
__global__ __launch_bounds__(256, 1) void k_decay_pair(DecayArgs p, uint32_t blocks) {
    using A = DecayTiles<T, DBP, CT>;
    using B = DecayTiles<T, DBP2, CT2>;
    __shared__ alignas(16) char lds[sizeof(A) > sizeof(B) ? sizeof(A) : sizeof(B)];
    if (blockIdx.x < blocks) decay_walk<T, KIND, DBP, CT, DOTS>(p, blockIdx.x, reinterpret_cast<A*>(lds));
    else decay_walk<T, KIND2, DBP2, CT2, false>(p, blockIdx.x - blocks, reinterpret_cast<B*>(lds));
}

// Along the segments of each sequence that has several, in place: what a
// segment adds becomes the state on its far side, X' = decay X + U. A workgroup
// per (sequence, head, block of elements): each element is read and written
// once, kBatch states under way.
template <bool REV>
__device__ __forceinline__ void decay_join(const DecayArgs& p, int s, int hv, int block, int blocks) {
    const Seq q = seq_at(p.cu, s, p.T);
    const int n = (q.len - 1) / p.seg;  // states between its segments
    if (q.len == 0 || n == 0) return;
    const int64_t state0 = q.start / p.seg;
    const size_t size = (size_t)p.Dk * p.Dv, step = size * p.Hv;
    float* const x = p.joint[REV] + (size_t)state0 * step + hv * size;
    const float* const d = p.seg_decay[REV] + state0 * p.Hv + hv;
    const float* first = REV ? p.dhT : p.h0;
    if (first) first += ((size_t)s * p.Hv + hv) * size;
    for (size_t e = ((size_t)block * 256 + threadIdx.x) * 4; e < size; e += (size_t)blocks * 1024) {
        f32x4 v = first ? *reinterpret_cast<const f32x4*>(first + e) : f32x4{0, 0, 0, 0};
        constexpr int kBatch = 8;
        for (int i = 0; i < n; i += kBatch) {
            f32x4 u[kBatch];
            float w[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int at = min(i + j, n - 1), to = REV ? n - 1 - at : at;
                u[j] = *reinterpret_cast<const f32x4*>(x + to * step + e);
                w[j] = d[to * p.Hv];
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                if (i + j < n) {
                    v = v * w[j] + u[j];
                    *reinterpret_cast<f32x4*>(x + (REV ? n - 1 - i - j : i + j) * step + e) = v;
                }
        }
    }
}
// ways: 1 for S alone, 2 for dS as well
template <int kUnused = 0>
__global__ __launch_bounds__(256) void k_decay_join(DecayArgs p, int blocks, int ways) {
    const int64_t i = blockIdx.x / ways;
    const int s = (int)(i / ((int64_t)p.Hv * blocks)), hv = (int)(i / blocks % p.Hv), block = (int)(i % blocks);
    if (ways == 1 || blockIdx.x % 2 == 0) decay_join<false>(p, s, hv, block, blocks);
    else decay_join<true>(p, s, hv, block, blocks);
}

// Columns of c that a workgroup takes, in tiles of 16 a wave: two, or one where
// there are no more or where fp32's planes of rows over 64 leave LDS for no more
template <typename T>
constexpr int decay_tiles(bool wide_b, bool wide_c) {
    return wide_c && !(kExact<T> == 3 && wide_b) ? 2 : 1;
}
inline int decay_blocks_of(int32_t Db, int32_t Dc, int32_t dtype) {
    const int cols = 64 * (dtype == SSMP_F32 ? decay_tiles<float>(Db > 64, Dc > 64) : decay_tiles<uint16_t>(Db > 64, Dc > 64));
    return (Dc + cols - 1) / cols;
}
// The walks' workgroups, by kind: those of heads that share a and b, or c, on
// one XCD.
inline int64_t decay_walk_blocks(const DecayArgs& a, int kind, int32_t dtype, int heads = 1) {
    const bool keys = decay_by_key(kind);
    const int blocks = keys ? a.slices * decay_blocks_of(a.Dv, a.Dk, dtype) : decay_blocks_of(a.Dk, a.Dv, dtype);
    return spread_blocks((a.T / a.seg + a.nseq) * a.Hk, a.Hv / a.Hk / heads * blocks);
}
// f(fp32, Dk over 64, Dv over 64), as constants
template <typename F>
void decay_dispatch(const DecayArgs& a, int32_t dtype, F f) {
    using Y = std::true_type;
    using N = std::false_type;
    const auto with = [&](auto t) {
        if (a.Dk > 64) a.Dv > 64 ? f(t, Y{}, Y{}) : f(t, Y{}, N{});
        else a.Dv > 64 ? f(t, N{}, Y{}) : f(t, N{}, N{});
    };
    if (dtype == SSMP_F32) with(Y{});
    else with(N{});
}
template <int KIND, bool WK, bool WV, typename T>
struct DecayForm {  // of a walk, for heads of Dk and Dv over 64 or not
    static constexpr bool B = decay_by_key(KIND) ? WV : WK, C = decay_by_key(KIND) ? WK : WV;
    static constexpr int DBP = B ? 128 : 64, CT = decay_tiles<T>(B, C);
};
template <bool FP32>
using DecayType = typename std::conditional<FP32, float, uint16_t>::type;
template <int KIND, bool DOTS>
int launch_decay_walk(const DecayArgs& a, int32_t dtype, hipStream_t s) {
    if constexpr (decay_by_key(KIND)) {
        if (a.heads == 2) {
            const unsigned n = (unsigned)decay_walk_blocks(a, KIND, dtype, 2);
            decay_dispatch(a, SSMP_BF16, [&](auto, auto wk, auto wv) {
                using F = DecayForm<KIND, decltype(wk)::value, decltype(wv)::value, uint16_t>;
                k_decay_heads<KIND, F::DBP, F::CT, DOTS><<<n, 512, 0, s>>>(a);
            });
            SSMP_LAUNCH_CHECK();
            return SSMP_OK;
        }
    }
    const unsigned n = (unsigned)decay_walk_blocks(a, KIND, dtype);
    decay_dispatch(a, dtype, [&](auto fp32, auto wk, auto wv) {
        using T = DecayType<decltype(fp32)::value>;
        using F = DecayForm<KIND, decltype(wk)::value, decltype(wv)::value, T>;
        k_decay_walk<T, KIND, F::DBP, F::CT, DOTS><<<n, 256, 0, s>>>(a);
    });
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
// Both walks, beside each other where they are small
template <int KIND, bool DOTS, int KIND2>
int launch_decay_pair(const DecayArgs& a, int32_t dtype, hipStream_t s) {
    const unsigned n = (unsigned)decay_walk_blocks(a, KIND, dtype), m = n + (unsigned)decay_walk_blocks(a, KIND2, dtype);
    if (m > kPairBlocks || (decay_by_key(KIND) && a.heads == 2)) {
        if (const int st = launch_decay_walk<KIND, DOTS>(a, dtype, s)) return st;
        return launch_decay_walk<KIND2, false>(a, dtype, s);
    }
    decay_dispatch(a, dtype, [&](auto fp32, auto wk, auto wv) {
        using T = DecayType<decltype(fp32)::value>;
        using F = DecayForm<KIND, decltype(wk)::value, decltype(wv)::value, T>;
        using G = DecayForm<KIND2, decltype(wk)::value, decltype(wv)::value, T>;
        k_decay_pair<T, KIND, F::DBP, F::CT, DOTS, KIND2, G::DBP, G::CT><<<m, 256, 0, s>>>(a, n);
    });
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
// Up to so many states between segments are added up by the walks themselves,
// each reading those on its way: a prompt of 513 tokens x 32 heads of 128 x 128
// in 5 segments takes 38 us with a join between the walks and 29 without.
constexpr int kFewStates = 5;
inline int launch_decay_join(const DecayArgs& a, int ways, hipStream_t s) {
    if (a.few) return SSMP_OK;
    const int64_t per = ((int64_t)a.Dk * a.Dv + 1023) / 1024;  // blocks of an element a thread
    int64_t blocks = 2048 / ((int64_t)a.nseq * a.Hv);
    blocks = blocks < 1 ? 1 : blocks > per ? per : blocks;
    k_decay_join<><<<(unsigned)((int64_t)a.nseq * a.Hv * blocks * ways), 256, 0, s>>>(a, (int)blocks, ways);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}
// Both value heads of a key head in a workgroup, where there are two, and more
// workgroups than the card has at a time: no parts are written and added up,
// while eight waves in step take about a fifth longer. Backward, in us, with
// one head a workgroup and with two; above the rule's border
//   tokens, sequences    2048, 8   4096, 8   8192, 8   32768, 35
//   32 heads 128 x 128   174, 161  333, 297  519, 467  1560, 1420
//   others: 16384, 1, 16 of 128 x 64: 403, 326; 8192, 8, 32 of 64 x 64: 245,
//   228; 32768, 29, 32 of 64 x 64: 795, 770; 8192, 8, 8 of 128 x 128: 184, 174
// and below it
//   513, 1, 32 of 128 x 128: 91, 125; 1024, 2, 16 of 128 x 128: 86, 114; 1024, 1,
//   8 of 128 x 64: 68, 86; 1237, 12, 8 of 64 x 64: 51, 64; 600, 20, 8 of 128 x
//   128: 50, 53
// (Two of 24 heads, which halves the parts: 16384, 8, of 128 x 64: 568, 551;
// 4096: 191, 198; 32768: 995, 1013. fp32 walks have no room for it.)
inline int decay_heads_of(const DecayArgs& a, int32_t dtype) {
    if (dtype == SSMP_F32 || a.Hv != 2 * a.Hk || a.slices > 1) return 1;
    return decay_walk_blocks(a, kDk, dtype) + decay_walk_blocks(a, kDv, dtype) > kPairBlocks ? 2 : 1;
}
// compiled in sources of their own
int launch_decay_dq(const DecayArgs& a, int32_t dtype, hipStream_t s);
int launch_decay_dkv(const DecayArgs& a, int32_t dtype, hipStream_t s);

inline int decay_check(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype) {
    if (const int st = delta_check(T, nseq, Hk, Hv, Dk, Dv, dtype)) return st;
    const int64_t slices = (Dv + kDecayMaxDb - 1) / kDecayMaxDb;
    if (Hv * slices * Dk > kMaxRow) return SSMP_ERR_SHAPE;  // a row of dq's parts
    // a walk's workgroups: segments of kSegMin at least, blocks of 64 columns or more
    if ((T / kSegMin + nseq + 7) * (int64_t)Hv * slices * 2 >= kMaxBlocks) return SSMP_ERR_SHAPE;
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
