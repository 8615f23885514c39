// What the forward and the backward of the gated delta rule make of every chunk
// before they go along the sequences: nothing here depends on the states.
#pragma once

#include "delta_common.h"

namespace ssmp {

// The sequences by chunks, most first, for the chains: a chain takes as long as
// its sequence, and a long one that starts last is waited for alone. Sorted by
// counting in one workgroup beside those that prepare the chunks; the order
// among equals is left to chance and changes no result. h: 2048 ints of LDS.
constexpr int kOrderMax = 4096;  // sequences one workgroup sorts beside the others; more start as they lie
__device__ __forceinline__ void order_sequences(const DeltaArgs& a, int* h) {
    constexpr int kBins = 1024;
    const int tid = threadIdx.x;
    const auto bin = [&](int s) {
        const int n = (seq_at(a.cu, s, a.T).len + kC - 1) / kC;
        return kBins - 1 - (n < kBins ? n : kBins - 1);
    };
    for (int i = tid; i < kBins; i += 256) h[i] = 0;
    __syncthreads();
    for (int s = tid; s < a.nseq; s += 256) atomicAdd(&h[bin(s)], 1);
    __syncthreads();
    int own = 0;  // of four bins
    for (int i = 0; i < 4; ++i) own += h[tid * 4 + i];
    h[kBins + tid] = own;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < tid; ++i) before += h[kBins + i];
    for (int i = 0; i < 4; ++i) {
        const int n = h[tid * 4 + i];
        h[tid * 4 + i] = before;
        before += n;
    }
    __syncthreads();
    for (int s = tid; s < a.nseq; s += 256) a.order[atomicAdd(&h[bin(s)], 1)] = s;
}

// One workgroup per (slot, value head); the heads of a group run on one XCD,
// whose L2 then holds their keys and queries.
//   forward:  (I + L diag(beta))^-1 and P,           both lower triangular
//   backward: (I + diag(beta) L)^-T and scale P^T,   both upper triangular
// The inverse is one dependent sequence of small products, which four
// workgroups a CU hide from each other: 175 us forward, 183 us backward for
// 32768 tokens x 32 heads of 128 in bf16, 0.76 GB at 4.2 TB/s.
template <typename T, int DKP, bool BWD>
__global__ __launch_bounds__(256, kExact<T> == 1 ? 4 : 1) void k_delta_prepare(DeltaArgs a) {
    constexpr int NX = kExact<T>;
    using Rows = Tile<T, DKP>;
    constexpr int kKeys = kC * DKP * (int)sizeof(T), kMats = kC * kLdA * 4;
    // keys and queries; then, once they are multiplied, the matrix and its inverse
    __shared__ alignas(16) char lds[2 * (kKeys > kMats ? kKeys : kMats)];
    __shared__ double G[kC];
    __shared__ float beta[kC];
    T* const Kl = reinterpret_cast<T*>(lds);
    T* const Ql = Kl + kC * DKP;
    float* const A = reinterpret_cast<float*>(lds);
    float* const X = A + kC * kLdA;
    if (a.order && blockIdx.x == gridDim.x - 1) return order_sequences(a, reinterpret_cast<int*>(lds));
    const int members = a.Hv / a.Hk;
    const Spread sp = spread(blockIdx.x, members);
    const int64_t slots = delta_slots(a.T, a.nseq);
    if (sp.group >= slots * a.Hk) return;
    const int64_t slot = sp.group / a.Hk;
    const int hk = (int)(sp.group % a.Hk), hv = hk * members + sp.member;
    Chunk c;
    if (!chunk_at(a.cu, a.nseq, a.T, slot, c)) return;
    const int tid = threadIdx.x, wave = wave_id(), l = lane_id(), l16 = l & 15, l4 = l >> 4;
    const size_t sh = (size_t)slot * a.Hv + hv;
    constexpr int kUnits = DKP / 8, kN = kC * kUnits / 256;
    // every load is under way before the first is waited for
    const auto brows = rows_rsrc(a.beta + (size_t)c.start * a.Hv + hv, c.n, a.Hv, 1);
    const auto grows = rows_rsrc(a.g + (size_t)c.start * a.Hv + hv, c.n, a.Hv, 1);
    const uint32_t gl = Elt<float>::raw_rsrc(grows, (uint32_t)(l * a.Hv) * 4u);
    const uint32_t bl = Elt<float>::raw_rsrc(brows, (uint32_t)(l * a.Hv) * 4u);
    const size_t from = ((size_t)c.start * a.Hk + hk) * a.Dk;
    const int stride = a.Hk * a.Dk;
    const auto krows = rows_rsrc(static_cast<const T*>(a.k) + from, c.n, stride, a.Dk);
    const auto qrows = rows_rsrc(static_cast<const T*>(a.q) + from, c.n, stride, a.Dk);
    Unit<T> ku[kN], qu[kN];
#pragma unroll
    for (int x = 0; x < kN; ++x) {
        const int u = tid + x * 256, i = u / kUnits, k8 = u % kUnits;
        const uint32_t o = k8 * 8 < a.Dk ? (uint32_t)(i * stride + k8 * 8) * (uint32_t)sizeof(T) : kNowhere;
        ku[x].load(krows, o);
        qu[x].load(qrows, o);
    }
    if (wave == 0) {
        const double s = chunk_decay_sum(Elt<float>::cvt(gl));
        G[l] = s;
        beta[l] = Elt<float>::cvt(bl);
        const double last = read_lane(s, kC - 1);
        reinterpret_cast<double*>(a.dec + sh * kDec)[l] = s;
        a.dec[sh * kDec + 2 * kC + l] = decay_of(s);
        a.dec[sh * kDec + 3 * kC + l] = decay_of(last - s);
    }
#pragma unroll
    for (int x = 0; x < kN; ++x) {
        const int u = tid + x * 256, at = Rows::at(u / kUnits, u % kUnits);
        ku[x].put_half(Kl + at, 0);
        ku[x].put_half(Kl + at + 4, 1);
        qu[x].put_half(Ql + at, 0);
        qu[x].put_half(Ql + at + 4, 1);
    }
    __syncthreads();
    // The products' 16 x 16 tiles that hold anything are five for each wave:
    //   forward:  K K^T rows w, columns 0 .. w; K Q^T rows w, columns w .. 3
    //   backward: Q K^T rows w, columns 0 .. w; K K^T rows 3 - w, columns 0 .. 3 - w
    // (K Q^T, as a lane then holds four contiguous keys of one query's row; in
    // the backward four queries of one key.) Which is which is a matter of
    // addresses, so that no tile hangs on a branch.
    const auto first = [&](int t) { return t <= wave; };  // of the two products
    const auto tile_row = [&](int t) { return BWD && !first(t) ? 3 - wave : wave; };
    const auto tile_col = [&](int t) { return first(t) ? t : (BWD ? t - wave - 1 : t - 1); };
    f32x4 acc[5] = {};
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
        const int u = s * 4 + l4;
        Frag<NX> fa[2], fb[5];
        fa[0] = tile_frag((BWD ? Ql : Kl) + Rows::at(wave * 16 + l16, u));
        fa[1] = BWD ? tile_frag(Kl + Rows::at((3 - wave) * 16 + l16, u)) : fa[0];
#pragma unroll
        for (int t = 0; t < 5; ++t)
            fb[t] = tile_frag((BWD || first(t) ? Kl : Ql) + Rows::at(tile_col(t) * 16 + l16, u));
#pragma unroll
        for (int t = 0; t < 5; ++t) mma<NX>(acc[t], first(t) ? fa[0] : fa[1], fb[t]);
    }
    __syncthreads();
    float* const att = a.att + sh * kTri;
#pragma unroll
    for (int t = 0; t < 5; ++t) {
        const int i0 = tile_row(t) * 16 + l4 * 4, j = tile_col(t) * 16 + l16;
        if (first(t) != BWD) {  // K K^T: rows are later tokens
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + r;
                A[i * kLdA + j] = i > j ? (BWD ? beta[i] : beta[j]) * decay_of(G[i] - G[j]) * acc[t][r] : 0.0f;
            }
        } else {
            f32x4 p;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = i0 + r;
                if constexpr (BWD) p[r] = i >= j ? decay_of(G[i] - G[j]) * acc[t][r] * a.scale : 0.0f;
                else p[r] = j >= i ? decay_of(G[j] - G[i]) * acc[t][r] : 0.0f;
            }
            *reinterpret_cast<f32x4*>(att + tri_row<BWD>(j, i0) * 32 + (kplace(i0) & 31)) = p;
        }
    }
    // the two empty tiles in the stored blocks
    if ((wave & 1) != BWD) {
        const int row = (BWD ? wave + 1 : wave - 1) * 16 + l16, k = wave * 16 + l4 * 4;
        *reinterpret_cast<f32x4*>(att + tri_row<BWD>(row, k) * 32 + (kplace(k) & 31)) = f32x4{0, 0, 0, 0};
    }
    __syncthreads();
    chunk_inverse(A, X);
    float* const inv = a.inv + sh * kTri;
    for (int e = tid; e < kTri / 4; e += 256) {
        const int t = e >> 3, q = e & 7;
        const bool second = t >= 64;  // place q of block: k = 4 g, g = q / 2 + 4 (q % 2)
        const int row = BWD ? (second ? t - 64 : t) : (second ? t - 32 : t);
        const int k = (BWD != second ? 32 : 0) + ((q >> 1) + (q & 1) * 4) * 4;
        f32x4 v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = BWD ? X[(k + x) * kLdA + row] : X[row * kLdA + k + x];
        *reinterpret_cast<f32x4*>(inv + t * 32 + q * 4) = v;
    }
}

template <typename T, int DKP, bool BWD>
int launch_delta_prepare(const DeltaArgs& a, hipStream_t s) {
    const int64_t blocks = spread_blocks(delta_slots(a.T, a.nseq) * a.Hk, a.Hv / a.Hk) + (a.order ? 1 : 0);
    k_delta_prepare<T, DKP, BWD><<<(unsigned)blocks, 256, 0, s>>>(a);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

// ---------------------------------------------------------------------------
// The operands of one chunk that a chain holds in LDS for all its waves, and
// the registers in which the next chunk's are under way meanwhile: keys and
// queries, the inverse and the products. 68 KB for bf16 heads of 128.
template <typename T, int DKP>
struct ChainTiles {
    RowTile<T, DKP> k, q;
    __bf16 inv[3 * kTri];
    __bf16 att[3 * kTri];
    float eg[kC], el[kC], beta[kC];
};

// Where the operands of a chain's chunks lie; they go on by the same step
// from chunk to chunk, which costs a scalar addition each.
template <typename T>
struct ChainAt {
    const T *k, *q;
    const float *inv, *att, *dec, *beta;

    __device__ __forceinline__ ChainAt(const DeltaArgs& a, int64_t slot, int64_t start, int hk, int hv) {
        const size_t sh = (size_t)slot * a.Hv + hv, row = ((size_t)start * a.Hk + hk) * a.Dk;
        k = static_cast<const T*>(a.k) + row;
        q = static_cast<const T*>(a.q) + row;
        inv = a.inv + sh * kTri;
        att = a.att + sh * kTri;
        dec = a.dec + sh * kDec + 2 * kC;
        beta = a.beta + (size_t)start * a.Hv + hv;
    }
    __device__ __forceinline__ void step(const DeltaArgs& a, int chunks) {
        k += (int64_t)chunks * kC * a.Hk * a.Dk;
        q += (int64_t)chunks * kC * a.Hk * a.Dk;
        inv += (int64_t)chunks * a.Hv * kTri;
        att += (int64_t)chunks * a.Hv * kTri;
        dec += (int64_t)chunks * a.Hv * kDec;
        beta += (int64_t)chunks * kC * a.Hv;
    }
};

template <typename T, int DKP, int THREADS>
struct ChainLoads {
    using Tiles = ChainTiles<T, DKP>;
    static constexpr int kN = DKP * kC / 8 / THREADS;                         // units of 8 elements a thread
    static constexpr int kM = (kTri / 4 + THREADS - 1) / THREADS;             // units of 4 of a triangle
    static __device__ __forceinline__ bool tri_on(int x) {
        return (x + 1) * THREADS <= kTri / 4 || threadIdx.x + x * THREADS < kTri / 4;
    }
    Unit<T> k[kN], q[kN];
    Unit<float4> inv[kM], att[kM];
    uint32_t dec, beta;

    // The chunk of n tokens at `p` (n <= 0: none, all zeros). The loads are
    // the same in every wave and on every path, so that a wait for an older
    // load can count the ones behind it and need not wait for these too.
    __device__ __forceinline__ void load_rows(const DeltaArgs& a, const ChainAt<T>& p, int n) {
        const int stride = a.Hk * a.Dk;
        const auto kr = rows_rsrc(p.k, n, stride, a.Dk), qr = rows_rsrc(p.q, n, stride, a.Dk);
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int u = threadIdx.x + x * THREADS, i = u / (DKP / 8), k8 = u % (DKP / 8);
            const uint32_t o = k8 * 8 < a.Dk ? (uint32_t)(i * stride + k8 * 8) * (uint32_t)sizeof(T) : kNowhere;
            k[x].load(kr, o);
            q[x].load(qr, o);
        }
    }
    __device__ __forceinline__ void load_rest(const DeltaArgs& a, const ChainAt<T>& p, int n) {
        const int tid = threadIdx.x;
        const auto ir = bytes_rsrc(p.inv, n > 0 ? kTri * 4 : 0), ar = bytes_rsrc(p.att, n > 0 ? kTri * 4 : 0);
#pragma unroll
        for (int x = 0; x < kM; ++x) {
            inv[x].load(ir, (uint32_t)(tid + x * THREADS) * 16u);
            att[x].load(ar, (uint32_t)(tid + x * THREADS) * 16u);
        }
        dec = Elt<float>::raw_rsrc(bytes_rsrc(p.dec, n > 0 ? 2 * kC * 4 : 0), (uint32_t)tid * 4u);
        beta = Elt<float>::raw_rsrc(rows_rsrc(p.beta, n, a.Hv, 1),
                                    tid < 2 * kC ? kNowhere : (uint32_t)((tid - 2 * kC) * a.Hv) * 4u);
    }
    __device__ __forceinline__ void put_rows(Tiles& t) const {
#pragma unroll
        for (int x = 0; x < kN; ++x) {
            const int u = threadIdx.x + x * THREADS, i = u / (DKP / 8), k8 = u % (DKP / 8);
            t.k.put(i, k8, k[x]);
            t.q.put(i, k8, q[x]);
        }
    }
    __device__ __forceinline__ void put_rest(Tiles& t) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int x = 0; x < kM; ++x)
            if (tri_on(x)) {
                tri_put4<3>(t.inv, tid + x * THREADS, inv[x].w);
                tri_put4<3>(t.att, tid + x * THREADS, att[x].w);
            }
        if (tid < kC) t.eg[tid] = Elt<float>::cvt(dec);
        else if (tid < 2 * kC) t.el[tid - kC] = Elt<float>::cvt(dec);
        else if (tid < 3 * kC) t.beta[tid - 2 * kC] = Elt<float>::cvt(beta);
    }
};

// Sets of a chain's operands in LDS: two where they fit and cost no workgroup
// beside it, so that the next chunk's are put while this one's are read and a
// chunk has one barrier. Against one set, keeping / backward, heads of 128 in
// bf16 (us): 8 waves, 16 sequences of 2048 tokens x 32 heads, 670 / 634 against
// 789 / 698; 4 waves, 6 sequences of 2731 x 12, 275 / 258 against 274 / 271;
// one of 513 tokens x 32 heads 49 / 46 against 49 / 48.
template <typename Tiles, int DKP, int NW>
constexpr int kSets = 2 * sizeof(Tiles) <= 160 * 1024 && (DKP > 64 || NW == 8) ? 2 : 1;

// Waves of a chain's workgroup. Eight (128 columns) read a chunk's operands
// once for a whole head and give each SIMD two waves, one of which works while
// the other waits; while every workgroup of four finds a CU of its own, each
// chunk of a chain ends sooner there. Keeping forward / backward in bf16, heads
// of 128 (us, 32768 tokens): 128 chains 654 / 587 with eight and 521 / 470 with
// four; 192 chains (24576 tokens) 334 / 299 and 439 / 405; 512 chains 670 / 634
// and 950 / 860. fp32 keys over 64 keep four: eight waves have half the registers
// each, and 104 to 177 of them spill (512 chains of 512 tokens, 663 / 587 against
// 427 / 441). With keys of 64, 4 to 13 spill, which costs less than four waves do
// (199 / 219 against 278 / 279).
constexpr int kCUs = 256;
template <typename T, int DKP>
constexpr bool kWide = kExact<T> == 1 || DKP <= 64;
inline int64_t chain_groups(const DeltaArgs& a, int waves) {
    return (int64_t)a.nseq * a.Hv * ((a.Dv + waves * kWaveCols - 1) / (waves * kWaveCols));
}
template <typename T, int DKP>
int chain_waves(const DeltaArgs& a) {
    return kWide<T, DKP> && a.Dv > 4 * kWaveCols && chain_groups(a, 4) > kCUs ? 8 : 4;
}
// Whether the chains are started by length: where they are more than the CUs
// take at once (31 sequences of 64 to 2048 tokens x 32 heads: 674 us against
// 789 keeping, 650 against 750 backward).
inline bool chain_ordered(const DeltaArgs& a, int waves) {
    return a.nseq > 1 && a.nseq <= kOrderMax && chain_groups(a, waves) > kCUs;
}
// Long sequences in few heads are split into parts, so that more than a few
// CUs work on them. The state that leaves a part is A S + B with S the one that
// enters: a first walk over all parts at once forms B, from S = 0, and A, whose
// columns are those of S = 1 with no values read; k_delta_join goes from part
// to part; a second walk, from the states it found, does what the walk of
// whole sequences does. Backwards the same with the gradient of the state.
// That is (Dv + Dk) / Dv and 1 times the steps of the plain walk, so it takes
// few chains and long ones. A part has at least the square root of half the
// chunks (the walks take 2 parts' time, the join 5.5 us for each part), and
// there are no more parts than CUs take at once. Forward / keeping / backward of
// one sequence, heads of 128 x 128 in bf16 (us):
//   tokens x heads (chains)   whole                 split
//   16384 x  4 (8)            1133 / 1202 / 1201     234 /  243 /  257
//   16384 x 16 (32)           1228 / 1423 / 1285     587 /  666 /  679
//   16384 x 24 (48)           1248 / 1435 / 1314     855 /  972 /  998
//   16384 x 32 (64)           1251 / 1472 / 1347    1126 / 1292 / 1294
//   16384 x 48 (96)           1261 / 1581 / 1407    1693 / 1945 / 1408
//    4096 x 16 (32)            292 /  310 /  306     166 /  177 /  192
//    4096 x 24 (48)            291 /  313 /  310     224 /  237 /  260
//    4096 x 32 (64)            287 /  323 /  316     280 /  305 /  331
//    2048 x  4 (8, 32 chunks)  145 /  155 /  149      89 /   93 /   94
//    1024 x  4 (8, 16 chunks)   75 /   81 /   77      64 /   66 /   69
// The two sides meet at 64 chains; the bound stands below that, and leaves whole
// what has 33 to 63 of them, which the split would take a quarter from. At 16
// chunks two more launches take most of what is gained.
constexpr int kSplitChains = 32, kSplitChunks = 32;
inline int split_chunks(int64_t T, int32_t nseq, int32_t Hv, int32_t Dv) {
    const int64_t chains = (int64_t)nseq * Hv * ((Dv + 63) / 64), chunks = T / kC / nseq;
    if (chains > kSplitChains || chunks < kSplitChunks) return 0;
    int64_t p = chunks * chains / (kCUs / 2);
    if (p < 4) p = 4;
    while (2 * p * p < chunks) ++p;
    return (int)p;
}
__host__ __device__ inline int64_t split_parts(const DeltaArgs& a) { return a.T / ((int64_t)kC * a.split) + a.nseq; }
// A part's matrix in `joint`: DKP rows of B's columns (whole waves of them; the
// state that enters, once it is known), then A's.
__host__ __device__ inline int joint_b(int Dv) { return (Dv + 63) / 64 * 64; }
// Room for the parts of every pack of up to T tokens and nseq sequences, so that
// a scratch made for the largest pack serves the smaller ones: fewer tokens may
// have more parts, and fewer sequences may be split where these are not. With
// `per` chains a sequence, packs of n <= kSplitChains / per sequences of kSplitChunks
// chunks or more are split, and they have at most T / (4 kC) + n parts. With
// q = chunks n per / (kCUs / 2) a part has at least max(4, 4 q / 5) chunks, so that
// there are at most (kCUs / 2) 5 / 4 (1 + 1 / kSplitChunks) / per + n parts as well.
constexpr int kMaxParts = kCUs / 2 * 5 / 4 * (kSplitChunks + 1) / kSplitChunks;
inline size_t joint_bytes(int64_t T, int32_t nseq, int32_t Hv, int dkp, int32_t Dv) {
    const int64_t per = (int64_t)Hv * ((Dv + 63) / 64);
    int64_t n = T / kC / kSplitChunks;
    if (n > nseq) n = nseq;
    if (n > kSplitChains / per) n = kSplitChains / per;
    if (n < 1) return 0;
    const int64_t parts = T / (4 * kC) < kMaxParts / per ? T / (4 * kC) : kMaxParts / per;
    return round256((size_t)(parts + n) * Hv * dkp * (joint_b(Dv) + dkp) * sizeof(float));
}

inline unsigned chain_blocks(const DeltaArgs& a, int waves) {
    const int ncb = (a.Dv + waves * kWaveCols - 1) / (waves * kWaveCols);
    return (unsigned)spread_blocks((a.split ? split_parts(a) : (int64_t)a.nseq) * a.Hk, ncb * (a.Hv / a.Hk));
}
// of the first walk over parts, by workgroups of four waves
inline unsigned split_blocks(const DeltaArgs& a, int dkp) {
    return (unsigned)spread_blocks(split_parts(a) * a.Hk, (joint_b(a.Dv) + dkp) / 64 * (a.Hv / a.Hk));
}

// What a chain walks: a sequence, or a part of one.
struct Walk {
    int64_t start, slot0;
    int32_t len, seq;
    int64_t part;      // its place in `joint`
    bool first, last;  // of its sequence
};
template <bool SPLIT>
__device__ __forceinline__ bool walk_at(const DeltaArgs& a, int64_t i, Walk& w) {
    if (SPLIT && a.split) {
        Chunk c;
        if (!chunk_at(a.cu, a.nseq, a.T, i, c, kC * a.split)) return false;
        const int64_t slot0 = (c.start - c.index * kC * a.split) / kC + c.seq;
        w = {c.start, slot0 + c.index * a.split, c.n, c.seq, i, c.index == 0, c.last};
        return true;
    }
    const int s = a.order ? a.order[i] : (int)i;
    const Seq q = seq_at(a.cu, s, a.T);
    w = {q.start, q.slot0, q.len, s, 0, true, true};
    return true;
}

// A lane's elements of a (tokens, Dv) tensor of one head, as a result of 4
// tiles holds them: tokens 16 m + 4 (l / 16) + r of its column (kNowhere where
// the column is none).
struct Column {
    uint32_t o;  // byte offset of its first element
    int stride;  // bytes between tokens
};
template <typename T>
__device__ __forceinline__ Column column_of(int H, int Dv, int col) {
    const int stride = H * Dv * (int)sizeof(T), l4 = lane_id() >> 4;
    return {col < Dv ? (uint32_t)(l4 * 4 * stride + col * (int)sizeof(T)) : kNowhere, stride};
}
template <typename T>
__device__ __forceinline__ void load_column(const T* first, int n, int H, int Dv, const Column& c, uint32_t (&v)[16]) {
    const auto r = rows_rsrc(first, n, H * Dv, Dv);
    const uint32_t o = fresh(c.o);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = Elt<T>::raw_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride);
}
template <typename T>
__device__ __forceinline__ void store_column(T* first, int n, int H, int Dv, const Column& c, const f32x4 (&v)[4],
                                             float scale) {
    const auto r = rows_rsrc(first, n, H * Dv, Dv);
    const uint32_t o = fresh(c.o);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        Elt<T>::st_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride, scale * v[i >> 2][i & 3]);
}
// the same of a caller's state (rows, Dv)
template <int MT>
__device__ __forceinline__ void store_state(float* p, int rows, int Dv, const Column& c, const f32x4 (&v)[MT]) {
    const auto r = rows_rsrc(p, rows, Dv, Dv);
    const uint32_t o = fresh(c.o);
#pragma unroll
    for (int i = 0; i < MT * 4; ++i)
        Elt<float>::st_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride, v[i >> 2][i & 3]);
}
template <int MT>
__device__ __forceinline__ void load_state(const float* p, int rows, int Dv, const Column& c, f32x4 (&v)[MT]) {
    const auto r = rows_rsrc(p, p ? rows : 0, Dv, Dv);
#pragma unroll
    for (int i = 0; i < MT * 4; ++i)
        v[i >> 2][i & 3] = Elt<float>::cvt(
            Elt<float>::raw_rsrc(r, c.o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (uint32_t)c.stride));
}
// the states of A's columns, and no state in B's (e < 0)
template <int DKP>
__device__ __forceinline__ void unit_state(f32x4 (&v)[DKP / 16], int e) {
#pragma unroll
    for (int i = 0; i < DKP / 4; ++i)
        v[i >> 2][i & 3] = (i >> 2) * 16 + (lane_id() >> 4) * 4 + (i & 3) == e ? 1.0f : 0.0f;
}
// and of a kept matrix (kept_at)
template <int MT>
__device__ __forceinline__ void store_kept(float* p, int Dv, int col, const f32x4 (&v)[MT]) {
    const auto r = bytes_rsrc(p, (uint32_t)(kept_cols(Dv) * MT * 16) * 4u);
    const uint32_t o = fresh(col < Dv ? (uint32_t)kept_at(MT * 16, (lane_id() >> 4) * 4, col) * 4u : kNowhere);
#pragma unroll
    for (int i = 0; i < MT * 4; ++i)
        Elt<float>::st_rsrc(r, o + (uint32_t)((i >> 2) * 16 + (i & 3)) * (kKeptCols * 4u), v[i >> 2][i & 3]);
}

// From part to part of a split sequence: 16 columns of the state a wave. `from`
// enters the first part (backwards: its gradient leaves the last); where there
// are no tokens it goes to `to` as it is. Bound by what one CU can read: A is 64
// KiB a part at keys of 128, 5.5 us. (The next part's A on its way in registers
// meanwhile gained nothing, 6.0 us.)
template <int DKP, bool BWD>
__global__ __launch_bounds__(64) void k_delta_join(DeltaArgs a, const float* from, float* to) {
    constexpr int MT = DKP / 16;
    const int ncb = (a.Dv + 15) / 16, l = lane_id(), l16 = l & 15, l4 = l >> 4;
    const int col = (int)(blockIdx.x % ncb) * 16 + l16, hv = (int)(blockIdx.x / ncb % a.Hv);
    const int seq = (int)(blockIdx.x / ncb / a.Hv);
    const Seq q = seq_at(a.cu, seq, a.T);
    const int64_t size = (int64_t)kC * a.split, first = q.start / size + seq;
    const int n = (int)((q.len + size - 1) / size), b = joint_b(a.Dv), width = b + DKP;
    const size_t state = ((size_t)seq * a.Hv + hv) * a.Dk * a.Dv;
    const Column cs = column_of<float>(1, a.Dv, col), cj = column_of<float>(1, width, col);
    f32x4 S[MT];
    load_state(from ? from + state : nullptr, a.Dk, a.Dv, cs, S);
    if (n == 0 && to) store_state(to + state, a.Dk, a.Dv, cs, S);
    for (int i = 0; i < n; ++i) {
        float* const J = a.joint + ((size_t)(first + (BWD ? n - 1 - i : i)) * a.Hv + hv) * DKP * width;
        f32x4 next[MT];
        load_state(i + 1 < n ? J : nullptr, DKP, width, cj, next);
        store_state(J, DKP, width, cj, S);
        if (i + 1 == n) break;
#pragma unroll
        for (int s = 0; s < DKP / 32; ++s) {
            const auto sb = split_tiles<3>(S[2 * s], S[2 * s + 1]);
            Frag<3> fa[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float* const row = J + (size_t)(m * 16 + l16) * width + b + s * 32 + l4 * 4;
                fa[m] = split_tiles<3>(*reinterpret_cast<const f32x4*>(row), *reinterpret_cast<const f32x4*>(row + 16));
            }
            mma_tiles<3, 0, MT>(next, fa, sb);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) S[m] = next[m];
    }
}
template <int DKP, bool BWD>
void launch_delta_join(const DeltaArgs& a, const float* from, float* to, hipStream_t s) {
    k_delta_join<DKP, BWD><<<(unsigned)(a.nseq * a.Hv * ((a.Dv + 15) / 16)), 64, 0, s>>>(a, from, to);
}

}  // namespace ssmp
