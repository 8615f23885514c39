// Shared by the delta-rule and head-norm kernels: chunk numbering, operands
// of the matrix instructions, and the small 64-token matrices of a chunk.
#pragma once

#include "common.h"

namespace ssmp {

// Host-side: whether every pointer is a multiple of 16 (wide loads want that).
template <typename... P>
inline bool aligned16(P... p) {
    return ((reinterpret_cast<uintptr_t>(p) % 16 == 0) && ...);
}

// A value again, in a way that the compiler does not see through: it would
// else form the addresses of a loop's every access ahead of the loop and keep
// them, dozens of registers that these kernels do not have.
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

// The wave's number in its workgroup, as a scalar: branches on it are the
// wave's own, as matrix instructions, which heed no lane mask, need them to be.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)); }

// Sums over the 8 or 16 lanes that share l / 8 or l / 16, in every lane:
// neighbours, pairs, then the mirrored half (no address registers, unlike a
// shuffle through LDS).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float sum8(float v) { return dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))); }
__device__ __forceinline__ float sum16(float v) { return dpp_add<0x140>(sum8(v)); }

// A launch takes fewer than 2^32 threads: fewer than this many workgroups of 256.
constexpr int64_t kMaxBlocks = int64_t(1) << 24;

// ---------------------------------------------------------------------------
// Chunks. A chunk is up to 64 tokens of one sequence, counted from its first
// token. Sequence s has its chunks in the slots floor(cu[s] / 64) + s + c,
// c = 0 .. ceil(len / 64) - 1: since floor((x + len) / 64) + 1 >= floor(x / 64)
// + ceil(len / 64), the slots of two sequences never meet, and T / 64 + nseq
// slots are enough for any division of T tokens, so no prefix sum over the
// sequences is needed. cu_seqlens is clamped to [0, T], so that no content of
// it leads outside the tensors or slots.
constexpr int kC = 64;

__host__ __device__ inline int64_t delta_slots(int64_t T, int32_t nseq) { return T / kC + nseq; }

struct Seq {
    int64_t start;
    int32_t len;
    int64_t slot0;
};
__device__ __forceinline__ Seq seq_at(const int32_t* __restrict__ cu, int s, int64_t T) {
    int64_t a = cu[s], b = cu[s + 1];
    a = a < 0 ? 0 : (a > T ? T : a);
    b = b < a ? a : (b > T ? T : b);
    return {a, (int32_t)(b - a), a / kC + s};
}

// The chunk in a slot: false where the slot holds none. Called by whole waves;
// 64 boundaries are looked at in one step, so one trip to memory finds a
// sequence among 64, two among 4096. (Pieces of another size than kC lie in
// slots by the same rule. `empties`: a sequence without tokens counts as one of
// no tokens, in the slot that it has all the same.)
struct Chunk {
    int64_t start;   // its first token
    int32_t n;       // tokens
    int32_t seq;
    int64_t index;   // in its sequence
    bool last;       // of its sequence
};
__device__ __forceinline__ bool chunk_at(const int32_t* __restrict__ cu, int32_t nseq, int64_t T, int64_t slot,
                                         Chunk& c, int size = kC, bool empties = false) {
    const int top = (int)T, lane = lane_id();
    int lo = 0, hi = nseq;
    while (true) {
        const int step = (hi - lo + 63) / 64, i = lo + lane * step;
        int a = cu[i < nseq ? i : nseq];
        a = a < 0 ? 0 : (a > top ? top : a);
        int n = __popcll(__ballot(i < hi && (int64_t)(a / size) + i <= slot));
        n = n < 1 ? 1 : n;
        if (step > 1) {
            lo += (n - 1) * step;
            hi = lo + step < hi ? lo + step : hi;
            continue;
        }
        lo += n - 1;  // the sequence
        const int first = __builtin_amdgcn_readlane(a, n - 1);
        int end;
        if (n < 64) {
            end = __builtin_amdgcn_readlane(a, n);
        } else {
            end = cu[lo + 1];
            end = end < 0 ? 0 : (end > top ? top : end);
        }
        c.index = slot - (first / size + lo);
        const int64_t at = c.index * size;
        if (at < 0 || (at >= end - first && !(empties && at == 0))) return false;
        c.start = first + at;
        c.last = end - first - at <= size;
        c.n = c.last ? (int32_t)(end - first - at) : size;
        c.seq = lo;
        return true;
    }
}

// ---------------------------------------------------------------------------
// Matrix products. States, the chunk's inverse and every value derived from
// them are fp32; v_mfma_f32_16x16x32_bf16 multiplies bf16. An fp32 operand is
// split into bf16 planes x = x0 + x1 + x2 (8 bits each, together fp32's 24),
// and a product adds the plane products down to the bits that count: with one
// side exactly bf16 all 3; with three planes a side 6 of 9, which leaves out
// 2^-24 of the product in the root mean square and 2^-21.1 at most (the planes
// are cut off, so it is left out with the product's sign: 2^-24.6 on average). That is 2.7 to 5.3 times the rate of the fp32 matrix
// instruction, whose rate is a sixteenth of bf16's.
//
// Operands: lane l of A holds row l % 16, elements k = 8 (l / 16) .. + 7; of B
// column l % 16, the same k; the result D has column l % 16, rows 4 (l / 16)
// .. + 3. Both operands want their k contiguous, so in memory A is [m][k] and
// B is [n][k].
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int NP>
struct Frag {
    bf16x8 p[NP];
};

// d += a b, the terms i + j < LIM of the plane products, small ones first
template <int LIM, int NA, int NB>
__device__ __forceinline__ void mma(f32x4& d, const Frag<NA>& a, const Frag<NB>& b) {
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], d, 0, 0, 0);
}

// One of the plane products of mma, the TERM-th in its order, if there are as
// many: for products on several results to take turns.
template <int LIM, int TERM, int NA, int NB>
__device__ __forceinline__ void mma_term(f32x4& d, const Frag<NA>& a, const Frag<NB>& b) {
    int t = 0;
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB) {
                if (t == TERM) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[s - i], d, 0, 0, 0);
                ++t;
            }
}

// d[m] += a[m] b for tiles FROM .. TO - 1, one plane product after the other
// over all tiles: a matrix instruction waits for the last one on its tile.
template <int LIM, int FROM, int TO, int NA, int NB, int N, int NF>
__device__ __forceinline__ void mma_tiles(f32x4 (&d)[N], const Frag<NA> (&a)[NF], const Frag<NB>& b) {
#pragma unroll
    for (int s = LIM - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NA; ++i)
            if (s - i >= 0 && s - i < NB)
#pragma unroll
                for (int m = FROM; m < TO; ++m)
                    d[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[m - FROM].p[i], b.p[s - i], d[m], 0, 0, 0);
}

// The order of one step of a chain: its LDS reads, then per matrix
// instruction V of the other operations (the next step's splitting), which
// run in its shadow.
template <int READS, int MFMAS, int V>
__device__ __forceinline__ void step_order() {
    __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
#pragma unroll
    for (int i = 0; i < MFMAS; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, V, 0);
    }
}

// Two values as bf16 planes, packed: v = p[0] + p[1] + ... Three planes take
// the leading 8 bits that are left each, which holds all 24 of an fp32; one is
// for values that are bf16 already. (Cutting off takes two thirds of the time of
// rounding: 34 against 52 cycles a pair on one SIMD, and a chain spends more
// cycles on splitting than on its products.)
template <int NP>
__device__ __forceinline__ void split2(float v0, float v1, uint32_t (&p)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const uint32_t a = __builtin_bit_cast(uint32_t, v0), b = __builtin_bit_cast(uint32_t, v1);
        p[i] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        if (i + 1 < NP) {
            v0 -= __builtin_bit_cast(float, a & 0xffff0000u);
            v1 -= __builtin_bit_cast(float, b & 0xffff0000u);
        }
    }
}
template <int NP>
__device__ __forceinline__ Frag<NP> split8(const float (&v)[8]) {
    u32x4 w[NP];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        uint32_t p[NP];
        split2<NP>(v[2 * e], v[2 * e + 1], p);
#pragma unroll
        for (int i = 0; i < NP; ++i) w[i][e] = p[i];
    }
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = __builtin_bit_cast(bf16x8, w[i]);
    return f;
}

// planes that hold an input of this type exactly
template <typename T>
constexpr int kExact = std::is_same<T, float>::value ? 3 : 1;

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
    }
}

// NP planes of `plane` elements each, at one place
template <int NP>
__device__ __forceinline__ Frag<NP> tile_planes(const __bf16* base, int plane, int at) {
    Frag<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        f.p[i] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(base + i * plane + at));
    return f;
}
// four values along k (a lane's rows of a result) into the planes
template <int NP>
__device__ __forceinline__ void lds_put4(__bf16* base, int plane, int at, const float (&v)[4]) {
    uint32_t p[2][NP];
    split2<NP>(v[0], v[1], p[0]);
    split2<NP>(v[2], v[3], p[1]);
#pragma unroll
    for (int i = 0; i < NP; ++i)
        *reinterpret_cast<u32x2*>(base + i * plane + at) = u32x2{p[0][i], p[1][i]};
}

// Results as operands. The order of a product's k is free as long as both
// operands have the same, so k = 4 g + e (g < 8) of each block of 32 is put at
// place 8 (g % 4) + 4 (g / 4) + e: lane group l / 16 then holds as operand the
// very rows 4 (l / 16) + e and 16 + 4 (l / 16) + e that two tiles of a result
// left with it, and a result becomes the next product's right operand by
// rounding alone, without a trip through LDS. Left operands are stored in
// this order.
__host__ __device__ constexpr int kplace(int k) { return (k & ~31) | (((k >> 2) & 3) << 3) | (((k >> 4) & 1) << 2) | (k & 3); }
template <int NP>
__device__ __forceinline__ Frag<NP> split_tiles(const f32x4& lo, const f32x4& hi) {
    const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return split8<NP>(v);
}

// Rows of a chunk through a buffer resource: 32-bit lane offsets, and what
// lies behind the chunk's last row, or is marked kNowhere, reads as zero and
// is not written. Rows of up to kMaxRow elements keep offsets below 2^31.
constexpr uint32_t kNowhere = 0x80000000u;
constexpr int64_t kMaxRow = int64_t(1) << 20;
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const T* first, int rows, int stride, int width) {
    return bytes_rsrc(first, rows > 0 ? (uint32_t)((rows - 1) * stride + width) * (uint32_t)sizeof(T) : 0u);
}

// 8 elements on their way from memory to LDS
template <typename T>
struct Unit;
template <>
struct Unit<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t o) {
        w = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)o, 0, 0));
    }
    __device__ __forceinline__ void put_half(uint16_t* p, int h) const {
        *reinterpret_cast<u32x2*>(p) = h ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]};
    }
    __device__ __forceinline__ void pack(const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = (uint32_t)f32_to_bf16(v[2 * e]) | ((uint32_t)f32_to_bf16(v[2 * e + 1]) << 16);
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t o) const {
        __builtin_amdgcn_raw_buffer_store_b128(w, r, (int)o, 0, 0);
    }
};
template <>
struct Unit<float4> {  // four of fp32
    f32x4 w;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t o) {
        w = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)o, 0, 0));
    }
};
template <>
struct Unit<float> {
    f32x4 w[2];
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t o) {
        w[0] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)o, 0, 0));
        w[1] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(o + 16), 0, 0));
    }
    __device__ __forceinline__ void put_half(float* p, int h) const { *reinterpret_cast<f32x4*>(p) = w[h]; }
    __device__ __forceinline__ void pack(const float (&v)[8]) {
        w[0] = f32x4{v[0], v[1], v[2], v[3]};
        w[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t o) const {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w[0]), r, (int)o, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, w[1]), r, (int)(o + 16), 0, 0);
    }
};
__device__ __forceinline__ Frag<1> unit_planes(const Unit<uint16_t>& u) { return {{__builtin_bit_cast(bf16x8, u.w)}}; }
__device__ __forceinline__ Frag<3> unit_planes(const Unit<float>& u) { return split_tiles<3>(u.w[0], u.w[1]); }
// Left operands in LDS: rows of W elements of E in 16-byte units (32 for fp32:
// what one lane reads), without padding; unit u of row r lies at u ^ swz(r),
// so that the 16 rows a read touches fall into different banks.
template <typename E, int W>
struct Tile {
    static constexpr int kUnits = W / 8;
    static constexpr int kPer = W * (int)sizeof(E) >= 256 ? 1 : 256 / (W * (int)sizeof(E));  // rows to a turn of the banks
    static __device__ __forceinline__ int at(int row, int unit) {
        return row * W + ((unit ^ ((row / kPer) & (kUnits - 1))) << 3);
    }
};
__device__ __forceinline__ Frag<1> tile_frag(const uint16_t* p) {
    return {{__builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p))}};
}
__device__ __forceinline__ Frag<3> tile_frag(const float* p) {
    float v[8];
    load8(p, v);
    return split8<3>(v);
}

// Rows of keys or queries in LDS as [token][d], d in places, and their two
// readings as operands: along d, and along the tokens of a block of 32 for the
// 16 columns d = 16 m .. + 15. The second is a transposing read of 8 bytes for
// bf16 (in a group of 16 lanes, lane j points at token j / 4, four columns
// from 4 (j % 4), and receives column j of the four tokens), single elements
// for fp32. So keys need no transposed copy.
template <typename T, int DKP>
struct RowTile {
    using L = Tile<T, DKP>;
    T x[kC * DKP];

    __device__ __forceinline__ Frag<kExact<T>> frag(int token, int unit) const { return tile_frag(x + L::at(token, unit)); }
    // lane l: tokens 16 t + 4 (l / 16) .. + 3 of column 16 m + l % 16
    __device__ __forceinline__ void column4(int l, int t, int m, uint32_t (&v)[kExact<T> == 1 ? 2 : 4]) const {
        const int l16 = l & 15, l4 = l >> 4;
        if constexpr (kExact<T> == 1) {
            const int token = t * 16 + l4 * 4 + (l16 >> 2);
            const T* p = x + L::at(token, (m >> 1) * 4 + (l16 & 3)) + (m & 1) * 4;
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            const s16x4 r = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
            const u32x2 w = __builtin_bit_cast(u32x2, r);
            v[0] = w[0];
            v[1] = w[1];
        } else {
            const int p = kplace(m * 16 + l16);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_bit_cast(uint32_t, x[L::at(t * 16 + l4 * 4 + e, p >> 3) + (p & 7)]);
        }
    }
    __device__ __forceinline__ void values4(int l, int t, int m, float (&f)[4]) const {
        if constexpr (kExact<T> == 1) {
            uint32_t v[2];
            column4(l, t, m, v);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[2 * e] = bf16_to_f32(v[e]);
                f[2 * e + 1] = bf16_hi_to_f32(v[e]);
            }
        } else {
            uint32_t v[4];
            column4(l, t, m, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = __builtin_bit_cast(float, v[e]);
        }
    }
    // tokens of block s of 32 as k, in places
    __device__ __forceinline__ Frag<kExact<T>> token_frag(int l, int s, int m) const {
        if constexpr (kExact<T> == 1) {
            uint32_t a[2], b[2];
            column4(l, 2 * s, m, a);
            column4(l, 2 * s + 1, m, b);
            return {{__builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]})}};
        } else {
            float a[4], b[4];
            values4(l, 2 * s, m, a);
            values4(l, 2 * s + 1, m, b);
            return split8<3>({a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
        }
    }
    // a unit of 8 elements of token i from column 8 k8 on
    __device__ __forceinline__ void put(int i, int k8, const Unit<T>& u) {
        const int p0 = kplace(k8 * 8), p1 = kplace(k8 * 8 + 4);
        u.put_half(x + L::at(i, p0 >> 3) + (p0 & 4), 0);
        u.put_half(x + L::at(i, p1 >> 3) + (p1 & 4), 1);
    }
};

// The triangular matrices of a chunk (the inverse, the decayed products) in
// memory: fp32, in places, the blocks of 32 columns that hold anything:
// lower: columns 0-31 of all 64 rows, then 32-63 of rows 32-63;
// upper: columns 32-63 of all 64 rows, then 0-31 of rows 0-31.
constexpr int kTriRows = 96, kTri = kTriRows * 32;
template <bool UPPER>
__device__ __forceinline__ int tri_row(int row, int col) {
    if constexpr (UPPER) return col >= 32 ? row : 64 + row;
    else return col < 32 ? row : 32 + row;
}
// the same in LDS: NP planes of 96 rows of 32 places
template <int NP>
__device__ __forceinline__ void tri_put4(__bf16* base, int idx4, const f32x4& v) {
    const int row = idx4 >> 3, q = idx4 & 7;
    const float x[4] = {v[0], v[1], v[2], v[3]};
    lds_put4<NP>(base, kTri, Tile<uint16_t, 32>::at(row, q >> 1) + (q & 1) * 4, x);
}
template <int NP>
__device__ __forceinline__ Frag<NP> tri_frag(const __bf16* base, int row, int unit) {
    return tile_planes<NP>(base, kTri, Tile<uint16_t, 32>::at(row, unit));
}

// The workgroups that share keys and queries (the column blocks of a head,
// the value heads of a key head) on one XCD, one after another: workgroups go
// to the 8 XCDs in turn, and each has its own L2.
struct Spread {
    int64_t group;
    int member;
};
__device__ __forceinline__ Spread spread(int64_t block, int members) {
    const int64_t i = block >> 3;
    return {(i / members) * 8 + (block & 7), (int)(i % members)};
}
inline int64_t spread_blocks(int64_t groups, int members) { return (groups + 7) / 8 * 8 * members; }

// ---------------------------------------------------------------------------
// Decays of a chunk: G = running sum of g / log 2 in 64 bits (32-bit sums would lose
// the small steps behind a large one), lane l holding token l. g below
// kGMin is taken as kGMin: e^g is zero all the same, and a full reset
// (g = -infinity) does not turn G's differences into NaN.
constexpr double kGMin = -4096.0;
// e^(sum of g over some tokens) from G's difference: rounded to 32 bits only
// here, where an exponent of size |d| errs by |d| 2^-24 of a result 2^d
__device__ __forceinline__ float decay_of(double d) { return exp2_fast((float)d); }
template <int CTRL>
__device__ __forceinline__ double dpp_add_f64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double read_lane(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// G from g of this lane's token (zero behind the chunk's end): sums within
// the rows of 16 lanes, then those of the rows before
__device__ __forceinline__ double chunk_decay_sum(float g) {
    const int lane = lane_id();
    double v = (double)g;
    v = (v < kGMin ? kGMin : v) * 1.4426950408889634074;
    v = dpp_add_f64<0x111>(v);
    v = dpp_add_f64<0x112>(v);
    v = dpp_add_f64<0x114>(v);
    v = dpp_add_f64<0x118>(v);
    const double a = read_lane(v, 15), b = a + read_lane(v, 31), c = b + read_lane(v, 47);
    return v + (lane < 16 ? 0.0 : lane < 32 ? a : lane < 48 ? b : c);
}

// The inverse of I + A for strictly lower triangular A (64 x 64, fp32 in LDS
// with row length kLdA): X = (I + A)^-1 in X. By forward substitution in the
// four 16 x 16 blocks of the diagonal (lane = block and column), then
//   X_ba = -X_bb (A_ba X_aa)
// for the blocks between them, twice, with the fp32 matrix instruction, whose
// k order is free: a result's rows 4 (l / 16) + r serve as the next product's
// k without leaving their registers. Called by workgroups of 256.
constexpr int kLdA = 68;
__device__ __forceinline__ f32x4 mma16(const float* a, const f32x4& b, f32x4 d) {
    // d += A b, A 16 x 16 at a (row length kLdA), b as a result of this layout
    const int l = lane_id();
    const f32x4 r = *reinterpret_cast<const f32x4*>(a + (l & 15) * kLdA + (l >> 4) * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x4f32(r[i], b[i], d, 0, 0, 0);
    return d;
}
__device__ __forceinline__ f32x4 tile16(const float* x) {
    const int l = lane_id();
    f32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = x[((l >> 4) * 4 + i) * kLdA + (l & 15)];
    return r;
}
__device__ __forceinline__ void put_tile16(float* x, const f32x4& v) {
    const int l = lane_id();
#pragma unroll
    for (int i = 0; i < 4; ++i) x[((l >> 4) * 4 + i) * kLdA + (l & 15)] = v[i];
}
__device__ __forceinline__ void chunk_inverse(const float* A, float* X) {
    const int tid = threadIdx.x, wave = wave_id(), l = lane_id();
    // zero the blocks (0, 1) and (2, 3), the only ones above the diagonal's that are read
#pragma unroll
    for (int i = tid; i < 512; i += 256) X[((i >> 8) * 32 + ((i >> 4) & 15)) * kLdA + (i >> 8) * 32 + 16 + (i & 15)] = 0.0f;
    if (wave == 0) {
        const int at = (l >> 4) * 16, c = l & 15;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == c ? 1.0f : 0.0f;
#pragma unroll
            for (int j = 0; j < i; ++j) s = fmaf(-A[(at + i) * kLdA + at + j], x[j], s);
            x[i] = s;
            X[(at + i) * kLdA + at + c] = s;
        }
    }
    __syncthreads();
    if (wave < 2) {  // blocks (1, 0) and (3, 2)
        const int a = wave * 32, b = a + 16;
        const f32x4 zero = {0, 0, 0, 0};
        const f32x4 y = mma16(A + b * kLdA + a, tile16(X + a * kLdA + a), zero);
        const f32x4 z = mma16(X + b * kLdA + b, y, zero);
        put_tile16(X + b * kLdA + a, -z);
    }
    __syncthreads();
    if (wave < 2) {  // the lower left 32 x 32, one column of blocks a wave
        const int n = wave * 16;
        f32x4 y[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const f32x4 b = tile16(X + k * 16 * kLdA + n);
#pragma unroll
            for (int m = 0; m < 2; ++m) y[m] = mma16(A + (32 + m * 16) * kLdA + k * 16, b, y[m]);
        }
        const f32x4 zero = {0, 0, 0, 0};
        f32x4 z0 = mma16(X + 32 * kLdA + 32, y[0], zero);
        f32x4 z1 = mma16(X + 48 * kLdA + 32, y[0], zero);
        z1 = mma16(X + 48 * kLdA + 48, y[1], z1);
        put_tile16(X + 32 * kLdA + n, -z0);
        put_tile16(X + 48 * kLdA + n, -z1);
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Sizes and buffers
constexpr int kMaxDk = 128;
constexpr int kWaveCols = 16;  // state columns a wave of the chains takes

__host__ __device__ inline int delta_dkp(int Dk) { return Dk <= 64 ? 64 : 128; }
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

constexpr int kDec = 4 * kC;

// What goes from the chains to the gradients, S, E, dS' and dU of each chunk:
// fp32 in blocks of 32 columns, [block][row][32], as k_delta_grads reads them:
// in rows of all columns it would read 128 bytes of each 512 at a time (1500 us
// where it takes 1415, 32768 tokens x 32 heads of 128 x 128).
constexpr int kKeptCols = 32;
__host__ __device__ inline int kept_cols(int Dv) { return (Dv + kKeptCols - 1) / kKeptCols * kKeptCols; }
__device__ __forceinline__ int kept_at(int rows, int row, int col) {
    return ((col / kKeptCols) * rows + row) * kKeptCols + col % kKeptCols;
}
struct DeltaArgs {
    const void *q, *k, *v, *dout;
    const float *g, *beta;
    const int32_t* cu;
    void *out, *dq, *dk, *dv;
    float *dg, *dbeta;
    const float *h0, *dhT;
    float *hT, *dh0;
    int64_t T;
    int32_t nseq, Hk, Hv, Dk, Dv;
    float scale;
    // kept from the forward to the backward, by slot and value head
    float *S0, *E;   // the state that enters the chunk (rows: Dk padded), the errors (64 rows)
    // scratch, by slot and head
    float* dec;      // G (64 doubles), e^{G_i}, e^{G_last - G_i}: kDec
    float* inv;      // the chunk's inverse: kTri
    float* att;      // the decayed products of q and k: kTri
    float *dS1, *dU; // backward: gradients of the state that leaves the chunk, and of U
    float* rows;     // backward: per 64 columns of dq and dk, what k_delta_dg adds up: 64
    int32_t* order;  // the sequences by length (null: as they come)
    float* joint;    // of split sequences, by part and value head: what joins them
    int32_t split;   // chunks of a part (0: sequences are not split)
};

inline size_t kept_bytes(int64_t T, int32_t nseq, int32_t Hv, int rows, int32_t Dv) {
    return round256((size_t)delta_slots(T, nseq) * Hv * rows * kept_cols(Dv) * sizeof(float));
}

inline int delta_check(int64_t T, int32_t nseq, int32_t Hk, int32_t Hv, int32_t Dk, int32_t Dv, int32_t dtype) {
    if (T < 0 || T >= (int64_t(1) << 31) || nseq < 1 || Hk < 1 || Hv < 1 || Dk < 1 || Dv < 1) return SSMP_ERR_SHAPE;
    if (Hv % Hk || Hv > 65535 || nseq > (1 << 24)) return SSMP_ERR_SHAPE;
    if ((int64_t)Hv * Dv > kMaxRow || (int64_t)Hk * Dk > kMaxRow) return SSMP_ERR_SHAPE;
    if (T * Hv * (int64_t)(Dv > Dk ? Dv : Dk) >= (int64_t(1) << 40)) return SSMP_ERR_SHAPE;
    // the chains' and the chunks' workgroups (of chunks two a head: 64 columns of dq and dk)
    if ((int64_t)(nseq + 7) * Hv * ((Dv + 127) / 128 * 2) >= kMaxBlocks) return SSMP_ERR_SHAPE;
    if ((T / kC + nseq + 7) * Hv * 2 >= kMaxBlocks) return SSMP_ERR_SHAPE;
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    if (Dk % 8 || Dv % 8 || Dk > kMaxDk) return SSMP_ERR_UNSUPPORTED;
    return SSMP_OK;
}

}  // namespace ssmp
