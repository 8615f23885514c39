// qk_norm_pack: norms of the query and key heads of a packed batch, with the
// position rotation in the same pass, and their gradients.
//
//   r = (mean_d x_d^2 + eps)^(-1/2)  (RMS)   or   (sum_d x_d^2 + eps)^(-1/2)  (L2)
//   y = R(pos) (x r w)
// R turns the pairs (i, i + rot/2), or (2i, 2i + 1), of the first `rot`
// components by pos * inv_freq[i]. With h = R^T dy and c = h w the gradients are
//   dw = sum_rows h x r,   dx = r (c - x r m),   m = mean_d or sum_d of c x r.
//
// Bound by HBM: each row is read and written once. A row lies across 1 to 64
// lanes, 8 components in each, so that a wave reads 1 KiB (bf16) at a time;
// a wave takes the heads of one token together, which turn by the same
// angles, and forms its lanes' cosines and sines once. In bf16, heads of 128:
// 32768 tokens of 32 heads 94 us forward and 157 us backward, 5.7 and 5.1 TB/s;
// 16384 tokens of 40, with weights and half turned, 85 us forward (3.9 TB/s) and
// 111 + 7 us backward (4.3 TB/s), the angles in 64 bits on top.
#include "delta_common.h"

namespace ssmp {

constexpr int kNormVec = 8;      // components a lane holds
constexpr int kNormMaxD = 512;   // 64 lanes
constexpr int kNormWaves = 4;    // per workgroup
constexpr int64_t kNormBwdBlocks = 1024;  // most workgroups of the backward: one row of weight sums each

struct NormArgs {
    const void* x[2];     // q, k
    const void* dy[2];
    const float* w[2];
    void* y[2];           // the forward's outputs, or dq, dk
    float* part;          // backward: (workgroups, 2, D) weight sums
    const int32_t* pos;
    const float* inv_freq;
    int64_t T;
    int32_t H[2];
    int32_t D, rot, interleaved;
    float inv_n, eps;     // 1/D or 1
    int32_t hsplit;       // waves that share a token's heads
};

// a lane's components as they lie in memory, so that the next row's are under
// way while the present ones are worked on
template <typename T>
struct NormRow;
template <>
struct NormRow<float> {
    f32x4 w[2];
    __device__ __forceinline__ void load(const float* p, bool on) {
        w[0] = w[1] = f32x4{0, 0, 0, 0};
        if (on) {
            w[0] = reinterpret_cast<const f32x4*>(p)[0];
            w[1] = reinterpret_cast<const f32x4*>(p)[1];
        }
    }
    __device__ __forceinline__ void values(float (&v)[kNormVec]) const {
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) v[e] = w[e >> 2][e & 3];
    }
};
template <>
struct NormRow<uint16_t> {
    u32x4 w;
    __device__ __forceinline__ void load(const uint16_t* p, bool on) {
        w = u32x4{0, 0, 0, 0};
        if (on) w = *reinterpret_cast<const u32x4*>(p);
    }
    __device__ __forceinline__ void values(float (&v)[kNormVec]) const {
#pragma unroll
        for (int e = 0; e < kNormVec / 2; ++e) {
            v[2 * e] = bf16_to_f32(w[e]);
            v[2 * e + 1] = bf16_hi_to_f32(w[e]);
        }
    }
};
__device__ __forceinline__ void norm_store(float* p, const float (&v)[kNormVec]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void norm_store(uint16_t* p, const float (&v)[kNormVec]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)f32_to_bf16(v[2 * i]) | ((uint32_t)f32_to_bf16(v[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
    if constexpr (LPR >= 2) v = dpp_add<0xB1>(v);
    if constexpr (LPR >= 4) v = dpp_add<0x4E>(v);
    if constexpr (LPR >= 8) v = dpp_add<0x141>(v);
    if constexpr (LPR >= 16) v = dpp_add<0x140>(v);
#pragma unroll
    for (int m = 16; m < LPR; m <<= 1) v += __shfl_xor(v, m);
    return v;
}

// Where a wave's rows of a token lie: the heads of q, then those of k.
struct NormAt {
    size_t at;
    bool isk, on;
};
__device__ __forceinline__ NormAt norm_at(const NormArgs& a, int64_t t, int h, int col) {
    const bool isk = h >= a.H[0];
    const size_t row = isk ? (size_t)t * a.H[1] + (h - a.H[0]) : (size_t)t * a.H[0] + h;
    return {row * a.D + col, isk, col < a.D && h < a.H[0] + a.H[1]};
}

// The turn of a lane's components at one position: y_e = x_e c_e + p_e s_e with
// p_e the other member of e's pair and the sign in s_e. The angle in turns is
// formed in 64 bits (a 32-bit one is off by radians at positions near 1e7) and
// reduced to half a turn either way; what its rounding to 32 leaves out, up to
// 2^-25 of a half turn, turns the result once more to first order, so that small
// cosines and sines have all their bits. The wave's
// lanes form one angle each (rot / 2 of them in all) and pass them on through
// LDS: formed where they are used, they would take longer than the heads do
// (16384 tokens of 40 heads of 128, half turned: 118 us against 87).
struct Turn {
    float c[kNormVec], s[kNormVec];
    int partner;  // lane that holds the other members (half-split pairs)
    int n;        // how many of this lane's components are turned (in adjacent pairs perhaps not all)
};
__device__ __forceinline__ void make_turn(Turn& t, const NormArgs& a, int32_t pos, int lane, int col, float2* cs) {
    const int half = a.rot >> 1;
    wave_sync();  // the last token's have been read
    for (int i = lane; i < half; i += kWave) {
        const double turns = (double)pos * (double)a.inv_freq[i] * 0.15915494309189533577;
        const double halves = 2.0 * (turns - rint(turns));
        const float main = (float)halves, rest = (float)((halves - (double)main) * 3.14159265358979323846);
        float sn, co;
        sincospif(main, &sn, &co);
        cs[i] = make_float2(fmaf(-sn, rest, co), fmaf(co, rest, sn));
    }
    wave_sync();
    t.n = a.rot - col;
    t.partner = lane;
    if (!a.interleaved && t.n > 0) t.partner = col < half ? lane + half / kNormVec : lane - half / kNormVec;
#pragma unroll
    for (int e = 0; e < kNormVec; ++e) {
        const int d = col + e;
        const int i = a.interleaved ? d >> 1 : (d < half ? d : d - half);
        const bool first = a.interleaved ? (e & 1) == 0 : d < half;
        const float2 v = d < a.rot ? cs[i] : make_float2(1.0f, 0.0f);
        t.c[e] = v.x;
        t.s[e] = first ? -v.y : v.y;
    }
}
template <bool BACK>
__device__ __forceinline__ void apply_turn(const Turn& t, int interleaved, float (&v)[kNormVec]) {
    float p[kNormVec];
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) p[e] = v[e ^ 1];
    } else {
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) p[e] = __shfl(v[e], t.partner);
    }
#pragma unroll
    for (int e = 0; e < kNormVec; ++e) {
        const float turned = BACK ? fmaf(-p[e], t.s[e], v[e] * t.c[e]) : fmaf(p[e], t.s[e], v[e] * t.c[e]);
        v[e] = e < t.n ? turned : v[e];
    }
}

// One wave per (token, share of its heads).
template <typename T, int LPR, bool ROT>
__global__ __launch_bounds__(kNormWaves* kWave) void k_qk_norm_fwd(NormArgs a) {
    constexpr int RPW = kWave / LPR;  // rows a wave holds at a time
    __shared__ float2 cs[ROT ? kNormWaves : 1][ROT ? kNormMaxD / 2 : 1];
    const int lane = lane_id();
    const int64_t task = (int64_t)blockIdx.x * kNormWaves + (threadIdx.x >> 6);
    if (task >= a.T * a.hsplit) return;
    const int64_t t = task / a.hsplit;
    const int share = (int)(task % a.hsplit);
    const int col = (lane & (LPR - 1)) * kNormVec;
    const bool in = col < a.D;
    const int heads = a.H[0] + a.H[1], step = a.hsplit * RPW;
    int h = share * RPW + lane / LPR;
    NormAt p = norm_at(a, t, h, col);
    NormRow<T> row;
    row.load(static_cast<const T*>(a.x[p.isk]) + p.at, p.on);
    float w[2][kNormVec];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) w[n][e] = a.w[n] && in ? a.w[n][col + e] : 1.0f;
    Turn turn;
    if constexpr (ROT) make_turn(turn, a, a.pos[t], lane, col, cs[threadIdx.x >> 6]);
    for (int h0 = share * RPW; h0 < heads; h0 += step) {
        h += step;
        const NormAt pn = norm_at(a, t, h, col);
        NormRow<T> next;
        next.load(static_cast<const T*>(a.x[pn.isk]) + pn.at, pn.on);
        float v[kNormVec];
        row.values(v);
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) ss = fmaf(v[e], v[e], ss);
        const float r = rsqrtf(fmaf(row_sum<LPR>(ss), a.inv_n, a.eps));
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) v[e] = v[e] * r * (p.isk ? w[1][e] : w[0][e]);
        if constexpr (ROT) apply_turn<false>(turn, a.interleaved, v);
        if (p.on) norm_store(static_cast<T*>(a.y[p.isk]) + p.at, v);
        p = pn;
        row = next;
    }
}

// As the forward; a wave goes over tokens with a fixed stride and keeps its
// lanes' weight sums in registers, which the workgroup adds in a fixed order. A
// lane may have thousands of rows, so the sums of kNormRun tokens go to sums of 64
// bits in LDS. 16384 tokens of 40 turned heads of 128 in bf16 take 111 us so, 105
// with sums of 32 bits alone, and 141 with those of 64 in registers, which leave
// a SIMD three waves instead of four.
constexpr int kNormRun = 8;
template <typename T, int LPR, bool ROT, bool DW>
__global__ __launch_bounds__(kNormWaves* kWave) void k_qk_norm_bwd(NormArgs a) {
    constexpr int RPW = kWave / LPR;
    __shared__ float2 cs[ROT ? kNormWaves : 1][ROT ? kNormMaxD / 2 : 1];
    __shared__ double sums[DW ? kNormWaves : 1][2][DW ? LPR * kNormVec : 1];
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    const int col = (lane & (LPR - 1)) * kNormVec;
    const bool in = col < a.D;
    const int heads = a.H[0] + a.H[1], step = a.hsplit * RPW;
    float w[2][kNormVec], dw[2][kNormVec];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < kNormVec; ++e) {
            w[n][e] = a.w[n] && in ? a.w[n][col + e] : 1.0f;
            dw[n][e] = 0.0f;
            if (DW && lane < LPR) sums[wave][n][col + e] = 0.0;
        }
    const auto put_sums = [&] {  // each lane to places of its own
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < kNormVec; ++e) {
                float s = dw[n][e];
#pragma unroll
                for (int m = LPR; m < kWave; m <<= 1) s += __shfl_xor(s, m);
                if (lane < LPR) sums[wave][n][col + e] += (double)s;
                dw[n][e] = 0.0f;
            }
    };
    int run = 0;
    const int64_t tasks = a.T * a.hsplit;
    for (int64_t task = (int64_t)blockIdx.x * kNormWaves + wave; task < tasks; task += (int64_t)gridDim.x * kNormWaves) {
        const int64_t t = task / a.hsplit;
        const int share = (int)(task % a.hsplit);
        int h = share * RPW + lane / LPR;
        NormAt p = norm_at(a, t, h, col);
        NormRow<T> xr, gr;
        xr.load(static_cast<const T*>(a.x[p.isk]) + p.at, p.on);
        gr.load(static_cast<const T*>(a.dy[p.isk]) + p.at, p.on);
        Turn turn;
        if constexpr (ROT) make_turn(turn, a, a.pos[t], lane, col, cs[wave]);
        for (int h0 = share * RPW; h0 < heads; h0 += step) {
            h += step;
            const NormAt pn = norm_at(a, t, h, col);
            NormRow<T> xn, gn;
            xn.load(static_cast<const T*>(a.x[pn.isk]) + pn.at, pn.on);
            gn.load(static_cast<const T*>(a.dy[pn.isk]) + pn.at, pn.on);
            const bool isk = p.isk, on = p.on;
            float v[kNormVec], g[kNormVec];
            xr.values(v);
            gr.values(g);
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < kNormVec; ++e) ss = fmaf(v[e], v[e], ss);
            const float r = rsqrtf(fmaf(row_sum<LPR>(ss), a.inv_n, a.eps));
            if constexpr (ROT) apply_turn<true>(turn, a.interleaved, g);
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < kNormVec; ++e) {
                v[e] *= r;
                if constexpr (DW) {
                    const float p = on ? g[e] * v[e] : 0.0f;  // r may be infinite where there is no row
                    dw[0][e] += isk ? 0.0f : p;
                    dw[1][e] += isk ? p : 0.0f;
                }
                g[e] *= isk ? w[1][e] : w[0][e];
                m = fmaf(g[e], v[e], m);
            }
            m = row_sum<LPR>(m) * a.inv_n;
#pragma unroll
            for (int e = 0; e < kNormVec; ++e) v[e] = r * fmaf(-v[e], m, g[e]);
            if (on) norm_store(static_cast<T*>(a.y[isk]) + p.at, v);
            p = pn;
            xr = xn;
            gr = gn;
        }
        if constexpr (DW)
            if (++run == kNormRun) {
                put_sums();
                run = 0;
            }
    }
    if constexpr (DW) {
        put_sums();
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
            const int n = i / a.D, d = i % a.D;
            double s = 0.0;
#pragma unroll
            for (int q = 0; q < kNormWaves; ++q) s += sums[q][n][d];
            a.part[(size_t)blockIdx.x * 2 * a.D + i] = (float)s;
        }
    }
}

// dw = the sum of the workgroups' rows, in order, in 64 bits: the rows' signs
// differ, and 32-bit sums over a thousand of them would lose several bits.
// One wave per component: lane l adds rows l, l + 64, ...
template <int kUnused = 0>
__global__ __launch_bounds__(kWave) void k_qk_norm_dw(const float* __restrict__ part, int64_t blocks, int32_t D,
                                                      float* __restrict__ dwq, float* __restrict__ dwk) {
    const int i = blockIdx.x;
    double s = 0.0;
    for (int64_t b = threadIdx.x; b < blocks; b += kWave) s += (double)part[(size_t)b * 2 * D + i];
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) s += __shfl_xor(s, m);
    float* out = i < D ? dwq : dwk;
    if (threadIdx.x == 0 && out) out[i < D ? i : i - D] = (float)s;
}

inline int norm_lanes(int D) {
    int l = 1;
    while (l * kNormVec < D) l <<= 1;
    return l;
}
// Heads of one token go to one wave unless there are too few tokens to give
// every SIMD two waves (2048): then as many waves share them as there are
// wave-fulls of rows.
inline int norm_hsplit(int64_t T, int heads, int D) {
    const int rpw = kWave / norm_lanes(D), full = (heads + rpw - 1) / rpw;
    int64_t s = T > 0 ? (2047 + T) / T : 1;
    return (int)(s > full ? full : s);
}
inline int64_t norm_bwd_blocks(int64_t T, int hsplit) {
    const int64_t b = (T * hsplit + kNormWaves - 1) / kNormWaves;
    return b < kNormBwdBlocks ? b : kNormBwdBlocks;
}
// The most of them for any number of tokens up to T, so that a workspace made
// for T serves fewer: T hsplit is at most T + 2047 below 2048 tokens, then T.
inline int64_t norm_bwd_rows(int64_t T, int heads, int D) {
    const int rpw = kWave / norm_lanes(D), full = (heads + rpw - 1) / rpw;
    int64_t most = (T < 2047 ? T : 2047) + 2047;
    if (most < T) most = T;
    return norm_bwd_blocks(T * full < most ? T * full : most, 1);
}

template <typename T, int LPR>
void launch_norm(const NormArgs& a, bool bwd, bool dw, int64_t blocks, hipStream_t s) {
    const dim3 g((unsigned)blocks), b(kNormWaves * kWave);
    if (!bwd) {
        if (a.rot) k_qk_norm_fwd<T, LPR, true><<<g, b, 0, s>>>(a);
        else k_qk_norm_fwd<T, LPR, false><<<g, b, 0, s>>>(a);
    } else if (a.rot) {
        if (dw) k_qk_norm_bwd<T, LPR, true, true><<<g, b, 0, s>>>(a);
        else k_qk_norm_bwd<T, LPR, true, false><<<g, b, 0, s>>>(a);
    } else {
        if (dw) k_qk_norm_bwd<T, LPR, false, true><<<g, b, 0, s>>>(a);
        else k_qk_norm_bwd<T, LPR, false, false><<<g, b, 0, s>>>(a);
    }
}
template <typename T>
void launch_norm_d(const NormArgs& a, bool bwd, bool dw, int64_t blocks, hipStream_t s) {
    switch (norm_lanes(a.D)) {
        case 1: return launch_norm<T, 1>(a, bwd, dw, blocks, s);
        case 2: return launch_norm<T, 2>(a, bwd, dw, blocks, s);
        case 4: return launch_norm<T, 4>(a, bwd, dw, blocks, s);
        case 8: return launch_norm<T, 8>(a, bwd, dw, blocks, s);
        case 16: return launch_norm<T, 16>(a, bwd, dw, blocks, s);
        case 32: return launch_norm<T, 32>(a, bwd, dw, blocks, s);
        default: return launch_norm<T, 64>(a, bwd, dw, blocks, s);
    }
}

inline bool norm_sizes_ok(int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
    return T >= 0 && T <= (kMaxBlocks - 1) * kNormWaves && Hq >= 0 && Hk >= 0 && Hq <= 65536 && Hk <= 65536 && Hq + Hk >= 1 &&
           D >= 1 && T * ((int64_t)Hq + Hk) * D < (int64_t(1) << 40);
}
inline int norm_check(int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t rot, int32_t dtype, int32_t norm,
                      int32_t interleaved, const int32_t* pos, const float* inv_freq) {
    if (!norm_sizes_ok(T, Hq, Hk, D)) return SSMP_ERR_SHAPE;
    if (rot < 0 || rot > D) return SSMP_ERR_SHAPE;
    if (D % kNormVec || D > kNormMaxD || rot % (interleaved ? 2 : 16)) return SSMP_ERR_UNSUPPORTED;
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    if (norm != SSMP_NORM_RMS && norm != SSMP_NORM_L2) return SSMP_ERR_UNSUPPORTED;
    if (rot > 0 && ((T > 0 && !pos) || !inv_freq)) return SSMP_ERR_NULL;
    return SSMP_OK;
}
inline NormArgs norm_args(int64_t T, int32_t Hq, int32_t Hk, int32_t D, int32_t rot, int32_t norm, float eps,
                          int32_t interleaved, const float* wq, const float* wk, const int32_t* pos,
                          const float* inv_freq) {
    NormArgs a = {};
    a.w[0] = wq;
    a.w[1] = wk;
    a.pos = pos;
    a.inv_freq = inv_freq;
    a.T = T;
    a.H[0] = Hq;
    a.H[1] = Hk;
    a.D = D;
    a.rot = rot;
    a.interleaved = interleaved;
    a.inv_n = norm == SSMP_NORM_RMS ? 1.0f / (float)D : 1.0f;
    a.eps = eps;
    a.hsplit = norm_hsplit(T, Hq + Hk, D);
    return a;
}

}  // namespace ssmp

extern "C" int qk_norm_pack_fwd(const void* q, const void* k, const float* wq, const float* wk, const int32_t* pos,
                                const float* inv_freq, void* yq, void* yk, int64_t T, int32_t Hq, int32_t Hk,
                                int32_t D, int32_t rot, int32_t dtype, int32_t norm, float eps, int32_t interleaved,
                                void* stream) {
    using namespace ssmp;
    if (const int st = norm_check(T, Hq, Hk, D, rot, dtype, norm, interleaved, pos, inv_freq)) return st;
    if (T == 0) return SSMP_OK;
    if ((Hq && (!q || !yq)) || (Hk && (!k || !yk))) return SSMP_ERR_NULL;
    if (!aligned16(q, k, yq, yk)) return SSMP_ERR_ALIGN;
    NormArgs a = norm_args(T, Hq, Hk, D, rot, norm, eps, interleaved, wq, wk, pos, inv_freq);
    a.x[0] = q;
    a.x[1] = k;
    a.y[0] = yq;
    a.y[1] = yk;
    const int64_t blocks = (T * a.hsplit + kNormWaves - 1) / kNormWaves;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dtype == SSMP_F32) launch_norm_d<float>(a, false, false, blocks, s);
    else launch_norm_d<uint16_t>(a, false, false, blocks, s);
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

extern "C" size_t qk_norm_pack_bwd_workspace_bytes(int64_t T, int32_t Hq, int32_t Hk, int32_t D) {
    using namespace ssmp;
    if (!norm_sizes_ok(T, Hq, Hk, D) || D > kNormMaxD || T == 0) return 0;
    return (size_t)norm_bwd_rows(T, Hq + Hk, D) * 2 * D * sizeof(float);
}

extern "C" int qk_norm_pack_bwd(const void* q, const void* k, const float* wq, const float* wk, const int32_t* pos,
                                const float* inv_freq, const void* dyq, const void* dyk, void* dq, void* dk,
                                float* dwq, float* dwk, void* workspace, size_t workspace_bytes, int64_t T,
                                int32_t Hq, int32_t Hk, int32_t D, int32_t rot, int32_t dtype, int32_t norm,
                                float eps, int32_t interleaved, void* stream) {
    using namespace ssmp;
    if (const int st = norm_check(T, Hq, Hk, D, rot, dtype, norm, interleaved, pos, inv_freq)) return st;
    if ((dwq && !wq) || (dwk && !wk)) return SSMP_ERR_NULL;
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (T == 0) {
        if (const int st = zero_f32(dwq, D, s)) return st;
        return zero_f32(dwk, D, s);
    }
    if ((Hq && (!q || !dyq || !dq)) || (Hk && (!k || !dyk || !dk))) return SSMP_ERR_NULL;
    if (!aligned16(q, k, dyq, dyk, dq, dk)) return SSMP_ERR_ALIGN;
    const bool dw = dwq || dwk;
    if (dw && (!workspace || workspace_bytes < qk_norm_pack_bwd_workspace_bytes(T, Hq, Hk, D)))
        return SSMP_ERR_WORKSPACE;
    if (dw && !aligned16(workspace)) return SSMP_ERR_ALIGN;
    NormArgs a = norm_args(T, Hq, Hk, D, rot, norm, eps, interleaved, wq, wk, pos, inv_freq);
    a.x[0] = q;
    a.x[1] = k;
    a.dy[0] = dyq;
    a.dy[1] = dyk;
    a.y[0] = dq;
    a.y[1] = dk;
    a.part = static_cast<float*>(workspace);
    const int64_t blocks = norm_bwd_blocks(T, a.hsplit);
    if (dtype == SSMP_F32) launch_norm_d<float>(a, true, dw, blocks, s);
    else launch_norm_d<uint16_t>(a, true, dw, blocks, s);
    SSMP_LAUNCH_CHECK();
    if (dw) {
        k_qk_norm_dw<><<<(unsigned)(2 * D), kWave, 0, s>>>(a.part, blocks, D, dwq, dwk);
        SSMP_LAUNCH_CHECK();
    }
    return SSMP_OK;
}
