// dropout_pack: y = residual + drop(x), and its gradient drop(dy).
// Bound by HBM: 32768 rows of 4096 in bf16, other tensors at each call, take
// 133 us with a residual (6.0 TB/s) beside the generator's ten rounds for every
// eight elements.
#include "dropout.h"

namespace ssmp {

template <typename T, bool ADD, bool ONCE>
__global__ __launch_bounds__(256) void k_dropout(const T* x, const T* r, T* y, Drop d, int64_t n) {
    const Philox ph(d);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i * 8 < n; i += (int64_t)gridDim.x * 256) {
        if (i * 8 + 8 <= n) {
            Piece<T, 8> a, b;
            a.template load<ONCE>(x + i * 8);
            if constexpr (ADD) b.template load<ONCE>(r + i * 8);
            float v[8], w[8];
            a.get(v);
            drop8(ph, d, (uint64_t)i, v);
            if constexpr (ADD) {
                b.get(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
            }
            Piece<T, 8>::template store<ONCE>(y + i * 8, v);
        } else {
            for (int64_t j = i * 8; j < n; ++j) {
                const float v = drop1(ph, d, (uint64_t)j, Elt<T>::ld(x, j));
                Elt<T>::st(y, j, ADD ? v + Elt<T>::ld(r, j) : v);
            }
        }
    }
}

// From this size of each tensor on, nothing of it would stay in the last cache
// (256 MiB) until it is used again, and accesses say so. Dropout with a
// residual, alone and with a norm that reads the result, in us:
//   MiB a tensor    16           32           64           128           256
//   said            9.9, 26.1    17.6, 42.0   33.7, 72.6   65.2, 130     133, 253
//   not said       11.4, 26.0    19.5, 40.3   37.0, 72.5   72.4, 140     143, 264
constexpr int64_t kOnceBytes = int64_t(128) << 20;
template <typename T, bool ADD>
void launch_dropout(const void* x, const void* r, void* y, const Drop& d, int64_t n, hipStream_t s) {
    const int64_t want = ((n + 7) / 8 + 255) / 256;
    const unsigned blocks = (unsigned)(want < 16384 ? want : 16384);
    const T *const xp = static_cast<const T*>(x), *const rp = static_cast<const T*>(r);
    if (n * (int64_t)sizeof(T) >= kOnceBytes) k_dropout<T, ADD, true><<<blocks, 256, 0, s>>>(xp, rp, static_cast<T*>(y), d, n);
    else k_dropout<T, ADD, false><<<blocks, 256, 0, s>>>(xp, rp, static_cast<T*>(y), d, n);
}

inline int dropout(const void* x, const void* residual, const uint64_t* rng, void* y, int64_t n, int32_t dtype, double p,
                   void* stream) {
    if (n < 0 || n >= (int64_t(1) << 40)) return SSMP_ERR_SHAPE;
    if (dtype != SSMP_F32 && dtype != SSMP_BF16) return SSMP_ERR_UNSUPPORTED;
    Drop d;
    if (!make_drop(p, rng, d)) return SSMP_ERR_SHAPE;
    if (n == 0) return SSMP_OK;
    if (!x || !y || !rng) return SSMP_ERR_NULL;
    if (!aligned16(x, residual, y)) return SSMP_ERR_ALIGN;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const auto launch = [&](auto add) {
        constexpr bool ADD = decltype(add)::value;
        if (dtype == SSMP_F32) launch_dropout<float, ADD>(x, residual, y, d, n, s);
        else launch_dropout<uint16_t, ADD>(x, residual, y, d, n, s);
    };
    if (residual) launch(std::true_type{});
    else launch(std::false_type{});
    SSMP_LAUNCH_CHECK();
    return SSMP_OK;
}

}  // namespace ssmp

extern "C" int dropout_pack_fwd(const void* x, const void* residual, const uint64_t* rng, void* y, int64_t n,
                                int32_t dtype, double p, void* stream) {
    return ssmp::dropout(x, residual, rng, y, n, dtype, p, stream);
}
extern "C" int dropout_pack_bwd(const void* dy, const uint64_t* rng, void* dx, int64_t n, int32_t dtype, double p,
                                void* stream) {
    return ssmp::dropout(dy, nullptr, rng, dx, n, dtype, p, stream);
}
