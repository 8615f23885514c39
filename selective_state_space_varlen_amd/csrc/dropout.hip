// dropout_pack: y = residual + drop(x), and its gradient drop(dy).
// Bound by HBM beside the generator's products.
#include "dropout.h"

namespace ssmp {

template <typename T, bool ADD>
__global__ __launch_bounds__(256) void k_dropout(const T* x, const T* r, T* y, Drop d, int64_t n) {
    const Philox ph(d);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i * 8 < n; i += (int64_t)gridDim.x * 256) {
        if (i * 8 + 8 <= n) {
            Piece<T, 8> a, b;
            a.load(x + i * 8);
            if constexpr (ADD) b.load(r + i * 8);
            float v[8], w[8];
            a.get(v);
            drop8(ph, d, (uint64_t)i, v);
            if constexpr (ADD) {
                b.get(w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
            }
            Piece<T, 8>::store(y + i * 8, v);
        } else {
            for (int64_t j = i * 8; j < n; ++j) {
                const float v = drop1(ph, d, (uint64_t)j, Elt<T>::ld(x, j));
                Elt<T>::st(y, j, ADD ? v + Elt<T>::ld(r, j) : v);
            }
        }
    }
}

template <typename T>
void launch_dropout(const void* x, const void* r, void* y, const Drop& d, int64_t n, hipStream_t s) {
    const int64_t want = ((n + 7) / 8 + 255) / 256;
    const unsigned blocks = (unsigned)(want < 16384 ? want : 16384);
    if (r) k_dropout<T, true><<<blocks, 256, 0, s>>>(static_cast<const T*>(x), static_cast<const T*>(r), static_cast<T*>(y), d, n);
    else k_dropout<T, false><<<blocks, 256, 0, s>>>(static_cast<const T*>(x), nullptr, static_cast<T*>(y), d, n);
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
    if (dtype == SSMP_F32) launch_dropout<float>(x, residual, y, d, n, s);
    else launch_dropout<uint16_t>(x, residual, y, d, n, s);
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
