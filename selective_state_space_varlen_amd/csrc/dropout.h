// Dropout from a counter: which elements are kept follows from their index
// and two numbers in device memory, so the backward forms the mask again and
// nothing stores it. The numbers are those of Philox4x32-10 (J. Salmon et al.,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): its 128 bits are the
// eight 16-bit numbers of eight consecutive elements.
#pragma once

#include <math.h>

#include "delta_common.h"

namespace ssmp {

// An element is dropped where its number is below cut: with probability
// cut / 65536. Sixteen bits an element, as ten rounds for every four elements
// would take longer than their bytes: 20 32-bit products a round trip, at a
// quarter of the rate of others.
struct Drop {
    const uint64_t* rng;  // the seed (Philox's key) and the stream (the counter's upper half)
    uint32_t cut;
    float by;             // 1 / (1 - cut / 65536)
};
// false: p is not in [0, 1) at that resolution
inline bool make_drop(double p, const uint64_t* rng, Drop& d) {
    if (!(p >= 0.0) || p >= 1.0) return false;
    const long cut = lrint(65536.0 * p);
    if (cut > 65535) return false;
    d.rng = rng;
    d.cut = (uint32_t)cut;
    d.by = (float)(65536.0 / (double)(65536 - cut));
    return true;
}

struct Philox {
    uint32_t k0, k1, s0, s1;
    __device__ __forceinline__ explicit Philox(const Drop& d) {
        const uint64_t seed = d.rng[0], stream = d.rng[1];
        k0 = (uint32_t)seed;
        k1 = (uint32_t)(seed >> 32);
        s0 = (uint32_t)stream;
        s1 = (uint32_t)(stream >> 32);
    }
    // numbers 8 n .. 8 n + 7, two to a word, the lower half first
    __device__ __forceinline__ u32x4 operator()(uint64_t n) const {
        uint32_t a = (uint32_t)n, b = (uint32_t)(n >> 32), c = s0, d = s1, x = k0, y = k1;
#pragma unroll
        for (int r = 0; r < 10; ++r) {
            const uint64_t u = (uint64_t)a * 0xD2511F53u, w = (uint64_t)c * 0xCD9E8D57u;
            a = (uint32_t)(w >> 32) ^ b ^ x;
            b = (uint32_t)w;
            c = (uint32_t)(u >> 32) ^ d ^ y;
            d = (uint32_t)u;
            x += 0x9E3779B9u;
            y += 0xBB67AE85u;
        }
        return u32x4{a, b, c, d};
    }
};
__device__ __forceinline__ uint32_t number_of(const u32x4& w, int e) {
    return e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xffffu;
}
// v[e] of elements 8 n + e: kept and divided by what is kept, or zero whatever it was
__device__ __forceinline__ void drop8(const Philox& ph, const Drop& d, uint64_t n, float (&v)[8]) {
    const u32x4 w = ph(n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = number_of(w, e) >= d.cut ? v[e] * d.by : 0.0f;
}
__device__ __forceinline__ float drop1(const Philox& ph, const Drop& d, uint64_t i, float v) {
    const u32x4 w = ph(i >> 3);
    const int e = (int)(i & 7);
    const uint32_t x = e & 4 ? (e & 2 ? w[3] : w[2]) : (e & 2 ? w[1] : w[0]);
    return (e & 1 ? x >> 16 : x & 0xffffu) >= d.cut ? v * d.by : 0.0f;
}

// V elements of a row on their way: 8 as two or one wide access, or a single
// one. ONCE: with a temporal hint that nothing of it is to stay in the caches.
template <typename T, int V>
struct Piece;
template <typename T>
struct Piece<T, 8> {
    Unit<T> u;
    using W = typename std::conditional<sizeof(T) == 2, u32x4, f32x4>::type;  // of a wide access
    template <bool ONCE = false>
    static __device__ __forceinline__ W wide(const W* p) {
        if constexpr (ONCE) return __builtin_nontemporal_load(p);
        else return *p;
    }
    template <bool ONCE = false>
    static __device__ __forceinline__ void wide(W* p, const W& w) {
        if constexpr (ONCE) __builtin_nontemporal_store(w, p);
        else *p = w;
    }
    template <bool ONCE = false>
    __device__ __forceinline__ void load(const T* p) {
        const W* const at = reinterpret_cast<const W*>(p);
        if constexpr (sizeof(T) == 2) {
            u.w = wide<ONCE>(at);
        } else {
            u.w[0] = wide<ONCE>(at);
            u.w[1] = wide<ONCE>(at + 1);
        }
    }
    __device__ __forceinline__ void zero() { u = {}; }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = bf16_to_f32(u.w[e]);
                v[2 * e + 1] = bf16_hi_to_f32(u.w[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = u.w[e >> 2][e & 3];
        }
    }
    template <bool ONCE = false>
    static __device__ __forceinline__ void store(T* p, const float (&v)[8]) {
        Unit<T> o;
        o.pack(v);
        W* const at = reinterpret_cast<W*>(p);
        if constexpr (sizeof(T) == 2) {
            wide<ONCE>(at, o.w);
        } else {
            wide<ONCE>(at, o.w[0]);
            wide<ONCE>(at + 1, o.w[1]);
        }
    }
};
template <typename T>
struct Piece<T, 1> {
    T x;
    __device__ __forceinline__ void load(const T* p) { x = *p; }
    __device__ __forceinline__ void zero() { x = {}; }
    __device__ __forceinline__ void get(float (&v)[1]) const {
        if constexpr (sizeof(T) == 2) v[0] = bf16_to_f32(x);
        else v[0] = x;
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { Elt<T>::st(p, 0, v[0]); }
};

}  // namespace ssmp
