// element.cuh -- element types of the layer kernels (f32, f16, bf16) and their
// vector accesses: V elements as one 16-byte access, or one element.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "hash32.cuh"
#include "internal.h"

namespace rngk {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two f32 rounded to a pair of 16-bit values in one register, a in the low half.
template <class T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}

// The bits of V elements of T as they travel: whole 32-bit registers, or one
// element.
template <class T, int V>
struct Raw {
    static_assert(V * sizeof(T) % 4 == 0, "whole registers");
    uint32_t w[V * sizeof(T) / 4];
};
template <>
struct Raw<__half, 1> {
    __half w;
};
template <>
struct Raw<__nv_bfloat16, 1> {
    __nv_bfloat16 w;
};

// V elements at p: 16-byte accesses (p aligned to them), or one element.  Streaming (evict-first) for activations,
// which are read once; plain for weights, which every row reads.
template <bool kStream, class T, int V>
__device__ __forceinline__ Raw<T, V> load(const T *p)
{
    Raw<T, V> r;
    if constexpr (V == 1) {
        *reinterpret_cast<T *>(&r) = kStream ? __ldcs(p) : *p;
    } else {
#pragma unroll
        for (int i = 0; i < static_cast<int>(V * sizeof(T) / 16); ++i) {
            const uint4 *q = reinterpret_cast<const uint4 *>(p) + i;
            const uint4 a = kStream ? __ldcs(q) : *q;
            r.w[4 * i] = a.x, r.w[4 * i + 1] = a.y, r.w[4 * i + 2] = a.z, r.w[4 * i + 3] = a.w;
        }
    }
    return r;
}

template <class T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V> &r, float (&o)[V])
{
    if constexpr (V == 1) {
        o[0] = to_f32(*reinterpret_cast<const T *>(&r));
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = __uint_as_float(r.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            if constexpr (sizeof(T) == 2) {
                if constexpr (std::is_same<T, __nv_bfloat16>::value) {  // a bfloat16 is the high half of its f32
                    o[2 * i] = __uint_as_float(r.w[i] << 16), o[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&r.w[i]));
                    o[2 * i] = f.x, o[2 * i + 1] = f.y;
                }
            }
        }
    }
}

template <class T, int V>
__device__ __forceinline__ void store(T *p, const float (&v)[V])
{
    if constexpr (V == 1) {
        *p = from_f32<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i)
            __stcs(reinterpret_cast<float4 *>(p) + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < V / 8; ++i)
            __stcs(reinterpret_cast<uint4 *>(p) + i,
                   make_uint4(pack2<T>(v[8 * i], v[8 * i + 1]), pack2<T>(v[8 * i + 2], v[8 * i + 3]),
                              pack2<T>(v[8 * i + 4], v[8 * i + 5]), pack2<T>(v[8 * i + 6], v[8 * i + 7])));
    }
}

// What rounding a pair to T's packed h has left of it, rounded likewise.
template <class T>
__device__ __forceinline__ uint32_t rest2(float2 v, uint32_t h)
{
    Raw<T, 8> r;
    r.w[0] = h, r.w[1] = r.w[2] = r.w[3] = 0;
    float o[8];
    unpack<T, 8>(r, o);
    return pack2<T>(v.x - o[0], v.y - o[1]);
}

// Two f32 at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)),
          "l"(*reinterpret_cast<uint64_t *>(&c)));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(*reinterpret_cast<uint64_t *>(&d))
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return d;
}

// The same over V elements (one by one for V = 1): d = a b + c, d = a + b.
template <int V>
__device__ __forceinline__ void fma_all(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V])
{
    if constexpr (V == 1) {
        d[0] = fmaf(a[0], b[0], c[0]);
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 r = fma2(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]), make_float2(c[k], c[k + 1]));
            d[k] = r.x, d[k + 1] = r.y;
        }
    }
}
template <int V>
__device__ __forceinline__ void fma_all(float (&d)[V], const float (&a)[V], float b, float c)
{
    if constexpr (V == 1) {
        d[0] = fmaf(a[0], b, c);
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 r = fma2(make_float2(a[k], a[k + 1]), make_float2(b, b), make_float2(c, c));
            d[k] = r.x, d[k + 1] = r.y;
        }
    }
}
template <int V>
__device__ __forceinline__ void fma_all(float (&d)[V], const float (&a)[V], float b, const float (&c)[V])
{
    if constexpr (V == 1) {
        d[0] = fmaf(a[0], b, c[0]);
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 r = fma2(make_float2(a[k], a[k + 1]), make_float2(b, b), make_float2(c[k], c[k + 1]));
            d[k] = r.x, d[k + 1] = r.y;
        }
    }
}
template <int V>
__device__ __forceinline__ void add_all(float (&d)[V], const float (&a)[V], const float (&b)[V])
{
    if constexpr (V == 1) {
        d[0] = a[0] + b[0];
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 r = add2(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]));
            d[k] = r.x, d[k + 1] = r.y;
        }
    }
}
template <int V>
__device__ __forceinline__ void mul_all(float (&d)[V], const float (&a)[V], const float (&b)[V])
{
    if constexpr (V == 1) {
        d[0] = a[0] * b[0];
    } else {
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            const float2 r = mul2(make_float2(a[k], a[k + 1]), make_float2(b[k], b[k + 1]));
            d[k] = r.x, d[k + 1] = r.y;
        }
    }
}

// V weights, ones where there are none.
template <class W, int V>
__device__ __forceinline__ Raw<W, V> load_or_one(const void *p, uint32_t at)
{
    if (p) return load<false, W, V>(static_cast<const W *>(p) + at);
    Raw<W, V> r;
    W *w = reinterpret_cast<W *>(&r);
#pragma unroll
    for (int k = 0; k < V; ++k) w[k] = from_f32<W>(1.0f);
    return r;
}

// Dropout as the layer kernels apply it: keep iff the draw's low 23 bits m
// reach the threshold T = ceil(p 2^23); the scale 1 / (1 - p) is multiplied by
// the caller.  threshold 0 (p = 0) keeps everything.
//
// The attention kernels are bound by the hash's logic operations (the ALU pipe
// takes one warp instruction in two cycles), so there the decision is made on
// the FMA pipe (11.9 cycles a warp and scheduler for 32 decisions and products,
// against 14.3 with a compare and a select):
// 1 + m 2^-23 is put together from the draw by one byte permutation and one
// logic operation, and 2^30 (1 + m 2^-23) - (2^30 + 2^7 (T - 1)) = 2^7 (m - T +
// 1), which a multiply-add gives exactly, saturates to 1 for m >= T and to 0
// below.
struct Mask {
    uint32_t key, threshold;
    float scale;
    float bar;  // -(2^30 + 2^7 (T - 1)), exact for T >= 1
};

inline Mask make_mask(float p, uint32_t seed)
{
    // keep iff m 2^-23 >= p  <=>  m >= ceil(p 2^23), exact in binary64
    const uint32_t t = static_cast<uint32_t>(std::ceil(static_cast<double>(p) * 8388608.0));
    return Mask{seed_key(seed), t, 1.0f / (1.0f - p), -(1073741824.0f + 128.0f * (static_cast<float>(t) - 1.0f))};
}

// The decision itself, for kernels that HBM bounds and whose dropped values
// may be infinite or NaN (a product with 0 would keep those).
__device__ __forceinline__ bool keeps(const Mask &m, uint32_t c)
{
    return (draw32(m.key, c) & 0x7FFFFFu) >= m.threshold;
}

// V adjacent elements dropped or scaled by 1 / (1 - p).  Their counters c, c + 1,
// ... share the high half but for one group in 2^16 / V.
template <int V>
__device__ __forceinline__ void drop_all(const Mask &m, uint32_t c, float (&v)[V])
{
    if (V > 1 && ((c ^ (c + (V - 1u))) >> 16) == 0u) {
        const uint32_t key = m.key ^ (c >> 16);
#pragma unroll
        for (uint32_t k = 0; k < V; ++k)
            v[k] = (lowbias32::hash32_rounds((c + k) ^ key) & 0x7FFFFFu) >= m.threshold ? v[k] * m.scale : 0.0f;
    } else {
#pragma unroll
        for (uint32_t k = 0; k < V; ++k) v[k] = keeps(m, c + k) ? v[k] * m.scale : 0.0f;
    }
}

// 1 for a kept element, 0 for a dropped one, from hash32 after its first
// xorshift with the key.
__device__ __forceinline__ float kept_of(const Mask &m, uint32_t x)
{
    x *= 0x7FEB352Du;
    x ^= x >> 15;
    x *= 0x846CA68Bu;
    const uint32_t high = __byte_perm(x, 0x3F800000u, 0x7632);  // x >> 16 under the exponent of 1.0
    float k;
    asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(k) : "f"(__uint_as_float(high ^ (x & 0x7FFFFFu))), "f"(1073741824.0f), "f"(m.bar));
    return k;
}
__device__ __forceinline__ float kept(const Mask &m, uint32_t c) { return kept_of(m, c ^ (c >> 16) ^ m.key); }

// Whether the counters c .. c + n - 1 share their high halves, in every lane of
// the warp: then kept_of(m, (c + e) ^ high_key(m, c)) is kept(m, c + e).
__device__ __forceinline__ bool one_high_half(uint32_t c, uint32_t n)
{
    return __all_sync(0xFFFFFFFFu, ((c ^ (c + (n - 1u))) >> 16) == 0u);
}
__device__ __forceinline__ uint32_t high_key(const Mask &m, uint32_t c) { return m.key ^ (c >> 16); }

// f(e, k) for e = 0 .. 31 in steps of 2, k the pair of factors (1 kept, 0
// dropped) of the counters c + e and c + e + 1.
template <bool kDrop, class F>
__device__ __forceinline__ void for_pairs32(const Mask &m, uint32_t c, F &&f)
{
    if (!kDrop) {
#pragma unroll
        for (uint32_t e = 0; e < 32; e += 2) f(e, make_float2(1.0f, 1.0f));
    } else if (one_high_half(c, 32)) {
        const uint32_t key = high_key(m, c);
#pragma unroll
        for (uint32_t e = 0; e < 32; e += 2)
            f(e, make_float2(kept_of(m, (c + e) ^ key), kept_of(m, (c + e + 1) ^ key)));
    } else {  // the high half changes on the way
#pragma unroll
        for (uint32_t e = 0; e < 32; e += 2) f(e, make_float2(kept(m, c + e), kept(m, c + e + 1)));
    }
}

}  // namespace rngk
