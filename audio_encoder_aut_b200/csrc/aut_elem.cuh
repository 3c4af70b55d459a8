// Loads and stores of 8 consecutive elements (16 or 32 bytes) of any of the
// element types, as fp32 in registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "aut_ptx.cuh"

namespace aut {

// Eight elements as they are in memory.
template <typename T>
struct Pack8 {
    uint32_t w[4];  // two 16-bit elements each
    AUT_DEV void load(const T *p) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x;
        w[1] = u.y;
        w[2] = u.z;
        w[3] = u.w;
    }
    AUT_DEV void values(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = pair(w[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    static AUT_DEV float2 pair(uint32_t u) {
        if constexpr (std::is_same<T, __half>::value)
            return __half22float2(*reinterpret_cast<const __half2 *>(&u));
        else  // bf16 is the upper half of the fp32 word
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
};
template <>
struct Pack8<float> {
    uint32_t w[8];
    AUT_DEV void load(const float *p) {
        const uint4 a = reinterpret_cast<const uint4 *>(p)[0], b = reinterpret_cast<const uint4 *>(p)[1];
        w[0] = a.x;
        w[1] = a.y;
        w[2] = a.z;
        w[3] = a.w;
        w[4] = b.x;
        w[5] = b.y;
        w[6] = b.z;
        w[7] = b.w;
    }
    AUT_DEV void values(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
    }
};

template <typename T>
AUT_DEV void load8(const T *p, float (&v)[8]) {
    Pack8<T> r;
    r.load(p);
    r.values(v);
}

// Two fp32 values as a packed pair of 16-bit ones, rounded to nearest even.
template <typename T>
AUT_DEV uint32_t pack2(float a, float b);
template <>
AUT_DEV uint32_t pack2<__nv_bfloat16>(float a, float b) {
    return pack_bf16x2(a, b);
}
template <>
AUT_DEV uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <typename T>
AUT_DEV void store8(T *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]),
                   pack2<T>(v[6], v[7]));
}
template <>
AUT_DEV void store8<float>(float *p, const float (&v)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace aut
