// What the sequence operators (the causal convolution and the selective scan)
// share: element types, vector loads and stores, the activations.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convfwd {

typedef __bf16 bf16_t;
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

#define SEQ_DEV __device__ __forceinline__

// V elements of T moved as one access (V * sizeof(T) is 2, 4, 8 or 16 bytes)
template <typename T, int V> struct Pack {
    typedef T type __attribute__((ext_vector_type(V)));
};
template <typename T> struct Pack<T, 1> {
    typedef T type;
};

template <typename T, int V> SEQ_DEV float pack_get(const typename Pack<T, V>::type &q, int i)
{
    if constexpr (V == 1) return (float)q;
    else return (float)q[i];
}

template <typename T, int V> SEQ_DEV void load_f32(const T *p, float (&v)[V])
{
    if constexpr (V == 1) {
        v[0] = (float)p[0];
    } else {
        const typename Pack<T, V>::type q = *reinterpret_cast<const typename Pack<T, V>::type *>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)q[i];
    }
}

// the one rounding of a result (nearest-even for bf16)
template <typename T, int V> SEQ_DEV void store_f32(T *p, const float (&v)[V])
{
    if constexpr (V == 1) {
        p[0] = (T)v[0];
    } else {
        typename Pack<T, V>::type q;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = (T)v[i];
        *reinterpret_cast<typename Pack<T, V>::type *>(p) = q;
    }
}
// ... of an output that no kernel of the call reads back, past the caches
template <typename T, int V> SEQ_DEV void stream_f32(T *p, const float (&v)[V])
{
    if constexpr (V == 1) {
        __builtin_nontemporal_store((T)v[0], p);
    } else {
        typename Pack<T, V>::type q;
#pragma unroll
        for (int i = 0; i < V; ++i) q[i] = (T)v[i];
        __builtin_nontemporal_store(q, reinterpret_cast<typename Pack<T, V>::type *>(p));
    }
}

constexpr float kLog2e = 1.4426950408889634f;

SEQ_DEV float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// 1 / (1 + e^-v): e^-v overflows to infinity for v < -88 and the reciprocal is 0
SEQ_DEV float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.0f + exp2_fast(-kLog2e * v)); }

// log(1 + e^v) without overflow, and exact to a few ulp where e^v is small
SEQ_DEV float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

// a sequence's length, within its row of L tokens whatever the caller's array holds
SEQ_DEV int64_t seq_len(const int32_t *lengths, int64_t n, int64_t L)
{
    if (!lengths) return L;
    const int64_t v = lengths[n];
    return v < 0 ? 0 : v > L ? L : v;
}

}  // namespace convfwd
