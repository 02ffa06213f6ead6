// Device helpers shared by the operators around the WKV recurrence: the causal convolution, the
// selective scan and the layer norm.
#pragma once

#include "wkv_common.cuh"

namespace rwkv {

// V consecutive elements as floats; one access where V elements are 4, 8 or 16 bytes (the caller
// then guarantees that alignment), element by element otherwise.
template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
  if constexpr (sizeof(T) == 4 && V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      f[i] = x.x, f[i + 1] = x.y, f[i + 2] = x.z, f[i + 3] = x.w;
    }
  } else if constexpr (sizeof(T) == 4 && V == 2) {
    const float2 x = *reinterpret_cast<const float2*>(p);
    f[0] = x.x, f[1] = x.y;
  } else if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    constexpr int W = V / 2;  // 32-bit words
    uint32_t w[W];
    if constexpr (W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 2 * i);
        w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
      }
    } else if constexpr (W == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    } else {
      static_assert(W == 1, "16, 8 or 4 bytes");
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    static_assert(V == 1, "vector width");
    f[0] = IO<T>::to_f(*p);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The inverse of load_vec: rounds to nearest once.
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  if constexpr (sizeof(T) == 4 && V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else if constexpr (sizeof(T) == 4 && V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else if constexpr (sizeof(T) == 2 && V % 8 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 8)
      *reinterpret_cast<uint4*>(p + i) = make_uint4(pack_bf16(f[i], f[i + 1]), pack_bf16(f[i + 2], f[i + 3]),
                                                    pack_bf16(f[i + 4], f[i + 5]), pack_bf16(f[i + 6], f[i + 7]));
  } else if constexpr (sizeof(T) == 2 && V == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
  } else if constexpr (sizeof(T) == 2 && V == 2) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(f[0], f[1]);
  } else {
    static_assert(V == 1, "vector width");
    *p = IO<T>::from_f(f[0]);
  }
}

// The first n of V elements (the rest read as zero); one wide access when `vec` and all are there.
template <typename T, int V>
__device__ __forceinline__ void load_part(const T* p, int n, bool vec, float (&f)[V]) {
  if (vec && n >= V) {
    load_vec<T, V>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i < n ? IO<T>::to_f(p[i]) : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_part(T* p, int n, bool vec, const float (&f)[V]) {
  if (vec && n >= V) {
    store_vec<T, V>(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = IO<T>::from_f(f[i]);
  }
}

// V elements as loaded, kept for later: unpacking them only where they are used leaves the load in
// flight until then.
template <typename T, int V>
struct Raw {
  static constexpr int kBytes = V * (int)sizeof(T);
  uint32_t w[(kBytes + 3) / 4];

  // The first n of the V elements at p (the rest zero); `vec` as in load_part.
  __device__ __forceinline__ void load(const T* p, int n, bool vec) {
    if (vec && n >= V) {
      load(p);
    } else {
#pragma unroll
      for (int i = 0; i < (kBytes + 3) / 4; ++i) w[i] = 0u;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i >= n) continue;
        if constexpr (sizeof(T) == 4)
          w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else
          w[i / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(p)[i] << (16 * (i & 1));
      }
    }
  }
  // All V elements (aligned for wide accesses, or V = 1).
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 x = reinterpret_cast<const uint4*>(p)[i];
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      static_assert(kBytes == 2, "vector width");
      w[0] = *reinterpret_cast<const unsigned short*>(p);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kBytes + 3) / 4; ++i) w[i] = 0u;
  }
  // Elements lo .. hi - 1 of the V at p (the rest zero), one by one.
  __device__ __forceinline__ void load_range(const T* p, int lo, int hi) {
    zero();
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < lo || i >= hi) continue;
      if constexpr (sizeof(T) == 4)
        w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else
        w[i / 2] |= (uint32_t) reinterpret_cast<const unsigned short*>(p)[i] << (16 * (i & 1));
    }
  }
  // Zero outside elements lo .. hi - 1.
  __device__ __forceinline__ void keep_range(int lo, int hi) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i >= lo && i < hi) continue;
      if constexpr (sizeof(T) == 4)
        w[i] = 0u;
      else
        w[i / 2] &= (i & 1) != 0 ? 0xFFFFu : 0xFFFF0000u;
    }
  }
  // Elements 2 i and 2 i + 1 (0 behind the last).
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2((*this)[2 * i], 2 * i + 1 < V ? (*this)[2 * i + 1] : 0.f);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float((i & 1) != 0 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};

// Two fp32 operations in one instruction (sm_100 packed arithmetic); each half rounds as the single
// instruction does.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 dup2(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 ex2_2(float2 x) { return make_float2(ex2(x.x), ex2(x.y)); }

__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 e = ex2_2(mul2(x, dup2(-kL2eHi)));
  const float2 d = add2(e, dup2(1.f));
  return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
// V elements held as pairs, rounded once each.
template <typename T, int V>
__device__ __forceinline__ void store_pairs_as(T* p, const float2 (&v)[(V + 1) / 2]) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = i & 1 ? v[i / 2].y : v[i / 2].x;
  store_vec<T, V>(p, f);
}

// Logistic sigmoid 1 / (1 + 2^(-x log2 e)); saturates to 0 and 1 without NaN.
__device__ __forceinline__ float sigmoid_ex2(float x) { return rcp_approx(1.f + ex2(-kL2eHi * x)); }

}  // namespace rwkv
