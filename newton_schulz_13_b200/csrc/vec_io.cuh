// Loads and stores of bf16 or fp32 values as fp32: eight at a time (16-byte accesses; the element
// index and the base must make them aligned) or one at a time.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace muon {

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t idx, float (&v)[8]) {
  if constexpr (BF16) {
    const uint4 raw = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + idx);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + idx);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t idx, const float (&v)[8]) {
  if constexpr (BF16) {
    uint4 raw;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + idx) = raw;
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + idx);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

template <bool BF16>
__device__ __forceinline__ float load1(const void* base, int64_t idx) {
  if constexpr (BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[idx]);
  else return static_cast<const float*>(base)[idx];
}

template <bool BF16>
__device__ __forceinline__ void store1(void* base, int64_t idx, float v) {
  if constexpr (BF16) static_cast<__nv_bfloat16*>(base)[idx] = __float2bfloat16_rn(v);
  else static_cast<float*>(base)[idx] = v;
}

// Eight values, or one, as loaded: kept so while several loads are in flight, and widened at use.
template <int V, bool BF16>
struct Raw;
template <>
struct Raw<8, true> {
  uint4 r;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    r = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  // adds v in fp32 and rounds
  __device__ __forceinline__ void add(const float (&v)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __fadd2_rn(make_float2(v[2 * i], v[2 * i + 1]), __bfloat1622float2(h[i]));
      h[i] = __floats2bfloat162_rn(f.x, f.y);
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) = r;
  }
};
template <>
struct Raw<8, false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void add(const float (&v)[8]) {
    a = make_float4(a.x + v[0], a.y + v[1], a.z + v[2], a.w + v[3]);
    b = make_float4(b.x + v[4], b.y + v[5], b.z + v[6], b.w + v[7]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = a;
    q[1] = b;
  }
};
template <>
struct Raw<1, true> {
  __nv_bfloat16 r;
  __device__ __forceinline__ void load(const void* p, int64_t i) { r = static_cast<const __nv_bfloat16*>(p)[i]; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = __bfloat162float(r); }
};
template <>
struct Raw<1, false> {
  float r;
  __device__ __forceinline__ void load(const void* p, int64_t i) { r = static_cast<const float*>(p)[i]; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = r; }
};

// Four consecutive elements at any element index, zeros past the `left` that remain in the row (at
// least one). bf16 come in the aligned words that hold them; each word read holds one that remains.
template <bool BF16>
__device__ __forceinline__ void load4_any(const void* base, int64_t idx, int64_t left, float (&v)[4]) {
  if constexpr (BF16) {
    const uintptr_t p = (uintptr_t)(static_cast<const __nv_bfloat16*>(base) + idx), off = p & 2;
    const uint32_t* const at = reinterpret_cast<const uint32_t*>(p - off);
    const int64_t bytes = left * 2 + (int64_t)off;
    const uint32_t w0 = at[0], w1 = bytes > 4 ? at[1] : 0u, w2 = off && bytes > 8 ? at[2] : 0u;
    const uint32_t a = __funnelshift_r(w0, w1, off * 8), b = __funnelshift_r(w1, w2, off * 8);
    v[0] = __uint_as_float(a << 16);
    v[1] = left > 1 ? __uint_as_float(a & 0xffff0000u) : 0.0f;
    v[2] = left > 2 ? __uint_as_float(b << 16) : 0.0f;
    v[3] = left > 3 ? __uint_as_float(b & 0xffff0000u) : 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = e < left ? static_cast<const float*>(base)[idx + e] : 0.0f;
  }
}

// Four elements at an index aligned to four.
template <bool BF16>
__device__ __forceinline__ void store4(void* base, int64_t idx, const float (&v)[4]) {
  if constexpr (BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + idx) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(base) + idx) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// V = 8 or 1 elements, for kernels that serve aligned and unaligned rows with one body.
template <int V, bool BF16>
__device__ __forceinline__ void load_v(const void* base, int64_t idx, float (&v)[V]) {
  if constexpr (V == 8) load8<BF16>(base, idx, v);
  else v[0] = load1<BF16>(base, idx);
}

template <int V, bool BF16>
__device__ __forceinline__ void store_v(void* base, int64_t idx, const float (&v)[V]) {
  if constexpr (V == 8) store8<BF16>(base, idx, v);
  else store1<BF16>(base, idx, v[0]);
}

}  // namespace muon
