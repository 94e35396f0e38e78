// 8-bit activation checkpoints (mx.cuh): store (quantise) and restore.
//
// Bound by HBM: 2 or 4 bytes read and 1 + 1/32 written per element on the way in, the reverse on
// the way out. Aligned rows: a thread owns 16 consecutive elements, two lanes a 32-element block;
// other rows: a lane owns one element, a warp one block.
#include <cuda_bf16.h>
#include <stdint.h>

#include "mx.cuh"
#include "ops_internal.h"
#include "vec_io.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;

template <bool X_BF16>
__global__ void __launch_bounds__(kThreads) mx_store_kernel(MxArgs a) {
  const int64_t per_row = (a.dim + 31) / 32 * 2;   // 16-element pieces, an even number
  const int64_t total = a.rows * per_row;
  // the loop bound is the same for both lanes of a block (total is even)
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / per_row, p = t - row * per_row;
    const int64_t c = p * 16;
    const bool ok = c < a.dim;   // dim is a multiple of 16
    float v[2][8] = {};
    if (ok) {
      load8<X_BF16>(a.x, row * a.xs + c, v[0]);
      load8<X_BF16>(a.x, row * a.xs + c + 8, v[1]);
    }
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, max(__float_as_uint(v[0][e]) & 0x7fffffffu, __float_as_uint(v[1][e]) & 0x7fffffffu));
    const uint32_t pair = 3u << (threadIdx.x & 30);
    m = max(m, __shfl_xor_sync(pair, m, 1));
    const uint32_t code = mx_scale_code(m);
    if (ok) {
      const uint2 lo = mx_pack8(v[0], code), hi = mx_pack8(v[1], code);
      *reinterpret_cast<uint4*>(a.q + row * a.qs + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      if (!(p & 1)) a.sc[row * a.scs + p / 2] = (uint8_t)code;
    }
  }
}

template <bool X_BF16>
__global__ void __launch_bounds__(kThreads) mx_store_any_kernel(MxArgs a) {
  const int64_t per_row = (a.dim + 31) / 32, total = a.rows * per_row;
  const int lane = threadIdx.x & 31;
  for (int64_t b = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; b < total; b += ((int64_t)gridDim.x * kThreads) >> 5) {
    const int64_t row = b / per_row, blk = b - row * per_row;
    const int64_t c = blk * 32 + lane;
    const bool ok = c < a.dim;
    const float v = ok ? load1<X_BF16>(a.x, row * a.xs + c) : 0.0f;
    uint32_t m = __float_as_uint(v) & 0x7fffffffu;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t code = mx_scale_code(m);
    if (ok) a.q[row * a.qs + c] = (uint8_t)mx_pack1(v, code);
    if (lane == 0) a.sc[row * a.scs + blk] = (uint8_t)code;
  }
}

template <bool O_BF16>
__global__ void __launch_bounds__(kThreads) mx_restore_kernel(MxArgs a) {
  const int64_t per_row = a.dim / 16, total = a.rows * per_row;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / per_row, p = t - row * per_row;
    const uint4 raw = *reinterpret_cast<const uint4*>(a.q + row * a.qs + p * 16);
    const float s = mx_scale(a.sc[row * a.scs + p / 2]);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = mx_unpack2(w[i >> 1] >> (16 * (i & 1)));
      v[i >> 2][(2 * i) & 7] = f.x * s;
      v[i >> 2][(2 * i + 1) & 7] = f.y * s;
    }
    store8<O_BF16>(a.out, row * a.xs + p * 16, v[0]);
    store8<O_BF16>(a.out, row * a.xs + p * 16 + 8, v[1]);
  }
}

template <bool O_BF16>
__global__ void __launch_bounds__(kThreads) mx_restore_any_kernel(MxArgs a) {
  const int64_t total = a.rows * a.dim;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / a.dim, c = t - row * a.dim;
    const float v = mx_unpack1(a.q[row * a.qs + c]) * mx_scale(a.sc[row * a.scs + c / 32]);
    store1<O_BF16>(a.out, row * a.xs + c, v);
  }
}

bool vec16(const MxArgs& a, const void* x) {
  return a.dim % 16 == 0 && (uintptr_t)x % 16 == 0 && a.xs % 8 == 0 && (uintptr_t)a.q % 16 == 0 && a.qs % 16 == 0;
}

int grid_of(int64_t threads, int sms) {
  const int64_t b = (threads + kThreads - 1) / kThreads;
  const int64_t cap = (int64_t)sms * 32;
  return (int)(b < 1 ? 1 : (b < cap ? b : cap));
}

}  // namespace

cudaError_t launch_mx_store(const MxArgs& a, int x_bf16, int sms, cudaStream_t s) {
  if (vec16(a, a.x)) {
    const int g = grid_of(a.rows * ((a.dim + 31) / 32 * 2), sms);
    if (x_bf16) mx_store_kernel<true><<<g, kThreads, 0, s>>>(a);
    else mx_store_kernel<false><<<g, kThreads, 0, s>>>(a);
  } else {
    const int g = grid_of(a.rows * ((a.dim + 31) / 32) * 32, sms);
    if (x_bf16) mx_store_any_kernel<true><<<g, kThreads, 0, s>>>(a);
    else mx_store_any_kernel<false><<<g, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_mx_restore(const MxArgs& a, int out_bf16, int sms, cudaStream_t s) {
  if (vec16(a, a.out)) {
    const int g = grid_of(a.rows * (a.dim / 16), sms);
    if (out_bf16) mx_restore_kernel<true><<<g, kThreads, 0, s>>>(a);
    else mx_restore_kernel<false><<<g, kThreads, 0, s>>>(a);
  } else {
    const int g = grid_of(a.rows * a.dim, sms);
    if (out_bf16) mx_restore_any_kernel<true><<<g, kThreads, 0, s>>>(a);
    else mx_restore_any_kernel<false><<<g, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace muon
