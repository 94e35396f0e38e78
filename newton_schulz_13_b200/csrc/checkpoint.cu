// 8-bit activation checkpoints (mx.cuh): store (quantise) and restore.
//
// Bound by HBM: 2 or 4 bytes read and 1 + 1/32 written per element on the way in, the reverse on
// the way out (8192 x 14336 bf16: 57 us stored, 53 restored, 6.3 and 6.7 TB/s). Aligned rows: a thread
// owns eight consecutive elements of two places, four lanes a 32-element block; other rows: four
// elements of four places, eight lanes a block.
#include <cuda_bf16.h>
#include <stdint.h>

#include "fast_div.cuh"
#include "mx.cuh"
#include "ops_internal.h"
#include "ptx.cuh"
#include "vec_io.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;

constexpr int kAcc = 2;   // accesses per thread, kThreads apart

// per_row: 8-element accesses of a row, padded to whole blocks (a multiple of 4); total: of all
// rows, below 2^31.
template <bool X_BF16>
__global__ void __launch_bounds__(kThreads) mx_store_kernel(MxArgs a, Div per_row, uint32_t total) {
  const uint32_t t0 = blockIdx.x * (kAcc * kThreads) + threadIdx.x;
  Raw<8, X_BF16> raw[kAcc];
  uint32_t row[kAcc], c[kAcc];
  bool ok[kAcc];
#pragma unroll
  for (int j = 0; j < kAcc; ++j) {
    const uint32_t t = t0 + j * kThreads;
    row[j] = per_row.quot(t);
    c[j] = (t - row[j] * per_row.d) * 8;
    ok[j] = t < total && c[j] < a.dim;   // dim is a multiple of 8
    if (ok[j]) raw[j].load(a.x, (int64_t)row[j] * a.xs + c[j]);
  }
#pragma unroll
  for (int j = 0; j < kAcc; ++j) {
    float v[8] = {};
    if (ok[j]) raw[j].get(v);
    uint32_t m = mx_amax8(v);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));   // the four lanes of a block
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t code = mx_scale_code(m);
    if (ok[j]) {
      *reinterpret_cast<uint2*>(a.q + (int64_t)row[j] * a.qs + c[j]) = mx_pack8(v, code);
      if (!(c[j] & (kMxBlock - 1))) a.sc[(int64_t)row[j] * a.scs + c[j] / kMxBlock] = (uint8_t)code;
    }
  }
}

// Any rows: a thread has four consecutive elements of kQuad places, eight lanes a 32-element block.
// per_row: four-element groups of a row, padded to whole blocks (a multiple of 8).
constexpr int kQuad = 4;

template <bool X_BF16>
__global__ void __launch_bounds__(kThreads) mx_store_any_kernel(MxArgs a, Div per_row, uint32_t total) {
  const uint32_t t0 = blockIdx.x * (kQuad * kThreads) + threadIdx.x;
  float v[kQuad][4];
#pragma unroll
  for (int j = 0; j < kQuad; ++j) {
    const uint32_t t = t0 + j * kThreads, row = per_row.quot(t), c = (t - row * per_row.d) * 4;
    if (t < total && c < a.dim) load4_any<X_BF16>(a.x, (int64_t)row * a.xs + c, a.dim - c, v[j]);
    else v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < kQuad; ++j) {
    const uint32_t t = t0 + j * kThreads, row = per_row.quot(t), c = (t - row * per_row.d) * 4;
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, __float_as_uint(v[j][e]) & 0x7fffffffu);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (t >= total || c >= a.dim) continue;
    const uint32_t code = mx_scale_code(m);
    uint32_t w = 0x7f7f7f7fu;
    if (code != kMxNan) {
      const float s = mx_inv_scale(code);
      w = mx_pack2(v[j][0] * s, v[j][1] * s) | (mx_pack2(v[j][2] * s, v[j][3] * s) << 16);
    }
    uint8_t* const q = a.q + (int64_t)row * a.qs + c;
    if (c + 4 <= a.dim && ((uintptr_t)q & 3) == 0) {
      *reinterpret_cast<uint32_t*>(q) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.dim) q[e] = (uint8_t)(w >> (8 * e));
    }
    if (!(c & (kMxBlock - 1))) a.sc[(int64_t)row * a.scs + c / kMxBlock] = (uint8_t)code;
  }
}

__device__ __forceinline__ void zero_words(const MxArgs& a) {
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.zeros; i += kThreads) a.zero[i] = 0;
}

template <bool O_BF16>
__global__ void __launch_bounds__(kThreads) mx_restore_kernel(MxArgs a, Div per_row, uint32_t total) {
  grid_launch_dependents();
  zero_words(a);
  const uint32_t t0 = blockIdx.x * (kAcc * kThreads) + threadIdx.x;
  uint2 raw[kAcc];
  uint32_t row[kAcc], c[kAcc], code[kAcc];
#pragma unroll
  for (int j = 0; j < kAcc; ++j) {
    const uint32_t t = t0 + j * kThreads;
    row[j] = per_row.quot(t);
    c[j] = (t - row[j] * per_row.d) * 8;
    if (t >= total) continue;
    raw[j] = *reinterpret_cast<const uint2*>(a.q + (int64_t)row[j] * a.qs + c[j]);
    code[j] = a.sc[(int64_t)row[j] * a.scs + c[j] / kMxBlock];
  }
#pragma unroll
  for (int j = 0; j < kAcc; ++j) {
    if (t0 + j * kThreads >= total) break;
    const float s = mx_scale(code[j]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __fmul2_rn(mx_unpack2((i < 2 ? raw[j].x : raw[j].y) >> (16 * (i & 1))), make_float2(s, s));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
    store8<O_BF16>(a.out, (int64_t)row[j] * a.xs + c[j], v);
  }
}

// Any rows: a thread has four elements of kQuad places, from the two aligned words that hold their
// codes; out4: groups of four of out are aligned.
template <bool O_BF16>
__global__ void __launch_bounds__(kThreads) mx_restore_any_kernel(MxArgs a, Div per_row, uint32_t total, int out4) {
  grid_launch_dependents();
  zero_words(a);
  const uint32_t t0 = blockIdx.x * (kQuad * kThreads) + threadIdx.x;
  uint32_t w[kQuad], code[kQuad];
#pragma unroll
  for (int j = 0; j < kQuad; ++j) {
    const uint32_t t = t0 + j * kThreads, row = per_row.quot(t), c = (t - row * per_row.d) * 4;
    if (t >= total) continue;
    const uint8_t* const p = a.q + (int64_t)row * a.qs + c;
    const uint32_t off = (uint32_t)((uintptr_t)p & 3);
    const uint32_t* const at = reinterpret_cast<const uint32_t*>(p - off);
    // the first word holds a code of this row, and so does the second if it begins before the row's end
    const uint32_t lo = at[0], hi = off && c + 4 - off < a.dim ? at[1] : 0u;
    w[j] = __funnelshift_r(lo, hi, off * 8);
    code[j] = a.sc[(int64_t)row * a.scs + c / kMxBlock];
  }
#pragma unroll
  for (int j = 0; j < kQuad; ++j) {
    const uint32_t t = t0 + j * kThreads, row = per_row.quot(t), c = (t - row * per_row.d) * 4;
    if (t >= total) break;
    const float s = mx_scale(code[j]);
    const float2 lo = mx_unpack2(w[j]), hi = mx_unpack2(w[j] >> 16);
    const float v[4] = {lo.x * s, lo.y * s, hi.x * s, hi.y * s};
    const int64_t to = (int64_t)row * a.xs + c;
    if (out4 && c + 4 <= a.dim) {
      store4<O_BF16>(a.out, to, v);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < a.dim) store1<O_BF16>(a.out, to + e, v[e]);
    }
  }
}

bool vec8(const MxArgs& a, const void* x) {
  return a.dim % 8 == 0 && (uintptr_t)x % 16 == 0 && a.xs % 8 == 0 && (uintptr_t)a.q % 8 == 0 && a.qs % 8 == 0;
}

// A row-contiguous matrix whose rows end on a block is one long row.
MxArgs flat(MxArgs a) {
  if (a.xs == a.dim && a.qs == a.dim && a.scs * 32 == a.dim && a.rows * a.dim < (int64_t(1) << 31)) {
    a.dim *= a.rows;
    a.xs = a.qs = a.dim;
    a.scs = a.dim / 32;
    a.rows = 1;
  }
  return a;
}

// Launches over all rows, `per_row` work items each and `per_block` of them per block, in
// runs of rows that keep the item index below 2^31.
template <class K, class... More>
cudaError_t launch_rows(MxArgs a, int64_t x_size, int64_t per_row, int64_t per_block, cudaStream_t s, K kernel, More... more) {
  const int64_t most = ((int64_t(1) << 31) - 1) / per_row;
  for (int64_t r = 0; r < a.rows; r += most) {
    MxArgs b = a;
    b.rows = a.rows - r < most ? a.rows - r : most;
    if (a.x) b.x = static_cast<const char*>(a.x) + r * a.xs * x_size;
    if (a.out) b.out = static_cast<char*>(a.out) + r * a.xs * x_size;
    b.q = a.q + r * a.qs;
    b.sc = a.sc + r * a.scs;
    const int64_t total = b.rows * per_row;
    kernel<<<(unsigned)((total + per_block - 1) / per_block), kThreads, 0, s>>>(b, Div((uint32_t)per_row), (uint32_t)total, more...);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_mx_store(const MxArgs& args, int x_bf16, cudaStream_t s) {
  const MxArgs a = flat(args);
  const int64_t size = x_bf16 ? 2 : 4, blocks = (a.dim + 31) / 32;
  if (vec8(a, a.x)) return launch_rows(a, size, blocks * 4, kAcc * kThreads, s, x_bf16 ? mx_store_kernel<true> : mx_store_kernel<false>);
  return launch_rows(a, size, blocks * 8, kQuad * kThreads, s, x_bf16 ? mx_store_any_kernel<true> : mx_store_any_kernel<false>);
}

cudaError_t launch_mx_restore(const MxArgs& args, int out_bf16, cudaStream_t s) {
  const MxArgs a = flat(args);
  const int64_t size = out_bf16 ? 2 : 4;
  if (vec8(a, a.out)) return launch_rows(a, size, a.dim / 8, kAcc * kThreads, s, out_bf16 ? mx_restore_kernel<true> : mx_restore_kernel<false>);
  const int out4 = (uintptr_t)a.out % 16 == 0 && a.xs % 4 == 0;
  return launch_rows(a, size, (a.dim + 3) / 4, kQuad * kThreads, s, out_bf16 ? mx_restore_any_kernel<true> : mx_restore_any_kernel<false>,
                     out4);
}

}  // namespace muon
