// Root-mean-square norm with the residual's addition and an output in 8 bits with scales, and its
// gradient:
//   h = round(x + r)   (in r's type; h = x without a residual)
//   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w,   checkpoint of y (mx.cuh)
//   with n = h rstd and a = dy w:   dx = rstd (a - n mean(a n)) + dh,   dw (+)= sum over rows dy n
// All sums and statistics are fp32. The norm is taken of the rounded h, which is what the gradient
// reads back, and the checkpoint of the unrounded y, so each of its values is rounded once.
//
// Both are bound by HBM: every element is read and written once. A row belongs to `tpr` threads
// (a multiple of 32) that hold it in registers, VPT accesses of V elements each: V = 8 (16-byte
// accesses) when every row is aligned to eight elements, V = 1 otherwise, where a warp reads 32
// consecutive elements per access. In both, a 32-element checkpoint block lies within a warp: four
// lanes of one access (V = 8) or all 32 (V = 1).
#include <cuda_bf16.h>
#include <stdint.h>

#include "mx.cuh"
#include "ops_internal.h"
#include "ptx.cuh"
#include "vec_io.cuh"

namespace muon {
namespace {

// Sum over the `tpr` threads of a row (threadIdx.x), broadcast to all of them. red: 33 floats per
// row of the block. Every thread of the block calls it.
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x == 32) return v;
  const int nw = blockDim.x >> 5;
  red += threadIdx.y * 32;
  __syncthreads();   // the values of the previous call have been read
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int V>
__device__ __forceinline__ void load_w(const void* w, int w_bf16, int64_t i, float (&v)[V]) {
  if (w_bf16) load_v<V, true>(w, i, v);
  else load_v<V, false>(w, i, v);
}

template <int V, int VPT, bool X_BF16, bool R_BF16>
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormArgs a) {
  __shared__ float red[32 * 32];
  const int tid = threadIdx.x, tpr = blockDim.x;
  const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const bool on = row < a.rows;
  const int64_t nv = a.dim / V;   // dim is a multiple of V
  float h[VPT][V];
  if (on && a.r) {
    float r[VPT][V];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t i = (int64_t)j * tpr + tid;
      if (i < nv) {
        load_v<V, X_BF16>(a.x, row * a.xs + i * V, h[j]);
        load_v<V, R_BF16>(a.r, row * a.rs + i * V, r[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t i = (int64_t)j * tpr + tid;
      if (i < nv) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          h[j][e] += r[j][e];
          if constexpr (R_BF16) h[j][e] = __bfloat162float(__float2bfloat16_rn(h[j][e]));
        }
        store_v<V, R_BF16>(a.h, row * a.hs + i * V, h[j]);
      }
    }
  } else if (on) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t i = (int64_t)j * tpr + tid;
      if (i < nv) load_v<V, X_BF16>(a.x, row * a.xs + i * V, h[j]);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (!on || (int64_t)j * tpr + tid >= nv) {
#pragma unroll
      for (int e = 0; e < V; ++e) h[j][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sum += h[j][e] * h[j][e];
  }
  sum = row_sum(sum, red);
  const float rstd = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
  if (on && tid == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int64_t i = (int64_t)j * tpr + tid;
    const bool ok = on && i < nv;
    float y[V];
#pragma unroll
    for (int e = 0; e < V; ++e) y[e] = 0.0f;
    if (ok) {
      float w[V];
      load_w<V>(a.w, a.w_bf16, i * V, w);
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] = h[j][e] * rstd * w[e];
      if (a.y) store_v<V, X_BF16>(a.y, row * a.ys + i * V, y);
    }
    if (a.q) {   // every lane of the warp takes part: lanes past the row hold zeros
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < V; ++e) m = max(m, __float_as_uint(y[e]) & 0x7fffffffu);
#pragma unroll
      for (int o = kMxBlock / V / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (ok) {
        const uint32_t code = mx_scale_code(m);
        uint8_t* q = a.q + row * a.qs + i * V;
        if constexpr (V == 8) *reinterpret_cast<uint2*>(q) = mx_pack8(y, code);
        else *q = (uint8_t)mx_pack1(y[0], code);
        if (i % (kMxBlock / V) == 0) a.sc[row * a.scs + i / (kMxBlock / V)] = (uint8_t)code;
      }
    }
  }
}

// One row at a time per row group; each thread keeps the weight gradient of its own columns in
// registers over all rows that its block takes (in a fixed order), and the blocks' sums are added
// by norm_dw_kernel.
template <int V, int VPT, bool DY_BF16, bool H_BF16>
__global__ void __launch_bounds__(1024) rms_norm_grad_kernel(NormGradArgs a) {
  extern __shared__ float dws[];   // [dim], only with several row groups
  __shared__ float red[32 * 32];
  grid_launch_dependents();
  const int tid = threadIdx.x, tpr = blockDim.x;
  const int64_t nv = a.dim / V;
  const float inv_dim = 1.0f / (float)a.dim;
  float dw[VPT][V];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.0f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  for (int64_t row0 = (int64_t)blockIdx.x * blockDim.y; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + threadIdx.y;
    const bool on = row < a.rows;
    float g[VPT][V], n[VPT][V];
    float rstd = 0.0f;
    if (on) {
      rstd = a.rstd[row];
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int64_t i = (int64_t)j * tpr + tid;
        if (i < nv) {
          load_v<V, DY_BF16>(a.dy, row * a.dys + i * V, g[j]);
          load_v<V, H_BF16>(a.h, row * a.hs + i * V, n[j]);
        }
      }
    }
    float c = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t i = (int64_t)j * tpr + tid;
      if (on && i < nv) {
        float w[V];
        load_w<V>(a.w, a.w_bf16, i * V, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          n[j][e] *= rstd;
          dw[j][e] += g[j][e] * n[j][e];
          g[j][e] *= w[e];
          c += g[j][e] * n[j][e];
        }
      }
    }
    c = row_sum(c, red) * inv_dim;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t i = (int64_t)j * tpr + tid;
      if (on && i < nv) {
        float d[V];
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = rstd * (g[j][e] - n[j][e] * c);
        if (a.dh) {
          float r[V];
          load_v<V, H_BF16>(a.dh, row * a.dhs + i * V, r);
#pragma unroll
          for (int e = 0; e < V; ++e) d[e] += r[e];
        }
        store_v<V, H_BF16>(a.dx, row * a.dxs + i * V, d);
      }
    }
  }
  // the block's sum over its row groups, in their order
  if (blockDim.y > 1) {
    for (int gr = 0; gr < (int)blockDim.y; ++gr) {
      __syncthreads();
      if ((int)threadIdx.y == gr) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
          const int64_t i = (int64_t)j * tpr + tid;
          if (i < nv) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const int64_t at = i * V + e;
              if (gr == 0) dws[at] = dw[j][e];
              else if (gr + 1 < (int)blockDim.y) dws[at] += dw[j][e];
              else a.partial[(int64_t)blockIdx.x * a.dim + at] = dws[at] + dw[j][e];
            }
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int64_t i = (int64_t)j * tpr + tid;
      if (i < nv) store_v<V, false>(a.partial, (int64_t)blockIdx.x * a.dim + i * V, dw[j]);
    }
  }
}

// dw (+)= the sum of the blocks' partial sums: 32 columns per block, eight warps that take every
// eighth partial in order, then the eight sums in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* __restrict__ partial, float* dw, int blocks,
                                                      int64_t dim, int accumulate) {
  __shared__ float part[8][33];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < dim) {
#pragma unroll 8
    for (int b = w; b < blocks; b += 8) s += partial[(int64_t)b * dim + col];
  }
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < dim) {
    s = accumulate ? dw[col] : 0.0f;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += part[k][lane];
    dw[col] = s + t;
  }
}

// Threads per row and accesses per thread for a row of nv accesses.
struct RowShape {
  int tpr, vpt, groups;
};

RowShape row_shape(int64_t nv, int want_vpt, int block) {
  RowShape s;
  s.tpr = 32;
  while (s.tpr < 1024 && (int64_t)s.tpr * want_vpt < nv) s.tpr *= 2;
  s.vpt = (int)((nv + s.tpr - 1) / s.tpr);
  s.groups = s.tpr < block ? block / s.tpr : 1;
  return s;
}

bool aligned8(const void* p, int64_t stride, int bf16) {
  return (uintptr_t)p % 16 == 0 && stride % 8 == 0 && (bf16 || stride % 4 == 0);
}

template <int V, int VPT>
cudaError_t norm_types(const NormArgs& a, int xb, int rb, RowShape s, cudaStream_t st) {
  const dim3 block(s.tpr, s.groups);
  const dim3 grid((unsigned)((a.rows + s.groups - 1) / s.groups));
  if (xb && rb) rms_norm_kernel<V, VPT, true, true><<<grid, block, 0, st>>>(a);
  else if (xb) rms_norm_kernel<V, VPT, true, false><<<grid, block, 0, st>>>(a);
  else if (rb) rms_norm_kernel<V, VPT, false, true><<<grid, block, 0, st>>>(a);
  else rms_norm_kernel<V, VPT, false, false><<<grid, block, 0, st>>>(a);
  return cudaGetLastError();
}

template <int V, int VPT, bool D, bool H>
cudaError_t norm_grad_one(const NormGradArgs& a, RowShape s, int blocks, cudaStream_t st) {
  const size_t smem = s.groups > 1 ? (size_t)a.dim * sizeof(float) : 0;   // at most 32 x VPT x V floats
  rms_norm_grad_kernel<V, VPT, D, H><<<blocks, dim3(s.tpr, s.groups), smem, st>>>(a);
  return cudaGetLastError();
}

template <int V, int VPT>
cudaError_t norm_grad_types(const NormGradArgs& a, int db, int hb, RowShape s, int blocks, cudaStream_t st) {
  if (db && hb) return norm_grad_one<V, VPT, true, true>(a, s, blocks, st);
  if (db) return norm_grad_one<V, VPT, true, false>(a, s, blocks, st);
  if (hb) return norm_grad_one<V, VPT, false, true>(a, s, blocks, st);
  return norm_grad_one<V, VPT, false, false>(a, s, blocks, st);
}

int norm_grad_blocks(int64_t rows) {
  const int64_t cap = (int64_t)kSms * 4;
  return (int)(rows < cap ? rows : cap);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int x_bf16, int r_bf16, int sms, cudaStream_t st) {
  const bool w_ok = (uintptr_t)a.w % 16 == 0;
  const bool v8 = a.dim % 8 == 0 && w_ok && aligned8(a.x, a.xs, x_bf16) &&
                  (!a.r || (aligned8(a.r, a.rs, r_bf16) && aligned8(a.h, a.hs, r_bf16))) &&
                  (!a.y || aligned8(a.y, a.ys, x_bf16)) &&
                  (!a.q || ((uintptr_t)a.q % 8 == 0 && a.qs % 8 == 0));
  if (v8) {
    const RowShape s = row_shape(a.dim / 8, a.rows < 2 * sms ? 1 : 2, 128);
    if (s.vpt <= 1) return norm_types<8, 1>(a, x_bf16, r_bf16, s, st);
    if (s.vpt <= 2) return norm_types<8, 2>(a, x_bf16, r_bf16, s, st);
    return norm_types<8, 4>(a, x_bf16, r_bf16, s, st);
  }
  const RowShape s = row_shape(a.dim, 8, 128);
  if (s.vpt <= 8) return norm_types<1, 8>(a, x_bf16, r_bf16, s, st);
  return norm_types<1, 32>(a, x_bf16, r_bf16, s, st);
}

int64_t norm_grad_workspace(int64_t rows, int64_t dim) {
  return (int64_t)norm_grad_blocks(rows) * dim * (int64_t)sizeof(float);
}

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, int dy_bf16, int h_bf16, int sms, int64_t* launches,
                                 cudaStream_t st) {
  if (a.rows == 0) {   // the empty sum
    norm_dw_kernel<<<(unsigned)((a.dim + 31) / 32), 256, 0, st>>>(a.partial, a.dw, 0, a.dim, a.accumulate);
    ++*launches;
    return cudaGetLastError();
  }
  const bool v8 = a.dim % 8 == 0 && (uintptr_t)a.w % 16 == 0 && aligned8(a.dy, a.dys, dy_bf16) &&
                  aligned8(a.h, a.hs, h_bf16) && aligned8(a.dx, a.dxs, h_bf16) &&
                  (!a.dh || aligned8(a.dh, a.dhs, h_bf16));
  const RowShape s = v8 ? row_shape(a.dim / 8, 2, 128) : row_shape(a.dim, 8, 128);
  int blocks = norm_grad_blocks((a.rows + s.groups - 1) / s.groups);
  cudaError_t e;
  if (v8) {
    e = s.vpt <= 1   ? norm_grad_types<8, 1>(a, dy_bf16, h_bf16, s, blocks, st)
        : s.vpt <= 2 ? norm_grad_types<8, 2>(a, dy_bf16, h_bf16, s, blocks, st)
                     : norm_grad_types<8, 4>(a, dy_bf16, h_bf16, s, blocks, st);
  } else {
    e = s.vpt <= 8 ? norm_grad_types<1, 8>(a, dy_bf16, h_bf16, s, blocks, st)
                   : norm_grad_types<1, 32>(a, dy_bf16, h_bf16, s, blocks, st);
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_dependent(norm_dw_kernel, dim3((unsigned)((a.dim + 31) / 32)), dim3(256), 0, st,
                       (const float*)a.partial, a.dw, blocks, a.dim, a.accumulate);
  ++*launches;
  return e;
}

}  // namespace muon
