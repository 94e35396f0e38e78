// Root-mean-square norm with the residual's addition and an output in 8 bits with scales, and its
// gradient:
//   h = round(x + r)   (in r's type; h = x without a residual)
//   rstd = 1 / sqrt(mean(h^2) + eps),   y = h rstd w,   checkpoint of y (mx.cuh)
//   with n = h rstd and a = dy w:   dx = rstd (a - n mean(a n)) + dh,   dw (+)= sum over rows dy n
// All sums and statistics are fp32. The norm is taken of the rounded h, which is what the gradient
// reads back, and the checkpoint of the unrounded y, so each of its values is rounded once.
//
// Both are bound by HBM: every element is read and written once (16384 x 4096 bf16 with residual, y
// and checkpoint: 95 us on fixed buffers, 6.3 TB/s; the gradient with dh: 85 us, 6.3 TB/s; plain loads
// and stores of the same bytes take 94 and 78 us). Not so unaligned rows (8000 x 4093: 143 and 84 us,
// floors 45 and 40), whose outputs leave one element at a time, rows over 8192 columns (4096 x 14336: 164
// and 322, floors 81 and 72), which come without copies ahead and in the gradient twice, and narrow rows,
// of which a warp holds one (131072 x 128: 47 and 57, floors 23 and 21; half of its lanes idle). A row belongs to `tpr` threads (a multiple of 32) that hold it
// in registers, VPT accesses of V elements each: V = 8 (16-byte accesses) when every row is aligned
// to eight elements, V = 1 otherwise, where a warp reads 32 consecutive elements per access. In both,
// a 32-element checkpoint block lies within a warp: four lanes of one access (V = 8) or all 32 (V = 1).
#include <cuda_bf16.h>
#include <stdint.h>

#include "device_once.h"
#include "muon_internal.h"
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
      if constexpr (V == 1) {
        m = __reduce_max_sync(0xffffffffu, m);
      } else {
#pragma unroll
        for (int o = kMxBlock / V / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      }
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

// The same for many rows: a row group takes every (gridDim.x * groups)-th row, whose x and residual
// come by one bulk copy each into a ring of stages, S rows ahead (a row lies in registers once its sum
// is taken, and frees its stage). Three rows ahead of two groups of 4096 columns, 96 KB per SM, suffice:
// with 192 KB (three blocks of four) 16384 x 4096 takes 118 us instead of 95.
constexpr int kMaxGroups = 32, kRingStages = 3, kGradStages = 4;
constexpr uint64_t kTimeoutNs = 2000000000ull;

// A row of n bytes at p by bulk copy: the 16-byte granules that hold it, of which it begins at byte
// p % 16 (0 where V = 8); `room` is the most that they take. Each granule holds a byte of the row, so
// it lies in the row's allocation; what it holds of others is not used.
template <int V>
__host__ __device__ constexpr int row_room(int n) {
  return V == 8 ? n : (n + 30) / 16 * 16;
}
template <int V>
__device__ __forceinline__ uint32_t row_off(const void* base, int64_t bytes) {
  return V == 8 ? 0u : (uint32_t)((uintptr_t)base + bytes) & 15u;
}
template <int V>
__device__ __forceinline__ uint32_t row_span(const void* base, int64_t bytes, int n) {
  return V == 8 ? (uint32_t)n : (row_off<V>(base, bytes) + n + 15u) & ~15u;
}
template <int V>
__device__ __forceinline__ void row_load(void* to, const void* base, int64_t bytes, int n, uint64_t* bar) {
  bulk_load(to, static_cast<const char*>(base) + bytes - row_off<V>(base, bytes), row_span<V>(base, bytes, n), bar);
}

template <int V, bool X_BF16, bool R_BF16>
__global__ void __launch_bounds__(V == 8 ? 512 : 1024, 1) rms_norm_ring_kernel(NormArgs a) {
  extern __shared__ __align__(128) char stages[];
  constexpr int VPT = V == 8 ? 2 : 8, S = kRingStages, kX = X_BF16 ? 2 : 4, kR = R_BF16 ? 2 : 4;
  __shared__ float red[2][32];
  __shared__ uint64_t full[kMaxGroups][S];
  __shared__ int abort_word[2];   // a wait gave up; never set (for the last waits)
  const int tid = threadIdx.x, tpr = blockDim.x, warps = tpr >> 5, group = threadIdx.y;
  const int dim = (int)a.dim;
  const float inv_dim = 1.0f / (float)dim;
  const int64_t step = (int64_t)gridDim.x * blockDim.y, first = (int64_t)blockIdx.x * blockDim.y + group;
  const bool leader = tid == 0;
  if (leader) {
    for (int s = 0; s < S; ++s) mbar_init(&full[group][s], 1);
    if (group == 0) abort_word[0] = abort_word[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const int r_at = row_room<V>(dim * kX), part = r_at + (a.r ? row_room<V>(dim * kR) : 0), stage_bytes = part * blockDim.y;
  char* const part0 = stages + part * group;
  bool timed_out = false;
  int64_t fetched = 0;   // by this thread
  auto fetch = [&](int64_t row, int s) {
    if (!leader || timed_out || row >= a.rows) return;
    char* const to = part0 + s * stage_bytes;
    uint64_t* bar = &full[group][s];
    mbar_arrive_expect_tx(bar, row_span<V>(a.x, row * a.xs * kX, dim * kX) + (a.r ? row_span<V>(a.r, row * a.rs * kR, dim * kR) : 0u));
    ++fetched;
    row_load<V>(to, a.x, row * a.xs * kX, dim * kX, bar);
    if (a.r) row_load<V>(to + r_at, a.r, row * a.rs * kR, dim * kR, bar);
  };
  for (int s = 0; s < S; ++s) fetch(first + s * step, s);
  float w[VPT][V];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    if ((j * tpr + tid) * V < dim) load_w<V>(a.w, a.w_bf16, (int64_t)(j * tpr + tid) * V, w[j]);
  int s = 0, phase = 0, parity = 0;
#pragma unroll 1
  for (int64_t row = first; row - group < a.rows; row += step) {
    const bool on = row < a.rows;
    if (on && !mbar_wait_bounded(&full[group][s], phase, abort_word, a.wait_ns ? a.wait_ns : kTimeoutNs)) {
      timed_out = true;
      *(volatile int*)abort_word = 1;
    }
    const char* const from = part0 + s * stage_bytes;
    const char *const x = from + row_off<V>(a.x, row * a.xs * kX), *const r = from + r_at + row_off<V>(a.r, row * a.rs * kR);
    float h[VPT][V];
    float2 part_sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j * tpr * V >= dim) break;
      const int c = (j * tpr + tid) * V;
      if (on && c < dim) {
        load_v<V, X_BF16>(x, c, h[j]);
        if (a.r) {   // h = round(h + r)
          if constexpr (V == 8) {
            Raw<8, R_BF16> raw;
            raw.load(r, c);
            raw.add(h[j]);
            raw.store(a.h, row * a.hs + c);
            raw.get(h[j]);
          } else {
            h[j][0] += load1<R_BF16>(r, c);
            if constexpr (R_BF16) h[j][0] = __bfloat162float(__float2bfloat16_rn(h[j][0]));
            store1<R_BF16>(a.h, row * a.hs + c, h[j][0]);
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e) h[j][e] = 0.0f;
      }
      if constexpr (V == 8) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 p = make_float2(h[j][e], h[j][e + 1]);
          part_sum = __ffma2_rn(p, p, part_sum);
        }
      } else {
        part_sum.x += h[j][0] * h[j][0];
      }
    }
    float sum = part_sum.x + part_sum.y;
    // the row's sum; the other half of red was last read before the barrier of the row before
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (warps > 1) {
      if ((tid & 31) == 0) red[parity][group * warps + (tid >> 5)] = sum;
      __syncthreads();
      sum = (tid & 31) < warps ? red[parity][group * warps + (tid & 31)] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      parity ^= 1;
    }
    // past this barrier (of the warp, if it is the group) nobody reads the stage of this row
    fetch(row + S * step, s);
    const float rstd = 1.0f / sqrtf(sum * inv_dim + a.eps);
    if (on && leader) a.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j * tpr * V >= dim) break;
      const int c = (j * tpr + tid) * V;
      const bool ok = on && c < dim;
      float y[V];
      if constexpr (V == 8) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 p = __fmul2_rn(__fmul2_rn(make_float2(h[j][e], h[j][e + 1]), make_float2(rstd, rstd)),
                                      make_float2(w[j][e], w[j][e + 1]));
          y[e] = p.x;
          y[e + 1] = p.y;
        }
      } else {
        y[0] = h[j][0] * rstd * w[j][0];
      }
      if (ok && a.y) store_v<V, X_BF16>(a.y, row * a.ys + c, y);
      if (a.q) {   // every lane of the warp takes part: lanes past the row count as zeros
        uint32_t m;
        if constexpr (V == 8) {
          m = ok ? mx_amax8(y) : 0u;
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
          m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        } else {
          m = __reduce_max_sync(0xffffffffu, ok ? __float_as_uint(y[0]) & 0x7fffffffu : 0u);
        }
        if (ok) {
          const uint32_t code = mx_scale_code(m);
          uint8_t* const q = a.q + row * a.qs + c;
          if constexpr (V == 8) *reinterpret_cast<uint2*>(q) = mx_pack8(y, code);
          else *q = (uint8_t)mx_pack1(y[0], code);
          if ((c & (kMxBlock - 1)) == 0) a.sc[row * a.scs + c / kMxBlock] = (uint8_t)code;
        }
      }
    }
    if (++s == S) {
      s = 0;
      phase ^= 1;
    }
  }
  if (timed_out) atomicOr(a.status, kStatusTimeout);
  if (timed_out && leader) {
    // no copy may land after the block has gone: wait for each stage's last one
    for (int64_t f = fetched > S ? fetched - S : 0; f < fetched; ++f)
      mbar_wait_bounded(&full[group][f % S], (f / S) & 1, abort_word + 1, kTimeoutNs);
  }
}

// How a row reaches the threads of the gradient:
//   kBulk    one bulk copy per row and tensor into a ring of stages, S - 1 rows ahead
//   kDirect  no copies: a thread loads its accesses, twice (rows too long for the ring)
// 16384 x 4096 bf16 with dh, 537 MB: kBulk 82 us, asynchronous copies per thread 116-131 us, kDirect
// 125 us.
enum class Feed { kBulk, kDirect };

// A row group takes every (gridDim.x * groups)-th row; each thread keeps the weight gradient of its
// own columns in registers over all of them (in a fixed order), and the blocks' sums are added by
// norm_dw_kernel. A row costs one block barrier, its sum's.
template <int V, int VPT, bool DY_BF16, bool H_BF16, Feed FEED, int S>
__global__ void __launch_bounds__(FEED == Feed::kDirect ? 1024 : 512) rms_norm_grad_kernel(NormGradArgs a) {
  extern __shared__ __align__(128) char slots[];   // the stages; after the rows, [dim] floats with several row groups
  constexpr bool BULK = FEED == Feed::kBulk;
  constexpr int kDy = DY_BF16 ? 2 : 4, kH = H_BF16 ? 2 : 4;
  __shared__ float red[2][32];
  __shared__ uint64_t full[kMaxGroups][kGradStages];
  __shared__ int abort_word[2];   // a wait gave up; never set (for the last waits)
  grid_launch_dependents();
  const int tid = threadIdx.x, tpr = blockDim.x, warps = tpr >> 5, group = threadIdx.y;
  const int nv = (int)(a.dim / V), mine = tid < nv ? (nv - tid + tpr - 1) / tpr : 0;   // accesses of this thread
  const float inv_dim = 1.0f / (float)a.dim;
  const int64_t step = (int64_t)gridDim.x * blockDim.y, first = (int64_t)blockIdx.x * blockDim.y + group;
  const bool leader = tid == 0;
  bool timed_out = false;
  int64_t fetched = 0;   // by this thread (kBulk)
  if constexpr (BULK) {
    if (leader) {
      for (int s = 0; s < S; ++s) mbar_init(&full[group][s], 1);
      if (group == 0) abort_word[0] = abort_word[1] = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  // where a group's tensors lie in its part of a stage
  const int dim = (int)a.dim, h_at = row_room<V>(dim * kDy), dh_at = h_at + row_room<V>(dim * kH);
  const int part = dh_at + (a.dh ? row_room<V>(dim * kH) : 0), stage_bytes = part * blockDim.y;
  char* const part0 = slots + part * group;
  auto fetch = [&](int64_t row, int s) {
    if constexpr (BULK) {
      if (!leader || timed_out || row >= a.rows) return;
      char* const to = part0 + s * stage_bytes;
      uint64_t* bar = &full[group][s];
      const int64_t dy_b = row * a.dys * kDy, h_b = row * a.hs * kH, dh_b = row * a.dhs * kH;
      mbar_arrive_expect_tx(bar, row_span<V>(a.dy, dy_b, dim * kDy) + row_span<V>(a.h, h_b, dim * kH) +
                                     (a.dh ? row_span<V>(a.dh, dh_b, dim * kH) : 0u));
      ++fetched;
      row_load<V>(to, a.dy, dy_b, dim * kDy, bar);
      row_load<V>(to + h_at, a.h, h_b, dim * kH, bar);
      if (a.dh) row_load<V>(to + dh_at, a.dh, dh_b, dim * kH, bar);
    }
  };
  float dw[VPT][V], w[VPT][V];
#pragma unroll
  for (int s = 0; s < S - 1; ++s) fetch(first + s * step, s);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    if (FEED != Feed::kDirect && j < mine) load_w<V>(a.w, a.w_bf16, (int64_t)(j * tpr + tid) * V, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.0f;
  }
  float rstd_next = first < a.rows ? a.rstd[first] : 0.0f;
  int s = 0, phase = 0, parity = 0;
#pragma unroll 1
  for (int64_t row = first; row - group < a.rows; row += step) {
    const bool on = row < a.rows;
    const float rstd = rstd_next;
    rstd_next = row + step < a.rows ? a.rstd[row + step] : 0.0f;
    const char* const from = part0 + s * stage_bytes;
    const int previous = s == 0 ? S - 1 : s - 1;
    if constexpr (BULK) {
      if (on && !mbar_wait_bounded(&full[group][s], phase, abort_word, a.wait_ns ? a.wait_ns : kTimeoutNs)) {
        timed_out = true;
        *(volatile int*)abort_word = 1;
      }
    }
    const char *const dy_row = from + row_off<V>(a.dy, row * a.dys * kDy), *const h_row = from + h_at + row_off<V>(a.h, row * a.hs * kH),
               *const dh_row = from + dh_at + row_off<V>(a.dh, row * a.dhs * kH);
    constexpr int KEEP = FEED == Feed::kDirect ? 1 : VPT;
    float g[KEEP][V], n[KEEP][V];
    // dy and h of access j (and its weights, where they are not kept)
    auto read = [&](int j, float (&gj)[V], float (&nj)[V]) {
      if constexpr (FEED != Feed::kDirect) {
        load_v<V, DY_BF16>(dy_row, (j * tpr + tid) * V, gj);
        load_v<V, H_BF16>(h_row, (j * tpr + tid) * V, nj);
      } else {
        const int64_t c = (int64_t)(j * tpr + tid) * V;
        load_v<V, DY_BF16>(a.dy, row * a.dys + c, gj);
        load_v<V, H_BF16>(a.h, row * a.hs + c, nj);
        load_w<V>(a.w, a.w_bf16, c, w[0]);
      }
    };
    float c = 0.0f;
    if (on) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j >= mine) break;
        float (&gj)[V] = g[KEEP > 1 ? j : 0], (&nj)[V] = n[KEEP > 1 ? j : 0], (&wj)[V] = w[KEEP > 1 ? j : 0];
        read(j, gj, nj);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          nj[e] *= rstd;
          dw[j][e] += gj[e] * nj[e];
          gj[e] *= wj[e];
          c += gj[e] * nj[e];
        }
      }
    }
    // the row's sum; the other half of red was last read before the barrier of the row before
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if (warps > 1) {
      if ((tid & 31) == 0) red[parity][group * warps + (tid >> 5)] = c;
      __syncthreads();
      c = (tid & 31) < warps ? red[parity][group * warps + (tid & 31)] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
      parity ^= 1;
    }
    c *= inv_dim;
    // past this barrier (of the warp, if it is the group) nobody reads the stage of the row before
    if constexpr (BULK) fetch(row + (S - 1) * step, previous);
    if (on) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (j >= mine) break;
        float (&gj)[V] = g[KEEP > 1 ? j : 0], (&nj)[V] = n[KEEP > 1 ? j : 0];
        if constexpr (FEED == Feed::kDirect) {
          read(j, gj, nj);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            nj[e] *= rstd;
            gj[e] *= w[0][e];
          }
        }
        float d[V];
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = rstd * (gj[e] - nj[e] * c);
        const int64_t col = (int64_t)(j * tpr + tid) * V;
        if (a.dh) {
          float r[V];
          if constexpr (FEED != Feed::kDirect) load_v<V, H_BF16>(dh_row, (j * tpr + tid) * V, r);
          else load_v<V, H_BF16>(a.dh, row * a.dhs + col, r);
#pragma unroll
          for (int e = 0; e < V; ++e) d[e] += r[e];
        }
        store_v<V, H_BF16>(a.dx, row * a.dxs + col, d);
      }
    }
    if (++s == S) {
      s = 0;
      phase ^= 1;
    }
  }
  if constexpr (BULK) {
    if (timed_out) atomicOr(a.status, kStatusTimeout);
    if (timed_out && leader) {
      // no copy may land after the block has gone: wait for each stage's last one
      for (int64_t f = fetched > S ? fetched - S : 0; f < fetched; ++f)
        mbar_wait_bounded(&full[group][f % S], (f / S) & 1, abort_word + 1, kTimeoutNs);
    }
  }
  float* dws = reinterpret_cast<float*>(slots);
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

// dw (+)= the sum of the blocks' partial sums: 32 columns per block, 32 warps that take every 32nd
// partial in order, then the 32 sums in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ partial, float* dw, int blocks,
                                                       int64_t dim, int accumulate) {
  __shared__ float part[32][33];
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (col < dim) {
#pragma unroll 8
    for (int b = w; b < blocks; b += 32) s += partial[(int64_t)b * dim + col];
  }
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < dim) {
    s = accumulate ? dw[col] : 0.0f;
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) t += part[k][lane];
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

constexpr int kRingSmem = 220 * 1024;   // of an SM, for the stages of its blocks

// One block per SM, whose stages (at most 64 KB each) always fit: of 512 threads with 16 elements each,
// or of 1024 with 8 where they take single accesses.
template <int V, bool X, bool R>
cudaError_t norm_ring(const NormArgs& a, cudaStream_t st) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = (cudaError_t)once.run(dev, [&] {
    return (int)cudaFuncSetAttribute(rms_norm_ring_kernel<V, X, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
  });
  if (e != cudaSuccess) return e;
  const RowShape s = V == 8 ? row_shape(a.dim / 8, 2, 512) : row_shape(a.dim, 8, 1024);
  const int64_t groups = (a.rows + s.groups - 1) / s.groups;
  const int dim = (int)a.dim;
  const size_t smem = (size_t)kRingStages * s.groups * (row_room<V>(dim * (X ? 2 : 4)) + (a.r ? row_room<V>(dim * (R ? 2 : 4)) : 0));
  rms_norm_ring_kernel<V, X, R><<<(unsigned)(groups < kSms ? groups : kSms), dim3(s.tpr, s.groups), smem, st>>>(a);
  return cudaGetLastError();
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

template <int V, int VPT, bool D, bool H, Feed F, int S>
cudaError_t norm_grad_one(const NormGradArgs& a, RowShape s, int64_t stage, int per_sm, int* blocks, cudaStream_t st) {
  const int64_t sums = s.groups > 1 ? a.dim * (int64_t)sizeof(float) : 0, stages = S * stage;
  const size_t smem = (size_t)(stages > sums ? stages : sums);
  const int64_t groups = (a.rows + s.groups - 1) / s.groups, cap = (int64_t)kSms * per_sm;
  *blocks = (int)(groups < cap ? groups : cap);
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = (cudaError_t)once.run(dev, [&] {
    return (int)cudaFuncSetAttribute(rms_norm_grad_kernel<V, VPT, D, H, F, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kRingSmem);
  });
  if (e != cudaSuccess) return e;
  rms_norm_grad_kernel<V, VPT, D, H, F, S><<<*blocks, dim3(s.tpr, s.groups), smem, st>>>(a);
  return cudaGetLastError();
}

// Blocks of 256 threads (512 for the longest rows), two per SM where their four stages leave room
// (4096 columns of fp32 with dh, one block with four stages or two with two: 84 and 91 us for 8192
// rows; bf16, 16384 rows, two with four, one with four, two with two: 85, 121 and 116 us).
template <int V, int VPT, bool D, bool H>
cudaError_t norm_grad_stages(const NormGradArgs& a, int* blocks, cudaStream_t st) {
  const RowShape s = row_shape(a.dim / V, VPT, 256);
  const int dim = (int)a.dim, h = row_room<V>(dim * (H ? 2 : 4));
  const int64_t stage = (int64_t)s.groups * (row_room<V>(dim * (D ? 2 : 4)) + (a.dh ? 2 : 1) * h);
  const int64_t fit = kRingSmem / (kGradStages * stage), most = s.tpr <= 256 ? 2 : 1;
  if (fit >= 1)
    return norm_grad_one<V, VPT, D, H, Feed::kBulk, kGradStages>(a, s, stage, (int)(fit < most ? fit : most), blocks, st);
  return norm_grad_one<V, VPT, D, H, Feed::kBulk, 2>(a, s, stage, 1, blocks, st);
}

template <bool D, bool H>
cudaError_t norm_grad_shapes(const NormGradArgs& a, bool v8, int* blocks, cudaStream_t st) {
  if (v8 && a.dim <= 8192) return norm_grad_stages<8, 2, D, H>(a, blocks, st);
  if (v8) return norm_grad_one<8, 4, D, H, Feed::kDirect, 1>(a, row_shape(a.dim / 8, 4, 256), 0, 1, blocks, st);
  if (a.dim <= 4096) return norm_grad_stages<1, 8, D, H>(a, blocks, st);
  if (a.dim <= 8192) return norm_grad_stages<1, 16, D, H>(a, blocks, st);
  return norm_grad_one<1, 32, D, H, Feed::kDirect, 1>(a, row_shape(a.dim, 32, 256), 0, 1, blocks, st);
}

// Whether many rows go through the ring (us with residual, y and checkpoint unless said otherwise, ring
// and not, of 2^24 elements in all; below 2^22 starting it costs up to 1 us more: 64 x 4096 bf16 3.6
// and 2.9):
//   unaligned rows: yes (31 columns 186 and 339, 257 113 and 124, 4093 76 and 128)
//   bf16: from 2304 columns on (2304 45 and 45, 4096 31 and 37, 8192 31 and 41), and below where the
//     row leaves no more than a quarter of its threads' accesses idle (1024 33 and 35, 768 40 and 39,
//     but 1280 46 and 43, 256 38 and 30, 128 72 and 47)
//   an fp32 tensor in it: from 4104 columns on (5120, residual fp32: 43 and 54; x fp32, no residual: 43
//     and 45), below no (4096, residual fp32: 45 and 42; 1024, x fp32, no residual: 33 and 31)
//   two: no (8192 57 and 51, 1024 57 and 50)
bool ring_pays(const NormArgs& a, bool v8, int x_bf16, int r_bf16) {
  if (!v8) return true;
  if (x_bf16 && r_bf16) return a.dim > 2048 || a.dim / 8 * 4 >= 3 * 2 * row_shape(a.dim / 8, 2, 512).tpr;
  return a.dim > 4096 && (!a.r || x_bf16 || r_bf16);
}

int norm_grad_blocks(int64_t rows) {
  const int64_t cap = (int64_t)kSms * 2;   // two blocks per SM at most
  return (int)(rows < cap ? rows : cap);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, int x_bf16, int r_bf16, int sms, cudaStream_t st) {
  const bool w_ok = (uintptr_t)a.w % 16 == 0;
  const bool v8 = a.dim % 8 == 0 && w_ok && aligned8(a.x, a.xs, x_bf16) &&
                  (!a.r || (aligned8(a.r, a.rs, r_bf16) && aligned8(a.h, a.hs, r_bf16))) &&
                  (!a.y || aligned8(a.y, a.ys, x_bf16)) &&
                  (!a.q || ((uintptr_t)a.q % 8 == 0 && a.qs % 8 == 0));
  if (a.dim <= 8192 && a.rows * a.dim >= (int64_t(1) << 22) && ring_pays(a, v8, x_bf16, r_bf16)) {
    if (v8) {
      if (x_bf16) return r_bf16 ? norm_ring<8, true, true>(a, st) : norm_ring<8, true, false>(a, st);
      return r_bf16 ? norm_ring<8, false, true>(a, st) : norm_ring<8, false, false>(a, st);
    }
    if (x_bf16) return r_bf16 ? norm_ring<1, true, true>(a, st) : norm_ring<1, true, false>(a, st);
    return r_bf16 ? norm_ring<1, false, true>(a, st) : norm_ring<1, false, false>(a, st);
  }
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

cudaError_t launch_rms_norm_grad(const NormGradArgs& a, int dy_bf16, int h_bf16, int64_t* launches,
                                 cudaStream_t st) {
  if (a.rows == 0) {   // the empty sum
    norm_dw_kernel<<<(unsigned)((a.dim + 31) / 32), 1024, 0, st>>>(a.partial, a.dw, 0, a.dim, a.accumulate);
    ++*launches;
    return cudaGetLastError();
  }
  const bool v8 = a.dim % 8 == 0 && (uintptr_t)a.w % 16 == 0 && aligned8(a.dy, a.dys, dy_bf16) &&
                  aligned8(a.h, a.hs, h_bf16) && aligned8(a.dx, a.dxs, h_bf16) &&
                  (!a.dh || aligned8(a.dh, a.dhs, h_bf16));
  int blocks = 0;   // at most norm_grad_blocks(rows)
  cudaError_t e = dy_bf16 ? (h_bf16 ? norm_grad_shapes<true, true>(a, v8, &blocks, st) : norm_grad_shapes<true, false>(a, v8, &blocks, st))
                          : (h_bf16 ? norm_grad_shapes<false, true>(a, v8, &blocks, st) : norm_grad_shapes<false, false>(a, v8, &blocks, st));
  if (e != cudaSuccess) return e;
  ++*launches;
  e = launch_dependent(norm_dw_kernel, dim3((unsigned)((a.dim + 31) / 32)), dim3(1024), 0, st,
                       (const float*)a.partial, a.dw, blocks, a.dim, a.accumulate);
  ++*launches;
  return e;
}

}  // namespace muon
