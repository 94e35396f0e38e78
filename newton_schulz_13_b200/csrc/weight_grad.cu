// Weight gradient from an 8-bit activation checkpoint: grad[n][k] (+)= sum over t of dy[t][n] x[t][k],
// with x the checkpoint's values (mx.cuh), which are exact in bf16. Compute-bound: 2 rows n k FLOPs
// on the tcgen05 tensor cores.
//
// Three launches:
//   stage    x (and dy, when its rows are not 16-byte aligned or it is fp32) written to the
//            workspace as bf16. An fp32 dy becomes three bf16 planes whose sum is dy exactly
//            (8 + 8 + 8 mantissa bits, by truncation), contracted one after the other, so nothing
//            of it is lost.
//   product  CTA pairs (cta_group::2) on 256 x 256 tiles; both operands are MN-major (the
//            contraction runs over rows t). Warp 0 loads 64-row slices with TMA, warp 1 of the even
//            CTA issues the MMAs, eight warps drain the accumulator. The accumulator is drained
//            every kChunk slices (1024 rows) into registers and added there in fp32: the tensor
//            core truncates its running sum at every step, a bias that grows with the number of
//            steps.
//   reduce   where the rows are split over several units of a tile (few tiles, many rows): the
//            parts, in fp32 in the workspace, are added in order.
// Waits are bounded as in the Newton-Schulz products (pair_pipe.cuh describes the unwinding).
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "device_once.h"
#include "muon_internal.h"
#include "mx.cuh"
#include "ops_internal.h"
#include "pair_pipe.cuh"
#include "ptx.cuh"
#include "vec_io.cuh"

namespace muon {
namespace {

constexpr int kTile = 256;                      // grad rows and columns per CTA pair
constexpr int kSlice = 64;                      // contraction rows per pipeline stage
constexpr int kChunk = 16;                      // slices between drains of the accumulator
constexpr int kStages = 6;
constexpr uint32_t kBox = 64 * 64 * 2;          // 64 contraction rows x 64 columns, bf16
constexpr uint32_t kOperand = 2 * kBox;         // a CTA's 128 columns of one operand
constexpr uint32_t kStage = 2 * kOperand;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kTransposeFloats = 32 * 33;  // per epilogue warp
constexpr size_t kSmem = 1024 + kStages * kStage + kEpiWarps * kTransposeFloats * 4 + 256;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kGroup = 8;                  // tile rows that sweep the columns together (L2 reuse)

struct ProductArgs {
  void* grad;               // the output, or (splits > 1) the fp32 parts [splits][n][k]
  int64_t gs;               // its row stride
  uint32_t n, k, tiles_n, tiles_k, splits;
  uint32_t slices;          // slices of one plane of dy
  uint32_t planes;
  uint32_t plane_rows;      // rows between planes of dy
  int accumulate;
  int* status;
  uint64_t wait_ns;
};

// Unit u of a launch: a tile and its range [s0, s1) of the planes * slices contraction slices.
struct Unit {
  uint32_t ti, tj, s0, s1, split;
};

__host__ __device__ inline Unit unit_of(const ProductArgs& a, uint32_t u) {
  const uint32_t tiles = a.tiles_n * a.tiles_k, all = a.slices * a.planes;
  Unit r;
  r.split = u / tiles;
  const uint32_t t = u - r.split * tiles;
  const uint32_t per = kGroup * a.tiles_k, g = t / per, first = g * kGroup;
  const uint32_t size = a.tiles_n - first < kGroup ? a.tiles_n - first : kGroup;
  r.ti = first + (t - g * per) % size;
  r.tj = (t - g * per) / size;
  r.s0 = (uint32_t)((uint64_t)all * r.split / a.splits);
  r.s1 = (uint32_t)((uint64_t)all * (r.split + 1) / a.splits);
  return r;
}

template <bool OUT_BF16>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_product_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
                         const ProductArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  float* transpose = reinterpret_cast<float*>(smem + kStages * kStage);
  uint64_t* full = reinterpret_cast<uint64_t*>(transpose + kEpiWarps * kTransposeFloats);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* zero_flag = abort_flag + 1;   // never set: the drain waits poll it
  volatile uint32_t* fill_count = reinterpret_cast<volatile uint32_t*>(zero_flag + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const uint32_t units = a.tiles_n * a.tiles_k * a.splits;
  const uint64_t wait_ns = a.wait_ns ? a.wait_ns : kTimeoutNs;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *zero_flag = 0;
    *fill_count = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  grid_dependency_wait();   // the staged operands
  grid_launch_dependents();

  bool timed_out = false;
  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, fills = 0;
      for (uint32_t u = pair; u < units && !timed_out; u += pairs) {
        const Unit w = unit_of(a, u);
        const int32_t n0 = (int32_t)(w.ti * kTile + rank * 128), k0 = (int32_t)(w.tj * kTile + rank * 128);
        for (uint32_t s = w.s0; s < w.s1; ++s) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, wait_ns)) {
            timed_out = true;
            break;
          }
          const uint32_t plane = s / a.slices, t0 = (s - plane * a.slices) * kSlice;
          const int32_t yd = (int32_t)(plane * a.plane_rows + t0), yx = (int32_t)t0;
          uint8_t* dst = smem + stage * kStage;
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStage);
          tma_load_2d_pair(dst, &map_dy, bar, n0, yd);
          tma_load_2d_pair(dst + kBox, &map_dy, bar, n0 + 64, yd);
          tma_load_2d_pair(dst + kOperand, &map_x, bar, k0, yx);
          tma_load_2d_pair(dst + kOperand + kBox, &map_x, bar, k0 + 64, yx);
          ++fills;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (timed_out) raise_abort(abort_flag, true, rank);
      *fill_count = fills;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      const uint32_t idesc = idesc_bf16_f32(kTile, kTile, 1, 1);
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      for (uint32_t u = pair; u < units && !timed_out; u += pairs) {
        const Unit w = unit_of(a, u);
        for (uint32_t c0 = w.s0; c0 < w.s1 && !timed_out; c0 += kChunk) {
          if (!mbar_wait_bounded(&tempty[acc], acc_phase ^ 1u, abort_flag, wait_ns)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          const uint32_t c1 = c0 + kChunk < w.s1 ? c0 + kChunk : w.s1;
          for (uint32_t s = c0; s < c1; ++s) {
            if (!mbar_wait_bounded(&full[stage], phase, abort_flag, wait_ns)) {
              timed_out = true;
              break;
            }
            tc_fence_after();
            const uint32_t ad = smem_u32(smem + stage * kStage), bd = ad + kOperand;
#pragma unroll
            for (uint32_t i = 0; i < kSlice / 16; ++i)
              tc_mma_f16_pair(tmem_base + acc * 256u, smem_desc_sw128(ad + i * 2048u, kBox, 1024),
                              smem_desc_sw128(bd + i * 2048u, kBox, 1024), idesc, s != c0 || i != 0 ? 1u : 0u);
            tc_commit_pair_mc(&empty[stage], 0x3);
            if (++stage == kStages) { stage = 0; phase ^= 1u; }
          }
          if (timed_out) break;
          tc_commit_pair_mc(&tfull[acc], 0x3);
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (timed_out) raise_abort(abort_flag, true, rank);
      tc_commit_pair(drain);   // all issued MMAs finish before the tensor memory is freed
      mbar_wait_bounded(drain, 0, zero_flag, kTimeoutNs);
    }
    __syncwarp();
  } else {
    // each warp: 32 accumulator rows (a lane each) x 128 of the tile's columns
    const uint32_t quarter = (uint32_t)(warp & 3), half = (uint32_t)(warp - 2) >> 2;
    float* stg = transpose + (uint32_t)(warp - 2) * kTransposeFloats;
    uint32_t acc = 0, acc_phase = 0;
    for (uint32_t u = pair; u < units; u += pairs) {
      const Unit w = unit_of(a, u);
      float sum[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) sum[i] = 0.0f;
      for (uint32_t c0 = w.s0; c0 < w.s1; c0 += kChunk) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&tfull[acc], acc_phase, abort_flag, wait_ns))) {
          timed_out = true;
          break;
        }
        tc_fence_after();
        const uint32_t at = tmem_base + ((quarter * 32u) << 16) + acc * 256u + half * 128u;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld_32x32b_x32_sync(at + g * 32, r);
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[g * 32 + i] += __uint_as_float(r[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&tempty[acc]), 0));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (timed_out) break;
      const int64_t r0 = (int64_t)w.ti * kTile + rank * 128 + quarter * 32;
      const int64_t base = a.splits > 1 ? (int64_t)w.split * a.n * a.k : 0;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int64_t col = (int64_t)w.tj * kTile + half * 128 + g * 32 + lane;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; ++i) stg[lane * 33 + i] = sum[g * 32 + i];
        __syncwarp();
        if (col < (int64_t)a.k) {
          const int rows = (int)min((int64_t)32, max((int64_t)0, (int64_t)a.n - r0));
#pragma unroll 8
          for (int r = 0; r < rows; ++r) {
            const int64_t at = base + (r0 + r) * a.gs + col;
            float v = stg[r * 33 + lane];
            if (a.splits > 1) {
              static_cast<float*>(a.grad)[at] = v;
            } else {
              if (a.accumulate) v += load1<OUT_BF16>(a.grad, at);
              store1<OUT_BF16>(a.grad, at, v);
            }
          }
        }
      }
    }
    if (timed_out && lane == 0) raise_abort(abort_flag, true, rank);
    __syncwarp();
  }

  if (timed_out) atomicOr(a.status, kStatusTimeout);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' roles have left their loops; the fill counts are visible
  if (warp == 0 && lane == 0 && leader) {
    const uint32_t peer = ld_shared_cluster(mapa_shared(smem_u32((const void*)fill_count), 1u));
    settle_pair_fills<kStages>(full, *fill_count, peer, kStage, zero_flag, kTimeoutNs);
  }
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, kTmemCols);
}

// grad (+)= the sum of the parts in order (zero parts: grad becomes 0).
template <bool OUT_BF16>
__global__ void __launch_bounds__(256) wgrad_reduce_kernel(const float* __restrict__ parts, void* grad, int64_t gs,
                                                           int64_t n, int64_t k, int splits, int accumulate) {
  grid_dependency_wait();
  const int64_t total = n * k;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < total; t += (int64_t)gridDim.x * 256) {
    const int64_t r = t / k, at = r * gs + (t - r * k);
    float v = 0.0f;
    for (int s = 0; s < splits; ++s) v += parts[s * total + t];
    if (accumulate) v += load1<OUT_BF16>(grad, at);
    store1<OUT_BF16>(grad, at, v);
  }
}

// Copies dy into bf16 rows of `pitch` elements; an fp32 dy into three planes, plane_rows apart.
template <bool DY_BF16>
__global__ void __launch_bounds__(256) wgrad_stage_dy_kernel(const void* dy, int64_t dys, int64_t rows, int64_t n,
                                                             __nv_bfloat16* out, int64_t pitch) {
  const int64_t total = rows * n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / n, c = i - t * n;
    if constexpr (DY_BF16) {
      out[t * pitch + c] = static_cast<const __nv_bfloat16*>(dy)[t * dys + c];
    } else {
      float v = static_cast<const float*>(dy)[t * dys + c];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        // the top 16 bits of a float are its value truncated to bf16; infinities and NaN stay whole
        uint32_t top = __float_as_uint(v) & 0xffff0000u;
        const bool finite = (top & 0x7f800000u) != 0x7f800000u;
        if (!finite && (__float_as_uint(v) & 0x7fffffu)) top |= 0x00400000u;
        out[(p * rows + t) * pitch + c] = __float2bfloat16_rn(__uint_as_float(top));
        v = finite ? v - __uint_as_float(top) : 0.0f;
      }
    }
  }
}

typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                           const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                           CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// MN-major operand view: boxes of 64 columns x 64 rows, 128-byte swizzle; outside reads zeros.
cudaError_t operand_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int64_t pitch) {
  static Encode encode = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)pitch * 2};
  const cuuint32_t box[2] = {64, 64}, one[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

struct Layout {
  int64_t x, dy, parts, bytes;    // workspace offsets
  int64_t x_pitch, dy_pitch;
  int planes, splits;
  bool copy_dy;
};

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

Layout layout_of(int64_t rows, int64_t n, int64_t k, int dy_bf16, int dy_aligned) {
  Layout l;
  l.planes = dy_bf16 ? 1 : 3;
  l.copy_dy = !dy_bf16 || !dy_aligned;
  l.x_pitch = up(k, 8);
  l.dy_pitch = up(n, 8);
  // splits of the contraction: rounds of units over the pairs x slices per unit, plus the parts'
  // way through memory, all in units of one slice's time (about 0.3 us; 1.2 MB of traffic)
  const int64_t tiles = (n + kTile - 1) / kTile * ((k + kTile - 1) / kTile), pairs = kSms / 2;
  const int64_t slices = (rows + kSlice - 1) / kSlice * l.planes;
  double best = 0;
  l.splits = 1;
  for (int64_t s = 1; s <= 64 && s <= slices; ++s) {
    const double rounds = (double)((tiles * s + pairs - 1) / pairs);
    double cost = rounds * ((double)((slices + s - 1) / s) + 4.0);
    if (s > 1) cost += 8.0 + 8.0 * (double)s * n * k / 1.2e6;
    if (s == 1 || cost < best) {
      best = cost;
      l.splits = (int)s;
    }
  }
  l.x = 0;
  l.dy = up(rows * l.x_pitch * 2, 256);
  l.parts = l.dy + (l.copy_dy ? up(rows * l.planes * l.dy_pitch * 2, 256) : 0);
  l.bytes = l.parts + (l.splits > 1 ? up((int64_t)l.splits * n * k * 4, 256) : 0);
  return l;
}

template <bool OUT_BF16>
cudaError_t launch_reduce(const float* parts, const WgradArgs& a, int splits, int sms, cudaStream_t s) {
  const int64_t blocks = (a.n * a.k + 255) / 256, cap = (int64_t)sms * 16;
  return launch_dependent(wgrad_reduce_kernel<OUT_BF16>, dim3((unsigned)(blocks < cap ? blocks : cap)), dim3(256), 0, s,
                          parts, a.grad, a.gs, a.n, a.k, splits, a.accumulate);
}

template <bool OUT_BF16>
cudaError_t launch_product(const CUtensorMap& md, const CUtensorMap& mx, const ProductArgs& p, int sms, cudaStream_t s) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = (cudaError_t)once.run(dev, [&] {
    return (int)cudaFuncSetAttribute(wgrad_product_kernel<OUT_BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kSmem);
  });
  if (e != cudaSuccess) return e;
  const uint32_t units = p.tiles_n * p.tiles_k * p.splits;
  const uint32_t pairs = units < (uint32_t)(sms / 2) ? units : (uint32_t)(sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, wgrad_product_kernel<OUT_BF16>, md, mx, p);
}

}  // namespace

int64_t wgrad_workspace(int64_t rows, int64_t n, int64_t k, int dy_bf16) {
  return layout_of(rows, n, k, dy_bf16, 0).bytes;   // with room for a copy of a dy that is not aligned
}

cudaError_t launch_wgrad(const WgradArgs& a, int dy_bf16, int grad_bf16, int sms, char* ws, int64_t* launches,
                         cudaStream_t s) {
  const int aligned = (uintptr_t)a.dy % 16 == 0 && a.dys % 8 == 0;
  const Layout l = layout_of(a.rows, a.n, a.k, dy_bf16, aligned);
  const float* parts = reinterpret_cast<const float*>(ws + l.parts);
  if (a.rows == 0) {
    ++*launches;
    return grad_bf16 ? launch_reduce<true>(parts, a, 0, sms, s) : launch_reduce<false>(parts, a, 0, sms, s);
  }
  MxArgs m = {};
  m.out = ws + l.x;
  m.q = const_cast<uint8_t*>(a.q);
  m.sc = const_cast<uint8_t*>(a.sc);
  m.rows = a.rows;
  m.dim = a.k;
  m.xs = l.x_pitch;
  m.qs = a.qs;
  m.scs = a.scs;
  cudaError_t e = launch_mx_restore(m, 1, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (l.copy_dy) {
    const int64_t blocks = (a.rows * a.n + 255) / 256, cap = (int64_t)sms * 16;
    const unsigned g = (unsigned)(blocks < cap ? blocks : cap);
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(ws + l.dy);
    if (dy_bf16) wgrad_stage_dy_kernel<true><<<g, 256, 0, s>>>(a.dy, a.dys, a.rows, a.n, out, l.dy_pitch);
    else wgrad_stage_dy_kernel<false><<<g, 256, 0, s>>>(a.dy, a.dys, a.rows, a.n, out, l.dy_pitch);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  CUtensorMap md, mx;
  e = l.copy_dy ? operand_map(&md, ws + l.dy, a.rows * l.planes, a.n, l.dy_pitch)
                : operand_map(&md, a.dy, a.rows, a.n, a.dys);
  if (e == cudaSuccess) e = operand_map(&mx, ws + l.x, a.rows, a.k, l.x_pitch);
  if (e != cudaSuccess) return e;
  ProductArgs p = {};
  p.grad = l.splits > 1 ? (void*)parts : a.grad;
  p.gs = l.splits > 1 ? a.k : a.gs;
  p.n = (uint32_t)a.n;
  p.k = (uint32_t)a.k;
  p.tiles_n = (uint32_t)((a.n + kTile - 1) / kTile);
  p.tiles_k = (uint32_t)((a.k + kTile - 1) / kTile);
  p.splits = (uint32_t)l.splits;
  p.slices = (uint32_t)((a.rows + kSlice - 1) / kSlice);
  p.planes = (uint32_t)l.planes;
  p.plane_rows = (uint32_t)a.rows;
  p.accumulate = a.accumulate;
  p.status = a.status;
  p.wait_ns = a.wait_ns;
  e = grad_bf16 ? launch_product<true>(md, mx, p, sms, s) : launch_product<false>(md, mx, p, sms, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (l.splits > 1) {
    e = grad_bf16 ? launch_reduce<true>(parts, a, l.splits, sms, s) : launch_reduce<false>(parts, a, l.splits, sms, s);
    ++*launches;
  }
  return e;
}

}  // namespace muon
