// Weight gradient from an 8-bit activation checkpoint: grad[n][k] (+)= sum over t of dy[t][n] x[t][k],
// with x the checkpoint's values (mx.cuh), which are exact in bf16. Compute-bound: 2 rows n k FLOPs
// on the tcgen05 tensor cores. 14336 x 4096 over 8192 rows: 664 us with the staging in short runs (1450
// TFLOP/s, the tensor pipe busy 88 % of the time), 780 to 810 over seconds under the power limit; 768 x
// 2304, accumulating in fp32: 47 us, 92 from an fp32 dy.
//
// Two launches:
//   stage    x (and dy, when its rows are not 16-byte aligned or it is fp32) written to the
//            workspace as bf16. An fp32 dy becomes three bf16 planes whose sum is dy (8 + 8 + 8
//            mantissa bits, by truncation): exactly from 2^-110 on; below, the third plane
//            ends at bf16's smallest number, 2^-133, and what is under it is cut off.
//   product  CTA pairs (cta_group::2) on 256 x 256 tiles; both operands are MN-major (the
//            contraction runs over rows t). Warp 0 loads 64-row slices with TMA (one of x, one of
//            each plane of dy), warp 1 of the even CTA issues the MMAs, eight warps drain the
//            accumulator. The accumulator is drained every 1024 rows (of one plane) into registers
//            and added there in fp32: the tensor core truncates its running sum at every step, a
//            bias that grows with the number of steps.
//            Whole tiles go to the pairs in rounds; the slices of the tiles left over after the
//            last full round are dealt out evenly. Where a tile so falls to several pairs, the one
//            with its last slices adds the others' sums, which come through the workspace in fp32,
//            to its own, always in the same order. The old gradient is added last. It waits only for pairs of lower numbers, whose
//            blocks start no later than its own, and for work that they do first.
// Waits are bounded as in the Newton-Schulz products (pair_pipe.cuh describes the unwinding).
#include <cuda.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "device_once.h"
#include "fast_div.cuh"
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
constexpr uint32_t kBox = 64 * 64 * 2;          // 64 contraction rows x 64 columns, bf16
constexpr uint32_t kOperand = 2 * kBox;         // a CTA's 128 columns of one operand
constexpr uint32_t kRing = 12 * kOperand;       // operand stages: 6 of x and dy, or 3 of x and three planes
constexpr int kEpiWarps = 8;
constexpr int kEpiFirst = 4;                    // warps 2 and 3 are idle: registers go by groups of four warps
constexpr int kThreads = 32 * (kEpiFirst + kEpiWarps);
// Registers per thread: 384 threads launch with at most 168; the first four warps hand most of
// theirs to the eight that hold 128 sums each (72 + 2 x 216 = 3 x 168).
constexpr uint32_t kRegsFew = 72, kRegsMany = 216;
constexpr uint32_t kTranspose = 32 * 32 * 4;    // bytes per epilogue warp
constexpr size_t kSmem = 1024 + kRing + kEpiWarps * kTranspose + 512;
static_assert(kSmem <= 232448, "dynamic shared memory per CTA");
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int64_t kCost = 8;                    // see layout_of
constexpr uint32_t kGroup = 8;                  // tile rows that sweep the columns together (L2 reuse)

constexpr int64_t kPart = kTile * kTile;        // floats of one part
constexpr uint32_t kPiece = 32 * 64 * 4, kJoin = 3;   // bytes of a warp's 64 columns of a part, and pieces ahead
static_assert(kJoin * kPiece * kEpiWarps <= kRing, "join");

struct ProductArgs {
  void* grad;
  int64_t gs;               // its row stride
  float* parts;             // [workers + left - 1][kPart]
  uint32_t* ready;          // [left][16]: parts written of each left-over tile, by epilogue warp of the pair
  uint32_t n, k, tiles_n, tiles_k;
  uint32_t whole, left;     // tiles given to the pairs whole, and the rest, whose slices are dealt out
  uint32_t workers;         // pairs that share them: each has `share` slices, the first `extra` one more
  uint32_t share, extra;
  uint32_t slices;
  uint32_t plane_rows;      // rows between planes of dy
  int accumulate;
  int vec;                  // groups of four columns of grad are aligned
  int* status;
  uint64_t wait_ns;
};

// Four consecutive, aligned columns of grad.
template <bool BF16>
__device__ __forceinline__ float4 load4(const void* p, int64_t at) {
  if constexpr (BF16) {
    const uint2 raw = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p) + at);
    return make_float4(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                       __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u));
  } else {
    return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  }
}

// An epilogue warp's 32 rows x 32 columns of grad (rows x cols of them exist) go through its 4 KB of
// shared memory. 16-byte chunk c of row r lies at chunk c ^ (r & 7) of its row: eight lanes that
// have a row's 32 columns, and lanes that each have a row, meet no bank twice. `at` is the place of
// the first row and column.
//
// A lane's eight accesses of whole, aligned blocks: rows 4 i + lane / 8, columns 4 (lane % 8) on.
template <bool BF16>
__device__ __forceinline__ void block_load(const ProductArgs& a, int64_t at, int lane, float4 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = load4<BF16>(a.grad, at + (4 * i + (lane >> 3)) * a.gs + (lane & 7) * 4);
}

__device__ __forceinline__ void block_sums(int lane, const float4* stg, bool add, const float4 (&old)[8], float4 (&v)[8]) {
  const int sub = lane >> 3, chunk = lane & 7;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = stg[(4 * i + sub) * 8 + (chunk ^ ((4 * i + sub) & 7))];
    if (add) v[i] = make_float4(v[i].x + old[i].x, v[i].y + old[i].y, v[i].z + old[i].z, v[i].w + old[i].w);
  }
}

template <bool BF16>
__device__ __forceinline__ void block_store(const ProductArgs& a, int64_t at, int lane, const float4 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    store4<BF16>(a.grad, at + (4 * i + (lane >> 3)) * a.gs + (lane & 7) * 4, {v[i].x, v[i].y, v[i].z, v[i].w});
}

// Any other block: a lane per column, eight rows at a time.
template <bool BF16>
__device__ __forceinline__ void block_out_any(const ProductArgs& a, int64_t at, int rows, int cols, int lane, const float4* stg) {
  if (lane >= cols) return;
  for (int r0 = 0; r0 < rows; r0 += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = a.accumulate && r0 + i < rows ? load1<BF16>(a.grad, at + (r0 + i) * a.gs + lane) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = r0 + i;
      if (r < rows)
        store1<BF16>(a.grad, at + r * a.gs + lane, v[i] + reinterpret_cast<const float*>(stg + r * 8 + ((lane >> 2) ^ (r & 7)))[lane & 3]);
    }
  }
}

// A tile and its range [s0, s1) of slices. part: where its sum goes among the parts, or -1: to
// grad, after `others` parts of the tile from `first_part` on.
struct Unit {
  uint32_t ti, tj, s0, s1, left_tile, others, first_part;
  int part;
};

// The units of one pair, in the order in which all of its warps take them: whole tiles, then, as
// worker q, its slices of the left-over tiles laid end to end (below 2^31 in all), last tile first.
// Its part of left-over tile t has place q + t, which no other pair and tile have.
struct Units {
  const ProductArgs& a;
  uint32_t next_whole, pairs, q;
  uint32_t begin, at;
  __device__ Units(const ProductArgs& a_, uint32_t pair, uint32_t pairs_) : a(a_), next_whole(pair), pairs(pairs_), q(pair) {
    begin = at = 0;
    if (pair < a.workers) {
      begin = pair * a.share + min(pair, a.extra);
      at = begin + a.share + (pair < a.extra ? 1 : 0);
    }
  }
  __device__ bool next(Unit& u) {
    uint32_t tile;
    u.s0 = 0;
    u.s1 = a.slices;
    u.part = -1;
    u.others = 0;
    if (next_whole < a.whole) {
      tile = next_whole;
      next_whole += pairs;
    } else if (at > begin) {
      const uint32_t t = (at - 1) / a.slices, t0 = t * a.slices;
      u.s0 = begin > t0 ? begin - t0 : 0;
      u.s1 = at - t0;
      at = t0 + u.s0;
      tile = a.whole + t;
      u.left_tile = t;
      if (u.s1 < a.slices) {
        u.part = (int)(q + t);
      } else if (u.s0 > 0) {
        const uint32_t more = a.extra * (a.share + 1);   // slices of the workers that have one more
        const uint32_t q0 = t0 < more ? t0 / (a.share + 1) : a.extra + (t0 - more) / a.share;   // has the tile's first
        u.others = q - q0;
        u.first_part = q0 + t;
      }
    } else {
      return false;
    }
    tile_place(a.tiles_n, a.tiles_k, tile, u.ti, u.tj);
    return true;
  }
  static __device__ void tile_place(uint32_t tiles_n, uint32_t tiles_k, uint32_t tile, uint32_t& ti, uint32_t& tj) {
    const uint32_t per = kGroup * tiles_k, g = tile / per, first = g * kGroup;
    const uint32_t size = min(kGroup, tiles_n - first);
    ti = first + (tile - g * per) % size;
    tj = (tile - g * per) / size;
  }
};

template <bool OUT_BF16, int PLANES>
__global__ void __launch_bounds__(kThreads, 1)
    wgrad_product_kernel(const __grid_constant__ CUtensorMap map_dy, const __grid_constant__ CUtensorMap map_x,
                         const ProductArgs a) {
  constexpr int kStages = PLANES == 1 ? 6 : 3;
  constexpr uint32_t kStage = (1 + PLANES) * kOperand;   // x, then the planes of dy
  constexpr uint32_t kChunk = 16 / PLANES;               // slices between drains: at most 64 steps
  static_assert(kStages * kStage == kRing, "stages");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  float4* transpose = reinterpret_cast<float4*>(smem + kRing);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing + kEpiWarps * kTranspose);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* join = drain + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(join + kEpiWarps * kJoin);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* zero_flag = abort_flag + 1;   // never set: the drain waits poll it
  volatile uint32_t* fill_count = reinterpret_cast<volatile uint32_t*>(zero_flag + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;
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
    for (uint32_t i = 0; i < kEpiWarps * kJoin; ++i) mbar_init(&join[i], 1);
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
  if (warp < kEpiFirst) {
    regs_dec<kRegsFew>();
    if (warp == 0 && lane == 0) {
      uint32_t stage = 0, phase = 0, fills = 0;
      Units units(a, pair, pairs);
      Unit w;
      while (!timed_out && units.next(w)) {
        const int32_t n0 = (int32_t)(w.ti * kTile + rank * 128), k0 = (int32_t)(w.tj * kTile + rank * 128);
        for (uint32_t s = w.s0; s < w.s1; ++s) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag, wait_ns)) {
            timed_out = true;
            break;
          }
          const int32_t t0 = (int32_t)(s * kSlice);
          uint8_t* dst = smem + stage * kStage;
          const uint32_t bar = mapa_shared(smem_u32(&full[stage]), 0);
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStage);
          tma_load_2d_pair(dst, &map_x, bar, k0, t0);
          tma_load_2d_pair(dst + kBox, &map_x, bar, k0 + 64, t0);
#pragma unroll
          for (int p = 0; p < PLANES; ++p) {
            const int32_t y = t0 + (int32_t)(p * a.plane_rows);
            tma_load_2d_pair(dst + (1 + p) * kOperand, &map_dy, bar, n0, y);
            tma_load_2d_pair(dst + (1 + p) * kOperand + kBox, &map_dy, bar, n0 + 64, y);
          }
          ++fills;
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (timed_out) raise_abort(abort_flag, true, rank);
      *fill_count = fills;
    }
    if (warp == 1 && lane == 0 && leader) {
      const uint32_t idesc = idesc_bf16_f32(kTile, kTile, 1, 1);
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      Units units(a, pair, pairs);
      Unit w;
      while (!timed_out && units.next(w)) {
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
            const uint32_t bd = smem_u32(smem + stage * kStage), ad = bd + kOperand;
#pragma unroll
            for (uint32_t p = 0; p < PLANES; ++p)
#pragma unroll
              for (uint32_t i = 0; i < kSlice / 16; ++i)
                tc_mma_f16_pair(tmem_base + acc * 256u, smem_desc_sw128(ad + p * kOperand + i * 2048u, kBox, 1024),
                                smem_desc_sw128(bd + i * 2048u, kBox, 1024), idesc, s != c0 || p != 0 || i != 0 ? 1u : 0u);
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
    regs_inc<kRegsMany>();
    // each warp: 32 accumulator rows (a lane each) x 128 of the tile's columns
    const uint32_t quarter = (uint32_t)(warp & 3), half = (uint32_t)(warp - kEpiFirst) >> 2;
    float4* stg = transpose + (uint32_t)(warp - kEpiFirst) * 256;
    uint32_t acc = 0, acc_phase = 0;
    Units units(a, pair, pairs);
    Unit w;
    while (units.next(w)) {
      const int64_t r0 = (int64_t)w.ti * kTile + rank * 128 + quarter * 32, col0 = (int64_t)w.tj * kTile + half * 128;
      const int rows = (int)min((int64_t)32, max((int64_t)0, (int64_t)a.n - r0));
      auto block = [&](int g, int& cols, bool& fast) {
        cols = (int)min((int64_t)32, max((int64_t)0, (int64_t)a.k - col0 - g * 32));
        fast = a.vec && rows == 32 && cols == 32;
        return r0 * a.gs + col0 + g * 32;
      };
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
      const uint32_t me = rank * 8 + quarter * 2 + half;   // among the pair's epilogue warps
      if (w.part >= 0) {
        // four columns of the warp's 32 rows together
        float4* out = reinterpret_cast<float4*>(a.parts + w.part * kPart + me * 4096) + lane;
#pragma unroll
        for (int i = 0; i < 32; ++i) out[i * 32] = make_float4(sum[i * 4], sum[i * 4 + 1], sum[i * 4 + 2], sum[i * 4 + 3]);
        __threadfence();
        __syncwarp();
        if (lane == 0) red_release_gpu_add(a.ready + w.left_tile * 16 + me, 1);
        continue;
      }
      // The old gradient is added last, once: to it, chunks of the sum that are each below half its
      // step would be lost one by one. It is read one block ahead of its use.
      float4 old[8];
      auto fetch_old = [&](int g) {
        int cols;
        bool fast;
        const int64_t at = block(g, cols, fast);
        if (a.accumulate && fast) block_load<OUT_BF16>(a, at, lane, old);
      };
      fetch_old(0);
      if (w.others) {
        // the last unit of the pair: the operand ring is free, and brings the parts in pieces of
        // 64 columns, kJoin of them ahead
        const float* from = a.parts + w.first_part * kPart + me * 4096;
        uint8_t* slots = smem + (uint32_t)(warp - kEpiFirst) * (kRing / kEpiWarps);
        uint64_t* landed = join + (warp - kEpiFirst) * kJoin;
        bool ok = lane != 0 || counter_wait_bounded(a.ready + w.left_tile * 16 + me, w.others, abort_flag, wait_ns);
        fence_proxy_async_global();
        const uint32_t pieces = w.others * 2;
        auto fetch = [&](uint32_t i) {
          if (lane != 0 || i >= pieces) return;
          uint64_t* bar = landed + i % kJoin;
          mbar_arrive_expect_tx(bar, kPiece);
          bulk_load(slots + i % kJoin * kPiece, from + (i >> 1) * kPart + (i & 1) * 2048, kPiece, bar);
        };
        ok = __all_sync(0xffffffffu, ok);
        if (ok)
          for (uint32_t i = 0; i < kJoin; ++i) fetch(i);
        for (uint32_t i = 0; ok && i < pieces; i += 2) {
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            // a copy that was asked for is waited for with the long limit: it must not land later
            if (!mbar_wait_bounded(landed + (i + h) % kJoin, (i + h) / kJoin & 1, zero_flag, kTimeoutNs)) timed_out = true;
            const float4* p = reinterpret_cast<const float4*>(slots + (i + h) % kJoin * kPiece) + lane;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float4 v = p[c * 32];
              sum[h * 64 + c * 4] += v.x;
              sum[h * 64 + c * 4 + 1] += v.y;
              sum[h * 64 + c * 4 + 2] += v.z;
              sum[h * 64 + c * 4 + 3] += v.w;
            }
            __syncwarp();
            fetch(i + h + kJoin);
          }
        }
        if (!ok) {
          timed_out = true;
          break;
        }
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        int cols;
        bool fast;
        const int64_t at = block(g, cols, fast);
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          stg[lane * 8 + (c ^ (lane & 7))] = make_float4(sum[g * 32 + c * 4], sum[g * 32 + c * 4 + 1],
                                                         sum[g * 32 + c * 4 + 2], sum[g * 32 + c * 4 + 3]);
        __syncwarp();
        if (fast) {
          float4 v[8];
          block_sums(lane, stg, a.accumulate, old, v);
          if (g < 3) fetch_old(g + 1);
          block_store<OUT_BF16>(a, at, lane, v);
        } else {
          block_out_any<OUT_BF16>(a, at, rows, cols, lane, stg);
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

// rows = 0: the empty sum.
template <bool OUT_BF16>
__global__ void __launch_bounds__(256) wgrad_zero_kernel(void* grad, int64_t gs, int64_t n, int64_t k) {
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n * k; t += (int64_t)gridDim.x * 256)
    store1<OUT_BF16>(grad, t / k * gs + t % k, 0.0f);
}

// Copies dy into bf16 rows of `pitch` elements (a multiple of 8); an fp32 dy into three planes,
// plane_rows apart. A thread has kStageAcc groups of V columns, 256 groups apart, all loaded before
// the first is stored: V = 8 where dy's rows are aligned, else 4. per_row: groups of a row (the last may end in the padding), total: of all
// rows, below 2^31.
template <int V>
constexpr int kStageAcc = V == 8 ? 1 : 4;

template <bool DY_BF16, int V>
__global__ void __launch_bounds__(256) wgrad_stage_dy_kernel(const void* dy, int64_t dys, int64_t n, int64_t plane_rows,
                                                             __nv_bfloat16* out, int64_t pitch, Div per_row, uint32_t total) {
  constexpr int A = kStageAcc<V>;
  const uint32_t i0 = blockIdx.x * (256 * A) + threadIdx.x;
  float all[A][V];
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const uint32_t i = i0 + j * 256, t = per_row.quot(i), c = (i - t * per_row.d) * V;
    if (i >= total) continue;
    if constexpr (V == 8) {
      load8<DY_BF16>(dy, t * dys + c, all[j]);
    } else {
      load4_any<DY_BF16>(dy, t * dys + c, n - c, all[j]);
    }
  }
  auto put = [&](int64_t to, const float (&v)[V]) {
    if constexpr (V == 8) {
      store8<true>(out, to, v);
    } else {
      store4<true>(out, to, v);
    }
  };
#pragma unroll
  for (int j = 0; j < A; ++j) {
    const uint32_t i = i0 + j * 256, t = per_row.quot(i), c = (i - t * per_row.d) * V;
    if (i >= total) break;
    float (&v)[V] = all[j];
    if constexpr (DY_BF16) {
      put(t * pitch + c, v);
    } else {
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        float part[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          // the top 16 bits of a float are its value truncated to bf16; infinities and NaN stay whole
          uint32_t top = __float_as_uint(v[e]) & 0xffff0000u;
          const bool finite = (top & 0x7f800000u) != 0x7f800000u;
          if (!finite && (__float_as_uint(v[e]) & 0x7fffffu)) top |= 0x00400000u;
          part[e] = __uint_as_float(top);
          v[e] = finite ? v[e] - part[e] : 0.0f;
        }
        put((p * plane_rows + t) * pitch + c, part);
      }
    }
  }
}

template <bool DY_BF16, int V>
cudaError_t launch_stage_dy(const WgradArgs& a, __nv_bfloat16* out, int64_t pitch, cudaStream_t s) {
  const int64_t per_row = (a.n + V - 1) / V, most = ((int64_t(1) << 31) - 1) / per_row;
  for (int64_t r = 0; r < a.rows; r += most) {
    const int64_t total = (a.rows - r < most ? a.rows - r : most) * per_row;
    const char* from = static_cast<const char*>(a.dy) + r * a.dys * (DY_BF16 ? 2 : 4);
    wgrad_stage_dy_kernel<DY_BF16, V><<<(unsigned)((total + 256 * kStageAcc<V> - 1) / (256 * kStageAcc<V>)), 256, 0, s>>>(
        from, a.dys, a.n, a.rows, out + r * pitch, pitch, Div((uint32_t)per_row), (uint32_t)total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
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
  int64_t x, dy, parts, ready, bytes;    // workspace offsets
  int64_t x_pitch, dy_pitch;
  int planes;
  uint32_t tiles_n, tiles_k, slices, whole, left, workers;
  bool copy_dy;
};

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

Layout layout_of(int64_t rows, int64_t n, int64_t k, int dy_bf16, int dy_aligned) {
  Layout l;
  l.planes = dy_bf16 ? 1 : 3;
  l.copy_dy = !dy_bf16 || !dy_aligned;
  l.x_pitch = up(k, 8);
  l.dy_pitch = up(n, 8);
  l.tiles_n = (uint32_t)((n + kTile - 1) / kTile);
  l.tiles_k = (uint32_t)((k + kTile - 1) / kTile);
  l.slices = (uint32_t)((rows + kSlice - 1) / kSlice);
  // The tiles of the last round whole, or dealt out to so many workers that the last of them ends
  // soonest, in slices of one plane (0.33 us each): its slices, 4 for each part that it adds (1.3 us)
  // and kCost for the joining.
  const int64_t tiles = (int64_t)l.tiles_n * l.tiles_k, pairs = kSms / 2, left = tiles % pairs, all = left * l.slices;
  int64_t workers = left, best = (int64_t)l.slices * l.planes;
  for (int64_t w = left + 1; left > 0 && w <= pairs && w <= all; ++w) {
    const int64_t per = (all + w - 1) / w, cost = per * l.planes + (l.slices + per - 1) / per * 4 + kCost;
    if (cost < best) {
      best = cost;
      workers = w;
    }
  }
  const bool deal = workers > left;
  l.left = (uint32_t)(deal ? left : 0);
  l.whole = (uint32_t)(tiles - l.left);
  l.workers = (uint32_t)(deal ? workers : 0);
  l.x = 0;
  l.dy = up(rows * l.x_pitch * 2, 256);
  l.parts = l.dy + (l.copy_dy ? up(rows * l.planes * l.dy_pitch * 2, 256) : 0);
  l.ready = l.parts + (deal ? (workers + left - 1) * kPart * 4 : 0);
  l.bytes = l.ready + l.left * 64;
  return l;
}

template <bool OUT_BF16, int PLANES>
cudaError_t launch_product(const CUtensorMap& md, const CUtensorMap& mx, const ProductArgs& p, cudaStream_t s) {
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = (cudaError_t)once.run(dev, [&] {
    return (int)cudaFuncSetAttribute(wgrad_product_kernel<OUT_BF16, PLANES>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)kSmem);
  });
  if (e != cudaSuccess) return e;
  uint32_t pairs = p.whole > p.workers ? p.whole : p.workers;
  if (pairs > kSms / 2) pairs = kSms / 2;
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
  return cudaLaunchKernelEx(&cfg, wgrad_product_kernel<OUT_BF16, PLANES>, md, mx, p);
}

}  // namespace

int64_t wgrad_workspace(int64_t rows, int64_t n, int64_t k, int dy_bf16) {
  return layout_of(rows, n, k, dy_bf16, 0).bytes;   // with room for a copy of a dy that is not aligned
}

cudaError_t launch_wgrad(const WgradArgs& a, int dy_bf16, int grad_bf16, int sms, char* ws, int64_t* launches,
                         cudaStream_t s) {
  const int aligned = (uintptr_t)a.dy % 16 == 0 && a.dys % 8 == 0;
  const Layout l = layout_of(a.rows, a.n, a.k, dy_bf16, aligned);
  if (a.rows == 0) {
    ++*launches;
    const int64_t blocks = (a.n * a.k + 255) / 256, cap = (int64_t)sms * 16;
    const unsigned g = (unsigned)(blocks < cap ? blocks : cap);
    if (grad_bf16) wgrad_zero_kernel<true><<<g, 256, 0, s>>>(a.grad, a.gs, a.n, a.k);
    else wgrad_zero_kernel<false><<<g, 256, 0, s>>>(a.grad, a.gs, a.n, a.k);
    return cudaGetLastError();
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
  m.zero = reinterpret_cast<uint32_t*>(ws + l.ready);
  m.zeros = (int)l.left * 16;
  cudaError_t e = launch_mx_restore(m, 1, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (l.copy_dy) {
    __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(ws + l.dy);
    const bool v8 = a.n % 8 == 0 && (uintptr_t)a.dy % 16 == 0 && a.dys % 4 == 0;
    if (dy_bf16) e = launch_stage_dy<true, 4>(a, out, l.dy_pitch, s);
    else if (v8) e = launch_stage_dy<false, 8>(a, out, l.dy_pitch, s);
    else e = launch_stage_dy<false, 4>(a, out, l.dy_pitch, s);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  CUtensorMap md, mx;
  e = l.copy_dy ? operand_map(&md, ws + l.dy, a.rows * l.planes, a.n, l.dy_pitch)
                : operand_map(&md, a.dy, a.rows, a.n, a.dys);
  if (e == cudaSuccess) e = operand_map(&mx, ws + l.x, a.rows, a.k, l.x_pitch);
  if (e != cudaSuccess) return e;
  ProductArgs p = {};
  p.grad = a.grad;
  p.gs = a.gs;
  p.parts = reinterpret_cast<float*>(ws + l.parts);
  p.ready = reinterpret_cast<uint32_t*>(ws + l.ready);
  p.n = (uint32_t)a.n;
  p.k = (uint32_t)a.k;
  p.tiles_n = l.tiles_n;
  p.tiles_k = l.tiles_k;
  p.whole = l.whole;
  p.left = l.left;
  p.workers = l.workers;
  p.share = l.workers ? l.left * l.slices / l.workers : 0;
  p.extra = l.workers ? l.left * l.slices % l.workers : 0;
  p.slices = l.slices;
  p.plane_rows = (uint32_t)a.rows;
  p.accumulate = a.accumulate;
  p.vec = (uintptr_t)a.grad % 16 == 0 && a.gs % 4 == 0;
  p.status = a.status;
  p.wait_ns = a.wait_ns;
  if (l.planes == 1) e = grad_bf16 ? launch_product<true, 1>(md, mx, p, s) : launch_product<false, 1>(md, mx, p, s);
  else e = grad_bf16 ? launch_product<true, 3>(md, mx, p, s) : launch_product<false, 3>(md, mx, p, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  return e;
}

}  // namespace muon
