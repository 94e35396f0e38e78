// Token embedding with scaling, and its gradient by sorted tokens:
//   out[t] = scale table[id_t];   grad[v] (+)= scale sum over t with id_t = v of dy[t].
// A negative id is padding: a zero row of out, nothing in grad. An id past the vocabulary is
// treated the same way and recorded in the device status word.
//
// The gradient in three launches, with no atomics on data, so that its sums have one order:
//   sort    each block owns a range of ids and reads all tokens: it counts the tokens below its
//           range (where its part of the sorted list begins) and places its own, stably, by
//           per-warp counts of each id. No block waits for another.
//   sums    blocks of kRun sorted positions x a slice of columns add the rows of each run of
//           equal ids in fp32; runs within a block go straight to grad, the parts of runs that
//           cross its borders to a workspace. Further blocks zero the rows of ids that no token has.
//   join    adds the parts of each crossing run in order.
#include <cuda_bf16.h>
#include <stdint.h>

#include "muon_internal.h"
#include "ops_internal.h"
#include "ptx.cuh"
#include "vec_io.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortIds = 1024;      // most ids of one block's range
constexpr int kRun = 32;            // sorted positions per block of the sums
constexpr int kFillRows = 16;       // ids per zero-filling block

template <bool ID64>
__device__ __forceinline__ int64_t load_id(const void* tokens, int64_t i) {
  if constexpr (ID64) return static_cast<const int64_t*>(tokens)[i];
  else return static_cast<const int32_t*>(tokens)[i];
}

template <int V, bool T_BF16, bool O_BF16, bool ID64>
__global__ void __launch_bounds__(kThreads) embedding_kernel(EmbedArgs a) {
  const int64_t per_row = a.dim / V, total = a.n * per_row;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < total; t += (int64_t)gridDim.x * kThreads) {
    const int64_t row = t / per_row, c = (t - row * per_row) * V;
    const int64_t id = load_id<ID64>(a.tokens, row);
    float v[V];
    if (id >= 0 && id < a.vocab) {
      load_v<V, T_BF16>(a.table, id * a.table_stride + c, v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] *= a.scale;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 0.0f;
      if (id >= a.vocab && c == 0) atomicOr(a.status, kStatusToken);
    }
    store_v<V, O_BF16>(a.out, row * a.out_stride + c, v);
  }
}

// ids: ids per block (at most kSortIds). Warps own consecutive segments of the tokens.
template <bool ID64>
__global__ void __launch_bounds__(kSortThreads, 1) token_sort_kernel(EmbedGradArgs a, int ids) {
  extern __shared__ int cnt[];   // [kSortWarps][ids]
  __shared__ int warp_part[kSortWarps];
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lo = (int64_t)blockIdx.x * ids;
  const int here = (int)min((int64_t)ids, a.vocab - lo);
  for (int i = threadIdx.x; i < kSortWarps * ids; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t seg = (a.n + kSortThreads - 1) / kSortThreads * 32;
  const int64_t t0 = warp * seg, t1 = min(a.n, t0 + seg);
  int* mine = cnt + warp * ids;
  int below = 0;
  bool bad = false;
  for (int64_t t = t0; t < t1; t += 32) {
    const int64_t id = t + lane < t1 ? load_id<ID64>(a.tokens, t + lane) : -1;
    below += id >= 0 && id < lo ? 1 : 0;
    bad |= id >= a.vocab;
    const bool in = id >= lo && id < lo + here;
    if (!__any_sync(0xffffffffu, in)) continue;
    const int b = in ? (int)(id - lo) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, b);
    if (in && lane == __ffs(same) - 1) mine[b] += __popc(same);
    __syncwarp();
  }
  if (blockIdx.x == 0 && bad) atomicOr(a.status, kStatusToken);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) below += __shfl_xor_sync(0xffffffffu, below, o);
  if (lane == 0) warp_part[warp] = below;
  __syncthreads();
  int first = 0;
  for (int w = 0; w < kSortWarps; ++w) first += warp_part[w];
  __syncthreads();
  // one thread per id: counts before each warp, then a block scan over the ids
  const int b = threadIdx.x;
  int total = 0;
  if (b < here) {
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * ids + b];
      cnt[w * ids + b] = total;
      total += c;
    }
  }
  int scan = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) warp_part[warp] = scan;
  __syncthreads();
  int before = first;
  for (int w = 0; w < warp; ++w) before += warp_part[w];
  const int begin = before + scan - total;
  if (b < here) {
    a.start[lo + b] = begin;
    for (int w = 0; w < kSortWarps; ++w) cnt[w * ids + b] += begin;
    if (lo + b == a.vocab - 1) a.start[a.vocab] = begin + total;
  }
  __syncthreads();
  for (int64_t t = t0; t < t1; t += 32) {
    const int64_t id = t + lane < t1 ? load_id<ID64>(a.tokens, t + lane) : -1;
    const bool in = id >= lo && id < lo + here;
    if (!__any_sync(0xffffffffu, in)) continue;
    const int k = in ? (int)(id - lo) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, k);
    if (in) {
      const int pos = mine[k] + __popc(same & ((1u << lane) - 1u));
      a.order[pos] = (int)(t + lane);
      a.keys[pos] = (int)id;
    }
    __syncwarp();
    if (in && lane == __ffs(same) - 1) mine[k] += __popc(same);
    __syncwarp();
  }
}

template <int V, bool G_BF16>
__device__ __forceinline__ void write_grad(const EmbedGradArgs& a, int64_t id, int64_t c, float (&v)[V]) {
  const int64_t at = id * a.grad_stride + c;
  if (a.accumulate) {
    float old[V];
    load_v<V, G_BF16>(a.grad, at, old);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = old[e] + a.scale * v[e];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] *= a.scale;
  }
  store_v<V, G_BF16>(a.grad, at, v);
}

// Blocks [0, chunks): sums of one chunk of sorted positions over columns blockIdx.y * kThreads * V
// onwards. Blocks [chunks, ...): zeros for ids without tokens (never launched when accumulating).
template <int V, bool D_BF16, bool G_BF16>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(EmbedGradArgs a, int chunks) {
  __shared__ int key[kRun + 2], ord[kRun];
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if ((int64_t)blockIdx.x >= chunks) {
    const int64_t v0 = ((int64_t)blockIdx.x - chunks) * kFillRows;
    const int64_t v1 = min(a.vocab, v0 + kFillRows);
    if (c >= a.dim) return;
    float z[V];
#pragma unroll
    for (int e = 0; e < V; ++e) z[e] = 0.0f;
    for (int64_t v = v0; v < v1; ++v)
      if (a.start[v] == a.start[v + 1]) store_v<V, G_BF16>(a.grad, v * a.grad_stride + c, z);
    return;
  }
  const int valid = a.start[a.vocab];
  const int p0 = blockIdx.x * kRun;
  if (p0 >= valid) return;
  const int m = min(kRun, valid - p0);
  for (int i = threadIdx.x; i < kRun + 2; i += blockDim.x) {   // key[i] belongs to position p0 + i - 1
    const int p = p0 + i - 1;
    key[i] = p >= 0 && p < valid ? a.keys[p] : -1;
    if (i < m) ord[i] = a.order[p0 + i];
  }
  __syncthreads();
  if (c >= a.dim) return;
  float sum[V];
#pragma unroll
  for (int e = 0; e < V; ++e) sum[e] = 0.0f;
  bool from_before = key[0] == key[1];
  constexpr int kAhead = 8;
  for (int i0 = 0; i0 < m; i0 += kAhead) {
    float v[kAhead][V];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (i0 + u < m) load_v<V, D_BF16>(a.dy, ord[i0 + u] * a.dy_stride + c, v[u]);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= m) break;
#pragma unroll
      for (int e = 0; e < V; ++e) sum[e] += v[u][e];
      const bool ends = key[i + 2] != key[i + 1];
      if (ends || i == m - 1) {
        if (ends && !from_before) {
          write_grad<V, G_BF16>(a, key[i + 1], c, sum);
        } else {   // slot 0: a run that came from before; slot 1: one that begins here and goes on
          store_v<V, false>(a.partial, ((int64_t)blockIdx.x * 2 + (from_before ? 0 : 1)) * a.dim + c, sum);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sum[e] = 0.0f;
        from_before = false;
      }
    }
  }
}

// Block x joins the run that begins in chunk x and goes on past it.
template <int V, bool G_BF16>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(EmbedGradArgs a) {
  grid_dependency_wait();
  const int valid = a.start[a.vocab];
  const int64_t p1 = ((int64_t)blockIdx.x + 1) * kRun;
  if (p1 >= valid) return;
  const int id = a.keys[p1];
  if (a.keys[p1 - 1] != id || a.start[id] < p1 - kRun) return;
  const int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V;
  if (c >= a.dim) return;
  const int last = (a.start[id + 1] - 1) / kRun;
  float sum[V];
  load_v<V, false>(a.partial, ((int64_t)blockIdx.x * 2 + 1) * a.dim + c, sum);
#pragma unroll 4
  for (int k = (int)blockIdx.x + 1; k <= last; ++k) {
    float v[V];
    load_v<V, false>(a.partial, (int64_t)k * 2 * a.dim + c, v);
#pragma unroll
    for (int e = 0; e < V; ++e) sum[e] += v[e];
  }
  write_grad<V, G_BF16>(a, id, c, sum);
}

bool aligned8(const void* p, int64_t stride) { return (uintptr_t)p % 16 == 0 && stride % 8 == 0; }

template <int V, bool T, bool O>
cudaError_t embed_ids(const EmbedArgs& a, int id64, cudaStream_t s) {
  const int64_t blocks = (a.n * (a.dim / V) + kThreads - 1) / kThreads;
  const int grid = (int)(blocks < (1 << 20) ? blocks : (1 << 20));
  if (id64) embedding_kernel<V, T, O, true><<<grid, kThreads, 0, s>>>(a);
  else embedding_kernel<V, T, O, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int V>
cudaError_t embed_types(const EmbedArgs& a, int tb, int ob, int id64, cudaStream_t s) {
  if (tb && ob) return embed_ids<V, true, true>(a, id64, s);
  if (tb) return embed_ids<V, true, false>(a, id64, s);
  if (ob) return embed_ids<V, false, true>(a, id64, s);
  return embed_ids<V, false, false>(a, id64, s);
}

template <int V, bool D, bool G>
cudaError_t embed_sums(const EmbedGradArgs& a, int64_t* launches, cudaStream_t s) {
  const int64_t per_row = a.dim / V;
  int threads = 32;
  while (threads < kThreads && threads < per_row) threads *= 2;
  const unsigned slices = (unsigned)((per_row + threads - 1) / threads);
  const int64_t chunks = (a.n + kRun - 1) / kRun;
  const int64_t fill = a.accumulate ? 0 : (a.vocab + kFillRows - 1) / kFillRows;
  cudaError_t e = launch_dependent(embed_sum_kernel<V, D, G>, dim3((unsigned)(chunks + fill), slices), dim3(threads), 0, s, a,
                                   (int)chunks);
  ++*launches;
  if (e != cudaSuccess || chunks < 2) return e;
  e = launch_dependent(embed_join_kernel<V, G>, dim3((unsigned)(chunks - 1), slices), dim3(threads), 0, s, a);
  ++*launches;
  return e;
}

template <int V>
cudaError_t embed_grad_types(const EmbedGradArgs& a, int db, int gb, int64_t* launches, cudaStream_t s) {
  if (db && gb) return embed_sums<V, true, true>(a, launches, s);
  if (db) return embed_sums<V, true, false>(a, launches, s);
  if (gb) return embed_sums<V, false, true>(a, launches, s);
  return embed_sums<V, false, false>(a, launches, s);
}

}  // namespace

cudaError_t launch_embedding(const EmbedArgs& a, int table_bf16, int out_bf16, int id64, cudaStream_t s) {
  if (a.dim % 8 == 0 && aligned8(a.table, a.table_stride) && aligned8(a.out, a.out_stride))
    return embed_types<8>(a, table_bf16, out_bf16, id64, s);
  return embed_types<1>(a, table_bf16, out_bf16, id64, s);
}

int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim, EmbedGradArgs* a, char* base) {
  auto up = [](int64_t b) { return (b + 255) / 256 * 256; };
  const int64_t order = 0, keys = order + up(n * 4), start = keys + up(n * 4), partial = start + up((vocab + 1) * 4);
  const int64_t chunks = (n + kRun - 1) / kRun;
  if (a) {
    a->order = reinterpret_cast<int*>(base + order);
    a->keys = reinterpret_cast<int*>(base + keys);
    a->start = reinterpret_cast<int*>(base + start);
    a->partial = reinterpret_cast<float*>(base + partial);
  }
  return partial + up(chunks * 2 * dim * 4);
}

cudaError_t launch_embedding_grad(const EmbedGradArgs& a, int dy_bf16, int grad_bf16, int id64, int sms,
                                  int64_t* launches, cudaStream_t s) {
  // ranges of equal length, about one per SM
  int64_t ids = (a.vocab + sms - 1) / sms;
  if (ids > kSortIds) ids = kSortIds;
  const int64_t blocks = (a.vocab + ids - 1) / ids;
  const size_t smem = (size_t)kSortWarps * ids * sizeof(int);
  const void* k = id64 ? (const void*)token_sort_kernel<true> : (const void*)token_sort_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortWarps * kSortIds * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  if (id64) token_sort_kernel<true><<<(unsigned)blocks, kSortThreads, smem, s>>>(a, (int)ids);
  else token_sort_kernel<false><<<(unsigned)blocks, kSortThreads, smem, s>>>(a, (int)ids);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  if (a.dim % 8 == 0 && aligned8(a.dy, a.dy_stride) && aligned8(a.grad, a.grad_stride))
    return embed_grad_types<8>(a, dy_bf16, grad_bf16, launches, s);
  return embed_grad_types<1>(a, dy_bf16, grad_bf16, launches, s);
}

}  // namespace muon
