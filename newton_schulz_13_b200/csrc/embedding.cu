// Token embedding with scaling, and its gradient by sorted tokens:
//   out[t] = scale table[id_t];   grad[v] (+)= scale sum over t with id_t = v of dy[t].
// A negative id is padding: a zero row of out, nothing in grad. An id past the vocabulary is
// treated the same way and recorded in the device status word. The lookup is bound by HBM (16384 rows
// of 768: 7.3 us, 6 TB/s).
//
// The gradient in two launches, with no atomics on data, so that its sums have one order:
//   sort    each block owns the ids of one residue modulo a power of two (frequent ids, which
//           neighbour one another in most vocabularies, so fall to different blocks) and reads all
//           tokens: it counts those of lower residues (where its part of the sorted list begins)
//           and places its own, stably, by per-warp counts of each id. No block waits for another.
//   sums    a warp adds, over 256 columns in fp32, the rows of the runs of equal ids (and of the
//           pieces of long runs) that begin in a window of the sorted list, kAhead rows on the way
//           at a time, and writes those parts of the gradient. Pieces' sums go to a workspace, and
//           the warp that finishes the last of eight adds them in their order, eight such sums
//           become one again, up to the run's. Between these blocks lie others that zero the rows
//           of absent ids: most of the bytes where the vocabulary is large.
// 16384 tokens into 128256 x 4096 bf16: 14 + 190 us (5.9 TB/s); 12276 into 50257 x 768 fp32: 12 + 16 us,
// bound by the sort's two serial walks over a warp's tokens and the levels of the joining.
#include <cuda_bf16.h>
#include <stdint.h>

#include "device_once.h"
#include "muon_internal.h"
#include "ops_internal.h"
#include "ptx.cuh"
#include "vec_io.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortIds = 1024;      // most ids of one block
constexpr int kBatch = 16;          // tokens per lane that a sort warp loads at a time
constexpr int kWindow = 8;          // sorted places per warp of the sums
constexpr int kFan = 8;             // sums that become one
constexpr int kPiece = 8;           // rows per piece of a long run (the last piece: up to 15)
constexpr int kLong = 16;           // runs from this length on are summed in pieces
static_assert(kWindow <= kPiece, "a long piece ends past its window");
constexpr int kCols = 256;          // columns per warp
constexpr int kFillRows = 32;       // ids per zero-filling block

template <bool ID64>
__device__ __forceinline__ int64_t load_id(const void* tokens, int64_t i) {
  if constexpr (ID64) return static_cast<const int64_t*>(tokens)[i];
  else return static_cast<const int32_t*>(tokens)[i];
}

// A warp per row and part of kPart accesses per lane: the id is read once, the row's loads are
// all in flight together.
constexpr int kPart = 4;

template <int V, bool T_BF16, bool O_BF16, bool ID64>
__global__ void __launch_bounds__(kThreads) embedding_kernel(EmbedArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= a.n) return;
  const int64_t id = load_id<ID64>(a.tokens, row);
  const int64_t c0 = ((int64_t)blockIdx.y * kPart * 32 + lane) * V;
  const bool have = id >= 0 && id < a.vocab;
  if (id >= a.vocab && c0 == 0) atomicOr(a.status + kStatusToken, 1);
  Raw<V, T_BF16> raw[kPart];
#pragma unroll
  for (int j = 0; j < kPart; ++j)
    if (have && c0 + j * 32 * V < a.dim) raw[j].load(a.table, id * a.table_stride + c0 + j * 32 * V);
#pragma unroll
  for (int j = 0; j < kPart; ++j) {
    const int64_t c = c0 + j * 32 * V;
    if (c >= a.dim) break;
    float v[V];
    if (have) {
      raw[j].get(v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] *= a.scale;
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = 0.0f;
    }
    store_v<V, O_BF16>(a.out, row * a.out_stride + c, v);
  }
}

// Block b of gridDim.x = 1 << shift takes the ids v with v mod gridDim.x = b; ids: how many there
// are at most. Warps own consecutive segments of the tokens and read them kBatch x 32 at a time; a
// segment of one batch (up to 16,384 tokens in all) is read once. Cnt holds counts up to n.
template <bool ID64, class Cnt>
__global__ void __launch_bounds__(kSortThreads, 1) token_sort_kernel(EmbedGradArgs a, int ids, int shift, int slices) {
  extern __shared__ int smem[];   // Cnt [kSortWarps][ids]: tokens of each id in each warp's segment
  __shared__ int warp_part[kSortWarps], base[kSortIds], length[kSortIds];
  Cnt* cnt = reinterpret_cast<Cnt*>(smem);
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int me = blockIdx.x, mask = (1 << shift) - 1;
  const int64_t seg = (a.n + kSortThreads - 1) / kSortThreads * 32;
  const int64_t t0 = min(a.n, warp * seg), t1 = min(a.n, t0 + seg);
  Cnt* mine = cnt + warp * ids;
  int below = 0;
  bool bad = false;
  int bin[kBatch];   // the id's number in this block, or -1
  auto read = [&](int64_t t, bool count) {
    int64_t id[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) id[j] = t + j * 32 + lane < t1 ? load_id<ID64>(a.tokens, t + j * 32 + lane) : -1;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const bool valid = id[j] >= 0 && id[j] < a.vocab;
      const int r = (int)id[j] & mask;
      if (count) {
        below += valid && r < me ? 1 : 0;
        bad |= id[j] >= a.vocab;
      }
      bin[j] = valid && r == me ? (int)(id[j] >> shift) : -1;
    }
  };
  // lanes of one id among the lanes that have one (match only where there are several)
  auto peers = [&](int k, uint32_t in) { return (in & (in - 1)) == 0 ? in : __match_any_sync(0xffffffffu, k); };
  const int64_t counts = (a.n + kPiece - 1) / kPiece * slices;
  for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x; i < counts; i += (int64_t)gridDim.x * kSortThreads)
    a.count[i] = 0;
  for (int i = threadIdx.x; i < (kSortWarps * ids * (int)sizeof(Cnt) + 3) / 4; i += kSortThreads) smem[i] = 0;
  if (t0 < t1) read(t0, true);
  __syncthreads();
  for (int64_t t = t0; t < t1; t += kBatch * 32) {
    if (t != t0) read(t, true);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const uint32_t in = __ballot_sync(0xffffffffu, bin[j] >= 0);
      if (!in) continue;
      const uint32_t same = peers(bin[j], in);
      if (bin[j] >= 0 && lane == __ffs(same) - 1) mine[bin[j]] += (Cnt)__popc(same);
      __syncwarp();
    }
  }
  if (me == 0 && bad) atomicOr(a.status + kStatusToken, 1);
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) warp_part[warp] = below;
  __syncthreads();
  const int first = __reduce_add_sync(0xffffffffu, warp_part[lane]);
  __syncthreads();
  // one thread per id: counts before each warp, then a block scan over the ids
  const int b = threadIdx.x;
  const int64_t id = ((int64_t)b << shift) + me;
  int total = 0;
  if (b < ids) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * ids + b];
      cnt[w * ids + b] = (Cnt)total;
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
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_part[lane] : 0);
  const int begin = first + before + scan - total;
  if (b < ids) {
    base[b] = begin;
    length[b] = total;
    if (id < a.vocab) a.total[id] = total;
  }
  if (me == mask && b == kSortThreads - 1) a.total[a.vocab] = begin + total;   // the last residue's end
  __syncthreads();
  for (int64_t t = t0; t < t1; t += kBatch * 32) {
    if (seg > kBatch * 32) read(t, false);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int k = bin[j];
      const uint32_t in = __ballot_sync(0xffffffffu, k >= 0);
      if (!in) continue;
      const uint32_t same = peers(k, in);
      if (k >= 0) {
        const int place = mine[k] + __popc(same & ((1u << lane) - 1u));
        a.sorted[base[k] + place] = make_int4((k << shift) + me, (int)(t + j * 32 + lane), place, length[k]);
      }
      __syncwarp();
      if (k >= 0 && lane == __ffs(same) - 1) mine[k] += (Cnt)__popc(same);
      __syncwarp();
    }
  }
}

// fp32 values that other SMs have written during this kernel: read from L2, not from this SM's L1.
template <int V>
__device__ __forceinline__ void load_cg(const float* p, float (&v)[V]) {
  if constexpr (V == 8) {
    const float4 a = __ldcg(reinterpret_cast<const float4*>(p)), b = __ldcg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    v[0] = __ldcg(p);
  }
}

// One lane's part of a warp's 256 columns: N accesses of V elements, 32 V apart.
template <int V>
struct Cols {
  static constexpr int N = kCols / 32 / V;
  int64_t c;       // first column
  int64_t dim;
  __device__ __forceinline__ bool ok(int j) const { return c + j * 32 * V < dim; }
  __device__ __forceinline__ int64_t at(int j) const { return c + j * 32 * V; }
};

template <int V, bool G_BF16>
__device__ __forceinline__ void write_grad(const EmbedGradArgs& a, int64_t id, const Cols<V>& w,
                                           const Raw<V, G_BF16> (&old)[Cols<V>::N], float (&sum)[Cols<V>::N][V]) {
#pragma unroll
  for (int j = 0; j < Cols<V>::N; ++j) {
    if (!w.ok(j)) continue;
    float o[V], v[V];
    if (a.accumulate) old[j].get(o);
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = a.accumulate ? o[e] + a.scale * sum[j][e] : a.scale * sum[j][e];
    store_v<V, G_BF16>(a.grad, id * a.grad_stride + w.at(j), v);
  }
}

// The sum of piece k of np of a run whose pieces' slots begin at `first` meets the others': true for
// the warp that has the run's sum in the end. Level by level, the last to finish of (up to) kFan
// neighbours adds them in order, into the first one's slot. Counters: of a group of several, the
// slot of its first member plus the level, which lies within the group.
template <int V>
__device__ __forceinline__ bool join_pieces(const EmbedGradArgs& a, const Cols<V>& w, int64_t first, int k, int np, int slice,
                                            int slices, int lane, float (&sum)[Cols<V>::N][V]) {
  constexpr int N = Cols<V>::N, kAtOnce = V == 8 ? 4 : 2;
  int64_t stride = 1;
  for (int level = 0; np > 1; ++level) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (w.ok(j)) store_v<V, false>(a.partial, (first + k * stride) * a.dim + w.at(j), sum[j]);
    const int group = k / kFan, members = min(kFan, np - group * kFan);
    if (members > 1) {
      __threadfence();
      __syncwarp();
      int done = 0;
      if (lane == 0) done = atomicAdd(a.count + (first + group * kFan * stride + level) * slices + slice, 1);
      if (__shfl_sync(0xffffffffu, done, 0) != members - 1) return false;
      __threadfence();
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[j][e] = 0.0f;
      for (int m = 0; m < members; m += kAtOnce) {
        float v[kAtOnce][N][V];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (m + u < members && w.ok(j)) load_cg<V>(a.partial + (first + (group * kFan + m + u) * stride) * a.dim + w.at(j), v[u][j]);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (m + u < members && w.ok(j)) {
#pragma unroll
              for (int e = 0; e < V; ++e) sum[j][e] += v[u][j][e];
            }
      }
    }
    k = group;
    np = (np + kFan - 1) / kFan;
    stride *= kFan;
  }
  return true;
}

// `sums` blocks of eight warps, a window and a slice of the columns each, spread evenly among the
// blocks that write zeros (none when accumulating): the sums wait on memory latency while the zeros
// fill its bandwidth.
template <int V, bool D_BF16, bool G_BF16>
__global__ void __launch_bounds__(kThreads, V == 8 ? 3 : 2) embed_sum_kernel(EmbedGradArgs a, int64_t sums, int64_t fills, int slices) {
  constexpr int N = Cols<V>::N, kAhead = V == 8 ? 4 : 2;
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t blk = blockIdx.x, all = sums + fills;
  const int64_t before = blk * sums / all;     // sums blocks among the blocks before this one
  if ((blk + 1) * sums / all == before) {
    const int64_t v0 = (blk - before) * kFillRows + warp * (kFillRows / 8);
    const bool mine = lane < kFillRows / 8 && v0 + lane < a.vocab;
    const uint32_t absent = __ballot_sync(0xffffffffu, mine && a.total[mine ? v0 + lane : 0] == 0);
    constexpr int kSize = G_BF16 ? 2 : 4, kPer = 16 / kSize;
    for (int r = 0; r < kFillRows / 8; ++r) {
      if (!(absent >> r & 1u)) continue;
      // 16 bytes at a time between the row's ends
      char* const row = static_cast<char*>(a.grad) + (v0 + r) * a.grad_stride * kSize;
      const int64_t before = min(a.dim, (int64_t)(-(uintptr_t)row % 16 / kSize)), whole = (a.dim - before) / kPer;
      uint4* const middle = reinterpret_cast<uint4*>(row + before * kSize);
#pragma unroll 4
      for (int64_t c = lane; c < whole; c += 32) middle[c] = make_uint4(0, 0, 0, 0);
      if (lane < before) store1<G_BF16>(row, lane, 0.0f);
      if (before + whole * kPer + lane < a.dim) store1<G_BF16>(row, before + whole * kPer + lane, 0.0f);
    }
    return;
  }
  // the places of the window and of the rows that its pieces may reach past it
  const int64_t item = before * (kThreads / 32) + warp, p0 = item / slices * kWindow;
  const int slice = (int)(item % slices);
  static_assert(kWindow + kLong - 1 <= 32, "a lane per place");
  int4 me = make_int4(0, 0, 0, 0);
  if (p0 + lane < a.n) me = a.sorted[p0 + lane];
  const int64_t valid = a.total[a.vocab];
  // the pieces that begin in this window: whole runs shorter than kLong, else every kPiece rows
  // (the last piece takes the rest, so that pieces of long runs are at least kPiece apart). One
  // follows the other, so their rows are the places from the first one's on.
  const int pieces = me.w < kLong ? 1 : me.w / kPiece;
  const bool head = lane < kWindow && p0 + lane < valid &&
                    (me.w < kLong ? me.z == 0 : me.z % kPiece == 0 && me.z / kPiece < pieces);
  const uint32_t heads = __ballot_sync(0xffffffffu, head);
  if (!heads) return;
  const int rows = pieces == 1 ? me.w : (me.z / kPiece == pieces - 1 ? me.w - me.z : kPiece);   // at most 15
  const uint32_t ends = __reduce_or_sync(0xffffffffu, head ? 1u << (lane + rows - 1) : 0u);
  const int stop = 32 - __clz(ends);
  const Cols<V> w = {(int64_t)slice * kCols + lane * V, a.dim};
  float sum[N][V];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) sum[j][e] = 0.0f;
  for (int i0 = __ffs(heads) - 1; i0 < stop; i0 += kAhead) {
    Raw<V, D_BF16> v[kAhead][N];
    Raw<V, G_BF16> old[kAhead][N];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= stop) break;
      const int64_t row = (int64_t)__shfl_sync(0xffffffffu, me.y, i) * a.dy_stride;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (w.ok(j)) v[u][j].load(a.dy, row + w.at(j));
      if (a.accumulate && (ends >> i & 1)) {
        const int src = 31 - __clz(heads & (2u << min(i, kWindow - 1)) - 1u);
        const int id = __shfl_sync(0xffffffffu, me.x, src), np = __shfl_sync(0xffffffffu, pieces, src);
        if (np == 1) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (w.ok(j)) old[u][j].load(a.grad, id * a.grad_stride + w.at(j));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u;
      if (i >= stop) break;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (!w.ok(j)) continue;
        float f[V];
        v[u][j].get(f);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[j][e] += f[e];
      }
      if (!(ends >> i & 1)) continue;
      const int src = 31 - __clz(heads & (2u << min(i, kWindow - 1)) - 1u);
      const int id = __shfl_sync(0xffffffffu, me.x, src), np = __shfl_sync(0xffffffffu, pieces, src);
      if (np > 1) break;   // a long run's piece, which reaches past the window: the last one
      write_grad<V, G_BF16>(a, id, w, old[u], sum);
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) sum[j][e] = 0.0f;
    }
  }
  const uint32_t longs = __ballot_sync(0xffffffffu, head && pieces > 1);
  if (!longs) return;
  const int src = __ffs(longs) - 1;
  const int id = __shfl_sync(0xffffffffu, me.x, src), off = __shfl_sync(0xffffffffu, me.z, src);
  const int np = __shfl_sync(0xffffffffu, pieces, src);
  // slot p / kPiece: no other piece of a long run has it. The run's slots follow one another.
  if (!join_pieces<V>(a, w, (p0 + src - off) / kPiece, off / kPiece, np, slice, slices, lane, sum)) return;
  Raw<V, G_BF16> old[N];
  if (a.accumulate) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (w.ok(j)) old[j].load(a.grad, id * a.grad_stride + w.at(j));
  }
  write_grad<V, G_BF16>(a, id, w, old, sum);
}

bool aligned8(const void* p, int64_t stride) { return (uintptr_t)p % 16 == 0 && stride % 8 == 0; }

template <int V, bool T, bool O>
cudaError_t embed_ids(const EmbedArgs& a, int id64, cudaStream_t s) {
  const dim3 grid((unsigned)((a.n + kThreads / 32 - 1) / (kThreads / 32)),
                  (unsigned)((a.dim + kPart * 32 * V - 1) / (kPart * 32 * V)));   // at most 8192 parts
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

int slices_of(int64_t dim) { return (int)((dim + kCols - 1) / kCols); }

template <int V, bool D, bool G>
cudaError_t embed_sums(const EmbedGradArgs& a, int64_t* launches, cudaStream_t s) {
  const int64_t sums = ((a.n + kWindow - 1) / kWindow * slices_of(a.dim) + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t fills = a.accumulate ? 0 : (a.vocab + kFillRows - 1) / kFillRows;
  ++*launches;
  return launch_dependent(embed_sum_kernel<V, D, G>, dim3((unsigned)(sums + fills)), dim3(kThreads), 0, s, a, sums, fills,
                          slices_of(a.dim));
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
  const int64_t slots = (n + kPiece - 1) / kPiece;
  const int64_t total = up(n * 16), partial = total + up((vocab + 1) * 4), count = partial + up(slots * dim * 4);
  if (a) {
    a->sorted = reinterpret_cast<int4*>(base);
    a->total = reinterpret_cast<int*>(base + total);
    a->partial = reinterpret_cast<float*>(base + partial);
    a->count = reinterpret_cast<int*>(base + count);
  }
  return count + up(slots * slices_of(dim) * 4);
}

cudaError_t launch_embedding_grad(const EmbedGradArgs& a, int dy_bf16, int grad_bf16, int id64,
                                  int64_t* launches, cudaStream_t s) {
  // 128 residues (fewer for a small vocabulary, more where a residue would have over kSortIds ids)
  int shift = 0;
  while (shift < 7 && (a.vocab >> shift) > 64) ++shift;
  while (((a.vocab - 1) >> shift) + 1 > kSortIds) ++shift;
  const int ids = (int)(((a.vocab - 1) >> shift) + 1);
  const bool small = a.n < 65536;   // counts fit 16 bits
  const size_t smem = (size_t)kSortWarps * ids * (small ? 2 : 4) + 4;
  using Kernel = void (*)(EmbedGradArgs, int, int, int);
  const Kernel kernels[4] = {token_sort_kernel<false, int>, token_sort_kernel<false, uint16_t>,
                             token_sort_kernel<true, int>, token_sort_kernel<true, uint16_t>};
  static PerDeviceOnce once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = (cudaError_t)once.run(dev, [&] {
    for (const Kernel k : kernels) {
      const cudaError_t r = cudaFuncSetAttribute((const void*)k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kSortWarps * kSortIds * 4 + 4);
      if (r != cudaSuccess) return (int)r;
    }
    return 0;
  });
  if (e != cudaSuccess) return e;
  kernels[(id64 ? 2 : 0) + (small ? 1 : 0)]<<<1u << shift, kSortThreads, smem, s>>>(a, ids, shift, slices_of(a.dim));
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  ++*launches;
  if (a.dim % 8 == 0 && aligned8(a.dy, a.dy_stride) && aligned8(a.grad, a.grad_stride))
    return embed_grad_types<8>(a, dy_bf16, grad_bf16, launches, s);
  return embed_grad_types<1>(a, dy_bf16, grad_bf16, launches, s);
}

}  // namespace muon
