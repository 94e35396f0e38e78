// Argument records and launchers of the operators that make the optimizer's gradients (embedding,
// RMS norm, 8-bit activation checkpoints, weight gradient). Row strides are in elements.
#pragma once

#include <cuda_runtime.h>

#include <string>
#include <stdint.h>

namespace muon {

// ---- embedding
struct EmbedArgs {
  const void* table;
  const void* tokens;
  void* out;
  int64_t n, vocab, dim, table_stride, out_stride;
  float scale;
  int* status;
};
cudaError_t launch_embedding(const EmbedArgs& a, int table_bf16, int out_bf16, int id64, cudaStream_t s);

struct EmbedGradArgs {
  const void* tokens;
  const void* dy;
  void* grad;
  int64_t n, vocab, dim, dy_stride, grad_stride;
  float scale;
  int accumulate;
  int* status;
  // workspace
  int4* sorted;    // [n] tokens grouped by id: id, position, place in the run of the id, length of the run
  int* total;      // [vocab + 1] tokens of each id; total[vocab] = tokens in all
  float* partial;  // [ceil(n / 8)][dim] sums of the pieces of long runs
  int* count;      // [ceil(n / 8)][slices] finished sums of each group of pieces
};
int64_t embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim, EmbedGradArgs* a, char* base);
cudaError_t launch_embedding_grad(const EmbedGradArgs& a, int dy_bf16, int grad_bf16, int id64,
                                  int64_t* launches, cudaStream_t s);

// ---- RMS norm
constexpr int64_t kNormMaxDim = 32768;
struct NormArgs {
  const void* x;
  const void* r;        // residual, or NULL
  const void* w;
  void* h;              // x + r in r's type (NULL when r is)
  void* y;              // x's type, or NULL
  uint8_t* q;           // e4m3 codes, or NULL
  uint8_t* sc;          // e8m0 codes
  float* rstd;
  int64_t rows, dim, xs, rs, hs, ys, qs, scs;
  float eps;
  int w_bf16;
  int* status;
  uint64_t wait_ns;
};
cudaError_t launch_rms_norm(const NormArgs& a, int x_bf16, int r_bf16, int sms, cudaStream_t s);

struct NormGradArgs {
  const void* dy;
  const void* h;
  const void* w;
  const float* rstd;
  const void* dh;       // h's type, or NULL
  void* dx;             // h's type
  float* dw;
  int64_t rows, dim, dys, hs, dhs, dxs;
  int w_bf16, accumulate;
  float* partial;       // workspace: [blocks][dim]
  int* status;
  uint64_t wait_ns;
};
int64_t norm_grad_workspace(int64_t rows, int64_t dim);
cudaError_t launch_rms_norm_grad(const NormGradArgs& a, int dy_bf16, int h_bf16, int64_t* launches,
                                 cudaStream_t s);

// ---- 8-bit activation checkpoints
struct MxArgs {
  const void* x;        // store: input
  void* out;            // restore: output
  uint8_t* q;
  uint8_t* sc;
  int64_t rows, dim, xs, qs, scs;
  uint32_t* zero;       // restore: `zeros` words that the first block also sets to 0
  int zeros;
};
cudaError_t launch_mx_store(const MxArgs& a, int x_bf16, cudaStream_t s);
cudaError_t launch_mx_restore(const MxArgs& a, int out_bf16, cudaStream_t s);

// ---- weight gradient
struct WgradArgs {
  const void* dy;
  const uint8_t* q;
  const uint8_t* sc;
  void* grad;
  int64_t rows, n, k, dys, qs, scs, gs;
  int accumulate;
  int* status;
  uint64_t wait_ns;
};
int64_t wgrad_workspace(int64_t rows, int64_t n, int64_t k, int dy_bf16);
cudaError_t launch_wgrad(const WgradArgs& a, int dy_bf16, int grad_bf16, int sms, char* ws, int64_t* launches,
                         cudaStream_t s);

// ---- launch with programmatic stream serialization: the kernel may be scheduled before the one
// before it has finished, and itself waits for it (grid_dependency_wait) before it touches memory.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ---- hooks of the main file: the calling thread's error message, the launch count, and the
// current device's record (sm count, status word, wait limit; any pointer may be NULL; fails off
// sm_100). Workspace sizes and splits go by kSms, not by the device, so that they can be asked for
// anywhere.
constexpr int kSms = 148;
void set_error_message(const std::string& msg);
void note_launches(int64_t n);
int current_device_info(int* sms, int** status, uint64_t* wait_ns);

}  // namespace muon
