// C entry points of the operators that make the optimizer's gradients: argument checks, then the
// launches (embedding.cu, rmsnorm.cu, checkpoint.cu, weight_grad.cu). They keep no state between
// calls and allocate nothing: workspaces are the caller's.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <string>

#include "../../include/muon.h"
#include "ops_internal.h"

namespace muon {
namespace {

int refuse(const char* msg) {
  set_error_message(msg);
  return MUON_ERR_INVALID_ARG;
}

int finish(cudaError_t e, const char* what, int64_t launches) {
  note_launches(launches);
  if (e == cudaSuccess) return MUON_OK;
  set_error_message(std::string(what) + ": " + cudaGetErrorString(e));
  return MUON_ERR_CUDA;
}

bool is_dtype(int t) { return t == MUON_BF16 || t == MUON_FP32; }
int64_t size_of(int t) { return t == MUON_BF16 ? 2 : 4; }

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxStride = int64_t(1) << 31;

// A row-major matrix: rows of `row_bytes` bytes, `stride` bytes apart.
struct Block {
  uintptr_t p;
  int64_t rows, row_bytes, stride;
  Block(const void* ptr, int64_t rows_, int64_t cols, int64_t stride_elems, int64_t elem)
      : p((uintptr_t)ptr), rows(rows_), row_bytes(cols * elem), stride(stride_elems * elem) {}
  uintptr_t end() const { return p + (uintptr_t)((rows - 1) * stride + row_bytes); }
};

// Whether two matrices share bytes (column ranges side by side in rows of one stride do not).
bool share(const Block& a, const Block& b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.row_bytes <= 0 || b.row_bytes <= 0) return false;
  if (a.end() <= b.p || b.end() <= a.p) return false;
  if (a.stride == b.stride && a.stride > 0) {
    const int64_t s = a.stride;
    const int64_t off = (int64_t)(((int64_t)(b.p - a.p) % s + s) % s);
    if (off >= a.row_bytes && off + b.row_bytes <= s) return false;
  }
  return true;
}

bool same(const Block& a, const Block& b) {
  return a.p == b.p && a.stride == b.stride && a.row_bytes == b.row_bytes;
}

const char* check_matrix(const void* p, int64_t rows, int64_t cols, int64_t stride, int dtype, const char* missing,
                         const char* bad_stride) {
  if (rows > 0 && !p) return missing;
  if (stride < cols || stride > kMaxStride) return bad_stride;
  if ((uintptr_t)p % (uintptr_t)size_of(dtype)) return "a pointer is not aligned to its element type";
  return nullptr;
}

#define REFUSE_IF(cond, msg) \
  do {                       \
    if (cond) return refuse(msg); \
  } while (0)
#define CHECK_MATRIX(name, p, rows, cols, stride, dtype)                                                \
  do {                                                                                                  \
    if (const char* m_ = check_matrix(p, rows, cols, stride, dtype, name " must not be NULL",           \
                                      name " row stride must be at least its row length (and <= 2^31)")) \
      return refuse(m_);                                                                                \
  } while (0)

int check_tokens(const void* tokens, int token_bits, int64_t n) {
  if (token_bits != 32 && token_bits != 64) return refuse("token_bits must be 32 or 64");
  if (n < 0 || n > kMaxRows) return refuse("n must be in [0, 2^31)");
  if (n > 0 && !tokens) return refuse("tokens must not be NULL");
  if ((uintptr_t)tokens % (token_bits / 8)) return refuse("tokens must be aligned to their type");
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

int muon_embedding(const void* tokens, int token_bits, int64_t n, const void* table, muon_dtype_t table_dtype,
                   int64_t table_stride, int64_t vocab, int64_t dim, float scale, void* out, muon_dtype_t out_dtype,
                   int64_t out_stride, muon_stream_t stream) {
  set_error_message("");
  if (int rc = check_tokens(tokens, token_bits, n)) return rc;
  REFUSE_IF(!is_dtype(table_dtype), "table_dtype");
  REFUSE_IF(!is_dtype(out_dtype), "out_dtype");
  REFUSE_IF(vocab < 1 || vocab > kMaxRows, "vocab must be in [1, 2^31)");
  REFUSE_IF(dim < 1 || dim > kMaxDim, "dim must be in [1, 2^20]");
  REFUSE_IF(!isfinite(scale), "scale must be finite");
  CHECK_MATRIX("table", table, vocab, dim, table_stride, table_dtype);
  CHECK_MATRIX("out", out, n, dim, out_stride, out_dtype);
  const Block o(out, n, dim, out_stride, size_of(out_dtype));
  REFUSE_IF(share(o, Block(table, vocab, dim, table_stride, size_of(table_dtype))) ||
                share(o, Block(tokens, 1, n, n, token_bits / 8)),
            "out overlaps an input");
  if (n == 0) return MUON_OK;
  EmbedArgs a = {};
  if (int rc = current_device_info(nullptr, &a.status, nullptr)) return rc;
  a.table = table;
  a.tokens = tokens;
  a.out = out;
  a.n = n;
  a.vocab = vocab;
  a.dim = dim;
  a.table_stride = table_stride;
  a.out_stride = out_stride;
  a.scale = scale;
  return finish(launch_embedding(a, table_dtype == MUON_BF16, out_dtype == MUON_BF16, token_bits == 64,
                                 reinterpret_cast<cudaStream_t>(stream)),
                "embedding launch", 1);
}

int64_t muon_embedding_grad_workspace(int64_t n, int64_t vocab, int64_t dim) {
  set_error_message("");
  if (n < 0 || n > kMaxRows || vocab < 1 || vocab > kMaxRows || dim < 1 || dim > kMaxDim)
    return refuse("n must be in [0, 2^31), vocab in [1, 2^31), dim in [1, 2^20]");
  return embed_grad_workspace(n, vocab, dim, nullptr, nullptr);
}

int muon_embedding_grad(const void* tokens, int token_bits, int64_t n, const void* dy, muon_dtype_t dy_dtype,
                        int64_t dy_stride, int64_t vocab, int64_t dim, float scale, void* grad, muon_dtype_t grad_dtype,
                        int64_t grad_stride, int accumulate, void* workspace, int64_t workspace_bytes,
                        muon_stream_t stream) {
  set_error_message("");
  if (int rc = check_tokens(tokens, token_bits, n)) return rc;
  REFUSE_IF(!is_dtype(dy_dtype), "dy_dtype");
  REFUSE_IF(!is_dtype(grad_dtype), "grad_dtype");
  REFUSE_IF(vocab < 1 || vocab > kMaxRows, "vocab must be in [1, 2^31)");
  REFUSE_IF(dim < 1 || dim > kMaxDim, "dim must be in [1, 2^20]");
  REFUSE_IF(!isfinite(scale), "scale must be finite");
  CHECK_MATRIX("dy", dy, n, dim, dy_stride, dy_dtype);
  CHECK_MATRIX("grad", grad, vocab, dim, grad_stride, grad_dtype);
  const int64_t need = embed_grad_workspace(n, vocab, dim, nullptr, nullptr);
  REFUSE_IF(!workspace || (uintptr_t)workspace % 256, "workspace must not be NULL and must be 256-byte aligned");
  REFUSE_IF(workspace_bytes < need, "workspace_bytes is less than muon_embedding_grad_workspace");
  const Block g(grad, vocab, dim, grad_stride, size_of(grad_dtype)), w(workspace, 1, need, need, 1);
  const Block d(dy, n, dim, dy_stride, size_of(dy_dtype)), t(tokens, 1, n, n, token_bits / 8);
  REFUSE_IF(share(g, d) || share(g, t) || share(w, g) || share(w, d) || share(w, t),
            "grad or the workspace overlaps another buffer");
  if (n == 0 && accumulate) return MUON_OK;
  EmbedGradArgs a = {};
  if (int rc = current_device_info(nullptr, &a.status, nullptr)) return rc;
  a.tokens = tokens;
  a.dy = dy;
  a.grad = grad;
  a.n = n;
  a.vocab = vocab;
  a.dim = dim;
  a.dy_stride = dy_stride;
  a.grad_stride = grad_stride;
  a.scale = scale;
  a.accumulate = accumulate != 0;
  embed_grad_workspace(n, vocab, dim, &a, static_cast<char*>(workspace));
  int64_t launches = 0;
  const cudaError_t e = launch_embedding_grad(a, dy_dtype == MUON_BF16, grad_dtype == MUON_BF16, token_bits == 64,
                                              &launches, reinterpret_cast<cudaStream_t>(stream));
  return finish(e, "embedding gradient launch", launches);
}

int muon_rms_norm(const void* x, muon_dtype_t x_dtype, int64_t x_stride, const void* residual, muon_dtype_t r_dtype,
                  int64_t r_stride, const void* weight, muon_dtype_t w_dtype, int64_t rows, int64_t dim, float eps,
                  void* h, int64_t h_stride, void* y, int64_t y_stride, void* codes, int64_t codes_stride, void* scales,
                  int64_t scales_stride, float* rstd, muon_stream_t stream) {
  set_error_message("");
  REFUSE_IF(!is_dtype(x_dtype), "x_dtype");
  REFUSE_IF(!is_dtype(w_dtype), "w_dtype");
  REFUSE_IF(residual && !is_dtype(r_dtype), "r_dtype");
  REFUSE_IF(rows < 0 || rows > kMaxRows, "rows must be in [0, 2^31)");
  REFUSE_IF(dim < 1 || dim > kNormMaxDim, "dim must be in [1, 32768]");
  REFUSE_IF(!(eps >= 0.0f) || !isfinite(eps), "eps must be finite and >= 0");
  REFUSE_IF(!residual != !h, "h and residual go together");
  REFUSE_IF(!codes != !scales, "codes and scales go together");
  if (rows == 0) return MUON_OK;
  REFUSE_IF(!y && !codes, "y, codes or both must be given");
  const int64_t xb = size_of(x_dtype), rb = size_of(r_dtype), blocks = (dim + 31) / 32;
  CHECK_MATRIX("x", x, rows, dim, x_stride, x_dtype);
  CHECK_MATRIX("weight", weight, 1, dim, dim, w_dtype);
  if (residual) CHECK_MATRIX("residual", residual, rows, dim, r_stride, r_dtype);
  if (residual) CHECK_MATRIX("h", h, rows, dim, h_stride, r_dtype);
  if (y) CHECK_MATRIX("y", y, rows, dim, y_stride, x_dtype);
  REFUSE_IF(codes && (codes_stride < dim || codes_stride > kMaxStride), "codes row stride must be at least dim (and <= 2^31)");
  REFUSE_IF(codes && (scales_stride < blocks || scales_stride > kMaxStride),
            "scales row stride must be at least ceil(dim / 32) (and <= 2^31)");
  REFUSE_IF(!rstd || (uintptr_t)rstd % 4, "rstd must not be NULL");
  const Block X(x, rows, dim, x_stride, xb), R(residual, rows, dim, r_stride, rb), W(weight, 1, dim, dim, size_of(w_dtype));
  const Block H(h, rows, dim, h_stride, rb), Y(y, rows, dim, y_stride, xb), Q(codes, rows, dim, codes_stride, 1);
  const Block S(scales, rows, blocks, scales_stride, 1), T(rstd, 1, rows, rows, 4);
  REFUSE_IF((share(H, X) && !same(H, X)) || (share(H, R) && !same(H, R)) || share(H, W), "h overlaps an input");
  REFUSE_IF((share(Y, X) && !same(Y, X)) || share(Y, R) || share(Y, W) || share(Y, H), "y overlaps another buffer");
  REFUSE_IF(share(Q, X) || share(Q, R) || share(Q, W) || share(Q, H) || share(Q, Y), "codes overlap another buffer");
  REFUSE_IF(share(S, X) || share(S, R) || share(S, W) || share(S, H) || share(S, Y) || share(S, Q),
            "scales overlap another buffer");
  REFUSE_IF(share(T, X) || share(T, R) || share(T, W) || share(T, H) || share(T, Y) || share(T, Q) || share(T, S),
            "rstd overlaps another buffer");
  NormArgs a = {};
  int sms = 0;
  if (int rc = current_device_info(&sms, &a.status, &a.wait_ns)) return rc;
  a.x = x;
  a.r = residual;
  a.w = weight;
  a.h = h;
  a.y = y;
  a.q = static_cast<uint8_t*>(codes);
  a.sc = static_cast<uint8_t*>(scales);
  a.rstd = rstd;
  a.rows = rows;
  a.dim = dim;
  a.xs = x_stride;
  a.rs = r_stride;
  a.hs = h_stride;
  a.ys = y_stride;
  a.qs = codes_stride;
  a.scs = scales_stride;
  a.eps = eps;
  a.w_bf16 = w_dtype == MUON_BF16;
  return finish(launch_rms_norm(a, x_dtype == MUON_BF16, residual ? r_dtype == MUON_BF16 : x_dtype == MUON_BF16, sms,
                                reinterpret_cast<cudaStream_t>(stream)),
                "rms_norm launch", 1);
}

int64_t muon_rms_norm_grad_workspace(int64_t rows, int64_t dim) {
  set_error_message("");
  if (rows < 0 || rows > kMaxRows || dim < 1 || dim > kNormMaxDim)
    return refuse("rows must be in [0, 2^31), dim in [1, 32768]");
  return norm_grad_workspace(rows, dim);
}

int muon_rms_norm_grad(const void* dy, muon_dtype_t dy_dtype, int64_t dy_stride, const void* h, muon_dtype_t h_dtype,
                       int64_t h_stride, const void* weight, muon_dtype_t w_dtype, const float* rstd, const void* dh,
                       int64_t dh_stride, int64_t rows, int64_t dim, void* dx, int64_t dx_stride, float* dweight,
                       int accumulate, void* workspace, int64_t workspace_bytes, muon_stream_t stream) {
  set_error_message("");
  REFUSE_IF(!is_dtype(dy_dtype), "dy_dtype");
  REFUSE_IF(!is_dtype(h_dtype), "h_dtype");
  REFUSE_IF(!is_dtype(w_dtype), "w_dtype");
  REFUSE_IF(rows < 0 || rows > kMaxRows, "rows must be in [0, 2^31)");
  REFUSE_IF(dim < 1 || dim > kNormMaxDim, "dim must be in [1, 32768]");
  CHECK_MATRIX("dweight", dweight, 1, dim, dim, MUON_FP32);
  const int64_t hb = size_of(h_dtype), db = size_of(dy_dtype), need = norm_grad_workspace(rows, dim);
  if (rows > 0) {
    CHECK_MATRIX("dy", dy, rows, dim, dy_stride, dy_dtype);
    CHECK_MATRIX("h", h, rows, dim, h_stride, h_dtype);
    CHECK_MATRIX("weight", weight, 1, dim, dim, w_dtype);
    CHECK_MATRIX("rstd", rstd, 1, rows, rows, MUON_FP32);
    if (dh) CHECK_MATRIX("dh", dh, rows, dim, dh_stride, h_dtype);
    CHECK_MATRIX("dx", dx, rows, dim, dx_stride, h_dtype);
    REFUSE_IF(!workspace || (uintptr_t)workspace % 256, "workspace must not be NULL and must be 256-byte aligned");
    REFUSE_IF(workspace_bytes < need, "workspace_bytes is less than muon_rms_norm_grad_workspace");
    const Block D(dy, rows, dim, dy_stride, db), H(h, rows, dim, h_stride, hb), G(dh, rows, dim, dh_stride, hb);
    const Block X(dx, rows, dim, dx_stride, hb), W(weight, 1, dim, dim, size_of(w_dtype)), T(rstd, 1, rows, rows, 4);
    const Block DW(dweight, 1, dim, dim, 4), B(workspace, 1, need, need, 1);
    REFUSE_IF((share(X, D) && !same(X, D)) || (share(X, H) && !same(X, H)) || (share(X, G) && !same(X, G)) ||
                  share(X, W) || share(X, T),
              "dx overlaps an input");
    REFUSE_IF(share(DW, D) || share(DW, H) || share(DW, G) || share(DW, W) || share(DW, T) || share(DW, X),
              "dweight overlaps another buffer");
    REFUSE_IF(share(B, D) || share(B, H) || share(B, G) || share(B, W) || share(B, T) || share(B, X) || share(B, DW),
              "the workspace overlaps another buffer");
  } else if (accumulate) {
    return MUON_OK;
  }
  NormGradArgs a = {};
  if (int rc = current_device_info(nullptr, &a.status, &a.wait_ns)) return rc;
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.rstd = rstd;
  a.dh = dh;
  a.dx = dx;
  a.dw = dweight;
  a.rows = rows;
  a.dim = dim;
  a.dys = dy_stride;
  a.hs = h_stride;
  a.dhs = dh_stride;
  a.dxs = dx_stride;
  a.w_bf16 = w_dtype == MUON_BF16;
  a.accumulate = accumulate != 0;
  a.partial = static_cast<float*>(workspace);
  int64_t launches = 0;
  const cudaError_t e = launch_rms_norm_grad(a, dy_dtype == MUON_BF16, h_dtype == MUON_BF16, &launches,
                                             reinterpret_cast<cudaStream_t>(stream));
  return finish(e, "rms_norm gradient launch", launches);
}

static int check_mx(const void* x, int dtype, int64_t stride, int64_t rows, int64_t dim, const void* codes,
                    int64_t codes_stride, const void* scales, int64_t scales_stride, const char* name) {
  const int64_t blocks = (dim + 31) / 32;
  if (!is_dtype(dtype)) return refuse("dtype");
  if (rows < 0 || rows > kMaxRows) return refuse("rows must be in [0, 2^31)");
  if (dim < 1 || dim > kMaxDim) return refuse("dim must be in [1, 2^20]");
  if (rows == 0) return MUON_OK;
  if (!x) {
    set_error_message(std::string(name) + " must not be NULL");
    return MUON_ERR_INVALID_ARG;
  }
  if (const char* m = check_matrix(x, rows, dim, stride, dtype, "", "row stride must be at least dim (and <= 2^31)"))
    return refuse(m);
  if (!codes || !scales) return refuse("codes and scales must not be NULL");
  if (codes_stride < dim || codes_stride > kMaxStride) return refuse("codes row stride must be at least dim (and <= 2^31)");
  if (scales_stride < blocks || scales_stride > kMaxStride)
    return refuse("scales row stride must be at least ceil(dim / 32) (and <= 2^31)");
  const Block X(x, rows, dim, stride, size_of(dtype)), Q(codes, rows, dim, codes_stride, 1);
  const Block S(scales, rows, blocks, scales_stride, 1);
  if (share(X, Q) || share(X, S) || share(Q, S)) return refuse("buffers overlap");
  return MUON_OK;
}

int muon_checkpoint_store(const void* x, muon_dtype_t x_dtype, int64_t x_stride, int64_t rows, int64_t dim, void* codes,
                          int64_t codes_stride, void* scales, int64_t scales_stride, muon_stream_t stream) {
  set_error_message("");
  if (int rc = check_mx(x, x_dtype, x_stride, rows, dim, codes, codes_stride, scales, scales_stride, "x")) return rc;
  if (rows == 0) return MUON_OK;
  if (int rc = current_device_info(nullptr, nullptr, nullptr)) return rc;
  MxArgs a = {x, nullptr, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), rows, dim, x_stride, codes_stride,
              scales_stride};
  return finish(launch_mx_store(a, x_dtype == MUON_BF16, reinterpret_cast<cudaStream_t>(stream)),
                "checkpoint store launch", 1);
}

int muon_checkpoint_restore(const void* codes, int64_t codes_stride, const void* scales, int64_t scales_stride,
                            int64_t rows, int64_t dim, void* x, muon_dtype_t x_dtype, int64_t x_stride,
                            muon_stream_t stream) {
  set_error_message("");
  if (int rc = check_mx(x, x_dtype, x_stride, rows, dim, codes, codes_stride, scales, scales_stride, "x")) return rc;
  if (rows == 0) return MUON_OK;
  if (int rc = current_device_info(nullptr, nullptr, nullptr)) return rc;
  MxArgs a = {nullptr, x, static_cast<uint8_t*>(const_cast<void*>(codes)),
              static_cast<uint8_t*>(const_cast<void*>(scales)), rows, dim, x_stride, codes_stride, scales_stride};
  return finish(launch_mx_restore(a, x_dtype == MUON_BF16, reinterpret_cast<cudaStream_t>(stream)),
                "checkpoint restore launch", 1);
}

static const char* check_wgrad_sizes(int64_t rows, int64_t n, int64_t k, int dy_dtype) {
  if (!is_dtype(dy_dtype)) return "dy_dtype";
  if (rows < 0 || rows > (int64_t(1) << 29)) return "rows must be in [0, 2^29]";
  if (n < 1 || n > kMaxDim || k < 1 || k > kMaxDim) return "n and k must be in [1, 2^20]";
  return nullptr;
}

int64_t muon_weight_grad_workspace(int64_t rows, int64_t n, int64_t k, muon_dtype_t dy_dtype) {
  set_error_message("");
  if (const char* m = check_wgrad_sizes(rows, n, k, dy_dtype)) return refuse(m);
  return wgrad_workspace(rows, n, k, dy_dtype == MUON_BF16);
}

int muon_weight_grad(const void* dy, muon_dtype_t dy_dtype, int64_t dy_stride, const void* codes, int64_t codes_stride,
                     const void* scales, int64_t scales_stride, int64_t rows, int64_t n, int64_t k, void* grad,
                     muon_dtype_t grad_dtype, int64_t grad_stride, int accumulate, void* workspace,
                     int64_t workspace_bytes, muon_stream_t stream) {
  set_error_message("");
  if (const char* m = check_wgrad_sizes(rows, n, k, dy_dtype)) return refuse(m);
  REFUSE_IF(!is_dtype(grad_dtype), "grad_dtype");
  CHECK_MATRIX("dy", dy, rows, n, dy_stride, dy_dtype);
  CHECK_MATRIX("grad", grad, n, k, grad_stride, grad_dtype);
  const int64_t blocks = (k + 31) / 32;
  REFUSE_IF(rows > 0 && (!codes || !scales), "codes and scales must not be NULL");
  REFUSE_IF(codes_stride < k || codes_stride > kMaxStride, "codes row stride must be at least k (and <= 2^31)");
  REFUSE_IF(scales_stride < blocks || scales_stride > kMaxStride,
            "scales row stride must be at least ceil(k / 32) (and <= 2^31)");
  const int64_t need = wgrad_workspace(rows, n, k, dy_dtype == MUON_BF16);
  REFUSE_IF(need > 0 && (!workspace || (uintptr_t)workspace % 256),
            "workspace must not be NULL and must be 256-byte aligned");
  REFUSE_IF(workspace_bytes < need, "workspace_bytes is less than muon_weight_grad_workspace");
  const Block D(dy, rows, n, dy_stride, size_of(dy_dtype)), Q(codes, rows, k, codes_stride, 1);
  const Block S(scales, rows, blocks, scales_stride, 1), G(grad, n, k, grad_stride, size_of(grad_dtype));
  const Block B(workspace, 1, need, need, 1);
  REFUSE_IF(share(G, D) || share(G, Q) || share(G, S) || share(B, G) || share(B, D) || share(B, Q) || share(B, S),
            "grad or the workspace overlaps another buffer");
  if (rows == 0 && accumulate) return MUON_OK;
  WgradArgs a = {};
  int sms = 0;
  if (int rc = current_device_info(&sms, &a.status, &a.wait_ns)) return rc;
  a.dy = dy;
  a.q = static_cast<const uint8_t*>(codes);
  a.sc = static_cast<const uint8_t*>(scales);
  a.grad = grad;
  a.rows = rows;
  a.n = n;
  a.k = k;
  a.dys = dy_stride;
  a.qs = codes_stride;
  a.scs = scales_stride;
  a.gs = grad_stride;
  a.accumulate = accumulate != 0;
  int64_t launches = 0;
  const cudaError_t e = launch_wgrad(a, dy_dtype == MUON_BF16, grad_dtype == MUON_BF16, sms, static_cast<char*>(workspace),
                                     &launches, reinterpret_cast<cudaStream_t>(stream));
  return finish(e, "weight gradient launch", launches);
}

}  // extern "C"
