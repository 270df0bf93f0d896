// mxg_api.cu -- the C ABI declared in include/mxg.h: argument validation,
// device checks and kernel dispatch.  Host code only; no allocation, no
// synchronisation.
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <mutex>

#include "mxg_device.cuh"

namespace mxg {
cudaError_t launch_group_offsets(const void* sizes, int is_int64, int G, int64_t mult,
                                 int64_t last_dim, int64_t cap, int64_t* ws, int32_t* status,
                                 cudaStream_t stream, int round128);
cudaError_t launch_mxfp8_quantize(bool row, bool col, const uint16_t* x, int64_t cap, int64_t cols,
                                  const int64_t* group_ws, int G, uint8_t* q_row, uint8_t* sf_row,
                                  uint8_t* q_col, uint8_t* sf_col, int32_t* status, int num_sms,
                                  cudaStream_t stream, bool unaligned);
cudaError_t launch_nvfp4_quantize(const uint16_t* x, int64_t cap, int64_t cols,
                                  const int64_t* group_ws, int G, uint8_t* q, uint8_t* sf,
                                  float* outer, int32_t* status, int num_sms, cudaStream_t stream);
cudaError_t launch_nvfp4_quantize_colwise(const uint16_t* x, int64_t cap, int64_t cols,
                                          const int64_t* group_ws, int G, uint8_t* qT,
                                          uint8_t* sfT, float* outer, int num_sms,
                                          cudaStream_t stream);
cudaError_t launch_dequantize(int nvfp4, int colwise, const uint8_t* q, const uint8_t* sf,
                              const float* outer, int64_t rows, int64_t cols, void* out, int bf16,
                              int num_sms, cudaStream_t stream);
cudaError_t launch_grouped_gemm(bool nvfp4, int mode, const void* a_data, const uint8_t* a_sf,
                                const float* a_outer, const void* b_data, const uint8_t* b_sf,
                                const float* b_outer, const int64_t* group_ws, int G, int64_t M_cap,
                                int64_t N, int64_t K, const float* alpha, const float* beta,
                                const float* bias, void* C, int out_bf16, int32_t* status,
                                int num_sms, int tile_n, int stage_bytes, int inject,
                                uint64_t timeout_ns, int unaligned, int64_t a_ld_bytes,
                                int64_t b_ld_bytes, cudaStream_t stream);
cudaError_t launch_wgrad_no_rows(int G, int64_t N, int64_t K, const float* beta, void* C,
                                 int out_bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_grouped_gemm16(int in_f16, int mode, const void* A, int64_t lda, const void* B,
                                  int64_t ldb, const int64_t* group_ws, int G, int64_t M_cap,
                                  int64_t N, int64_t K, const float* alpha, const float* beta,
                                  void* C, int64_t ldc, int out_type, int32_t* status, int num_sms,
                                  cudaStream_t stream);
int64_t block_norm_ws_bytes(int64_t rows, int64_t cols);
cudaError_t launch_block_norm(const mxg_block_norm_t& p, int num_sms, cudaStream_t stream);
cudaError_t launch_block_norm_backward(const mxg_block_norm_grad_t& p, float* ws, int num_sms,
                                       cudaStream_t stream);
size_t grad_ws_bytes();
cudaError_t launch_grad_clip(const mxg_grad_t* grads, int n, bool clip, float max_norm,
                             float* norm, void* ws, int num_sms, cudaStream_t stream,
                             int* launches);
size_t route_ws_bytes(int64_t tokens, int experts, int k);
cudaError_t launch_route(const mxg_route_t& d, void* workspace, int32_t* status,
                         cudaStream_t stream, int* launches);
cudaError_t launch_route_rows(const int32_t* expert, int64_t tokens, int experts, int k, int align,
                              int64_t capacity, int64_t last_dim, int32_t* counts, int32_t* row_of,
                              int64_t* group_ws, void* workspace, int32_t* status,
                              cudaStream_t stream, int* launches);
cudaError_t launch_route_backward(const mxg_route_grad_t& d, int num_sms, cudaStream_t stream);
cudaError_t launch_expert_rows(const mxg_expert_rows_t& d, int op, int num_sms,
                               cudaStream_t stream);
cudaError_t launch_gated_act(const mxg_gated_act_t& d, bool backward, int num_sms,
                             cudaStream_t stream);
constexpr uint64_t kDefaultWaitNs = 1000000000ull;
}  // namespace mxg

namespace {

std::atomic<uint64_t> g_launches{0};

constexpr int kMaxDevices = 64;
struct DevInfo {
  int checked = 0;  // 0 unknown, 1 sm_103, -1 other
  int num_sms = 0;
};
DevInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Confirms the current device is sm_103 (GB300) and returns its SM count.
mxg_status_t current_device(int* num_sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices)
    return MXG_ERR_UNSUPPORTED_ARCH;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DevInfo& d = g_dev[dev];
  if (d.checked == 0) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return MXG_ERR_UNSUPPORTED_ARCH;
    d.checked = (major == 10 && minor == 3) ? 1 : -1;
    d.num_sms = sms;
  }
  if (d.checked != 1) return MXG_ERR_UNSUPPORTED_ARCH;
  *num_sms = d.num_sms;
  return MXG_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool mult128(int64_t v) { return v >= 0 && (v & 127) == 0; }

mxg_status_t launched(cudaError_t e, uint64_t n) {
  if (e != cudaSuccess) return MXG_ERR_LAUNCH;
  g_launches.fetch_add(n, std::memory_order_relaxed);
  return MXG_OK;
}

// The kernels index rows (and the padded rows of groups of any size) with
// 32-bit integers in their group tables.
constexpr int64_t kMaxRows = 0x7FFFFF80LL;
constexpr int64_t kMaxNormCols = 16384;  // of the norms around a block

// Arguments of the offsets entry points.  Bounds on the multiplier (2^31)
// and on the capacity (2^62, and capacity * last_dim within int64) keep every
// product the kernel forms -- sanitised rows times the multiplier, offsets
// times last_dim -- inside 64 bits.
bool offsets_args_ok(const void* sizes, const int64_t* ws, int G, int64_t multiplier,
                     int64_t last_dim, int64_t rows_capacity) {
  return sizes != nullptr && ws != nullptr && G >= 1 && G <= 65536 && multiplier >= 1 &&
         multiplier <= (1LL << 31) && last_dim >= 1 && rows_capacity >= 0 &&
         rows_capacity <= (1LL << 62) && rows_capacity <= INT64_MAX / last_dim;
}

// Checks an operand descriptor's rows / cols (0 = as the mode implies) and
// leading dimension (0 = dense) and returns the data's row stride in bytes.
mxg_status_t operand_shape(const mxg_operand_t* op, int64_t rows, int64_t cols, bool nvfp4,
                           int64_t* ld_bytes) {
  if ((op->rows != 0 && op->rows != rows) || (op->cols != 0 && op->cols != cols))
    return MXG_ERR_INVALID_ARG;
  const int64_t ld = op->ld == 0 ? cols : op->ld;
  if (ld < cols) return MXG_ERR_INVALID_ARG;
  if (nvfp4 && (ld & 1)) return MXG_ERR_ALIGNMENT;
  const int64_t bytes = nvfp4 ? ld / 2 : ld;
  if (bytes % 16 != 0) return MXG_ERR_ALIGNMENT;
  *ld_bytes = bytes;
  return MXG_OK;
}

// Bytes of an element, or 0 for a value that is no mxg_dtype_t.
size_t dtype_bytes(mxg_dtype_t t) {
  return t == MXG_F32 ? 4 : (t == MXG_BF16 || t == MXG_F16 ? 2 : 0);
}

bool aligned_to(const void* p, size_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// The fields that the norms around a block share, in both directions.
// Fills in the dense leading dimensions.
template <typename Desc>
mxg_status_t norm_common(Desc& d) {
  const size_t e = dtype_bytes(d.dtype), r = dtype_bytes(d.res_dtype);
  if (e == 0 || r == 0 || (d.res_dtype != d.dtype && d.res_dtype != MXG_F32))
    return MXG_ERR_INVALID_ARG;
  if (d.rows < 0 || d.rows > kMaxRows || d.cols < 1 || d.cols > kMaxNormCols)
    return MXG_ERR_INVALID_ARG;
  if (!(d.eps > 0.0f) || std::isinf(d.eps) || !std::isfinite(d.res_scale))
    return MXG_ERR_INVALID_ARG;
  if (d.gate_mode < MXG_GATE_NONE || d.gate_mode > MXG_GATE_FULL) return MXG_ERR_INVALID_ARG;
  if (d.gate_mode != MXG_GATE_NONE && d.rows != 0 && (d.gate == nullptr || d.y == nullptr))
    return MXG_ERR_INVALID_ARG;
  // the gradient of a COL gate's row sums reads the gate even without rows
  if (d.gate_mode == MXG_GATE_COL && d.gate == nullptr) return MXG_ERR_INVALID_ARG;
  if (d.ldx == 0) d.ldx = d.cols;
  if (d.ldy == 0) d.ldy = d.cols;
  if (d.ldg == 0) d.ldg = d.cols;
  if (d.ldx < d.cols || d.ldy < d.cols || d.ldg < d.cols) return MXG_ERR_INVALID_ARG;
  const size_t gate_bytes = d.gate_mode == MXG_GATE_ROW ? 4 : e;
  if (!aligned_to(d.x, r) || !aligned_to(d.y, e) || !aligned_to(d.w_post, e) ||
      !aligned_to(d.w_pre, e) || !aligned_to(d.gate, gate_bytes))
    return MXG_ERR_ALIGNMENT;
  return MXG_OK;
}

mxg_status_t grad_args(const mxg_grad_t* grads, int n, bool clip, const float* norm,
                       const void* workspace, size_t workspace_bytes) {
  if (n < 0 || (n > 0 && grads == nullptr) || norm == nullptr || workspace == nullptr)
    return MXG_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    const mxg_grad_t& t = grads[i];
    const size_t se = dtype_bytes(t.src_type), de = dtype_bytes(t.dst_type);
    if (se == 0 || t.numel < 0 || t.numel > (1LL << 40) || (t.numel > 0 && t.src == nullptr))
      return MXG_ERR_INVALID_ARG;
    if (clip && (de == 0 || (t.numel > 0 && t.dst == nullptr) ||
                 (t.dst == t.src && t.numel > 0 && t.dst_type != t.src_type)))
      return MXG_ERR_INVALID_ARG;
    if (!aligned_to(t.src, se) || (clip && !aligned_to(t.dst, de))) return MXG_ERR_ALIGNMENT;
  }
  if (!aligned_to(norm, 4) || !aligned16(workspace)) return MXG_ERR_ALIGNMENT;
  if (workspace_bytes < mxg::grad_ws_bytes()) return MXG_ERR_WORKSPACE_TOO_SMALL;
  return MXG_OK;
}

mxg_status_t grad_impl(const mxg_grad_t* grads, int n, bool clip, float max_norm, float* norm,
                       void* workspace, size_t workspace_bytes, mxg_stream_t stream) {
  mxg_status_t st = grad_args(grads, n, clip, norm, workspace, workspace_bytes);
  if (st != MXG_OK) return st;
  int sms = 0;
  if ((st = current_device(&sms)) != MXG_OK) return st;
  int launches = 0;
  const cudaError_t e =
      mxg::launch_grad_clip(grads, n, clip, max_norm, norm, workspace, sms,
                            reinterpret_cast<cudaStream_t>(stream), &launches);
  return launched(e, static_cast<uint64_t>(launches));
}

// Sizes of a routed batch.  The bounds keep every index of a choice or a row in 32 bits.
constexpr int kMaxExperts = 1024;
constexpr int kMaxChosen = 32;
constexpr int64_t kMaxRowCols = 1LL << 20;
constexpr int64_t kMaxLd = 1LL << 36;  // elements between rows

bool route_sizes_ok(int64_t tokens, int experts, int k) {
  return tokens >= 0 && tokens <= kMaxRows && experts >= 1 && experts <= kMaxExperts && k >= 1 &&
         k <= kMaxChosen && k <= experts && tokens * k <= kMaxRows;
}

// counts, and the rows where they are wanted.
mxg_status_t route_rows_args(int64_t tokens, const int32_t* counts, const int32_t* row_of,
                             const int64_t* group_ws, int align, int64_t rows_capacity,
                             int64_t last_dim) {
  if (counts == nullptr) return MXG_ERR_INVALID_ARG;
  if (align < 1 || align > 1024 || rows_capacity < 0 || rows_capacity > kMaxRows || last_dim < 1 ||
      (rows_capacity > 0 && last_dim > INT64_MAX / rows_capacity))
    return MXG_ERR_INVALID_ARG;
  if ((row_of != nullptr && group_ws == nullptr) ||
      (group_ws != nullptr && row_of == nullptr && tokens != 0))
    return MXG_ERR_INVALID_ARG;
  if (!aligned_to(counts, 4) || !aligned_to(row_of, 4) || !aligned_to(group_ws, 8))
    return MXG_ERR_ALIGNMENT;
  return MXG_OK;
}

// The workspace, and the word that a kernel's atomics may write.
mxg_status_t route_memory(int64_t tokens, int experts, int k, const void* workspace,
                          size_t workspace_bytes, const int32_t* dev_status) {
  if (workspace == nullptr) return MXG_ERR_INVALID_ARG;
  if (!aligned16(workspace) || !aligned_to(dev_status, 4)) return MXG_ERR_ALIGNMENT;
  return workspace_bytes < mxg::route_ws_bytes(tokens, experts, k) ? MXG_ERR_WORKSPACE_TOO_SMALL
                                                                   : MXG_OK;
}

// Checks a matrix's leading dimension, filling in a dense one.
bool fill_ld(int64_t* ld, int64_t cols) {
  if (*ld == 0) *ld = cols;
  return *ld >= cols && *ld <= kMaxLd;
}

// op: 0 dispatch, 1 combine, 2 its gradients.
mxg_status_t expert_rows_impl(const mxg_expert_rows_t* desc, int op, mxg_stream_t stream) {
  if (desc == nullptr) return MXG_ERR_INVALID_ARG;
  mxg_expert_rows_t d = *desc;
  const size_t size = dtype_bytes(d.dtype);
  if (size == 0 || d.n < 0 || d.n > kMaxRows || d.k < 1 || d.k > kMaxChosen ||
      d.n * d.k > kMaxRows || d.cols < 1 || d.cols > kMaxRowCols || d.rows_capacity < 0 ||
      d.rows_capacity > kMaxRows)
    return MXG_ERR_INVALID_ARG;
  const bool any = d.n != 0, rows = d.rows_capacity != 0;
  if (any && (d.tokens == nullptr || d.row_of == nullptr)) return MXG_ERR_INVALID_ARG;
  if (op != 2 && ((rows && d.rows == nullptr) || d.y_rows != nullptr || d.dweight != nullptr))
    return MXG_ERR_INVALID_ARG;
  if (op == 0 && d.weight != nullptr) return MXG_ERR_INVALID_ARG;
  if (op == 2 && any && ((d.dweight != nullptr && rows && d.y_rows == nullptr) ||
                         (d.dweight == nullptr && rows && d.rows == nullptr)))
    return MXG_ERR_INVALID_ARG;
  if (op == 2 && d.dweight == nullptr && d.y_rows != nullptr) return MXG_ERR_INVALID_ARG;
  // padding: all three or none
  const bool padded = d.counts != nullptr;
  if (padded != (d.group_ws != nullptr) || padded != (d.experts != 0) ||
      (padded && (op == 1 || d.experts < 1 || d.experts > kMaxExperts ||
                  (rows && d.rows == nullptr))))
    return MXG_ERR_INVALID_ARG;
  if (!fill_ld(&d.ldt, d.cols) || !fill_ld(&d.ldr, d.cols) || !fill_ld(&d.ldy, d.cols) ||
      (d.y_rows != nullptr && d.y_rows == d.rows && d.ldy != d.ldr))
    return MXG_ERR_INVALID_ARG;
  if (!aligned_to(d.tokens, size) || !aligned_to(d.rows, size) || !aligned_to(d.y_rows, size) ||
      !aligned_to(d.row_of, 4) || !aligned_to(d.weight, 4) || !aligned_to(d.dweight, 4) ||
      !aligned_to(d.counts, 4) || !aligned_to(d.group_ws, 8))
    return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  if (!rows) {  // nothing lies there
    d.rows = nullptr;
    d.y_rows = nullptr;
  }
  if (op == 1 ? !any : !any && !(padded && rows)) return MXG_OK;
  if (op == 0 && !rows) return MXG_OK;
  return launched(mxg::launch_expert_rows(d, op, sms, reinterpret_cast<cudaStream_t>(stream)), 1);
}

mxg_status_t gated_act_impl(const mxg_gated_act_t* desc, bool backward, mxg_stream_t stream) {
  if (desc == nullptr) return MXG_ERR_INVALID_ARG;
  mxg_gated_act_t d = *desc;
  if ((d.dtype != MXG_BF16 && d.dtype != MXG_F16) ||
      (d.act != MXG_ACT_SILU && d.act != MXG_ACT_GELU_TANH) || d.rows < 0 || d.rows > kMaxRows ||
      d.cols < 1 || d.cols > kMaxRowCols || (d.gated != 0 && d.gated != 1))
    return MXG_ERR_INVALID_ARG;
  if (d.G < 0 || d.G > kMaxExperts || (d.G != 0) != (d.group_ws != nullptr))
    return MXG_ERR_INVALID_ARG;
  const bool any = d.rows != 0;
  if (backward ? d.gate != nullptr || d.up != nullptr
               : d.dh != nullptr || d.dgate != nullptr || d.dup != nullptr)
    return MXG_ERR_INVALID_ARG;
  if (any) {
    if (backward && (d.q == nullptr || d.sf == nullptr || d.dh == nullptr || d.dgate == nullptr ||
                     (d.dup != nullptr) != (d.gated != 0)))
      return MXG_ERR_INVALID_ARG;
    if (!backward && (d.gate == nullptr || d.h == nullptr || (d.up != nullptr) != (d.gated != 0) ||
                      (d.q != nullptr) != (d.sf != nullptr)))
      return MXG_ERR_INVALID_ARG;
  }
  if (!fill_ld(&d.ldg, d.cols) || !fill_ld(&d.ldu, d.cols) || !fill_ld(&d.ldh, d.cols) ||
      !fill_ld(&d.ldq, d.cols * (1 + d.gated)) || !fill_ld(&d.lddh, d.cols) ||
      !fill_ld(&d.lddg, d.cols) || !fill_ld(&d.lddu, d.cols))
    return MXG_ERR_INVALID_ARG;
  // in place: the same element at the same time
  if (d.h != nullptr && ((d.h == d.gate && d.ldh != d.ldg) || (d.h == d.up && d.ldh != d.ldu)))
    return MXG_ERR_INVALID_ARG;
  if (d.dh != nullptr &&
      ((d.dh == d.dgate && d.lddh != d.lddg) || (d.dh == d.dup && d.lddh != d.lddu)))
    return MXG_ERR_INVALID_ARG;
  for (const void* p : {d.gate, d.up, static_cast<const void*>(d.h), d.dh,
                        static_cast<const void*>(d.dgate), static_cast<const void*>(d.dup)})
    if (!aligned_to(p, 2)) return MXG_ERR_ALIGNMENT;
  if (!aligned_to(d.group_ws, 8)) return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  if (!any) return MXG_OK;
  return launched(mxg::launch_gated_act(d, backward, sms, reinterpret_cast<cudaStream_t>(stream)),
                  1);
}

}  // namespace

extern "C" {

size_t mxg_offsets_workspace_bytes(int G) {
  return G < 1 ? 0 : static_cast<size_t>(2 * G + 1) * sizeof(int64_t);
}

mxg_status_t mxg_group_offsets(const void* sizes, int sizes_is_int64, int G, int64_t multiplier,
                               int64_t last_dim, int64_t rows_capacity, int64_t* ws,
                               int32_t* dev_status, mxg_stream_t stream) {
  if (!offsets_args_ok(sizes, ws, G, multiplier, last_dim, rows_capacity))
    return MXG_ERR_INVALID_ARG;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  return launched(mxg::launch_group_offsets(sizes, sizes_is_int64 ? 1 : 0, G, multiplier, last_dim,
                                            rows_capacity, ws, dev_status,
                                            reinterpret_cast<cudaStream_t>(stream), 1),
                  1);
}

mxg_status_t mxg_group_offsets_unaligned(const void* sizes, int sizes_is_int64, int G,
                                         int64_t multiplier, int64_t last_dim,
                                         int64_t rows_capacity, int64_t* ws, int32_t* dev_status,
                                         mxg_stream_t stream) {
  if (!offsets_args_ok(sizes, ws, G, multiplier, last_dim, rows_capacity))
    return MXG_ERR_INVALID_ARG;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  return launched(mxg::launch_group_offsets(sizes, sizes_is_int64 ? 1 : 0, G, multiplier, last_dim,
                                            rows_capacity, ws, dev_status,
                                            reinterpret_cast<cudaStream_t>(stream), 0),
                  1);
}

int64_t mxg_unaligned_rows_capacity(int64_t rows_capacity, int G) {
  if (rows_capacity < 0 || G < 1) return 0;
  return rows_capacity + 128 * static_cast<int64_t>(G);
}

mxg_status_t mxg_group_quantize_unaligned(mxg_qlayout_t layout, const void* x,
                                          int64_t rows_capacity, int64_t cols,
                                          const int64_t* group_ws, int G, uint8_t* q_row,
                                          uint8_t* sf_row, uint8_t* q_col, uint8_t* sf_col,
                                          int32_t* dev_status, mxg_stream_t stream) {
  if (x == nullptr || group_ws == nullptr || G < 1 || G > 1024) return MXG_ERR_INVALID_ARG;
  if (layout != MXG_ROWWISE && layout != MXG_COLWISE && layout != MXG_BOTH)
    return MXG_ERR_INVALID_ARG;
  const bool row = (layout & MXG_ROWWISE) != 0, col = (layout & MXG_COLWISE) != 0;
  if ((row && (q_row == nullptr || sf_row == nullptr)) ||
      (col && (q_col == nullptr || sf_col == nullptr)))
    return MXG_ERR_INVALID_ARG;
  if (!mult128(rows_capacity) || !mult128(cols) || cols == 0) return MXG_ERR_ALIGNMENT;
  if (rows_capacity + 128 * static_cast<int64_t>(G) > kMaxRows) return MXG_ERR_INVALID_ARG;
  if (!aligned16(x) || (row && (!aligned16(q_row) || !aligned16(sf_row))) ||
      (col && (!aligned16(q_col) || !aligned16(sf_col))))
    return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  if (rows_capacity == 0) return MXG_OK;
  return launched(mxg::launch_mxfp8_quantize(row, col, static_cast<const uint16_t*>(x),
                                             rows_capacity, cols, group_ws, G, q_row, sf_row,
                                             q_col, sf_col, dev_status, sms,
                                             reinterpret_cast<cudaStream_t>(stream), true),
                  1);
}

mxg_status_t mxg_group_quantize(mxg_format_t fmt, mxg_qlayout_t layout, const void* x,
                                int64_t rows_capacity, int64_t cols, const int64_t* group_ws,
                                int G, void* q_row, uint8_t* sf_row, void* q_col, uint8_t* sf_col,
                                float* outer_row, float* outer_col, int32_t* dev_status,
                                mxg_stream_t stream) {
  if (x == nullptr || (group_ws != nullptr && (G < 1 || G > 65536))) return MXG_ERR_INVALID_ARG;
  if (layout != MXG_ROWWISE && layout != MXG_COLWISE && layout != MXG_BOTH)
    return MXG_ERR_INVALID_ARG;
  const bool row = (layout & MXG_ROWWISE) != 0, col = (layout & MXG_COLWISE) != 0;
  if (fmt == MXG_MXFP8_E4M3) {
    if ((row && (q_row == nullptr || sf_row == nullptr)) ||
        (col && (q_col == nullptr || sf_col == nullptr)))
      return MXG_ERR_INVALID_ARG;
  } else if (fmt == MXG_NVFP4_ROWSCALED) {
    if ((row && (q_row == nullptr || sf_row == nullptr || outer_row == nullptr)) ||
        (col && (q_col == nullptr || sf_col == nullptr || outer_col == nullptr)) ||
        (col && group_ws != nullptr && G > 1024))
      return MXG_ERR_INVALID_ARG;
  } else {
    return MXG_ERR_INVALID_ARG;
  }
  if (!mult128(rows_capacity) || !mult128(cols) || cols == 0) return MXG_ERR_ALIGNMENT;
  if (!aligned16(x) || (row && (!aligned16(q_row) || !aligned16(sf_row))) ||
      (col && (!aligned16(q_col) || !aligned16(sf_col))))
    return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (rows_capacity == 0) {
    // no rows: every group is empty, and the NVFP4 colwise outer scales of an
    // empty group are 0 (the colwise kernel needs rows for its tensor map)
    if (fmt == MXG_NVFP4_ROWSCALED && col &&
        cudaMemsetAsync(outer_col, 0,
                        static_cast<size_t>(group_ws ? G : 1) * static_cast<size_t>(cols) *
                            sizeof(float),
                        s) != cudaSuccess)
      return MXG_ERR_LAUNCH;
    return MXG_OK;
  }
  if (fmt == MXG_MXFP8_E4M3)
    return launched(mxg::launch_mxfp8_quantize(row, col, static_cast<const uint16_t*>(x),
                                               rows_capacity, cols, group_ws, G,
                                               static_cast<uint8_t*>(q_row), sf_row,
                                               static_cast<uint8_t*>(q_col), sf_col, dev_status,
                                               sms, s, false),
                    1);
  if (row) {
    const mxg_status_t r = launched(
        mxg::launch_nvfp4_quantize(static_cast<const uint16_t*>(x), rows_capacity, cols, group_ws,
                                   G, static_cast<uint8_t*>(q_row), sf_row, outer_row, dev_status,
                                   sms, s),
        1);
    if (r != MXG_OK || !col) return r;
  }
  return launched(mxg::launch_nvfp4_quantize_colwise(static_cast<const uint16_t*>(x), rows_capacity,
                                                     cols, group_ws, G,
                                                     static_cast<uint8_t*>(q_col), sf_col,
                                                     outer_col, sms, s),
                  1);
}

static mxg_status_t grouped_gemm_impl(mxg_format_t fmt, mxg_gemm_mode_t mode,
                                      const mxg_operand_t* A, const mxg_operand_t* B,
                                      const int64_t* group_ws, int G, int64_t M_cap, int64_t N,
                                      int64_t K, const float* alpha, const float* beta,
                                      const float* bias, void* C, mxg_out_t out_type,
                                      int32_t* dev_status, int tile_n, int stage_bytes,
                                      int inject, uint64_t timeout_ns, mxg_stream_t stream,
                                      int unaligned) {
  if (A == nullptr || B == nullptr || C == nullptr || group_ws == nullptr || G < 1 || G > 1024)
    return MXG_ERR_INVALID_ARG;
  if (fmt != MXG_MXFP8_E4M3 && fmt != MXG_NVFP4_ROWSCALED) return MXG_ERR_INVALID_ARG;
  if (mode != MXG_FPROP_TN && mode != MXG_WGRAD_NT && mode != MXG_DGRAD_NN)
    return MXG_ERR_INVALID_ARG;
  if (out_type != MXG_OUT_F32 && out_type != MXG_OUT_BF16) return MXG_ERR_INVALID_ARG;
  if (A->data == nullptr || A->scale == nullptr || B->data == nullptr || B->scale == nullptr)
    return MXG_ERR_INVALID_ARG;
  const bool nv = fmt == MXG_NVFP4_ROWSCALED;
  if (nv && (mode == MXG_DGRAD_NN || beta != nullptr || A->outer == nullptr || B->outer == nullptr))
    return MXG_ERR_INVALID_ARG;  // row-scaled NVFP4: fprop and wgrad, no beta
  if (bias != nullptr && mode == MXG_WGRAD_NT) return MXG_ERR_INVALID_ARG;
  // unaligned groups: MXFP8 on the CTA-pair kernel, whose B spans >= 256 rows
  if (unaligned && (nv || (mode == MXG_FPROP_TN ? N * static_cast<int64_t>(G) : K) < 256))
    return MXG_ERR_INVALID_ARG;
  if (!mult128(M_cap) || !mult128(N) || !mult128(K) || N == 0 || K == 0)
    return MXG_ERR_ALIGNMENT;

  if (M_cap + (unaligned ? 128 * static_cast<int64_t>(G) : 0) > kMaxRows ||
      N * static_cast<int64_t>(G) > kMaxRows)
    return MXG_ERR_INVALID_ARG;
  if (!aligned16(A->data) || !aligned16(A->scale) || !aligned16(B->data) || !aligned16(B->scale) ||
      !aligned16(C))
    return MXG_ERR_ALIGNMENT;
  // operand shapes the mode implies (rows x contraction elements) and the
  // leading dimensions of the data, in bytes
  const int64_t M_pad = M_cap + (unaligned ? 128 * static_cast<int64_t>(G) : 0);
  const int64_t a_rows = mode == MXG_WGRAD_NT ? N : M_cap;
  const int64_t a_cols = mode == MXG_FPROP_TN ? K : (mode == MXG_WGRAD_NT ? M_pad : N);
  const int64_t b_rows = mode == MXG_FPROP_TN ? N * static_cast<int64_t>(G) : K;
  const int64_t b_cols = mode == MXG_FPROP_TN ? K : (mode == MXG_WGRAD_NT ? M_pad : N * G);
  int64_t a_ld = 0, b_ld = 0;
  mxg_status_t sh = operand_shape(A, a_rows, a_cols, nv, &a_ld);
  if (sh != MXG_OK) return sh;
  if ((sh = operand_shape(B, b_rows, b_cols, nv, &b_ld)) != MXG_OK) return sh;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  if (M_cap == 0) {
    // no rows: the fprop and dgrad outputs are empty; every wgrad group is
    // empty, and each dW_g is written as for an empty group
    if (mode != MXG_WGRAD_NT) return MXG_OK;
    return launched(mxg::launch_wgrad_no_rows(G, N, K, beta, C, out_type == MXG_OUT_BF16 ? 1 : 0,
                                              sms, reinterpret_cast<cudaStream_t>(stream)),
                    1);
  }
  return launched(mxg::launch_grouped_gemm(
                      nv, mode == MXG_WGRAD_NT ? 1 : (mode == MXG_DGRAD_NN ? 2 : 0), A->data, A->scale, A->outer, B->data,
                      B->scale, B->outer, group_ws, G, M_cap, N, K, alpha, beta, bias, C,
                      out_type == MXG_OUT_BF16 ? 1 : 0, dev_status, sms, tile_n, stage_bytes,
                      inject, timeout_ns, unaligned, a_ld, b_ld,
                      reinterpret_cast<cudaStream_t>(stream)),
                  1);
}

mxg_status_t mxg_grouped_gemm(mxg_format_t fmt, mxg_gemm_mode_t mode, const mxg_operand_t* A,
                              const mxg_operand_t* B, const int64_t* group_ws, int G,
                              int64_t M_cap, int64_t N, int64_t K, const float* alpha,
                              const float* beta, const float* bias, void* C, mxg_out_t out_type,
                              void* workspace, size_t workspace_bytes, int32_t* dev_status,
                              mxg_stream_t stream) {
  (void)workspace;
  (void)workspace_bytes;
  return grouped_gemm_impl(fmt, mode, A, B, group_ws, G, M_cap, N, K, alpha, beta, bias, C,
                           out_type, dev_status, 0, 0, 0, mxg::kDefaultWaitNs, stream, 0);
}

mxg_status_t mxg_grouped_gemm_debug(mxg_format_t fmt, mxg_gemm_mode_t mode, const mxg_operand_t* A,
                                    const mxg_operand_t* B, const int64_t* group_ws, int G,
                                    int64_t M_cap, int64_t N, int64_t K, const float* alpha,
                                    const float* beta, const float* bias, void* C,
                                    mxg_out_t out_type, int32_t* dev_status, int tile_n,
                                    int stage_bytes, int inject_flags, int64_t wait_timeout_ns,
                                    mxg_stream_t stream) {
  if (wait_timeout_ns < 0 || (inject_flags & ~1)) return MXG_ERR_INVALID_ARG;
  if ((tile_n != 0 && tile_n != 128 && tile_n != 256) || (stage_bytes != 0 && stage_bytes != 128))
    return MXG_ERR_INVALID_ARG;
  const uint64_t t = wait_timeout_ns == 0 ? mxg::kDefaultWaitNs
                                          : static_cast<uint64_t>(wait_timeout_ns);
  return grouped_gemm_impl(fmt, mode, A, B, group_ws, G, M_cap, N, K, alpha, beta, bias, C,
                           out_type, dev_status, tile_n, stage_bytes, inject_flags, t, stream, 0);
}

mxg_status_t mxg_grouped_gemm_unaligned(mxg_gemm_mode_t mode, const mxg_operand_t* A,
                                        const mxg_operand_t* B, const int64_t* group_ws, int G,
                                        int64_t M_cap, int64_t N, int64_t K, const float* alpha,
                                        const float* beta, const float* bias, void* C,
                                        mxg_out_t out_type, int32_t* dev_status,
                                        mxg_stream_t stream) {
  return grouped_gemm_impl(MXG_MXFP8_E4M3, mode, A, B, group_ws, G, M_cap, N, K, alpha, beta, bias,
                           C, out_type, dev_status, 0, 0, 0, mxg::kDefaultWaitNs, stream, 1);
}

size_t mxg_grouped_gemm_workspace_bytes(mxg_format_t fmt, mxg_gemm_mode_t mode, int G,
                                        int64_t M_cap, int64_t N) {
  (void)fmt;
  (void)mode;
  (void)G;
  (void)M_cap;
  (void)N;
  return 0;
}

mxg_status_t mxg_dequantize(mxg_format_t fmt, mxg_qlayout_t layout, const void* q,
                            const uint8_t* sf, const float* outer, int64_t rows, int64_t cols,
                            void* out, mxg_out_t out_type, mxg_stream_t stream) {
  if (q == nullptr || sf == nullptr || out == nullptr) return MXG_ERR_INVALID_ARG;
  if (fmt != MXG_MXFP8_E4M3 && fmt != MXG_NVFP4_ROWSCALED) return MXG_ERR_INVALID_ARG;
  if (layout != MXG_ROWWISE && layout != MXG_COLWISE) return MXG_ERR_INVALID_ARG;
  if (out_type != MXG_OUT_F32 && out_type != MXG_OUT_BF16) return MXG_ERR_INVALID_ARG;
  if (fmt == MXG_NVFP4_ROWSCALED && layout == MXG_COLWISE) return MXG_ERR_UNSUPPORTED;
  if (!mult128(rows) || !mult128(cols)) return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  return launched(mxg::launch_dequantize(fmt == MXG_NVFP4_ROWSCALED ? 1 : 0,
                                         layout == MXG_COLWISE ? 1 : 0,
                                         static_cast<const uint8_t*>(q), sf, outer, rows, cols, out,
                                         out_type == MXG_OUT_BF16 ? 1 : 0, sms,
                                         reinterpret_cast<cudaStream_t>(stream)),
                  1);
}

mxg_status_t mxg_grouped_gemm_16bit(mxg_dtype_t in_type, mxg_gemm_mode_t mode, const void* A,
                                    int64_t lda, const void* B, int64_t ldb,
                                    const int64_t* group_ws, int G, int64_t M_cap, int64_t N,
                                    int64_t K, const float* alpha, const float* beta, void* C,
                                    int64_t ldc, mxg_dtype_t out_type, int32_t* dev_status,
                                    mxg_stream_t stream) {
  const bool wgrad = mode == MXG_WGRAD_NT;
  // a ragged matrix without rows (M_cap = 0) needs no memory
  if ((A == nullptr && M_cap != 0) || (B == nullptr && !(wgrad && M_cap == 0)) ||
      (C == nullptr && !(!wgrad && M_cap == 0)) || group_ws == nullptr || G < 1 || G > 1024)
    return MXG_ERR_INVALID_ARG;
  if ((in_type != MXG_BF16 && in_type != MXG_F16) || (out_type != MXG_F32 && out_type != in_type))
    return MXG_ERR_INVALID_ARG;
  if (mode != MXG_FPROP_TN && mode != MXG_WGRAD_NT && mode != MXG_DGRAD_NN)
    return MXG_ERR_INVALID_ARG;
  if (M_cap < 0 || N < 1 || K < 1 || M_cap > kMaxRows || N > kMaxRows || K > kMaxRows)
    return MXG_ERR_INVALID_ARG;
  const int64_t a_cols = mode == MXG_FPROP_TN ? K : N;
  const int64_t c_cols = mode == MXG_FPROP_TN ? N : K;
  if (lda == 0) lda = a_cols;
  if (ldb == 0) ldb = K;
  if (ldc == 0) ldc = c_cols;
  // a row stride past 2^36 elements would leave the tensor maps' range
  constexpr int64_t kMaxLd = 1LL << 36;
  if (lda < a_cols || ldb < K || ldc < c_cols || lda > kMaxLd || ldb > kMaxLd || ldc > kMaxLd ||
      N > (1LL << 38) / ldb)
    return MXG_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(B) || lda % 8 != 0 || ldb % 8 != 0 ||
      !aligned_to(C, dtype_bytes(out_type)))
    return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  if (M_cap == 0 && !wgrad) return MXG_OK;
  return launched(mxg::launch_grouped_gemm16(
                      in_type == MXG_F16 ? 1 : 0,
                      mode == MXG_WGRAD_NT ? 1 : (mode == MXG_DGRAD_NN ? 2 : 0), A, lda, B, ldb,
                      group_ws, G, M_cap, N, K, alpha, beta, C, ldc, out_type, dev_status, sms,
                      reinterpret_cast<cudaStream_t>(stream)),
                  1);
}

mxg_status_t mxg_block_norm(const mxg_block_norm_t* desc, mxg_stream_t stream) {
  if (desc == nullptr) return MXG_ERR_INVALID_ARG;
  mxg_block_norm_t d = *desc;
  if (d.rows != 0 && (d.x == nullptr || (d.y == nullptr && d.n_out == nullptr) ||
                      (d.y != nullptr && d.x_out == nullptr)))
    return MXG_ERR_INVALID_ARG;
  mxg_status_t st = norm_common(d);
  if (st == MXG_ERR_INVALID_ARG) return st;
  if (d.ldxo == 0) d.ldxo = d.cols;
  if (d.ldn == 0) d.ldn = d.cols;
  if (d.ldxo < d.cols || d.ldn < d.cols || (d.x_out == d.x && d.x != nullptr && d.ldxo != d.ldx))
    return MXG_ERR_INVALID_ARG;
  if (st != MXG_OK) return st;
  if (!aligned_to(d.x_out, dtype_bytes(d.res_dtype)) || !aligned_to(d.n_out, dtype_bytes(d.dtype)))
    return MXG_ERR_ALIGNMENT;
  int sms = 0;
  if ((st = current_device(&sms)) != MXG_OK) return st;
  if (d.rows == 0) return MXG_OK;
  return launched(mxg::launch_block_norm(d, sms, reinterpret_cast<cudaStream_t>(stream)), 1);
}

size_t mxg_block_norm_workspace_bytes(int64_t rows, int64_t cols) {
  // a width that the calls refuse has no shape of teams to ask for
  if (rows < 0 || cols < 1 || cols > kMaxNormCols) return 0;
  return static_cast<size_t>(mxg::block_norm_ws_bytes(rows, cols));
}

mxg_status_t mxg_block_norm_backward(const mxg_block_norm_grad_t* desc, void* workspace,
                                     size_t workspace_bytes, mxg_stream_t stream) {
  if (desc == nullptr) return MXG_ERR_INVALID_ARG;
  mxg_block_norm_grad_t d = *desc;
  if (d.rows != 0 && (d.dx == nullptr || (d.dx_out == nullptr && d.dn == nullptr) ||
                      (d.dn != nullptr && d.x == nullptr) || (d.y != nullptr && d.dy == nullptr)))
    return MXG_ERR_INVALID_ARG;
  mxg_status_t st = norm_common(d);
  if (st == MXG_ERR_INVALID_ARG) return st;
  if (d.lddxo == 0) d.lddxo = d.cols;
  if (d.lddn == 0) d.lddn = d.cols;
  if (d.lddx == 0) d.lddx = d.cols;
  if (d.lddy == 0) d.lddy = d.cols;
  if (d.lddg == 0) d.lddg = d.cols;
  if (d.lddxo < d.cols || d.lddn < d.cols || d.lddx < d.cols || d.lddy < d.cols ||
      d.lddg < d.cols || (d.dx == d.dx_out && d.dx != nullptr && d.lddx != d.lddxo) ||
      (d.y != nullptr && ((d.dy == d.y && d.lddy != d.ldy) || (d.dy == d.dn && d.lddy != d.lddn))))
    return MXG_ERR_INVALID_ARG;
  if (st != MXG_OK) return st;
  const size_t e = dtype_bytes(d.dtype), r = dtype_bytes(d.res_dtype);
  if (!aligned_to(d.dx_out, r) || !aligned_to(d.dx, r) || !aligned_to(d.dn, e) ||
      !aligned_to(d.dy, e) || !aligned_to(d.dw_post, 4) || !aligned_to(d.dw_pre, 4) ||
      !aligned_to(d.dgate, d.gate_mode == MXG_GATE_FULL ? e : 4) || !aligned16(workspace))
    return MXG_ERR_ALIGNMENT;
  const size_t need = mxg_block_norm_workspace_bytes(d.rows, d.cols);
  if (workspace_bytes < need) return MXG_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && workspace == nullptr) return MXG_ERR_INVALID_ARG;
  int sms = 0;
  if ((st = current_device(&sms)) != MXG_OK) return st;
  return launched(mxg::launch_block_norm_backward(d, static_cast<float*>(workspace), sms,
                                                  reinterpret_cast<cudaStream_t>(stream)),
                  d.rows > 0 ? 2 : 1);
}

size_t mxg_grad_workspace_bytes(void) { return mxg::grad_ws_bytes(); }

mxg_status_t mxg_grad_norm(const mxg_grad_t* grads, int n, float* norm, void* workspace,
                           size_t workspace_bytes, mxg_stream_t stream) {
  return grad_impl(grads, n, false, 0.0f, norm, workspace, workspace_bytes, stream);
}

mxg_status_t mxg_grad_clip(const mxg_grad_t* grads, int n, float max_norm, float* norm,
                           void* workspace, size_t workspace_bytes, mxg_stream_t stream) {
  if (!(max_norm >= 0.0f)) return MXG_ERR_INVALID_ARG;
  return grad_impl(grads, n, true, max_norm, norm, workspace, workspace_bytes, stream);
}

size_t mxg_route_workspace_bytes(int64_t tokens, int experts, int k) {
  return route_sizes_ok(tokens, experts, k) ? mxg::route_ws_bytes(tokens, experts, k) : 0;
}

mxg_status_t mxg_route(const mxg_route_t* desc, void* workspace, size_t workspace_bytes,
                       int32_t* dev_status, mxg_stream_t stream) {
  if (desc == nullptr) return MXG_ERR_INVALID_ARG;
  mxg_route_t d = *desc;
  const size_t size = dtype_bytes(d.dtype);
  if (size == 0 || !route_sizes_ok(d.tokens, d.experts, d.k) ||
      (d.score != MXG_SCORE_SOFTMAX && d.score != MXG_SCORE_SIGMOID) ||
      !std::isfinite(d.scale) || !std::isfinite(d.balance))
    return MXG_ERR_INVALID_ARG;
  if (d.tokens != 0 && (d.logits == nullptr || d.expert == nullptr || d.weight == nullptr))
    return MXG_ERR_INVALID_ARG;
  if (!fill_ld(&d.ld, d.experts)) return MXG_ERR_INVALID_ARG;
  mxg_status_t st = route_rows_args(d.tokens, d.counts, d.row_of, d.group_ws, d.align,
                                    d.rows_capacity, d.last_dim);
  if (st != MXG_OK) return st;
  if (!aligned_to(d.logits, size) || !aligned_to(d.expert, 4) || !aligned_to(d.weight, 4) ||
      !aligned_to(d.loss, 4) || !aligned_to(d.slope, 4))
    return MXG_ERR_ALIGNMENT;
  st = route_memory(d.tokens, d.experts, d.k, workspace, workspace_bytes, dev_status);
  if (st != MXG_OK) return st;
  int sms = 0;
  if ((st = current_device(&sms)) != MXG_OK) return st;
  int launches = 0;
  const cudaError_t e = mxg::launch_route(d, workspace, dev_status,
                                          reinterpret_cast<cudaStream_t>(stream), &launches);
  return launched(e, static_cast<uint64_t>(launches));
}

mxg_status_t mxg_route_rows(const int32_t* expert, int64_t tokens, int experts, int k, int align,
                            int64_t rows_capacity, int64_t last_dim, int32_t* counts,
                            int32_t* row_of, int64_t* group_ws, void* workspace,
                            size_t workspace_bytes, int32_t* dev_status, mxg_stream_t stream) {
  if (!route_sizes_ok(tokens, experts, k) || (tokens != 0 && expert == nullptr))
    return MXG_ERR_INVALID_ARG;
  mxg_status_t st =
      route_rows_args(tokens, counts, row_of, group_ws, align, rows_capacity, last_dim);
  if (st != MXG_OK) return st;
  if (!aligned_to(expert, 4)) return MXG_ERR_ALIGNMENT;
  st = route_memory(tokens, experts, k, workspace, workspace_bytes, dev_status);
  if (st != MXG_OK) return st;
  int sms = 0;
  if ((st = current_device(&sms)) != MXG_OK) return st;
  int launches = 0;
  const cudaError_t e = mxg::launch_route_rows(
      expert, tokens, experts, k, align, rows_capacity, last_dim, counts, row_of, group_ws,
      workspace, dev_status, reinterpret_cast<cudaStream_t>(stream), &launches);
  return launched(e, static_cast<uint64_t>(launches));
}

mxg_status_t mxg_route_backward(const mxg_route_grad_t* desc, mxg_stream_t stream) {
  if (desc == nullptr) return MXG_ERR_INVALID_ARG;
  mxg_route_grad_t d = *desc;
  const size_t size = dtype_bytes(d.dtype);
  if (size == 0 || !route_sizes_ok(d.tokens, d.experts, d.k) ||
      (d.score != MXG_SCORE_SOFTMAX && d.score != MXG_SCORE_SIGMOID) || !std::isfinite(d.scale) ||
      (d.slope != nullptr) != (d.dloss != nullptr))
    return MXG_ERR_INVALID_ARG;
  if (d.tokens != 0 && (d.logits == nullptr || d.expert == nullptr || d.dlogits == nullptr))
    return MXG_ERR_INVALID_ARG;
  if (!fill_ld(&d.ld, d.experts) || !fill_ld(&d.ldd, d.experts) ||
      (d.dlogits != nullptr && d.dlogits == d.logits && d.ld != d.ldd))
    return MXG_ERR_INVALID_ARG;
  if (!aligned_to(d.logits, size) || !aligned_to(d.dlogits, size) || !aligned_to(d.expert, 4) ||
      !aligned_to(d.dweight, 4) || !aligned_to(d.slope, 4) || !aligned_to(d.dloss, 4))
    return MXG_ERR_ALIGNMENT;
  int sms = 0;
  const mxg_status_t st = current_device(&sms);
  if (st != MXG_OK) return st;
  if (d.tokens == 0) return MXG_OK;
  return launched(
      mxg::launch_route_backward(d, sms, reinterpret_cast<cudaStream_t>(stream)), 1);
}

mxg_status_t mxg_dispatch(const mxg_expert_rows_t* desc, mxg_stream_t stream) {
  return expert_rows_impl(desc, 0, stream);
}

mxg_status_t mxg_combine(const mxg_expert_rows_t* desc, mxg_stream_t stream) {
  return expert_rows_impl(desc, 1, stream);
}

mxg_status_t mxg_combine_backward(const mxg_expert_rows_t* desc, mxg_stream_t stream) {
  return expert_rows_impl(desc, 2, stream);
}

mxg_status_t mxg_gated_act(const mxg_gated_act_t* desc, mxg_stream_t stream) {
  return gated_act_impl(desc, false, stream);
}

mxg_status_t mxg_gated_act_backward(const mxg_gated_act_t* desc, mxg_stream_t stream) {
  return gated_act_impl(desc, true, stream);
}

const char* mxg_status_string(mxg_status_t status) {
  switch (status) {
    case MXG_OK: return "MXG_OK";
    case MXG_ERR_INVALID_ARG: return "MXG_ERR_INVALID_ARG";
    case MXG_ERR_ALIGNMENT: return "MXG_ERR_ALIGNMENT";
    case MXG_ERR_UNSUPPORTED_ARCH: return "MXG_ERR_UNSUPPORTED_ARCH";
    case MXG_ERR_LAUNCH: return "MXG_ERR_LAUNCH";
    case MXG_ERR_WORKSPACE_TOO_SMALL: return "MXG_ERR_WORKSPACE_TOO_SMALL";
    case MXG_ERR_UNSUPPORTED: return "MXG_ERR_UNSUPPORTED";
  }
  return "MXG_ERR_UNKNOWN";
}

int mxg_version(void) { return 100; }

uint64_t mxg_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

}  // extern "C"
