// ops_internal.h -- what the operators' host code shares (ops_api.cu): the
// handle, error reporting, workspace carving, padded copies and the planning
// and launch of one block product.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "../../include/gemm_ops.h"
#include "block_params.h"

namespace spgemm {
constexpr int kSmallCluster = 8;  // CTAs of a cluster of the on-chip iteration, at most
}

// What persists between calls: limits of the device and its status word.  Calls
// only read it (but for the flag), so that it serves any streams, captured graphs
// among them.
struct gemm_ops {
  int device = 0;
  int sm_count = 0;
  int pairs = 0;                 // co-resident CTA pairs
  // Co-resident clusters of the on-chip iteration, by its row blocks (less
  // one) and the cluster's CTAs.
  int small_clusters[2][spgemm::kSmallCluster + 1] = {};
  size_t smem_optin = 0;
  int64_t l2_bytes = 0;
  unsigned long long timeout_ns = 0;
  int debug_fault = 0;
  int* d_status = nullptr;       // [0] code, [1] detail
  std::atomic<bool> layer_norm_ready{false};  // its kernels' attributes are set
};

namespace spgemm {

void set_last_error(const char* text);  // gemm_api.cu

gemm_status_t ops_fail(gemm_status_t st, const char* fmt, ...);
gemm_status_t ops_cuda_fail(cudaError_t e, const char* what);

constexpr unsigned long long kOpsTimeoutNs = 2000000000ull;  // 2 s per wait
constexpr int64_t kOpsMaxDim = (int64_t{1} << 31) - 1;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Restores the caller's current device on scope exit.
struct OpsDevice {
  int prev = -1;
  bool switched = false;
  cudaError_t err;
  explicit OpsDevice(int dev);
  ~OpsDevice();
};

// Hands out 256-byte aligned pieces of a workspace, or, with a null base,
// only counts them.
struct Carver {
  uint8_t* base;
  size_t used = 0;
  explicit Carver(void* p) : base(static_cast<uint8_t*>(p)) {}
  void* take(size_t bytes) {
    void* p = base ? base + used : nullptr;
    used += align256(bytes);
    return p;
  }
};

// A matrix (or a batch of them) as a product's operand or output.
struct Matrix {
  const void* ptr = nullptr;
  int64_t rows = 0, cols = 0, ld = 0, batch_stride = 0;
};

// Whether the copy engine can read the matrix where it lies.
inline bool copyable(const Matrix& m) {
  return (reinterpret_cast<uintptr_t>(m.ptr) & 15u) == 0 && m.ld % 8 == 0;
}

// A batch of row-major 16-bit matrices as a 3-D map, box `box_cols` x
// `box_rows` of one matrix, 128-byte swizzle.
gemm_status_t encode_map(CUtensorMap* map, bool bf16, const Matrix& m, int64_t batch, uint32_t box_cols,
                         uint32_t box_rows, CUtensorMapL2promotion l2);

// Whether two ranges of bytes share one (NULL or empty ones share none).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

// Up to kPackJobs matrices copied to rows of a 16-byte multiple, in one launch.
constexpr int kPackJobs = 4;
struct PackJob {
  const uint16_t* src;
  uint16_t* dst;
  int64_t rows, cols, ld, ldp;
};
struct PackJobs {
  PackJob job[kPackJobs];
  int count = 0;
};
cudaError_t launch_pack(const PackJobs& jobs, int sm_count, cudaStream_t stream);

// One product of the block kernels.
struct BlockProblem {
  enum Kind { kNT, kNN, kTN, kDiagOut, kDiagRows, kDiagCols, kGated, kGatedBwd } kind = kNT;
  int64_t M = 0, N = 0, K = 0;   // output extent (gated: N columns of H) and reduction
  int64_t batch = 1;
  Matrix a, b, d;                // d: added with weight beta (fp16; the kDiag kinds)
  bool bf16 = false, out_bf16 = false;
  bool symmetric = false;
  float alpha = 1.0f, beta = 0.0f;
  float* diag = nullptr;         // the kDiag kinds: diag_batch elements a matrix, at least M
  int64_t diag_batch = 0;        // (kDiagOut, kDiagRows) or N rounded up to 64 (kDiagCols)
  int act = 0;
  Matrix out0, out1;             // cols: the columns of each row that may be written (>= N)
  float* pre = nullptr;
  bool stream_b = false;         // B is read once: evict-first copies
};

// A call's workspace for its products' split tiles: fp32 partials, and the flags
// that say they are there (4 per CTA, raised and reset within a launch).  They
// are a call's own, because calls on other streams and replayed graphs may run
// beside it.  Whatever runs first in a call and needs no flags zeroes them.
struct BlockScratch {
  float* partials = nullptr;
  int* flags = nullptr;
  int count = 0;         // flags
  bool zeroed = false;   // by what was launched before
};
BlockScratch take_scratch(const gemm_ops* ops, Carver& c);  // enough for any product

cudaError_t logprobs_set_smem();  // logprobs.cu
cudaError_t adamw_set_smem();  // adamw.cu

gemm_status_t run_block(const gemm_ops* ops, const BlockProblem& pr, BlockScratch& scratch, cudaStream_t stream);

}  // namespace spgemm
