// ops_api.cu -- the operators' handle (include/gemm_ops.h) and the planning
// and launch of their products.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>

#include "few_tokens.h"
#include "ops_internal.h"
#include "orthogonal_small.h"
#include "ptx.cuh"

namespace spgemm {

gemm_status_t ops_fail(gemm_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  try {
    set_last_error(buf);
  } catch (...) {  // out of host memory: the status still says what failed
  }
  return st;
}

gemm_status_t ops_cuda_fail(cudaError_t e, const char* what) {
  return ops_fail(GEMM_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

OpsDevice::OpsDevice(int dev) {
  err = cudaGetDevice(&prev);
  if (err == cudaSuccess && prev != dev) {
    err = cudaSetDevice(dev);
    switched = err == cudaSuccess;
  }
}
OpsDevice::~OpsDevice() {
  if (switched) cudaSetDevice(prev);
}

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// A batch of row-major 16-bit matrices as a 3-D map, box `box_cols` x
// `box_rows` of one matrix, 128-byte swizzle.
gemm_status_t encode(CUtensorMap* map, bool bf16, const Matrix& m, int64_t batch, uint32_t box_cols,
                     uint32_t box_rows, CUtensorMapL2promotion l2) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc) return ops_fail(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
  const int64_t step = batch > 1 ? m.batch_stride : m.rows * m.ld;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(m.cols), static_cast<cuuint64_t>(m.rows),
                              static_cast<cuuint64_t>(batch)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(m.ld) * 2u,
                                 static_cast<cuuint64_t>(step) * 2u};
  const cuuint32_t box[3] = {box_cols, box_rows, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  const CUresult r =
      enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
          const_cast<void*>(m.ptr), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, l2, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return ops_fail(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled failed (CUresult %d) for %lld x %lld x %lld",
                    static_cast<int>(r), static_cast<long long>(batch),
                    static_cast<long long>(m.rows), static_cast<long long>(m.cols));
  return GEMM_OK;
}

// The bulk-store path needs every row (and matrix) of the output 16-byte
// aligned.  A bulk store is clipped to whole 16-byte units (loads to single
// elements), so the output must also own its rows (Matrix::cols) up to the
// next multiple of 8 elements.
BlockOut describe_out(const Matrix& m, int64_t N, int64_t batch) {
  BlockOut o{};
  o.ptr = const_cast<void*>(m.ptr);
  o.ld = m.ld;
  o.batch = m.batch_stride;
  o.tma = copyable(m) && m.cols >= round8(N) && (batch == 1 || m.batch_stride % 8 == 0) ? 1 : 0;
  return o;
}

constexpr int kZeroThreads = 256;

// Flags of a call whose first product already needs them.  The product starts
// beside this kernel and waits for it.
__global__ void __launch_bounds__(kZeroThreads) zero_flags_kernel(int* flags, int count) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  for (int i = threadIdx.x; i < count; i += kZeroThreads) flags[i] = 0;
}

cudaError_t launch_zero_flags(const BlockScratch& s, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kZeroThreads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, zero_flags_kernel, s.flags, s.count);
}

constexpr size_t kStagingBytes = 4u * 2u * kStoreBuf;

size_t block_smem(int cg, int stages, int a_rows) {
  const size_t slice = static_cast<size_t>(a_rows) * kBK * 2 +
                       static_cast<size_t>(block_bn(cg) / cg) * kBK * 2;
  return kAlignSlack + slice * block_sub(cg) * stages + kStagingBytes + kBarrierBytes;
}

}  // namespace

BlockScratch take_scratch(const gemm_ops* ops, Carver& c) {
  BlockScratch s;
  s.partials = static_cast<float*>(
      c.take(ops->sm_count * std::max(block_partial_bytes(1), block_partial_bytes(2))));
  s.count = 4 * ops->sm_count;
  s.flags = static_cast<int*>(c.take(s.count * sizeof(int)));
  return s;
}

gemm_status_t run_block(const gemm_ops* ops, const BlockProblem& pr, BlockScratch& scratch, cudaStream_t stream) {
  const bool gated = pr.kind == BlockProblem::kGated;
  const bool a_t = pr.kind == BlockProblem::kTN;
  const bool use_d = pr.kind == BlockProblem::kDiagOut || pr.kind == BlockProblem::kDiagRows ||
                     pr.kind == BlockProblem::kDiagCols;
  const bool b_n = pr.kind == BlockProblem::kNN || pr.kind == BlockProblem::kTN ||
                   pr.kind == BlockProblem::kDiagRows ||
                   pr.kind == BlockProblem::kGatedBwd;
  BlockMaps maps;
  BlockParams p;
  std::memset(&p, 0, sizeof(p));

  auto tiles = [&](int cg, int64_t* tm, int64_t* tn) -> int64_t {
    *tm = ceil_div(pr.M, static_cast<int64_t>(kBM) * cg);
    *tn = ceil_div(pr.N, gated ? block_bn(cg) / 2 : block_bn(cg));
    return (pr.symmetric ? *tn * (*tn + 1) / 2 : *tm * *tn) * pr.batch;
  };
  // The cheapest of three schedules, by a model of their times in us (fitted
  // to time stamps of launches between 3 and 600 us).  A pair multiplies a 256
  // x 256 x 128 slot in kPairSlot; a single CTA's 128 x 128 x 64 slot moves
  // twice the operand bytes per product and is bound by what an SM takes in,
  // kSoloSlot.  A wave of tiles adds its start and its epilogue.  Splitting K
  // costs its exchange: kSplitCost through a cluster's shared memory; through
  // the workspace kPairStream or kSoloStream and, for every partial that a
  // tile's owner adds one after another, kPairPart or kSoloPart.
  constexpr double kPairSlot = 0.65, kSoloSlot = 0.30, kPairWave = 5.0, kSoloWave = 3.5;
  constexpr double kSplitCost = 4.0, kPairStream = 8.0, kSoloStream = 4.0;
  constexpr double kPairPart = 2.5, kSoloPart = 1.5;
  constexpr double kHbmBytesPerUs = 6.5e6;
  int64_t tm, tn, walkers = 0, sk = 0;
  int cg = 1, splits = 1;
  double best = 1e300;
  auto offer = [&](double cost, int c, int s, int64_t w, int64_t k) {
    if (cost < best) {
      best = cost;
      cg = c;
      splits = s;
      walkers = w;
      sk = k;
    }
  };
  for (int c = 1; c <= 2; ++c) {
    if (c == 2 && (pr.M <= kBM || ops->pairs < 1)) break;
    const int64_t most = c == 2 ? ops->pairs : ops->sm_count;
    const int64_t nt = tiles(c, &tm, &tn);
    const int64_t kb = ceil_div(pr.K, static_cast<int64_t>(kBK) * block_sub(c));
    const double slot = c == 2 ? kPairSlot : kSoloSlot;
    // Later waves' epilogues hide behind the next tiles' main loops where those are longer.
    const double wave = c == 2 ? kPairWave : kSoloWave;
    const double waves = static_cast<double>(ceil_div(nt, most));
    offer(wave + kb * slot + (waves - 1) * std::max(kb * slot, 0.6 * wave), c, 1, std::min(nt, most), 0);
    // Stream-K: the last one to two waves' slots shared out evenly, or fewer
    // tiles than walkers over up to four walkers each.  The walkers are then
    // at different places along K, so operands beyond L2 are read from HBM
    // once per tile instead of once per wave.
    for (int64_t per = 1; per <= 4 && nt % most != 0; ++per) {
      const int64_t w = nt < most ? std::min(most, nt * (per + 1)) : most;
      if (nt * kb < 2 * w) break;
      const int64_t shared = nt < w ? nt : nt % w + w;
      const double parts = static_cast<double>(nt < w ? ceil_div(w, nt) - 1 : 1);
      double cost = wave + static_cast<double>(nt) * kb / w * slot +
                    (c == 2 ? kPairStream + parts * kPairPart : kSoloStream + parts * kSoloPart);
      const double operands = 2.0 * (pr.M + pr.N * (gated ? 2 : 1)) * pr.K * pr.batch;
      if (operands > 0.75 * ops->l2_bytes && pr.M > kBM) {
        const double reads = 2.0 * shared * (kBM * c + block_bn(c)) * pr.K / kHbmBytesPerUs;
        cost += std::max(0.0, reads - static_cast<double>(shared) * kb / w * slot);
      }
      offer(cost, c, 1, w, shared);
      if (w == most) break;
    }
    if (c == 1)
      for (int s = 2; s <= kMaxSplits; s *= 2)
        if (nt * s <= most && kb >= 2 * s)
          offer(wave + ceil_div(kb, s) * slot + kSplitCost, c, s, nt * s, 0);
  }
  const int64_t nt = tiles(cg, &tm, &tn);
  const int64_t kb = ceil_div(pr.K, static_cast<int64_t>(kBK) * block_sub(cg));
  if (nt > kOpsMaxDim) return ops_fail(GEMM_ERR_INVALID_ARG, "too many output tiles");

  const int a_rows = a_t || cg == 2 || pr.M > 64 ? kBM : static_cast<int>(round8(pr.M));
  int stages = kMaxStages;
  while (stages > 1 && block_smem(cg, stages, a_rows) > ops->smem_optin) --stages;
  const size_t smem = block_smem(cg, stages, a_rows);
  if (smem > ops->smem_optin) return ops_fail(GEMM_ERR_SMEM_BUDGET, "no ring fits shared memory");

  p.M = static_cast<int>(pr.M);
  p.N = static_cast<int>(pr.N);
  p.K = static_cast<int>(pr.K);
  p.tiles_m = static_cast<int>(tm);
  p.tiles_n = static_cast<int>(tn);
  p.num_tiles = static_cast<int>(nt);
  p.tiles_per = static_cast<int>(nt / pr.batch);
  p.batch = static_cast<int>(pr.batch);
  p.k_blocks = static_cast<int>(kb);
  p.stages = stages;
  p.raster_group = cg == 2 ? 8 : 16;
  p.walkers = static_cast<int>(walkers);
  p.splits = splits;
  p.sk_tiles = static_cast<int>(sk);
  p.dp_tiles = static_cast<int>(nt - sk);
  p.sk_ws = scratch.partials;
  p.sk_flags = scratch.flags;
  p.zero_flags = scratch.zeroed || sk > 0 ? 0 : scratch.count;
  p.a_box_rows = a_rows;
  p.b_stream = pr.stream_b && tm == 1 ? 1 : 0;
  p.l2_prefetch_first = p.b_stream;
  p.bf16 = pr.bf16 ? 1 : 0;
  p.idesc = ptx::instr_desc_f16(kBM * cg, block_bn(cg), pr.bf16, b_n) | (a_t ? 1u << 15 : 0u);
  p.status = ops->d_status;
  p.timeout_ns = ops->timeout_ns;
  p.inject_fault = ops->debug_fault;
  p.symmetric = pr.symmetric ? 1 : 0;
  p.out_bf16 = pr.out_bf16 ? 1 : 0;
  p.act = pr.act;
  p.gate_rows = gated ? static_cast<int>(pr.N) : 0;
  // Two epilogue warps per lane quarter halve an epilogue that no main loop
  // hides: single CTAs, one wave (or less) of tiles, and pairs whose K is
  // short next to what their epilogue moves (one warp a quarter -> two, in us:
  // gated backward and dX of 2048 x 2048 x 8192 176 -> 161, the forward pass
  // that keeps its projections 142 -> 138; updates of 2048 x 8192 552 -> 534;
  // at K = 16384 no difference).
  const int64_t short_k = pr.kind == BlockProblem::kGatedBwd ? 8192
                          : gated || use_d                   ? 2048
                                                             : 1024;
  p.epi = cg == 1 || pr.K <= short_k || nt <= walkers ? 2 : 1;
  p.alpha = pr.alpha;
  p.beta = pr.beta;
  p.diag = pr.diag;
  p.diag_batch = pr.diag_batch;
  p.out0 = describe_out(pr.out0, pr.N, pr.batch);
  p.out1 = describe_out(pr.out1, pr.N, pr.batch);
  p.pre = pr.pre;
  p.pre_half = ceil_div(pr.M, 32) * 32 * pr.N;

  const CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  const CUtensorMapL2promotion none = CU_TENSOR_MAP_L2_PROMOTION_NONE;
  const uint32_t b_rows = gated && cg == 1 ? block_bn(1) / 2 : block_bn(cg) / cg;
  gemm_status_t st = encode(&maps.a, pr.bf16, pr.a, pr.batch, kBK,
                            a_t ? kBK : static_cast<uint32_t>(a_rows), l2);
  if (st == GEMM_OK) st = encode(&maps.b, pr.bf16, pr.b, pr.batch, kBK, b_n ? kBK : b_rows, l2);
  Matrix o0 = pr.out0, o1 = pr.out1;
  o0.rows = o1.rows = pr.M;
  o0.cols = o1.cols = pr.N;
  maps.c0 = maps.c1 = maps.d = maps.a;  // valid maps where a product has no such operand
  if (st == GEMM_OK && p.out0.tma) st = encode(&maps.c0, pr.out_bf16, o0, pr.batch, 64, 32, none);
  if (st == GEMM_OK && p.out1.ptr && p.out1.tma)
    st = encode(&maps.c1, pr.out_bf16, o1, pr.batch, 64, 32, none);
  if (st == GEMM_OK && use_d) st = encode(&maps.d, false, pr.d, pr.batch, 64, 32, none);
  if (st != GEMM_OK) return st;

  const int grid = static_cast<int>(walkers) * cg;
  cudaError_t e = cudaSuccess;
  if (sk > 0 && !scratch.zeroed) e = launch_zero_flags(scratch, stream);
  if (e != cudaSuccess) return ops_cuda_fail(e, "flag clearing launch");
  scratch.zeroed = true;
  switch (pr.kind) {
    case BlockProblem::kNT: e = block_launch_nt(maps, p, cg, grid, smem, stream); break;
    case BlockProblem::kNN: e = block_launch_nn(maps, p, cg, grid, smem, stream); break;
    case BlockProblem::kTN: e = block_launch_tn(maps, p, cg, grid, smem, stream); break;
    case BlockProblem::kDiagOut: e = block_launch_diag_out(maps, p, cg, grid, smem, stream); break;
    case BlockProblem::kDiagRows: e = block_launch_diag_rows(maps, p, cg, grid, smem, stream); break;
    case BlockProblem::kDiagCols: e = block_launch_diag_cols(maps, p, cg, grid, smem, stream); break;
    case BlockProblem::kGated: e = block_launch_gated(maps, p, cg, grid, smem, stream); break;
    default: e = block_launch_gated_bwd(maps, p, cg, grid, smem, stream); break;
  }
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "block product launch");
}

}  // namespace spgemm

using namespace spgemm;

extern "C" {

gemm_status_t gemm_ops_create(gemm_ops_t** out, int device) {
  ops_fail(GEMM_OK, "%s", "");
  if (!out) return ops_fail(GEMM_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (device < 0) return ops_fail(GEMM_ERR_INVALID_ARG, "device %d < 0", device);
  int ndev = 0;
  cudaError_t e = cudaGetDeviceCount(&ndev);
  if (e != cudaSuccess) return ops_cuda_fail(e, "cudaGetDeviceCount");
  if (device >= ndev)
    return ops_fail(GEMM_ERR_INVALID_ARG, "device %d >= count %d", device, ndev);
  gemm_device_desc_t desc;
  const gemm_status_t st = gemm_device_query(device, &desc);
  if (st != GEMM_OK) return st;
  OpsDevice guard(device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  gemm_ops* ops = new (std::nothrow) gemm_ops();
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "out of host memory");
  ops->device = device;
  ops->sm_count = desc.sm_count;
  ops->pairs = desc.pair_clusters;
  ops->smem_optin = static_cast<size_t>(desc.smem_optin);
  ops->l2_bytes = desc.l2_bytes;
  ops->timeout_ns = kOpsTimeoutNs;
  for (auto set : {block_set_smem_nt, block_set_smem_nn, block_set_smem_tn, block_set_smem_diag_out,
                   block_set_smem_diag_rows, block_set_smem_diag_cols, block_set_smem_gated,
                   block_set_smem_gated_bwd})
    if (e == cudaSuccess) e = set(ops->smem_optin);
  if (e == cudaSuccess) e = logprobs_set_smem();
  if (e == cudaSuccess) e = small_newton_init(ops);
  if (e == cudaSuccess) e = few_tokens_init(ops);
  if (e == cudaSuccess) e = cudaMalloc(&ops->d_status, 4 * sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(ops->d_status, 0, 4 * sizeof(int));
  // cudaMemset runs on the default stream; another stream's first call must not overtake it.
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) {
    gemm_ops_destroy(ops);
    return ops_cuda_fail(e, "operator handle set-up");
  }
  *out = ops;
  return GEMM_OK;
}

void gemm_ops_destroy(gemm_ops_t* ops) {
  if (!ops) return;
  OpsDevice guard(ops->device);
  cudaDeviceSynchronize();
  if (ops->d_status) cudaFree(ops->d_status);
  delete ops;
}

gemm_status_t gemm_ops_configure(gemm_ops_t* ops, int64_t timeout_ns, int debug_fault) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  if (timeout_ns < 0) return ops_fail(GEMM_ERR_INVALID_ARG, "negative timeout_ns");
  if (debug_fault < 0 || debug_fault > 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "debug_fault %d not in {0, 1}", debug_fault);
  ops->timeout_ns = timeout_ns > 0 ? static_cast<unsigned long long>(timeout_ns) : kOpsTimeoutNs;
  ops->debug_fault = debug_fault;
  return GEMM_OK;
}

gemm_status_t gemm_ops_check(gemm_ops_t* ops, int32_t* device_status, int32_t* detail) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops || !device_status) return ops_fail(GEMM_ERR_INVALID_ARG, "NULL argument");
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return ops_cuda_fail(e, "cudaDeviceSynchronize");
  int h[4] = {0, 0, 0, 0};
  e = cudaMemcpy(h, ops->d_status, sizeof(h), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess) e = cudaMemset(ops->d_status, 0, sizeof(h));
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) return ops_cuda_fail(e, "read or clear the status word");
  *device_status = h[0];
  if (detail) *detail = h[1];
  return GEMM_OK;
}

}  // extern "C"
