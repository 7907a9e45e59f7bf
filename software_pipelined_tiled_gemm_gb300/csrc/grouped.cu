// grouped.cu -- the products grouped by expert: argument checks, padded copies
// of operands that need them, the copies of the groups' last tokens, and the
// launches of the forward and backward products (grouped_kernel.cuh).
#include "grouped_kernel.cuh"

#include <algorithm>

#include "grouped_few.h"
#include "ops_internal.h"

using namespace spgemm;

namespace {

// Rows [m - m % 16, m) of each group of m rows, padded with zeros to 16: the
// last, partial step of the sums over tokens.  At most 15 rows a group move,
// so this is bound by its launch (2 us).
struct TailJob {
  const uint16_t* src;
  uint16_t* dst;  // groups x 16 rows, pitch ldp
  int64_t ld, ldp;
  int cols;
};
struct TailJobs {
  TailJob job[2];
};
constexpr int kTailThreads = 256;

__global__ void __launch_bounds__(kTailThreads)
    tail_kernel(const TailJobs jobs, const int64_t* offsets, int64_t rows) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  const int e = blockIdx.x;
  const int64_t first = offsets[e], end = offsets[e + 1];
  if (first < 0 || first > end || end > rows) return;  // the products report it
  const int tail = static_cast<int>((end - first) % kGroupedTail);
  if (tail == 0) return;
  const TailJob& j = jobs.job[blockIdx.z];
  const int vectors = (j.cols + 7) / 8;
  for (int i = blockIdx.y * kTailThreads + threadIdx.x; i < kGroupedTail * vectors; i += gridDim.y * kTailThreads) {
    const int r = i / vectors, v = i - r * vectors;
    uint4 out = make_uint4(0u, 0u, 0u, 0u);
    if (r < tail) {
      const uint16_t* src = j.src + (end - tail + r) * j.ld + 8 * v;
      if (8 * v + 8 <= j.cols) {
        out = __ldcg(reinterpret_cast<const uint4*>(src));
      } else {
        uint32_t wd[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (8 * v + c < j.cols) wd[c >> 1] |= static_cast<uint32_t>(src[c]) << ((c & 1) * 16);
        out = make_uint4(wd[0], wd[1], wd[2], wd[3]);
      }
    }
    *reinterpret_cast<uint4*>(j.dst + (static_cast<int64_t>(e) * kGroupedTail + r) * j.ldp + 8 * v) = out;
  }
}

template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Grouped {
  const gemm_grouped_args_t* a;
  Matrix x, w, dy, tail_x, tail_dy;
  PackJobs pack;
};

constexpr int64_t kMostRows = (int64_t{1} << 31) - 65536;

gemm_status_t check(const gemm_grouped_args_t* a, bool backward) {
  if (!a) return ops_fail(GEMM_ERR_INVALID_ARG, "args is NULL");
  if (a->rows < 0 || a->n < 1 || a->k < 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "rows %lld < 0 or n %lld, k %lld < 1", (long long)a->rows,
                    (long long)a->n, (long long)a->k);
  if (a->groups < 1 || a->groups > GEMM_GROUPED_MAX_GROUPS)
    return ops_fail(GEMM_ERR_INVALID_ARG, "%lld groups not in 1 .. %d", (long long)a->groups,
                    GEMM_GROUPED_MAX_GROUPS);
  if (a->n > kOpsMaxDim || a->k > kOpsMaxDim) return ops_fail(GEMM_ERR_INVALID_ARG, "size above 2^31-1");
  // The kernels count rows in 32 bits, a tile's or a launch's warps beyond the last.
  if (a->rows > kMostRows) return ops_fail(GEMM_ERR_INVALID_ARG, "more than 2^31 - 65536 rows");
  // The tiles of 32 output rows that all products could need.
  const int64_t most = std::max(ceil_div(a->n, int64_t{kGroupedLanes}), ceil_div(a->k, int64_t{kGroupedLanes}));
  if (most * (ceil_div(a->rows, int64_t{kGroupedUnit}) + a->groups) > kOpsMaxDim / 2 ||
      a->groups * most * ceil_div(std::max(a->n, a->k), int64_t{kGroupedUnit}) > kOpsMaxDim / 2)
    return ops_fail(GEMM_ERR_INVALID_ARG, "too many output tiles");
  if (a->dtype != GEMM_F16 && a->dtype != GEMM_BF16)
    return ops_fail(GEMM_ERR_INVALID_ARG, "dtype %d out of range", static_cast<int>(a->dtype));
  if (a->ldx < a->k) return ops_fail(GEMM_ERR_INVALID_ARG, "ldx %lld < k", (long long)a->ldx);
  if (backward && a->lddy < a->n) return ops_fail(GEMM_ERR_INVALID_ARG, "lddy %lld < n", (long long)a->lddy);
  if (a->zero_rest != 0 && a->zero_rest != 1)
    return ops_fail(GEMM_ERR_INVALID_ARG, "zero_rest %d not in {0, 1}", a->zero_rest);
  if (!a->offsets) return ops_fail(GEMM_ERR_INVALID_ARG, "offsets is NULL");
  if (reinterpret_cast<uintptr_t>(a->offsets) & 7u)
    return ops_fail(GEMM_ERR_INVALID_ARG, "offsets must be 8-byte aligned");
  if (a->rows > 0) {
    if (!a->x || !a->w) return ops_fail(GEMM_ERR_INVALID_ARG, "x or w is NULL");
    if (backward && !a->dy) return ops_fail(GEMM_ERR_INVALID_ARG, "dy is NULL");
    if (!backward && !a->y) return ops_fail(GEMM_ERR_INVALID_ARG, "y is NULL");
  }
  const void* ptrs[] = {a->x, a->w, a->y, a->dy, a->dx, a->dw};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 1u)
      return ops_fail(GEMM_ERR_INVALID_ARG, "matrices must be 2-byte aligned");
  return GEMM_OK;
}

// Outputs against inputs and each other.
gemm_status_t check_overlap(const gemm_grouped_args_t* a, bool backward, const void* ws, size_t ws_bytes) {
  const size_t R = a->rows, N = a->n, K = a->k, E = a->groups;
  struct Range {
    const void* p;
    size_t n;
    const char* name;
  };
  const Range in[] = {{a->x, R ? ((R - 1) * a->ldx + K) * 2 : 0, "x"},
                      {a->w, 2 * E * N * K, "w"},
                      {a->offsets, 8 * (E + 1), "offsets"},
                      {backward ? a->dy : nullptr, R && backward ? ((R - 1) * a->lddy + N) * 2 : 0, "dy"}};
  const Range out[] = {{backward ? nullptr : a->y, 2 * R * N, "y"},
                       {backward ? a->dx : nullptr, 2 * R * K, "dx"},
                       {backward ? a->dw : nullptr, 2 * E * N * K, "dw"},
                       {ws, ws_bytes, "the workspace"}};
  constexpr int kOut = sizeof(out) / sizeof(out[0]);
  for (int i = 0; i < kOut; ++i) {
    for (const Range& r : in)
      if (overlap(out[i].p, out[i].n, r.p, r.n))
        return ops_fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return ops_fail(GEMM_ERR_INVALID_ARG, "%s overlaps %s", out[i].name, out[j].name);
  }
  return GEMM_OK;
}

// Lays out the workspace (with a null base: only measures it).  An operand
// the copy engine cannot read is replaced by a padded copy.
size_t layout(const gemm_ops* ops, const gemm_grouped_args_t* a, bool backward, void* workspace, Grouped* g) {
  g->a = a;
  g->x = {a->x, a->rows, a->k, a->ldx, 0};
  g->w = {a->w, a->groups * a->n, a->k, a->k, 0};
  g->dy = {a->dy, a->rows, a->n, a->lddy, 0};
  g->pack.count = 0;
  Carver c(workspace);
  auto padded = [&](Matrix* m) {
    if (copyable(*m)) return;
    const int64_t ldp = round8(m->cols);
    uint16_t* dst = static_cast<uint16_t*>(c.take(static_cast<size_t>(m->rows) * ldp * 2));
    g->pack.job[g->pack.count++] = {static_cast<const uint16_t*>(m->ptr), dst, m->rows, m->cols, m->ld, ldp};
    m->ptr = dst;
    m->ld = ldp;
  };
  if (a->rows == 0) return 0;
  if (!backward && grouped_few_fits(ops, a)) return 0;  // goes over the operands as they lie
  if (!backward || a->dw) padded(&g->x);
  if (!backward || a->dx) padded(&g->w);
  if (backward && (a->dx || a->dw)) padded(&g->dy);
  if (backward && a->dw) {
    auto tail = [&](const Matrix& m) {
      const int64_t ld = round8(m.cols);
      return Matrix{c.take(static_cast<size_t>(a->groups) * kGroupedTail * ld * 2), kGroupedTail, m.cols, ld,
                    kGroupedTail * ld};
    };
    g->tail_x = tail(g->x);
    g->tail_dy = tail(g->dy);
  }
  g->w.rows = a->n;  // one group's, of a batch
  g->w.batch_stride = a->n * g->w.ld;
  return c.used;
}

gemm_status_t prepare(gemm_ops_t* ops, const gemm_grouped_args_t* a, bool backward, void* workspace, size_t bytes,
                      Grouped* g) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops) return ops_fail(GEMM_ERR_INVALID_ARG, "ops is NULL");
  const gemm_status_t st = check(a, backward);
  if (st != GEMM_OK) return st;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return ops_fail(GEMM_ERR_INVALID_ARG, "the workspace must be 256-byte aligned");
  const size_t need = layout(ops, a, backward, workspace, g);
  if (need > 0 && (!workspace || bytes < need))
    return ops_fail(GEMM_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace ? bytes : 0, need);
  return check_overlap(a, backward, workspace, need);
}

gemm_status_t run_product(const gemm_ops* ops, const Grouped& g, int kind, void* out, cudaStream_t stream) {
  const gemm_grouped_args_t* a = g.a;
  const bool bf16 = a->dtype == GEMM_BF16;
  GroupedParams p{};
  GroupedMaps maps;
  p.offsets = a->offsets;
  p.groups = static_cast<int>(a->groups);
  p.rows = static_cast<int>(a->rows);
  p.reduce = static_cast<int>(kind == kGroupedForward ? a->k : a->n);
  p.lanes = static_cast<int>(kind == kGroupedForward ? a->n : a->k);
  p.cols = static_cast<int>(a->n);
  p.tiles_lane = static_cast<int>(ceil_div(p.lanes, int64_t{kGroupedLanes}));
  p.zero_rest = a->zero_rest;
  p.out = static_cast<uint16_t*>(out);
  p.ldo = p.lanes;
  p.out_group = a->n * a->k;
  p.wide = p.lanes % 2 == 0 && (reinterpret_cast<uintptr_t>(out) & 3u) == 0 ? 1 : 0;
  p.bf16 = bf16 ? 1 : 0;
  p.status = ops->d_status;
  p.timeout_ns = ops->timeout_ns;
  p.inject_fault = ops->debug_fault;

  if (ops->pairs < 1) return ops_fail(GEMM_ERR_UNSUPPORTED, "no CTA pair fits the device");
  p.cap = kGroupedCols;
  int64_t tiles = p.tiles_lane * (a->rows / grouped_cap(kGroupedCaps - 1) + std::min(a->groups, a->rows));  // at most
  if (kind == kGroupedWeight) {
    const int slots = static_cast<int>(a->rows / a->groups / kGroupedK) + 2, strips = static_cast<int>(a->groups) * p.tiles_lane;
    float best = -1.0f;
    for (int i = 0; i < kGroupedCaps; ++i) {
      const int cap = grouped_cap(i), n = strips * grouped_tiles(p.cols, cap);
      const float clocks = grouped_clocks(static_cast<float>(strips) * grouped_strip_clocks(p.cols, cap, slots), n, cap, slots, ops->pairs);
      if (best >= 0.0f && clocks >= best) continue;
      best = clocks;
      tiles = n;
      p.cap = cap;
    }
  }
  p.pairs = static_cast<int>(std::min<int64_t>(ops->pairs, tiles));

  p.stages = kGroupedStages;
  while (p.stages > 1 && grouped_smem_bytes(p.stages, p.groups) > ops->smem_optin) --p.stages;
  const size_t smem = grouped_smem_bytes(p.stages, p.groups);
  if (smem > ops->smem_optin) return ops_fail(GEMM_ERR_SMEM_BUDGET, "no ring fits shared memory");

  const CUtensorMapL2promotion l2 = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  gemm_status_t st;
  if (kind == kGroupedWeight) {
    st = encode_map(&maps.a, bf16, g.x, 1, 64, kGroupedK, l2);
    if (st == GEMM_OK) st = encode_map(&maps.b[0], bf16, g.dy, 1, 64, kGroupedK, l2);
    if (st == GEMM_OK) st = encode_map(&maps.b[1], bf16, g.tail_x, a->groups, 64, kGroupedTail, l2);
    if (st == GEMM_OK) st = encode_map(&maps.b[2], bf16, g.tail_dy, a->groups, 64, kGroupedTail, l2);
    maps.b[3] = maps.b[0];
  } else {
    st = kind == kGroupedForward ? encode_map(&maps.a, bf16, g.w, a->groups, kBK, kBM, l2)
                                 : encode_map(&maps.a, bf16, g.w, a->groups, 64, kGroupedK, l2);
    for (int i = 0; i < 4 && st == GEMM_OK; ++i)
      st = encode_map(&maps.b[i], bf16, kind == kGroupedForward ? g.x : g.dy, 1, kBK, kGroupedTail << i, l2);
  }
  if (st != GEMM_OK) return st;
  const cudaError_t e = grouped_launch(kind, maps, p, smem, stream);
  return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "grouped product launch");
}

template <int kKind>
cudaError_t launch_kind(const GroupedMaps& m, const GroupedParams& p, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(2 * p.pairs, 1, 1);
  cfg.blockDim = dim3(kGroupedThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_kernel<kKind>, m, p);
}

}  // namespace

namespace spgemm {

cudaError_t grouped_set_smem(size_t smem) {
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int bytes = static_cast<int>(smem);
  cudaError_t e = cudaFuncSetAttribute(grouped_kernel<kGroupedForward>, attr, bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_kernel<kGroupedInput>, attr, bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(grouped_kernel<kGroupedWeight>, attr, bytes);
  return e;
}

cudaError_t grouped_launch(int kind, const GroupedMaps& m, const GroupedParams& p, size_t smem,
                           cudaStream_t stream) {
  if (kind == kGroupedForward) return launch_kind<kGroupedForward>(m, p, smem, stream);
  if (kind == kGroupedInput) return launch_kind<kGroupedInput>(m, p, smem, stream);
  return launch_kind<kGroupedWeight>(m, p, smem, stream);
}

}  // namespace spgemm

extern "C" {

gemm_status_t gemm_grouped_workspace(gemm_ops_t* ops, const gemm_grouped_args_t* args, int backward, size_t* bytes) {
  ops_fail(GEMM_OK, "%s", "");
  if (!ops || !bytes) return ops_fail(GEMM_ERR_INVALID_ARG, "NULL argument");
  const gemm_status_t st = check(args, backward != 0);
  if (st != GEMM_OK) return st;
  Grouped g;
  *bytes = layout(ops, args, backward != 0, nullptr, &g);
  return GEMM_OK;
}

gemm_status_t gemm_grouped_run(gemm_ops_t* ops, const gemm_grouped_args_t* args, void* workspace,
                               size_t workspace_bytes, void* stream_handle) {
  Grouped g;
  const gemm_status_t st = prepare(ops, args, false, workspace, workspace_bytes, &g);
  if (st != GEMM_OK || args->rows == 0) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  cudaError_t e;
  if (grouped_few_fits(ops, args)) {
    e = grouped_few_launch(ops, args, stream);
    return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "grouped product launch");
  }
  e = launch_pack(g.pack, ops->sm_count, stream);
  if (e != cudaSuccess) return ops_cuda_fail(e, "padding copy launch");
  return run_product(ops, g, kGroupedForward, args->y, stream);
}

gemm_status_t gemm_grouped_backward(gemm_ops_t* ops, const gemm_grouped_args_t* args, void* workspace,
                                    size_t workspace_bytes, void* stream_handle) {
  Grouped g;
  gemm_status_t st = prepare(ops, args, true, workspace, workspace_bytes, &g);
  if (st != GEMM_OK) return st;
  OpsDevice guard(ops->device);
  if (guard.err != cudaSuccess) return ops_cuda_fail(guard.err, "cudaSetDevice");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_handle);
  if (args->rows == 0) {  // sums over no tokens
    if (!args->dw) return GEMM_OK;
    const cudaError_t e =
        cudaMemsetAsync(args->dw, 0, static_cast<size_t>(2) * args->groups * args->n * args->k, stream);
    return e == cudaSuccess ? GEMM_OK : ops_cuda_fail(e, "cudaMemsetAsync(weight gradients)");
  }
  cudaError_t e = launch_pack(g.pack, ops->sm_count, stream);
  if (e != cudaSuccess) return ops_cuda_fail(e, "padding copy launch");
  if (args->dw) {
    TailJobs jobs;
    const Matrix* from[2] = {&g.x, &g.dy};
    const Matrix* to[2] = {&g.tail_x, &g.tail_dy};
    for (int i = 0; i < 2; ++i)
      jobs.job[i] = {static_cast<const uint16_t*>(from[i]->ptr),
                     static_cast<uint16_t*>(const_cast<void*>(to[i]->ptr)), from[i]->ld, to[i]->ld,
                     static_cast<int>(from[i]->cols)};
    const int64_t blocks = ceil_div(kGroupedTail * ceil_div(std::max(args->n, args->k), int64_t{8}), int64_t{4 * kTailThreads});
    e = launch(tail_kernel, dim3(static_cast<unsigned>(args->groups), static_cast<unsigned>(std::min<int64_t>(blocks, 64)), 2),
               kTailThreads, stream, jobs, args->offsets, args->rows);
    if (e != cudaSuccess) return ops_cuda_fail(e, "group tails launch");
  }
  if (args->dx) st = run_product(ops, g, kGroupedInput, args->dx, stream);
  if (st == GEMM_OK && args->dw) st = run_product(ops, g, kGroupedWeight, args->dw, stream);
  return st;
}

}  // extern "C"
