// grouped_few.cu -- the products grouped by expert for a few rows a group.
//
// With one or a few rows a group a product is a pass over the weights of the
// groups that have rows, as in few_tokens.cu (see there for the instruction and
// the operands' order): a warp reads rows of the weights from memory straight
// into the registers of mma.sync, tokens as columns, whether or not the rows are
// 16-byte aligned.  What differs: every block reads the offsets and lists the
// groups that have rows; the rows of their weights, one group after another, are
// shared out evenly over the blocks, so a block's share may end inside one group
// and begin inside another.  A group with more tokens than shared memory (or the
// instance) holds takes several passes over the share.
//
// Bound by the weights' bytes: 8 rows over 64 experts of 2048 x 4096 (134 MB of
// weights used) take 25.7 us in a stream of calls (5.2 TB/s), on TMEM tiles 29 us.
// Unaligned weights save the padded copy of all of them, which moves three times
// their bytes.
#include <algorithm>

#include "../../include/gemm_ops.h"
#include "few_tokens.cuh"
#include "gemm_kernel.cuh"
#include "grouped_few.h"

namespace spgemm {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int steps_ahead(bool shifted) { return shifted ? 4 : 8; }

struct Args {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* w;   // groups x n x k, dense
  uint16_t* y;         // rows x n, dense
  const int64_t* offsets;
  int groups, n, k;
  int64_t rows;
  int tokens;          // that shared memory holds, at most 8 kTiles
  int zero_rest;
  int x_shifted;       // rows of tokens are not 16-byte aligned
  int* status;
};

// kTiles: groups of eight tokens.  kShifted: rows of weights that are not
// 16-byte aligned, or of no multiple of eight elements.
template <bool kBf16, int kTiles, bool kShifted>
__global__ void __launch_bounds__(kThreads, 1) grouped_few_kernel(const Args a) {
  constexpr int kSteps = steps_ahead(kShifted);
  extern __shared__ uint4 xs[];  // tokens of token_pitch(k), then the list of groups with rows
  __shared__ float4 partial[kWarps][kTiles][32];
  __shared__ int found;
  const int pitch = token_pitch(a.k);
  int* list = reinterpret_cast<int*>(xs + static_cast<size_t>(a.tokens) * pitch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int vecs = (a.k + 7) / 8, steps = (vecs + 3) / 4;
  const uint16_t* w_end = a.w + static_cast<int64_t>(a.groups) * a.n * a.k;

  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();
  int bad = 0;
  for (int e = threadIdx.x; e <= a.groups; e += kThreads) {
    const int64_t at = a.offsets[e], next = e < a.groups ? a.offsets[e + 1] : a.rows;
    bad |= at < 0 || at > next || next > a.rows;
  }
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && threadIdx.x == 0)
      record_error(a.status, static_cast<int>(GEMM_ERR_INVALID_ARG), GEMM_CHECK_OFFSETS);
    return;
  }
  if (warp == 0) {
    int count = 0;
    for (int e0 = 0; e0 < a.groups; e0 += 32) {
      const int e = e0 + lane;
      const bool some = e < a.groups && a.offsets[e + 1] > a.offsets[e];
      const uint32_t votes = __ballot_sync(0xffffffffu, some);
      if (some) list[count + __popc(votes & ((1u << lane) - 1u))] = e;
      count += __popc(votes);
    }
    if (lane == 0) found = count;
  } else if (a.zero_rest) {
    const int64_t first = a.offsets[0], last = a.offsets[a.groups], rest = first + (a.rows - last);
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kWarps - 1) + warp - 1; i < rest;
         i += static_cast<int64_t>(gridDim.x) * (kWarps - 1)) {
      uint16_t* dst = a.y + (i < first ? i : last + (i - first)) * a.n;
      for (int c = lane; c < a.n; c += 32) dst[c] = 0;
    }
  }
  __syncthreads();

  const int64_t all = static_cast<int64_t>(found) * a.n;
  int64_t at = all * blockIdx.x / gridDim.x;
  const int64_t share_end = all * (blockIdx.x + 1) / gridDim.x;
  while (at < share_end) {
    // The part of this block's share that is one group's: rows [first_row, last_row) of its weights.
    const int index = static_cast<int>(at / a.n);
    const int first_row = static_cast<int>(at - static_cast<int64_t>(index) * a.n);
    const int last_row = static_cast<int>(min(static_cast<int64_t>(a.n), first_row + (share_end - at)));
    at += last_row - first_row;
    const int e = list[index];
    const int64_t token0 = a.offsets[e], token_end = a.offsets[e + 1];
    const uint16_t* we = a.w + static_cast<int64_t>(e) * a.n * a.k;
    // Warps of 16 rows: as many as the block has for them, while each has words to read.
    const int sets = (last_row - first_row + 15) / 16;
    int share = 1;
    while (share < kWarps && sets * share * 2 <= kWarps && steps >= share * 8) share *= 2;
    const int slots = kWarps / share, slot = warp / share, part = warp % share;
    const int begin = static_cast<int>(static_cast<int64_t>(steps) * part / share);
    const int end = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / share);
    const int rounds = (sets + slots - 1) / slots;

    uint4 w[2][kShifted ? 1 : kSteps];
    Window window[2][kShifted ? kSteps : 1];
    auto load = [&](int round, int s0) {
      const int row = first_row + (round * slots + slot) * 16 + g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool exists = row + 8 * h < last_row;
        const uint16_t* src = we + (static_cast<int64_t>(row) + 8 * h) * a.k;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int v = 4 * (s0 + i) + t;
          const uint16_t* p = reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint4*>(src) + v);
          const bool in = exists && s0 + i < end && v < vecs;
          if constexpr (kShifted)
            window[h][i].load(p, w_end, in);
          else
            w[h][i] = in ? __ldcs(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    for (int64_t token = token0; token < token_end; token += a.tokens) {
      const int m = static_cast<int>(min(static_cast<int64_t>(a.tokens), token_end - token));
      int round = 0, s0 = begin;
      if (rounds > 0) load(0, s0);
      const uint16_t* x = a.x + token * a.ldx;
      __syncthreads();  // the tokens before these have been read
      if (kShifted || a.x_shifted) {
        const uint16_t* x_end = a.x + (a.rows - 1) * a.ldx + a.k;
#pragma unroll 4
        for (int i = threadIdx.x; i < m * vecs; i += kThreads) {
          const int n = i / vecs, v = i - n * vecs;
          const uint16_t* src = x + n * a.ldx + 8 * v;
          Window one;
          one.load(src, x_end, true);
          xs[n * pitch + v] = one.get(src, a.k - 8 * v);
        }
      } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < m * vecs; i += kThreads) {
          const int n = i / vecs, v = i - n * vecs;
          xs[n * pitch + v] = __ldcg(reinterpret_cast<const uint4*>(x + n * a.ldx) + v);
        }
      }
      __syncthreads();

      float acc[kTiles][4];
#pragma unroll
      for (int n = 0; n < kTiles; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[n][c] = 0.0f;
      while (round < rounds) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          uint4 w0, w1;
          if constexpr (kShifted) {
            const int row = first_row + (round * slots + slot) * 16 + g, k = 8 * (4 * (s0 + i) + t);
            const uint16_t* src = we + static_cast<int64_t>(row) * a.k + k;
            w0 = window[0][i].get(src, a.k - k);
            w1 = window[1][i].get(src + static_cast<int64_t>(8) * a.k, a.k - k);
          } else {
            w0 = w[0][i];
            w1 = w[1][i];
          }
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            // Past the end of a warp's share the weights are 0: no token is read there.
            const int v = 4 * (s0 + i) + t;
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (8 * n + g < m && s0 + i < end && v < vecs) u = xs[(8 * n + g) * pitch + v];
            mma<kBf16>(acc[n], w0.x, w1.x, w0.y, w1.y, u.x, u.y);
            mma<kBf16>(acc[n], w0.z, w1.z, w0.w, w1.w, u.z, u.w);
          }
        }
        const int done = round;
        s0 += kSteps;
        if (s0 >= end) {
          s0 = begin;
          ++round;
        }
        if (round < rounds) load(round, s0);
        if (round == done) continue;

        // Sixteen rows are complete; add the warps' shares of their K.
        if (share > 1) {
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
            partial[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
          __syncthreads();
          if (part == 0)
            for (int s = 1; s < share; ++s)
#pragma unroll
              for (int n = 0; n < kTiles; ++n) {
                const float4 v = partial[warp + s][n][lane];
                acc[n][0] += v.x;
                acc[n][1] += v.y;
                acc[n][2] += v.z;
                acc[n][3] += v.w;
              }
          if (round < rounds) __syncthreads();  // read before the next round's
        }
        const int row = first_row + (done * slots + slot) * 16 + g;
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int i = 8 * n + 2 * t + c;
            if (part == 0 && i < m) {
              uint16_t* out = a.y + (token + i) * a.n + row;
              if (row < last_row) out[0] = round16<kBf16>(acc[n][c]);
              if (row + 8 < last_row) out[8] = round16<kBf16>(acc[n][2 + c]);
            }
          }
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[n][c] = 0.0f;
      }
    }
  }
}

using Kernel = void (*)(const Args);

// (Aligned weights come here with two rows a group at most: `two` is never set for them.)
Kernel kernel_of(bool bf16, bool two, bool shifted) {
  if (!shifted) return bf16 ? grouped_few_kernel<true, 1, false> : grouped_few_kernel<false, 1, false>;
  return bf16 ? (two ? grouped_few_kernel<true, 2, true> : grouped_few_kernel<true, 1, true>)
              : (two ? grouped_few_kernel<false, 2, true> : grouped_few_kernel<false, 1, true>);
}

bool aligned_rows(const Matrix& m) { return m.cols % 8 == 0 && copyable(m); }

// Shared memory for tokens and the list of groups, beside the partials.
size_t few_smem(const gemm_ops* ops) { return ops->smem_optin - sizeof(float4) * kWarps * 32 * 2 - 64; }

int tokens_that_fit(const gemm_ops* ops, int64_t groups, int64_t k) {
  const size_t row = static_cast<size_t>(token_pitch(static_cast<int>(k))) * 16, list = 4u * static_cast<size_t>(groups);
  return static_cast<int>(std::min<size_t>(16, (few_smem(ops) - list) / row));
}

}  // namespace

// Aligned weights: up to two rows a group (above, TMEM tiles reach the memory's
// rate too); others, whose padded copy is saved, up to eight.  Measured, in us, these
// passes and TMEM tiles, by rows a group:
//   16 x 2048 x 4096    1: 37, 50    2: 48, 52    4: 60, 54
//   16 x 2047 x 4095    1: 82, 136   8: 107, 144  12: 179, 144
//   64 x 1023 x 1021    1: 52, 72    8: 76, 80    12: 109, 80
// That is with rows evenly spread.  The host does not know how they are: where one group has
// all of them, each 8 (16) rows are another pass over its weights.  64 x 2048 x 4096 with 128
// rows: 181, 170 evenly spread, 55, 21 in one group; 64 x 1023 x 1021 with 512: 70, 77 and
// 146, 60; 1024 x 512 x 512 with 2048: 85, 99 and 471, 18.
bool grouped_few_fits(const gemm_ops* ops, const gemm_grouped_args_t* a) {
  const Matrix w{a->w, a->groups * a->n, a->k, a->k, 0};
  const int64_t most = (aligned_rows(w) ? 2 : 8) * a->groups;
  return a->rows <= most && a->k <= kOpsMaxDim - 64 && ops->smem_optin >= 227 * 1024 && ops->debug_fault == 0 &&
         tokens_that_fit(ops, a->groups, a->k) >= 1;
}

cudaError_t grouped_few_init(const gemm_ops* ops) {
  cudaError_t e = cudaSuccess;
  if (ops->smem_optin < 227 * 1024) return e;  // not used
  for (int i = 0; i < 6 && e == cudaSuccess; ++i)
    e = cudaFuncSetAttribute(kernel_of((i & 1) != 0, i >= 4, i >= 2), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(few_smem(ops)));
  return e;
}

cudaError_t grouped_few_launch(const gemm_ops* ops, const gemm_grouped_args_t* a, cudaStream_t stream) {
  const Matrix w{a->w, a->groups * a->n, a->k, a->k, 0}, x{a->x, a->rows, a->k, a->ldx, 0};
  Args p{};
  p.x = static_cast<const uint16_t*>(a->x);
  p.ldx = a->ldx;
  p.w = static_cast<const uint16_t*>(a->w);
  p.y = static_cast<uint16_t*>(a->y);
  p.offsets = a->offsets;
  p.groups = static_cast<int>(a->groups);
  p.n = static_cast<int>(a->n);
  p.k = static_cast<int>(a->k);
  p.rows = a->rows;
  // Two tiles of eight tokens where a group may well have more than eight.
  const bool two = a->rows > 8 && a->rows > 2 * a->groups;
  p.tokens = std::min(two ? 16 : 8, tokens_that_fit(ops, a->groups, a->k));
  p.zero_rest = a->zero_rest;
  p.x_shifted = aligned_rows(x) ? 0 : 1;
  p.status = ops->d_status;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(ops->sm_count, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.tokens) * token_pitch(p.k) * 16 + 4u * static_cast<size_t>(a->groups);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel_of(a->dtype == GEMM_BF16, two, !aligned_rows(w)), p);
}

}  // namespace spgemm
