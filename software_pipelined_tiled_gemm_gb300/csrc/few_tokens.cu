// few_tokens.cu -- the gated block's products for a few tokens.
//
// With so few rows a product is a pass over its weights, and what counts is the
// time around that pass.  A product on TMEM tiles spends 8 to 9 us there:
// barriers, the ring's first fill, a tile's exchange between the CTAs that share
// its K, its epilogue and store.  Here a warp reads its rows of the weights from
// memory straight into the registers of mma.sync (m16n8k16, fp32 sums), tokens
// as columns; the instruction's rate, a fraction of tcgen05's, is far above what
// the memory delivers, and what costs fp32 arithmetic several instructions a
// weight and token costs it none.
//
// A sum over K may take its terms in any order, as long as weights and tokens
// agree: a lane's 16-byte word, eight neighbours of a row, is the operand of two
// instructions, and the same eight elements of a token their other operand.
//
//   gate and up   the instruction's rows are 8 gate rows and the up rows of the
//                 same outputs, so act(G) U needs no exchange;
//   down          16 rows.
//
// A block takes a contiguous share of the rows, so the bytes are shared out
// evenly; its warps take groups of those, or, where there are fewer groups than
// warps, shares of a group's K (added in a fixed order).  The tokens lie in
// shared memory; where they do not fit, a product takes the tiles.  Rows that
// are not 16-byte aligned are read as they lie, a vector from the two words
// around it.
//
// Forward pass in us, here and on tiles (bytes at 6780 GB/s): 4096 / 16384, 1
// token 62 and 74 (59); 2048 / 4096, 1 token 12 and 27 (7), 8 tokens 14 and 27,
// 32 tokens of 1024 / 1024 11 and 19 (1).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "block_math.cuh"
#include "byte_shift.cuh"
#include "few_tokens.h"
#include "ops_internal.h"
#include "ptx.cuh"

namespace spgemm {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
// Steps (a vector of eight weights from each of two rows) that a lane has in
// flight; a vector of an unaligned row takes two words.
constexpr int steps_ahead(bool shifted) { return shifted ? 4 : 8; }

struct Args {
  const uint16_t* x;   // M x K
  int64_t ldx;
  const uint16_t* w;   // rows x K; gated: the up rows follow the gate rows
  int64_t ldw;
  int m, rows, k;
  int share;           // warps of a group
  int x_shifted;       // rows of tokens are not 16-byte aligned
  int weights_ready;   // the previous kernel on the stream has waited for what writes w
  uint16_t* out;       // M x rows
  int64_t ldo;
  float* pre;          // gated: kept projections, or nullptr
  int64_t pre_half;
  int act;
};

// 16-byte words of a token's row in shared memory: an odd multiple of 64 bytes,
// so that the rows of an instruction's tokens lie in different banks.
__host__ __device__ constexpr int token_pitch(int k) { return (k + 63) / 64 * 8 + 4; }

template <bool kBf16>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ float activate(int act, float g) {
  if (act == kActSilu) return gate_act<kActSilu>(g);
  if (act == kActGelu) return gate_act<kActGelu>(g);
  return gate_act<kActRelu>(g);
}

// c += rows (16 x 16) times tokens (16 x 8).
template <bool kBf16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The eight elements from p on (`end`: past the array's last), as the aligned
// words around them.  The second is read only if it holds an element of the
// array; each has one, so both lie in its allocation.
struct Window {
  uint4 lo, hi;
  __device__ __forceinline__ void load(const uint16_t* p, const uint16_t* end, bool in) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p), base = at & ~uintptr_t{15};
    lo = hi = make_uint4(0u, 0u, 0u, 0u);
    if (in) lo = __ldcg(reinterpret_cast<const uint4*>(base));
    if (in && at != base && base + 16 < reinterpret_cast<uintptr_t>(end))
      hi = __ldcg(reinterpret_cast<const uint4*>(base + 16));
  }
  // The first `count` of them, 0 after those.
  __device__ __forceinline__ uint4 get(const uint16_t* p, int count) const {
    const uint4 v = shift_window(lo, hi, static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u));
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (count < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= count) w[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// kTiles: groups of eight tokens.  kShifted: rows of weights that are not
// 16-byte aligned, or of no multiple of eight elements.  The tokens are read
// once, however they lie, so that theirs need no instance.
template <bool kBf16, int kTiles, bool kGated, bool kShifted>
__global__ void __launch_bounds__(kThreads, 1) few_tokens_kernel(const Args a) {
  constexpr int kGroup = kGated ? 8 : 16;  // rows of a group
  constexpr int kSteps = steps_ahead(kShifted);
  extern __shared__ uint4 xs[];  // M rows of token_pitch(k)
  __shared__ float4 partial[kWarps][kTiles][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int vecs = (a.k + 7) / 8, steps = (vecs + 3) / 4;
  const int share = a.share, slots = kWarps / share;
  const int slot = warp / share, part = warp % share;
  const int begin = static_cast<int>(static_cast<int64_t>(steps) * part / share);
  const int end = static_cast<int>(static_cast<int64_t>(steps) * (part + 1) / share);
  const int first_row = static_cast<int>(static_cast<int64_t>(a.rows) * blockIdx.x / gridDim.x);
  const int last_row = static_cast<int>(static_cast<int64_t>(a.rows) * (blockIdx.x + 1) / gridDim.x);
  const int groups = (last_row - first_row + kGroup - 1) / kGroup;
  const int rounds = (groups + slots - 1) / slots;

  // Words of step s0 + i: row g of the group's first eight, and of its others.
  uint4 w[2][kShifted ? 1 : kSteps];
  Window window[2][kShifted ? kSteps : 1];
  const uint16_t* w_end = a.w + (static_cast<int64_t>(kGated ? 2 : 1) * a.rows - 1) * a.ldw + a.k;
  auto each_word = [&](int round, int s0, auto&& f) {
    const int row = first_row + (round * slots + slot) * kGroup + g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool exists = row + (kGated ? 0 : 8 * h) < last_row;
      const uint16_t* src = a.w + (static_cast<int64_t>(row) + (kGated ? h * a.rows : 8 * h)) * a.ldw;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int v = 4 * (s0 + i) + t;
        // Sixteen bytes a step, so that the steps' loads share one address (src +
        // 8 v made each its own: 1 to 2 us a call).
        f(h, i, reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint4*>(src) + v),
          exists && s0 + i < end && v < vecs);
      }
    }
  };
  auto load = [&](int round, int s0) {
    each_word(round, s0, [&](int h, int i, const uint16_t* src, bool in) {
      if constexpr (kShifted)
        window[h][i].load(src, w_end, in);
      else
        w[h][i] = in ? __ldcs(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
    });
  };
  // The first weights come while the previous kernel ends: into registers
  // where that one is known to have waited for whatever writes them, otherwise
  // only into L2.  The next kernel may start once this one has waited.
  int round = 0, s0 = begin;
  if (rounds > 0) {
    if (a.weights_ready)
      load(0, s0);
    else
      each_word(0, s0, [](int, int, const uint16_t* src, bool in) {
        if (in) asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
      });
  }
  ptx::pdl_wait_prior_grid();
  ptx::pdl_launch_dependents();
  if (rounds > 0 && !a.weights_ready) load(0, s0);
  const int pitch = token_pitch(a.k);
  if (kShifted || a.x_shifted) {
    const uint16_t* x_end = a.x + (a.m - 1) * a.ldx + a.k;
#pragma unroll 4
    for (int i = threadIdx.x; i < a.m * vecs; i += kThreads) {
      const int n = i / vecs, v = i - n * vecs;
      const uint16_t* src = a.x + n * a.ldx + 8 * v;
      Window window;
      window.load(src, x_end, true);
      xs[n * pitch + v] = window.get(src, a.k - 8 * v);
    }
  } else {
#pragma unroll 8
    for (int i = threadIdx.x; i < a.m * vecs; i += kThreads) {
      const int n = i / vecs, v = i - n * vecs;
      xs[n * pitch + v] = __ldcg(reinterpret_cast<const uint4*>(a.x + n * a.ldx) + v);
    }
  }
  __syncthreads();

  float acc[kTiles][4];
#pragma unroll
  for (int n = 0; n < kTiles; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
  while (round < rounds) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      uint4 w0, w1;
      if constexpr (kShifted) {
        const int row = first_row + (round * slots + slot) * kGroup + g, k = 8 * (4 * (s0 + i) + t);
        const uint16_t* src = a.w + static_cast<int64_t>(row) * a.ldw + k;
        w0 = window[0][i].get(src, a.k - k);
        w1 = window[1][i].get(src + static_cast<int64_t>(kGated ? a.rows : 8) * a.ldw, a.k - k);
      } else {
        w0 = w[0][i];
        w1 = w[1][i];
      }
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        // Past the end of a warp's share the weights are 0: no token is read there.
        const int v = 4 * (s0 + i) + t;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (8 * n + g < a.m && s0 + i < end && v < vecs) x = xs[(8 * n + g) * pitch + v];
        mma<kBf16>(acc[n], w0.x, w1.x, w0.y, w1.y, x.x, x.y);
        mma<kBf16>(acc[n], w0.z, w1.z, w0.w, w1.w, x.z, x.w);
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

    // The group is complete; add the warps' shares of its K.
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
    const int row = first_row + (done * slots + slot) * kGroup + g;
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int token = 8 * n + 2 * t + e;
        if (part == 0 && token < a.m) {
          uint16_t* out = a.out + token * a.ldo + row;
          if constexpr (kGated) {
            if (row < last_row) {
              if (a.pre != nullptr) {
                a.pre[static_cast<int64_t>(row) * 32 + token] = acc[n][e];
                a.pre[a.pre_half + static_cast<int64_t>(row) * 32 + token] = acc[n][2 + e];
              }
              *out = round16<kBf16>(activate(a.act, acc[n][e]) * acc[n][2 + e]);
            }
          } else {
            if (row < last_row) out[0] = round16<kBf16>(acc[n][e]);
            if (row + 8 < last_row) out[8] = round16<kBf16>(acc[n][2 + e]);
          }
        }
      }
#pragma unroll
    for (int n = 0; n < kTiles; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
  }
}

using Kernel = void (*)(const Args);

template <bool kBf16, bool kGated, bool kShifted>
Kernel kernel_of(int64_t m) {
  return m <= 8    ? few_tokens_kernel<kBf16, 1, kGated, kShifted>
         : m <= 16 ? few_tokens_kernel<kBf16, 2, kGated, kShifted>
                   : few_tokens_kernel<kBf16, 4, kGated, kShifted>;
}

Kernel kernel_of(bool bf16, bool gated, bool shifted, int64_t m) {
  if (shifted) {
    if (bf16) return gated ? kernel_of<true, true, true>(m) : kernel_of<true, false, true>(m);
    return gated ? kernel_of<false, true, true>(m) : kernel_of<false, false, true>(m);
  }
  if (bf16) return gated ? kernel_of<true, true, false>(m) : kernel_of<true, false, false>(m);
  return gated ? kernel_of<false, true, false>(m) : kernel_of<false, false, false>(m);
}

}  // namespace

// Whether whole 16-byte words of the rows can be read where they lie.
bool aligned_rows(const Matrix& m) { return m.cols % 8 == 0 && copyable(m); }

size_t token_bytes(int64_t m, int64_t k) { return static_cast<size_t>(m) * token_pitch(static_cast<int>(k)) * 16; }

// Shared memory for the tokens, beside the partials.
size_t token_limit(int64_t m) {
  const int tiles = m <= 8 ? 1 : m <= 16 ? 2 : 4;
  return 226 * 1024 - sizeof(float4) * kWarps * 32 * tiles;
}

// Up to eight tokens wherever they fit.  Each eight more are another pair of
// instructions and another read of shared memory a word, and a long pass is
// then bound by those: 9 to 16 tokens up to 256 MB of weights (us here and on
// tiles: 36 and 51 where gate and up are 108 MB, 73 and 74 at 268 MB, 135 to
// 159 and 132 at 537 MB), 17 to 32 up to 48 MB (23 and 27 at 34 MB, 90 and 74
// at 268 MB).
//
// Rows of weights that are not 16-byte aligned cost twice the loads here, and a
// padded copy of all weights on tiles: up to eight tokens always gain (1 of
// 2049 / 2051 23 and 45, of 4095 / 8193 81 and 122), 9 to 16 where what they
// fill of shared memory is below 160 KB (16 of 4095 / 4097, 132 KB, 68 and 80;
// 12 of 6045 / 1617, 146 KB, 52 and 63; 16 of those, 195 KB, 76 and 63), 17 to
// 32 there up to 32 MB of weights (17 tokens where gate and up are 25 MB 44 and
// 53, 39 MB 64 and 61, 49 MB 72 and 67).
bool few_tokens_fits(const gemm_ops* ops, int64_t m, int64_t rows, const Matrix& w) {
  const int64_t k = w.cols, limit = int64_t{1} << 20;
  const bool aligned = aligned_rows(w);
  const int64_t most = m <= 8 ? kOpsMaxDim * limit : m <= 16 ? 256 * limit : (aligned ? 48 : 32) * limit;
  if (m < 1 || m > kFewTokens || k > kOpsMaxDim - 64 || ops->smem_optin < 227 * 1024) return false;
  return 2 * rows * k <= most && token_bytes(m, k) <= (aligned || m <= 8 ? token_limit(m) : 160 * 1024);
}

cudaError_t few_tokens_init(const gemm_ops* ops) {
  cudaError_t e = cudaSuccess;
  if (ops->smem_optin < 227 * 1024) return e;  // not used
  for (int n = 0; n < 24 && e == cudaSuccess; ++n) {
    const int m = n < 8 ? 8 : n < 16 ? 16 : 32;
    e = cudaFuncSetAttribute(kernel_of((n & 1) != 0, (n & 2) != 0, (n & 4) != 0, m), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(token_limit(m)));
  }
  return e;
}

cudaError_t few_tokens_launch(const gemm_ops* ops, const FewTokens& f, cudaStream_t stream) {
  Args a{};
  a.x = static_cast<const uint16_t*>(f.x.ptr);
  a.ldx = f.x.ld;
  a.w = static_cast<const uint16_t*>(f.w.ptr);
  a.ldw = f.w.ld;
  a.m = static_cast<int>(f.x.rows);
  a.rows = static_cast<int>(f.rows);
  a.k = static_cast<int>(f.x.cols);
  a.out = f.out;
  a.ldo = f.ldo;
  a.pre = f.pre;
  a.pre_half = f.rows * 32;
  a.act = f.act;
  a.weights_ready = f.weights_ready ? 1 : 0;
  // Warps of a group: as many as the block has for its groups, while each has
  // words to read.
  const int64_t groups = ceil_div(ceil_div(f.rows, ops->sm_count), f.gated ? 8 : 16);
  a.share = 1;
  while (a.share < kWarps && groups * a.share * 2 <= kWarps && ceil_div(f.x.cols, 32) >= a.share * 2)
    a.share *= 2;
  const bool shifted = !aligned_rows(f.w);
  a.x_shifted = aligned_rows(f.x) ? 0 : 1;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(ops->sm_count, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = token_bytes(f.x.rows, f.x.cols);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel_of(f.bf16, f.gated, shifted, f.x.rows), a);
}

}  // namespace spgemm
