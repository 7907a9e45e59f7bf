// orthogonal_small.cu -- the orthogonalised update of matrices whose short
// side is at most 256, in one launch with the iterate on chip.
//
// With Z the matrix laid with its short side s down (Z = G, or G^T of a tall
// one; the iteration commutes with transposition) and l its long side, each
// step is A = Z Z^T, B = b A + c A^2, Z' = a Z + B Z.  A cluster of CTAs holds
// Z in shared memory, each its own columns, for all steps.  A^2 and B Z need
// only those columns and the s x s matrix, which every CTA keeps and squares
// for itself; A sums over the long side, so with more than one CTA the fp32
// partials go through L2: each CTA adds a share of A's elements in CTA order
// and all read the fp16 sums back.  Only blocks on and above the diagonal are
// multiplied, the rest is mirrored.
//
// Where six panels or fewer are a CTA's, what rounding the iterate to fp16
// loses is kept beside it (kLow) and carried in the term a Z: its errors along
// small singular values grow up to a^5 = 480 times, so that of 8 x 8 or 64 x 64
// matrices a few end several times further off than the mean.  It costs 3 us;
// 64 x 64 ends 1.9e-3 from the exact result, of which 1.65e-3 is bf16's.
//
// Latency is what bounds it: separate products spend 5 to 7.5 us a launch on
// matrices of this size, nearly all of it launch, first copies and the last
// store.  Here a step on one CTA is three bursts of tcgen05.mma with an
// epilogue each: 128 x 128, 6,000 cycles a step (3.2 us) and 20 us for five
// steps (15 products and 2 passes: 93 us); 128 x 512, 9,000 cycles and 39 us.
// A step of 256 x 640 on four CTAs takes 29,000 cycles: products 9,000,
// epilogues 5,000, and 15,000 for the exchange, of which the 192 KB of
// partials leave an SM at its 32 bytes a cycle in 6,200.
//
// Shared memory: 64-column panels, rows of 128 bytes, 128-byte swizzle, of
// the s x s matrix (A, then B in its place) and of Z.  A panel serves as a
// K-major operand (A = Z Z^T contracts over its columns) and as an MN-major
// one (B Z contracts over its rows) where it lies.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "gemm_kernel.cuh"
#include "ops_internal.h"
#include "orthogonal_load.cuh"
#include "orthogonal_small.h"
#include "ptx_block.cuh"

namespace spgemm {

namespace {

// Warps: four lane quarters x kGroups groups of columns.
constexpr int kGroups = 4, kThreads = 128 * kGroups;

// R: row blocks of 128 of the padded short side.
template <int R>
struct Small {
  static constexpr int kSide = 128 * R;
  static constexpr uint32_t kPanel = kSide * 128u;
  static constexpr uint32_t kSquare = 2u * R * kPanel;        // the s x s matrix
  static constexpr int kPanels = small_newton_panels(R);      // of Z in a CTA, at most
  static constexpr int kCols = R == 1 ? 128 : 384;            // accumulator columns of A's upper blocks
  static constexpr int kElems = kCols * 128;
  // As many as leave room for the iterate's low parts (kLow).
  static constexpr int kLowPanels = R == 1 ? 6 : 0;
  static constexpr uint32_t kBytes = kSquare + (R == 1 ? 2 * kLowPanels : kPanels) * kPanel;
};

// Byte offset of element (row, col) from the first panel.
template <int R>
__device__ __forceinline__ uint32_t element(int row, int col) {
  return static_cast<uint32_t>(col >> 6) * Small<R>::kPanel + static_cast<uint32_t>(row) * 128u +
         (((static_cast<uint32_t>(col) >> 3 & 7u) ^ (static_cast<uint32_t>(row) & 7u)) << 4) +
         (static_cast<uint32_t>(col) & 7u) * 2u;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_bf162(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// What two values rounded to `high` lost.
__device__ __forceinline__ uint32_t low_half2(uint32_t high, float lo, float hi) {
  const float2 f = unpack_half2(high);
  return pack_half2(lo - f.x, hi - f.y);
}

// How a CTA's part of Z is read from G, in items of which neighbouring threads
// take neighbours: aligned 16-byte words of a row; eight elements of a column
// of a tall G; or single elements of a row.
enum Access { kWords, kColumns, kElements };

// Calls f(values, row, panel column) for this thread's items of columns
// [first, first + 64 panels) of Z; what lies outside G is 0.  The loops are
// short: each is run once or twice a launch, on a cold instruction cache
// (sixteen items of straight-line code took twice as long as eight).  Loads
// have no branch, so that the next need not wait for them.
template <typename T, int R, int kAccess, typename F>
__device__ __forceinline__ void read_slice(const SmallNewton& p, const T* g, int64_t first, int panels, F&& f) {
  constexpr int kSide = Small<R>::kSide;
  const int t = threadIdx.x;
  if constexpr (kAccess == kColumns) {
    constexpr int kParts = kThreads / kSide;
    const int row = t % kSide;
    const T* src = g + (row < p.s ? row : 0);
#pragma unroll 2
    for (int c = t / kSide * 8; c < panels * 64; c += 8 * kParts) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in = row < p.s && first + c + i < p.l;
        const float x = to_float<T>(__ldg(src + (in ? (first + c + i) * p.ld : 0)));
        v[i] = in ? x : 0.0f;
      }
      f(v, row, c);
    }
  } else {
    constexpr int kCount = kAccess == kWords ? 16 / sizeof(T) : 1;
    constexpr int kInRow = 64 / kCount, kRows = kThreads / kInRow;
    for (int n = 0; n < panels; ++n) {
      const int c = 64 * n + t % kInRow * kCount;
      const bool in_row = first + c < p.l;  // a word: whole, l is a multiple of it
      const T* src = g + (in_row ? first + c : 0);
#pragma unroll 4
      for (int row = t / kInRow; row < kSide; row += kRows) {
        const bool in = in_row && row < p.s;
        const T* at = src + (in ? row * p.ld : 0);
        float v[kCount];
        if constexpr (kCount == 1) {
          const float x = to_float<T>(__ldg(at));
          v[0] = in ? x : 0.0f;
        } else {
          const uint4 w = __ldg(reinterpret_cast<const uint4*>(at));
          const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
          for (int i = 0; i < kCount; ++i) v[i] = in ? to_float<T>(e[i]) : 0.0f;
        }
        f(v, row, c);
      }
    }
  }
}

// Z's rows to a wide output, in units of W (l is a multiple of its elements).
template <int R, typename W>
__device__ __forceinline__ void store_rows(const SmallNewton& p, uint16_t* out, const uint8_t* z, int64_t first,
                                           int elements) {
  constexpr int kUnit = sizeof(W) / 2, kInRow = 64 / kUnit;
#pragma unroll 4
  for (int v = threadIdx.x; v < elements / kUnit; v += kThreads) {
    const int row = v / kInRow % Small<R>::kSide;
    const int col = v / (kInRow * Small<R>::kSide) * 64 + v % kInRow * kUnit;
    if (row < p.s && first + col < p.l)
      *reinterpret_cast<W*>(out + static_cast<int64_t>(row) * p.l + first + col) =
          *reinterpret_cast<const W*>(z + element<R>(row, col));
  }
}

// Calls f(matrix m of G in its type, how it is read).
template <typename F>
__device__ __forceinline__ void with_type(const SmallNewton& p, int m, F&& f) {
  const int64_t at = m * p.g_batch;
  auto call = [&](auto* g) {
    if (p.tall)
      f(g, std::integral_constant<int, kColumns>{});
    else if (p.aligned && p.l % (16 / sizeof(*g)) == 0)
      f(g, std::integral_constant<int, kWords>{});
    else
      f(g, std::integral_constant<int, kElements>{});
  };
  if (p.type == GEMM_IN_F32)
    call(static_cast<const float*>(p.g) + at);
  else if (p.type == GEMM_IN_BF16)
    call(static_cast<const __nv_bfloat16*>(p.g) + at);
  else
    call(static_cast<const __half*>(p.g) + at);
}

// The block right of the first diagonal block of the s x s matrix, from the
// one below it: a thread transposes an 8 x 8 tile.  Neighbouring threads take
// tiles along a diagonal, so neither reads nor writes meet in a bank.
__device__ __forceinline__ void mirror_block(uint8_t* square) {
  if (threadIdx.x >= 256) return;  // one tile a thread
  const int tc = threadIdx.x & 15, u = threadIdx.x >> 4, tr = (u & 8) | ((u + tc) & 7);
  uint32_t w[8][4];  // row j, columns 2 i and 2 i + 1
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 x = *reinterpret_cast<const uint4*>(square + element<2>(128 + 8 * tr + j, 8 * tc));
    w[j][0] = x.x;
    w[j][1] = x.y;
    w[j][2] = x.z;
    w[j][3] = x.w;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // column j of the tile
    uint32_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = __byte_perm(w[2 * i][j >> 1], w[2 * i + 1][j >> 1], j & 1 ? 0x7632 : 0x5410);
    *reinterpret_cast<uint4*>(square + element<2>(8 * tc + j, 128 + 8 * tr)) =
        make_uint4(t[0], t[1], t[2], t[3]);
  }
}

// This CTA's share of A: the cluster's partials of each element added in CTA
// order, several vectors' loads in flight.
template <int R, int C>
__device__ __forceinline__ void add_partials(const float* parts, uint16_t* gram, int rank, float alpha) {
  constexpr int kVectors = Small<R>::kElems / 4, kN = 48 / kGroups / C;
  const int v1 = kVectors * (rank + 1) / C;
#pragma unroll 1
  for (int v0 = kVectors * rank / C + threadIdx.x; v0 < v1; v0 += kThreads * kN) {
    float4 x[kN][C];
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)  // past the end: the last vector again, not used
        x[i][c] = __ldcg(reinterpret_cast<const float4*>(parts + c * Small<R>::kElems) +
                         min(v0 + i * kThreads, v1 - 1));
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      float4 t = x[i][0];
#pragma unroll
      for (int c = 1; c < C; ++c) {
        t.x += x[i][c].x;
        t.y += x[i][c].y;
        t.z += x[i][c].z;
        t.w += x[i][c].w;
      }
      if (v0 + i * kThreads < v1)
        __stcg(reinterpret_cast<uint2*>(gram) + v0 + i * kThreads,
               make_uint2(pack_half2(alpha * t.x, alpha * t.y), pack_half2(alpha * t.z, alpha * t.w)));
    }
  }
}

template <int R, bool kLow>
__global__ void __launch_bounds__(kThreads, 1) small_newton_kernel(const __grid_constant__ SmallNewton p) {
  using K = Small<R>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ double shared[kThreads / 32];
  __shared__ float shared_scale;
  __shared__ float diag[K::kSide];  // of B, in fp32 (see orthogonal.cu); 0 in the square
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  uint8_t* square = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  uint8_t* z = square + K::kSquare;
  uint8_t* z_low = z + K::kLowPanels * K::kPanel;
  const uint32_t square_addr = ptx::smem_addr(square), z_addr = square_addr + K::kSquare;
  const uint32_t bar = square_addr + K::kBytes;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(square + K::kBytes + 8u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, group = warp >> 2;
  const int C = p.cluster;
  const int rank = C > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int slot = static_cast<int>(blockIdx.x) / C, slots = static_cast<int>(gridDim.x) / C;
  const int total = (p.l + 63) / 64;
  const int panel0 = total * rank / C, panels = total * (rank + 1) / C - panel0;
  if (SPGEMM_OUT_OF_BOUNDS((square_addr - raw_addr) + K::kBytes + 16u <= ptx::dynamic_smem_bytes() &&
                               total <= C * K::kPanels && p.s <= K::kSide,
                           p.base, kCheckSmemLayout))
    return;

  if (threadIdx.x == 0) {
    ptx::mbar_init(bar, 1);
    ptx::fence_barrier_init();
  }
  __syncwarp();
  if (warp == 0) {
    ptx::tmem_alloc<1>(ptx::smem_addr(tmem_slot), 512u);
    ptx::tmem_relinquish<1>();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(q * 32) << 16);
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();

  uint32_t phase = 0;
  bool ok = true;        // the same in every thread of the CTA
  bool hook = p.base.inject_fault == 1 && blockIdx.x == 0;
  // One burst of products by thread 0, on shared memory that all threads have
  // written and TMEM that all have read, and the wait for its end.
  auto multiply = [&](auto&& issue) {
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (ok) {
      if (threadIdx.x == 0 && !hook) {  // test hook: the first burst never starts
        ptx::tc_fence_after_sync();
        issue();
        ptx::mma_commit<1>(bar);
      }
      hook = false;
      __syncwarp();
      const bool done = wait_bounded(bar, phase, p.base, kDetailMmaFull);
      phase ^= 1u;
      ok = __syncthreads_and(done) != 0;
    }
    ptx::tc_fence_after_sync();
  };
  // Accumulator columns of A's (B's) row block i, which begin at column 128 i.
  constexpr uint32_t kRow1 = K::kSide;
  const float inv = 1.0f / kIterateScale;
  double* norms = p.norms + static_cast<int64_t>(slot) * C;
  float* parts = p.parts + static_cast<int64_t>(slot) * C * K::kElems;
  uint16_t* gram = p.gram + static_cast<int64_t>(slot) * K::kElems;
  const int64_t first = static_cast<int64_t>(panel0) * 64;
  const int elements = panels * K::kSide * 64;

  for (int m = slot; m < p.batch; m += slots) {
    // Z = 2^8 G / max(|G|, eps).
    SquareSum squares;
    with_type(p, m, [&](auto* g, auto access) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(g)>>;
      read_slice<T, R, decltype(access)::value>(p, g, first, panels, [&](const auto& v, int, int) {
        for (float x : v) squares.mid = fmaf(x, x, squares.mid);
      });
    });
    double sum = squares.block_total<kThreads>(shared);
    if (!__syncthreads_and(threadIdx.x > 0 || plain_sum_holds(sum))) {
      squares = SquareSum();
      with_type(p, m, [&](auto* g, auto access) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(g)>>;
        read_slice<T, R, decltype(access)::value>(p, g, first, panels, [&](const auto& v, int, int) {
          for (float x : v) squares.add<T>(x);
        });
      });
      sum = squares.block_total<kThreads>(shared);
    }
    if (C > 1) {
      if (threadIdx.x == 0) norms[rank] = sum;
      __syncwarp();
      ptx::cluster_sync();
      if (threadIdx.x == 0) {
        sum = 0.0;
        for (int c = 0; c < C; ++c) sum += __ldcg(norms + c);
      }
    }
    if (threadIdx.x == 0) shared_scale = half_scale(sum, p.eps);
    __syncthreads();
    const float scale = shared_scale;
    with_type(p, m, [&](auto* g, auto access) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(g)>>;
      constexpr int kAccess = decltype(access)::value;
      read_slice<T, R, kAccess>(p, g, first, panels, [&](const auto& v, int row, int col) {
        uint8_t* dst = z + element<R>(row, col);
        constexpr int kCount = sizeof(v) / sizeof(float);
        if constexpr (kCount == 1) {
          const float x = v[0] * scale * scale;
          const __half high = __float2half_rn(x);
          *reinterpret_cast<__half*>(dst) = high;
          if (kLow)
            *reinterpret_cast<__half*>(z_low + element<R>(row, col)) = __float2half_rn(x - __half2float(high));
        } else {
#pragma unroll
          for (int j = 0; j < kCount; j += 4) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = v[j + e] * scale * scale;
            const uint2 high = make_uint2(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]));
            *reinterpret_cast<uint2*>(dst + 2 * j) = high;
            if (kLow)
              *reinterpret_cast<uint2*>(z_low + element<R>(row, col) + 2 * j) =
                  make_uint2(low_half2(high.x, x[0], x[1]), low_half2(high.y, x[2], x[3]));
          }
        }
      });
    });

    for (int step = 0; step < p.steps; ++step) {
      const bool last = step + 1 == p.steps;
      // A = Z Z^T over this CTA's columns.
      multiply([&] {
        for (int i = 0; i < R; ++i) {
          const uint32_t idesc = ptx::instr_desc_f16(128, K::kSide - 128 * i, false);
          for (int n = 0; n < panels; ++n) {
            const uint64_t d = ptx::smem_desc_k_sw128(z_addr + n * K::kPanel + i * 16384u);
            for (int k = 0; k < 4; ++k)
              ptx::mma_f16_ss<1>(tmem + i * kRow1, d + 2u * k, d + 2u * k, idesc, (n | k) != 0);
          }
        }
      });
      const float alpha = inv * inv;
      if (C == 1) {
        for (int i = 0; i < R; ++i) {
          const int row = i * 128 + q * 32 + lane;
#pragma unroll 1
          for (int c = group * 16; c < K::kSide - 128 * i; c += 16 * kGroups) {
            uint32_t r[16], w[8];
            ptx::tmem_ld_32x32b_x16(t_lane + i * kRow1 + c, r);
            ptx::tmem_wait_ld();
            const int col = 128 * i + c;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              w[j] = pack_half2(alpha * __uint_as_float(r[2 * j]), alpha * __uint_as_float(r[2 * j + 1]));
            *reinterpret_cast<uint4*>(square + element<R>(row, col)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(square + element<R>(row, col + 8)) = make_uint4(w[4], w[5], w[6], w[7]);
            if (R == 2 && i == 0 && c >= 128) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                *reinterpret_cast<uint16_t*>(square + element<R>(col + j, row)) =
                    static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
            }
          }
        }
      } else {
        // Partials: accumulator column by column, 128 rows each.
        for (int i = 0; i < R; ++i) {
          float* dst = parts + static_cast<int64_t>(rank) * K::kElems + i * kRow1 * 128 + q * 32 + lane;
#pragma unroll 1
          for (int c = group * 32; c < K::kSide - 128 * i; c += 32 * kGroups) {
            uint32_t r[32];
            ptx::tmem_ld_32x32b_x32(t_lane + i * kRow1 + c, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) __stcg(dst + (c + j) * 128, __uint_as_float(r[j]));
          }
        }
        ptx::cluster_sync();
        switch (C) {
          case 2: add_partials<R, 2>(parts, gram, rank, alpha); break;
          case 3: add_partials<R, 3>(parts, gram, rank, alpha); break;
          case 4: add_partials<R, 4>(parts, gram, rank, alpha); break;
          case 5: add_partials<R, 5>(parts, gram, rank, alpha); break;
          case 6: add_partials<R, 6>(parts, gram, rank, alpha); break;
          case 7: add_partials<R, 7>(parts, gram, rank, alpha); break;
          default: add_partials<R, 8>(parts, gram, rank, alpha); break;
        }
        ptx::cluster_sync();
        // Element (row, col) of a block is element (col, row) of its mirror
        // image: eight rows of a column are eight columns of a row there.
        constexpr int kRead = 16 / kGroups;
#pragma unroll 1
        for (int v0 = threadIdx.x; v0 < K::kElems / 8; v0 += kThreads * kRead) {
          uint4 x[kRead];
#pragma unroll
          for (int n = 0; n < kRead; ++n) {
            const int v = v0 + n * kThreads;
            x[n] = __ldcg(reinterpret_cast<const uint4*>(gram) + v);
          }
#pragma unroll
          for (int n = 0; n < kRead; ++n) {
            const int v = v0 + n * kThreads, ac = v / 16;
            const int i = R == 2 && ac >= static_cast<int>(kRow1) ? 1 : 0;
            const int col = i ? ac - static_cast<int>(kRow1) + 128 : ac, row = 128 * i + v % 16 * 8;
            *reinterpret_cast<uint4*>(square + element<R>(col, row)) = x[n];
          }
        }
        if (R == 2) {
          __syncthreads();
          mirror_block(square);
        }
      }

      // B = b A + c A^2, in A's place.
      multiply([&] {
        for (int i = 0; i < R; ++i) {
          const uint32_t idesc = ptx::instr_desc_f16(128, K::kSide - 128 * i, false);
          for (int n = 0; n < 2 * R; ++n) {
            const uint64_t d = ptx::smem_desc_k_sw128(square_addr + n * K::kPanel + i * 16384u);
            for (int k = 0; k < 4; ++k)
              ptx::mma_f16_ss<1>(tmem + i * kRow1, d + 2u * k, d + 2u * k, idesc, (n | k) != 0);
          }
        }
      });
      for (int i = 0; i < R; ++i) {
        const int row = i * 128 + q * 32 + lane;
#pragma unroll 1
        for (int c = group * 16; c < K::kSide - 128 * i; c += 16 * kGroups) {
          uint32_t r[16], w[8];
          ptx::tmem_ld_32x32b_x16(t_lane + i * kRow1 + c, r);
          const int col = 128 * i + c;
          uint4* at0 = reinterpret_cast<uint4*>(square + element<R>(row, col));
          uint4* at1 = reinterpret_cast<uint4*>(square + element<R>(row, col + 8));
          const uint4 a0 = *at0, a1 = *at1;
          const uint32_t old[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 f = unpack_half2(old[j]);
            w[j] = pack_half2(fmaf(p.c, __uint_as_float(r[2 * j]), p.b * f.x),
                              fmaf(p.c, __uint_as_float(r[2 * j + 1]), p.b * f.y));
          }
          if (col >> 5 == row >> 5) {  // the warp's rows meet the diagonal here
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 f = unpack_half2(old[j]);
              if (row == col + 2 * j) {
                diag[row] = fmaf(p.c, __uint_as_float(r[2 * j]), p.b * f.x);
                w[j] &= 0xFFFF0000u;
              }
              if (row == col + 2 * j + 1) {
                diag[row] = fmaf(p.c, __uint_as_float(r[2 * j + 1]), p.b * f.y);
                w[j] &= 0x0000FFFFu;
              }
            }
          }
          *at0 = make_uint4(w[0], w[1], w[2], w[3]);
          *at1 = make_uint4(w[4], w[5], w[6], w[7]);
          if (R == 2 && i == 0 && c >= 128) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              *reinterpret_cast<uint16_t*>(square + element<R>(col + j, row)) =
                  static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
          }
        }
      }

      // Z' = a Z + B Z, up to 256 of this CTA's columns a product.
      multiply([&] {
        for (int i = 0; i < R; ++i)
          for (int n = 0; n < panels; n += 4) {
            const uint32_t idesc = ptx::instr_desc_f16(128, 64 * min(4, panels - n), false, true);
            for (int k = 0; k < K::kSide / 16; ++k) {
              const uint64_t da =
                  ptx::smem_desc_k_sw128(square_addr + (k >> 2) * K::kPanel + i * 16384u) + 2u * (k & 3);
              const uint64_t db =
                  ptx::smem_desc_mn_sw128(z_addr + n * K::kPanel + k * 2048u, K::kPanel, 1024u);
              ptx::mma_f16_ss<1>(tmem + (i * K::kPanels + n) * 64u, da, db, idesc, k != 0);
            }
          }
      });
      const float wm = last ? inv : 1.0f;
      uint16_t* out = p.out + static_cast<int64_t>(m) * p.s * p.l;
      for (int i = 0; i < R; ++i) {
        const int row = i * 128 + q * 32 + lane;
        const float weight = p.a + diag[row], wa = wm * weight;
#pragma unroll 1
        for (int c = group * 32; c < panels * 64; c += 32 * kGroups) {
          uint32_t r[32], w[16];
          ptx::tmem_ld_32x32b_x32(t_lane + static_cast<uint32_t>(i * K::kPanels * 64 + c), r);
          uint4 old[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) old[j] = *reinterpret_cast<const uint4*>(z + element<R>(row, c + 8 * j));
          ptx::tmem_wait_ld();
          if (kLow) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 o = *reinterpret_cast<const uint4*>(z_low + element<R>(row, c + 8 * j));
              const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = unpack_half2(ow[e]);
                const int n = 8 * j + 2 * e;
                r[n] = __float_as_uint(fmaf(weight, f.x, __uint_as_float(r[n])));
                r[n + 1] = __float_as_uint(fmaf(weight, f.y, __uint_as_float(r[n + 1])));
              }
            }
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint4& o = old[j >> 2];
            const float2 f = unpack_half2((j & 3) == 0 ? o.x : (j & 3) == 1 ? o.y : (j & 3) == 2 ? o.z : o.w);
            const float x = fmaf(wm, __uint_as_float(r[2 * j]), wa * f.x);
            const float y = fmaf(wm, __uint_as_float(r[2 * j + 1]), wa * f.y);
            w[j] = last ? pack_bf162(x, y) : pack_half2(x, y);
            r[2 * j] = __float_as_uint(x);
            r[2 * j + 1] = __float_as_uint(y);
          }
          if (last && p.tall) {  // a column of Z is a row of the output
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (row < p.s && first + c + j < p.l)
                out[(first + c + j) * p.s + row] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(z + element<R>(row, c + 8 * j)) =
                  make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            if (kLow && !last) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[j] = low_half2(w[j], __uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(z_low + element<R>(row, c + 8 * j)) =
                    make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            }
          }
        }
      }
      if (last && !p.tall) {
        __syncthreads();
        const uintptr_t base = reinterpret_cast<uintptr_t>(out);
        if (p.l % 8 == 0 && base % 16 == 0)
          store_rows<R, uint4>(p, out, z, first, elements);
        else if (p.l % 2 == 0 && base % 4 == 0)
          store_rows<R, uint32_t>(p, out, z, first, elements);
        else
          store_rows<R, uint16_t>(p, out, z, first, elements);
      }
    }
    __syncthreads();
  }
  ptx::tc_fence_before_sync();
  __syncthreads();
  if (warp == 0) ptx::tmem_dealloc<1>(tmem, 512u);
}

constexpr size_t kStaticBytes = 1536;  // left for the kernel's own static shared memory

// The whole opt-in shared memory, whatever the panels need: a second CTA on
// an SM could not have its TMEM.
size_t smem_bytes(const gemm_ops* ops) { return ops->smem_optin - kStaticBytes; }

void configure(const gemm_ops* ops, int cluster, int grid, cudaStream_t stream, cudaLaunchConfig_t* cfg,
               cudaLaunchAttribute (&attr)[2]) {
  *cfg = cudaLaunchConfig_t{};
  cfg->gridDim = dim3(grid, 1, 1);
  cfg->blockDim = dim3(kThreads, 1, 1);
  cfg->dynamicSmemBytes = smem_bytes(ops);
  cfg->stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg->attrs = attr;
  cfg->numAttrs = cluster > 1 ? 2 : 1;
}

template <int R>
cudaError_t init(gemm_ops* ops) {
  const cudaFuncAttribute attribute = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int bytes = static_cast<int>(smem_bytes(ops));
  cudaError_t e = cudaFuncSetAttribute(small_newton_kernel<R, false>, attribute, bytes);
  if (e == cudaSuccess && R == 1) e = cudaFuncSetAttribute(small_newton_kernel<R, R == 1>, attribute, bytes);
  ops->small_clusters[R - 1][1] = ops->sm_count;
  for (int c = 2; c <= kSmallCluster && e == cudaSuccess; ++c) {
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    configure(ops, c, c, nullptr, &cfg, attr);
    e = cudaOccupancyMaxActiveClusters(&ops->small_clusters[R - 1][c], small_newton_kernel<R, false>, &cfg);
  }
  return e;
}

template <int R>
cudaError_t launch(const gemm_ops* ops, const SmallNewton& p, int grid, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  configure(ops, p.cluster, grid, stream, &cfg, attr);
  if (R == 1 && ceil_div(ceil_div(p.l, 64), p.cluster) <= Small<R>::kLowPanels)
    return cudaLaunchKernelEx(&cfg, small_newton_kernel<R, R == 1>, p);
  return cudaLaunchKernelEx(&cfg, small_newton_kernel<R, false>, p);
}

}  // namespace

cudaError_t small_newton_init(gemm_ops* ops) {
  if (ops->smem_optin < Small<2>::kBytes + 1024 + 16 + kStaticBytes) return cudaSuccess;  // no clusters: not used
  cudaError_t e = init<1>(ops);
  return e == cudaSuccess ? init<2>(ops) : e;
}

// Short sides up to 128 always (us, this kernel / separate products, five
// steps of fp32: 128 x 128 20 / 93, 128 x 512 39 / 102, 600 x 128 x 512 179 /
// 508, 128 x 4096 58 / 129, 64 x 128 x 4096 372 / 407).  Up to 256 a single
// CTA's always too (192 x 192 56 / 95, 608 of them 239 / 596); with the
// exchange a step is long and it pays while all matrices run at once (8 x 256
// x 640 90 / 117, 8 x 256 x 1536 93 / 142, but 80 x 256 x 640 372 / 229).
SmallPlan small_newton_plan(const gemm_ops* ops, int64_t m, int64_t n, int64_t batch) {
  SmallPlan plan;
  const int64_t s = std::min(m, n), l = std::max(m, n);
  if (s > 256) return plan;
  const int rows = s > 128 ? 2 : 1;
  const int64_t cluster = ceil_div(ceil_div(l, 64), small_newton_panels(rows));
  if (cluster > kSmallCluster) return plan;
  const int64_t slots = ops->small_clusters[rows - 1][cluster];
  if (slots < 1 || (rows == 2 && cluster > 1 && batch > slots)) return plan;
  plan.rows = rows;
  plan.cluster = static_cast<int>(cluster);
  plan.slots = static_cast<int>(std::min(batch, slots));
  const size_t elems = rows == 1 ? Small<1>::kElems : Small<2>::kElems;
  if (cluster > 1) {
    plan.norm_bytes = static_cast<size_t>(plan.slots) * cluster * sizeof(double);
    plan.part_bytes = plan.slots * cluster * elems * sizeof(float);
    plan.gram_bytes = plan.slots * elems * sizeof(uint16_t);
  }
  return plan;
}

cudaError_t small_newton_launch(const gemm_ops* ops, const SmallPlan& plan, SmallNewton& p,
                                cudaStream_t stream) {
  p.base.status = ops->d_status;
  p.base.timeout_ns = ops->timeout_ns;
  p.base.inject_fault = ops->debug_fault;
  p.cluster = plan.cluster;
  const int grid = plan.slots * plan.cluster;
  return plan.rows == 1 ? launch<1>(ops, p, grid, stream) : launch<2>(ops, p, grid, stream);
}

}  // namespace spgemm
