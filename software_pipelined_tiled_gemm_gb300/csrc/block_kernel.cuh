// block_kernel.cuh -- the products of the gated feed-forward block and of the
// Newton-Schulz iteration, on the roles of gemm_kernel.cuh (one TMA producer
// thread, one tcgen05.mma issuer thread, four or eight epilogue warps; see
// there for the ring and accumulator protocol).  What differs:
//
//   operands    each K-major (rows of K) or MN-major (stored K x M / K x N).
//               An MN-major slice of 64 K rows arrives as boxes of 64 columns
//               x 64 rows, 8 KiB each: swizzle atoms of 8 K rows are 1024 B
//               apart along K and 8 KiB apart along M/N.  Two-dimensional
//               boxes are clipped at the matrix's own edge, so no extent has
//               to be a multiple of 64.
//   tiles       256 x 256 on a CTA pair with two K slices per ring slot, or
//               128 x 128 on one CTA; of a batch of matrices; optionally only
//               those on and above the diagonal of a symmetric product.
//   gated       the tile's B rows are half gate rows, half up rows of the
//               same output columns, so act(gate) * up needs no other tile.
//               With a pair, the even CTA copies the gate rows and the odd
//               one the up rows.
//   split K     a product of few tiles gives each tile to a cluster of 2 or 4
//               single CTAs, each with a share of K.  Once a CTA's own
//               products are done its ring is idle: it stages its fp32
//               partial there, bulk-copies each CTA of the cluster the rows
//               that one will store (a quarter or half of the tile), and adds
//               its own and what it receives in CTA order while it stores its
//               rows: the epilogue is shared out as well.
//   last wave   stream-K with any number of walkers per tile: the walker
//               holding a tile's first K slices owns it, the others publish
//               fp32 partials (each at most one, in a slot of its own, as its
//               first piece of work), and the owner adds them in walker order.
//               Every sum has a fixed order, so results repeat bit for bit.
#pragma once

#include "block_math.cuh"
#include "block_params.h"
#include "gemm_kernel.cuh"
#include "ptx_block.cuh"

namespace spgemm {

struct BlockTile {
  int mb, nb, z;
};

// Tile t of the launch: which matrix of the batch, and where in it.
__device__ __forceinline__ BlockTile block_tile(int t, const BlockParams& p) {
  BlockTile x;
  x.z = t / p.tiles_per;
  const int r = t - x.z * p.tiles_per;
  if (!p.symmetric) {
    tile_coords(r, p, x.mb, x.nb);
    return x;
  }
  // Upper triangle, row by row: row i starts at i n - i (i - 1) / 2.
  const int n = p.tiles_n;
  const float b = 2.0f * n + 1.0f;
  int i = static_cast<int>((b - sqrtf(fmaxf(b * b - 8.0f * r, 0.0f))) * 0.5f);
  i = min(max(i, 0), n - 1);
  while (i > 0 && i * n - i * (i - 1) / 2 > r) --i;
  while (i + 1 < n && (i + 1) * n - (i + 1) * i / 2 <= r) ++i;
  x.mb = i;
  x.nb = i + (r - (i * n - i * (i - 1) / 2));
  return x;
}

// A piece of work: K slots [k0, k1) of a tile.
struct BlockUnit {
  int tile, k0, k1, role;
};

// A walker's pieces: first its contiguous share of the stream-K tiles' K
// slots (its partial for another walker, if any, comes first of all), then
// its whole tiles.
struct BlockIter {
  int u;
  int64_t it, end;
  int split;  // this CTA's share of a split tile, not yet taken; -1: none
  __device__ BlockIter(int walker, const BlockParams& p) : u(walker) {
    split = p.splits > 1 ? walker % p.splits : -1;
    if (p.splits > 1) {
      u = walker / p.splits;
      it = end = 0;
      return;
    }
    const int64_t total = static_cast<int64_t>(p.sk_tiles) * p.k_blocks;
    it = total * walker / p.walkers;
    end = total * (walker + 1) / p.walkers;
  }
  __device__ bool next(const BlockParams& p, BlockUnit& x) {
    if (p.splits > 1) {
      if (split < 0) return false;
      x.tile = u;
      x.k0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * split / p.splits);
      x.k1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (split + 1) / p.splits);
      x.role = kWhole;
      split = -1;
      return true;
    }
    if (it < end) {
      x.tile = static_cast<int>(it / p.k_blocks);
      x.k0 = static_cast<int>(it - static_cast<int64_t>(x.tile) * p.k_blocks);
      const int64_t left = end - it;
      x.k1 = static_cast<int>(x.k0 + left < p.k_blocks ? x.k0 + left : p.k_blocks);
      x.role = x.k0 > 0 ? kContrib : (x.k1 < p.k_blocks ? kOwner : kWhole);
      it += x.k1 - x.k0;
      return true;
    }
    if (u < p.dp_tiles) {
      x.tile = p.sk_tiles + u;
      x.k0 = 0;
      x.k1 = p.k_blocks;
      x.role = kWhole;
      u += p.walkers;
      return true;
    }
    return false;
  }
};

// The walkers after `walker` that hold a piece of its last stream-K tile.
__device__ __forceinline__ int block_contributors(int walker, const BlockUnit& x,
                                                  const BlockParams& p) {
  const int64_t total = static_cast<int64_t>(p.sk_tiles) * p.k_blocks;
  const int64_t tile_end = static_cast<int64_t>(x.tile + 1) * p.k_blocks;
  int n = 0;
  while (walker + n + 1 < p.walkers && total * (walker + n + 1) / p.walkers < tile_end) ++n;
  return n;
}

// The epilogue works on 16 columns at a time (lane = row) in rolled loops: a
// launch of a small product runs its epilogue once, on a cold instruction
// cache, and straight-line code for 64 columns took two to three times as
// long there as a loop whose later turns find their instructions.
//
// A 32-row x 64-column block of a 16-bit output goes through the warp's
// staging buffer (already free) in the layout of a 128-byte-swizzled box.
// stage16: columns [16 c, 16 c + 16) of the block, as 8 words of this row.
__device__ __forceinline__ void stage16(uint8_t* sb, int lane, int c, const uint32_t (&w)[8]) {
  uint8_t* row = sb + lane * 128u;
  const uint32_t sw = lane & 7u, j = 2u * static_cast<uint32_t>(c);
  *reinterpret_cast<uint4*>(row + ((j ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(row + (((j + 1) ^ sw) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
}

// The staged block (visible to the warp and the copy engine), out with one
// bulk store, or row by row where the output's rows are not 16-byte aligned
// (columns below `cols`).
__device__ __forceinline__ void block_store(const BlockParams& p, const BlockOut& o,
                                            const CUtensorMap& map, uint8_t* sb, int lane, int row0,
                                            int col0, int z, int cols) {
  if (o.tma) {
    if (lane == 0) {
      ptx::tma_store_3d(&map, ptx::smem_addr(sb), col0, row0, z);
      ptx::bulk_commit_group();
    }
    return;
  }
  const int ncols = min(64, cols - col0);
  const int nrows = min(32, p.M - row0);
  uint16_t* base = static_cast<uint16_t*>(o.ptr) + z * o.batch + static_cast<int64_t>(row0) * o.ld + col0;
#pragma unroll 4
  for (int r = 0; r < nrows; ++r) {
    uint16_t* crow = base + r * o.ld;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int cc = lane + 32 * h;
      const uint32_t byte = static_cast<uint32_t>(cc) * 2u;
      const uint32_t off = static_cast<uint32_t>(r) * 128u +
                           (((byte >> 4) ^ (static_cast<uint32_t>(r) & 7u)) << 4) + (byte & 15u);
      if (cc < ncols) crow[cc] = *reinterpret_cast<const uint16_t*>(sb + off);
    }
  }
}

// 16 columns of the block transposed, into the same output: a column is 32
// consecutive elements of row col0 + column.  Neighbouring lanes first
// exchange words, so that each lane stores two rows' worth of one column.
__device__ __forceinline__ void mirror16(const uint32_t (&w)[8], const BlockParams& p,
                                         const BlockOut& o, int lane, int row0, int col0, int z) {
  const bool odd = lane & 1;
  const int r = row0 + (lane & ~1);  // this lane's pair of source rows
  uint16_t* dst = static_cast<uint16_t*>(o.ptr) + z * o.batch +
                  static_cast<int64_t>(col0 + (odd ? 1 : 0)) * o.ld + r;
  const int n = p.N - col0 - (odd ? 1 : 0);  // columns that exist from this lane's first
  uint32_t pair[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    // w[j]: columns 2j, 2j + 1 of this row.  The even lane keeps column 2j
    // and takes its neighbour's; the odd lane column 2j + 1.
    const uint32_t got = __shfl_xor_sync(0xffffffffu, w[j], 1);
    pair[j] = odd ? __byte_perm(got, w[j], 0x7632) : __byte_perm(w[j], got, 0x5410);
  }
  if (row0 + 32 <= p.M && col0 + 16 <= p.N) {
#pragma unroll
    for (int j = 0; j < 8; ++j)  // r is even and the pitch a multiple of 8
      *reinterpret_cast<uint32_t*>(dst + 2 * j * o.ld) = pair[j];
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (2 * j < n) {
      if (r + 1 < p.M)
        *reinterpret_cast<uint32_t*>(dst + 2 * j * o.ld) = pair[j];
      else if (r < p.M)
        dst[2 * j * o.ld] = static_cast<uint16_t>(pair[j]);
    }
}

// Adds the contributors' partials to a tile's accumulator in TMEM, in order:
// columns [c, c + 32) for c = first, first + stride, ...
__device__ __forceinline__ void block_add_partials(uint32_t t_row, const float* partial,
                                                   size_t partial_step, int parts, int first,
                                                   int columns, int stride, int lane) {
#pragma unroll 1
  for (int c = first; c < columns; c += stride) {
    uint32_t r[32];
    ptx::tmem_ld_32x32b_x32(t_row + c, r);
    ptx::tmem_wait_ld();
    const float* src = partial + static_cast<size_t>(c) * 32 + lane;
#pragma unroll 1
    for (int n = 0; n < parts; n += 2, src += 2 * partial_step) {  // two partials' loads in flight
      const bool both = n + 1 < parts;
      float v[2][32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[0][j] = __ldcg(src + j * 32);
        v[1][j] = both ? __ldcg(src + partial_step + j * 32) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        float sum = __uint_as_float(r[j]) + v[0][j];
        if (both) sum += v[1][j];
        r[j] = __float_as_uint(sum);
      }
    }
    ptx::tmem_st_32x32b_x32(t_row + c, r);
  }
  ptx::tmem_wait_st();
}

// act(gate) * up of 16 columns, packed two to a word.
template <int ACT>
__device__ __forceinline__ void gated16(const uint32_t (&g)[16], const uint32_t (&u)[16],
                                        uint32_t (&pk)[8], bool bf16) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    pk[j] = pack2(gate_act<ACT>(__uint_as_float(g[2 * j])) * __uint_as_float(u[2 * j]),
                  gate_act<ACT>(__uint_as_float(g[2 * j + 1])) * __uint_as_float(u[2 * j + 1]), bf16);
}

// dGate and dUp of 16 columns.
template <int ACT>
__device__ __forceinline__ void gated_bwd16(const uint32_t (&dh)[16], const float (&g)[16],
                                            const float (&u)[16], uint32_t (&pg)[8],
                                            uint32_t (&pu)[8], bool bf16) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float dg[2], du[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, d;
      gate_act_grad<ACT>(g[2 * j + i], a, d);
      const float h = __uint_as_float(dh[2 * j + i]);
      dg[i] = h * u[2 * j + i] * d;
      du[i] = h * a;
    }
    pg[j] = pack2(dg[0], dg[1], bf16);
    pu[j] = pack2(du[0], du[1], bf16);
  }
}

// CG: 2 for CTA pairs, 1 for single CTAs.  kAT: A stored K x M.  kBN: B
// stored K x N.  kEpi: the epilogue (block_params.h).
// kG: epilogue warps per TMEM lane quarter.  With two, they share the
// quarter's staging buffers and each takes 32 of a chunk's 64 columns.
template <int CG, bool kAT, bool kBN, int kEpi, int kG>
__global__ void __launch_bounds__(kernel_threads(kG), 1)
    block_kernel(const __grid_constant__ BlockMaps maps, const __grid_constant__ BlockParams p) {
  constexpr int BN = block_bn(CG);
  constexpr int kSub = block_sub(CG);
  constexpr int kBRows = BN / CG;                 // B rows this CTA copies
  constexpr uint32_t kStageB = kBRows * kBK * 2;
  constexpr int kTileM = kBM * CG;
  constexpr bool kUseD = kEpi >= kEpiDiagOut;
  constexpr int kOutN = kEpi == kEpiGated ? BN / 2 : BN;  // output columns of a tile
  constexpr uint32_t kBoxBytes = 64u * kBK * 2u;          // MN-major box: 64 columns x 64 K rows
  // K-major A of a single row of tiles: only the rows that exist are copied
  // (see Params::a_box_rows); the MMA's other rows read what follows in the
  // slot and feed output rows that are never stored.
  const uint32_t slice_a = kAT ? kStageA : static_cast<uint32_t>(p.a_box_rows) * (kBK * 2u);
  const uint32_t slot_a = slice_a * kSub;
  const uint32_t slot_bytes = slot_a + kStageB * kSub;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = ptx::smem_addr(smem);
  const int S = p.stages;
  const uint32_t ring_bytes = static_cast<uint32_t>(S) * slot_bytes;
  uint8_t* staging = smem + ring_bytes;
  constexpr uint32_t staging_bytes = 4u * 2u * kStoreBuf;
  const uint32_t bar_base = sbase + ring_bytes + staging_bytes;
  if (SPGEMM_OUT_OF_BOUNDS(S >= 1 && S <= kMaxStages &&
                               (sbase - raw_addr) + ring_bytes + staging_bytes +
                                       8u * (2 * kMaxStages + 5 + 2 * kEpiWarps) + 4u <=
                                   ptx::dynamic_smem_bytes(),
                           p, kCheckSmemLayout))
    return;
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (kMaxStages + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * kMaxStages + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * kMaxStages + 2 + a); };
  const uint32_t done_bar = bar_base + 8u * (2 * kMaxStages + 4);
  const uint32_t inbox_bar = bar_base + 8u * (2 * kMaxStages + 13);
  auto d_bar = [&](int e, int b) { return bar_base + 8u * (2 * kMaxStages + 5 + 2 * e + b); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + ring_bytes + staging_bytes +
                                                    8u * (2 * kMaxStages + 5 + 2 * kEpiWarps));

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  constexpr uint32_t tmem_cols = 2u * BN;  // two accumulators
  const uint32_t rank = (CG == 2) ? ptx::cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int walker = static_cast<int>(blockIdx.x) / CG;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), 4 * kG * CG);
    }
    ptx::mbar_init(done_bar, 1);
    for (int e = 0; e < 4; ++e)
      for (int b = 0; b < 2; ++b) ptx::mbar_init(d_bar(e, b), 1);
    ptx::mbar_init(inbox_bar, 1);
    ptx::fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    ptx::tma_prefetch_desc(&maps.a);
    ptx::tma_prefetch_desc(&maps.b);
  }
  if (warp == 1) {
    ptx::tmem_alloc<CG>(ptx::smem_addr(tmem_slot), tmem_cols);
    ptx::tmem_relinquish<CG>();
  }
  ptx::tc_fence_before_sync();
  if (CG == 2)
    ptx::cluster_sync();
  else
    __syncthreads();
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  ptx::pdl_launch_dependents();

  // First B row of a tile for this CTA, and (gated, single CTA) of its up half.
  auto b_first = [&](int nb) {
    if constexpr (kEpi == kEpiGated)
      return nb * kOutN + (CG == 2 && rank == 1 ? p.gate_rows : 0);
    else
      return nb * BN + static_cast<int>(rank) * kBRows;
  };

  // Split K: the two points that all warps of the cluster pass, whatever
  // their role met (rings free; partials received).
  auto split_syncs = [&]() {
    if (CG == 1 && p.splits > 1) {
      ptx::cluster_sync();
      ptx::cluster_sync();
    }
  };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;
      const uint64_t pol_b = (CG == 1 && p.b_stream) ? ptx::l2_policy_evict_first() : 0;
      bool ok = true;
      const uint32_t bytes =
          (slice_a + static_cast<uint32_t>(kStageB)) * static_cast<uint32_t>(CG * kSub);
      BlockIter it(walker, p);
      BlockUnit x;
      // Warm L2 with the weights of the first slots while the previous kernel
      // in the stream finishes (only lines move; the copies come after the wait).
      if (CG == 1 && p.l2_prefetch_first) {
        BlockIter it0(walker, p);
        if (it0.next(p, x)) {
          const BlockTile t = block_tile(x.tile, p);
          for (int i = 0; i < S && x.k0 + i < x.k1; ++i) {
            const int kx = (x.k0 + i) * kBK;
            if constexpr (kBN) {
              ptx::tma_prefetch_l2_3d(&maps.b, b_first(t.nb), kx, t.z);
              ptx::tma_prefetch_l2_3d(&maps.b, b_first(t.nb) + 64, kx, t.z);
            } else {
              ptx::tma_prefetch_l2_3d(&maps.b, kx, b_first(t.nb), t.z);
              if constexpr (kEpi == kEpiGated)
                ptx::tma_prefetch_l2_3d(&maps.b, kx, b_first(t.nb) + p.gate_rows, t.z);
            }
          }
        }
      }
      bool waited = false;  // on the previous kernel: finding the first tile overlaps it
      while (ok && it.next(p, x)) {
        const BlockTile t = block_tile(x.tile, p);
        if (SPGEMM_OUT_OF_BOUNDS(x.tile >= 0 && x.tile < p.num_tiles && t.z < p.batch &&
                                     t.mb >= 0 && t.mb < p.tiles_m && t.nb >= 0 && t.nb < p.tiles_n,
                                 p, kCheckTile) ||
            SPGEMM_OUT_OF_BOUNDS(x.k0 >= 0 && x.k0 < x.k1 && x.k1 <= p.k_blocks, p, kCheckKSlice)) {
          ok = false;
          break;
        }
        const int a_row = t.mb * kTileM + static_cast<int>(rank) * kBM;
        const int b_row = b_first(t.nb);
        for (int kb = x.k0; kb < x.k1; ++kb) {
          if (!wait_bounded(empty_bar(stage), phase ^ 1u, p, kDetailProducerEmpty)) {
            ok = false;
            break;
          }
          if (SPGEMM_OUT_OF_BOUNDS(stage < S && (a_row & 7) == 0 && (!kBN || (b_row & 7) == 0), p,
                                   kCheckTmaCoord)) {
            ok = false;
            break;
          }
          const uint32_t sa = sbase + stage * slot_bytes;
          uint32_t fb = full_bar(stage);
          if constexpr (CG == 2) fb = ptx::map_shared_rank(fb, 0);
          if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), bytes);
          if (!waited) {
            ptx::pdl_wait_prior_grid();
            waited = true;
          }
          // Test hook: the first slot of the first CTA is announced but never copied.
          const bool skip = p.inject_fault == 1 && blockIdx.x == 0 && issued == 0;
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub) {
            if (skip) break;
            const int kx = (kb * kSub + sub) * kBK;
            const uint32_t da = sa + sub * slice_a, db = sa + slot_a + sub * kStageB;
            if constexpr (CG == 2) {
              if constexpr (kAT) {
                ptx::tma_load_3d_pair(da, &maps.a, a_row, kx, t.z, fb);
                ptx::tma_load_3d_pair(da + kBoxBytes, &maps.a, a_row + 64, kx, t.z, fb);
              } else {
                ptx::tma_load_3d_pair(da, &maps.a, kx, a_row, t.z, fb);
              }
              if constexpr (kBN) {
                ptx::tma_load_3d_pair(db, &maps.b, b_row, kx, t.z, fb);
                ptx::tma_load_3d_pair(db + kBoxBytes, &maps.b, b_row + 64, kx, t.z, fb);
              } else {
                ptx::tma_load_3d_pair(db, &maps.b, kx, b_row, t.z, fb);
              }
            } else {
              if constexpr (kAT) {
                ptx::tma_load_3d(da, &maps.a, a_row, kx, t.z, fb);
                ptx::tma_load_3d(da + kBoxBytes, &maps.a, a_row + 64, kx, t.z, fb);
              } else {
                ptx::tma_load_3d(da, &maps.a, kx, a_row, t.z, fb);
              }
              auto load_b = [&](uint32_t dst, int cx, int cy) {
                if (p.b_stream)
                  ptx::tma_load_3d_hint(dst, &maps.b, cx, cy, t.z, fb, pol_b);
                else
                  ptx::tma_load_3d(dst, &maps.b, cx, cy, t.z, fb);
              };
              if constexpr (kBN) {
                load_b(db, b_row, kx);
                load_b(db + kBoxBytes, b_row + 64, kx);
              } else if constexpr (kEpi == kEpiGated) {  // 64 gate rows, then 64 up rows
                load_b(db, kx, b_row);
                load_b(db + kStageB / 2, kx, b_row + p.gate_rows);
              } else {
                load_b(db, kx, b_row);
              }
            }
          }
          issued |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // Every copy this CTA (pair) started must have landed before it exits.
      if (leader) {
        for (int s = 0; s < S; ++s)
          if (issued & (1u << s))
            wait_bounded(full_bar(s), (issued_parity >> s) & 1u, p, kDetailProducerDrain);
      }
    }
    __syncwarp();
    split_syncs();
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      BlockIter it(walker, p);
      BlockUnit x;
      while (ok && it.next(p, x)) {
        if (!wait_bounded_cluster<CG>(tempty_bar(acc), acc_phase ^ 1u, p, kDetailMmaAccEmpty)) break;
        ptx::tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = x.k0; kb < x.k1; ++kb) {
          if (!wait_bounded(full_bar(stage), phase, p, kDetailMmaFull) ||
              SPGEMM_OUT_OF_BOUNDS(stage >= 0 && stage < S, p, kCheckMmaSlot)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after_sync();
          const uint32_t sa = sbase + stage * slot_bytes;
          const uint64_t a_desc = kAT ? ptx::smem_desc_mn_sw128(sa, kBoxBytes, 1024u)
                                      : ptx::smem_desc_k_sw128(sa);
          const uint64_t b_desc = kBN ? ptx::smem_desc_mn_sw128(sa + slot_a, kBoxBytes, 1024u)
                                      : ptx::smem_desc_k_sw128(sa + slot_a);
          // A 16-wide K step is 32 B inside a K-major swizzle row, or two
          // 1024-byte atoms of 8 K rows of an MN-major box.
          constexpr uint32_t a_step = kAT ? 2048u / 16u : 2u, b_step = kBN ? 2048u / 16u : 2u;
#pragma unroll
          for (int k = 0; k < kSub * (kBK / kUmmaK); ++k) {
            const uint32_t sub = static_cast<uint32_t>(k) / 4u, kk = static_cast<uint32_t>(k) % 4u;
            ptx::mma_f16_ss<CG>(d_tmem, a_desc + sub * (slice_a / 16u) + a_step * kk,
                                b_desc + sub * (kStageB / 16u) + b_step * kk, p.idesc,
                                (kb != x.k0 || k != 0) ? 1u : 0u);
          }
          if constexpr (CG == 2)
            ptx::mma_commit_multicast_pair(empty_bar(stage), 0x3);
          else
            ptx::mma_commit<1>(empty_bar(stage));
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if constexpr (CG == 2)
          ptx::mma_commit_multicast_pair(tfull_bar(acc), 0x3);
        else
          ptx::mma_commit<1>(tfull_bar(acc));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      ptx::mma_commit<CG>(done_bar);
      wait_bounded(done_bar, 0, p, kDetailMmaDrain);
    }
    __syncwarp();
    split_syncs();
  } else {
    // --------------------------------------------------------- epilogue --
    ptx::pdl_wait_prior_grid();
    if (blockIdx.x == 0)
      for (int i = static_cast<int>(threadIdx.x) - 64; i < p.zero_flags; i += 128 * kG) p.sk_flags[i] = 0;
    const int q = warp & 3;         // TMEM lane quarter
    const int ew = (warp - 2) & 3;  // index of the quarter's staging, partials and flags
    const int g = (warp - 2) >> 2;  // which of the quarter's warps
    const bool lead = g == 0 && lane == 0;
    // Sub-steps of 16 columns of a chunk that this warp takes.
    constexpr int kSteps = 4 / kG;
    const int s0 = g * kSteps;
    auto quarter_sync = [&]() {  // the quarter's warps
      if constexpr (kG == 2)
        ptx::named_barrier_sync(2 + q, 64);
      else
        __syncwarp();
    };
    // Whether every wait of the quarter's warps ended well: they leave a
    // unit together, or one would wait for the other at their barrier.
    auto quarter_all = [&](bool ok) -> bool {
      if constexpr (kG == 2)
        return ptx::named_barrier_all(2 + q, 64, ok);
      else
        return __all_sync(0xffffffffu, ok);
    };
    uint8_t* my_stage = staging + ew * 2 * kStoreBuf;
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t d_phase = 0;  // parity of the next fill of D buffer b in bit b
    int buf = 0;
    const bool bf16_out = p.out_bf16 != 0;
    constexpr size_t kPartial = block_partial_bytes(CG) / 4;  // floats of a CTA's partial
    // beta D: one chunk into staging buffer b.
    auto load_d = [&](int b, int row0, int col, int z) {
      if (lead) {
        ptx::bulk_wait_group_read<0>();  // the buffer's last store has been read out
        ptx::fence_proxy_async_smem();   // (by the warp itself, where rows are stored one by one)
        ptx::mbar_arrive_expect_tx(d_bar(ew, b), kStoreBuf);
        ptx::tma_load_3d(ptx::smem_addr(my_stage + b * kStoreBuf), &maps.d, col, row0, z,
                         d_bar(ew, b));
      }
    };
    auto wait_d = [&]() { return wait_bounded(d_bar(ew, buf), (d_phase >> buf) & 1u, p, kDetailSkCopy); };

    // The diagonal's elements for this lane's row, or for two of a chunk's
    // columns: read a chunk (or a tile) before they are used.
    float diag0 = 0.0f, diag1 = 0.0f;
    auto load_diag = [&](int row0, int col0, int z) {
      const float* diag = p.diag + z * p.diag_batch;
      if constexpr (kEpi == kEpiDiagRows) diag0 = row0 + lane < p.M ? __ldcg(diag + row0 + lane) : 0.0f;
      if constexpr (kEpi == kEpiDiagCols) {
        diag0 = __ldcg(diag + col0 + lane);
        diag1 = __ldcg(diag + col0 + 32 + lane);
      }
    };

    // The staged block out, once the quarter's warps have written it.
    auto store = [&](const BlockOut& o, const CUtensorMap& map, uint8_t* sb, int row0, int col0, int z) {
      if (o.tma) ptx::fence_proxy_async_smem();
      quarter_sync();
      if (g == 0) block_store(p, o, map, sb, lane, row0, col0, z, p.N);
      if (!o.tma) quarter_sync();  // the buffer has been read
    };

    // 32 rows x 64 output columns from column n0 + cc: acc(c, r) gives the 16
    // accumulator columns from tile column c for this lane's row.  more: the
    // next chunk of these rows follows (its D is fetched meanwhile).
    auto chunk = [&](auto&& acc_cols, int row0, int n0, int cc, int z, bool more) -> bool {
      const int col0 = n0 + cc;
      uint8_t* sb = my_stage + buf * kStoreBuf;
      if constexpr (kEpi == kEpiGated) {
        if (lead) ptx::bulk_wait_group_read<1>();
        quarter_sync();
        float* dst = p.pre + (static_cast<int64_t>(row0 / 32) * p.N + col0 + 16 * s0) * 32 + lane;
#pragma unroll 1
        for (int s = s0; s < s0 + kSteps; ++s) {
          uint32_t gate[16], up[16], pk[8];
          acc_cols(cc + 16 * s, gate);
          acc_cols(BN / 2 + cc + 16 * s, up);
          if (p.pre != nullptr) {
            const int n = p.N - (col0 + 16 * s);  // columns that exist
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (j < n) {
                __stcs(dst + j * 32, __uint_as_float(gate[j]));
                __stcs(dst + p.pre_half + j * 32, __uint_as_float(up[j]));
              }
            dst += 16 * 32;
          }
          if (p.act == kActSilu)
            gated16<kActSilu>(gate, up, pk, bf16_out);
          else if (p.act == kActGelu)
            gated16<kActGelu>(gate, up, pk, bf16_out);
          else
            gated16<kActRelu>(gate, up, pk, bf16_out);
          stage16(sb, lane, s, pk);
        }
        store(p.out0, maps.c0, sb, row0, col0, z);
        buf ^= 1;
      } else if constexpr (kEpi == kEpiGatedBwd) {
        const float* src = p.pre + (static_cast<int64_t>(row0 / 32) * p.N + col0) * 32 + lane;
        const int n = p.N - col0;
        float gate[2][16], up[2][16];  // this step's and the next one's
        auto load_pre = [&](int s, float (&gs)[16], float (&us)[16]) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const bool in = 16 * s + j < n;
            gs[j] = in ? __ldcs(src + (16 * s + j) * 32) : 0.0f;
            us[j] = in ? __ldcs(src + p.pre_half + (16 * s + j) * 32) : 0.0f;
          }
        };
        auto step = [&](int s, const float (&gs)[16], const float (&us)[16]) {
          uint32_t dh[16], pg[8], pu[8];
          acc_cols(cc + 16 * s, dh);
          if (p.act == kActSilu)
            gated_bwd16<kActSilu>(dh, gs, us, pg, pu, bf16_out);
          else if (p.act == kActGelu)
            gated_bwd16<kActGelu>(dh, gs, us, pg, pu, bf16_out);
          else
            gated_bwd16<kActRelu>(dh, gs, us, pg, pu, bf16_out);
          stage16(my_stage, lane, s, pg);
          stage16(my_stage + kStoreBuf, lane, s, pu);
        };
        load_pre(s0, gate[0], up[0]);
        load_pre(s0 + 1, gate[1], up[1]);
        if (lead) ptx::bulk_wait_group_read<0>();
        quarter_sync();
#pragma unroll 1
        for (int s = s0; s < s0 + kSteps; s += 2) {
          step(s, gate[0], up[0]);
          if (s + 2 < s0 + kSteps) load_pre(s + 2, gate[0], up[0]);
          step(s + 1, gate[1], up[1]);
          if (s + 3 < s0 + kSteps) load_pre(s + 3, gate[1], up[1]);
        }
        store(p.out0, maps.c0, my_stage, row0, col0, z);
        store(p.out1, maps.c1, my_stage + kStoreBuf, row0, col0, z);
      } else {
        const float beta = fmaf(p.alpha, diag0, p.beta), beta2 = fmaf(p.alpha, diag1, p.beta);
        if (kEpi == kEpiDiagCols && more) load_diag(row0, col0 + 64, z);
        if constexpr (kUseD) {
          const bool got = wait_d();
          d_phase ^= 1u << buf;
          if (!quarter_all(got)) return false;
          if (more) load_d(buf ^ 1, row0, col0 + 64, z);
        } else {
          if (lead) ptx::bulk_wait_group_read<1>();
          quarter_sync();
        }
        const bool mirror = p.symmetric && row0 / kTileM != col0 / BN;
#pragma unroll 1
        for (int s = s0; s < s0 + kSteps; ++s) {
          uint32_t r[16], pk[8];
          acc_cols(cc + 16 * s, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(p.alpha * __uint_as_float(r[j]));
          if constexpr (kUseD) {
            auto weight = [&](int i) {
              return kEpi == kEpiDiagCols
                         ? __shfl_sync(0xffffffffu, s < 2 ? beta : beta2, 16 * (s & 1) + i)
                         : beta;
            };
            // D is fp16 (the iterate's type), in the swizzled layout of the box.
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t c = static_cast<uint32_t>(2 * s + j);
              const uint4 v = *reinterpret_cast<const uint4*>(sb + lane * 128u + ((c ^ (lane & 7u)) << 4));
              const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&wd[e]));
                const int i = 8 * j + 2 * e;
                r[i] = __float_as_uint(fmaf(weight(i), f.x, __uint_as_float(r[i])));
                r[i + 1] = __float_as_uint(fmaf(weight(i + 1), f.y, __uint_as_float(r[i + 1])));
              }
            }
          }
          if constexpr (kEpi == kEpiDiagOut) {
            if ((col0 + 16 * s) >> 5 == row0 >> 5) {
              float* diag = p.diag + z * p.diag_batch;
              const int at = row0 + lane - (col0 + 16 * s);  // the diagonal's of these columns
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (j == at) {
                  if (row0 + lane < p.M) __stcg(diag + row0 + lane, __uint_as_float(r[j]));
                  r[j] = 0u;
                }
            }
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            pk[j] = pack2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), bf16_out);
          if (mirror) mirror16(pk, p, p.out0, lane, row0, col0 + 16 * s, z);
          stage16(sb, lane, s, pk);
        }
        store(p.out0, maps.c0, sb, row0, col0, z);
        buf ^= 1;
      }
      return true;
    };

    BlockIter it(walker, p);
    BlockUnit x;
    if (CG == 1 && p.splits > 1) {
      // ------------------------------------------ a share of a split tile --
      const int part = walker % p.splits;
      it.next(p, x);
      const BlockTile t = block_tile(x.tile, p);
      const int n0 = t.nb * kOutN;
      // This CTA's rows of the tile, in blocks of 32, and of those the
      // chunks that exist: (block, chunk) units, taken by the warps in turn.
      const int row_blocks = 4 / p.splits;
      constexpr int kChunks = kOutN / 64;
      const int first_row = t.mb * kTileM + part * row_blocks * 32;
      auto unit_exists = [&](int u) {
        return u < row_blocks * kChunks && first_row + (u / kChunks) * 32 < p.M &&
               n0 + (u % kChunks) * 64 < p.N;
      };
      if (kUseD && unit_exists(ew))
        load_d(buf, first_row + (ew / kChunks) * 32, n0 + (ew % kChunks) * 64, t.z);
      // The idle ring: this CTA's partial, [quarter][column][row], then what it
      // receives, [CTA][quarter of this CTA's][column][row].
      constexpr uint32_t kQuarter = kSplitBytes / 4;
      const uint32_t inbox = sbase + kSplitBytes;
      const int expected = [&]() {  // quarters of this CTA's rows that exist
        int n = 0;
        for (int i = 0; i < row_blocks; ++i) n += first_row + i * 32 < p.M ? 1 : 0;
        return n;
      }();
      int ok = SPGEMM_OUT_OF_BOUNDS(2 * kSplitBytes <= ring_bytes, p, kCheckFixup) ? 0 : 1;
      if (lane == 0 && ok) ok = wait_bounded<true>(tfull_bar(0), 0, p, kDetailEpiFull) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (lead && ew == 0 && expected > 0)
        ptx::mbar_arrive_expect_tx(inbox_bar, static_cast<uint32_t>(expected * (p.splits - 1)) * kQuarter);
      __syncwarp();
      // The accumulator is full, so every copy into the ring has been
      // consumed: this CTA's ring is free.
      ptx::cluster_arrive();
      const uint32_t mine = sbase + static_cast<uint32_t>(q) * kQuarter;
      if (ok) {
        ptx::tc_fence_after_sync();
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
        float* own = reinterpret_cast<float*>(smem) + q * (kQuarter / 4);
#pragma unroll 1
        for (int c = 32 * g; c < BN; c += 32 * kG) {
          uint32_t v[32];
          ptx::tmem_ld_32x32b_x32(t_row + c, v);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) own[(c + j) * 32 + lane] = __uint_as_float(v[j]);
        }
        ptx::fence_proxy_async_smem();
      }
      ptx::cluster_wait();  // every ring of the cluster is free
      // The stores below are shared out by chunk, so a warp also reads what
      // the other quarters' warps staged: their arrivals at the cluster's
      // barrier came before that.
      ptx::named_barrier_sync(1, 128 * kG);
      const int to = q / row_blocks;  // the CTA that stores this quarter's rows
      if (quarter_all(ok != 0) && lead && to != part && t.mb * kTileM + q * 32 < p.M)
        ptx::bulk_copy_to_peer(
            ptx::map_shared_rank(inbox + static_cast<uint32_t>(part * row_blocks + q % row_blocks) * kQuarter, to),
            mine, kQuarter, ptx::map_shared_rank(inbox_bar, to));
      int got = 1;
      if (expected > 0 && lane == 0) got = wait_bounded_cluster<2>(inbox_bar, 0, p, kDetailSkCopy) ? 1 : 0;
      got = __shfl_sync(0xffffffffu, got, 0);
      if (expected > 0 && got) (void)ptx::mbar_try_wait_cluster(inbox_bar, 0);  // every lane acquires
      // Received; a CTA may leave when all have (its copies then are read out).
      ptx::cluster_arrive();
      if (quarter_all(got != 0))
        for (int u = ew; unit_exists(u); u += 4) {
          const int rb = u / kChunks;
          const float* in = reinterpret_cast<const float*>(smem + kSplitBytes) + rb * (kQuarter / 4) + lane;
          const float* own = reinterpret_cast<const float*>(smem) + (part * row_blocks + rb) * (kQuarter / 4) + lane;
          const int step = row_blocks * (kQuarter / 4);
          if (kUseD) load_diag(first_row + rb * 32, n0 + (u % kChunks) * 64, t.z);
          auto from_inbox = [&](int c, uint32_t (&r)[16]) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
            for (int n = 0; n < p.splits; ++n) {
              const float* src = n == part ? own : in + n * step;
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] += src[(c + j) * 32];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(v[j]);
          };
          if (!chunk(from_inbox, first_row + (u / kChunks) * 32, n0, (u % kChunks) * 64, t.z, false)) break;
        }
      ptx::cluster_wait();
    } else
    while (it.next(p, x)) {
      const BlockTile t = block_tile(x.tile, p);
      const int row0 = t.mb * kTileM + static_cast<int>(rank) * kBM + q * 32;
      const int n0 = t.nb * kOutN;
      const bool rows = row0 < p.M;
      const bool stores = x.role != kContrib && rows;
      if (SPGEMM_OUT_OF_BOUNDS(row0 >= 0 && row0 < p.tiles_m * kTileM && n0 >= 0 && (n0 & 63) == 0,
                               p, kCheckStore) ||
          SPGEMM_OUT_OF_BOUNDS(x.role == kWhole || (p.sk_ws != nullptr && p.sk_flags != nullptr), p,
                               kCheckPartial))
        break;
      // The tile's first chunk of D arrives while the accumulator fills.
      const bool d_first = kUseD && stores;
      if (d_first) {
        load_d(buf, row0, n0, t.z);
        load_diag(row0, n0, t.z);
      }
      // The kept projections of these rows, a contiguous run each, into L2.
      if (kEpi == kEpiGatedBwd && stores && g == 0 && lane < 2) {
        const uint32_t n = static_cast<uint32_t>(min(BN, p.N - n0));
        ptx::bulk_prefetch_l2(p.pre + lane * p.pre_half + (static_cast<int64_t>(row0 / 32) * p.N + n0) * 32,
                              n * 128u);
      }

      int ready = 1;
      if (lane == 0) ready = wait_bounded<true>(tfull_bar(acc), acc_phase, p, kDetailEpiFull) ? 1 : 0;
      ready = __shfl_sync(0xffffffffu, ready, 0);
      if (!quarter_all(ready != 0)) {
        if (d_first) wait_d();  // a copy in flight lands before this warp's memory goes
        break;
      }
      ptx::tc_fence_after_sync();
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);

      if (x.role == kContrib) {
        if (rows) {
          const int slot = walker * CG + static_cast<int>(rank);
          float* partial = p.sk_ws + slot * kPartial + static_cast<size_t>(ew) * BN * 32;
#pragma unroll 1
          for (int c = 32 * g; c < BN; c += 32 * kG) {
            uint32_t v[32];
            ptx::tmem_ld_32x32b_x32(t_row + c, v);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              __stcg(partial + (c + j) * 32 + lane, __uint_as_float(v[j]));
          }
          __threadfence();
          quarter_sync();
          if (lead) atomicExch(p.sk_flags + slot * 4 + ew, 1);
        }
      } else if (rows) {
        // Partials of the walkers after this one.
        int parts = 0;
        const float* partial = nullptr;
        const int slot = (walker + 1) * CG + static_cast<int>(rank);
        if (x.role == kOwner) {
          parts = block_contributors(walker, x, p);
          partial = p.sk_ws + slot * kPartial + static_cast<size_t>(ew) * BN * 32;
          int ok = 1;
          if (lane == 0)
            for (int n = 0; n < parts && ok; ++n)
              ok = wait_flag(p.sk_flags + (slot + n * CG) * 4 + ew, p, kDetailSkFlag) ? 1 : 0;
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!quarter_all(ok != 0)) {
            if (d_first) wait_d();
            break;
          }
          for (int n = 0; n < parts; ++n)  // every lane acquires the partials
            (void)ld_acquire_gpu(p.sk_flags + (slot + n * CG) * 4 + ew);
        }
        if (parts > 0) block_add_partials(t_row, partial, kPartial * CG, parts, 32 * g, BN, 32 * kG, lane);
        auto from_tmem = [&](int c, uint32_t (&r)[16]) {
          ptx::tmem_ld_32x32b_x16(t_row + c, r);
          ptx::tmem_wait_ld();
        };
        bool ok = true;
#pragma unroll 1
        for (int cc = 0; ok && cc < kOutN && n0 + cc < p.N; cc += 64)
          ok = chunk(from_tmem, row0, n0, cc, t.z, cc + 64 < kOutN && n0 + cc + 64 < p.N);
        if (!ok) break;
        if (x.role == kOwner) {
          quarter_sync();  // every lane has read the partials
          if (lead)
            for (int n = 0; n < parts; ++n) p.sk_flags[(slot + n * CG) * 4 + ew] = 0;
        }
      }
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2)
          ptx::mbar_arrive_cluster(ptx::map_shared_rank(tempty_bar(acc), 0));
        else
          ptx::mbar_arrive(tempty_bar(acc));
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (lane == 0) ptx::bulk_wait_group_all();
    __syncwarp();
  }

  ptx::tc_fence_before_sync();
  if (CG == 2)
    ptx::cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc<CG>(tmem_base, tmem_cols);
  }
}

template <bool kAT, bool kBN, int kEpi>
cudaError_t block_set_smem(size_t smem) {
  const cudaFuncAttribute attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int bytes = static_cast<int>(smem);
  cudaError_t e = cudaFuncSetAttribute(block_kernel<1, kAT, kBN, kEpi, 2>, attr, bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(block_kernel<2, kAT, kBN, kEpi, 1>, attr, bytes);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(block_kernel<2, kAT, kBN, kEpi, 2>, attr, bytes);
  return e;
}

// `grid` CTAs, in clusters of a pair or of a tile's K splits; the launch may
// overlap the previous kernel's tail (programmatic dependent launch).
template <bool kAT, bool kBN, int kEpi>
cudaError_t block_launch(const BlockMaps& m, const BlockParams& p, int cg, int grid, size_t smem,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kernel_threads(p.epi), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  const int cluster = cg == 2 ? 2 : p.splits;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cg == 1) return cudaLaunchKernelEx(&cfg, block_kernel<1, kAT, kBN, kEpi, 2>, m, p);
  return p.epi == 2 ? cudaLaunchKernelEx(&cfg, block_kernel<2, kAT, kBN, kEpi, 2>, m, p)
                    : cudaLaunchKernelEx(&cfg, block_kernel<2, kAT, kBN, kEpi, 1>, m, p);
}

}  // namespace spgemm

#define SPGEMM_DEFINE_BLOCK(NAME, AT, BN, EPI)                                                 \
  namespace spgemm {                                                                           \
  cudaError_t block_set_smem_##NAME(size_t smem) { return block_set_smem<AT, BN, EPI>(smem); } \
  cudaError_t block_launch_##NAME(const BlockMaps& m, const BlockParams& p, int cg, int grid,  \
                                  size_t smem, cudaStream_t stream) {                          \
    return block_launch<AT, BN, EPI>(m, p, cg, grid, smem, stream);                            \
  }                                                                                            \
  }
