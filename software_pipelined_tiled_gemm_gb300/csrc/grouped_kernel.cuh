// grouped_kernel.cuh -- matrix products of many groups of rows, each with a
// weight of its own, on the roles of gemm_kernel.cuh (TMA producers, one
// tcgen05.mma issuer thread, eight epilogue warps; see there for the ring and
// accumulator protocol).  Bound by the tensor pipe where groups have hundreds of
// rows (16384 rows over 16 experts of 4096 x 4096: 332 us, 1.66 PFLOP/s), by the
// weights' bytes below (512 rows over 64 experts of 4096 x 2048: 171 us in a
// stream of calls, 6.3 TB/s).  What differs:
//
//   sizes       The groups' offsets are read on the device.  Every CTA loads
//               them, checks them and counts the tiles of each group, so the
//               launch needs no more than an upper bound and the host no copy.
//   copies      A copy costs some 90 clocks beside its bytes, whoever issues it, so
//               an operand stored along the sum comes as boxes of 64 columns x 128
//               rows, two slices of 64 in a slot (boxes of 64 rows: dW took a tenth
//               longer; boxes of two panels, 3- or 4-dimensional, longer still).
//               A's and B's are issued by a warp each.
//   schedule    Finding a tile's place takes some hundred instructions, and the
//               producer is never far ahead of the tensor cores (a slot's copies
//               take about as long as the ring's other slots last), so a
//               warp of its own describes a CTA's tiles ahead of time: the other
//               roles read some words (found by each role itself: 1 us a tile).
//               Pairs take tiles in turn: handed out from a counter as pairs become
//               free they ended 1 to 2 % sooner where groups differ, and 17 % later
//               where all pairs had the same number of equal tiles.
//   tiles       256 x n on a CTA pair, n a multiple of 32 up to 256.  The
//               weights' features lie along the MMA's M side and a group's
//               tokens along its N side, so a tile is as wide as the group's
//               rows need: a group of 300 rows costs the products of 320, not
//               of 512, and a few tokens cost what their weights' bytes do.
//   epilogue    A lane holds one feature, a column one token: neighbouring
//               lanes exchange halves, and a warp writes 64 contiguous bytes
//               of two tokens with each store.  A group's last rows need no
//               clipping by the copy engine, whose box would reach into the
//               next group, and no staging memory: the ring has all of it.
//   dW          The sum runs over a group's tokens, any number of them.  MMA
//               steps of 16 tokens that are all the group's read x and dy
//               where they lie; the last 1 to 15 come from a copy padded with
//               zeros (grouped.cu): the next group's rows would be products'
//               operands otherwise, and zero times their NaN is NaN.
//
// Under the power cap a busy wait costs clocks, so the long ones suspend: for a
// ring slot, for a full accumulator, for room in the queue of tiles (1 % of long
// calls back to back).
//
// Every sum has a fixed order, so results repeat bit for bit.
#pragma once

#include "../../include/gemm_ops.h"
#include "gemm_kernel.cuh"
#include "grouped_params.h"
#include "ptx_block.cuh"

namespace spgemm {
// What a CTA's scheduler tells the other roles of a tile.
struct alignas(16) GroupedTile {
  int rows;         // output rows that exist; 0: there are no more tiles
  int group;
  int lane0;        // first feature
  int row0;         // first output row: of the tokens, or of dW_e
  int width;        // the MMA's columns
  int slots;        // ring slots of the sum
  int first;        // kWeight: first token of the group
  int full;         // kWeight: slots whose tokens are all the group's
  int part;         // kWeight: whole steps after them
  int tail;         // kWeight: 1 where a last partial step follows
  int pad[2];
};
static_assert(sizeof(GroupedTile) == 48);

// Tile t.  `offsets` and `first_tile` (tiles along the tokens before each
// group) are this CTA's tables.
template <int kKind>
__device__ __forceinline__ GroupedTile grouped_tile(int t, const GroupedParams& p, const int* offsets,
                                                    const int* first_tile, int cap) {
  GroupedTile x{};
  if constexpr (kKind == kGroupedWeight) {
    const int tiles = grouped_tiles(p.cols, cap);
    const int per = p.tiles_lane * tiles;
    x.group = t / per;
    const int r = t - x.group * per;
    x.lane0 = (r / tiles) * kGroupedLanes;
    x.row0 = (r % tiles) * cap;
    x.rows = min(cap, p.cols - x.row0);
    x.first = offsets[x.group];
    const int m = offsets[x.group + 1] - x.first;
    x.full = m / kGroupedK;
    x.part = (m % kGroupedK) / kGroupedTail;
    x.tail = m % kGroupedTail != 0 ? 1 : 0;
    x.slots = x.full + (x.part > 0 ? 1 : 0) + x.tail;
  } else {
    int lo = 0, hi = p.groups;  // the last group whose first tile is not after t
    const int row = t / p.tiles_lane;  // (a group's tiles are tiles_lane times as many)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first_tile[mid] <= row)
        lo = mid;
      else
        hi = mid;
    }
    x.group = lo;
    const int tiles = first_tile[lo + 1] - first_tile[lo];
    const int r = t - first_tile[lo] * p.tiles_lane;
    // Eight tiles of tokens at a time, lane tile by lane tile: their rows stay
    // in L2 while the weights pass once.
    const int g = r / (8 * p.tiles_lane);
    const int high = min(8, tiles - 8 * g);
    const int s = r - g * 8 * p.tiles_lane;
    x.lane0 = (s / high) * kGroupedLanes;
    const int at = (8 * g + s % high) * cap;
    x.row0 = offsets[lo] + at;
    x.rows = min(cap, offsets[lo + 1] - x.row0);
    x.slots = (p.reduce + kGroupedK - 1) / kGroupedK;
  }
  x.width = (x.rows + kGroupedUnit - 1) / kGroupedUnit * kGroupedUnit;
  return x;
}

// Rows of no group become zero: this warp's share.
__device__ __forceinline__ void grouped_zero_rest(const GroupedParams& p, int first, int last, int worker,
                                                  int workers, int lane) {
  const int rest = first + (p.rows - last);
  for (int i = worker; i < rest; i += workers) {
    const int row = i < first ? i : last + (i - first);
    uint16_t* dst = p.out + row * p.ldo;
    for (int c = lane; c < p.lanes; c += 32) dst[c] = 0;
  }
}

template <int kKind>
__global__ void __launch_bounds__(kGroupedThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps maps, const __grid_constant__ GroupedParams p) {
  constexpr bool kAN = kKind != kGroupedForward;   // A stored (sum) x (lanes)
  constexpr bool kBN = kKind == kGroupedWeight;    // B stored (sum) x (columns)
  constexpr uint32_t kBoxBytes = 64u * kGroupedK * 2u;  // MN-major box: 64 columns x 128 rows of the sum
  constexpr uint32_t kTailBytes = 64u * kGroupedTail * 2u;
  constexpr uint32_t tmem_cols = 2u * kGroupedCols;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  const uint32_t sbase = ptx::smem_addr(smem);
  const int S = p.stages;
  const uint32_t ring_bytes = static_cast<uint32_t>(S) * kGroupedSlot;
  const uint32_t bar_base = sbase + ring_bytes;
  constexpr uint32_t kBars = 8u * (2 * kGroupedStages + 5 + 2 * kGroupedAhead);
  auto full_bar = [&](int s) { return bar_base + 8u * s; };
  auto empty_bar = [&](int s) { return bar_base + 8u * (kGroupedStages + s); };
  auto tfull_bar = [&](int a) { return bar_base + 8u * (2 * kGroupedStages + a); };
  auto tempty_bar = [&](int a) { return bar_base + 8u * (2 * kGroupedStages + 2 + a); };
  const uint32_t done_bar = bar_base + 8u * (2 * kGroupedStages + 4);
  auto next_full_bar = [&](int d) { return bar_base + 8u * (2 * kGroupedStages + 5 + d); };
  auto next_empty_bar = [&](int d) { return bar_base + 8u * (2 * kGroupedStages + 5 + kGroupedAhead + d); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + ring_bytes + kBars);
  int* cap_slot = reinterpret_cast<int*>(tmem_slot + 1);
  // (the queue of tiles 16-byte aligned)
  GroupedTile* queue = reinterpret_cast<GroupedTile*>(smem + ((ring_bytes + kBars + 8u + 15u) & ~15u));
  int* offsets = reinterpret_cast<int*>(queue + kGroupedAhead);
  int* first_tile = offsets + p.groups + 1;
  if (SPGEMM_OUT_OF_BOUNDS(S >= 1 && S <= kGroupedStages &&
                               (sbase - raw_addr) + ring_bytes + kBars + 24u + 48u * kGroupedAhead + 8u * (p.groups + 1) <=
                                   ptx::dynamic_smem_bytes(),
                           p, kCheckSmemLayout))
    return;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int walker = static_cast<int>(blockIdx.x) / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(full_bar(s), 1);
      ptx::mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), 2 * 8);
    }
    ptx::mbar_init(done_bar, 1);
    for (int d = 0; d < kGroupedAhead; ++d) {
      ptx::mbar_init(next_full_bar(d), 1);
      ptx::mbar_init(next_empty_bar(d), leader ? 11 : 10);  // producers, MMA issuer, epilogue warps
    }
    ptx::fence_barrier_init();
    ptx::tma_prefetch_desc(&maps.a);
    ptx::tma_prefetch_desc(&maps.b[0]);
  }
  if (warp == 1) {
    ptx::tmem_alloc<2>(ptx::smem_addr(tmem_slot), tmem_cols);
    ptx::tmem_relinquish<2>();
  }
  ptx::pdl_launch_dependents();
  ptx::pdl_wait_prior_grid();

  // The groups' offsets and, for tiles along the tokens, how many come before each group.
  int bad = 0;
  for (int e = threadIdx.x; e <= p.groups; e += kGroupedThreads) {
    const int64_t at = p.offsets[e], next = e < p.groups ? p.offsets[e + 1] : static_cast<int64_t>(p.rows);
    bad |= at < 0 || at > next || next > p.rows;
    offsets[e] = static_cast<int>(at);
  }
  bad = __syncthreads_or(bad);
  if constexpr (kKind != kGroupedWeight) {
    if (warp == 0 && !bad) {
      // The width of full tiles that takes the least time.
      const int slots = (p.reduce + kGroupedK - 1) / kGroupedK;
      int tiles[kGroupedCaps] = {};
      float clocks[kGroupedCaps] = {};
      for (int e = lane; e < p.groups; e += 32) {
        const int m = offsets[e + 1] - offsets[e];
#pragma unroll
        for (int i = 0; i < kGroupedCaps; ++i) {
          tiles[i] += grouped_tiles(m, grouped_cap(i));
          clocks[i] += grouped_strip_clocks(m, grouped_cap(i), slots);
        }
      }
      uint32_t best = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < kGroupedCaps; ++i) {
        const int n = __reduce_add_sync(0xffffffffu, tiles[i]) * p.tiles_lane;
        float c = clocks[i];
#pragma unroll
        for (int d = 16; d > 0; d /= 2) c += __shfl_xor_sync(0xffffffffu, c, d);
        c = grouped_clocks(c * static_cast<float>(p.tiles_lane), n, grouped_cap(i), slots, p.pairs);
        // Positive floats order as their bits; two of those make room for the width.
        best = min(best, (__float_as_uint(c) & ~3u) | static_cast<uint32_t>(i));
      }
      const int cap = grouped_cap(best & 3u);
      static_assert(kGroupedCaps == 4);
      if (lane == 0) *cap_slot = cap;
      int before = 0;
      for (int e0 = 0; e0 < p.groups; e0 += 32) {
        const int e = e0 + lane;
        const int m = e < p.groups ? offsets[e + 1] - offsets[e] : 0;
        int n = grouped_tiles(m, cap);
        for (int d = 1; d < 32; d *= 2) {
          const int up = __shfl_up_sync(0xffffffffu, n, d);
          if (lane >= d) n += up;
        }
        if (e < p.groups) first_tile[e + 1] = before + n;
        before += __shfl_sync(0xffffffffu, n, 31);
      }
      if (lane == 0) first_tile[0] = 0;
    }
  }
  ptx::tc_fence_before_sync();
  ptx::cluster_sync();
  ptx::tc_fence_after_sync();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);

  const int cap = kKind == kGroupedWeight ? p.cap : *cap_slot;
  int total = 0;
  if (!bad)
    total = p.tiles_lane * (kKind == kGroupedWeight ? p.groups * grouped_tiles(p.cols, cap) : first_tile[p.groups]);
  else if (blockIdx.x == 0 && threadIdx.x == 0)
    record_error(p.status, static_cast<int>(GEMM_ERR_INVALID_ARG), GEMM_CHECK_OFFSETS);

  // The next tile for one thread of a role that has met `n` tiles so far; rows 0: none.
  auto next_of = [&](int& n) -> GroupedTile {
    const int d = n % kGroupedAhead;
    const uint32_t parity = static_cast<uint32_t>(n / kGroupedAhead) & 1u;
    ++n;
    GroupedTile x{};
    if (!wait_bounded(next_full_bar(d), parity, p, GEMM_WAIT_NEXT_TILE)) return x;
    const uint32_t at = ptx::smem_addr(queue + d);
    const uint4 v0 = ptx::ld_shared_v4(at), v1 = ptx::ld_shared_v4(at + 16u), v2 = ptx::ld_shared_v4(at + 32u);
    memcpy(&x, &v0, 16);
    memcpy(&x.width, &v1, 16);
    memcpy(&x.part, &v2, 16);
    ptx::mbar_arrive(next_empty_bar(d));
    return x;
  };

  if (warp == 0 || warp == 11) {
    // ----------------------------------------------------- TMA producers --
    const bool for_a = warp == 0;  // the other brings B
    if (lane == 0) {
      int met = 0;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, issued_parity = 0;
      bool ok = true;
      for (GroupedTile x = next_of(met); x.rows > 0; x = next_of(met)) {
        if (SPGEMM_OUT_OF_BOUNDS(x.group >= 0 && x.group < p.groups && x.width >= kGroupedUnit &&
                                     x.width <= kGroupedCols && x.lane0 >= 0 && x.lane0 < p.lanes,
                                 p, kCheckTile)) {
          ok = false;
          break;
        }
        const int half = x.width / 2;  // columns this CTA copies
        const int a0 = x.lane0 + static_cast<int>(rank) * kBM;
        const int b0 = x.row0 + static_cast<int>(rank) * half;
        // kWeight: 64-column boxes; otherwise the smallest box of rows that holds them.
        const int box = grouped_box(x.width);
        const int boxes = (half + 63) / 64;
        for (int s = 0; s < x.slots; ++s) {
          if (!wait_bounded<true>(empty_bar(stage), phase ^ 1u, p, kDetailProducerEmpty)) {
            ok = false;
            break;
          }
          const bool tail = kBN && x.tail && s == x.slots - 1;
          const uint32_t da = sbase + stage * kGroupedSlot, db = da + kGroupedOperand;
          const uint32_t fb = ptx::map_shared_rank(full_bar(stage), 0);
          if (for_a) {
            const uint32_t bytes =
                !kBN ? kGroupedOperand + (static_cast<uint32_t>(kGroupedTail) << box) * (kGroupedK * 2u)
                     : (tail ? kTailBytes : kBoxBytes) * static_cast<uint32_t>(2 + boxes);
            if (leader) ptx::mbar_arrive_expect_tx(full_bar(stage), 2u * bytes);
            // Test hook: the first slot of the first CTA is announced but never copied.
            if (p.inject_fault != 1 || blockIdx.x != 0 || issued != 0) {
              if constexpr (!kAN) {
#pragma unroll
                for (int i = 0; i < kGroupedSlices; ++i)
                  ptx::tma_load_3d_pair(da + i * kStageA, &maps.a, s * kGroupedK + i * kBK, a0, x.group, fb);
              } else {
                const int at = !kBN ? s * kGroupedK : tail ? 0 : x.first + s * kGroupedK;
                const int z = !kBN || tail ? x.group : 0;
                const CUtensorMap* map = kBN && tail ? &maps.b[1] : &maps.a;
                ptx::tma_load_3d_pair(da, map, a0, at, z, fb);
                ptx::tma_load_3d_pair(da + kBoxBytes, map, a0 + 64, at, z, fb);
              }
            }
            issued |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          } else if constexpr (!kBN) {
#pragma unroll
            for (int i = 0; i < kGroupedSlices; ++i)
              ptx::tma_load_3d_pair(db + i * kStageA, &maps.b[box], s * kGroupedK + i * kBK, b0, 0, fb);
          } else {
            const int at = tail ? 0 : x.first + s * kGroupedK;
            const int z = tail ? x.group : 0;
            const CUtensorMap* map = tail ? &maps.b[2] : &maps.b[0];
            ptx::tma_load_3d_pair(db, map, b0, at, z, fb);
            if (boxes > 1) ptx::tma_load_3d_pair(db + kBoxBytes, map, b0 + 64, at, z, fb);
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
      }
      // Every copy this pair started must have landed before it exits.
      if (leader && for_a) {
        for (int s = 0; s < S; ++s)
          if (issued & (1u << s))
            wait_bounded(full_bar(s), (issued_parity >> s) & 1u, p, kDetailProducerDrain);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    if (lane == 0 && leader) {
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      int met = 0;
      for (GroupedTile x = next_of(met); ok && x.rows > 0; x = next_of(met)) {
        const int slots = x.slots;
        if (slots == 0) continue;  // an empty group's dW: the epilogue writes zeros
        if (!wait_bounded_cluster<2>(tempty_bar(acc), acc_phase ^ 1u, p, kDetailMmaAccEmpty)) break;
        ptx::tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kGroupedCols);
        const uint32_t idesc = ptx::instr_desc_f16(kGroupedLanes, x.width, p.bf16 != 0, kBN) |
                               (kAN ? 1u << 15 : 0u);
        for (int s = 0; s < slots; ++s) {
          if (!wait_bounded<true>(full_bar(stage), phase, p, kDetailMmaFull) ||
              SPGEMM_OUT_OF_BOUNDS(stage >= 0 && stage < S, p, kCheckMmaSlot)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after_sync();
          const uint32_t sa = sbase + stage * kGroupedSlot, sb = sa + kGroupedOperand;
          const uint64_t a_desc = kAN ? ptx::smem_desc_mn_sw128(sa, kBoxBytes, 1024u) : ptx::smem_desc_k_sw128(sa);
          const uint64_t b_desc = kBN ? ptx::smem_desc_mn_sw128(sb, kBoxBytes, 1024u) : ptx::smem_desc_k_sw128(sb);
          int steps = kGroupedK / kUmmaK;
          if (kBN && s >= x.full) steps = s == x.full && x.part > 0 ? x.part : 1;
          // A step: 32 bytes of a K-major row, the slices 16 KiB apart, or two atoms of 8 rows of the sum.
#pragma unroll
          for (int k = 0; k < kGroupedK / kUmmaK; ++k) {
            constexpr uint32_t kRows = 2048u / 16u, kSlice = kStageA / 16u;
            const uint32_t along = static_cast<uint32_t>(k) / 4u * kSlice + static_cast<uint32_t>(k) % 4u * 2u;
            if (k < steps)
              ptx::mma_f16_ss<2>(d_tmem, a_desc + (kAN ? kRows * k : along), b_desc + (kBN ? kRows * k : along), idesc,
                                 (s | k) != 0 ? 1u : 0u);
          }
          ptx::mma_commit_multicast_pair(empty_bar(stage), 0x3);
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        ptx::mma_commit_multicast_pair(tfull_bar(acc), 0x3);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      ptx::mma_commit<2>(done_bar);
      wait_bounded(done_bar, 0, p, kDetailMmaDrain);
    }
    __syncwarp();
  } else if (warp == 10) {
    // -------------------------------------------------------- scheduler --
    if (lane == 0) {
      int n = 0;
      for (int t = walker;; t += p.pairs, ++n) {
        const int d = n % kGroupedAhead;
        const uint32_t parity = static_cast<uint32_t>(n / kGroupedAhead) & 1u;
        GroupedTile x{};
        if (t < total) x = grouped_tile<kKind>(t, p, offsets, first_tile, cap);
        if (!wait_bounded<true>(next_empty_bar(d), parity ^ 1u, p, GEMM_WAIT_NEXT_FREE)) break;
        queue[d] = x;
        ptx::mbar_arrive(next_full_bar(d));
        if (t >= total) break;
      }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue --
    const int q = warp & 3;         // TMEM lane quarter
    const int g = (warp - 2) >> 2;  // which of the quarter's two warps
    const bool bf16 = p.bf16 != 0, odd = lane & 1;
    if (kKind != kGroupedWeight && p.zero_rest && !bad)
      grouped_zero_rest(p, offsets[0], offsets[p.groups], static_cast<int>(blockIdx.x) * 8 + warp - 2,
                        static_cast<int>(gridDim.x) * 8, lane);
    int acc = 0, met = 0;
    uint32_t acc_phase = 0;
    auto next_of_warp = [&]() {
      GroupedTile x{};
      if (lane == 0) x = next_of(met);
      x.rows = __shfl_sync(0xffffffffu, x.rows, 0);
      x.group = __shfl_sync(0xffffffffu, x.group, 0);
      x.lane0 = __shfl_sync(0xffffffffu, x.lane0, 0);
      x.row0 = __shfl_sync(0xffffffffu, x.row0, 0);
      x.slots = __shfl_sync(0xffffffffu, x.slots, 0);
      return x;
    };
    for (GroupedTile x = next_of_warp(); x.rows > 0; x = next_of_warp()) {
      const bool some = x.slots > 0;
      if (some) {
        int ready = 1;
        if (lane == 0) ready = wait_bounded<true>(tfull_bar(acc), acc_phase, p, kDetailEpiFull) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, ready, 0)) break;
        ptx::tc_fence_after_sync();
      }
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kGroupedCols);
      const int f = x.lane0 + static_cast<int>(rank) * kBM + q * 32 + lane;  // this lane's feature
      uint16_t* base = p.out + (kKind == kGroupedWeight ? x.group * p.out_group : 0) + x.row0 * p.ldo;
      if (x.lane0 + static_cast<int>(rank) * kBM + q * 32 < p.lanes) {
#pragma unroll 1
        for (int c = 32 * g; c < x.rows; c += 64) {
          uint32_t v[32];
          if (some) {
            ptx::tmem_ld_32x32b_x32(t_row + c, v);
            ptx::tmem_wait_ld();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0u;
          }
          const int left = x.rows - c;
          if (p.wide) {
            // Two tokens of one feature a word -> two features of one token: even lanes
            // store token 2j, odd lanes token 2j + 1.
            uint16_t* dst = base + (c + (odd ? 1 : 0)) * p.ldo + (f & ~1);
            const bool in = (f & ~1) < p.lanes;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t w = pack2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]), bf16);
              const uint32_t got = __shfl_xor_sync(0xffffffffu, w, 1);
              const uint32_t word = odd ? __byte_perm(got, w, 0x7632) : __byte_perm(w, got, 0x5410);
              if (in && 2 * j + (odd ? 1 : 0) < left) *reinterpret_cast<uint32_t*>(dst) = word;
              dst += 2 * p.ldo;
            }
          } else {
            uint16_t* dst = base + c * p.ldo + f;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (f < p.lanes && j < left)
                *dst = static_cast<uint16_t>(pack2(__uint_as_float(v[j]), 0.0f, bf16));
              dst += p.ldo;
            }
          }
        }
      }
      if (!some) continue;
      ptx::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(ptx::map_shared_rank(tempty_bar(acc), 0));
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    __syncwarp();
  }

  ptx::tc_fence_before_sync();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after_sync();
    ptx::tmem_dealloc<2>(tmem_base, tmem_cols);
  }
}

}  // namespace spgemm
