// fp8_linear.cu -- product of FP8 activations with FP8 weights, both with scales for blocks
// of 128 along the sum.
//
// Mathematics. out[m][n] = sum over blocks b of sx[m][b] sw[n / 128][b] P_b[m][n], where P_b is
// the product of 128 columns. The tensor core sums P_b (tcgen05.mma, four steps of 32 codes)
// into TMEM; the epilogue warps read it, multiply by the two scales and add to the running
// sum in registers, all FP32. While they do, the next block's product goes to another part of
// TMEM, and TMA loads the blocks after that.
//
// Two layouts. TMEM's 128 lanes are rows of one operand, its columns rows of the other:
//  * weights on the lanes, 16 to 128 tokens on the columns, for few tokens: time goes into
//    reading the weights once, so the tile is narrow and many loads are in flight. One scale
//    per column; a sum of many blocks is split over the CTAs of a cluster where there are
//    too few tiles for the SMs, and joined through distributed shared memory in a fixed order.
//  * tokens on the lanes, 256 weight rows on the columns, for many: a lane has one scale a
//    block, kept in a register.
//
// Measured: one token, 1536 into 8960 6.9 us (13.8 MB: 2.0 us of copy; the launch, one block's way through and the joining
// of the parts are the rest), 4096 into 14336 12.5; 64 tokens, 1536 into 151936 39.8 us, 6.4 TB/s of the copy's 6.8; 8192 tokens,
// 4096 into 14336 408 to 434 us, 2.22 to 2.36 PFLOP/s, bound by the way of a block's sums between products and epilogue: the
// products alone take 207 us, with the loads 276, with the hand-over of TMEM's two slots, nothing read, 387.
//
// Warps: 0 and 2 load (one thread each), 1 and 3 issue products (one thread each), the others are the epilogue.
// Every wait has a time limit; one that runs out records PULSE_ERR_TIMEOUT and ends the roles one after the other. A CTA leaves
// with nothing under way into its memory: the loaders wait for the last products to let go of their stages (what arrives there
// last); after a wait that ran out, one thread goes by the counts of what each role has begun.
#include <atomic>

#include "pulse.h"
#include "pulse_internal.h"
#include "tcgen05.cuh"

namespace pulse {
namespace {

constexpr uint32_t kLanes = 128, kBlock = 128;
constexpr uint32_t kLaneTile = kLanes * kBlock;  // bytes of the lane side's tile

__device__ __forceinline__ bool withholds(const Fp8LinearArgs& a, uint32_t rank, bool weights, uint32_t block) {
  return block == a.withheld && (a.withheld_by >> (2 * (rank & 1u) + (weights ? 1u : 0u)) & 1u);
}
// After a wait that ran out: the arrivals of the products that the two issuers, each with every other block, have begun.
template <uint32_t kStages, uint32_t kSlots>
__device__ __forceinline__ void settle_products(const uint32_t* issued, uint64_t* empty, uint64_t* tmem_full, uint64_t limit_ns) {
  for (uint32_t q = 0; q < 2; ++q) {
    const uint32_t n = issued[q];
    for (uint32_t d = n > kStages / 2 ? n - kStages / 2 : 0; d < n; ++d) {
      const uint32_t b = q + 2 * d;
      mbar_wait_often(&empty[b % kStages], (b / kStages) & 1u, limit_ns);
      if (d + kSlots / 2 >= n) mbar_wait_often(&tmem_full[b % kSlots], (b / kSlots) & 1u, limit_ns);
    }
  }
}

struct Work {
  uint32_t lane_tiles, col_tiles;
  uint32_t splits;  // CTAs of a cluster that share a tile's blocks
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const uint32_t b = cvt_bf16x2_rn(lo, hi);
  return any_nan2(lo, hi) ? canon_nan_pair(b, lo, hi) : b;
}
__device__ __forceinline__ void store_out(const Fp8LinearArgs& a, uint64_t at, float v) {
  if (a.out_bf16)
    static_cast<uint16_t*>(a.out)[at] = uint16_t(bf16_rne_bits(__float_as_uint(v)));
  else
    static_cast<float*>(a.out)[at] = v;
}

// 32 rows of a warp's columns, a row a lane in registers, to rows of the output: through 128 bytes
// of shared memory a row, 16-byte pieces swapped within groups of 8 rows so that neither
// side meets a bank twice.
template <int kCols, typename T>
__device__ __forceinline__ void store_rows(const Fp8LinearArgs& a, uint8_t* stage, uint64_t m0, uint64_t n0, const float (&acc)[kCols]) {
  constexpr int kPiece = 16 / sizeof(T), kPart = 128 / sizeof(T);  // values of 16 bytes, of a row's 128
  const uint32_t lane = threadIdx.x & 31u;
  T* out = static_cast<T*>(a.out);
#pragma unroll
  for (int p = 0; p < kCols / kPart; ++p) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float* v = acc + p * kPart + j * kPiece;
      uint4 q;
      if (sizeof(T) == 4) {
        q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = bf16_pair(v[2 * i < kPiece ? 2 * i : 0], v[2 * i + 1 < kPiece ? 2 * i + 1 : 0]);
        q = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = q;
    }
    __syncwarp();
    const uint64_t n = n0 + p * kPart;
    if (n >= a.n) return;
    if (a.out_vec && n + kPart <= a.n) {
#pragma unroll
      for (uint32_t r = 0; r < 32; r += 4) {
        const uint32_t row = r + (lane >> 3), j = lane & 7u;
        const uint4 q = *reinterpret_cast<const uint4*>(stage + row * 128 + ((j ^ (row & 7)) << 4));
        if (m0 + row < a.rows) *reinterpret_cast<uint4*>(out + (m0 + row) * a.out_stride + n + j * kPiece) = q;
      }
    } else {
      for (uint32_t row = 0; row < 32 && m0 + row < a.rows; ++row)
#pragma unroll
        for (uint32_t c = lane; c < kPart; c += 32)
          if (n + c < a.n)
            out[(m0 + row) * a.out_stride + n + c] =
                *reinterpret_cast<const T*>(stage + row * 128 + (((c / kPiece) ^ (row & 7)) << 4) + c % kPiece * sizeof(T));
    }
  }
}

// A lane's column of the output, one value for each of a warp's tokens. The type is chosen outside and the address moved by a
// row: with both found anew for each value 64 x 1536 x 151936 took 45 us instead of 39, 256 x 1024 x 4096 6.3 instead of 5.1.
template <int kCols, typename T>
__device__ __forceinline__ void store_columns(const Fp8LinearArgs& a, uint64_t m0, uint64_t n, const unsigned long long (&sums)[kCols / 2]) {
  if (n >= a.n) return;
  const uint32_t left = m0 < a.rows ? uint32_t(a.rows - m0) : 0u;
  T* p = static_cast<T*>(a.out) + m0 * a.out_stride + n;
#pragma unroll
  for (uint32_t c = 0; c < kCols; c += 2) {
    float v[2];
    unpair(sums[c / 2], v[0], v[1]);
    const uint32_t both = sizeof(T) == 2 ? bf16_pair(v[0], v[1]) : 0u;
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i, p += a.out_stride) {
      if (c + i >= left) continue;
      if constexpr (sizeof(T) == 2)
        *p = uint16_t(both >> (16 * i));
      else
        *p = v[i];
    }
  }
}

// Adds the next block's product to a warp's running sums: its 32 lanes, columns from `at` on. `scales(k)`
// gives the factors of columns k .. k + 3.
template <int kCols, int kChunk, typename Scales, typename Done>
__device__ __forceinline__ void add_product(unsigned long long (&sums)[kCols / 2], uint32_t at, Scales scales, Done done) {
#pragma unroll
  for (int c = 0; c < kCols; c += kChunk) {
    unsigned long long d[kChunk / 2];
    tmem_read(d, at + c);
    if (c + kChunk == kCols) {
      tmem_fence_before();
      done();
    }
#pragma unroll
    for (int k = 0; k < kChunk; k += 4) {
      const ulonglong2 f = scales(c + k);
      fma2(sums[(c + k) / 2], d[k / 2], f.x);
      fma2(sums[(c + k) / 2 + 1], d[k / 2 + 1], f.y);
    }
  }
}

// ------------------------------------------------- many tokens: tokens on the lanes
//
// A pair of CTAs takes 256 tokens x 256 weight rows; each loads half of both operands and holds the
// sums of its 128 tokens.
// 6 stages and the output's rows are what shared memory holds. 16 epilogue warps of 64 columns, with 5 stages: 477 us for
// 8192 x 4096 x 14336 instead of 410.
constexpr int kPairStages = 6, kPairWarps = 8, kPairThreads = 128 + 32 * kPairWarps;
constexpr uint32_t kPairStage = 2 * kLaneTile;
constexpr uint32_t kPairBytes = 1024 + kPairStages * kPairStage + kPairWarps * 4096;
constexpr uint32_t kPairSlots = 2;  // products in TMEM
constexpr uint32_t kPairCols = 256 / (kPairWarps / 4);  // columns of an epilogue warp
constexpr uint32_t kPairFew = 40, kPairMany = 232;  // registers of the first four warps' threads and of the epilogue's

struct PairBars {
  uint64_t full[kPairStages], empty[kPairStages], tmem_full[kPairSlots], tmem_empty[kPairSlots];
  uint32_t tmem, stop;
  uint32_t loaded[4];  // blocks that the loaders have begun, of the even CTA's tokens, weights, of the odd one's (in the even CTA)
  uint32_t issued[2];  // blocks that the issuers have (in both)
};

__global__ void __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap token_map, const __grid_constant__ CUtensorMap weight_map,
                   Fp8LinearArgs a, Work work) {
  extern __shared__ uint8_t raw[];
  __shared__ PairBars bars;
  uint8_t* tiles = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u, rank = cluster_rank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
    for (int i = 0; i < int(kPairSlots); ++i) mbar_init(&bars.tmem_full[i], 1), mbar_init(&bars.tmem_empty[i], 2 * kPairWarps);
    bars.stop = 0;
    fence_mbar_init();
    prefetch_map(&token_map);
    prefetch_map(&weight_map);
  }
  if (warp == 2) tmem_alloc_pair(&bars.tmem, 512);
  __syncwarp();
  tmem_fence_before();
  cluster_sync();  // the other CTA's barriers, too
  tmem_fence_after();
  stream_ready();
  const uint32_t tmem = bars.tmem;

  const uint32_t tiles_all = work.lane_tiles * work.col_tiles, first = blockIdx.x >> 1, step = gridDim.x >> 1;
  volatile uint32_t* stop = &bars.stop;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*stop == 0 && mbar_wait_often(bar, parity, a.wait_ns)) return true;
    if (*stop == 0) record_error(a.error_word, kErrTimeout);
    *stop = 1;
    peer_store(&bars.stop, rank ^ 1u, 1);
    return false;
  };

  // 384 threads of 168 registers become 128 of 40 and 256 of 232 (pairs_fit: these are not more)
  if (warp < 4) {
    fewer_registers<kPairFew>();
    if ((warp & 1u) == 0 && lane == 0) {
      // two threads load: tokens, and weights
      const bool tokens = warp == 0;
      const uint64_t keep = l2_policy_evict_last();
      const CUtensorMap* map = tokens ? &token_map : &weight_map;
      uint32_t stage = 0, phase = 0, loaded = 0;
      bool live = true;
      for (uint32_t t = first; t < tiles_all && live; t += step) {
        const uint32_t ct = t / work.lane_tiles, lt = t - ct * work.lane_tiles, from = (tokens ? lt : ct) * 256 + rank * 128;
        for (uint32_t b = 0; b < a.blocks; ++b) {
          live = !withholds(a, rank, !tokens, loaded) && wait(&bars.empty[stage], phase ^ 1u);
          if (!live) break;
          if (tokens && rank == 0) mbar_arrive_expect_tx(&bars.full[stage], 2 * kPairStage);
          tma_load_2d_pair(tiles + stage * kPairStage + (tokens ? 0u : kLaneTile), map, b * kBlock, from,
                           peer_addr(&bars.full[stage], 0), keep);
          ++loaded;
          if (++stage == kPairStages) stage = 0, phase ^= 1u;
        }
      }
      for (int i = 0; i < kPairStages && live; ++i) {
        live = wait(&bars.empty[stage], phase ^ 1u);
        if (++stage == kPairStages) stage = 0, phase ^= 1u;
      }
      peer_store(&bars.loaded[2 * rank + (tokens ? 0 : 1)], 0, loaded);
    } else if ((warp & 1u) && lane == 0 && rank == 0) {
      // Two threads issue, each for one slot of TMEM: between two blocks a thread spends some 600 cycles
      // in waits and commits, longer than the products that are queued behind one another.
      constexpr uint32_t instruction = fp8_instruction(256, 256);
      const uint32_t slot = warp >> 1, total = (tiles_all - first + step - 1) / step * a.blocks;  // first < tiles_all
      uint32_t stage = slot, phase = 0, done = 0;
      bool live = true;
      for (uint32_t b = slot; b < total; b += 2, ++done) {
        live = wait(&bars.full[stage], phase) && wait(&bars.tmem_empty[slot], (done & 1u) ^ 1u);
        if (!live) break;
        tmem_fence_after();
        const uint64_t ad = smem_desc(tiles + stage * kPairStage), bd = smem_desc(tiles + stage * kPairStage + kLaneTile);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) mma_fp8_pair(tmem + slot * 256u, ad + 2 * k, bd + 2 * k, instruction, k > 0);
        mma_commit_pair(&bars.tmem_full[slot]);
        mma_commit_pair(&bars.empty[stage]);
        if ((stage += 2) >= kPairStages) stage -= kPairStages, phase ^= 1u;
      }
      for (uint32_t r = 0; r < 2; ++r) peer_store(&bars.issued[slot], r, done);
    }
  } else {
    more_registers<kPairMany>();
    const uint32_t quarter = warp & 3u, part = (warp - 4u) >> 2;  // lanes and columns of the warp
    const uint32_t row = quarter * 32u + lane;
    uint8_t* stage_out = tiles + kPairStages * kPairStage + (warp - 4u) * 4096u;
    uint32_t slot = 0, slot_phase = 0;
    bool live = true;
    for (uint32_t t = first; t < tiles_all && live; t += step) {
      const uint32_t ct = t / work.lane_tiles, lt = t - ct * work.lane_tiles;
      const uint64_t token = uint64_t(lt) * 256 + rank * 128 + row, group = uint64_t(ct) * 2 + part * kPairCols / 128;
      const bool there = token < a.rows && group * 128 < a.n;
      const float* sx = a.x_scales + (there ? token * a.x_scales_stride : 0);
      const float* sw = a.w_scales + (there ? group * a.w_scales_stride : 0);
      unsigned long long sums[kPairCols / 2];
#pragma unroll
      for (uint32_t c = 0; c < kPairCols / 2; ++c) sums[c] = 0;
      // one scale a lane and block, asked for a block ahead
      float x_next = there ? sx[0] : 0.0f, w_next = there ? sw[0] : 0.0f;
      for (uint32_t b = 0; b < a.blocks && live; ++b) {
        const unsigned long long f = pair_of(x_next * w_next, x_next * w_next);
        if (there && b + 1 < a.blocks) x_next = sx[b + 1], w_next = sw[b + 1];
        live = __all_sync(0xFFFFFFFFu, wait(&bars.tmem_full[slot], slot_phase));
        if (!live) break;
        tmem_fence_after();
        const uint32_t at = tmem + slot * 256u + part * kPairCols + ((quarter * 32u) << 16);
        add_product<kPairCols, 16>(sums, at, [&](int) { return make_ulonglong2(f, f); },
                             [&] { if (lane == 0) mbar_arrive_at(peer_addr(&bars.tmem_empty[slot], 0)); });
        if (++slot == kPairSlots) slot = 0, slot_phase ^= 1u;
      }
      if (!live) break;
      float acc[kPairCols];
#pragma unroll
      for (uint32_t c = 0; c < kPairCols; c += 2) unpair(sums[c / 2], acc[c], acc[c + 1]);
      const uint64_t m0 = uint64_t(lt) * 256 + rank * 128 + quarter * 32u, n0 = uint64_t(ct) * 256 + part * kPairCols;
      if (a.out_bf16)
        store_rows<kPairCols, uint16_t>(a, stage_out, m0, n0, acc);
      else
        store_rows<kPairCols, float>(a, stage_out, m0, n0, acc);
    }
  }
  __syncwarp();
  tmem_fence_before();
  cluster_sync();  // no CTA leaves while the other arrives at its barriers or reads its operands
  if (*stop != 0) {  // known to both CTAs
    if (warp == 2 && lane == 0) {
      if (rank == 0) {  // the copies of both CTAs arrive here
        uint32_t most = 0;
        for (int k = 0; k < 4; ++k) most = max(most, bars.loaded[k]);
        for (uint32_t i = most > kPairStages ? most - kPairStages : 0; i < most; ++i) {
          uint64_t* bar = &bars.full[i % kPairStages];
          uint32_t bytes = 0;
          for (int k = 0; k < 4; ++k) bytes += i < bars.loaded[k] ? kLaneTile : 0u;
          if (i >= bars.loaded[0])
            mbar_arrive_expect_tx(bar, bytes);
          else if (bytes < 2 * kPairStage)
            mbar_complete_tx(bar, 2 * kPairStage - bytes);
          mbar_wait_often(bar, (i / kPairStages) & 1u, a.wait_ns);
        }
      }
      settle_products<kPairStages, kPairSlots>(bars.issued, bars.empty, bars.tmem_full, a.wait_ns);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 2) {
    tmem_fence_after();
    tmem_free_pair(tmem, 512);
  }
}

// ------------------------------------------------- few tokens: weights on the lanes
template <int kCols>
struct Narrow {
  // of the columns, each with four epilogue warps: with one half for 64 columns 64 x 1536 x 151936 took 54 us, with two 45
  static constexpr int kHalves = kCols >= 64 ? 2 : 1;
  static constexpr int kWarps = 4 * kHalves, kThreads = 128 + 32 * kWarps;
  static constexpr int kWarpCols = kCols / kHalves;
  static constexpr int kSlots = 4;  // products in TMEM
  static constexpr uint32_t kTmemCols = kSlots * kCols;
  static constexpr uint32_t kStageBytes = kLaneTile + kCols * kBlock;
  static constexpr int kStages = kCols <= 32 ? 10 : kCols <= 64 ? 8 : 6;
  static constexpr uint32_t kBytes = 1024 + kStages * kStageBytes + 2 * 4 * kCols * 4;
};

struct NarrowBars {
  uint64_t full[16], empty[16], tmem_full[4], tmem_empty[4];
  uint32_t tmem, stop;
  uint32_t loaded[2], issued[2];  // blocks that the loaders (tokens, weights) and the issuers have begun
};

template <int kCols>
__global__ void __launch_bounds__(Narrow<kCols>::kThreads, 1)
linear_narrow_kernel(const __grid_constant__ CUtensorMap weight_map, const __grid_constant__ CUtensorMap token_map,
                     Fp8LinearArgs a, Work work) {
  using S = Narrow<kCols>;
  extern __shared__ uint8_t raw[];
  __shared__ NarrowBars bars;
  uint8_t* tiles = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  float* col_scales = reinterpret_cast<float*>(tiles + S::kStages * S::kStageBytes);  // [2][4][kCols]
  const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31u;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(&bars.full[i], 1), mbar_init(&bars.empty[i], 1);
    for (int i = 0; i < S::kSlots; ++i) mbar_init(&bars.tmem_full[i], 1), mbar_init(&bars.tmem_empty[i], S::kWarps);
    bars.stop = 0;
    fence_mbar_init();
    prefetch_map(&weight_map);
    prefetch_map(&token_map);
  }
  if (warp == 2) tmem_alloc(&bars.tmem, S::kTmemCols);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  stream_ready();
  const uint32_t tmem = bars.tmem;

  const uint32_t tiles_all = work.lane_tiles * work.col_tiles;
  const uint32_t rank = blockIdx.x % work.splits, first = blockIdx.x / work.splits, step = gridDim.x / work.splits;
  const uint32_t b0 = uint32_t(uint64_t(rank) * a.blocks / work.splits);
  const uint32_t b1 = uint32_t(uint64_t(rank + 1) * a.blocks / work.splits);
  volatile uint32_t* stop = &bars.stop;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*stop == 0 && mbar_wait_often(bar, parity, a.wait_ns)) return true;
    if (*stop == 0) record_error(a.error_word, kErrTimeout);
    *stop = 1;
    return false;
  };

  if (warp < 4 && (warp & 1u) == 0 && lane == 0) {  // two threads load: weights, and tokens
    const bool weights = warp == 0;
    const uint64_t policy = weights && work.col_tiles == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
    const CUtensorMap* map = weights ? &weight_map : &token_map;
    uint32_t stage = 0, phase = 0, loaded = 0;
    bool live = true;
    for (uint32_t t = first; t < tiles_all && live; t += step) {  // tiles of the same weights follow one another
      const uint32_t lt = t / work.col_tiles, ct = t - lt * work.col_tiles, from = weights ? lt * kLanes : ct * kCols;
      for (uint32_t b = b0; b < b1; ++b) {
        live = !withholds(a, rank, weights, loaded) && wait(&bars.empty[stage], phase ^ 1u);
        if (!live) break;
        if (weights) mbar_arrive_expect_tx(&bars.full[stage], S::kStageBytes);
        tma_load_2d(tiles + stage * S::kStageBytes + (weights ? 0u : kLaneTile), map, b * kBlock, from, &bars.full[stage], policy);
        ++loaded;
        if (++stage == S::kStages) stage = 0, phase ^= 1u;
      }
    }
    for (int i = 0; i < S::kStages && live; ++i) {
      live = wait(&bars.empty[stage], phase ^ 1u);
      if (++stage == S::kStages) stage = 0, phase ^= 1u;
    }
    bars.loaded[weights ? 1 : 0] = loaded;
  } else if (warp < 4 && lane == 0) {  // two threads issue, each for every other slot of TMEM
    constexpr uint32_t instruction = fp8_instruction(kLanes, kCols);
    const uint32_t total = (tiles_all - first + step - 1) / step * (b1 - b0);  // first < tiles_all
    uint32_t stage = warp >> 1, phase = 0, slot = warp >> 1, slot_phase = 0, done = 0;
    bool live = true;
    for (uint32_t b = warp >> 1; b < total; b += 2, ++done) {
      live = wait(&bars.full[stage], phase) && wait(&bars.tmem_empty[slot], slot_phase ^ 1u);
      if (!live) break;
      tmem_fence_after();
      const uint64_t ad = smem_desc(tiles + stage * S::kStageBytes);
      const uint64_t bd = smem_desc(tiles + stage * S::kStageBytes + kLaneTile);
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) mma_fp8(tmem + slot * kCols, ad + 2 * k, bd + 2 * k, instruction, k > 0);
      mma_commit(&bars.tmem_full[slot]);
      mma_commit(&bars.empty[stage]);
      if ((stage += 2) >= S::kStages) stage -= S::kStages, phase ^= 1u;
      if ((slot += 2) >= S::kSlots) slot -= S::kSlots, slot_phase ^= 1u;
    }
    bars.issued[warp >> 1] = done;
  } else if (warp >= 4) {
    const uint32_t me = threadIdx.x - 128u, quarter = warp & 3u, row = quarter * 32u + lane;
    const uint32_t col0 = (warp - 4u) / 4u * S::kWarpCols;  // first of the warp's columns
    uint32_t slot = 0, slot_phase = 0, flip = 0;
    bool live = true;  // a warp that gave up still meets the others at their barrier
    for (uint32_t t = first; t < tiles_all; t += step) {
      const uint32_t lt = t / work.col_tiles, ct = t - lt * work.col_tiles;
      // this thread's scales: of one column's token
      const uint64_t token = uint64_t(ct) * kCols + (me < kCols ? me : 0);
      const bool there = token < a.rows;
      const float* sx = a.x_scales + (there ? token * a.x_scales_stride : 0);
      const float* sw = a.w_scales + lt * a.w_scales_stride;
      // four blocks' at a time through shared memory, asked for four blocks ahead
      float x_next[4], w_next[4];
      auto fetch = [&](uint32_t b) {
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          const bool some = there && b + i < b1;
          x_next[i] = some ? sx[b + i] : 0.0f;
          w_next[i] = some ? sw[b + i] : 0.0f;
        }
      };
      unsigned long long sums[S::kWarpCols / 2];
#pragma unroll
      for (int c = 0; c < S::kWarpCols / 2; ++c) sums[c] = 0;
      fetch(b0);
      for (uint32_t b = b0; b < b1; b += 4) {
        float* set = col_scales + flip * 4 * kCols;  // two sets: a warp writes the next one while another reads this one
        if (me < kCols)
#pragma unroll
          for (int i = 0; i < 4; ++i) set[i * kCols + me] = x_next[i] * w_next[i];
        asm volatile("bar.sync 1, %0;" ::"n"(32 * S::kWarps) : "memory");
        fetch(b + 4);
        flip ^= 1u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          if (b + i >= b1) break;
          if (live) live = wait(&bars.tmem_full[slot], slot_phase);
          live = __all_sync(0xFFFFFFFFu, live);
          if (live) {
            tmem_fence_after();
            add_product<S::kWarpCols, 16>(
                sums, tmem + slot * kCols + col0 + ((quarter * 32u) << 16),
                [&](int k) { return *reinterpret_cast<const ulonglong2*>(set + i * kCols + col0 + k); },
                [&] { if (lane == 0) mbar_arrive(&bars.tmem_empty[slot]); });
          }
          if (++slot == S::kSlots) slot = 0, slot_phase ^= 1u;
        }
      }
      if (!live) continue;
      if (work.splits > 1) {  // the only tile of this cluster: its loads and products are done, their memory is free
        float* part = reinterpret_cast<float*>(tiles) + col0 * kLanes + row;
#pragma unroll
        for (int c = 0; c < S::kWarpCols; c += 2) unpair(sums[c / 2], part[c * kLanes], part[(c + 1) * kLanes]);
      } else if (a.out_bf16) {
        store_columns<S::kWarpCols, uint16_t>(a, uint64_t(ct) * kCols + col0, uint64_t(lt) * kLanes + row, sums);
      } else {
        store_columns<S::kWarpCols, float>(a, uint64_t(ct) * kCols + col0, uint64_t(lt) * kLanes + row, sums);
      }
    }
  }

  __syncwarp();
  if (work.splits > 1) {
    cluster_sync();
    if (warp >= 4) {
      const uint32_t lt = first / work.col_tiles, ct = first - lt * work.col_tiles;
      const uint32_t row = (warp & 3u) * 32u + lane;
      const uint64_t n = uint64_t(lt) * kLanes + row;
      const float* part = reinterpret_cast<const float*>(tiles);
      const uint32_t c0 = rank * kCols / work.splits, c1 = (rank + 1) * kCols / work.splits;
      // eight columns of two CTAs at once: a read of another CTA's memory takes some 0.3 us (256 x 1024 x 4096 with one at
      // a time 14.8 us)
      constexpr uint32_t kBatch = 8;
      for (uint32_t c = c0 + (warp - 4u) / 4u; c < c1; c += S::kHalves * kBatch) {
        float sum[kBatch] = {};
        for (uint32_t r = 0; r < work.splits; r += 2) {
          float v[2][kBatch];
#pragma unroll
          for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
            for (uint32_t j = 0; j < kBatch; ++j)
              v[i][j] = c + j * S::kHalves < c1 ? peer_load(part + (c + j * S::kHalves) * kLanes + row, r + i) : 0.0f;
#pragma unroll
          for (uint32_t j = 0; j < kBatch; ++j) sum[j] = sum[j] + v[0][j] + v[1][j];
        }
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
          const uint64_t m = uint64_t(ct) * kCols + c + j * S::kHalves;
          if (c + j * S::kHalves < c1 && m < a.rows && n < a.n) store_out(a, m * a.out_stride + n, sum[j]);
        }
      }
    }
    cluster_sync();  // no CTA leaves while another reads its part
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == 2) {
    if (lane == 0 && *stop != 0) {
      const uint32_t tokens = bars.loaded[0], weights = bars.loaded[1], most = max(tokens, weights);
      for (uint32_t i = most > S::kStages ? most - S::kStages : 0; i < most; ++i) {
        uint64_t* bar = &bars.full[i % S::kStages];
        if (i >= weights)
          mbar_arrive_expect_tx(bar, kCols * kBlock);
        else if (i >= tokens)
          mbar_complete_tx(bar, kCols * kBlock);
        mbar_wait_often(bar, (i / S::kStages) & 1u, a.wait_ns);
      }
      settle_products<S::kStages, S::kSlots>(bars.issued, bars.empty, bars.tmem_full, a.wait_ns);
    }
    __syncwarp();
    tmem_fence_after();
    tmem_free(tmem, S::kTmemCols);
  }
}

// ----------------------------------------------------------------- the host side

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {  // asked for again where it was not to be had
  static std::atomic<EncodeTiled> known{nullptr};
  EncodeTiled f = known.load(std::memory_order_acquire);
  if (f != nullptr) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiled>(p);
  known.store(f, std::memory_order_release);
  return f;
}

// Boxes of 128 codes by `box` rows; what lies outside of the matrix reads as 0.
bool make_map(CUtensorMap* map, const uint8_t* p, uint64_t rows, uint64_t cols, uint64_t stride, uint32_t box) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {rows > 1 ? stride : (cols + 15) / 16 * 16};
  const cuuint32_t boxes[2] = {kBlock, box}, steps[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, boxes, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Lets a kernel use its shared memory on the current device, once for each.
bool allow_shared(const void* kernel, uint32_t bytes, std::atomic<uint64_t>& ready) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return false;
  const uint64_t bit = device < 64 ? uint64_t(1) << device : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) != cudaSuccess) return false;
  ready.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

template <typename K>
int launch(K kernel, uint32_t ctas, uint32_t threads, uint32_t bytes, uint32_t cluster, const CUtensorMap& first,
           const CUtensorMap& second, const Fp8LinearArgs& a, const Work& w, cudaStream_t stream) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(ctas);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = bytes;
  c.stream = stream;
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, first, second, a, w) == cudaSuccess ? PULSE_OK : PULSE_ERR_CUDA;
}

// Whether the pair kernel was compiled with the registers that its warps share out anew: more than the launch has would be
// waited for without end. 168 a thread are just enough; a compiler that gives it fewer leaves it out.
bool pairs_fit() {
  static std::atomic<int> known{0};
  int registers = known.load(std::memory_order_relaxed);
  if (registers == 0) {
    cudaFuncAttributes f{};
    if (cudaFuncGetAttributes(&f, linear_pair_kernel) != cudaSuccess) return false;
    known.store(registers = f.numRegs, std::memory_order_relaxed);
  }
  return registers * kPairThreads >= int(128 * kPairFew + 32 * kPairWarps * kPairMany);
}

int launch_pair(const Fp8LinearArgs& a, int sms, cudaStream_t stream) {
  static std::atomic<uint64_t> ready{0};
  if (!allow_shared(reinterpret_cast<const void*>(linear_pair_kernel), kPairBytes, ready)) return PULSE_ERR_CUDA;
  CUtensorMap tokens, weights;
  if (!make_map(&tokens, a.x, a.rows, a.k, a.x_stride, 128) || !make_map(&weights, a.w, a.n, a.k, a.w_stride, 128))
    return PULSE_ERR_CUDA;
  Work w{(a.rows + 255) / 256, (a.n + 255) / 256, 1};
  const uint64_t all = uint64_t(w.lane_tiles) * w.col_tiles, pairs = uint64_t(sms) / 2;
  if (all >= (1ull << 31)) return PULSE_ERR_RANGE;
  return launch(linear_pair_kernel, uint32_t(all < pairs ? all : pairs) * 2, kPairThreads, kPairBytes, 2, tokens, weights, a, w, stream);
}

template <int kCols>
int launch_narrow(const Fp8LinearArgs& a, int sms, cudaStream_t stream) {
  using S = Narrow<kCols>;
  static std::atomic<uint64_t> ready{0};
  if (!allow_shared(reinterpret_cast<const void*>(linear_narrow_kernel<kCols>), S::kBytes, ready)) return PULSE_ERR_CUDA;
  CUtensorMap tokens, weights;
  if (!make_map(&tokens, a.x, a.rows, a.k, a.x_stride, kCols) || !make_map(&weights, a.w, a.n, a.k, a.w_stride, kLanes))
    return PULSE_ERR_CUDA;
  Work w{(a.n + kLanes - 1) / kLanes, (a.rows + kCols - 1) / kCols, 1};
  const uint64_t all = uint64_t(w.lane_tiles) * w.col_tiles;
  if (all >= (1ull << 31)) return PULSE_ERR_RANGE;
  // As many CTAs a tile as the SMs hold at once, two blocks each at least. Eight need eight SMs of one cluster's group
  // free, which 16 clusters do not find at once: 128 x 4096 x 2048 (16 tiles) 18.3 us with eight, 10.5 with four; 8 tiles
  // (128 x 8192 x 1024) 11.3 with eight, 14.0 with four. More CTAs than SMs do not pay, even to even out a second round: 171
  // tiles (7 x 11008 x 21888) 49.7 us, in halves 49.5, in quarters 53.9; 224 tiles (1 x 4096 x 28672) 22.0, 28.2, 43.7.
  auto fits = [&](uint64_t splits) { return all * splits <= uint64_t(sms) / (splits == 8 ? 2 : 1) && a.blocks >= splits * 2; };
  while (w.splits < 8 && fits(w.splits * 2)) w.splits *= 2;
  const uint64_t ctas = w.splits > 1 ? all * w.splits : all < uint64_t(sms) ? all : uint64_t(sms);
  return launch(linear_narrow_kernel<kCols>, uint32_t(ctas), S::kThreads, S::kBytes, w.splits, weights, tokens, a, w, stream);
}

}  // namespace

// Few tokens: the narrowest tile that holds them, since a narrower one than needed reads the weights again and a wider one
// multiplies zeros (weights of 151936 x 1536, us with 16, 32, 64, 128 columns: 16 tokens 37, 39, 47, 67; 32 tokens 51, 37, 39, 63;
// 64 tokens 94, 56, 39, 54; 128 tokens 181, 105, 69, 55 and by pairs 68). More: the widest tiles that still give every SM one
// at most; where even those of 128 columns do not, the pair's, which read half as much for a product (4096 columns into n
// outputs, us with 64, 128, pair: 256 tokens, n = 4096 12.2, 15.0, 20.6; n = 9728 21.6, 19.1, 21.1; n = 14336 30.8, 34.9, 21.7;
// 512 tokens, n = 2048 12.0, 14.8, 20.5; n = 4096 21.4, 18.7, 20.7; n = 9728 39.9, 34.6, 21.7).
int launch_fp8_linear(const Fp8LinearArgs& a, int sms, bool pairs, cudaStream_t stream) {
  auto tiles = [&](uint32_t cols) { return uint64_t((a.rows + cols - 1) / cols) * ((a.n + kLanes - 1) / kLanes); };
  if (a.rows <= 16) return launch_narrow<16>(a, sms, stream);
  if (a.rows <= 32) return launch_narrow<32>(a, sms, stream);
  if (a.rows <= 64 || tiles(64) <= uint64_t(sms)) return launch_narrow<64>(a, sms, stream);
  if (a.rows <= 128 || tiles(128) <= uint64_t(sms) || !pairs || !pairs_fit()) return launch_narrow<128>(a, sms, stream);
  return launch_pair(a, sms, stream);
}

}  // namespace pulse
