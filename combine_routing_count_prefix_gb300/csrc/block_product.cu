// block_product.cu -- llmoe_expert_product (include/llmoe_block.h): matrix
// products grouped by expert over the received rows.
//
// The weights are the M side of the tensor-core product and the received rows
// its N side: D[feature][row] = sum_k w[feature][k] x[row][k].  An expert has
// from none to thousands of rows; N takes any multiple of 32 up to 256, so few
// rows cost few columns, while the weights, which are most of the bytes there,
// stream through full 256-row tiles.  A pair of CTAs (one cluster) works on one
// tile of 256 features x up to kMaxRows rows: each CTA holds 128 of the
// features and half of the rows in shared memory and 128 x N sums in its tensor
// memory (tcgen05, cta_group::2).
//
// The rows of an expert lie in R buckets of consecutive rows.  A tile takes
// them in groups of four (a bucket's last group may reach past its count: those
// columns are computed from whatever lies there and never stored), and runs of
// groups load as boxes of 4 to 128 rows.
//
// Persistent pairs; every pair takes tiles pair, pair + pairs, ... of a list
// that each CTA derives from the counts in its prologue.  Inside a CTA:
//   warps 0, 3  load: one TMA box of w, and a few of x, per 128 bytes of K into
//               a ring (warp 3 also allocates the tensor memory)
//   warp 1      (first CTA of the pair) issues the products
//   warp 2      plans: the tile's expert, features and received rows
//   warps 4-11  epilogue: sums from tensor memory, SwiGLU, rounding, stores,
//               while the next tile's products run into the other accumulator
//   warps 12-15 8-bit operands: move the scales to shared memory
// Every wait is bounded (kSpinLimit cycles); on expiry the role records
// LLMOE_DEV_TIMEOUT and leaves its loop, the others follow when their own waits
// expire, and all meet at the end to free the tensor memory.  A copy in flight
// then was issued at least one expired wait (a second) earlier.
//
// What bounds it, and what was measured on a GB300 (6.69 TB/s copy rate, 1.90
// PFLOP/s cuBLAS bf16 in a burst, 1.73 in a loop under the power cap):
// - few rows per expert: the weights' bytes.  256 experts x ~32 rows, 7168 ->
//   2 x 2048: 2.19-2.26 ms bf16 (6.7-6.9 TB/s), 1.14-1.19 ms MX8.  The ring is
//   what covers HBM's latency: MX8 tiles of 192 rows, which leave room for a
//   seventh stage, took 2% less here and 5% more with many rows.
// - many rows: the tensor cores, then power.  16 experts x ~1024 rows: 527-555
//   us in a burst (1.73-1.82 PFLOP/s), 620-655 us steadily.  A row costs its
//   columns padded to 4 per bucket and 32 per share.  MX8 (2048 -> 7168): 182-188
//   us in a burst (2.6 PFLOP/s), 212-218 steadily; there the epilogue and the
//   scale copies of a tile of 16 steps take what the tensor cores leave.
// - one row: eight experts' weights, 76-79 us of 70; 6 us are launch, plan, the
//   first load's latency and the last tile's stores.
// What the structure bought, in microseconds (dense bf16 / decode bf16 / decode
// MX8): rows by four-row gathers and one load warp 2311 / 3433 / 3547; boxes of
// consecutive rows, one box of w, four scale warps 722 / 2289 / 1582; one
// elected thread per role (a lane predicate leaves every TMA and tensor
// instruction in a loop over lanes) 683 / 2267 / 1520; two boxes per run, two
// epilogue sets 656 / 2272 / 1285; no cluster release in the scale warps (2600
// cycles each) 651 / 2265 / 1177; loads by two warps, the epilogue as below 620
// / 2197 / 1136.
#include "block_plan.cuh"

namespace {

// Per operand type: the most rows per tile and the ring stage's layout (128
// bytes of K: 64 values of 16 bits or 128 of 8 bits).
template <bool kMx>
struct Shape {
  static constexpr int kThreads = kMx ? 512 : 384;
  // two accumulators of kMaxRows columns
  static constexpr int kMaxRows = kMx ? 224 : 256;
  static constexpr int kBytesA = 128 * 128, kBytesB = kMaxRows / 2 * 128;
  static constexpr int kStage = kBytesA + kBytesB;
  // 8-bit operands: scales in slots of four steps; a step's are 512 bytes for
  // the CTA's 128 rows of w and 1024 for up to 256 rows of x, and 12 columns
  // of tensor memory, reused after kScaleRing steps
  static constexpr int kSlots = kMx ? 3 : 0;
  static constexpr int kSlot = 4 * (512 + 1024);
  static constexpr int kScaleColumns = 12, kScaleRing = 5;
  static_assert(2 * kMaxRows + (kMx ? kScaleRing * kScaleColumns : 0) <= 512, "tensor memory has 512 columns");
};

// Byte offsets in dynamic shared memory, from its first 1024-byte boundary.
struct SmemLayout {
  uint32_t scales, boxes, rows, tiles, amax, bars, tmem, part, prefix, total;
};
template <bool kMx>
__host__ __device__ inline SmemLayout smem_layout(int stages, int E) {
  using S = Shape<kMx>;
  SmemLayout l;
  uint32_t at = stages * S::kStage;
  l.scales = at, at += S::kSlots * S::kSlot;
  l.boxes = at, at += kPlanDepth * 32 * 16;
  l.rows = at, at += kPlanDepth * S::kMaxRows * 4;
  l.tiles = at, at += kPlanDepth * (uint32_t)sizeof(Tile);
  l.amax = at, at += 2 * 8 * 32 * 4;
  l.bars = at, at += (2 * kStages + 4 + 2 * kPlanDepth + 4 + 2 * 4) * 8;
  l.tmem = at, at += 16;
  l.part = at, at += 64;
  l.prefix = at, at += (E + 1) * 4;
  l.total = at + 1024;  // the base may have to move up to its boundary
  return l;
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------
// 32 columns of 16 gate and 16 up features (swiglu_columns).  MX8 output: amax is
// the exchange's buffer, bar its barrier, parity its phase; false when the wait
// expired.
__device__ __forceinline__ bool store_swiglu(const ProductArgs& a, const float (&v)[32], int first, const int* list,
                                             uint32_t* amax, int warp, uint32_t bar, uint32_t parity) {
  const int lane = threadIdx.x & 31, up = lane >> 3 & 1;
  if (a.out_dtype != LLMOE_DTYPE_MX8) {
    store_swiglu_values(a, v, first, list);
    return true;
  }
  // a group of 32 outputs is this warp's 16 and its neighbour's: the two swap
  // their largest magnitudes through shared memory
  float h[16];
  swiglu_columns(v, h);
  int at;
  const uint32_t most = largest_of_columns(h, at);
  amax[warp * 32 + up * 16 + at] = most;
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
  if (!mbar_wait_warp(bar, parity, a.err)) return false;
  uint32_t mine = 0;  // the scale code of column 2 at + up
  float inverse[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t code = scale_code(max(amax[warp * 32 + up * 16 + i], amax[(warp ^ 1) * 32 + up * 16 + i]));
    if (i == at) mine = code;
    inverse[i] = scale_inverse(code);
  }
  store_codes(a, h, inverse, first, list);
  const int my_row = swiglu_feature(first) < a.out && !(warp & 1) ? list[2 * at + up] : -1;
  if (my_row >= 0) {
    uint8_t* s = in_row(a, a.y + a.out + first / 32, my_row);
    *s = (uint8_t)mine;
    if (first + 32 == a.out)
      for (uint8_t* end = in_row(a, a.y + a.y_row, my_row); ++s < end;) *s = 0;
  }
  return true;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <bool kMx, bool kSwiglu>
__global__ void __launch_bounds__(Shape<kMx>::kThreads, 1) __cluster_dims__(2, 1, 1)
    product_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ ProductMaps maps) {
  using S = Shape<kMx>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - raw % 1024) % 1024);
  const uint32_t sbase = smem_addr(smem);
  const SmemLayout l = smem_layout<kMx>(a.stages, a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  int* rows = reinterpret_cast<int*>(smem + l.rows);
  Box* boxes = reinterpret_cast<Box*>(smem + l.boxes);
  Tile* tiles = reinterpret_cast<Tile*>(smem + l.tiles);
  int* prefix = reinterpret_cast<int*>(smem + l.prefix);
  const uint32_t full = sbase + l.bars, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, plan_full = acc_empty + 16, plan_empty = plan_full + 8 * kPlanDepth,
                 halves = plan_empty + 8 * kPlanDepth, scale_full = halves + 32, scale_empty = scale_full + 32;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&maps.w);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(scale_full + 8 * s, 8);  // the scale warps of both CTAs
      mbar_init(scale_empty + 8 * s, 1);
    }
    for (int b = 0; b < 4; ++b) mbar_init(halves + 8 * b, 2);  // the two epilogue warps of an output group
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, 16);  // the epilogue warps of both CTAs
    }
    for (int p = 0; p < kPlanDepth; ++p) {
      mbar_init(plan_full + 8 * p, 1);
      mbar_init(plan_empty + 8 * p, 10 + (leader ? 1 : 0) + (kMx ? 4 : 0));  // warps that read a plan
    }
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc_pair(sbase + l.tmem, 512);
  wait_prior_grid();
  release_next_grid();
  count_shares<S::kMaxRows, S::kThreads>(a, prefix, reinterpret_cast<int*>(smem + l.part));
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + l.tmem);

  const RingBars bars{full, empty, plan_full, plan_empty};
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, ntiles = prefix[a.E] * a.blocks;

  if (warp == 0 || warp == 3) {
    if (elect_one())
      load_tiles<S::kStage, S::kBytesA, kMx ? 128 : 64, kSwiglu, 6>(a, maps, sbase, bars, tiles, boxes, warp == 3, rank, pair,
                                                                 pairs, ntiles);
  } else if (warp == 1 && leader) {
    // ---- products: one thread -----------------------------------------------------
    if (elect_one()) {
      int stage = 0, i = 0, sslot = 0, ring = 0;
      uint32_t phase = 0, sphase = 0;
      // 8-bit: steps whose products are known to be done, and the last one's stage and phase
      int issued = 0, done = 0, done_stage = a.stages - 1;
      uint32_t done_phase = 1;
      bool ok = true;
      const uint32_t desc = tile_desc(sbase), sdesc = scale_desc(sbase + l.scales);  // they count 16 bytes
      for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
        const int slot = i % kPlanDepth, buf = i & 1;
        if (!(ok = mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
        const int n = columns(tiles[slot].groups);
        mbar_arrive(plan_empty + 8 * slot);
        if (!(ok = mbar_wait(acc_empty + 8 * buf, ((i >> 1) & 1) ^ 1, a.err))) break;
        tc_fence_after();
        const uint32_t d = tmem + buf * S::kMaxRows, idesc = a.idesc | (uint32_t)(n >> 3) << 17;
        if constexpr (kMx) {
          // two steps a turn: this thread's instructions, not the tensor core,
          // bound the 8-bit product (496 cycles a step alone, of 422)
          for (int k = 0; k < a.steps && ok; k += 2) {
            const int m = k + 1 < a.steps ? 2 : 1;
            const bool last = k + 2 >= a.steps;
            if ((k & 2) == 0 && !(ok = mbar_wait(scale_full + 8 * sslot, sphase, a.err))) break;
            issued += m;
            if (issued - S::kScaleRing > done) {  // the columns' last users
              done_stage += issued - S::kScaleRing - done;
              done = issued - S::kScaleRing;
              if (done_stage >= a.stages) done_stage -= a.stages, done_phase ^= 1;
              if (!(ok = mbar_wait(empty + 8 * done_stage, done_phase, a.err))) break;
            }
            const uint32_t sa = sdesc + (uint32_t)((sslot * S::kSlot + (k & 2) * 512) >> 4),
                           sb = sdesc + (uint32_t)((sslot * S::kSlot + 2048 + (k & 2) * 1024) >> 4);
            uint32_t ta[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              ta[u] = tmem + 2 * S::kMaxRows + ring * S::kScaleColumns;
              if (u < m) {
                copy_scales(ta[u], sa + u * (512 >> 4));
                copy_scales(ta[u] + 4, sb + u * (1024 >> 4));
                if (n > 128) copy_scales(ta[u] + 8, sb + u * (1024 >> 4) + (512 >> 4));
                if (++ring == S::kScaleRing) ring = 0;
              }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (u < m && ok) {
                const uint32_t da = desc + (uint32_t)(stage * (S::kStage >> 4)), db = da + (S::kBytesA >> 4);
                if (!(ok = mbar_wait(full + 8 * stage, phase, a.err))) break;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < 4; ++j)  // 32 bytes of K; scale j of each row's four
                  mma_mx8(d, da + 2 * j, db + 2 * j, idesc | (uint32_t)j << 4 | (uint32_t)j << 29, ta[u], ta[u] + 4,
                          k + u > 0 || j > 0);
                mma_commit_pair(empty + 8 * stage);
                if (++stage == a.stages) stage = 0, phase ^= 1;
              }
            }
            if (((k & 2) != 0 || last) && ok) {
              mma_commit_pair(scale_empty + 8 * sslot);
              if (++sslot == S::kSlots) sslot = 0, sphase ^= 1;
            }
          }
        } else {
          for (int k = 0; k < a.steps; ++k) {
            const uint32_t da = desc + (uint32_t)(stage * (S::kStage >> 4)), db = da + (S::kBytesA >> 4);
            if (!(ok = mbar_wait(full + 8 * stage, phase, a.err))) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_16bit(d, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
            mma_commit_pair(empty + 8 * stage);
            if (++stage == a.stages) stage = 0, phase ^= 1;
          }
        }
        if (ok) mma_commit_pair(acc_full + 8 * buf);
      }
    }
  } else if (warp == 2) {
    // ---- plan ------------------------------------------------------------------
    int i = 0;
    Buckets buckets{-1, 0, 0, 0};
    for (int t = pair; t < ntiles; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!mbar_wait_warp(plan_empty + 8 * slot, ((i / kPlanDepth) & 1) ^ 1, a.err)) break;
      plan_tile<S::kMaxRows, true>(a, prefix, t, (int)rank, buckets, tiles + slot, rows + slot * S::kMaxRows, boxes + 32 * slot);
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_full + 8 * slot);
    }
  } else if (warp >= 4 && warp < 12) {
    // ---- epilogue ------------------------------------------------------------------
    // two sets of four warps, each taking every other 32 columns
    const int w = warp & 3, set = warp >= 8;  // tensor-memory lanes 32 w ..
    uint32_t* amax = reinterpret_cast<uint32_t*>(smem + l.amax) + set * 256;
    int i = 0, flip = 0;
    for (int t = pair; t < ntiles; t += pairs, ++i) {
      const int slot = i % kPlanDepth, buf = i & 1;
      if (!mbar_wait_warp(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err)) break;
      const Tile tile = tiles[slot];
      const int* list = rows + slot * S::kMaxRows;
      const int first = kSwiglu ? tile.block * 128 + (int)rank * 64 + w * 16
                                : tile.block * kTileFeatures + (int)rank * 128 + w * 32;
      if (!mbar_wait_warp(acc_full + 8 * buf, (i >> 1) & 1, a.err)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * w) << 16) + buf * S::kMaxRows;
      bool ok = true;
      for (int c = 32 * set; c < tile.groups * kGroup && ok; c += 64) {
        float v[32];
        tmem_load32(acc + c, v);
        if constexpr (kSwiglu) {
          // two buffers in turn: a warp that fills one again has met its
          // neighbour at the other since, so the neighbour has read it
          ok = store_swiglu(a, v, first, list + c, amax + 128 * flip, w, halves + 8 * (2 * set + (w >> 1)), flip);
          flip ^= 1;
        } else {
          store_plain(a, v, first, list + c);
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_tensor(map_rank(acc_empty + 8 * buf, 0));
        mbar_arrive(plan_empty + 8 * slot);
      }
    }
  } else if (kMx && warp >= 12) {
    // ---- scales ------------------------------------------------------------------
    // Warp q's lane l moves the scales of row 32 q + l of the CTA's 128 rows of w
    // and of columns 32 q + l and 128 + 32 q + l: 16 bytes of a row at a time,
    // for four steps, kAhead such chunks ahead.  A step's scales of 128 rows are
    // 32 lines of 16 bytes, line l holding rows l, l + 32, l + 64, l + 96: what
    // lane l of tensor memory takes.
    constexpr int kAhead = 3;
    const int q = warp & 3, nscale = a.in / 32, chunks = (a.steps + 3) / 4;
    int i = 0, sslot = 0;
    uint32_t sphase = 0;
    bool ok = true;
    for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!(ok = mbar_wait_warp(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
      const Tile tile = tiles[slot];
      const int n = columns(tile.groups), m = 32 * q + lane;
      const int f = min(kSwiglu ? (m >> 3 & 1) * a.out + tile.block * 128 + (int)rank * 64 + (m >> 4) * 8 + (m & 7)
                                : tile.block * kTileFeatures + (int)rank * 128 + m,
                        a.n - 1);  // past the expert's last row: its products are not stored
      const int r0 = m < n ? rows[slot * S::kMaxRows + m] : -1;
      const int r1 = 128 + m < n ? rows[slot * S::kMaxRows + 128 + m] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
      const uint4* src[3] = {
          reinterpret_cast<const uint4*>(a.w + ((uint64_t)tile.expert * a.n + f) * a.x_row + a.in),
          reinterpret_cast<const uint4*>(a.x + (uint64_t)max(r0, 0) * a.x_row + a.in),
          reinterpret_cast<const uint4*>(a.x + (uint64_t)max(r1, 0) * a.x_row + a.in)};
      const bool have[3] = {true, r0 >= 0, r1 >= 0};
      uint4 ahead[kAhead][3];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          ahead[u][j] = make_uint4(0, 0, 0, 0);
          if (have[j] && u < chunks) ahead[u][j] = src[j][u];
        }
      for (int c0 = 0; c0 < chunks && ok; c0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int c = c0 + u;
          if (c >= chunks || !ok) break;
          if (!(ok = mbar_wait_warp(scale_empty + 8 * sslot, sphase ^ 1, a.err))) break;
          uint8_t* dst = smem + l.scales + sslot * S::kSlot + lane * 16 + q * 4;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            // scales past the row's last are 1: the codes there are zeros, and 0 * NaN would not be
            const int left = nscale - 4 * (4 * c + b);
            const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << 8 * left) - 1;
#pragma unroll
            for (int j = 0; j < 3; ++j) {
              const uint4& v = ahead[u][j];
              const uint32_t word = b == 0 ? v.x : b == 1 ? v.y : b == 2 ? v.z : v.w;
              if (have[j])
                *reinterpret_cast<uint32_t*>(dst + (j == 0 ? b * 512 : 2048 + b * 1024 + (j - 1) * 512)) =
                    (word & keep) | (0x7f7f7f7fu & ~keep);
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(map_rank(scale_full + 8 * sslot, 0));
          if (++sslot == S::kSlots) sslot = 0, sphase ^= 1;
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (have[j] && c + kAhead < chunks) ahead[u][j] = src[j][c + kAhead];
        }
      }
    }
    for (int s = 0; s < S::kSlots && ok; ++s) {  // as the ring
      ok = mbar_wait_warp(scale_empty + 8 * sslot, sphase ^ 1, a.err);
      if (++sslot == S::kSlots) sslot = 0, sphase ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 3) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Checks a product's arguments and fills its geometry.
int product_args(const void* x, const void* w, void* y, const int64_t* counts, int in, int out, int dtype,
                 int out_dtype, uint32_t flags, const llmoe_buf_set_t* bs, ProductArgs* a) {
  if ((flags & ~LLMOE_PRODUCT_SWIGLU) != 0 || !product_buckets(counts, bs, a)) return LLMOE_ERR_INVALID_ARGUMENT;
  const bool swiglu = (flags & LLMOE_PRODUCT_SWIGLU) != 0;
  switch (dtype) {
    case LLMOE_DTYPE_BF16:
    case LLMOE_DTYPE_FP16:
      if (out_dtype != dtype && out_dtype != LLMOE_DTYPE_FP32) return LLMOE_ERR_INVALID_ARGUMENT;
      break;
    case LLMOE_DTYPE_MX8:
      if ((out_dtype == LLMOE_DTYPE_MX8 && !swiglu) || out_dtype == LLMOE_DTYPE_FP8B) return LLMOE_ERR_INVALID_ARGUMENT;
      break;
    default: return LLMOE_ERR_INVALID_ARGUMENT;
  }
  const uint64_t xr = row_bytes(in, dtype);
  if (!product_rows(x, y, in, out, dtype, out_dtype, swiglu, a) || w == nullptr || !aligned(w, 16) ||
      xr > kMostBytes / ((uint64_t)a->n * a->E))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t rows = (uint64_t)a->E * a->R * a->T;
  if (overlap(y, rows * a->y_row, w, (uint64_t)a->n * a->E * xr)) return LLMOE_ERR_INVALID_ARGUMENT;
  a->w = static_cast<const uint8_t*>(w);
  return LLMOE_SUCCESS;
}

template <bool kMx, bool kSwiglu>
int launch_product(ProductArgs& a, llmoe_stream_t stream) {
  using S = Shape<kMx>;
  a.steps = (int)(((int64_t)a.in * (kMx ? 1 : 2) + 127) / 128);
  a.blocks = (a.n + kTileFeatures - 1) / kTileFeatures;
  // tiles at full counts
  const uint64_t groups = (uint64_t)((a.T + kGroup - 1) / kGroup) * a.R, share = S::kMaxRows / kGroup;
  const uint64_t most = (groups + share - 1) / share * a.E * a.blocks;
  if (most > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  a.stages = kStages;
  while (smem_layout<kMx>(a.stages, a.E).total > kMaxSmem) --a.stages;
  const size_t smem = smem_layout<kMx>(a.stages, a.E).total;
  // both operands 16-bit or both e4m3 (0), fp32 sums, M = 256; 8-bit: e8m0 scales
  const uint32_t type = a.dtype == LLMOE_DTYPE_BF16 ? 1 : 0;
  a.idesc = (uint32_t)(kTileFeatures >> 4) << 24 | type << 7 | type << 10 | (kMx ? 1u << 23 : 1u << 4);

  ProductMaps maps;
  const cuuint32_t k_box = kMx ? 128 : 64;
  for (int b = 0; b < kBoxes; ++b) {
    if (b > 0 && (uint64_t)kGroup << (b - 1) >= (uint64_t)a.R * a.T) break;  // a run is at most an expert's rows
    const cuuint64_t dims[2] = {(cuuint64_t)a.in, (cuuint64_t)a.E * a.R * a.T}, strides[1] = {a.x_row};
    const cuuint32_t box[2] = {k_box, (cuuint32_t)kGroup << b};
    if (!make_map(&maps.x[b], a.x, a.dtype, dims, strides, box, 2)) return LLMOE_ERR_CUDA;
  }
  if (kSwiglu) {
    // gate and up in turn, eight rows of each: a box is (K, 8 rows, gate / up, 8 such)
    const cuuint64_t dims[5] = {(cuuint64_t)a.in, 8, 2, (cuuint64_t)a.out / 8, (cuuint64_t)a.E},
                     strides[4] = {a.x_row, a.x_row * (uint64_t)a.out, a.x_row * 8, a.x_row * (uint64_t)a.n};
    const cuuint32_t box[5] = {k_box, 8, 2, 8, 1};
    if (!make_map(&maps.w, a.w, a.dtype, dims, strides, box, 5)) return LLMOE_ERR_CUDA;
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)a.in, (cuuint64_t)a.n, (cuuint64_t)a.E},
                     strides[2] = {a.x_row, a.x_row * (uint64_t)a.n};
    const cuuint32_t box[3] = {k_box, 128, 1};
    if (!make_map(&maps.w, a.w, a.dtype, dims, strides, box, 3)) return LLMOE_ERR_CUDA;
  }
  static_assert((kStages - 1) * S::kStage > kMaxSmem / 2, "one CTA per SM");
  const int pairs = resident_pairs<product_kernel<kMx, kSwiglu>>(S::kThreads);
  if (pairs < 1) return LLMOE_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min<uint64_t>(most, pairs));
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, product_kernel<kMx, kSwiglu>, a, maps) != cudaSuccess) {
    cudaGetLastError();
    return LLMOE_ERR_CUDA;
  }
  return LLMOE_SUCCESS;
}

}  // namespace

extern "C" int llmoe_expert_product(const void* x, const void* w, void* y, const int64_t* counts, int in_features,
                                    int out_features, int dtype, int out_dtype, uint32_t flags,
                                    const llmoe_buf_set_t* bs, llmoe_stream_t stream) {
  ProductArgs a;
  const int rc = product_args(x, w, y, counts, in_features, out_features, dtype, out_dtype, flags, bs, &a);
  if (rc != LLMOE_SUCCESS) return rc;
  const bool swiglu = (flags & LLMOE_PRODUCT_SWIGLU) != 0;
  if (dtype == LLMOE_DTYPE_MX8)
    return swiglu ? launch_product<true, true>(a, stream) : launch_product<true, false>(a, stream);
  return swiglu ? launch_product<false, true>(a, stream) : launch_product<false, false>(a, stream);
}
