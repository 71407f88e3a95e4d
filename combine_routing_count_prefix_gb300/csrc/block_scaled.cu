// block_scaled.cu -- llmoe_expert_product_fp8b (include/llmoe_block.h): matrix
// products grouped by expert over received FP8B rows.
//
// Tiles, plan, ring and pairs are block_product.cu's: the weights on the M side,
// 256 features to a pair of CTAs, up to kMaxRows received rows on the N side.
// What differs is where the sums live.  A block's scales are fp32, so the tensor
// core cannot apply them: it makes the sums of one block of 128 (one step of the
// ring, four instructions) in one of two buffers of tensor memory, and eight warps
// add them, times their scales, to sums that they hold in registers:
//   acc[f][r] += P[f][r] * (s[r] * ws),
// 128 values a thread for a full tile.  ws is one number for a CTA's 128 features
// (two with SwiGLU, gate and up), s one for a column.  A warp reads tensor memory
// so that a thread holds pairs of neighbouring columns of four features each: a
// pair's two scales are one 8-byte load for four packed multiply-adds.
//
// Inside a CTA of 16 warps:
//   warps 0, 3  load (warp 3 also allocates the tensor memory)
//   warp 1      (first CTA of the pair) issues the products
//   warp 2      plans
//   warps 4-11  sums, then the tile's epilogue
//   warps 12-15 move the scales of x's rows (times ws without SwiGLU) and of w to
//               shared memory, four steps at a time
// The eight warps have kManyRegisters registers a thread, the others kFewRegisters.
// Every wait is bounded, as there.
#include "block_plan.cuh"

namespace {

constexpr int kMaxRows = 256, kThreads = 512;
constexpr int kBytesA = 128 * 128, kBytesB = kMaxRows / 2 * 128, kStage = kBytesA + kBytesB;
constexpr int kManyRegisters = 200, kFewRegisters = 56;
static_assert(256 * (kManyRegisters + kFewRegisters) <= 65536, "what a launch of 512 threads has");
constexpr int kSlots = 3;                      // of scales, four steps each
constexpr int kSlot = 4 * kMaxRows * 4;        // bytes of a slot's row scales
constexpr int kChunks = kMaxRows / 64;         // of 32 columns, for each set of four warps

struct ScaledArgs {
  ProductArgs p;
  const float* w_scale;
  int down, across;  // blocks of 128 down and across one matrix of w
};

// Byte offsets in dynamic shared memory, from its first 1024-byte boundary.
struct ScaledSmem {
  uint32_t scales, w_scales, turn, codes, boxes, rows, tiles, bars, tmem, part, prefix, total;
};
__host__ __device__ inline ScaledSmem scaled_smem(int stages, int E) {
  ScaledSmem l;
  uint32_t at = stages * kStage;
  l.scales = at, at += kSlots * kSlot;
  l.w_scales = at, at += kSlots * 4 * 2 * 4;
  at = (at + 127) / 128 * 128;
  l.turn = at, at += 8 * kMaxRows * 4;  // 1 KB a warp to turn outputs in, or the largest magnitudes of eight warps
  l.codes = at, at += 8 * 512;  // a warp's 32 columns of 16 codes
  l.boxes = at, at += kPlanDepth * 32 * 16;
  l.rows = at, at += kPlanDepth * kMaxRows * 4;
  l.tiles = at, at += kPlanDepth * (uint32_t)sizeof(Tile);
  l.bars = at, at += (2 * kStages + 4 + 2 * kPlanDepth + 2 * kSlots + 4) * 8;
  l.tmem = at, at += 16;
  l.part = at, at += 64;
  l.prefix = at, at += (E + 1) * 4;
  l.total = at + 1024;  // the base may have to move up to its boundary
  return l;
}

// One thread's sums of 32 columns: [half][j][features l / + 8], columns 8 j + 2 q
// and the next (tmem_load_pairs).
using Sums = Pair[2][4][2];

// ---------------------------------------------------------------------------
// epilogue: 32 columns of a warp's 32 lanes; turn: 1 KB of the warp's own
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store_plain(const ProductArgs& a, const Sums& acc, int first, const int* list,
                                            uint32_t turn) {
  const int lane = threadIdx.x & 31, l = lane >> 2, q = lane & 3;
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int2 row = *reinterpret_cast<const int2*>(list + 8 * j + 2 * q);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float2 v = unpair(acc[b >> 1][j][b & 1]);
        const int feature = first + 8 * b + l;
        if (feature >= a.out) continue;
        uint8_t* at = a.y + (uint64_t)feature * 4;
        if (row.x >= 0) *reinterpret_cast<float*>(in_row(a, at, row.x)) = v.x;
        if (row.y >= 0) *reinterpret_cast<float*>(in_row(a, at, row.y)) = v.y;
      }
    }
    return;
  }
  // 8 columns of 32 features at a time: 64 bytes a column, its 16-byte pieces
  // placed so that neither the turned stores nor the loads meet in a bank
  const bool fp16 = a.out_dtype == LLMOE_DTYPE_FP16;
  const uint32_t put = turn + (lane & 7) * 64 + (((lane >> 3) ^ (lane >> 1 & 3)) << 4);
  const uint32_t get = turn + l * 64 + ((q ^ (l >> 1 & 3)) << 4);
  const int feature = first + 8 * q;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t u[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float2 v = unpair(acc[b >> 1][j][b & 1]);
      u[b] = pack2(v.x, v.y, fp16);
    }
    store_turned(put + (j & 1) * 512, u[0], u[1], u[2], u[3]);
    __syncwarp();  // and the buffer's use before the last one is over
    const uint4 v = shared_load16(get + (j & 1) * 512);
    const int row = list[8 * j + l];
    if (row >= 0 && feature < a.out) *reinterpret_cast<uint4*>(in_row(a, a.y + (uint64_t)feature * 2, row)) = v;
  }
}

// Lanes 0-7 and 16-23 of a warp are gate features, the others up; h of 16
// features, 8 half + l, in place of the gate's sums.
template <bool kAccurate>
__device__ __forceinline__ void swiglu(Sums& acc) {
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 g = unpair(acc[half][j][0]), u = unpair(acc[half][j][1]);
      acc[half][j][0] = kAccurate ? pair(silu(g.x) * u.x, silu(g.y) * u.y) : pair(near_silu(g.x) * u.x, near_silu(g.y) * u.y);
    }
}

__device__ __forceinline__ void store_swiglu(const ProductArgs& a, const Sums& acc, int first, const int* list,
                                             uint32_t turn) {
  const int lane = threadIdx.x & 31, l = lane >> 2, q = lane & 3;
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int2 row = *reinterpret_cast<const int2*>(list + 8 * j + 2 * q);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const float2 v = unpair(acc[half][j][0]);
        const int feature = first + 8 * half + l;
        if (feature >= a.out) continue;
        uint8_t* at = a.y + (uint64_t)feature * 4;
        if (row.x >= 0) *reinterpret_cast<float*>(in_row(a, at, row.x)) = v.x;
        if (row.y >= 0) *reinterpret_cast<float*>(in_row(a, at, row.y)) = v.y;
      }
    }
    return;
  }
  // 16 columns of 16 features at a time, 32 bytes a column
  const bool fp16 = a.out_dtype == LLMOE_DTYPE_FP16;
  const uint32_t put = turn + ((lane >> 4) * 8 + (lane & 7)) * 32 + (((lane >> 3 & 1) ^ (lane >> 2 & 1)) << 4);
  const uint32_t get = turn + (lane >> 1) * 32 + (((lane & 1) ^ (lane >> 3 & 1)) << 4);
  const int feature = first + 8 * (lane & 1);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t u[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float2 v = unpair(acc[m & 1][2 * i + (m >> 1)][0]);
      u[m] = pack2(v.x, v.y, fp16);
    }
    store_turned(put + i * 512, u[0], u[1], u[2], u[3]);
    __syncwarp();
    const uint4 v = shared_load16(get + i * 512);
    const int row = list[16 * i + (lane >> 1)];
    if (row >= 0 && feature < a.out) *reinterpret_cast<uint4*>(in_row(a, a.y + (uint64_t)feature * 2, row)) = v;
  }
}

// Largest magnitude of the warp's 16 features of h in each of 32 columns: lane's
// column is the one returned in `column`.
__device__ __forceinline__ uint32_t largest(const Sums& acc, int& column) {
  const int lane = threadIdx.x & 31;
  uint32_t m[8];  // columns 8 j + 2 q + i as 2 j + i
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 a = unpair(acc[0][j][0]), b = unpair(acc[1][j][0]);
    m[2 * j] = max(magnitude(a.x), magnitude(b.x));
    m[2 * j + 1] = max(magnitude(a.y), magnitude(b.y));
  }
  // lanes of the same q halve the columns they keep at each of three exchanges
  int at = 0;
#pragma unroll
  for (int step = 0; step < 3; ++step) {
    const int d = 4 << step, keep = 4 >> step;
    const bool high = lane & d;
#pragma unroll
    for (int i = 0; i < keep; ++i) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? m[i] : m[i + keep], d);
      m[i] = max(high ? m[i + keep] : m[i], got);
    }
    at += high ? keep : 0;
  }
  column = 8 * (at >> 1) + 2 * (lane & 3) + (at & 1);
  return m[0];
}

// Codes of 32 columns; inv: of column `lane`.
__device__ __forceinline__ void store_codes(const ProductArgs& a, const Sums& acc, int first, const int* list, float inv,
                                            uint32_t turn) {
  const int lane = threadIdx.x & 31, q = lane & 3;
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Pair i2 = pair(__shfl_sync(0xffffffffu, inv, 8 * j + 2 * q), __shfl_sync(0xffffffffu, inv, 8 * j + 2 * q + 1));
    const float2 lo = unpair(mul2(acc[0][j][0], i2)), hi = unpair(mul2(acc[1][j][0], i2));
    u[j] = pack_e4m3x2(lo.x, hi.x) | pack_e4m3x2(lo.y, hi.y) << 16;  // a 16-bit value: features l and 8 + l
  }
  store_turned(turn + lane * 16, u[0], u[1], u[2], u[3]);
  __syncwarp();
  const uint4 v = shared_load16(turn + lane * 16);
  __syncwarp();  // read, before the next columns' are stored
  const int row = list[lane];
  if (row >= 0 && first < a.out)
    *reinterpret_cast<uint4*>(in_row(a, a.y + first, row)) =
        make_uint4(__byte_perm(v.x, v.y, 0x6420), __byte_perm(v.z, v.w, 0x6420), __byte_perm(v.x, v.y, 0x7531),
                   __byte_perm(v.z, v.w, 0x7531));
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    scaled_kernel(const __grid_constant__ ScaledArgs s, const __grid_constant__ ProductMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  const ProductArgs& a = s.p;
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - raw % 1024) % 1024);
  const uint32_t sbase = smem_addr(smem);
  const ScaledSmem l = scaled_smem(a.stages, a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  int* rows = reinterpret_cast<int*>(smem + l.rows);
  Box* boxes = reinterpret_cast<Box*>(smem + l.boxes);
  Tile* tiles = reinterpret_cast<Tile*>(smem + l.tiles);
  int* prefix = reinterpret_cast<int*>(smem + l.prefix);
  const uint32_t full = sbase + l.bars, empty = full + 8 * kStages, acc_full = empty + 8 * kStages,
                 acc_empty = acc_full + 16, plan_full = acc_empty + 16, plan_empty = plan_full + 8 * kPlanDepth,
                 scale_full = plan_empty + 8 * kPlanDepth, scale_empty = scale_full + 8 * kSlots,
                 amax_full = scale_empty + 8 * kSlots, amax_empty = amax_full + 16;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&maps.w);
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(scale_full + 8 * i, 4);
      mbar_init(scale_empty + 8 * i, 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 16);  // the summing warps of both CTAs
      mbar_init(amax_full + 8 * i, 8);   // a set's warps of both CTAs
      mbar_init(amax_empty + 8 * i, 8);
    }
    for (int i = 0; i < kPlanDepth; ++i) {
      mbar_init(plan_full + 8 * i, 1);
      mbar_init(plan_empty + 8 * i, 14 + (leader ? 1 : 0));  // warps that read a plan
    }
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc_pair(sbase + l.tmem, 512);
  wait_prior_grid();
  release_next_grid();
  count_shares<kMaxRows, kThreads>(a, prefix, reinterpret_cast<int*>(smem + l.part));
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + l.tmem);

  const RingBars bars{full, empty, plan_full, plan_empty};
  const int pair_id = blockIdx.x >> 1, pairs = gridDim.x >> 1, ntiles = prefix[a.E] * a.blocks;

  if (warp < 4) {
    fewer_registers<kFewRegisters>();
    if (warp == 0 || warp == 3) {
      if (elect_one())
        load_tiles<kStage, kBytesA, 128, kSwiglu>(a, maps, sbase, bars, tiles, boxes, warp == 3, rank, pair_id, pairs,
                                                  ntiles);
    } else if (warp == 1) {
      // ---- products: one thread -----------------------------------------------------
      if (leader && elect_one()) {
        int stage = 0, i = 0;
        uint32_t phase = 0, step = 0;  // step: over all tiles, two buffers in turn
        bool ok = true;
        const uint32_t desc = tile_desc(sbase);
        for (int t = pair_id; t < ntiles && ok; t += pairs, ++i) {
          const int slot = i % kPlanDepth;
          if (!(ok = mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
          const uint32_t idesc = a.idesc | (uint32_t)(columns(tiles[slot].groups) >> 3) << 17;
          mbar_arrive(plan_empty + 8 * slot);
          for (int k = 0; k < a.steps; ++k, ++step) {
            const uint32_t buf = step & 1, d = tmem + buf * kMaxRows;
            const uint32_t da = desc + (uint32_t)(stage * (kStage >> 4)), db = da + (kBytesA >> 4);
            if (!(ok = mbar_wait(acc_empty + 8 * buf, (step >> 1 & 1) ^ 1, a.err))) break;
            if (!(ok = mbar_wait(full + 8 * stage, phase, a.err))) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_8bit(d, da + 2 * j, db + 2 * j, idesc, j > 0);
            mma_commit_pair(empty + 8 * stage);
            mma_commit_pair(acc_full + 8 * buf);
            if (++stage == a.stages) stage = 0, phase ^= 1;
          }
        }
      }
    } else {
      // ---- plan ------------------------------------------------------------------
      int i = 0;
      Buckets buckets{-1, 0, 0, 0};
      for (int t = pair_id; t < ntiles; t += pairs, ++i) {
        const int slot = i % kPlanDepth;
        if (!mbar_wait_warp(plan_empty + 8 * slot, ((i / kPlanDepth) & 1) ^ 1, a.err)) break;
        plan_tile<kMaxRows>(a, prefix, t, (int)rank, buckets, tiles + slot, rows + slot * kMaxRows, boxes + 32 * slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(plan_full + 8 * slot);
      }
    }
  } else if (warp < 12) {
    more_registers<kManyRegisters>();
    // ---- sums and epilogue ---------------------------------------------------------
    // two sets of four warps, each taking every other 32 columns
    const int w = warp & 3, set = warp >= 8;  // tensor-memory lanes 32 w ..
    const uint32_t turn = sbase + l.turn + (warp - 4) * 1024;
    uint32_t* amax = reinterpret_cast<uint32_t*>(smem + l.turn);  // [warp of the pair's set][column]
    const uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16) + 32 * set;
    const uint32_t leader_empty = map_rank(acc_empty, 0);
    int i = 0, sslot = 0;
    uint32_t step = 0, sphase = 0;
    bool ok = true;
    for (int t = pair_id; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!(ok = mbar_wait_warp(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
      const Tile tile = tiles[slot];
      const int chunks = (columns(tile.groups) / 32 + 1 - set) / 2;
      Sums acc[kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; ++c)
#pragma unroll
        for (int h = 0; h < 16; ++h) acc[c][h >> 3][h >> 1 & 3][h & 1] = 0;
      for (int k = 0; k < a.steps; ++k, ++step) {
        const uint32_t buf = step & 1;
        if ((k & 3) == 0 && !(ok = mbar_wait_warp(scale_full + 8 * sslot, sphase, a.err))) break;
        if (!(ok = mbar_wait_warp(acc_full + 8 * buf, step >> 1 & 1, a.err))) break;
        tc_fence_after();
        const float* sx = reinterpret_cast<const float*>(smem + l.scales + sslot * kSlot) + (k & 3) * kMaxRows + 32 * set +
                          2 * (lane & 3);
        Pair wg = 0, wu = 0;
        if constexpr (kSwiglu) {
          const float2 ws = *reinterpret_cast<const float2*>(smem + l.w_scales + (sslot * 4 + (k & 3)) * 8);
          wg = pair(ws.x, ws.x), wu = pair(ws.y, ws.y);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c < chunks) {
            uint32_t v[2][4][4];
            tmem_load_pairs(lanes + buf * kMaxRows + 64 * c, v);
            if (c == chunks - 1) {  // all of the buffer is in registers
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_peer(leader_empty + 8 * buf);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = *reinterpret_cast<const float2*>(sx + 64 * c + 8 * j);
              const Pair sc = pair(f.x, f.y);
              const Pair g = kSwiglu ? mul2(sc, wg) : sc, u = kSwiglu ? mul2(sc, wu) : sc;
#pragma unroll
              for (int half = 0; half < 2; ++half) {
                const uint32_t(&p)[4] = v[half][j];
                acc[c][half][j][0] = fma2(pair(__uint_as_float(p[0]), __uint_as_float(p[1])), g, acc[c][half][j][0]);
                acc[c][half][j][1] = fma2(pair(__uint_as_float(p[2]), __uint_as_float(p[3])), u, acc[c][half][j][1]);
              }
            }
          }
        }
        if (chunks == 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(leader_empty + 8 * buf);
        }
        if ((k & 3) == 3 || k + 1 == a.steps) {
          __syncwarp();
          if (lane == 0) mbar_arrive(scale_empty + 8 * sslot);
          if (++sslot == kSlots) sslot = 0, sphase ^= 1;
        }
      }
      if (!ok) break;
      const int* list = rows + slot * kMaxRows + 32 * set;
      if constexpr (!kSwiglu) {
        const int first = tile.block * kTileFeatures + (int)rank * 128 + w * 32;
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c < chunks) store_plain(a, acc[c], first, list + 64 * c, turn);
      } else {
        const int first = tile.block * 128 + (int)rank * 64 + w * 16;
        if (a.out_dtype == LLMOE_DTYPE_FP8B) {
          // a block of 128 outputs is the pair's: its eight warps of this set swap
          // their largest magnitudes, once the last tile's have been read
          if (!(ok = mbar_wait_warp(amax_empty + 8 * set, (i & 1) ^ 1, a.err))) break;
          const uint32_t mine = smem_addr(amax + (rank * 4 + w) * kMaxRows + 32 * set), peer = map_rank(mine, rank ^ 1);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              swiglu<false>(acc[c]);
              int column;
              const uint32_t m = largest(acc[c], column);
              amax[(rank * 4 + w) * kMaxRows + 32 * set + 64 * c + column] = m;
              shared_store_peer(peer + 4 * (64 * c + column), m);
            }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(amax_full + 8 * set);
            mbar_arrive_peer_release(map_rank(amax_full + 8 * set, rank ^ 1));
          }
          if (!(ok = mbar_wait_warp(amax_full + 8 * set, i & 1, a.err))) break;
          float scale[kChunks];
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              uint32_t m = 0;
#pragma unroll
              for (int j = 0; j < 8; ++j) m = max(m, amax[j * kMaxRows + 32 * set + 64 * c + lane]);
              scale[c] = block_scale(__uint_as_float(m));
            }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(amax_empty + 8 * set);
            mbar_arrive_peer_release(map_rank(amax_empty + 8 * set, rank ^ 1));
          }
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              store_codes(a, acc[c], first, list + 64 * c, __frcp_rn(scale[c]), sbase + l.codes + (warp - 4) * 512);
              const int row = list[64 * c + lane];
              if (leader && w == 0 && row >= 0) {
                uint8_t* at = in_row(a, a.y + a.out + 4 * tile.block, row);
                *reinterpret_cast<float*>(at) = scale[c];
                if (tile.block + 1 == a.blocks)
                  for (uint8_t* end = in_row(a, a.y + a.y_row, row); (at += 4) < end;) *reinterpret_cast<uint32_t*>(at) = 0;
              }
            }
        } else {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              if (a.out_dtype == LLMOE_DTYPE_FP32)
                swiglu<true>(acc[c]);
              else
                swiglu<false>(acc[c]);
              store_swiglu(a, acc[c], first, list + 64 * c, turn);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
    }
  } else {
    fewer_registers<kFewRegisters>();
    // ---- scales ------------------------------------------------------------------
    // Warp q's lane moves those of columns 32 q + lane and 128 + 32 q + lane, 16
    // bytes of a row (four steps) at a time, kAhead such chunks ahead; and lane % 4
    // (with SwiGLU lane % 8) w's of a step (and of gate or up).
    constexpr int kAhead = 3, kParts = kSwiglu ? 2 : 1;
    const int q = warp & 3, chunks = (a.steps + 3) / 4;
    int i = 0, sslot = 0;
    uint32_t sphase = 0;
    bool ok = true;
    for (int t = pair_id; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!(ok = mbar_wait_warp(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
      const Tile tile = tiles[slot];
      const int n = columns(tile.groups), m = 32 * q + lane;
      const int r0 = m < n ? rows[slot * kMaxRows + m] : -1;
      const int r1 = 128 + m < n ? rows[slot * kMaxRows + 128 + m] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
      const uint4* src[2] = {reinterpret_cast<const uint4*>(a.x + (uint64_t)max(r0, 0) * a.x_row + a.in),
                             reinterpret_cast<const uint4*>(a.x + (uint64_t)max(r1, 0) * a.x_row + a.in)};
      const bool have[2] = {r0 >= 0, r1 >= 0};
      // the CTA's features are in one block of w (of gate, of up); past the last one nothing is stored
      const int block = min(kSwiglu ? tile.block : 2 * tile.block + (int)rank, s.down - 1);
      const float* wsrc = s.w_scale + (((int64_t)tile.expert * kParts + (kSwiglu ? lane >> 2 & 1 : 0)) * s.down + block) *
                                          (int64_t)s.across;
      const auto load_w = [&](int c) { return 4 * c + (lane & 3) < s.across ? wsrc[4 * c + (lane & 3)] : 0.0f; };
      uint4 ahead[kAhead][2];
      float w_ahead[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          ahead[u][j] = make_uint4(0, 0, 0, 0);
          if (have[j] && u < chunks) ahead[u][j] = src[j][u];
        }
        w_ahead[u] = load_w(u);
      }
      for (int c0 = 0; c0 < chunks && ok; c0 += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int c = c0 + u;
          if (c >= chunks || !ok) break;
          if (!(ok = mbar_wait_warp(scale_empty + 8 * sslot, sphase ^ 1, a.err))) break;
          float* dst = reinterpret_cast<float*>(smem + l.scales + sslot * kSlot) + m;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float ws = kSwiglu ? 1.0f : __shfl_sync(0xffffffffu, w_ahead[u], b);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4& v = ahead[u][j];
              const float x = __uint_as_float(b == 0 ? v.x : b == 1 ? v.y : b == 2 ? v.z : v.w);
              if (have[j]) dst[b * kMaxRows + j * 128] = kSwiglu ? x : x * ws;
            }
          }
          if (kSwiglu && q == 0 && lane < 8)
            reinterpret_cast<float*>(smem + l.w_scales)[(sslot * 4 + (lane & 3)) * 2 + (lane >> 2)] = w_ahead[u];
          __syncwarp();
          if (lane == 0) mbar_arrive(scale_full + 8 * sslot);
          if (++sslot == kSlots) sslot = 0, sphase ^= 1;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (have[j] && c + kAhead < chunks) ahead[u][j] = src[j][c + kAhead];
          w_ahead[u] = load_w(c + kAhead);
        }
      }
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
template <bool kSwiglu>
int launch_scaled(ScaledArgs& s, llmoe_stream_t stream) {
  ProductArgs& a = s.p;
  a.steps = s.across;
  a.blocks = (a.n + kTileFeatures - 1) / kTileFeatures;
  // tiles at full counts
  const uint64_t groups = (uint64_t)((a.T + kGroup - 1) / kGroup) * a.R, share = kMaxRows / kGroup;
  const uint64_t most = (groups + share - 1) / share * a.E * a.blocks;
  if (most > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  a.stages = kStages;
  while (scaled_smem(a.stages, a.E).total > kMaxSmem) --a.stages;
  const size_t smem = scaled_smem(a.stages, a.E).total;
  a.idesc = (uint32_t)(kTileFeatures >> 4) << 24 | 1u << 4;  // e4m3 operands, fp32 sums, M = 256

  ProductMaps maps;
  const cuuint64_t w_row = (cuuint64_t)a.in;
  for (int b = 0; b < kBoxes; ++b) {
    if (b > 0 && (uint64_t)kGroup << (b - 1) >= (uint64_t)a.R * a.T) break;  // a run is at most an expert's rows
    const cuuint64_t dims[2] = {(cuuint64_t)a.in, (cuuint64_t)a.E * a.R * a.T}, strides[1] = {a.x_row};
    const cuuint32_t box[2] = {128, (cuuint32_t)kGroup << b};
    if (!make_map(&maps.x[b], a.x, a.dtype, dims, strides, box, 2)) return LLMOE_ERR_CUDA;
  }
  if (kSwiglu) {
    // gate and up in turn, eight rows of each: a box is (K, 8 rows, gate / up, 8 such)
    const cuuint64_t dims[5] = {(cuuint64_t)a.in, 8, 2, (cuuint64_t)a.out / 8, (cuuint64_t)a.E},
                     strides[4] = {w_row, w_row * (uint64_t)a.out, w_row * 8, w_row * (uint64_t)a.n};
    const cuuint32_t box[5] = {128, 8, 2, 8, 1};
    if (!make_map(&maps.w, a.w, a.dtype, dims, strides, box, 5)) return LLMOE_ERR_CUDA;
  } else {
    const cuuint64_t dims[3] = {(cuuint64_t)a.in, (cuuint64_t)a.n, (cuuint64_t)a.E},
                     strides[2] = {w_row, w_row * (uint64_t)a.n};
    const cuuint32_t box[3] = {128, 128, 1};
    if (!make_map(&maps.w, a.w, a.dtype, dims, strides, box, 3)) return LLMOE_ERR_CUDA;
  }
  static_assert((kStages - 1) * kStage > kMaxSmem / 2, "one CTA per SM");
  const int pairs = resident_pairs<scaled_kernel<kSwiglu>>(kThreads);
  if (pairs < 1) return LLMOE_ERR_CUDA;
  return launch_block(scaled_kernel<kSwiglu>, 2 * (unsigned)std::min<uint64_t>(most, pairs), kThreads, smem, stream, s,
                      maps);
}

}  // namespace

extern "C" int llmoe_expert_product_fp8b(const void* x, const void* w, const float* w_scale, void* y,
                                         const int64_t* counts, int in_features, int out_features, int out_dtype,
                                         uint32_t flags, const llmoe_buf_set_t* bs, llmoe_stream_t stream) {
  ScaledArgs s;
  ProductArgs& a = s.p;
  const bool swiglu = (flags & LLMOE_PRODUCT_SWIGLU) != 0;
  if ((flags & ~LLMOE_PRODUCT_SWIGLU) != 0 || !product_buckets(counts, bs, &a) ||
      !(out_dtype == LLMOE_DTYPE_BF16 || out_dtype == LLMOE_DTYPE_FP16 || out_dtype == LLMOE_DTYPE_FP32 ||
        (out_dtype == LLMOE_DTYPE_FP8B && swiglu)) ||
      !product_rows(x, y, in_features, out_features, LLMOE_DTYPE_FP8B, out_dtype, swiglu, &a))
    return LLMOE_ERR_INVALID_ARGUMENT;
  s.down = (out_features + LLMOE_FP8B_BLOCK - 1) / LLMOE_FP8B_BLOCK;
  s.across = (int)(((int64_t)in_features + LLMOE_FP8B_BLOCK - 1) / LLMOE_FP8B_BLOCK);
  const uint64_t matrices = (uint64_t)a.E * (swiglu ? 2 : 1), codes = (uint64_t)out_features * in_features;
  if (w == nullptr || w_scale == nullptr || !aligned(w, 16) || !aligned(w_scale, 4) || codes > kMostBytes / matrices)
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t y_bytes = (uint64_t)a.E * a.R * a.T * a.y_row;
  if (overlap(y, y_bytes, w, matrices * codes) || overlap(y, y_bytes, w_scale, matrices * s.down * s.across * 4))
    return LLMOE_ERR_INVALID_ARGUMENT;
  a.w = static_cast<const uint8_t*>(w);
  s.w_scale = w_scale;
  return swiglu ? launch_scaled<true>(s, stream) : launch_scaled<false>(s, stream);
}
