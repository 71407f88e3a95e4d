// block_scaled.cu -- llmoe_expert_product_fp8b (include/llmoe_block.h): matrix
// products grouped by expert over received FP8B rows.
//
// Ring, plan and pairs of CTAs are block_product.cu's: a tile is 256 features and
// up to kMaxRows received rows, 128 features and half of the rows in each CTA.
// What differs is where the sums live.  A block's scales are fp32, so the tensor
// core cannot apply them: it makes the sums of one block of 128 (one step of the
// ring, four instructions) in one of two to eight buffers of tensor memory, and
// eight warps add them, times their scales, to sums that they hold in registers:
//   acc[f][r] += P[f][r] * (s[r] * ws),
// s a row's scale, ws one number for a CTA's 128 features (with SwiGLU one for its
// gate and one for its up features).  Tiles come in two kinds:
//   wide (more than kNarrowRows rows): the rows on the M side, the features on the
//     N side.  A thread of the eight warps is one row and 128 features: it needs one
//     scale a step (two with SwiGLU), read from memory four steps ahead, and has a
//     row's features side by side.
//   narrow: the features on the M side, up to 128 rows on the N side, so that few
//     rows cost few columns.  A thread is one feature and up to 64 rows, whose s * ws
//     it reads four at a time from shared memory.
// The operands in shared memory are the same for both; only the roles differ.
//
// Inside a CTA of 16 warps:
//   warps 0, 3  load (warp 3 also allocates the tensor memory)
//   warp 1      (first CTA of the pair) issues the products
//   warp 2      plans
//   warps 4-11  sums, then the tile's epilogue
//   warps 12-15 make narrow tiles' products of scales in shared memory, four steps at
//               a time, and tell the peer which swaps of magnitudes have been read
// The eight warps have kManyRegisters registers a thread, the others kFewRegisters.
// Every wait is bounded, as there.
//
// What bounds it, on one GB300:
// - few rows per expert: the weights' bytes.  256 experts x ~32 rows, 7168 -> 2 x
//   2048, rows to rows: 1.14-1.17 ms of 1.14 (6.5-6.7 TB/s); 2048 -> 7168, 0.59 of
//   0.58.  One row: eight experts' weights, 44 us of 35; 6 are launch, plan, first
//   load and last stores, and the tiles are 1.7 rounds of the pairs.
// - many rows: the summing warps.  A step of a wide tile is 505 cycles of the tensor
//   core and 750 to 800 of a warp: a wait, loads of 128 columns, 128
//   multiply-adds, the arrival that hands the buffer back, each in the shadow of the
//   tensor core's and the loads' traffic (an access to shared memory takes 140 cycles
//   there).  16 experts x ~1024 rows, 7168 -> 2 x 2048: 442-452 us steadily, 403-414 in
//   a burst (2.3-2.4 PFLOP/s); 2048 -> 7168: 264-274, a quarter of it the epilogues of
//   tiles of 16 steps.
// Three of the four kernels spill a few registers (bytes stored / loaded): with wide
// tiles 116 / 152 with SwiGLU and 48 / 136 plain, without them 40 / 100 plain.
#include "block_plan.cuh"

namespace {

constexpr int kMaxRows = 256, kNarrowRows = 128, kThreads = 512;
constexpr int kBytesA = 128 * 128;
// Bytes and number of the ring's stages.  kFew: a call whose experts have room for
// kNarrowRows rows at most, so that no tile is wide; a stage then has half the room
// for rows, and there are more of them under way (one token, 128 tiles: 44.0 us
// against 45.1 with the other kernel).
template <bool kFew>
constexpr int kStage = kBytesA + (kFew ? kNarrowRows : kMaxRows) / 2 * 128;
template <bool kFew>
constexpr int kRing = kFew ? 8 : kStages;
static_assert(kRing<true> * kStage<true> == kRing<false> * kStage<false>, "the same room");
constexpr int kManyRegisters = 200, kFewRegisters = 56;
static_assert(256 * (kManyRegisters + kFewRegisters) <= 65536, "what a launch of 512 threads has");
constexpr int kBuffers = 8;  // of tensor memory: 8 of 64 columns, 4 of 128 or, for wide tiles, 2 of 256
constexpr int kSlots = 2;    // of scales, four steps each
// A slot: a narrow tile's products of scales [step][gate, up][row], the up ones 16
// bytes further so that a warp's loads of both do not meet in a bank
constexpr int kNarrowStride = kNarrowRows + 4;
constexpr int kSlot = 4 * 2 * kNarrowStride * 4;

struct ScaledArgs {
  ProductArgs p;
  const float* w_scale;
  int down, across;  // blocks of 128 down and across one matrix of w
};

// Byte offsets in dynamic shared memory, from its first 1024-byte boundary.
struct ScaledSmem {
  uint32_t scales, amax, row_max, boxes, rows, tiles, bars, tmem, part, prefix, total;
};
__host__ __device__ inline ScaledSmem scaled_smem(int stages, int stage, int E) {
  ScaledSmem l;
  uint32_t at = stages * stage;
  l.scales = at, at += kSlots * kSlot;
  l.amax = at, at += 2 * 8 * kNarrowRows * 4;  // narrow: [swap's parity][warp of the pair's set][row]
  l.row_max = at, at += 2 * 2 * 128 * 4;       // wide: [tile's parity][set][row]
  l.boxes = at, at += kPlanDepth * 32 * 16;
  l.rows = at, at += kPlanDepth * kMaxRows * 4;
  l.tiles = at, at += kPlanDepth * (uint32_t)sizeof(Tile);
  l.bars = at, at += (2 * kRing<true> + 2 * kBuffers + 2 * kPlanDepth + 2 * kSlots + 12 + 4) * 8;
  l.tmem = at, at += 16;
  l.part = at, at += 64;
  l.prefix = at, at += (E + 1) * 4;
  l.total = at + 1024;  // the base may have to move up to its boundary
  return l;
}

// Buffers a tile uses in turn: as many as its columns leave room for, so that the
// products of narrow tiles run on while the last tile is stored.  A buffer's phase is
// a bit of a word that the issuing thread and the summing warps each keep.
__device__ __forceinline__ int buffers_of(int columns) { return columns > kNarrowRows ? 2 : columns > 64 ? 4 : 8; }
__device__ __forceinline__ bool is_wide(const Tile& t) { return t.groups > kNarrowRows / kGroup; }

// The scales of w for a tile's gate (part 0) or up features, or for those of the
// pair's first or second CTA: one for each step.  Past the last block of features,
// where nothing is stored, the last one's.
template <bool kSwiglu>
__device__ __forceinline__ const float* weight_scales(const ScaledArgs& s, const Tile& tile, int part) {
  const int64_t matrix = kSwiglu ? 2 * (int64_t)tile.expert + part : tile.expert;
  return s.w_scale + (matrix * s.down + (kSwiglu ? tile.block : min(2 * tile.block + part, s.down - 1))) * (int64_t)s.across;
}

// ---------------------------------------------------------------------------
// narrow tiles: lane = feature, 32 rows in a chunk
// ---------------------------------------------------------------------------
// acc += v * scale; scale: shared address
template <int kOffset, int kColumn = 0>
__device__ __forceinline__ void add_rows(const uint32_t (&v)[32], uint32_t scale, float (&acc)[32]) {
  const float4 f = shared_load4<kOffset + 4 * kColumn>(scale);
  acc[kColumn] = __fmaf_rn(__uint_as_float(v[kColumn]), f.x, acc[kColumn]);
  acc[kColumn + 1] = __fmaf_rn(__uint_as_float(v[kColumn + 1]), f.y, acc[kColumn + 1]);
  acc[kColumn + 2] = __fmaf_rn(__uint_as_float(v[kColumn + 2]), f.z, acc[kColumn + 2]);
  acc[kColumn + 3] = __fmaf_rn(__uint_as_float(v[kColumn + 3]), f.w, acc[kColumn + 3]);
  if constexpr (kColumn + 4 < 32) add_rows<kOffset, kColumn + 4>(v, scale, acc);
}

// ---------------------------------------------------------------------------
// wide tiles: lane = row, 32 features in a chunk
// ---------------------------------------------------------------------------
// acc += v * scale, from column kFrom of 32 on; with SwiGLU the features are eight of
// gate, eight of up in turn.
template <bool kSwiglu, int kFrom, int N>
__device__ __forceinline__ void add_features(const uint32_t (&v)[N], float gate, float up, float (&acc)[32]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    acc[kFrom + i] = __fmaf_rn(__uint_as_float(v[i]), kSwiglu && (i & 8) ? up : gate, acc[kFrom + i]);
}

// 32 bytes of each lane's row to y, `at` bytes into the row: neighbours swap halves,
// so that two lanes store the 32 bytes of one of their rows, then the other's.
__device__ __forceinline__ void store_pieces(const ProductArgs& a, const uint4& first, const uint4& second, int row,
                                             int neighbour, uint32_t at, uint32_t end) {
  const bool odd = threadIdx.x & 1;
  uint4 got;
  got.x = __shfl_xor_sync(0xffffffffu, odd ? first.x : second.x, 1);
  got.y = __shfl_xor_sync(0xffffffffu, odd ? first.y : second.y, 1);
  got.z = __shfl_xor_sync(0xffffffffu, odd ? first.z : second.z, 1);
  got.w = __shfl_xor_sync(0xffffffffu, odd ? first.w : second.w, 1);
  at += odd ? 16 : 0;
  const int even_row = odd ? neighbour : row, odd_row = odd ? row : neighbour;
  if (at >= end) return;
  if (even_row >= 0) *reinterpret_cast<uint4*>(in_row(a, a.y + at, even_row)) = odd ? got : first;
  if (odd_row >= 0) *reinterpret_cast<uint4*>(in_row(a, a.y + at, odd_row)) = odd ? second : got;
}

// N values of the lane's row from feature `first` on, to fp32, bf16 or fp16 (N: 16 or 32).
template <int N>
__device__ __forceinline__ void store_values(const ProductArgs& a, const float (&v)[N], int first, int row,
                                             int neighbour) {
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      uint4 q[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        q[u] = make_uint4(__float_as_uint(v[i + 4 * u]), __float_as_uint(v[i + 4 * u + 1]), __float_as_uint(v[i + 4 * u + 2]),
                          __float_as_uint(v[i + 4 * u + 3]));
      store_pieces(a, q[0], q[1], row, neighbour, (uint32_t)(first + i) * 4, (uint32_t)a.out * 4);
    }
    return;
  }
  const bool fp16 = a.out_dtype == LLMOE_DTYPE_FP16;
#pragma unroll
  for (int i = 0; i < N; i += 16) {
    uint4 q[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
      q[u] = make_uint4(pack2(v[i + 8 * u], v[i + 8 * u + 1], fp16), pack2(v[i + 8 * u + 2], v[i + 8 * u + 3], fp16),
                        pack2(v[i + 8 * u + 4], v[i + 8 * u + 5], fp16), pack2(v[i + 8 * u + 6], v[i + 8 * u + 7], fp16));
    store_pieces(a, q[0], q[1], row, neighbour, (uint32_t)(first + i) * 2, (uint32_t)a.out * 2);
  }
}

// h of a chunk's 16 features.
template <bool kAccurate>
__device__ __forceinline__ void swiglu_row(const float (&acc)[32], float (&h)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float gate = acc[i / 8 * 16 + i % 8], up = acc[i / 8 * 16 + 8 + i % 8];
    h[i] = (kAccurate ? silu(gate) : near_silu(gate)) * up;
  }
}

// ---------------------------------------------------------------------------
// a tile's sums
// ---------------------------------------------------------------------------
// What a summing warp keeps from tile to tile.  Under the tensor core's and the
// loads' traffic an access to shared memory takes about 140 cycles, a test of a
// barrier among them, so a step's are issued during the step before: whether its
// sums are there, and its scales.  The steps of a slot of scales are unrolled, so
// that buffers and addresses are constants.
// (Few registers are left beside a wide tile's 128 sums and 64 loaded ones: so one
// address for all barriers here, and what is constant of the call from its arguments.)
struct Sums {
  static constexpr int kScaleFull = 8 * (2 * kBuffers + 2 * kPlanDepth), kScaleEmpty = kScaleFull + 8 * kSlots;
  uint32_t acc_full;     // the first barrier; those of the scales are behind it
  uint32_t leader_empty;
  uint32_t scales;
  uint32_t phases, slots;  // of buffers; slots of scales used
  uint32_t next_done;      // the next step's sums were there when last looked
  bool ok;

  // ok is a lane's own until the tile's end: a vote in every step took 4% of a dense call.
  __device__ __forceinline__ void wait(const ProductArgs& a, int buffer) {
    if (!next_done && ok) ok = mbar_wait_tensor(acc_full + 8 * buffer, phases >> buffer & 1, a.err);
    __syncwarp();
    phases ^= 1u << buffer;
    tc_fence_after();
  }
  __device__ __forceinline__ void look(int buffer) {
    next_done = mbar_test_tensor(acc_full + 8 * buffer, phases >> buffer & 1);
  }
  // this warp has read the buffer
  __device__ __forceinline__ void release(int buffer) {
    tc_fence_before();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_tensor(leader_empty + 8 * buffer);
  }
  static_assert(kSlots == 2, "slots alternate");
  __device__ __forceinline__ uint32_t slot() const { return slots & 1; }
  __device__ __forceinline__ void wait_scales(const ProductArgs& a) {
    if (ok) ok = mbar_wait_cta(acc_full + kScaleFull + 8 * slot(), slots >> 1 & 1, a.err);
    __syncwarp();
  }
  __device__ __forceinline__ void release_scales() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(acc_full + kScaleEmpty + 8 * slot());
    ++slots;
  }

  // Narrow: kChunks times 32 rows, 64 columns apart from address `at` on in buffer 0;
  // scale: their place in the slot's scales; first: the first of the slot's buffers
  // (kCount of them in turn).
  template <int kChunks, int kCount, int kStep>
  __device__ __forceinline__ void narrow_step(const ProductArgs& a, float (&acc)[4][32], uint32_t at, uint32_t scale,
                                              int first) {
    constexpr int kScale = 4 * 2 * kStep * kNarrowStride, kOffset = 512 / kCount * kStep;
    const int next = kStep < 3 ? first + kStep + 1 : kCount == 8 ? first ^ 4 : 0;
    wait(a, first + kStep);
    if constexpr (kChunks > 0) {
      uint32_t v[32];
      tmem_load_begin<kOffset>(at, v);
      tmem_load_end(v);
      if (kChunks == 1) {
        release(first + kStep);
        look(next);
      }
      add_rows<kScale>(v, scale, acc[0]);
    }
    if constexpr (kChunks > 1) {
      uint32_t v[32];
      tmem_load_begin<kOffset + 64>(at, v);
      tmem_load_end(v);
      release(first + kStep);
      look(next);
      add_rows<kScale + 256>(v, scale, acc[1]);
    }
    if constexpr (kChunks == 0) {
      release(first + kStep);
      look(next);
    }
  }
  template <int kChunks, int kCount>
  __device__ __forceinline__ void narrow(const ProductArgs& a, float (&acc)[4][32], uint32_t at, uint32_t scale) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int n = 0; n < 32; ++n) acc[c][n] = 0;
    next_done = 0;
    for (int k = 0; k < a.steps; k += 4) {
      wait_scales(a);
      const int first = kCount == 8 ? k & 4 : 0;
      const uint32_t from = scales + slot() * kSlot + scale, here = at + 64 * first;
      narrow_step<kChunks, kCount, 0>(a, acc, here, from, first);
      if (k + 1 < a.steps) narrow_step<kChunks, kCount, 1>(a, acc, here, from, first);
      if (k + 2 < a.steps) narrow_step<kChunks, kCount, 2>(a, acc, here, from, first);
      if (k + 3 < a.steps) narrow_step<kChunks, kCount, 3>(a, acc, here, from, first);
      release_scales();
    }
  }

  // Wide: the set's 128 features from address `at` on in buffer 0; some: whether the
  // warp has rows at all.  A thread reads its row's scales from memory itself, four
  // steps at a time and four ahead, and w's of a step with a lane each.
  struct Scales {
    const float4* row;   // of the thread's row
    const float* w;      // of step lane % 4: gate or up with SwiGLU, or the first or the last 64 features (lane / 4 % 2)
    float4 now, next;    // of four steps and the next four
    float w_now, w_next;
    float r, w0, w1;     // the step's
    __device__ __forceinline__ void load(int k, int steps) {
      next = make_float4(0, 0, 0, 0), w_next = 0;
      if (k < steps) next = row[k >> 2];
      if (k + (int)(threadIdx.x & 3) < steps) w_next = w[k];
    }
    template <int kStep, bool kBoth>
    __device__ __forceinline__ void take(int kFirst) {
      r = kStep == 0 ? now.x : kStep == 1 ? now.y : kStep == 2 ? now.z : now.w;
      w0 = __shfl_sync(0xffffffffu, w_now, kFirst + kStep);
      if (kBoth) w1 = __shfl_sync(0xffffffffu, w_now, 4 + kStep);
    }
  };
  // The step's columns from kAt on: N load while the last N are added.
  template <bool kSwiglu, int kStep, int kAt, int N>
  __device__ __forceinline__ void wide_columns(uint32_t (&v)[2][N], float (&acc)[4][32], uint32_t at, int set, float g,
                                               float u, Scales& s) {
    constexpr int kBuffer = kStep & 1, kNext = kBuffer ^ 1, kNow = kAt / N & 1;
    tmem_load_end(v[kNow]);
    if constexpr (kAt + N < 128) {
      tmem_load_begin<256 * kBuffer + kAt + N>(at, v[kNow ^ 1]);
    } else {
      release(kBuffer);
      look(kNext);
    }
    add_features<kSwiglu, kAt % 32>(v[kNow], g, u, acc[kAt / 32]);
    if constexpr (kAt + N == 32) {
      if (kStep == 3) s.now = s.next, s.w_now = s.w_next;
      s.take<(kStep + 1) % 4, kSwiglu>(kSwiglu ? 0 : 4 * set);
    }
    if constexpr (kAt + N < 128) wide_columns<kSwiglu, kStep, kAt + N>(v, acc, at, set, g, u, s);
  }
  template <bool kSwiglu, int kStep>
  __device__ __forceinline__ void wide_step(const ProductArgs& a, float (&acc)[4][32], uint32_t at, int set, Scales& s) {
    constexpr int kBuffer = kStep & 1;
    wait(a, kBuffer);
    // 16 columns at a time in the plain product, whose rows' and features' epilogue then
    // spills half the registers (2048 -> 7168 of 2048 rows an expert 264 us, 274 with 32);
    // with SwiGLU 32 (7168 -> 2 x 2048 410 us, 422 with 16)
    uint32_t v[2][kSwiglu ? 32 : 16];
    tmem_load_begin<256 * kBuffer>(at, v[0]);
    const float g = s.r * s.w0, u = kSwiglu ? s.r * s.w1 : g;
    wide_columns<kSwiglu, kStep, 0>(v, acc, at, set, g, u, s);
  }
  template <bool kSwiglu>
  __device__ __forceinline__ void wide(const ProductArgs& a, float (&acc)[4][32], uint32_t at, int set, bool some,
                                       Scales& s) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int n = 0; n < 32; ++n) acc[c][n] = 0;
    next_done = 0;
    if (!some) {
#pragma unroll 1
      for (int k = 0; k < a.steps; ++k) {
        wait(a, k & 1);
        release(k & 1);
        look(k & 1 ^ 1);
      }
      return;
    }
    s.now = s.next, s.w_now = s.w_next;
    s.take<0, kSwiglu>(kSwiglu ? 0 : 4 * set);
    for (int k = 0; k < a.steps; k += 4) {
      s.load(k + 4, a.steps);
      wide_step<kSwiglu, 0>(a, acc, at, set, s);
      if (k + 1 < a.steps) wide_step<kSwiglu, 1>(a, acc, at, set, s);
      if (k + 2 < a.steps) wide_step<kSwiglu, 2>(a, acc, at, set, s);
      if (k + 3 < a.steps) wide_step<kSwiglu, 3>(a, acc, at, set, s);
    }
  }
};

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <bool kSwiglu, bool kFew>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    scaled_kernel(const __grid_constant__ ScaledArgs s, const __grid_constant__ ProductMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  const ProductArgs& a = s.p;
  const uint32_t raw = smem_addr(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - raw % 1024) % 1024);
  const uint32_t sbase = smem_addr(smem);
  const ScaledSmem l = scaled_smem(a.stages, kStage<kFew>, a.E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  int* rows = reinterpret_cast<int*>(smem + l.rows);
  Box* boxes = reinterpret_cast<Box*>(smem + l.boxes);
  Tile* tiles = reinterpret_cast<Tile*>(smem + l.tiles);
  int* prefix = reinterpret_cast<int*>(smem + l.prefix);
  const uint32_t full = sbase + l.bars, empty = full + 8 * kRing<kFew>, acc_full = empty + 8 * kRing<kFew>,
                 acc_empty = acc_full + 8 * kBuffers, plan_full = acc_empty + 8 * kBuffers,
                 plan_empty = plan_full + 8 * kPlanDepth, scale_full = plan_empty + 8 * kPlanDepth,
                 scale_empty = scale_full + 8 * kSlots,
                 // [set][swap's parity]
                 amax_full = scale_empty + 8 * kSlots, amax_read = amax_full + 32, amax_empty = amax_read + 32,
                 row_full = amax_empty + 32;

  if (threadIdx.x == 0) {
    tma_prefetch_map(&maps.w);
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < kBuffers; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 16);  // the summing warps of both CTAs
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(scale_full + 8 * i, 4);
      mbar_init(scale_empty + 8 * i, 8);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(amax_full + 8 * i, 4);   // a set's warps, and the bytes that the peer's send
      mbar_init(amax_read + 8 * i, 4);   // a set's warps
      mbar_init(amax_empty + 8 * i, 1);  // the peer's warp that waits for its set's
    }
    for (int i = 0; i < 4; ++i) mbar_init(row_full + 8 * i, 2);  // the two warps of 32 rows
    for (int i = 0; i < kPlanDepth; ++i) {
      mbar_init(plan_full + 8 * i, 1);
      mbar_init(plan_empty + 8 * i, 14 + (leader ? 1 : 0));  // warps that read a plan
    }
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc_pair(sbase + l.tmem, 512);
  // The pair's barriers and tensor memory are there behind the wait, which the prior
  // grid's and the counting hide (a call of one tile a pair 7.5 us, 8.0 with both parts there)
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  wait_prior_grid();
  release_next_grid();
  count_shares<kMaxRows, kThreads>(a, prefix, reinterpret_cast<int*>(smem + l.part));
  __syncthreads();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + l.tmem);

  const RingBars bars{full, empty, plan_full, plan_empty};
  const int pair_id = blockIdx.x >> 1, pairs = gridDim.x >> 1, ntiles = prefix[a.E] * a.blocks;

  if (warp < 4) {
    fewer_registers<kFewRegisters>();
    if (warp == 0 || warp == 3) {
      if (elect_one())
        load_tiles<kStage<kFew>, kBytesA, 128, kSwiglu, 4>(a, maps, sbase, bars, tiles, boxes, warp == 3, rank, pair_id,
                                                           pairs, ntiles);
    } else if (warp == 1) {
      // ---- products: one thread -----------------------------------------------------
      if (leader && elect_one()) {
        int stage = 0, i = 0;
        uint32_t phase = 0, phases = 0;
        bool ok = true;
        int count = 0;  // of buffers
        const uint32_t desc = tile_desc(sbase);
        for (int t = pair_id; t < ntiles && ok; t += pairs, ++i) {
          const int slot = i % kPlanDepth;
          if (!(ok = mbar_wait_cta(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
          const int rows_n = columns(tiles[slot].groups), was = count;
          const bool wide = !kFew && rows_n > kNarrowRows;
          const uint32_t n = wide ? kTileFeatures : rows_n, idesc = a.idesc | (n >> 3) << 17;
          mbar_arrive(plan_empty + 8 * slot);
          count = buffers_of(rows_n);
          const uint32_t stride = 512 / count;
          if (count != was)  // other columns: every buffer has to be handed back
            for (int b = 0; b < kBuffers && ok; ++b) ok = mbar_wait_tensor(acc_empty + 8 * b, (phases >> b & 1) ^ 1, a.err);
          for (int k = 0; k < a.steps && ok; ++k) {
            const uint32_t w = desc + (uint32_t)(stage * (kStage<kFew> >> 4)), x = w + (kBytesA >> 4);
            const uint32_t m_side = wide ? x : w, n_side = wide ? w : x;
            const int b = k & (count - 1);
            // the later of the two, most often, last
            if (!(ok = mbar_wait(full + 8 * stage, phase, a.err))) break;
            if (!(ok = mbar_wait_tensor(acc_empty + 8 * b, (phases >> b & 1) ^ 1, a.err))) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_8bit(tmem + b * stride, m_side + 2 * j, n_side + 2 * j, idesc, j > 0);
            mma_commit_pair(acc_full + 8 * b);
            phases ^= 1u << b;
            mma_commit_pair(empty + 8 * stage);
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
        plan_tile<kMaxRows, false>(a, prefix, t, (int)rank, buckets, tiles + slot, rows + slot * kMaxRows, boxes + 32 * slot);
        __syncwarp();
        if (lane == 0) mbar_arrive(plan_full + 8 * slot);
      }
    }
  } else if (warp < 12) {
    more_registers<kManyRegisters>();
    // ---- sums and epilogue ---------------------------------------------------------
    // two sets of four warps, warp w of each on tensor-memory lanes 32 w ..
    const int w = warp & 3, set = warp >= 8;
    Sums sums;
    sums.acc_full = acc_full, sums.leader_empty = map_rank(acc_empty, 0);
    sums.scales = sbase + l.scales;
    sums.phases = sums.slots = 0;
    sums.ok = true;
    bool& ok = sums.ok;
    int i = 0, swaps = 0, wide_tiles = 0;  // swaps: of largest magnitudes with the peer
    // the i-th tile's plan; of a wide one this thread's row and first scales, which are
    // asked for before the tile before it is stored
    int row = -1;
    Sums::Scales scales;
    const auto open = [&] {
      const int slot = i % kPlanDepth;
      mbar_wait_cta_warp(plan_full + 8 * slot, (i / kPlanDepth) & 1, ok, a.err);
      const Tile tile = tiles[slot];
      if (!ok || kFew || !is_wide(tile)) return;
      const int half = columns(tile.groups) / 2;  // the pair's halves of the list
      row = 32 * w + lane < half ? rows[slot * kMaxRows + (int)rank * half + 32 * w + lane] : -1;
      scales.row = reinterpret_cast<const float4*>(a.x + (uint64_t)max(row, 0) * a.x_row + a.in);
      scales.w = weight_scales<kSwiglu>(s, tile, lane >> 2 & 1) + (lane & 3);
      scales.load(0, a.steps);
    };
    if (pair_id < ntiles) open();
    for (int t = pair_id; t < ntiles && ok; t += pairs) {
      const int slot = i % kPlanDepth;
      uint32_t lanes = tmem + ((uint32_t)(32 * w) << 16);
      asm volatile("" : "+r"(lanes));  // not kept, with sums of it, from tile to tile
      float acc[4][32];  // one for both kinds of tile: with an array each 1.4 KB of registers spill
      const Tile tile = tiles[slot];
      const int* list = rows + slot * kMaxRows;
      ++i;
      if (!kFew && is_wide(tile)) {
        // set: which half of each CTA's features
        const bool some = 32 * w < columns(tile.groups) / 2;
        constexpr int kChunks = 4;
        sums.wide<kSwiglu>(a, acc, lanes + 128 * set, set, some, scales);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int own = row, neighbour = __shfl_xor_sync(0xffffffffu, row, 1);
        if (t + pairs < ntiles) open();
        if (some) {
          if constexpr (!kSwiglu) {
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
              store_values(a, acc[c], tile.block * kTileFeatures + 128 * set + 32 * c, own, neighbour);
            }
          } else {
            const int first = tile.block * 128 + 64 * set;
            if (a.out_dtype != LLMOE_DTYPE_FP8B) {
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                float h[16];
                if (a.out_dtype == LLMOE_DTYPE_FP32)
                  swiglu_row<true>(acc[c], h);
                else
                  swiglu_row<false>(acc[c], h);
                store_values(a, h, first + 16 * c, own, neighbour);
              }
            } else {
              // a row's block of 128 outputs is this thread's and the other set's
              float h[kChunks][16];
              uint32_t most = 0;
#pragma unroll
              for (int c = 0; c < kChunks; ++c) {
                swiglu_row<false>(acc[c], h[c]);
#pragma unroll
                for (int n = 0; n < 16; ++n) most = max(most, magnitude(h[c][n]));
              }
              uint32_t* swap = reinterpret_cast<uint32_t*>(smem + l.row_max) + (wide_tiles & 1) * 256 + 32 * w + lane;
              swap[128 * set] = most;
              __syncwarp();
              if (lane == 0) mbar_arrive(row_full + 8 * w);
              mbar_wait_cta_warp(row_full + 8 * w, wide_tiles & 1, ok, a.err);
              if (!ok) break;
              most = max(most, swap[128 * (set ^ 1)]);
              const float scale = block_scale(__uint_as_float(most)), inverse = __frcp_rn(scale);
#pragma unroll
              for (int c = 0; c < kChunks; c += 2) {
                uint4 q[2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  uint32_t b[4];
#pragma unroll
                  for (int m = 0; m < 4; ++m)
                    b[m] = pack_e4m3x2(h[c + n][4 * m] * inverse, h[c + n][4 * m + 1] * inverse) |
                           pack_e4m3x2(h[c + n][4 * m + 2] * inverse, h[c + n][4 * m + 3] * inverse) << 16;
                  q[n] = make_uint4(b[0], b[1], b[2], b[3]);
                }
                store_pieces(a, q[0], q[1], own, neighbour, first + 16 * c, a.out);
              }
              if (set == 0 && own >= 0) {
                uint8_t* at = in_row(a, a.y + a.out + 4 * tile.block, own);
                *reinterpret_cast<float*>(at) = scale;
                if (tile.block + 1 == a.blocks)
                  for (uint8_t* end = in_row(a, a.y + a.y_row, own); (at += 4) < end;) *reinterpret_cast<uint32_t*>(at) = 0;
              }
              ++wide_tiles;
            }
          }
        }
      } else {
        // set: every other 32 rows
        const int chunks = (columns(tile.groups) / 32 + 1 - set) / 2, up = kSwiglu ? lane >> 3 & 1 : 0;
        constexpr int kChunks = kNarrowRows / 64;
        const uint32_t scale = 4 * (up * kNarrowStride + 32 * set);
        const uint32_t at = lanes + 32 * set;
        if (buffers_of(columns(tile.groups)) == 8) {
          if (chunks == 1)
            sums.narrow<1, 8>(a, acc, at, scale);
          else
            sums.narrow<0, 8>(a, acc, at, scale);
        } else {
          if (chunks == 2)
            sums.narrow<2, 4>(a, acc, at, scale);
          else
            sums.narrow<1, 4>(a, acc, at, scale);
        }
        static_assert(kChunks == 2, "all numbers of chunks");
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (t + pairs < ntiles) open();
        list += 32 * set;
        const int first = kSwiglu ? tile.block * 128 + (int)rank * 64 + w * 16
                                  : tile.block * kTileFeatures + (int)rank * 128 + w * 32;
        if (!kSwiglu || a.out_dtype != LLMOE_DTYPE_FP8B) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              if constexpr (kSwiglu)
                store_swiglu_values(a, acc[c], first, list + 64 * c);
              else
                store_plain(a, acc[c], first, list + 64 * c);
            }
        } else if (chunks > 0) {
          // A block of 128 outputs is the pair's: its eight warps of this set swap their
          // largest magnitudes, through one of two buffers in turn.  The peer may still
          // read the other one, and has read this one when amax_empty says so (below, at
          // the scales): its reads come before this warp's stores only by a release to
          // the cluster there and an acquire of it here.
          const uint32_t turn = 16 * set + 8 * (swaps & 1), swapped = amax_full + turn;
          if (ok && swaps > 1) ok = mbar_wait_warp(amax_empty + turn, (swaps >> 1 & 1) ^ 1, a.err);
          if (!ok) break;
          uint32_t* amax = reinterpret_cast<uint32_t*>(smem + l.amax) + (swaps & 1) * 8 * kNarrowRows + 32 * set;
          const int source = ((int)rank * 4 + w) * kNarrowRows;
          const uint32_t peer = map_rank(smem_addr(amax + source), rank ^ 1), told = map_rank(swapped, rank ^ 1);
          if (lane == 0) mbar_expect_bytes(swapped, 128 * chunks);
          float h[kChunks][16];
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              swiglu_columns(acc[c], h[c]);
              int at;
              const uint32_t most = largest_of_columns(h[c], at);
              const int column = 64 * c + 2 * at + up;
              amax[source + column] = most;
              shared_store_peer(peer + 4 * column, most, told);
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(swapped);
          ok = mbar_wait_warp(swapped, swaps >> 1 & 1, a.err);  // counted bytes, as loads are
          if (!ok) break;
          float scale[kChunks];  // of row `lane` of each 32
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              uint32_t most = 0;
#pragma unroll
              for (int j = 0; j < 8; ++j) most = max(most, amax[j * kNarrowRows + 64 * c + lane]);
              scale[c] = block_scale(__uint_as_float(most));
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(amax_read + turn);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
              const float mine = __frcp_rn(scale[c]);
              float inverse[16];
#pragma unroll
              for (int n = 0; n < 16; ++n) inverse[n] = __shfl_sync(0xffffffffu, mine, 2 * n + up);
              store_codes(a, h[c], inverse, first, list + 64 * c);
              const int row = list[64 * c + lane];
              if (leader && w == 0 && row >= 0) {
                uint8_t* at = in_row(a, a.y + a.out + 4 * tile.block, row);
                *reinterpret_cast<float*>(at) = scale[c];
                if (tile.block + 1 == a.blocks)
                  for (uint8_t* end = in_row(a, a.y + a.y_row, row); (at += 4) < end;) *reinterpret_cast<uint32_t*>(at) = 0;
              }
            }
          ++swaps;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
    }
  } else {
    fewer_registers<kFewRegisters>();
    // ---- scales ------------------------------------------------------------------
    // Of narrow tiles.  Warp q's lane makes those of row 32 q + lane of the tile's
    // list, 16 bytes of it (four steps) at a time, the next on their way; lane % 4
    // brings w's of a step (with SwiGLU of gate or, lane & 4, up).
    const int q = warp & 3, chunks = (a.steps + 3) / 4;
    // Warps 14 and 15 also tell the peer, once in a tile, that a set here has read the
    // largest magnitudes of the swap before the last, so that the next may take their
    // buffer.  A release to the cluster takes 1500 cycles and more, which the summing
    // warps do not have (decode 1257 us with it there, 1166 here).  Behind a tile's
    // second slot of scales they are at the end of the tile before, and the next slot is
    // long to come (8 steps a tile, 302 us; behind the first, 322).
    const int set = q - 2;
    int i = 0, sslot = 0, swaps = 0;
    uint32_t sphase = 0;
    bool ok = true;
    for (int t = pair_id; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      mbar_wait_cta_warp(plan_full + 8 * slot, (i / kPlanDepth) & 1, ok, a.err);
      if (!ok) break;
      const Tile tile = tiles[slot];
      const int m = 32 * q + lane, row = m < columns(tile.groups) && !is_wide(tile) ? rows[slot * kMaxRows + m] : -1;
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
      if (is_wide(tile)) continue;
      const uint4* src = reinterpret_cast<const uint4*>(a.x + (uint64_t)max(row, 0) * a.x_row + a.in);
      const float* wsrc = weight_scales<kSwiglu>(s, tile, kSwiglu ? lane >> 2 & 1 : (int)rank) + (lane & 3);
      uint4 next = make_uint4(0, 0, 0, 0);
      float w_next = 0;
      const auto load = [&](int c) {
        if (row >= 0 && c < chunks) next = src[c];
        if (4 * c + (lane & 3) < s.across) w_next = wsrc[4 * c];
      };
      load(0);
      for (int c = 0; c < chunks; ++c) {
        const uint4 v = next;
        const float wv = w_next;
        load(c + 1);
        mbar_wait_cta_warp(scale_empty + 8 * sslot, sphase ^ 1, ok, a.err);
        if (!ok) break;
        float* dst = reinterpret_cast<float*>(smem + l.scales + sslot * kSlot) + m;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float x = __uint_as_float(b == 0 ? v.x : b == 1 ? v.y : b == 2 ? v.z : v.w);
#pragma unroll
          for (int p = 0; p < (kSwiglu ? 2 : 1); ++p) {
            const float ws = __shfl_sync(0xffffffffu, wv, 4 * p + b);
            if (row >= 0) dst[(2 * b + p) * kNarrowStride] = x * ws;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(scale_full + 8 * sslot);
        if (++sslot == kSlots) sslot = 0, sphase ^= 1;
        if (kSwiglu && c == min(1, chunks - 1) && a.out_dtype == LLMOE_DTYPE_FP8B && set >= 0 && columns(tile.groups) > 32 * set) {
          const uint32_t turn = 16 * set + 8 * (swaps & 1);
          if (swaps > 1) {
            mbar_wait_cta_warp(amax_read + turn, (swaps >> 1 & 1) ^ 1, ok, a.err);
            if (!ok) break;
            if (lane == 0) mbar_arrive_peer_release(map_rank(amax_empty + turn, rank ^ 1));
          }
          ++swaps;
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
template <bool kSwiglu, bool kFew>
int launch_scaled(ScaledArgs& s, llmoe_stream_t stream) {
  ProductArgs& a = s.p;
  a.steps = s.across;
  a.blocks = (a.n + kTileFeatures - 1) / kTileFeatures;
  // tiles at full counts
  const uint64_t groups = (uint64_t)((a.T + kGroup - 1) / kGroup) * a.R, share = kMaxRows / kGroup;
  const uint64_t most = (groups + share - 1) / share * a.E * a.blocks;
  if (most > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  a.stages = kRing<kFew>;
  while (scaled_smem(a.stages, kStage<kFew>, a.E).total > kMaxSmem) --a.stages;
  const size_t smem = scaled_smem(a.stages, kStage<kFew>, a.E).total;
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
  static_assert((kRing<kFew> - 1) * kStage<kFew> > kMaxSmem / 2, "one CTA per SM");
  const int pairs = resident_pairs<scaled_kernel<kSwiglu, kFew>>(kThreads);
  if (pairs < 1) return LLMOE_ERR_CUDA;
  return launch_block(scaled_kernel<kSwiglu, kFew>, 2 * (unsigned)std::min<uint64_t>(most, pairs), kThreads, smem, stream, s,
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
  if ((int64_t)((a.T + kGroup - 1) / kGroup) * a.R <= kNarrowRows / kGroup)
    return swiglu ? launch_scaled<true, true>(s, stream) : launch_scaled<false, true>(s, stream);
  return swiglu ? launch_scaled<true, false>(s, stream) : launch_scaled<false, false>(s, stream);
}
