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
// Persistent pairs; every pair takes tiles pair, pair + pairs, ... of a list
// that each CTA derives from the counts in its prologue.  Inside a CTA:
//   warp 0     loads: one TMA tile of w and TMA gathers of x rows (four rows of
//              any index per instruction) per 128 bytes of K, into a ring
//   warp 1     (first CTA of the pair) issues the products
//   warp 2     plans: the tile's expert, features and received rows
//   warp 3     8-bit operands: moves the scales into the ring
//   warps 4-7  epilogue: sums from tensor memory, SwiGLU, rounding, stores,
//              while the next tile's products run into the other accumulator
// Every wait is bounded (kSpinLimit cycles); on expiry the role records
// LLMOE_DEV_TIMEOUT and leaves its loop, the others follow when their own waits
// expire, and all meet at the end to free the tensor memory.  A copy in flight
// then was issued at least one expired wait (a second) earlier.
#include "block_tensor.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kPlanDepth = 4;   // planned tiles in flight
constexpr int kMaxStages = 8;
constexpr int kTileFeatures = 256;  // rows of w per tile: 128 in each CTA

// Per operand type: the most rows per tile and the ring stage's layout (128
// bytes of K: 64 values of 16 bits or 128 of 8 bits).
template <bool kMx>
struct Shape {
  // two accumulators of kMaxRows columns; 8-bit scales need 12 more for each stage
  static constexpr int kMaxRows = kMx ? 192 : 256;
  static constexpr int kBytesA = 128 * 128, kBytesB = kMaxRows / 2 * 128;
  static constexpr int kStage = kBytesA + kBytesB;
  static constexpr int kScales = kMx ? 512 + 1024 : 0;  // of 128 w rows, of up to 256 x rows
  static constexpr int kScaleColumns = 12;
  static constexpr int kStages = kMx ? 7 : 6;
  static_assert(2 * kMaxRows + (kMx ? kStages * kScaleColumns : 0) <= 512, "tensor memory has 512 columns");
};

struct ProductArgs {
  const uint8_t* x;
  const uint8_t* w;
  uint8_t* y;
  const int64_t* counts;  // [E][R], or null: the signal words
  const uint8_t* base;    // rank buffers' signal words: base + (e / L) * rank_stride + sig_off
  uint64_t rank_stride, sig_off;
  int32_t* err;
  int T, R, E, L;
  int in, out, n;  // n: rows of w per expert
  uint64_t x_row, y_row;  // bytes
  int dtype, out_dtype;
  int blocks;   // feature tiles per expert
  int steps;    // 128-byte steps of K
  int stages;   // of the ring
  uint32_t idesc;  // instruction descriptor without N and scale ids
};

__device__ __forceinline__ int bucket_count(const ProductArgs& a, int e, int src) {
  const int64_t* p = a.counts != nullptr
                         ? a.counts + (int64_t)e * a.R + src
                         : reinterpret_cast<const int64_t*>(a.base + (e / a.L) * a.rank_stride + a.sig_off) +
                               ((int64_t)(e % a.L) * a.R + src);
  const int64_t c = *p;
  if (c < 0 || c > a.T) report(a.err, LLMOE_DEV_SLOT_RANGE);
  return (int)max((int64_t)0, min(c, (int64_t)a.T));
}

// A planned tile; its rows are in the plan's row list.
struct __align__(16) Tile {
  int expert, block, rows;
};

// Columns of a tile's product: a CTA pair's N is a multiple of 32.
__device__ __forceinline__ int padded(int rows) { return (rows + 31) / 32 * 32; }

// Byte offsets in dynamic shared memory, from its first 1024-byte boundary.
struct SmemLayout {
  uint32_t scales, rows, tiles, amax, bars, tmem, part, prefix, total;
};
template <bool kMx>
__host__ __device__ inline SmemLayout smem_layout(int stages, int E) {
  using S = Shape<kMx>;
  SmemLayout l;
  uint32_t at = stages * S::kStage;
  l.scales = at, at += stages * S::kScales;
  l.rows = at, at += kPlanDepth * S::kMaxRows * 4;
  l.tiles = at, at += kPlanDepth * 16;
  l.amax = at, at += 2 * 4 * 16 * 4;
  l.bars = at, at += (2 * kMaxStages + 4 + 2 * kPlanDepth + 2) * 8;
  l.tmem = at, at += 16;
  l.part = at, at += 32;
  l.prefix = at, at += (E + 1) * 4;
  l.total = at + 1024;  // the base may have to move up to its boundary
  return l;
}

// ---------------------------------------------------------------------------
// prologue: tiles before each expert
// ---------------------------------------------------------------------------
// prefix[e] = tiles of the experts before e (prefix[E]: all tiles).
template <bool kMx>
__device__ void count_tiles(const ProductArgs& a, int* prefix, int* part) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kMaxRows = Shape<kMx>::kMaxRows;
  if (a.R >= 32) {
    for (int e = warp; e < a.E; e += kThreads / 32) {
      int n = 0;
      for (int s = lane; s < a.R; s += 32) n += bucket_count(a, e, s);
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) prefix[e] = (n + kMaxRows - 1) / kMaxRows * a.blocks;
    }
  } else {
    for (int e = tid; e < a.E; e += kThreads) {
      int n = 0;
      for (int s = 0; s < a.R; ++s) n += bucket_count(a, e, s);
      prefix[e] = (n + kMaxRows - 1) / kMaxRows * a.blocks;
    }
  }
  __syncthreads();
  // exclusive scan: a contiguous segment per thread, the segments' sums across the CTA
  const int seg = (a.E + kThreads - 1) / kThreads, lo = min(a.E, tid * seg), hi = min(a.E, lo + seg);
  int sum = 0;
  for (int e = lo; e < hi; ++e) sum += prefix[e];
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  int run = incl - sum;
  for (int w = 0; w < warp; ++w) run += part[w];
  for (int e = lo; e < hi; ++e) {
    const int t = prefix[e];
    prefix[e] = run;
    run += t;
  }
  if (tid == kThreads - 1) prefix[a.E] = run;  // the last segments are empty or end at E
  __syncthreads();
}

// ---------------------------------------------------------------------------
// plan: one warp turns a tile's number into its expert, features and rows
// ---------------------------------------------------------------------------
// Rows of expert e in compact order: source ranks ascending, slots ascending.
// The tile's share [r0, r1) goes to list, padded to a multiple of 32 with its
// last row (the columns of the padding are never stored).
__device__ void plan_rows(const ProductArgs& a, int e, int r0, int r1, int* list) {
  const int lane = threadIdx.x & 31;
  int before = 0, last = 0;
  for (int s0 = 0; s0 < a.R && before < r1; s0 += 32) {
    const int c = s0 + lane < a.R ? bucket_count(a, e, s0 + lane) : 0;
    int incl = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    const int n = min(32, a.R - s0);
    for (int j = 0; j < n; ++j) {
      const int end = before + __shfl_sync(0xffffffffu, incl, j), cnt = __shfl_sync(0xffffffffu, c, j);
      const int beg = end - cnt, lo = max(beg, r0), hi = min(end, r1);
      if (lo >= hi) continue;
      const int first = (e * a.R + s0 + j) * a.T - beg;  // row of compact index i: first + i
      for (int i = lo + lane; i < hi; i += 32) list[i - r0] = first + i;
      last = first + hi - 1;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  const int pad = padded(r1 - r0);
  for (int i = r1 - r0 + lane; i < pad; i += 32) list[i] = last;
}

template <bool kMx>
__device__ void plan_tile(const ProductArgs& a, const int* prefix, int t, Tile* tile, int* list) {
  constexpr int kMaxRows = Shape<kMx>::kMaxRows;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = a.E - 1;  // the largest e with prefix[e] <= t: it has tiles, for t < prefix[e + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int e = lo, shares = (prefix[e + 1] - prefix[e]) / a.blocks;
  const int local = t - prefix[e], share = local % shares;
  int total = 0;
  for (int s = lane; s < a.R; s += 32) total += bucket_count(a, e, s);
  total = __reduce_add_sync(0xffffffffu, total);
  // equal shares: an expert of 300 rows is two tiles of 150
  const int r0 = (int)((int64_t)total * share / shares), r1 = (int)((int64_t)total * (share + 1) / shares);
  static_assert(kMaxRows % 32 == 0, "a share of at most kMaxRows rows pads to at most kMaxRows");
  plan_rows(a, e, r0, r1, list);
  if (lane == 0) *tile = Tile{e, local / shares, r1 - r0};
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------
__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// Two values of one row at `p`, of out_dtype BF16 or FP16.
__device__ __forceinline__ void store2(uint8_t* p, float lo, float hi, int out_dtype) {
  uint32_t u;
  if (out_dtype == LLMOE_DTYPE_FP16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    u = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    u = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint32_t*>(p) = u;
}

// 16 columns (rows of y) of 32 features: lane l holds feature first + l.
// list: the 16 rows; n of them are stored.
__device__ __forceinline__ void store_plain(const ProductArgs& a, const float (&v)[16], int first, const int* list,
                                            int n) {
  const int lane = threadIdx.x & 31;
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n && first + lane < a.out)
        reinterpret_cast<float*>(a.y + list[j] * a.y_row)[first + lane] = v[j];
    return;
  }
  // neighbours swap so that a lane holds two features of one column: even
  // lanes the first column of a pair, odd lanes the second
  const bool odd = lane & 1;
  const int feature = first + (lane & ~1);
#pragma unroll
  for (int j = 0; j < 16; j += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
    const int col = odd ? j + 1 : j;
    if (col < n && feature < a.out)
      store2(a.y + list[col] * a.y_row + (uint64_t)feature * 2, odd ? got : v[j], odd ? v[j + 1] : got, a.out_dtype);
  }
}

// 16 columns of 16 gate (lanes 0-15) and 16 up (lanes 16-31) features.  The
// halves swap so that lanes 0-15 end with h of even columns and lanes 16-31 of
// odd ones, for output feature first + lane % 16.
// MX8 output: amax is the exchange's buffer, bar its barrier, parity its phase;
// false when the wait expired.
__device__ __forceinline__ bool store_swiglu(const ProductArgs& a, const float (&v)[16], int first, const int* list,
                                             int n, uint32_t* amax, int warp, uint32_t bar, uint32_t parity) {
  const int lane = threadIdx.x & 31, half = lane >> 4;
  float h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float got = __shfl_xor_sync(0xffffffffu, half ? v[2 * i] : v[2 * i + 1], 16);
    h[i] = half ? silu(got) * v[2 * i + 1] : silu(v[2 * i]) * got;
  }
  const int feature = first + (lane & 15);
  if (a.out_dtype == LLMOE_DTYPE_MX8) {
    // a group of 32 outputs is this warp's 16 and its neighbour's: the two
    // exchange their largest magnitudes through shared memory
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = magnitude(h[i]);
#pragma unroll
      for (int d = 8; d; d >>= 1) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
      if ((lane & 15) == i) amax[warp * 16 + 2 * i + half] = m[i];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    if (!mbar_wait(bar, parity, a.err)) return false;
    const bool store = feature < a.out;  // whole groups: out is a multiple of 32
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int col = 2 * i + half;
      const uint32_t code = scale_code(max(m[i], amax[(warp ^ 1) * 16 + col]));
      if (col >= n || !store) continue;
      uint8_t* row = a.y + list[col] * a.y_row;
      row[feature] = (uint8_t)pack_e4m3x2(h[i] * scale_inverse(code), 0.0f);
      if ((lane & 15) == 0 && !(warp & 1)) {
        uint8_t* s = row + a.out + feature / 32;
        *s = (uint8_t)code;
        if (feature + 32 == a.out)
          for (uint8_t* end = row + a.y_row; ++s < end;) *s = 0;
      }
    }
    return true;
  }
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (2 * i + half < n && feature < a.out)
        reinterpret_cast<float*>(a.y + list[2 * i + half] * a.y_row)[feature] = h[i];
    return true;
  }
  const bool odd = lane & 1;
  const int even_feature = feature & ~1;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? h[i] : h[i + 1], 1);
    const int col = 2 * (odd ? i + 1 : i) + half;
    if (col < n && even_feature < a.out)
      store2(a.y + list[col] * a.y_row + (uint64_t)even_feature * 2, odd ? got : h[i], odd ? h[i + 1] : got,
             a.out_dtype);
  }
  return true;
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <bool kMx, bool kSwiglu>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    product_kernel(const __grid_constant__ ProductArgs a, const __grid_constant__ CUtensorMap map_x,
                   const __grid_constant__ CUtensorMap map_w) {
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
  Tile* tiles = reinterpret_cast<Tile*>(smem + l.tiles);
  int* prefix = reinterpret_cast<int*>(smem + l.prefix);
  const uint32_t full = sbase + l.bars, empty = full + 8 * kMaxStages, acc_full = empty + 8 * kMaxStages,
                 acc_empty = acc_full + 16, plan_full = acc_empty + 16, plan_empty = plan_full + 8 * kPlanDepth,
                 halves = plan_empty + 8 * kPlanDepth;

  release_next_grid();
  if (threadIdx.x == 0) {
    tma_prefetch_map(&map_x);
    tma_prefetch_map(&map_w);
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full + 8 * s, kMx ? 3 : 1);  // the leader's bytes-expected, each CTA's scales
      mbar_init(empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(halves + 8 * b, 2);  // the two epilogue warps of an output group
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, 8);  // the epilogue warps of both CTAs
    }
    for (int p = 0; p < kPlanDepth; ++p) {
      mbar_init(plan_full + 8 * p, 1);
      mbar_init(plan_empty + 8 * p, 5 + (leader ? 1 : 0) + (kMx ? 1 : 0));  // warps that read a plan
    }
    mbar_init_fence();
  }
  if (warp == 3) tmem_alloc_pair(sbase + l.tmem, 512);
  wait_prior_grid();
  count_tiles<kMx>(a, prefix, reinterpret_cast<int*>(smem + l.part));
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + l.tmem);

  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, ntiles = prefix[a.E];

  if (warp == 0) {
    // ---- loads -------------------------------------------------------------
    int stage = 0, i = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!(ok = mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
      const Tile tile = tiles[slot];
      const int half = padded(tile.rows) / 2;  // rows this CTA loads
      const int* list = rows + slot * S::kMaxRows + rank * half;
      int4 r = make_int4(0, 0, 0, 0);
      if (4 * lane < half) r = make_int4(list[4 * lane], list[4 * lane + 1], list[4 * lane + 2], list[4 * lane + 3]);
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
      // first row of w per load: one load of 128 rows, or with gate and up
      // eight of 16 rows, gate and up in turn, so that a tensor-memory lane and
      // the lane 16 further hold gate and up of one output
      const int feature = kSwiglu ? (lane & 1) * a.out + tile.block * 128 + (int)rank * 64 + (lane >> 1) * 16
                                  : tile.block * kTileFeatures + (int)rank * 128;
      for (int k = 0; k < a.steps; ++k) {
        if (!(ok = mbar_wait(empty + 8 * stage, phase ^ 1, a.err))) break;
        const uint32_t data = sbase + stage * S::kStage, bar = map_rank(full + 8 * stage, 0);
        const int k0 = k * (kMx ? 128 : 64);
        if (leader && lane == 0) mbar_expect_tx(full + 8 * stage, 2 * (S::kBytesA + half * 128));
        __syncwarp();
        if (lane < (kSwiglu ? 8 : 1)) tma_tile(data + (kSwiglu ? lane * 2048 : 0), &map_w, k0, feature, tile.expert, bar);
        if (4 * lane < half) tma_gather4(data + S::kBytesA + lane * 512, &map_x, k0, r, bar);
        __syncwarp();
        if (++stage == a.stages) stage = 0, phase ^= 1;
      }
    }
    // the ring drains: no product reads shared memory, and no arrival is under
    // way to this CTA, once every stage has been handed back
    for (int s = 0; s < a.stages && ok; ++s) {
      ok = mbar_wait(empty + 8 * stage, phase ^ 1, a.err);
      if (++stage == a.stages) stage = 0, phase ^= 1;
    }
  } else if (warp == 1 && leader) {
    // ---- products ------------------------------------------------------------
    int stage = 0, i = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth, buf = i & 1;
      if (!(ok = mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
      const int n = padded(tiles[slot].rows);
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
      if (!(ok = mbar_wait(acc_empty + 8 * buf, ((i >> 1) & 1) ^ 1, a.err))) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * S::kMaxRows, idesc = a.idesc | (uint32_t)(n >> 3) << 17;
      for (int k = 0; k < a.steps; ++k) {
        if (!(ok = mbar_wait(full + 8 * stage, phase, a.err))) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t data = sbase + stage * S::kStage;
          const uint64_t da = tile_desc(data), db = tile_desc(data + S::kBytesA);
          if constexpr (kMx) {
            const uint32_t sc = sbase + l.scales + stage * S::kScales;
            const uint32_t ta = tmem + 2 * S::kMaxRows + stage * S::kScaleColumns, tb = ta + 4;
            copy_scales(ta, scale_desc(sc));
            copy_scales(tb, scale_desc(sc + 512));
            if (n > 128) copy_scales(tb + 4, scale_desc(sc + 1024));
#pragma unroll
            for (int j = 0; j < 4; ++j)  // 32 bytes of K; scale j of each row's four
              mma_mx8(d, da + 2 * j, db + 2 * j, idesc | (uint32_t)j << 4 | (uint32_t)j << 29, ta, tb, k > 0 || j > 0);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_16bit(d, da + 2 * j, db + 2 * j, idesc, k > 0 || j > 0);
          }
          mma_commit_pair(empty + 8 * stage);
          if (k == a.steps - 1) mma_commit_pair(acc_full + 8 * buf);
        }
        __syncwarp();
        if (++stage == a.stages) stage = 0, phase ^= 1;
      }
    }
  } else if (warp == 2) {
    // ---- plan ------------------------------------------------------------------
    int i = 0;
    for (int t = pair; t < ntiles; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!mbar_wait(plan_empty + 8 * slot, ((i / kPlanDepth) & 1) ^ 1, a.err)) break;
      plan_tile<kMx>(a, prefix, t, tiles + slot,
                     rows + slot * S::kMaxRows);
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_full + 8 * slot);
    }
  } else if (warp == 3 && kMx) {
    // ---- scales ------------------------------------------------------------------
    // Lane l moves the scales of w rows l, l + 32, l + 64, l + 96 and of x rows
    // l, l + 32, ...: 4 bytes of each row per stage, which together are the 16
    // bytes that lane l's tensor-memory lane takes.  16 bytes of a row are read
    // at a time, for four stages, one such chunk ahead.
    int stage = 0, i = 0;
    uint32_t phase = 0;
    bool ok = true;
    const int nscale = a.in / 32, chunks = (a.steps + 3) / 4;
    for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
      const int slot = i % kPlanDepth;
      if (!(ok = mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
      const Tile tile = tiles[slot];
      const int n = padded(tile.rows);
      const uint8_t* src[12];  // 4 rows of w, 8 of x
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int m = lane + 32 * j;  // row of this CTA's 128
        int f = kSwiglu ? (m >> 4 & 1) * a.out + tile.block * 128 + (int)rank * 64 + (m >> 5) * 16 + (m & 15)
                        : tile.block * kTileFeatures + (int)rank * 128 + m;
        f = min(f, a.n - 1);  // past the expert's last row: its products are not stored
        src[j] = a.w + ((uint64_t)tile.expert * a.n + f) * a.x_row + a.in;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        src[4 + j] = a.x + rows[slot * S::kMaxRows + min(lane + 32 * j, n - 1)] * a.x_row + a.in;
      __syncwarp();
      if (lane == 0) mbar_arrive(plan_empty + 8 * slot);
      const int nx = n > 128 ? 12 : 8;
      uint4 q[12];
#pragma unroll
      for (int j = 0; j < 12; ++j)
        if (j < nx) q[j] = __ldg(reinterpret_cast<const uint4*>(src[j]));
      for (int c = 0; c < chunks && ok; ++c) {
        uint4 now[12];
#pragma unroll
        for (int j = 0; j < 12; ++j) now[j] = q[j];
        if (c + 1 < chunks) {
#pragma unroll
          for (int j = 0; j < 12; ++j)
            if (j < nx) q[j] = __ldg(reinterpret_cast<const uint4*>(src[j] + 16 * (c + 1)));
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int k = 4 * c + b;
          if (k >= a.steps || !ok) break;
          // scales past the row's last are 1: the codes there are zeros, and 0 * NaN would not be
          const int have = nscale - 4 * k;
          const uint32_t keep = have >= 4 ? 0xffffffffu : (1u << 8 * have) - 1, fill = 0x7f7f7f7fu & ~keep;
          uint32_t word[12];
#pragma unroll
          for (int j = 0; j < 12; ++j) {
            const uint32_t u = b == 0 ? now[j].x : b == 1 ? now[j].y : b == 2 ? now[j].z : now[j].w;
            word[j] = (u & keep) | fill;
          }
          if (!(ok = mbar_wait(empty + 8 * stage, phase ^ 1, a.err))) break;
          uint4* dst = reinterpret_cast<uint4*>(smem + l.scales + stage * S::kScales) + lane;
          dst[0] = make_uint4(word[0], word[1], word[2], word[3]);
          dst[32] = make_uint4(word[4], word[5], word[6], word[7]);
          if (n > 128) dst[64] = make_uint4(word[8], word[9], word[10], word[11]);
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_rank(full + 8 * stage, 0));
          if (++stage == a.stages) stage = 0, phase ^= 1;
        }
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue ------------------------------------------------------------------
    const int w = warp & 3;  // tensor-memory lanes 32 w ..
    uint32_t* amax = reinterpret_cast<uint32_t*>(smem + l.amax);
    int i = 0, flip = 0;
    for (int t = pair; t < ntiles; t += pairs, ++i) {
      const int slot = i % kPlanDepth, buf = i & 1;
      if (!mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err)) break;
      const Tile tile = tiles[slot];
      const int* list = rows + slot * S::kMaxRows;
      const int first = kSwiglu ? tile.block * 128 + (int)rank * 64 + w * 16
                                : tile.block * kTileFeatures + (int)rank * 128 + w * 32;
      if (!mbar_wait(acc_full + 8 * buf, (i >> 1) & 1, a.err)) break;
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * w) << 16) + buf * S::kMaxRows;
      bool ok = true;
      for (int c = 0; c < tile.rows && ok; c += 16) {
        float v[16];
        tmem_load16(acc + c, v);
        if constexpr (kSwiglu) {
          // two buffers in turn: a warp that fills one again has met its
          // neighbour at the other since, so the neighbour has read it
          ok = store_swiglu(a, v, first, list + c, tile.rows - c, amax + 64 * flip, w, halves + 8 * (w >> 1), flip);
          flip ^= 1;
        } else {
          store_plain(a, v, first, list + c, tile.rows - c);
        }
      }
      if (!ok) break;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_cluster(map_rank(acc_empty + 8 * buf, 0));
        mbar_arrive(plan_empty + 8 * slot);
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
// Checks a product's arguments and fills its geometry.
int product_args(const void* x, const void* w, void* y, const int64_t* counts, int in, int out, int dtype,
                 int out_dtype, uint32_t flags, const llmoe_buf_set_t* bs, ProductArgs* a) {
  if (bs == nullptr || (flags & ~LLMOE_PRODUCT_SWIGLU) != 0) return LLMOE_ERR_INVALID_ARGUMENT;
  const bool swiglu = (flags & LLMOE_PRODUCT_SWIGLU) != 0;
  const int T = bs->num_max_tokens, R = bs->num_ranks, E = bs->num_experts;
  if (T < 1 || R < 1 || E < R || E % R != 0 || E > LLMOE_MAX_EXPERTS || !aligned(bs->err, 4))
    return LLMOE_ERR_INVALID_ARGUMENT;
  if ((uint64_t)E * R > INT32_MAX || (uint64_t)E * R * T > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  switch (dtype) {
    case LLMOE_DTYPE_BF16:
    case LLMOE_DTYPE_FP16:
      if (out_dtype != dtype && out_dtype != LLMOE_DTYPE_FP32) return LLMOE_ERR_INVALID_ARGUMENT;
      break;
    case LLMOE_DTYPE_MX8:
      if (out_dtype == LLMOE_DTYPE_MX8 && !swiglu) return LLMOE_ERR_INVALID_ARGUMENT;
      break;
    default: return LLMOE_ERR_INVALID_ARGUMENT;
  }
  const uint64_t xr = row_bytes(in, dtype), yr = row_bytes(out, out_dtype);
  if (xr == 0 || yr == 0 || out > INT32_MAX / 2) return LLMOE_ERR_INVALID_ARGUMENT;
  if (x == nullptr || w == nullptr || y == nullptr || !aligned(x, 16) || !aligned(w, 16) || !aligned(y, 16) ||
      !aligned(counts, 8))
    return LLMOE_ERR_INVALID_ARGUMENT;
  const uint64_t rows = (uint64_t)E * R * T, n = (uint64_t)out * (swiglu ? 2 : 1);
  const uint64_t limit = (uint64_t)INT64_MAX / 2;
  if (xr > limit / rows || yr > limit / rows || xr > limit / (n * E)) return LLMOE_ERR_INVALID_ARGUMENT;
  if (overlap(y, rows * yr, x, rows * xr) || overlap(y, rows * yr, w, n * E * xr)) return LLMOE_ERR_INVALID_ARGUMENT;
  *a = ProductArgs{};
  if (counts == nullptr) {
    const size_t total = llmoe_layout_bytes_dtype(T, bs->hidden, R, E, bs->dtype);
    uint64_t sig = 0;
    if (total == 0 || bs->base == nullptr || !aligned(bs->base, 16) || bs->rank_stride % 16 != 0 ||
        bs->rank_stride < total || bs->rank_stride > limit / R ||
        llmoe_layout_offsets_dtype(T, bs->hidden, R, E, bs->dtype, bs->set, nullptr, nullptr, &sig) != LLMOE_SUCCESS ||
        sig % 8 != 0)
      return LLMOE_ERR_INVALID_ARGUMENT;
    a->base = static_cast<const uint8_t*>(bs->base);
    a->rank_stride = bs->rank_stride;
    a->sig_off = sig;
  }
  a->x = static_cast<const uint8_t*>(x);
  a->w = static_cast<const uint8_t*>(w);
  a->y = static_cast<uint8_t*>(y);
  a->counts = counts;
  a->err = bs->err;
  a->T = T;
  a->R = R;
  a->E = E;
  a->L = E / R;
  a->in = in;
  a->out = out;
  a->n = (int)n;
  a->x_row = xr;
  a->y_row = yr;
  a->dtype = dtype;
  a->out_dtype = out_dtype;
  return LLMOE_SUCCESS;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once (the library does not link libcuda).
EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> cache{nullptr};
  EncodeTiled f = cache.load(std::memory_order_acquire);
  if (f != nullptr) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
      found != cudaDriverEntryPointSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  f = reinterpret_cast<EncodeTiled>(p);
  cache.store(f, std::memory_order_release);
  return f;
}

// Rows of 128-byte steps along K, 128-byte swizzle; `dims` beyond the row.
bool make_map(CUtensorMap* m, const void* base, int dtype, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box, int rank) {
  const EncodeTiled encode = encode_tiled();
  if (encode == nullptr) return false;
  const CUtensorMapDataType type = dtype == LLMOE_DTYPE_BF16   ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == LLMOE_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const cuuint32_t ones[3] = {1, 1, 1};
  return encode(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kMaxSmem = 232448;  // 227 KB

// Opts the kernel in to its shared memory and asks how many pairs can be
// resident, once per device and shared-memory size.
template <bool kMx, bool kSwiglu>
int resident_pairs(size_t smem) {
  constexpr int kMaxDevices = 64;
  static std::atomic<uint64_t> cache[kMaxDevices];  // bytes << 32 | pairs
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kMaxDevices) {
    const uint64_t c = cache[dev].load(std::memory_order_relaxed);
    if (c >> 32 == smem) return (int)(uint32_t)c;
  }
  const auto kernel = product_kernel<kMx, kSwiglu>;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 0;
  }
  if (dev < kMaxDevices) cache[dev].store((uint64_t)smem << 32 | (uint32_t)n, std::memory_order_relaxed);
  return n;
}

template <bool kMx, bool kSwiglu>
int launch_product(ProductArgs& a, llmoe_stream_t stream) {
  using S = Shape<kMx>;
  a.steps = (int)(((int64_t)a.in * (kMx ? 1 : 2) + 127) / 128);
  a.blocks = (a.n + kTileFeatures - 1) / kTileFeatures;
  const uint64_t most = ((uint64_t)a.R * a.T + S::kMaxRows - 1) / S::kMaxRows * a.E * a.blocks;  // tiles at full counts
  if (most > INT32_MAX) return LLMOE_ERR_INVALID_ARGUMENT;
  a.stages = S::kStages;
  while (smem_layout<kMx>(a.stages, a.E).total > kMaxSmem) --a.stages;
  const size_t smem = smem_layout<kMx>(a.stages, a.E).total;
  // both operands 16-bit or both e4m3 (0), fp32 sums, M = 256; 8-bit: e8m0 scales
  const uint32_t type = a.dtype == LLMOE_DTYPE_BF16 ? 1 : 0;
  a.idesc = (uint32_t)(kTileFeatures >> 4) << 24 | type << 7 | type << 10 | (kMx ? 1u << 23 : 1u << 4);

  CUtensorMap map_x, map_w;
  const cuuint32_t k_box = kMx ? 128 : 64;
  {
    const cuuint64_t dims[2] = {(cuuint64_t)a.in, (cuuint64_t)a.E * a.R * a.T}, strides[1] = {a.x_row};
    const cuuint32_t box[2] = {k_box, 1};
    if (!make_map(&map_x, a.x, a.dtype, dims, strides, box, 2)) return LLMOE_ERR_CUDA;
  }
  {
    const cuuint64_t dims[3] = {(cuuint64_t)a.in, (cuuint64_t)a.n, (cuuint64_t)a.E},
                     strides[2] = {a.x_row, a.x_row * (uint64_t)a.n};
    const cuuint32_t box[3] = {k_box, kSwiglu ? 16u : 128u, 1};
    if (!make_map(&map_w, a.w, a.dtype, dims, strides, box, 3)) return LLMOE_ERR_CUDA;
  }
  const int pairs = resident_pairs<kMx, kSwiglu>(smem);
  if (pairs < 1) return LLMOE_ERR_CUDA;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (unsigned)std::min<uint64_t>(most, pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, product_kernel<kMx, kSwiglu>, a, map_x, map_w) != cudaSuccess) {
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
