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
#include "block_tensor.cuh"

namespace {

constexpr int kPlanDepth = 4;       // planned tiles in flight
constexpr int kStages = 6;          // of the ring at most; fewer where thousands of experts take their room
constexpr int kTileFeatures = 256;  // rows of w per tile: 128 in each CTA
constexpr int kGroup = 4;           // rows of x taken together
constexpr int kBoxes = 6;           // x loads of 1, 2, .. 32 groups

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
  uint64_t x_row;  // bytes of a row
  uint32_t y_row;
  int dtype, out_dtype;
  int blocks;   // feature tiles per expert
  int steps;    // 128-byte steps of K
  int stages;   // of the ring
  uint32_t idesc;  // instruction descriptor without N and scale ids
};

struct ProductMaps {
  CUtensorMap w, x[kBoxes];
};

// Received rows of the buckets (e, s), s = src, src + stride, ... below R, at
// most N of them (0 for the others); all loads before any check.
template <int N>
__device__ __forceinline__ void bucket_counts(const ProductArgs& a, int e, int src, int stride, int (&rows)[N]) {
  const int64_t* p = a.counts != nullptr
                         ? a.counts + (int64_t)e * a.R
                         : reinterpret_cast<const int64_t*>(a.base + (e / a.L) * a.rank_stride + a.sig_off) +
                               (int64_t)(e % a.L) * a.R;
  int64_t c[N];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = src + i * stride < a.R ? p[src + i * stride] : 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    bad |= c[i] < 0 || c[i] > a.T;
    rows[i] = (int)max((int64_t)0, min(c[i], (int64_t)a.T));
  }
  if (bad) report(a.err, LLMOE_DEV_SLOT_RANGE);
}
__device__ __forceinline__ int groups_of(int rows) { return (rows + kGroup - 1) / kGroup; }

// A planned tile; its rows are in the plan's row list.
struct __align__(16) Tile {
  int expert, block, groups;
  int boxes;  // loads of x rows in this CTA
  int bytes;  // that the loads of x rows of both CTAs bring
};

// One load of consecutive x rows: offset in the stage's rows, first row, and
// the power of two of its groups.
struct __align__(16) Box {
  int offset, row, size, unused;
};

// Columns of a tile's product: a CTA pair's N is a multiple of 32.
__device__ __forceinline__ int columns(int groups) { return (groups * kGroup + 31) / 32 * 32; }

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
// prologue: shares before each expert
// ---------------------------------------------------------------------------
// An expert's groups are cut into shares, the fewest of at most kMaxRows rows;
// every share meets a.blocks feature blocks.  prefix[e] = shares of the experts
// before e (prefix[E]: all).
template <bool kMx>
__device__ void count_shares(const ProductArgs& a, int* prefix, int* part) {
  constexpr int kThreads = Shape<kMx>::kThreads, kMost = Shape<kMx>::kMaxRows / kGroup, kBatch = 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (a.R >= 32) {  // a warp per expert
    for (int e = warp; e < a.E; e += kThreads / 32) {
      int n = 0;
      for (int s = lane; s < a.R; s += 32 * kBatch) {
        int c[kBatch];
        bucket_counts(a, e, s, 32, c);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) n += groups_of(c[i]);
      }
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) prefix[e] = (n + kMost - 1) / kMost;
    }
  } else {
    for (int e = tid; e < a.E; e += kThreads) {
      int n = 0;
      for (int s = 0; s < a.R; s += kBatch) {
        int c[kBatch];
        bucket_counts(a, e, s, 1, c);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) n += groups_of(c[i]);
      }
      prefix[e] = (n + kMost - 1) / kMost;
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
// One expert's buckets, 32 source ranks at a time: lane s holds rank s0 + s's
// rows, and the groups of the ranks from s0 up to and with it.
struct Buckets {
  int expert, s0;
  int rows, incl;
};
__device__ __forceinline__ void load_buckets(const ProductArgs& a, int e, int s0, Buckets& b) {
  if (b.expert == e && b.s0 == s0) return;  // the previous tile's
  const int lane = threadIdx.x & 31;
  b.expert = e;
  b.s0 = s0;
  int c[1];
  bucket_counts(a, e, s0 + lane, 1, c);
  b.rows = c[0];
  b.incl = groups_of(b.rows);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, b.incl, d);
    if (lane >= d) b.incl += v;
  }
}

// Groups of expert e in order: source ranks ascending, slots ascending.  The
// tile's share [g0, g1) goes to list, one entry per column: the row of x and y,
// or -1 where there is none.  A lane takes a group: it finds the group's bucket
// by a search over the lanes' sums.
__device__ void plan_rows(const ProductArgs& a, int e, int g0, int g1, Buckets& b, int* list) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int s0 = 0; s0 < a.R && before < g1; s0 += 32) {
    load_buckets(a, e, s0, b);
    const int end = before + __shfl_sync(0xffffffffu, b.incl, 31);
    for (int first = max(g0, before); first < min(g1, end); first += 32) {
      const int g = first + lane, target = g - before;
      int s = 0;  // the first lane whose sum is above target
#pragma unroll
      for (int d = 16; d; d >>= 1)
        if (__shfl_sync(0xffffffffu, b.incl, s + d - 1) <= target) s += d;
      s = min(s, 31);
      const int cnt = __shfl_sync(0xffffffffu, b.rows, s), incl = __shfl_sync(0xffffffffu, b.incl, s);
      if (g < min(g1, end)) {
        const int slot = (target - (incl - groups_of(cnt))) * kGroup, row = (e * a.R + s0 + s) * a.T + slot;
        static_assert(kGroup == 4, "a group is one 16-byte store");
        *reinterpret_cast<int4*>(list + (g - g0) * kGroup) =
            make_int4(row, slot + 1 < cnt ? row + 1 : -1, slot + 2 < cnt ? row + 2 : -1, slot + 3 < cnt ? row + 3 : -1);
      }
    }
    before = end;
  }
  for (int i = (g1 - g0) * kGroup + lane; i < columns(g1 - g0); i += 32) list[i] = -1;
}

// The box that starts at this lane's group, as the power of two of its groups,
// or -1: a CTA's share of a tile is `groups` groups, lane g's starting at row
// `row`.  A run of consecutive rows is one box, or two of the same size that
// overlap where its length is no power of two (the rows in both are written
// twice, with the same values): loads are bound by their number.
__device__ __forceinline__ int plan_box(int row, int groups) {
  const int lane = threadIdx.x & 31;
  const int prev = __shfl_up_sync(0xffffffffu, row, 1);
  const uint32_t heads = __ballot_sync(0xffffffffu, lane < groups && (lane == 0 || row != prev + kGroup));
  if (lane >= groups) return -1;
  const int head = 31 - __clz(heads & (0xffffffffu >> (31 - lane)));
  const uint32_t later = lane == 31 ? 0 : heads >> (lane + 1);
  const int len = (later ? lane + __ffs(later) : groups) - head, p = lane - head;
  const int size = 31 - __clz(len);
  return p == 0 || p == len - (1 << size) ? size : -1;
}

// Where tile t lies: expert, feature block, and which of the expert's shares.
struct Place {
  int expert, block, share, shares;
};
__device__ __forceinline__ Place find_tile(const ProductArgs& a, const int* prefix, int t) {
  // the largest e with prefix[e] <= t / blocks (it has shares, for the next is
  // above), 32 candidates at a time
  const int lane = threadIdx.x & 31, nth = t / a.blocks;
  int e = 0;
  for (int span = a.E; span > 1;) {
    const int step = (span + 31) / 32, at = e + lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, lane * step < span && prefix[at] <= nth);
    const int last = 31 - __clz(below);  // lane 0's is: prefix[e] <= nth
    e += last * step;
    span = min(step, span - last * step);
  }
  Place p{e, t - prefix[e] * a.blocks, 0, prefix[e + 1] - prefix[e]};
  if (p.shares > 1) {
    const int local = p.block;
    p.block = local / p.shares;
    p.share = local - p.block * p.shares;
  }
  return p;
}

template <bool kMx>
__device__ void plan_tile(const ProductArgs& a, const int* prefix, int t, int rank, Buckets& b, Tile* tile, int* list,
                          Box* boxes) {
  constexpr int kMaxRows = Shape<kMx>::kMaxRows;
  const int lane = threadIdx.x & 31;
  const Place place = find_tile(a, prefix, t);
  const int e = place.expert, shares = place.shares, share = place.share;
  int total = 0;
  for (int s0 = 0; s0 < a.R; s0 += 32) {
    load_buckets(a, e, s0, b);
    total += __shfl_sync(0xffffffffu, b.incl, 31);
  }
  // shares of whole 32s of columns, as equal as that allows, the remainder
  // last: 1040 rows are 4 x 224 + 144 columns, 1056 as padded (five equal
  // shares would pad to 1120).  shares is the fewest that hold the total, so the
  // last is never empty.
  const int per = shares == 1 ? total : columns((total + shares - 1) / shares) / kGroup;
  const int g0 = share * per, g1 = min(total, g0 + per);
  static_assert(kMaxRows % 32 == 0, "a share of at most kMaxRows rows pads to at most kMaxRows");
  plan_rows(a, e, g0, g1, b, list);
  __syncwarp();
  // the loads of each CTA's half of the columns
  const int half = columns(g1 - g0) / 2;
  int bytes = 0, count = 0;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int mine = max(0, min(g1 - g0 - r * (half / kGroup), half / kGroup));
    const int row = lane < mine ? list[r * half + lane * kGroup] : 0;
    const int box = plan_box(row, mine);
    const uint32_t all = __ballot_sync(0xffffffffu, box >= 0);
    bytes += __reduce_add_sync(0xffffffffu, box >= 0 ? kGroup * 128 << box : 0);
    if (r == rank) {
      count = __popc(all);
      if (box >= 0) boxes[__popc(all & ((1u << lane) - 1))] = Box{lane * (kGroup * 128), row, box, 0};
    }
  }
  if (lane == 0) *tile = Tile{e, place.block, g1 - g0, count, bytes};
}

// ---------------------------------------------------------------------------
// epilogue
// ---------------------------------------------------------------------------
// v / (1 + exp(-v)) in fp32, for fp32 outputs, which show its bits (4096 rows of
// 1024 -> 2 x 2048: 38 us against 33 with near_silu, one token 80.3 against 78.1).
__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }
// The same with the hardware's exponential and division, for outputs of 16 or 8
// bits: each within a few units of the last fp32 place (the exponential's also
// grow by |v| halves of one: 30 units at v = -75, a 64th of half an fp16 unit); a
// denominator above 2^126 gives 0 for what is below 2^-118.  silu() for those too
// took one token from 78.9 to 81.1 us.
__device__ __forceinline__ float near_silu(float v) { return __fdividef(v, 1.0f + __expf(-v)); }

// Two values as BF16 or FP16, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// `at`, an address in row 0 of y, moved to `row`.
__device__ __forceinline__ uint8_t* in_row(const ProductArgs& a, uint8_t* at, int row) {
  return at + (uint64_t)(uint32_t)row * a.y_row;
}

// 32 columns (rows of y) of 32 features: lane l holds feature first + l.
// list: the columns' rows, -1 where nothing is stored (read before the stores,
// which the compiler cannot tell from writes to it).
__device__ __forceinline__ void store_plain(const ProductArgs& a, const float (&v)[32], int first, const int* list) {
  const int lane = threadIdx.x & 31;
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
    if (first + lane >= a.out) return;
    uint8_t* at = a.y + (uint64_t)(first + lane) * 4;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
      const int4 row = *reinterpret_cast<const int4*>(list + j);
      if (row.x >= 0) *reinterpret_cast<float*>(in_row(a, at, row.x)) = v[j];
      if (row.y >= 0) *reinterpret_cast<float*>(in_row(a, at, row.y)) = v[j + 1];
      if (row.z >= 0) *reinterpret_cast<float*>(in_row(a, at, row.z)) = v[j + 2];
      if (row.w >= 0) *reinterpret_cast<float*>(in_row(a, at, row.w)) = v[j + 3];
    }
    return;
  }
  // neighbours swap so that a lane holds two features of one column: even
  // lanes the first column of a pair, odd lanes the second
  const bool odd = lane & 1, fp16 = a.out_dtype == LLMOE_DTYPE_FP16;
  const int feature = first + (lane & ~1);
  const bool in = feature < a.out;
  uint8_t* at = a.y + (uint64_t)feature * 2;
  int row[16];
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const int4 r = *reinterpret_cast<const int4*>(list + 2 * i);
    row[i] = odd ? r.y : r.x;
    row[i + 1] = odd ? r.w : r.z;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    // both columns of this lane's feature in one word: it keeps one half
    const uint32_t mine = pack2(v[2 * i], v[2 * i + 1], fp16), got = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint32_t u = __byte_perm(mine, got, odd ? 0x3276 : 0x5410);
    if (in && row[i] >= 0) *reinterpret_cast<uint32_t*>(in_row(a, at, row[i])) = u;
  }
}

// 32 columns of 16 gate and 16 up features, eight of each in turn: lane l holds
// gate (l & 8 == 0) or up of output feature first + l / 16 * 8 + l % 8.  The
// two swap so that gate lanes end with h of even columns and up lanes of odd
// ones.  MX8 output: amax is the exchange's buffer, bar its barrier, parity its
// phase; false when the wait expired.
__device__ __forceinline__ bool store_swiglu(const ProductArgs& a, const float (&v)[32], int first, const int* list,
                                             uint32_t* amax, int warp, uint32_t bar, uint32_t parity) {
  const int lane = threadIdx.x & 31, up = lane >> 3 & 1;
  const int feature = first + (lane >> 4) * 8 + (lane & 7);
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 8);
      const float h = silu(up ? got : v[2 * i]) * (up ? v[2 * i + 1] : got);
      const int row = list[2 * i + up];
      if (row >= 0 && feature < a.out) *reinterpret_cast<float*>(in_row(a, a.y + (uint64_t)feature * 4, row)) = h;
    }
    return true;
  }
  float h[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 8);
    h[i] = up ? near_silu(got) * v[2 * i + 1] : near_silu(v[2 * i]) * got;
  }
  if (a.out_dtype == LLMOE_DTYPE_MX8) {
    // a group of 32 outputs is this warp's 16 and its neighbour's.  The largest
    // magnitudes: lanes of the same columns halve the columns they keep at each
    // of four exchanges, so that lane at = 0..15 of them ends with column
    // 2 at + up's, and the two warps swap through shared memory
    uint32_t m[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) m[i] = magnitude(h[i]);
    int at = 0;
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      const int d = step == 3 ? 16 : 1 << step, keep = 8 >> step;  // lane bits 0, 1, 2, 4
      const bool high = lane & d;
#pragma unroll
      for (int i = 0; i < keep; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? m[i] : m[i + keep], d);
        m[i] = max(high ? m[i + keep] : m[i], got);
      }
      at += high ? keep : 0;
    }
    amax[warp * 32 + up * 16 + at] = m[0];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
    if (!mbar_wait_warp(bar, parity, a.err)) return false;
    uint32_t mine = 0;  // the scale code of column 2 at + up
    uint32_t code[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      code[i] = scale_code(max(amax[warp * 32 + up * 16 + i], amax[(warp ^ 1) * 32 + up * 16 + i]));
      if (i == at) mine = code[i];
    }
    const bool store = feature < a.out;  // whole groups: out is a multiple of 32
    const int q = lane & 3;
    int row[4];
#pragma unroll
    for (int g = 0; g < 4; ++g) row[g] = store ? list[2 * (4 * g + q) + up] : -1;
    const int my_row = store && !(warp & 1) ? list[2 * at + up] : -1;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      // four columns of one feature, turned over four lanes into four features of one column
      uint32_t b = pack_e4m3x2(h[4 * g] * scale_inverse(code[4 * g]), h[4 * g + 1] * scale_inverse(code[4 * g + 1])) |
                   pack_e4m3x2(h[4 * g + 2] * scale_inverse(code[4 * g + 2]),
                               h[4 * g + 3] * scale_inverse(code[4 * g + 3])) << 16;
      uint32_t got = __shfl_xor_sync(0xffffffffu, b, 1);
      b = __byte_perm(b, got, lane & 1 ? 0x3715 : 0x6240);
      got = __shfl_xor_sync(0xffffffffu, b, 2);
      b = __byte_perm(b, got, lane & 2 ? 0x3276 : 0x5410);
      if (row[g] >= 0) *reinterpret_cast<uint32_t*>(in_row(a, a.y + (feature - q), row[g])) = b;
    }
    if (my_row >= 0) {
      uint8_t* s = in_row(a, a.y + a.out + first / 32, my_row);
      *s = (uint8_t)mine;
      if (first + 32 == a.out)
        for (uint8_t* end = in_row(a, a.y + a.y_row, my_row); ++s < end;) *s = 0;
    }
    return true;
  }
  const bool odd = lane & 1, fp16 = a.out_dtype == LLMOE_DTYPE_FP16;
  const int even_feature = feature & ~1;
  int row[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) row[i] = even_feature < a.out ? list[4 * i + 2 * odd + up] : -1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t mine = pack2(h[2 * i], h[2 * i + 1], fp16), got = __shfl_xor_sync(0xffffffffu, mine, 1);
    const uint32_t u = __byte_perm(mine, got, odd ? 0x3276 : 0x5410);
    if (row[i] >= 0) *reinterpret_cast<uint32_t*>(in_row(a, a.y + (uint64_t)even_feature * 2, row[i])) = u;
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
  count_shares<kMx>(a, prefix, reinterpret_cast<int*>(smem + l.part));
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + l.tmem);

  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, ntiles = prefix[a.E] * a.blocks;

  if (warp == 0 || warp == 3) {
    // ---- loads: one thread of each of two warps, on alternate steps ----------------
    if (elect_one()) {
      int stage = warp == 3, i = 0;
      int turn = warp == 3;  // steps until this thread's next
      uint32_t phase = 0;
      bool ok = true;
      for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
        const int slot = i % kPlanDepth;
        if (!(ok = mbar_wait(plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
        const Tile tile = tiles[slot];
        // the first boxes stay in registers: read from shared memory at every
        // step, each load would wait for its box
        constexpr int kKept = 6;
        Box kept[kKept];
#pragma unroll
        for (int b = 0; b < kKept; ++b) kept[b] = b < tile.boxes ? boxes[32 * slot + b] : Box{};
        int k = turn;
        for (; k < a.steps; k += 2) {
          if (!(ok = mbar_wait(empty + 8 * stage, phase ^ 1, a.err))) break;
          const uint32_t data = sbase + stage * S::kStage, to = data + S::kBytesA, bar = map_rank(full + 8 * stage, 0);
          const int k0 = k * (kMx ? 128 : 64);
          if (leader) mbar_expect_tx(full + 8 * stage, 2 * S::kBytesA + tile.bytes);  // both CTAs', w and x
          if constexpr (kSwiglu)
            tma_tile5(data, &maps.w, k0, 0, 0, tile.block * 16 + (int)rank * 8, tile.expert, bar);
          else
            tma_tile3(data, &maps.w, k0, tile.block * kTileFeatures + (int)rank * 128, tile.expert, bar);
#pragma unroll
          for (int b = 0; b < kKept; ++b)
            if (b < tile.boxes) tma_rows(to + kept[b].offset, &maps.x[kept[b].size], k0, kept[b].row, bar);
          for (int b = kKept; b < tile.boxes; b += 4) {
            Box q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) q[u] = b + u < tile.boxes ? boxes[32 * slot + b + u] : Box{};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (b + u < tile.boxes) tma_rows(to + q[u].offset, &maps.x[q[u].size], k0, q[u].row, bar);
          }
          if ((stage += 2) >= a.stages) stage -= a.stages, phase ^= 1;
        }
        turn = k - a.steps;
        mbar_arrive(plan_empty + 8 * slot);
      }
      // the ring drains: no product reads shared memory, and no arrival is under
      // way to this CTA, once every stage has been handed back
      for (int n = turn; n < a.stages && ok; n += 2) {
        ok = mbar_wait(empty + 8 * stage, phase ^ 1, a.err);
        if ((stage += 2) >= a.stages) stage -= a.stages, phase ^= 1;
      }
    }
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
      plan_tile<kMx>(a, prefix, t, (int)rank, buckets, tiles + slot, rows + slot * S::kMaxRows, boxes + 32 * slot);
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
        mbar_arrive_peer(map_rank(acc_empty + 8 * buf, 0));
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
  if (xr == 0 || yr == 0 || yr > INT32_MAX || out > INT32_MAX / 2 || (swiglu && out % 8 != 0)) return LLMOE_ERR_INVALID_ARGUMENT;
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
  a->y_row = (uint32_t)yr;
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
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kMaxSmem = 232448;  // 227 KB

// Opts the kernel in to its shared memory and asks how many pairs can be
// resident, once per device.  Asked with the most shared memory: whatever a call
// uses is more than half of an SM's, so there is one CTA on an SM in any case.
template <bool kMx, bool kSwiglu>
int resident_pairs() {
  static_assert((kStages - 1) * Shape<kMx>::kStage > kMaxSmem / 2, "one CTA per SM");
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kMaxDevices) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  const auto kernel = product_kernel<kMx, kSwiglu>;
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(Shape<kMx>::kThreads);
  cfg.dynamicSmemBytes = kMaxSmem;
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
  if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
  return n;
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
  const int pairs = resident_pairs<kMx, kSwiglu>();
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
