// block_plan.cuh -- what the expert products share: their arguments, the plan
// that turns counts into tiles and loads, tensor maps, and SwiGLU.
#pragma once
#include "block_tensor.cuh"

namespace {

constexpr int kPlanDepth = 4;       // planned tiles in flight
constexpr int kStages = 6;          // of the ring at most; fewer where thousands of experts take their room
constexpr int kTileFeatures = 256;  // rows of w per tile: 128 in each CTA
constexpr int kGroup = 4;           // rows of x taken together
constexpr int kBoxes = 6;           // x loads of 1, 2, .. 32 groups

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
  uint64_t x_row;  // bytes of a row of x
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

// ---------------------------------------------------------------------------
// prologue: shares before each expert
// ---------------------------------------------------------------------------
// An expert's groups are cut into shares, the fewest of at most kMaxRows rows;
// every share meets a.blocks feature blocks.  prefix[e] = shares of the experts
// before e (prefix[E]: all).
template <int kMaxRows, int kThreads>
__device__ void count_shares(const ProductArgs& a, int* prefix, int* part) {
  constexpr int kMost = kMaxRows / kGroup, kBatch = 8;
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

template <int kMaxRows, bool kEven>
__device__ void plan_tile(const ProductArgs& a, const int* prefix, int t, int rank, Buckets& b, Tile* tile, int* list,
                          Box* boxes) {
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
  // (Not kEven: full shares and what is left.)
  const int per = shares == 1 ? total : kEven ? columns((total + shares - 1) / shares) / kGroup : kMaxRows / kGroup;
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
// loads
// ---------------------------------------------------------------------------
// Barriers of the ring and of the plans, as shared-memory addresses.
struct RingBars {
  uint32_t full, empty, plan_full, plan_empty;
};

// One thread of each of two warps, on alternate steps: one box of w and those of
// x's rows per 128 bytes of K.
template <int kStage, int kBytesA, int kStepValues, bool kSwiglu, int kKept>
__device__ __forceinline__ void load_tiles(const ProductArgs& a, const ProductMaps& maps, uint32_t sbase,
                                           const RingBars& bars, const Tile* tiles, const Box* boxes, bool second,
                                           uint32_t rank, int pair, int pairs, int ntiles) {
  int stage = second, i = 0;
  int turn = second;  // steps until this thread's next
  uint32_t phase = 0;
  bool ok = true;
  for (int t = pair; t < ntiles && ok; t += pairs, ++i) {
    const int slot = i % kPlanDepth;
    if (!(ok = mbar_wait(bars.plan_full + 8 * slot, (i / kPlanDepth) & 1, a.err))) break;
    const Tile tile = tiles[slot];
    // the first boxes stay in registers: read from shared memory at every
    // step, each load would wait for its box
    Box kept[kKept];
#pragma unroll
    for (int b = 0; b < kKept; ++b) kept[b] = b < tile.boxes ? boxes[32 * slot + b] : Box{};
    int k = turn;
    for (; k < a.steps; k += 2) {
      if (!(ok = mbar_wait(bars.empty + 8 * stage, phase ^ 1, a.err))) break;
      const uint32_t data = sbase + stage * kStage, to = data + kBytesA, bar = map_rank(bars.full + 8 * stage, 0);
      const int k0 = k * kStepValues;
      if (rank == 0) mbar_expect_tx(bars.full + 8 * stage, 2 * kBytesA + tile.bytes);  // both CTAs', w and x
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
    mbar_arrive(bars.plan_empty + 8 * slot);
  }
  // the ring drains: no product reads shared memory, and no arrival is under
  // way to this CTA, once every stage has been handed back
  for (int n = turn; n < a.stages && ok; n += 2) {
    ok = mbar_wait(bars.empty + 8 * stage, phase ^ 1, a.err);
    if ((stage += 2) >= a.stages) stage -= a.stages, phase ^= 1;
  }
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

// SwiGLU: 32 columns of 16 gate and 16 up features, eight of each in turn: lane l
// holds gate (l & 8 == 0) or up of output feature first + l / 16 * 8 + l % 8.
__device__ __forceinline__ int swiglu_feature(int first) {
  const int lane = threadIdx.x & 31;
  return first + (lane >> 4) * 8 + (lane & 7);
}
// Gate and up lanes swap, so that gate lanes end with h of even columns and up
// lanes of odd ones: h[i] is column 2 i + up's.
__device__ __forceinline__ void swiglu_columns(const float (&v)[32], float (&h)[16]) {
  const bool up = threadIdx.x >> 3 & 1;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 8);
    h[i] = up ? near_silu(got) * v[2 * i + 1] : near_silu(v[2 * i]) * got;
  }
}

// To rows of fp32, bf16 or fp16.
__device__ __forceinline__ void store_swiglu_values(const ProductArgs& a, const float (&v)[32], int first,
                                                    const int* list) {
  const int lane = threadIdx.x & 31, up = lane >> 3 & 1, feature = swiglu_feature(first);
  if (a.out_dtype == LLMOE_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[2 * i] : v[2 * i + 1], 8);
      const float h = silu(up ? got : v[2 * i]) * (up ? v[2 * i + 1] : got);
      const int row = list[2 * i + up];
      if (row >= 0 && feature < a.out) *reinterpret_cast<float*>(in_row(a, a.y + (uint64_t)feature * 4, row)) = h;
    }
    return;
  }
  float h[16];
  swiglu_columns(v, h);
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
}

// The largest magnitude of each column of the warp's 16 features: lanes of the
// same columns halve the columns they keep at each of four exchanges, so that
// lane at = 0..15 of them ends with column 2 at + up's.
__device__ __forceinline__ uint32_t largest_of_columns(const float (&h)[16], int& at) {
  const int lane = threadIdx.x & 31;
  uint32_t m[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) m[i] = magnitude(h[i]);
  at = 0;
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
  return m[0];
}

// h as e4m3 codes; inverse[i]: 1 / scale of column 2 i + up.  Where any feature of
// four is in y, all are (y's features are whole eights).
__device__ __forceinline__ void store_codes(const ProductArgs& a, const float (&h)[16], const float (&inverse)[16],
                                            int first, const int* list) {
  const int lane = threadIdx.x & 31, up = lane >> 3 & 1, feature = swiglu_feature(first), q = lane & 3;
  int row[4];
#pragma unroll
  for (int g = 0; g < 4; ++g) row[g] = feature < a.out ? list[2 * (4 * g + q) + up] : -1;
  // four columns of one feature, turned over four lanes into four features of one
  // column; each exchange for all four groups at once, for they take long
  uint32_t b[4], got[4];
#pragma unroll
  for (int g = 0; g < 4; ++g)
    b[g] = pack_e4m3x2(h[4 * g] * inverse[4 * g], h[4 * g + 1] * inverse[4 * g + 1]) |
           pack_e4m3x2(h[4 * g + 2] * inverse[4 * g + 2], h[4 * g + 3] * inverse[4 * g + 3]) << 16;
#pragma unroll
  for (int g = 0; g < 4; ++g) got[g] = __shfl_xor_sync(0xffffffffu, b[g], 1);
#pragma unroll
  for (int g = 0; g < 4; ++g) b[g] = __byte_perm(b[g], got[g], lane & 1 ? 0x3715 : 0x6240);
#pragma unroll
  for (int g = 0; g < 4; ++g) got[g] = __shfl_xor_sync(0xffffffffu, b[g], 2);
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    b[g] = __byte_perm(b[g], got[g], lane & 2 ? 0x3276 : 0x5410);
    if (row[g] >= 0) *reinterpret_cast<uint32_t*>(in_row(a, a.y + (feature - q), row[g])) = b[g];
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
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

constexpr uint64_t kMostBytes = (uint64_t)INT64_MAX / 2;

// The buckets of a product: fills their geometry and where their counts lie
// (llmoe_route's, or NULL: a buffer set's signal words); false where the
// arguments are not valid.
bool product_buckets(const int64_t* counts, const llmoe_buf_set_t* bs, ProductArgs* a) {
  if (bs == nullptr) return false;
  const int T = bs->num_max_tokens, R = bs->num_ranks, E = bs->num_experts;
  if (T < 1 || R < 1 || E < R || E % R != 0 || E > LLMOE_MAX_EXPERTS || !aligned(bs->err, 4) || !aligned(counts, 8))
    return false;
  if ((uint64_t)E * R > INT32_MAX || (uint64_t)E * R * T > INT32_MAX) return false;
  *a = ProductArgs{};
  if (counts == nullptr) {
    const size_t total = llmoe_layout_bytes_dtype(T, bs->hidden, R, E, bs->dtype);
    uint64_t sig = 0;
    if (total == 0 || bs->base == nullptr || !aligned(bs->base, 16) || bs->rank_stride % 16 != 0 ||
        bs->rank_stride < total || bs->rank_stride > kMostBytes / R ||
        llmoe_layout_offsets_dtype(T, bs->hidden, R, E, bs->dtype, bs->set, nullptr, nullptr, &sig) != LLMOE_SUCCESS ||
        sig % 8 != 0)
      return false;
    a->base = static_cast<const uint8_t*>(bs->base);
    a->rank_stride = bs->rank_stride;
    a->sig_off = sig;
  }
  a->counts = counts;
  a->err = bs->err;
  a->T = T;
  a->R = R;
  a->E = E;
  a->L = E / R;
  return true;
}

// A product's rows, x's of dtype and y's of out_dtype, for buckets that are filled in.
bool product_rows(const void* x, void* y, int in, int out, int dtype, int out_dtype, bool swiglu, ProductArgs* a) {
  const uint64_t xr = row_bytes(in, dtype), yr = row_bytes(out, out_dtype), rows = (uint64_t)a->E * a->R * a->T;
  if (xr == 0 || yr == 0 || yr > INT32_MAX || out > INT32_MAX / 2 || (swiglu && out % 8 != 0)) return false;
  if (x == nullptr || y == nullptr || !aligned(x, 16) || !aligned(y, 16)) return false;
  if (xr > kMostBytes / rows || yr > kMostBytes / rows || overlap(y, rows * yr, x, rows * xr)) return false;
  a->x = static_cast<const uint8_t*>(x);
  a->y = static_cast<uint8_t*>(y);
  a->in = in;
  a->out = out;
  a->n = out * (swiglu ? 2 : 1);
  a->x_row = xr;
  a->y_row = (uint32_t)yr;
  a->dtype = dtype;
  a->out_dtype = out_dtype;
  return true;
}

// Opts a kernel of CTA pairs in to its shared memory and asks how many pairs can
// be resident, once per device.  Asked with the most shared memory: whatever a
// call uses is more than half of an SM's, so there is one CTA on an SM in any case.
template <auto kKernel>
int resident_pairs(int threads) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
  if (dev < kMaxDevices) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * num_sms());
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = kMaxSmem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 0;
  }
  if (dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace
