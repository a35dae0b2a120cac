// Attention of every request's new rows over its paged keys and values.
//
// Three launches:
//  1. attend_prepare_kernel: the first workgroup lays out the work (below); the
//     others write the new rows' keys and values into their pages.
//  2. the product.  A unit of work is a block of rows (a row here is one query head
//     of one new token; the Hq / Hkv heads of a group and the request's new tokens
//     share their keys, so they share the block) over one request's tokens, for one
//     key-value head.  All units in a line are cut into equal shares, one per
//     workgroup and about as many as the chip holds at once, whatever the lengths.
//     A unit within one share writes its result; of one that is cut, every share
//     leaves (max, sum, sum p v).  Two kernels:
//       attend_few_kernel   up to 16 rows a block (single tokens): its four waves
//                           take the steps along the tokens in turn, each straight
//                           from memory into its products, and are joined in LDS;
//       attend_many_kernel  up to 64 rows: the waves take the rows, and each step's
//                           keys and values pass through LDS once for all of them.
//  3. attend_join_kernel joins what was cut.
//
// The products need no shuffle.  Scores are formed transposed, S^T = K Q^T, and
// the result too, O^T = V^T P^T: a lane then holds the same row of Q in S^T and in
// O^T, so maxima, sums and rescaling factors never cross lanes, and P^T leaves the
// first product in the register layout in which the second wants it.  For that the
// 32 keys of a bf16 step are entered in an order that gives a lane 8 consecutive
// ones, and values lie along the tokens in their pages, so that a lane's 8 are one
// 16-byte load.
//
// Bound: keys and values are read once from memory (2 Hkv D bytes a token for each
// of K and V); the products are 4 Hq D n operations a token, far below the matrix
// rate for the rows of a round.  Measured (128 requests of 1 to 17 new rows over up to
// 6000 tokens, 32 query and 8 key-value heads of 128, bf16, pages of 16; 1.60 GB):
// layout and append 10 us, product 325 us (4.9 TB/s), join 17 us.  256 single tokens
// over up to 4000 (2.10 GB): product 350 us (6.0 TB/s).  Three single fp32 tokens over
// up to 120000 (92 MB): 4 + 22 + 8 us.  A prompt is bound by its operations: one of
// 16000 rows takes 5.2 ms in the product, 403 TFLOP/s in bf16.
#include <limits.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kWaves = kBlock / kWave;
// Over all key-value heads: two workgroups a compute unit, as many as their registers
// and LDS allow.  Three or four would only queue (verified batch 378 and 337 us for
// 324 then, decoding 383 and 354 for 349).
constexpr int kShares = 2 * kComputeUnits;
constexpr int kCut = 128;         // a unit is cut at multiples of this many tokens
constexpr int kFixed = 64;        // a unit's fixed cost, in tokens (128 and 160: no change)
constexpr int kJoiners = 32;      // workgroups that join a request's rows, at most;
constexpr int kJoinGrid = 2048;   // more where requests are few, up to so many in all
constexpr int kAppend = 8;        // rows whose values a workgroup writes at a time
constexpr int kWindow = 1024;     // page numbers of a stretch that wait in LDS at a time
constexpr float kNone = -3e38f;   // running maximum of a row that has seen nothing
constexpr float kSlack = 8.0f;    // see weigh below

struct AttendParams {
  AttendLaunch L;
  int heads_per_group, block_rows;
  int most_shares;  // per key-value head
  // scratch
  int64_t *head;    // work units per share (tokens), of all requests
  int64_t *before;  // [R + 1] work units before each request
  int32_t *first;   // [most_shares] the request in which each share begins
  float2 *part_ml;  // [2 most_shares][Hkv][block_rows]: (max, sum)
  float *part_o;    // [2 most_shares][Hkv][block_rows][D]
};

struct Slice { int row0, n, len; };

// A request's rows and length; what is out of bounds counts as empty.
__device__ __forceinline__ Slice slice_of(const AttendLaunch &L, int r, int *bits) {
  Slice s;
  s.row0 = r;
  s.n = 1;
  if (L.row_offset != nullptr) {
    const int a = L.row_offset[r], b = L.row_offset[r + 1];
    const bool bad = a < 0 || b < a || b > L.rows_capacity;
    if (bad) *bits |= kErrLength;
    s.row0 = bad ? 0 : a;
    s.n = bad ? 0 : b - a;
  }
  s.len = L.kv_len[r];
  if (s.len < 0 || s.len > L.max_pages << L.page_shift) {
    *bits |= kErrLength;
    s.len = 0;
  }
  return s;
}

// First token that any of the request's rows sees, in whole steps of 32.
__device__ __forceinline__ int first_token(const AttendLaunch &L, const Slice &s) {
  if (L.window == 0) return 0;
  return max(0, s.len - s.n + 1 - L.window) & ~31;
}

// The units of a request: so many blocks of `size` work units each, over the tokens
// [t0, len).
struct Units { int blocks, size, t0; };
__device__ __forceinline__ Units units_of(const AttendParams &p, const Slice &s) {
  Units u;
  u.blocks = (int)(((int64_t)s.n * p.heads_per_group + p.block_rows - 1) / p.block_rows);
  u.t0 = first_token(p.L, s);
  u.size = kFixed + (s.len - u.t0);
  return u;
}
// The order of a request's units: the first block, the last, the second, ...  A block
// reads the tokens that its own rows see, so of a prompt's the first blocks are short
// and the last long, and this way a share takes as many of both (a prompt of 4000
// tokens, 32 and 8 heads of 128, bf16: 0.34 ms, 1.21 where every block passed over all
// tokens and masked).
__device__ __forceinline__ int block_at(int i, int blocks) {
  return i & 1 ? blocks - 1 - i / 2 : i / 2;
}
__device__ __forceinline__ int place_of_block(int b, int blocks) {
  return b < (blocks + 1) / 2 ? 2 * b : 2 * (blocks - 1 - b) + 1;
}
// Where a cut at `at` of a unit's `size` work units lies among its tokens.
__device__ __forceinline__ int cut_at(int64_t at, int size) {
  if (at >= size) return size - kFixed;
  return at <= kFixed ? 0 : ((int)at - kFixed) & ~(kCut - 1);
}

// Exclusive prefix over the workgroup, and the total.
__device__ __forceinline__ int64_t scan64(int64_t v, int64_t *scratch, int64_t *total) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int64_t x = __shfl_up((long long)inc, o);
    if (lane >= o) inc += x;
  }
  __syncthreads();
  if (lane == kWave - 1) scratch[w] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) before += scratch[i];
    all += scratch[i];
  }
  *total = all;
  return before + inc - v;
}

}  // namespace

// Equal shares of the units of all requests, of at least one cut.
__device__ __forceinline__ void lay_out(const AttendParams &p) {
  const AttendLaunch &L = p.L;
  __shared__ int64_t scratch[kWaves], from[kBlock];
  const int tid = threadIdx.x;
  int bits = 0;
  auto work_of = [&](int r) __attribute__((always_inline)) {
    if (r >= L.R) return (int64_t)0;
    const Units u = units_of(p, slice_of(L, r, &bits));
    return (int64_t)u.blocks * u.size;
  };
  int64_t all = 0, mine = 0;
  for (int r = tid; r < L.R; r += kBlock) mine += work_of(r);
  scan64(mine, scratch, &all);
  const int64_t even = (all + p.most_shares - 1) / p.most_shares;
  const int64_t share = even < kCut + kFixed ? kCut + kFixed : even;
  int64_t base = 0;
  for (int r0 = 0; r0 < L.R; r0 += kBlock) {
    const int r = r0 + tid;
    int64_t total;
    const int64_t at = base + scan64(work_of(r), scratch, &total);
    if (r < L.R) p.before[r] = at;
    from[tid] = at;
    __syncthreads();
    // shares that begin among these requests, by all threads: in the last request
    // that does not begin behind them
    const int here = min(L.R - r0, kBlock);
    for (int64_t i = (base + share - 1) / share + tid; i * share < base + total; i += kBlock) {
      int lo = 0;
#pragma unroll
      for (int step = kBlock / 2; step > 0; step >>= 1)
        if (lo + step < here && from[lo + step] <= i * share) lo += step;
      p.first[i] = r0 + lo;
    }
    __syncthreads();
    base += total;
  }
  if (tid == 0) {
    p.before[L.R] = all;
    p.head[0] = share;
    p.head[1] = all;
  }
  if (bits) flag_error(L.err, bits);
}

// Workgroups from 1 on: a quarter of the elements of up to kAppend rows of request
// (b - 1) % R at a time.  Values lie along the tokens, so neighbouring lanes take
// neighbouring rows: a store reaches 8 pieces of a page and not 64 (9 us for 10.5).
template <typename T>
__global__ __launch_bounds__(kBlock) void attend_prepare_kernel(AttendParams p) {
  if (blockIdx.x == 0) {
    lay_out(p);
    return;
  }
  const AttendLaunch &L = p.L;
  constexpr int kPer = Elem<T>::kPerVec;
  int bits = 0;
  const int b = blockIdx.x - 1, r = b % L.R, part = b / L.R / 4, parts = (gridDim.x - 1) / L.R / 4;
  const Slice s = slice_of(L, r, &bits);
  const int page_mask = (1 << L.page_shift) - 1;
  const int elems = L.Hkv * L.D / 4, e0 = b / L.R % 4 * elems;  // a multiple of 8
  bits = 0;  // the layout reports the slices
  // the page of row j, null where it is not to be written
  auto page_of = [&](int j, void *pages, int64_t stride) __attribute__((always_inline)) {
    const int t = s.len - s.n + j;
    const int id = t < 0 ? -1 : L.table[(int64_t)r * L.max_pages + (t >> L.page_shift)];
    if (t < 0) bits |= kErrLength;
    else if ((unsigned)id >= (unsigned)L.n_pages) bits |= kErrPage;
    return (unsigned)id < (unsigned)L.n_pages ? reinterpret_cast<T *>(pages) + (int64_t)id * stride
                                              : (T *)nullptr;
  };
  for (int j0 = part * kAppend; j0 < s.n; j0 += parts * kAppend) {
    const int rows = min(kAppend, s.n - j0);
    // keys: rows of D elements
    const int pieces = elems / kPer;
    for (int i = threadIdx.x; i < rows * pieces; i += kBlock) {
      const int j = j0 + i / pieces, e = e0 + i % pieces * kPer, h = e / L.D;
      T *page = page_of(j, L.k_pages, L.k_page_stride);
      if (page == nullptr) continue;
      const int slot = (s.len - s.n + j) & page_mask;
      const T *from = reinterpret_cast<const T *>(L.k_new) + (int64_t)(s.row0 + j) * L.kv_stride + e;
      *reinterpret_cast<u32x4 *>(page + (((int64_t)h << L.page_shift) + slot) * L.D + e - h * L.D) =
          *reinterpret_cast<const u32x4 *>(from);
    }
    // values: `lanes` neighbours take as many rows
    const int shift = rows > 4 ? 3 : rows > 2 ? 2 : rows > 1 ? 1 : 0;
    const int mine = threadIdx.x & ((1 << shift) - 1);
    if (mine < rows) {
      const int j = j0 + mine, slot = (s.len - s.n + j) & page_mask;
      T *page = page_of(j, L.v_pages, L.v_page_stride);
      const T *from = reinterpret_cast<const T *>(L.v_new) + (int64_t)(s.row0 + j) * L.kv_stride;
      if (page != nullptr) {
#pragma unroll 8
        for (int e = e0 + (threadIdx.x >> shift); e < e0 + elems; e += kBlock >> shift)
          page[((int64_t)e << L.page_shift) + slot] = from[e];
      }
    }
  }
  if (bits) flag_error(L.err, bits);
}

namespace {

// 16 bytes of keys or values.  A step reads 64 bytes of each of its rows of values.
// Where that is the whole row of a page, the step's lines are its own and pass the
// caches by (decoding 256 requests of up to 4000 tokens, pages of 16: 350 us, 381
// through the caches); where rows are longer, another wave wants the line's other
// half a moment later (pages of 64: 363 us through the caches, 414 past them).
template <bool kPast> __device__ __forceinline__ u32x4 ld_cache(const void *p) {
  if constexpr (kPast) return ld_stream4(p);
  else return *reinterpret_cast<const u32x4 *>(p);
}
// The matrix products of one step.  Lane l: column c = l % 16 of a 16-row tile of
// Q, group g = l / 16.  S^T tile: register i of the lane is key 4 g + i of the
// tile.  bf16: two tiles of 16 keys, entered so that the lane's two quads are the
// 8 consecutive keys 8 g..8 g + 7 of the step: tile t, matrix row m is key
// 8 (m / 4) + 4 t + m % 4.  fp32: one tile of 16 keys, the lane has 4 g..4 g + 3.
template <typename T> struct Step;

template <> struct Step<bf16_t> {
  static constexpr int kKeys = 32, kTiles = 2, kMine = 8;  // keys of a step, tiles, keys of a lane
  __device__ static __forceinline__ int key_of_row(int m, int t) {
    return 8 * (m >> 2) + 4 * t + (m & 3);
  }
  template <int D> struct K { u32x4 v[2][D / 32]; };
  template <int D> struct V { u32x4 v[D / 16]; };
  template <int D> struct Q { u32x4 v[D / 32]; };
  // key row `k` (this lane's), element order: contraction index 32 s + 8 g + e
  template <bool kPast, int D>
  __device__ static __forceinline__ void load_k(const bf16_t *k, int t, int g, K<D> &o) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) o.v[t][s] = ld_cache<kPast>(k + 32 * s + 8 * g);
  }
  template <int D>
  __device__ static __forceinline__ void load_q(const bf16_t *q, int g, Q<D> &o) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) o.v[s] = *reinterpret_cast<const u32x4 *>(q + 32 * s + 8 * g);
  }
  template <int D>
  __device__ static __forceinline__ floatx4 scores(const K<D> &k, int t, const Q<D> &q) {
    floatx4 a = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k.v[t][s]),
                                                  __builtin_bit_cast(bf16x8, q.v[s]), a, 0, 0, 0);
    return a;
  }
  // Probabilities as a bf16 and the bf16 of what it leaves: one rounding to 8
  // bits would be the largest error of the whole pass (as large as the rounding
  // of the result), and the matrix cores have room for the second product.
  struct P { bf16x8 hi, lo; };
  __device__ static __forceinline__ P pack(const float *p) {
    P o;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o.hi[i] = (__bf16)p[i];
      o.lo[i] = (__bf16)(p[i] - (float)o.hi[i]);
    }
    return o;
  }
  __device__ static __forceinline__ floatx4 product(const u32x4 &v, const P &p, floatx4 a) {
    const bf16x8 x = __builtin_bit_cast(bf16x8, v);
    a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, p.lo, a, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, p.hi, a, 0, 0, 0);
  }
  // v with the tokens behind the first `n` of its 8 (and before `from`) zeroed
  __device__ static __forceinline__ u32x4 keep(u32x4 v, int from, int n) {
    u16x8 x = __builtin_bit_cast(u16x8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i >= from && i < n ? x[i] : (uint16_t)0;
    return __builtin_bit_cast(u32x4, x);
  }
  __device__ static __forceinline__ bool not_finite(u32x4 v) {
    const u16x8 x = __builtin_bit_cast(u16x8, v);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) bad = bad || (x[i] & 0x7F80) == 0x7F80;
    return bad;
  }
};

template <> struct Step<float> {
  static constexpr int kKeys = 16, kTiles = 1, kMine = 4;
  __device__ static __forceinline__ int key_of_row(int m, int t) { return m; }
  template <int D> struct K { u32x4 v[1][D / 16]; };
  template <int D> struct V { u32x4 v[D / 16]; };
  template <int D> struct Q { u32x4 v[D / 16]; };
  // element order: product 4 s + e takes contraction index 16 s + 4 g + e
  template <bool kPast, int D>
  __device__ static __forceinline__ void load_k(const float *k, int t, int g, K<D> &o) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) o.v[t][s] = ld_cache<kPast>(k + 16 * s + 4 * g);
  }
  template <int D>
  __device__ static __forceinline__ void load_q(const float *q, int g, Q<D> &o) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) o.v[s] = *reinterpret_cast<const u32x4 *>(q + 16 * s + 4 * g);
  }
  template <int D>
  __device__ static __forceinline__ floatx4 scores(const K<D> &k, int t, const Q<D> &q) {
    floatx4 a = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        a = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k.v[t][s][e]),
                                                 __uint_as_float(q.v[s][e]), a, 0, 0, 0);
    return a;
  }
  struct P { floatx4 v; };
  __device__ static __forceinline__ P pack(const float *p) {
    P o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = p[i];
    return o;
  }
  __device__ static __forceinline__ floatx4 product(const u32x4 &v, const P &p, floatx4 a) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      a = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[e]), p.v[e], a, 0, 0, 0);
    return a;
  }
  __device__ static __forceinline__ u32x4 keep(u32x4 v, int from, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i >= from && i < n ? v[i] : 0u;
    return v;
  }
  __device__ static __forceinline__ bool not_finite(u32x4 v) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad = bad || (v[i] & 0x7F800000u) == 0x7F800000u;
    return bad;
  }
};

__device__ __forceinline__ void store4(float *p, const float *v) {
  *reinterpret_cast<floatx4 *>(p) = floatx4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store4(bf16_t *p, const float *v) {
  const uint32_t a = f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16;
  const uint32_t b = f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16;
  *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
}

}  // namespace

namespace {

template <int N> struct Count { static constexpr int value = N; };

// Where the window of page numbers that begins with token w0 ends: at a page's end,
// for w0 may lie inside one.
__device__ __forceinline__ int window_end(const AttendLaunch &L, int w0, int end) {
  return min(end, ((w0 >> L.page_shift) + kWindow) << L.page_shift);
}

// The page numbers of tokens [begin, end) to LDS (-1 where there is no such page);
// returns whether one is missing.  From LDS, because loads come back in order: a
// number read from memory would be waited for behind every key in flight.
__device__ __forceinline__ bool stage_ids(const AttendLaunch &L, const int32_t *table, int begin, int end,
                                          int32_t *ids) {
  bool bad = false;
  const int first = begin >> L.page_shift, n = ((end - 1) >> L.page_shift) - first + 1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kBlock) {
    const int id = table[first + i];
    const bool there = (unsigned)id < (unsigned)L.n_pages;
    ids[i] = there ? id : -1;
    bad = bad || !there;
  }
  return __syncthreads_or(bad);
}

// A share's stretches, one after the other.
struct Stretch {
  Slice sl;
  int r, block_row, rows, begin, end;
  int slot;  // where its part goes, -1: the unit is whole
};
struct Share {
  int64_t at, end;
  int r, index;
};
__device__ __forceinline__ bool share_of(const AttendParams &p, int index, Share *s) {
  s->index = index;
  s->at = index * p.head[0];
  s->end = min(s->at + p.head[0], p.head[1]);
  if (s->at >= s->end) return false;
  s->r = p.first[index];
  return true;
}
__device__ __forceinline__ bool next_stretch(const AttendParams &p, Share *s, Stretch *o) {
  if (s->at >= s->end) return false;
  while (s->at >= p.before[s->r + 1]) ++s->r;  // requests without rows have no units
  int bits = 0;
  o->r = s->r;
  o->sl = slice_of(p.L, s->r, &bits);
  const Units u = units_of(p, o->sl);
  const int64_t rel = s->at - p.before[s->r];
  const int i = (int)(rel / u.size);
  const int64_t x = rel - (int64_t)i * u.size, x1 = min((int64_t)u.size, x + (s->end - s->at));
  o->block_row = block_at(i, u.blocks) * p.block_rows;
  o->rows = min(p.block_rows, o->sl.n * p.heads_per_group - o->block_row);
  // of these tokens, those that some row of the block sees
  const int past = o->sl.len - o->sl.n + 1;
  const int high = max(0, past + (o->block_row + o->rows - 1) / p.heads_per_group);
  const int low = p.L.window > 0 ? max(0, past + o->block_row / p.heads_per_group - p.L.window) & ~31 : 0;
  o->begin = max(u.t0 + cut_at(x, u.size), low);
  o->end = min(u.t0 + cut_at(x1, u.size), high);
  // a share has at most one part that begins within a unit and one that ends within
  o->slot = x > 0 ? 2 * s->index : x1 < u.size ? 2 * s->index + 1 : -1;
  s->at += x1 - x;
  return true;
}

// One row (of Q) of a 16-row tile as a lane holds it: the tokens that it sees,
// [low, high), the subtrahend m and its lane's share of the sum.
struct RowState {
  int low, high;
  float m, l;
};

// Row `row` of the item's `rows` (block_row on): what it sees and its query.
template <typename T, int D>
__device__ __forceinline__ RowState row_state(const AttendParams &p, const Slice &sl, int block_row,
                                              int row, int rows, int hk, int g,
                                              typename Step<T>::template Q<D> &q) {
  const AttendLaunch &L = p.L;
  RowState s{0, 0, kNone, 0.0f};
#pragma unroll
  for (unsigned i = 0; i < sizeof(q.v) / 16; ++i) q.v[i] = u32x4{0, 0, 0, 0};
  if (row < rows) {
    const int group = p.heads_per_group, j = (block_row + row) / group, h = (block_row + row) % group;
    s.high = max(0, sl.len - sl.n + 1 + j);
    s.low = L.window > 0 ? max(0, s.high - L.window) : 0;
    Step<T>::template load_q<D>(reinterpret_cast<const T *>(L.q) + (int64_t)(sl.row0 + j) * L.q_stride +
                                    (int64_t)(hk * group + h) * D,
                                g, q);
  }
  return s;
}

// Masks a lane's scores of the tokens from t0 on.
template <int kMine>
__device__ __forceinline__ void mask_scores(float *s, const RowState &r, int t0, bool bad) {
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (bad || t0 + i < r.low || t0 + i >= r.high) s[i] = -INFINITY;
}

// Scores to probabilities against the row's subtrahend.  That follows the running
// maximum only when it is kSlack (a factor 2^8) behind: below that the sums just
// grow, and what is summed so far needs no rescaling.  The lanes of a row (16, 32
// and 48 apart) agree on it.  The difference is formed before the factor: a fused
// s to_log2 - m would leave the rounding of m, and beyond 2^30 that is an exponent.
template <typename T, int kOut>
__device__ __forceinline__ typename Step<T>::P weigh(float *s, float to_log2, RowState &r,
                                                     floatx4 (&o)[kOut]) {
  constexpr int kMine = Step<T>::kMine;
  float top = s[0];
#pragma unroll
  for (int i = 1; i < kMine; ++i) top = fmaxf(top, s[i]);
  if (__ballot((top - r.m) * to_log2 > kSlack) != 0) {
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float now = fmaxf(r.m, top), f = exp2_fast((r.m - now) * to_log2);
    r.m = now;
    r.l *= f;
#pragma unroll
    for (int d = 0; d < kOut; ++d) o[d] *= f;
  }
  float e[kMine], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    e[i] = exp2_fast((s[i] - r.m) * to_log2);
    sum += e[i];
  }
  r.l += sum;
  return Step<T>::pack(e);
}

// The product row by row, with the values that the row does not see zeroed:
// where a value that some of the rows see is not finite.
template <typename T>
__device__ __forceinline__ floatx4 product_mixed(const u32x4 &v, const typename Step<T>::P &pr,
                                                 const RowState &r, int t0, floatx4 o) {
  const int col = threadIdx.x & 15;
#pragma nounroll
  for (int c = 0; c < 16; ++c) {
    const int from = __shfl(r.low, c) - t0, to = __shfl(r.high, c) - t0;
    const floatx4 a = Step<T>::product(Step<T>::keep(v, from, to), pr, o);
    if (col == c) o = a;
  }
  return o;
}

// Four elements from d on of a row's result: the stretch's share, or the result.
template <typename T>
__device__ __forceinline__ void write_row(const AttendParams &p, const Slice &sl, int hk, int slot,
                                          int block_row, int row, int d, float m, float sum,
                                          const float *x) {
  const AttendLaunch &L = p.L;
  if (slot >= 0) {
    const int64_t at = ((int64_t)slot * L.Hkv + hk) * p.block_rows + row;
    store4(p.part_o + at * L.D + d, x);
    if (d == 0) p.part_ml[at] = make_float2(m, sum);
    return;
  }
  const float inv = sum > 0.0f ? 1.0f / sum : sum;  // nothing seen: 0; NaN stays
  const float y[4] = {x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv};
  const int group = p.heads_per_group;
  const int j = (block_row + row) / group, h = hk * group + (block_row + row) % group;
  const int64_t out_row = (int64_t)(sl.row0 + j) * L.Hq + h;
  store4(reinterpret_cast<T *>(L.out) + out_row * L.D + d, y);
  if (d == 0 && L.lse != nullptr)
    L.lse[out_row] = sum == 0.0f ? -INFINITY : fmaf(m, L.scale, logf(sum));
}

}  // namespace

// Up to 16 rows, each wave its own steps: nothing passes through LDS but page numbers
// and the joining of the waves, so the loads are bound by memory alone (6.0 TB/s with
// two steps of 16 KB in flight a wave).
template <typename T, int D, bool kPast>
__global__ __launch_bounds__(kBlock, D <= 128 ? 2 : 1) void attend_few_kernel(AttendParams p) {
  using St = Step<T>;
  constexpr int kKeys = St::kKeys, kMine = St::kMine, kTiles = St::kTiles;
  constexpr int kOut = D / 16;      // 16-wide tiles of the result
  constexpr int kPitch = D + 4;     // of a row in LDS, floats
  // two steps' keys and values (D / 2 registers each) beside the result and queries
  constexpr bool kAhead = D <= 128;
  __shared__ float lds_o[kWaves][16][kPitch];
  __shared__ float2 lds_ml[kWaves][16];
  __shared__ int32_t ids[kWindow];
  const AttendLaunch &L = p.L;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  const int group = p.heads_per_group;
  const float to_log2 = L.scale * kLog2e;
  const int page_mask = (1 << L.page_shift) - 1;

  const int hk = blockIdx.x % L.Hkv;
  Share share;
  if (!share_of(p, blockIdx.x / L.Hkv, &share)) return;
  Stretch st;
  while (next_stretch(p, &share, &st)) {
    const Slice &sl = st.sl;
    const int block_row = st.block_row, rows = st.rows, begin = st.begin, end = st.end, slot = st.slot;
    int bits = 0;
    const int32_t *table = L.table + (int64_t)st.r * L.max_pages;
    typename St::template Q<D> q;
    RowState row = row_state<T, D>(p, sl, block_row, col, rows, hk, g, q);
    // tokens before most_low or from least_high on are hidden from some row
    const int first_j = block_row / group, last_j = (block_row + rows - 1) / group;
    const int least_high = max(0, sl.len - sl.n + 1 + first_j);
    const int most_low = L.window > 0 ? sl.len - sl.n + 1 + last_j - L.window : 0;
    floatx4 o[kOut];
#pragma unroll
    for (int d = 0; d < kOut; ++d) o[d] = floatx4{0, 0, 0, 0};

    struct Data {
      typename St::template K<D> k;
      typename St::template V<D> v;
    };
    const T *kbase = reinterpret_cast<const T *>(L.k_pages) + ((int64_t)hk << L.page_shift) * D;
    const T *vbase = reinterpret_cast<const T *>(L.v_pages) + ((int64_t)hk * D << L.page_shift);
    const int stride = kWaves * kKeys;
    for (int w0 = begin, w1; w0 < end; w0 = w1) {
      w1 = window_end(L, w0, end);
      const bool any_bad = stage_ids(L, table, w0, w1, ids);
      const int first_page = w0 >> L.page_shift;
      // loads of the step at token t; tokens past the last read the last page again
      auto load = [&](int t, Data &x) __attribute__((always_inline)) {
        const int tk = t + St::key_of_row(col, 0), tv = t + kMine * g;
        const int ik = max(0, ids[(min(tk, w1 - 1) >> L.page_shift) - first_page]);
        const int iv = max(0, ids[(min(tv, w1 - 1) >> L.page_shift) - first_page]);
        const T *k = kbase + (int64_t)ik * L.k_page_stride;
        const T *v = vbase + (int64_t)iv * L.v_page_stride + (tv & page_mask) + (col << L.page_shift);
#pragma unroll
        for (int s = 0; s < kTiles; ++s)
          St::template load_k<kPast, D>(k + ((t + St::key_of_row(col, s)) & page_mask) * D, s, g, x.k);
#pragma unroll
        for (int d = 0; d < kOut; ++d) x.v.v[d] = ld_cache<kPast>(v + (16 * d << L.page_shift));
      };
      auto compute = [&](int t, Data &x) __attribute__((always_inline)) {
        const int t0 = t + kMine * g;  // this lane's first token
        const bool edge = any_bad || t + kKeys > least_high || t < most_low;  // uniform
        float s[kMine];
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          const floatx4 a = St::template scores<D>(x.k, u, q);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[4 * u + i] = a[i];
        }
        bool mixed = false;
        if (edge) {
          const bool bad = any_bad && ids[(min(t0, w1 - 1) >> L.page_shift) - first_page] < 0;
          if (bad) bits |= kErrPage;
          mask_scores<kMine>(s, row, t0, bad);
          bool odd = false;
#pragma unroll
          for (int d = 0; d < kOut; ++d) {
            x.v.v[d] = St::keep(x.v.v[d], 0, bad ? 0 : end - t0);
            odd = odd || St::not_finite(x.v.v[d]);
          }
          mixed = __ballot(odd) != 0;
        }
        const typename St::P pr = weigh<T, kOut>(s, to_log2, row, o);
        if (!mixed) {
#pragma unroll
          for (int d = 0; d < kOut; ++d) o[d] = St::product(x.v.v[d], pr, o[d]);
        } else {
#pragma unroll
          for (int d = 0; d < kOut; ++d) o[d] = product_mixed<T>(x.v.v[d], pr, row, t0, o[d]);
        }
      };

      // every wave its steps; where registers allow, the next one's loads are in
      // flight during this one's products
      int t = w0 + wave * kKeys;
      Data a;
      if constexpr (!kAhead) {
        for (; t < w1; t += stride) {
          load(t, a);
          compute(t, a);
        }
      } else if (t < w1) {
        Data b;
        load(t, a);
        for (;;) {
          const bool more = t + stride < w1;
          if (more) load(t + stride, b);
          compute(t, a);
          t += stride;
          if (!more) break;
          const bool again = t + stride < w1;
          if (again) load(t + stride, a);
          compute(t, b);
          t += stride;
          if (!again) break;
        }
      }
    }
    if (bits) flag_error(L.err, bits);

    // join the waves
    float sum = row.l;
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    __syncthreads();
    if (g == 0) lds_ml[wave][col] = make_float2(row.m, sum);
#pragma unroll
    for (int d = 0; d < kOut; ++d)
      *reinterpret_cast<floatx4 *>(&lds_o[wave][col][16 * d + 4 * g]) = o[d];
    __syncthreads();
    // 4 elements a thread at a time
    for (int i = threadIdx.x; i < rows * (D / 4); i += kBlock) {
      const int c = i / (D / 4), d = i % (D / 4) * 4;
      float mx = kNone;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) mx = fmaxf(mx, lds_ml[v][c].x);
      float all = 0.0f, x[4] = {0, 0, 0, 0};
#pragma unroll
      for (int v = 0; v < kWaves; ++v) {
        const float f = exp2_fast((lds_ml[v][c].x - mx) * to_log2);
        all += f * lds_ml[v][c].y;
        const floatx4 y = *reinterpret_cast<const floatx4 *>(&lds_o[v][c][d]);
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] += f * y[k];
      }
      write_row<T>(p, sl, hk, slot, block_row, c, d, mx, all, x);
    }
  }
}

// 16 rows a wave.  A step's keys and values are D / 8 pieces of 64 x 16 bytes, each
// an operand of the matrix cores in lane order: waves 0 and 1 fetch the keys', 2 and
// 3 the values', kDeep steps ahead in registers, and pass them on through two buffers
// in LDS of kGroup steps each.  In lane order every LDS access is 1 KB in a row; one
// barrier a buffer (timed in turn, two steps a barrier and one copy of the step's code
// took 317 us, one step and two copies 325).  64 rows: with 128, two tiles a wave, the results spill in the
// 256 registers that two workgroups a unit leave (verified batch 1207 us).
template <typename T, int D, bool kPast>
__global__ __launch_bounds__(kBlock, D <= 128 ? 2 : 1) void attend_many_kernel(AttendParams p) {
  using St = Step<T>;
  constexpr int kKeys = St::kKeys, kMine = St::kMine, kTiles = St::kTiles;
  constexpr int kOut = D / 16;
  constexpr int kPieces = D / 8, kFetch = kPieces / kWaves;  // of a step; of a wave
  constexpr int kGroup = D <= 128 ? 2 : 1, kDeep = 2;
  __shared__ u32x4 ring[2][kGroup][kPieces][kWave];
  __shared__ int32_t ids[kWindow];
  const AttendLaunch &L = p.L;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  const int group = p.heads_per_group;
  const float to_log2 = L.scale * kLog2e;
  const int page_mask = (1 << L.page_shift) - 1;
  const bool keys = wave < 2;  // what this wave fetches

  const int hk = blockIdx.x % L.Hkv;
  Share share;
  if (!share_of(p, blockIdx.x / L.Hkv, &share)) return;
  Stretch st;
  while (next_stretch(p, &share, &st)) {
    const Slice &sl = st.sl;
    const int block_row = st.block_row, rows = st.rows, begin = st.begin, end = st.end, slot = st.slot;
    int bits = 0;
    const int32_t *table = L.table + (int64_t)st.r * L.max_pages;
    typename St::template Q<D> q;
    RowState row = row_state<T, D>(p, sl, block_row, 16 * wave + col, rows, hk, g, q);
    floatx4 o[kOut];
#pragma unroll
    for (int d = 0; d < kOut; ++d) o[d] = floatx4{0, 0, 0, 0};
    const int first_j = block_row / group, last_j = (block_row + rows - 1) / group;
    const int least_high = max(0, sl.len - sl.n + 1 + first_j);
    const int most_low = L.window > 0 ? sl.len - sl.n + 1 + last_j - L.window : 0;

    // The lane's address within a page (element), and its token within a step:
    // keys: pieces [wave kFetch, ..) of the step's kTiles key tiles.
    const int tile = kTiles == 2 ? (wave & 1) : 0;
    const int s0 = kTiles == 2 ? 0 : (wave & 1) * kFetch;  // first piece of the tile
    const int my_token = keys ? St::key_of_row(col, tile) : kMine * g;
    const T *base = keys ? reinterpret_cast<const T *>(L.k_pages) + ((int64_t)hk << L.page_shift) * D +
                               4 * kMine * s0 + kMine * g
                         : reinterpret_cast<const T *>(L.v_pages) +
                               (((int64_t)hk * D + (wave - 2) * kFetch * 16 + col) << L.page_shift);
    const int64_t page_stride = keys ? L.k_page_stride : L.v_page_stride;
    const int piece_step = keys ? 4 * kMine : 16 << L.page_shift;  // elements from piece to piece
    const int slot_step = keys ? D : 1;
    for (int w0 = begin, w1; w0 < end; w0 = w1) {
      w1 = window_end(L, w0, end);
      const bool any_bad = stage_ids(L, table, w0, w1, ids);
      const int first_page = w0 >> L.page_shift;
      // tokens past the last read the last page again
      auto fetch = [&](int t, u32x4 (&x)[kFetch]) __attribute__((always_inline)) {
        const int id = max(0, ids[(min(t + my_token, w1 - 1) >> L.page_shift) - first_page]);
        const T *at = base + (int64_t)id * page_stride + ((t + my_token) & page_mask) * slot_step;
#pragma unroll
        for (int i = 0; i < kFetch; ++i) x[i] = ld_cache<kPast>(at + i * piece_step);
      };
      u32x4 ahead[kDeep][kFetch];
#pragma unroll
      for (int i = 0; i < kDeep; ++i)
        if (w0 + i * kKeys < w1) fetch(w0 + i * kKeys, ahead[i]);
      int buf = 0;
      for (int t1 = w0; t1 < w1; t1 += kDeep * kKeys) {
#pragma unroll
        for (int i0 = 0; i0 < kDeep; i0 += kGroup) {
          if (t1 + i0 * kKeys >= w1) break;  // uniform
#pragma unroll
          for (int i = i0; i < i0 + kGroup; ++i) {
            const int t = t1 + i * kKeys;
            if (t < w1) {
#pragma unroll
              for (int f = 0; f < kFetch; ++f) ring[buf][i - i0][wave * kFetch + f][lane] = ahead[i][f];
              if (t + kDeep * kKeys < w1) fetch(t + kDeep * kKeys, ahead[i]);
            }
          }
          // the steps' pieces are in LDS; the buffer written next was last read
          // before this barrier
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
          u32x4(*const here)[kPieces][kWave] = ring[buf];
          buf ^= 1;
          if (16 * wave >= rows) continue;  // no rows of this wave
          // one copy of the step for all of them: the kernel has to stay in the
          // instruction cache
#pragma nounroll
          for (int i = 0; i < kGroup; ++i) {
            const int t = t1 + (i0 + i) * kKeys, t0 = t + kMine * g;
            if (t >= w1) break;
            u32x4(*const to)[kWave] = here[i];
            const bool edge = any_bad || t + kKeys > least_high || t < most_low;  // uniform
            float s[kMine];
            {
              typename St::template K<D> k;
#pragma unroll
              for (int u = 0; u < kTiles; ++u)
#pragma unroll
                for (int f = 0; f < kOut / kTiles; ++f) k.v[u][f] = to[u * (kOut / kTiles) + f][lane];
#pragma unroll
              for (int u = 0; u < kTiles; ++u) {
                const floatx4 a = St::template scores<D>(k, u, q);
#pragma unroll
                for (int e = 0; e < 4; ++e) s[4 * u + e] = a[e];
              }
            }
            int seen = kMine;  // this lane's tokens whose values count
            if (edge) {
              const bool bad = any_bad && ids[(min(t0, w1 - 1) >> L.page_shift) - first_page] < 0;
              if (bad) bits |= kErrPage;
              mask_scores<kMine>(s, row, t0, bad);
              seen = bad ? 0 : end - t0;
            }
            const typename St::P pr = weigh<T, kOut>(s, to_log2, row, o);
            if (!edge) {
#pragma unroll
              for (int d = 0; d < kOut; ++d) o[d] = St::product(to[kOut + d][lane], pr, o[d]);
            } else {
#pragma unroll
              for (int d = 0; d < kOut; ++d) {
                const u32x4 v = St::keep(to[kOut + d][lane], 0, seen);
                if (__ballot(St::not_finite(v)) == 0) o[d] = St::product(v, pr, o[d]);
                else o[d] = product_mixed<T>(v, pr, row, t0, o[d]);
              }
            }
          }
        }
      }
    }
    if (bits) flag_error(L.err, bits);
    const int c = 16 * wave + col;
    float sum = row.l;
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (c < rows) {
#pragma unroll
      for (int d = 0; d < kOut; ++d) {
        const float x[4] = {o[d][0], o[d][1], o[d][2], o[d][3]};
        write_row<T>(p, sl, hk, slot, block_row, c, 16 * d + 4 * g, row.m, sum, x);
      }
    }
    __syncthreads();  // the ring is free for the next item
  }
}

// The parts of the rows of units that were cut.  A row's part takes D / 4 lanes, so a
// wave has 256 / D sides (two for D = 96), each with four or eight parts in flight.
// Where a row has few parts every side takes a row of its own; where it may have
// many, the workgroup's sides share one and are joined at the end (verified batch: 17
// us, 24 with a workgroup a row throughout).
template <typename T, int D>
__global__ __launch_bounds__(kBlock) void attend_join_kernel(AttendParams p) {
  constexpr int kLanes = D / 4, kSide = kWave / kLanes, kSides = kWaves * kSide;
  __shared__ float lds_x[kSides][D];
  __shared__ float2 lds_ml[kSides];
  const AttendLaunch &L = p.L;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = blockIdx.x;
  int bits = 0;
  const float to_log2 = L.scale * kLog2e;
  const Slice s = slice_of(L, r, &bits);
  const Units u = units_of(p, s);
  const int64_t share = p.head[0], at0 = p.before[r];
  if (u.blocks == 0 || at0 / share == (at0 + (int64_t)u.blocks * u.size - 1) / share) return;
  const int group = p.heads_per_group;
  const bool many = u.size / share + 2 > 8;  // parts of a unit, at most
  const int at_once = many ? 1 : kSides;     // rows
  const bool idle = lane / kLanes >= kSide;  // the last 16 lanes for D = 96
  const int side = wave * kSide + (idle ? 0 : lane / kLanes), d = lane % kLanes * 4;
  const int first = many ? side : 0, stride = many ? kSides : 1;
  int unit = -1, s0 = 0, splits = 0;
  for (int i0 = blockIdx.y * at_once; i0 < s.n * L.Hq; i0 += gridDim.y * at_once) {
    const int i = i0 + (many ? 0 : side);
    const bool there = i < s.n * L.Hq && !idle;
    const int j = there ? i / L.Hq : 0, h = there ? i % L.Hq : 0, hk = h / group;
    const int row = j * group + h % group, b = row / p.block_rows;
    if (b != unit) {  // most rows follow one of the same unit
      unit = b;
      const int64_t at = at0 + (int64_t)place_of_block(b, u.blocks) * u.size;
      s0 = (int)(at / share);
      splits = (int)((at + u.size - 1) / share) - s0 + 1;
    }
    // part k: what share s0 + k left, the first of them as its last
    const int64_t slot_size = (int64_t)L.Hkv * p.block_rows;
    const int64_t base = (int64_t)hk * p.block_rows + row % p.block_rows;
    float m = kNone, all = 0.0f, x[4] = {0, 0, 0, 0};
    auto take = [&](int k0, auto batch) __attribute__((always_inline)) {
      constexpr int kBatch = decltype(batch)::value;
      float2 ml[kBatch];
      floatx4 y[kBatch];
#pragma unroll
      for (int v = 0; v < kBatch; ++v) {
        const int k = min(k0 + v * stride, splits - 1);
        const int64_t at = base + (2 * (int64_t)(s0 + k) + (k == 0)) * slot_size;
        ml[v] = p.part_ml[at];
        y[v] = *reinterpret_cast<const floatx4 *>(p.part_o + at * D + d);
      }
      float now = m;
#pragma unroll
      for (int v = 0; v < kBatch; ++v) now = fmaxf(now, ml[v].x);  // a part twice does no harm here
      const float old = exp2_fast((m - now) * to_log2);
      m = now;
      all *= old;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] *= old;
#pragma unroll
      for (int v = 0; v < kBatch; ++v) {
        if (k0 + v * stride < splits) {
          const float f = exp2_fast((ml[v].x - m) * to_log2);
          all += f * ml[v].y;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += f * y[v][e];
        }
      }
    };
    if (there && splits > 1) {
      if (many)
        for (int k0 = first; k0 < splits; k0 += 8 * stride) take(k0, Count<8>{});
      else
        for (int k0 = 0; k0 < splits; k0 += 4) take(k0, Count<4>{});
    }
    if (many) {  // uniform
      __syncthreads();
      if (!idle) store4(&lds_x[side][d], x);
      if (!idle && d == 0) lds_ml[side] = make_float2(m, all);
      __syncthreads();
      m = kNone;
#pragma unroll
      for (int v = 0; v < kSides; ++v) m = fmaxf(m, lds_ml[v].x);
      all = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = 0.0f;
#pragma unroll
      for (int v = 0; v < kSides; ++v) {
        const float f = exp2_fast((lds_ml[v].x - m) * to_log2);
        all += f * lds_ml[v].y;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += f * lds_x[v][d + e];
      }
    }
    if (there && splits > 1 && (!many || side == 0)) {
      const int rr = row % p.block_rows;
      write_row<T>(p, s, hk, -1, row - rr, rr, d, m, all, x);
    }
  }
}

// ------------------------------------------------------------------- launch
namespace {

// Rows of a block.  Up to 16 rows a request on the mean (single tokens): 16, and
// the waves share the tokens.  Beyond: 64, 16 a wave.
int rows_of_block(int R, int rows_capacity, int group) {
  return (int64_t)rows_capacity * group <= (int64_t)16 * R ? 16 : 64;
}

struct Sizes {
  int block_rows, shares;
};
Sizes sizes_of(int R, int rows_capacity, int Hq, int Hkv, int D) {
  return {rows_of_block(R, rows_capacity, Hq / Hkv), (kShares + Hkv - 1) / Hkv};
}

template <typename T, int D, bool kPast>
void launch_rows(const AttendParams &p, int grid, hipStream_t stream) {
  if (p.block_rows == 16)
    DSPARK_LAUNCH("attend_few", stream, (attend_few_kernel<T, D, kPast>), grid, kBlock, p);
  else
    DSPARK_LAUNCH("attend_many", stream, (attend_many_kernel<T, D, kPast>), grid, kBlock, p);
}
template <typename T, int D>
void launch_product(const AttendParams &p, int grid, dim3 join_grid, hipStream_t stream) {
  // whether a step's 64 bytes are a page's whole row of values (see ld_cache)
  if ((sizeof(T) << p.L.page_shift) <= 64) launch_rows<T, D, true>(p, grid, stream);
  else launch_rows<T, D, false>(p, grid, stream);
  DSPARK_LAUNCH("attend_join", stream, (attend_join_kernel<T, D>), join_grid, kBlock, p);
}

template <typename T> hipError_t launch_attend_t(const AttendLaunch &L, hipStream_t stream) {
  const Sizes z = sizes_of(L.R, L.rows_capacity, L.Hq, L.Hkv, L.D);
  AttendParams p{};
  p.L = L;
  p.heads_per_group = L.Hq / L.Hkv;
  p.block_rows = z.block_rows;
  p.most_shares = z.shares;
  char *at = (char *)L.scratch;
  auto take = [&](size_t bytes) { char *c = at; at += ws_align(bytes); return c; };
  const size_t parts = (size_t)2 * z.shares * L.Hkv * z.block_rows;
  p.head = (int64_t *)take(256);
  p.before = (int64_t *)take(((size_t)L.R + 1) * 8);
  p.first = (int32_t *)take((size_t)z.shares * 4);
  p.part_ml = (float2 *)take(parts * 8);
  p.part_o = (float *)take(parts * L.D * 4);
  // four workgroups for every kAppend rows of the mean request
  const int64_t mean = (L.rows_capacity + L.R - 1) / L.R, sets = (mean + kAppend - 1) / kAppend;
  const int appenders = L.k_new == nullptr ? 0 : 4 * (int)(sets < 64 ? sets : 64);
  DSPARK_LAUNCH("attend_prepare", stream, attend_prepare_kernel<T>, 1 + L.R * appenders, kBlock, p);
  const int grid = z.shares * L.Hkv;
  const int64_t heads = mean * L.Hq;
  // joiners of a request: its rows by the sides of a workgroup, but where requests are
  // few (and may be in many parts) a workgroup a row
  const int64_t spread = (kComputeUnits + L.R - 1) / L.R, sides = kWaves * (256 / L.D);
  int64_t gy = (heads + sides - 1) / sides;
  if (gy < spread) gy = heads < spread ? heads : spread;
  const int64_t most = kJoiners * L.R < kJoinGrid ? kJoinGrid / L.R : kJoiners;
  const dim3 join(L.R, (unsigned)(gy < most ? gy : most));
  switch (L.D) {
    case 64: launch_product<T, 64>(p, grid, join, stream); break;
    case 96: launch_product<T, 96>(p, grid, join, stream); break;
    case 128: launch_product<T, 128>(p, grid, join, stream); break;
    default: launch_product<T, 256>(p, grid, join, stream); break;
  }
  return hipGetLastError();
}

}  // namespace

size_t attend_ws_bytes(int R, int rows_capacity, int Hq, int Hkv, int D, bool bf16) {
  (void)bf16;
  const Sizes z = sizes_of(R, rows_capacity, Hq, Hkv, D);
  const size_t parts = (size_t)2 * z.shares * Hkv * z.block_rows;
  return kWsHeader + 256 + ws_align(((size_t)R + 1) * 8) + ws_align((size_t)z.shares * 4) +
         ws_align(parts * 8) + ws_align(parts * D * 4);
}

hipError_t launch_attend(const AttendLaunch &L, hipStream_t stream) {
  return L.bf16 ? launch_attend_t<bf16_t>(L, stream) : launch_attend_t<float>(L, stream);
}

}  // namespace dspark
