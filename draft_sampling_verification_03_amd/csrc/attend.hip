// Attention of every request's new rows over its paged keys and values.
//
// Three launches:
//  1. attend_prepare_kernel: the first workgroup lays out the work (below); the
//     others write the new rows' keys and values into their pages.
//  2. attend_kernel: one work item is a block of up to 16 MT rows (a row here is
//     one query head of one new token; the Hq / Hkv heads of a group and the
//     request's new tokens share their keys, so they share the block), one
//     key-value head and a stretch of the request's tokens.  Its four waves take
//     the stretch's steps in turn and are joined in LDS.  A request in one
//     stretch writes its result, one in several leaves (max, sum, sum p v).
//  3. attend_join_kernel joins the stretches.
//
// The product in registers alone.  Scores are formed transposed, S^T = K Q^T, and
// the result too, O^T = V^T P^T: a lane then holds the same row of Q in S^T and in
// O^T, so maxima, sums and rescaling factors never cross lanes, and P^T leaves the
// first product in the register layout in which the second wants it.  For that the
// 32 keys of a bf16 step are entered in an order that gives a lane 8 consecutive
// ones, and values lie along the tokens in their pages, so that a lane's 8 are one
// 16-byte load.  No LDS and no shuffle stand between the loads and the products.
//
// Bound: keys and values are read once from memory (2 Hkv D bytes a token for each
// of K and V); the products are 4 Hq D n operations a token, far below the matrix
// rate for the rows of a round.
#include <limits.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kWaves = kBlock / kWave;
// Work items aimed at over all key-value heads (see lay_out).
constexpr int kTarget = 4 * kComputeUnits;
constexpr int kLeast = 128;       // tokens of a stretch, at least: one step of every wave
constexpr float kNone = -1e30f;   // running maximum of a row that has seen nothing
constexpr float kSlack = 8.0f;    // see rescale below

struct AttendParams {
  AttendLaunch L;
  int heads_per_group, block_rows;
  int most_items, most_slots;
  // scratch
  int32_t *head;    // [0] number of items, [1] split slots used
  int4 *items;      // (request, first row of the block, first token, slot or -1)
  int2 *stretches;  // [R]: (tokens of a stretch, first slot or -1)
  float2 *part_ml;  // [slots][Hkv][block_rows]: (max in log2 units, sum)
  float *part_o;    // [slots][Hkv][block_rows][D]
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

__device__ __forceinline__ int2 scan2(int2 v, int2 *scratch, int2 *total) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  int2 inc = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int x = __shfl_up(inc.x, o), y = __shfl_up(inc.y, o);
    if (lane >= o) { inc.x += x; inc.y += y; }
  }
  __syncthreads();
  if (lane == kWave - 1) scratch[w] = inc;
  __syncthreads();
  int2 before = {0, 0}, all = {0, 0};
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) { before.x += scratch[i].x; before.y += scratch[i].y; }
    all.x += scratch[i].x; all.y += scratch[i].y;
  }
  *total = all;
  return make_int2(before.x + inc.x - v.x, before.y + inc.y - v.y);
}

__device__ __forceinline__ double block_sum_f64(double v, double *scratch) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  __syncthreads();
  if ((threadIdx.x & (kWave - 1)) == 0) scratch[threadIdx.x / kWave] = v;
  __syncthreads();
  return ((scratch[0] + scratch[1]) + scratch[2]) + scratch[3];
}

}  // namespace

// Stretches so long that all blocks' tokens together make about kTarget items
// over all key-value heads (lengths may differ a lot: an item's work, not a
// request's, is what has to be alike); a request within one stretch is not
// split.  A split request has at least two stretches, each but the last full,
// so split items number at most 2 kTarget / Hkv: the slots.
__device__ __forceinline__ void lay_out(const AttendParams &p) {
  const AttendLaunch &L = p.L;
  __shared__ double sums[kWaves];
  __shared__ int2 scratch[kWaves];
  const int tid = threadIdx.x;
  int bits = 0;
  double work = 0.0;
  for (int r = tid; r < L.R; r += kBlock) {
    const Slice s = slice_of(L, r, &bits);
    const int blocks = (s.n * p.heads_per_group + p.block_rows - 1) / p.block_rows;
    work += (double)blocks * (s.len - first_token(L, s));
  }
  work = block_sum_f64(work, sums) * L.Hkv;
  const int64_t even = (int64_t)(work / kTarget) + 1;
  const int stretch = (int)min((int64_t)(even < kLeast ? kLeast : (even + 127) / 128 * 128),
                               (int64_t)1 << 30);
  int2 base = {0, 0};
  for (int r0 = 0; r0 < L.R; r0 += kBlock) {
    const int r = r0 + tid;
    int2 count = {0, 0};
    Slice s{};
    int blocks = 0, splits = 1, t0 = 0;
    if (r < L.R) {
      s = slice_of(L, r, &bits);
      t0 = first_token(L, s);
      blocks = (s.n * p.heads_per_group + p.block_rows - 1) / p.block_rows;
      splits = max(1, (int)(((int64_t)s.len - t0 + stretch - 1) / stretch));
      count = make_int2(blocks * splits, splits > 1 ? blocks * splits : 0);
    }
    int2 total;
    const int2 at = scan2(count, scratch, &total);
    if (r < L.R) {
      const int item0 = base.x + at.x, slot0 = base.y + at.y;
      p.stretches[r] = make_int2(stretch, splits > 1 ? slot0 : -1);
      for (int i = 0; i < blocks * splits; ++i) {
        // only slices that overlap (a row_offset that decreases) can pass the bounds
        if (item0 + i >= p.most_items || (splits > 1 && slot0 + i >= p.most_slots)) {
          bits |= kErrLength;
          break;
        }
        const int b = i % blocks, k = i / blocks;
        p.items[item0 + i] =
            make_int4(r, b * p.block_rows, t0 + k * stretch, splits > 1 ? slot0 + i : -1);
      }
    }
    base.x += total.x;
    base.y += total.y;
  }
  if (tid == 0) {
    p.head[0] = min(base.x, p.most_items);
    p.head[1] = base.y;
  }
  if (bits) flag_error(L.err, bits);
}

// Workgroups from 1 on: request (b - 1) % R, every n-th of its rows.
template <typename T>
__global__ __launch_bounds__(kBlock) void attend_prepare_kernel(AttendParams p) {
  if (blockIdx.x == 0) {
    lay_out(p);
    return;
  }
  const AttendLaunch &L = p.L;
  constexpr int kPer = Elem<T>::kPerVec;
  int bits = 0;
  const int b = blockIdx.x - 1, r = b % L.R, part = b / L.R, parts = (gridDim.x - 1) / L.R;
  const Slice s = slice_of(L, r, &bits);
  const int page_mask = (1 << L.page_shift) - 1;
  const int pieces = L.Hkv * L.D / kPer;
  bits = 0;  // the layout reports the slices
  for (int j = part; j < s.n; j += parts) {
    const int t = s.len - s.n + j;
    if (t < 0) {
      bits |= kErrLength;
      continue;
    }
    const int id = L.table[(int64_t)r * L.max_pages + (t >> L.page_shift)], slot = t & page_mask;
    if ((unsigned)id >= (unsigned)L.n_pages) {
      bits |= kErrPage;
      continue;
    }
    const T *kn = reinterpret_cast<const T *>(L.k_new) + (int64_t)(s.row0 + j) * L.kv_stride;
    const T *vn = reinterpret_cast<const T *>(L.v_new) + (int64_t)(s.row0 + j) * L.kv_stride;
    T *kp = reinterpret_cast<T *>(L.k_pages) + (int64_t)id * L.k_page_stride;
    T *vp = reinterpret_cast<T *>(L.v_pages) + (int64_t)id * L.v_page_stride;
    for (int i = threadIdx.x; i < pieces; i += kBlock) {
      const int h = i * kPer / L.D, d = i * kPer - h * L.D;
      const u32x4 k = *reinterpret_cast<const u32x4 *>(kn + i * kPer);
      *reinterpret_cast<u32x4 *>(kp + (((int64_t)h << L.page_shift) + slot) * L.D + d) = k;
    }
    for (int i = threadIdx.x; i < L.Hkv * L.D; i += kBlock)
      vp[((int64_t)i << L.page_shift) + slot] = vn[i];
  }
  if (bits && threadIdx.x == 0) flag_error(L.err, bits);
}

namespace {

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
  template <int D>
  __device__ static __forceinline__ void load_k(const bf16_t *k, int t, int g, K<D> &o) {
#pragma unroll
    for (int s = 0; s < D / 32; ++s) o.v[t][s] = ld_stream4(k + 32 * s + 8 * g);
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
  template <int D>
  __device__ static __forceinline__ void load_k(const float *k, int t, int g, K<D> &o) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) o.v[t][s] = ld_stream4(k + 16 * s + 4 * g);
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

template <typename T, int D, int MT>
__global__ __launch_bounds__(kBlock) void attend_kernel(AttendParams p) {
  using St = Step<T>;
  constexpr int kKeys = St::kKeys, kMine = St::kMine, kTiles = St::kTiles;
  constexpr int kOut = D / 16;      // 16-wide tiles of the result
  constexpr int kPitch = D + 4;     // of a row in LDS, floats
  // registers: D / 2 for a step's keys and values, 3 D / 8 for a tile's result and queries
  constexpr bool kAhead = D + MT * 3 * D / 8 <= 240;
  __shared__ float lds_o[kWaves][16][kPitch];
  __shared__ float2 lds_ml[kWaves][16];
  const AttendLaunch &L = p.L;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  const int n_items = p.head[0];
  const int group = p.heads_per_group;
  const float to_log2 = L.scale * kLog2e;

  for (int64_t w = blockIdx.x; w < (int64_t)n_items * L.Hkv; w += gridDim.x) {
    const int hk = (int)(w % L.Hkv);
    const int4 item = p.items[w / L.Hkv];
    const int r = item.x, block_row = item.y, begin = item.z, slot = item.w;
    int bits = 0;
    const Slice sl = slice_of(L, r, &bits);
    const int end = min(begin + p.stretches[r].x, sl.len);
    const int rows = min(p.block_rows, sl.n * group - block_row);
    const int32_t *table = L.table + (int64_t)r * L.max_pages;

    // this lane's row of each tile: tokens it sees are [low, high)
    typename St::template Q<D> q[MT];
    int low[MT], high[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int i = mt * 16 + col, j = (block_row + i) / group, h = (block_row + i) % group;
      low[mt] = high[mt] = 0;
#pragma unroll
      for (unsigned s = 0; s < sizeof(q[mt].v) / 16; ++s) q[mt].v[s] = u32x4{0, 0, 0, 0};
      if (i < rows) {
        high[mt] = max(0, sl.len - sl.n + 1 + j);
        low[mt] = L.window > 0 ? max(0, high[mt] - L.window) : 0;
        St::template load_q<D>(reinterpret_cast<const T *>(L.q) +
                                   (int64_t)(sl.row0 + j) * L.q_stride + (hk * group + h) * D,
                               g, q[mt]);
      }
    }
    const int first_j = block_row / group, last_j = (block_row + rows - 1) / group;
    const int least_high = max(0, sl.len - sl.n + 1 + first_j);
    const int most_low = L.window > 0 ? sl.len - sl.n + 1 + last_j - L.window : 0;

    floatx4 o[MT][kOut];
    float m[MT], l[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      m[mt] = kNone;
      l[mt] = 0.0f;
#pragma unroll
      for (int d = 0; d < kOut; ++d) o[mt][d] = floatx4{0, 0, 0, 0};
    }

    struct Data {
      typename St::template K<D> k;
      typename St::template V<D> v;
      bool bad;  // this lane's keys lie in a page that does not exist
    };
    const T *kbase = reinterpret_cast<const T *>(L.k_pages) + ((int64_t)hk << L.page_shift) * D;
    const T *vbase = reinterpret_cast<const T *>(L.v_pages) + ((int64_t)hk * D << L.page_shift);
    const int page_mask = (1 << L.page_shift) - 1;
    // loads of the step at token t; tokens past the last read the last page again
    auto load = [&](int t, Data &x) __attribute__((always_inline)) {
      const int last = sl.len - 1;
      const int tk = t + St::key_of_row(col, 0), tv = t + kMine * g;
      const int ik = table[min(tk, last) >> L.page_shift];
      const int iv = table[min(tv, last) >> L.page_shift];
      x.bad = (unsigned)iv >= (unsigned)L.n_pages;
      const T *k = kbase + (int64_t)((unsigned)ik < (unsigned)L.n_pages ? ik : 0) * L.k_page_stride;
      const T *v = vbase + (int64_t)(x.bad ? 0 : iv) * L.v_page_stride + (tv & page_mask);
#pragma unroll
      for (int s = 0; s < kTiles; ++s)
        St::template load_k<D>(k + (int64_t)((t + St::key_of_row(col, s)) & page_mask) * D, s, g, x.k);
#pragma unroll
      for (int d = 0; d < kOut; ++d)
        x.v.v[d] = ld_stream4(v + ((int64_t)(16 * d + col) << L.page_shift));
    };
    auto compute = [&](int t, Data &x) __attribute__((always_inline)) {
      const int t0 = t + kMine * g;  // this lane's first token
      const bool any_bad = __ballot(x.bad) != 0;
      const bool edge = any_bad || t + kKeys > least_high || t < most_low;  // uniform
      bool mixed = false;  // a value that is not finite, seen by some rows only
      if (edge) {
        if (x.bad) bits |= kErrPage;
        bool odd = false;
#pragma unroll
        for (int d = 0; d < kOut; ++d) {
          x.v.v[d] = St::keep(x.v.v[d], 0, x.bad ? 0 : sl.len - t0);
          odd = odd || St::not_finite(x.v.v[d]);
        }
        mixed = __ballot(odd) != 0;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (mt * 16 >= rows) continue;  // uniform
        float s[kMine];
#pragma unroll
        for (int u = 0; u < kTiles; ++u) {
          const floatx4 a = St::template scores<D>(x.k, u, q[mt]);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[4 * u + i] = a[i];
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < kMine; ++i)
            if (x.bad || t0 + i < low[mt] || t0 + i >= high[mt]) s[i] = -INFINITY;
        }
        // The subtrahend follows the running maximum only when that is kSlack
        // (a factor 2^8) ahead; below that the sums just grow, and the sums and
        // products need no rescaling.
        float top = s[0];
#pragma unroll
        for (int i = 1; i < kMine; ++i) top = fmaxf(top, s[i]);
        top *= to_log2;
        if (__ballot(top > m[mt] + kSlack) != 0) {
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const float now = fmaxf(m[mt], top), f = exp2_fast(m[mt] - now);
          m[mt] = now;
          l[mt] *= f;
#pragma unroll
          for (int d = 0; d < kOut; ++d) o[mt][d] *= f;
        }
        float e[kMine], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          e[i] = exp2_fast(fmaf(s[i], to_log2, -m[mt]));
          sum += e[i];
        }
        l[mt] += sum;
        const typename St::P pr = St::pack(e);
        if (!mixed) {
#pragma unroll
          for (int d = 0; d < kOut; ++d) o[mt][d] = St::product(x.v.v[d], pr, o[mt][d]);
        } else {
          // row by row, with what the row does not see zeroed in V
          for (int c = 0; c < 16; ++c) {
            const int from = __shfl(low[mt], c) - t0, to = __shfl(high[mt], c) - t0;
#pragma unroll
            for (int d = 0; d < kOut; ++d) {
              const floatx4 a = St::product(St::keep(x.v.v[d], from, to), pr, o[mt][d]);
              if (col == c) o[mt][d] = a;
            }
          }
        }
      }
    };

    // every wave its steps; where registers allow, the next one's loads are in
    // flight during this one's products
    const int stride = kWaves * kKeys;
    int t = begin + wave * kKeys;
    Data a;
    if constexpr (!kAhead) {
      for (; t < end; t += stride) {
        load(t, a);
        compute(t, a);
      }
    } else if (t < end) {
      Data b;
      load(t, a);
      for (;;) {
        const bool more = t + stride < end;
        if (more) load(t + stride, b);
        compute(t, a);
        t += stride;
        if (!more) break;
        const bool again = t + stride < end;
        if (again) load(t + stride, a);
        compute(t, b);
        t += stride;
        if (!again) break;
      }
    }
    if (bits) flag_error(L.err, bits);

    // join the waves, one tile of rows at a time
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (mt * 16 >= rows) continue;
      float sum = l[mt];
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      __syncthreads();
      if (g == 0) lds_ml[wave][col] = make_float2(m[mt], sum);
#pragma unroll
      for (int d = 0; d < kOut; ++d)
        *reinterpret_cast<floatx4 *>(&lds_o[wave][col][16 * d + 4 * g]) = o[mt][d];
      __syncthreads();
      // 4 elements a thread at a time
      for (int i = threadIdx.x; i < 16 * D / 4; i += kBlock) {
        const int c = i / (D / 4), d = i % (D / 4) * 4, row = mt * 16 + c;
        if (row >= rows) continue;
        float mx = kNone;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) mx = fmaxf(mx, lds_ml[v][c].x);
        float all = 0.0f, x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          const float f = exp2_fast(lds_ml[v][c].x - mx);
          all += f * lds_ml[v][c].y;
          const floatx4 y = *reinterpret_cast<const floatx4 *>(&lds_o[v][c][d]);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] += f * y[k];
        }
        if (slot >= 0) {
          const int64_t at = ((int64_t)slot * L.Hkv + hk) * p.block_rows + row;
          store4(p.part_o + at * D + d, x);
          if (d == 0) p.part_ml[at] = make_float2(mx, all);
        } else {
          const float inv = all > 0.0f ? 1.0f / all : (all == 0.0f ? 0.0f : all);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] *= inv;
          const int j = (block_row + row) / group, h = hk * group + (block_row + row) % group;
          const int64_t out_row = (int64_t)(sl.row0 + j) * L.Hq + h;
          store4(reinterpret_cast<T *>(L.out) + out_row * D + d, x);
          if (d == 0 && L.lse != nullptr)
            L.lse[out_row] = all == 0.0f ? -INFINITY : fmaf(mx, 0.6931471805599453f, logf(all));
        }
      }
    }
    __syncthreads();
  }
}

// One wave per (new token, query head) of the split requests.
template <typename T>
__global__ __launch_bounds__(kBlock) void attend_join_kernel(AttendParams p) {
  const AttendLaunch &L = p.L;
  if (p.head[1] == 0) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int r = blockIdx.x;
  const int2 st = p.stretches[r];
  if (st.y < 0) return;
  int bits = 0;
  const Slice s = slice_of(L, r, &bits);
  const int group = p.heads_per_group, D = L.D;
  const int blocks = (s.n * group + p.block_rows - 1) / p.block_rows;
  const int splits = (s.len - first_token(L, s) + st.x - 1) / st.x;
  const int waves = gridDim.y * kWaves;
  for (int i = blockIdx.y * kWaves + threadIdx.x / kWave; i < s.n * L.Hq; i += waves) {
    const int j = i / L.Hq, h = i % L.Hq, hk = h / group, row = j * group + h % group;
    const int b = row / p.block_rows;
    // slot of stretch k: st.y + k blocks + b
    const int64_t first = ((int64_t)(st.y + b) * L.Hkv + hk) * p.block_rows + row % p.block_rows;
    const int64_t next = (int64_t)blocks * L.Hkv * p.block_rows;
    float mx = kNone;
    for (int k = lane; k < splits; k += kWave) mx = fmaxf(mx, p.part_ml[first + k * next].x);
    mx = wave_max(mx);
    float all = 0.0f, x[4] = {0, 0, 0, 0};
    const int d = lane * 4;
    for (int k = 0; k < splits; ++k) {
      const float2 ml = p.part_ml[first + k * next];
      const float f = exp2_fast(ml.x - mx);
      all += f * ml.y;
      if (d < D) {
        const floatx4 y = *reinterpret_cast<const floatx4 *>(p.part_o + (first + k * next) * D + d);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += f * y[e];
      }
    }
    const float inv = all > 0.0f ? 1.0f / all : (all == 0.0f ? 0.0f : all);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= inv;
    const int64_t out_row = (int64_t)(s.row0 + j) * L.Hq + h;
    if (d < D) store4(reinterpret_cast<T *>(L.out) + out_row * D + d, x);
    if (lane == 0 && L.lse != nullptr)
      L.lse[out_row] = all == 0.0f ? -INFINITY : fmaf(mx, 0.6931471805599453f, logf(all));
  }
}

// ------------------------------------------------------------------- launch
namespace {

// Row tiles of a block: enough for the mean request's rows, so that the keys are
// read once for all of them (a request with more takes several blocks, which read
// them again from the caches); registers allow 4 tiles up to D = 128, 1 beyond.
int row_tiles(int R, int rows_capacity, int group, int D) {
  const int rows = (int)(((int64_t)rows_capacity * group + R - 1) / R);
  if (D > 128 || rows <= 16) return 1;
  return rows <= 32 ? 2 : 4;
}

struct Sizes {
  int tiles, block_rows;
  int64_t items, slots;
};
Sizes sizes_of(int R, int rows_capacity, int Hq, int Hkv, int D) {
  Sizes z;
  const int group = Hq / Hkv;
  z.tiles = row_tiles(R, rows_capacity, group, D);
  z.block_rows = 16 * z.tiles;
  z.slots = 2 * kTarget / Hkv + 2;
  z.items = R + ((int64_t)rows_capacity * group) / z.block_rows + z.slots;
  return z;
}

template <typename T, int D, int MT> void launch_one(const AttendParams &p, int grid, hipStream_t stream) {
  DSPARK_LAUNCH("attend", stream, (attend_kernel<T, D, MT>), grid, kBlock, p);
}
template <typename T, int D>
void launch_tiles(const AttendParams &p, int tiles, int grid, hipStream_t stream) {
  if constexpr (D <= 128) {
    if (tiles == 4) return launch_one<T, D, 4>(p, grid, stream);
    if (tiles == 2) return launch_one<T, D, 2>(p, grid, stream);
  }
  launch_one<T, D, 1>(p, grid, stream);
}

template <typename T> hipError_t launch_attend_t(const AttendLaunch &L, hipStream_t stream) {
  const Sizes z = sizes_of(L.R, L.rows_capacity, L.Hq, L.Hkv, L.D);
  AttendParams p{};
  p.L = L;
  p.heads_per_group = L.Hq / L.Hkv;
  p.block_rows = z.block_rows;
  p.most_items = (int)z.items;
  p.most_slots = (int)z.slots;
  char *at = (char *)L.scratch;
  auto take = [&](size_t bytes) { char *c = at; at += ws_align(bytes); return c; };
  p.head = (int32_t *)take(256);
  p.items = (int4 *)take((size_t)z.items * 16);
  p.stretches = (int2 *)take((size_t)L.R * 8);
  p.part_ml = (float2 *)take((size_t)z.slots * L.Hkv * z.block_rows * 8);
  p.part_o = (float *)take((size_t)z.slots * L.Hkv * z.block_rows * L.D * 4);
  // appenders: a workgroup for every 4 rows of a request or so
  const int64_t mean = (L.rows_capacity + L.R - 1) / L.R;
  const int parts = L.k_new == nullptr ? 0 : (int)(mean < 4 ? 1 : mean < 256 ? (mean + 3) / 4 : 64);
  DSPARK_LAUNCH("attend_prepare", stream, attend_prepare_kernel<T>, 1 + L.R * parts, kBlock, p);
  const int64_t most = z.items * L.Hkv;
  const int grid = (int)(most < 8 * kComputeUnits ? most : 8 * kComputeUnits);
  switch (L.D) {
    case 64: launch_tiles<T, 64>(p, z.tiles, grid, stream); break;
    case 96: launch_tiles<T, 96>(p, z.tiles, grid, stream); break;
    case 128: launch_tiles<T, 128>(p, z.tiles, grid, stream); break;
    default: launch_tiles<T, 256>(p, z.tiles, grid, stream); break;
  }
  const int64_t heads = mean * L.Hq;
  const int gy = (int)(heads < 4 * 64 ? (heads + 3) / 4 : 64);
  DSPARK_LAUNCH("attend_join", stream, attend_join_kernel<T>, dim3(L.R, gy), kBlock, p);
  return hipGetLastError();
}

}  // namespace

size_t attend_ws_bytes(int R, int rows_capacity, int Hq, int Hkv, int D, bool bf16) {
  (void)bf16;
  const Sizes z = sizes_of(R, rows_capacity, Hq, Hkv, D);
  const size_t parts = (size_t)z.slots * Hkv * z.block_rows;
  return kWsHeader + 256 + ws_align((size_t)z.items * 16) + ws_align((size_t)R * 8) +
         ws_align(parts * 8) + ws_align(parts * D * 4);
}

hipError_t launch_attend(const AttendLaunch &L, hipStream_t stream) {
  return L.bf16 ? launch_attend_t<bf16_t>(L, stream) : launch_attend_t<float>(L, stream);
}

}  // namespace dspark
