// Rotary positions: queries and keys of a batch (forward and gradient), and on the
// way into the paged cache, where values are laid along the tokens.
//
// The angle of pair i at position t is t f_i.  Frequencies come as turns a token in
// 64-bit fixed point, u_i = f_i 2^64 / (2 pi), so t u_i mod 2^64 is the angle without
// its whole turns, exactly, for any 32-bit t: one integer product and no table of
// cosines over the positions.  The nearest quarter turn is taken off as an integer too,
// and the rest, at most pi / 4, goes through the Taylor sums of sine and cosine.
//
// A workgroup takes up to 16 rows and a stretch of their heads; the cosines and sines
// of its rows go to LDS once and serve all of the stretch's heads.
//
// Bound: queries, keys and values are read and written once.  8191 rows of 32 + 8 heads of
// 128, bf16 (168 MB): 35 us, 4.8 TB/s (29 in a trace of two batches in turn); 23838 new rows
// of 12 + 2 * 4 heads of 96, fp32, into pages of 64 (366 MB; counters: 183 fetched, 184
// written): 91 us, 4.0 TB/s, where keys and values alone (146 MB) take 42: their 16 slots of
// a page are 64 bytes a row.  Four items of a thread read ahead of the first one's writing
// (95 us; rotary 40), or neighbouring groups on one XCD (98), gain nothing.  1152 rows of
// 128 requests (28 MB): 13.7 us, for values of groups that are not full are stored two bytes
// at a time, one turn after another.  Single tokens: 3.7 us, one launch.
#include <limits.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kWaves = kBlock / kWave;
constexpr int kRows = 16;      // rows of a workgroup; of a page, 16 slots from a multiple of 16 on
constexpr int kMostPairs = 128;
constexpr int kChunk = 32;     // elements of a head whose values one wave lays along the tokens

// How the pairs of a head are reached.
//   kPieces: halves whose both parts are whole 16-byte pieces; one item is a piece of each.
//   kInter:  interleaved; one item is a piece.
//   kSingle: halves that are not; one item is a pair.
enum Mode { kPieces, kInter, kSingle };

struct Turn {
  const uint64_t *turns;
  int rot, D, pair_shift;  // rot / 2 <= 1 << pair_shift
  float magnitude, sign;   // sign: -1 turns back
};

// cos and sin of position * turns, each off by at most 2 x 2^-24: the angle is rounded
// once from 64 bits (an error of 2^-25 of at most pi / 4), the sums end below 2^-25, and
// their last operations round.
__device__ __forceinline__ float2 cos_sin(int position, uint64_t turns) {
  const uint64_t angle = (uint64_t)(int64_t)position * turns;
  const uint32_t quarter = (uint32_t)((angle + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(angle - ((uint64_t)quarter << 62));
  constexpr double kRadians = 6.283185307179586476925 / 18446744073709551616.0;
  const float y = (float)((double)rest * kRadians), z = y * y;
  const float s =
      y + y * (z * (-1.0f / 6 + z * (1.0f / 120 + z * (-1.0f / 5040 + z * (1.0f / 362880)))));
  const float c = 1.0f + z * (-0.5f + z * (1.0f / 24 + z * (-1.0f / 720 +
                  z * (1.0f / 40320 + z * (-1.0f / 3628800)))));
  const float a = quarter & 1 ? s : c, b = quarter & 1 ? c : s;
  return make_float2(quarter == 1 || quarter == 2 ? -a : a, quarter >= 2 ? -b : b);
}

// magnitude (cos, sin) of `rows` positions into LDS
__device__ __forceinline__ void turn_rows(const Turn &t, int rows, const int *position,
                                          float (*cs)[kMostPairs], float (*sn)[kMostPairs]) {
  const int pairs = t.rot / 2;
  for (int x = threadIdx.x; x < rows << t.pair_shift; x += kBlock) {
    const int row = x >> t.pair_shift, i = x & ((1 << t.pair_shift) - 1);
    if (i >= pairs) continue;
    const float2 v = cos_sin(position[row], t.turns[i]);
    cs[row][i] = t.magnitude * v.x;
    sn[row][i] = t.sign * (t.magnitude * v.y);
  }
}

template <typename T> struct Piece {
  static constexpr int kPer = Elem<T>::kPerVec;
  __device__ static __forceinline__ void unpack(u32x4 v, float *x) {
    if constexpr (kPer == 8) {
      const u16x8 h = __builtin_bit_cast(u16x8, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = bf16_to_f32(h[i]);
    } else {
      const floatx4 f = __builtin_bit_cast(floatx4, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = f[i];
    }
  }
  __device__ static __forceinline__ u32x4 pack(const float *x) {
    if constexpr (kPer == 8) {
      bf16x8 h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (__bf16)x[i];
      return __builtin_bit_cast(u32x4, h);
    } else {
      return __builtin_bit_cast(u32x4, floatx4{x[0], x[1], x[2], x[3]});
    }
  }
};

// Items of a head.
template <typename T, Mode kMode> __device__ __forceinline__ int items_of(const Turn &t) {
  constexpr int kPer = Elem<T>::kPerVec;
  if constexpr (kMode == kPieces) return (t.D - t.rot / 2) / kPer;
  else if constexpr (kMode == kInter) return t.D / kPer;
  else return t.D - t.rot / 2;
}

// Item `it` of the head at `from`, turned by its row's cosines and sines, to `to`.
template <typename T, Mode kMode>
__device__ __forceinline__ void turn_item(const Turn &t, int it, const T *from, T *to, const float *cs,
                                          const float *sn) {
  constexpr int kPer = Elem<T>::kPerVec;
  const int pairs = t.rot / 2;
  if constexpr (kMode == kSingle) {
    if (it >= pairs) {
      if (from != to) to[it + pairs] = from[it + pairs];
      return;
    }
    const float a = Elem<T>::at(from, it), b = Elem<T>::at(from, it + pairs);
    store_elem(to, it, a * cs[it] - b * sn[it]);
    store_elem(to, it + pairs, b * cs[it] + a * sn[it]);
  } else if constexpr (kMode == kPieces) {
    const int e = it * kPer;
    if (e >= pairs) {  // behind the pairs
      if (from != to)
        *reinterpret_cast<u32x4 *>(to + e + pairs) = *reinterpret_cast<const u32x4 *>(from + e + pairs);
      return;
    }
    float a[kPer], b[kPer], x[kPer], y[kPer];
    const u32x4 va = *reinterpret_cast<const u32x4 *>(from + e);
    const u32x4 vb = *reinterpret_cast<const u32x4 *>(from + e + pairs);
    Piece<T>::unpack(va, a);
    Piece<T>::unpack(vb, b);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float c = cs[e + i], s = sn[e + i];
      x[i] = a[i] * c - b[i] * s;
      y[i] = b[i] * c + a[i] * s;
    }
    *reinterpret_cast<u32x4 *>(to + e) = Piece<T>::pack(x);
    *reinterpret_cast<u32x4 *>(to + e + pairs) = Piece<T>::pack(y);
  } else {
    const int e = it * kPer;
    const u32x4 v = *reinterpret_cast<const u32x4 *>(from + e);
    if (e >= t.rot) {
      if (from != to) *reinterpret_cast<u32x4 *>(to + e) = v;
      return;
    }
    float a[kPer], x[kPer];
    Piece<T>::unpack(v, a);
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
      const int p = (e + i) / 2;
      const bool in = p < pairs;
      const float c = in ? cs[p] : 1.0f, s = in ? sn[p] : 0.0f;
      x[i] = in ? a[i] * c - a[i + 1] * s : a[i];
      x[i + 1] = in ? a[i + 1] * c + a[i] * s : a[i + 1];
    }
    *reinterpret_cast<u32x4 *>(to + e) = Piece<T>::pack(x);
  }
}

// f(row, slot, item) for all items of `rows` rows and `slots` heads, one thread each;
// the place is carried along instead of divided for anew.
template <typename F> __device__ __forceinline__ void walk(int rows, int slots, int items, F f) {
  if (slots <= 0) return;
  int it = threadIdx.x, slot = it / items;
  it -= slot * items;
  int row = slot / slots;
  slot -= row * slots;
  const int by_slot = kBlock / items, by_it = kBlock - by_slot * items;
  const int by_row = by_slot / slots, by_rest = by_slot - by_row * slots;
  while (row < rows) {
    f(row, slot, it);
    it += by_it;
    slot += by_rest;
    row += by_row;
    if (it >= items) it -= items, ++slot;
    if (slot >= slots) slot -= slots, ++row;
  }
}

// The last i < n with key(i) <= x, keys ascending; -1 where there is none.  By a whole
// wave, 64 keys at a time: every wave has the answer.
template <typename F> __device__ __forceinline__ int last_not_above(int n, int x, F key) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0, hi = n;
  for (;;) {
    const int step = (hi - lo + kWave - 1) / kWave;
    const int i = lo + lane * step;
    const int c = __popcll(__ballot(i < hi && key(i) <= x));
    if (c == 0) return -1;
    lo += (c - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) return lo;
  }
}

// Whether any slice of row_offset is out of order or bounds (a whole workgroup, its own share
// each).  One workgroup of the grid checks them all: 65536 requests of one row 38 us for 21
// without row_offset, 1048576 634 for 284.
__device__ __forceinline__ bool bad_offsets(const int32_t *row_offset, int R, int n_rows) {
  bool bad = false;
  for (int r = threadIdx.x; r < R; r += kBlock) {
    const int a = row_offset[r], b = row_offset[r + 1];
    bad = bad || a < 0 || b < a || b > n_rows;
  }
  return bad;
}

}  // namespace

// ------------------------------------------------------------------- rotary
// blockIdx.x: a stretch of `block_rows` rows; blockIdx.y: a stretch of the heads.
template <typename T, Mode kMode>
__global__ __launch_bounds__(kBlock) void rotary_kernel(RotaryLaunch L, Turn t, int block_rows) {
  __shared__ float cs[kRows][kMostPairs], sn[kRows][kMostPairs];
  __shared__ int position[kRows];
  __shared__ uint32_t used;  // rows that some request has
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int row0 = blockIdx.x * block_rows, rows = min(block_rows, L.n_rows - row0);
  if (L.row_offset != nullptr && blockIdx.x == 0 && blockIdx.y == 0 &&
      bad_offsets(L.row_offset, L.R, L.n_rows))
    flag_error(L.err, kErrLength);
  if (tid < kWave) {  // the rows' requests and positions
    const int row = row0 + lane;
    bool in = lane < rows;
    int place = row;
    if (L.row_offset != nullptr) {
      const int r0 = last_not_above(L.R, row0, [&](int i) { return L.row_offset[i]; });
      int lo = max(r0, 0), hi = L.R;  // this lane's: the last request that begins by its row
      while (in && hi - lo > 1) {
        // requests of this stretch lie close by: steps of doubling width, then halving
        int step = 1;
        while (lo + step < hi && L.row_offset[lo + step] <= row) lo += step, step *= 2;
        hi = min(hi, lo + step);
      }
      const int a = L.row_offset[lo], b = L.row_offset[lo + 1];
      in = in && a >= 0 && a <= row && row < b && b <= L.n_rows;
      place = row - a;
      if (in && L.kv_len != nullptr) place += L.kv_len[lo] - (b - a);
    } else if (in && L.kv_len != nullptr) {
      place = L.kv_len[row] - 1;
    }
    if (in && L.positions != nullptr) place = L.positions[row];
    if (lane < kRows) position[lane] = in ? place : 0;
    const uint64_t all = __ballot(in);
    if (lane == 0) used = (uint32_t)all;
  }
  __syncthreads();
  turn_rows(t, rows, position, cs, sn);
  __syncthreads();
  const int slots = L.Hq + L.Hkv;
  const int s0 = (int)((int64_t)blockIdx.y * slots / gridDim.y);
  const int s1 = (int)((int64_t)(blockIdx.y + 1) * slots / gridDim.y);
  const uint32_t mine = used;
  walk(rows, s1 - s0, items_of<T, kMode>(t), [&](int row, int slot, int it) {
    if (!((mine >> row) & 1)) return;
    slot += s0;
    const bool is_q = slot < L.Hq;
    const int h = is_q ? slot : slot - L.Hq;
    const int64_t at = row0 + row;
    const T *from = reinterpret_cast<const T *>(is_q ? L.q : L.k) + at * (is_q ? L.q_stride : L.k_stride);
    T *to = reinterpret_cast<T *>(is_q ? L.q_out : L.k_out) + at * (is_q ? L.qo_stride : L.ko_stride);
    turn_item<T, kMode>(t, it, from + h * t.D, to + h * t.D, cs[row], sn[row]);
  });
}

// ------------------------------------------------------------- cache_append
// blockIdx.x: 16 slots of one request's page, from a multiple of 16 on.  Request r's
// first such group has the number key(r) = row_offset[r] / 16 + 2 r: n rows lie in at
// most n / 16 + 2 groups, so the numbers of two requests never meet, and no pass over
// the requests has to lay them out.  blockIdx.y: a stretch of the heads, queries first,
// then keys, then values.
template <typename T, Mode kMode>
__global__ __launch_bounds__(kBlock) void append_kernel(AppendLaunch L, Turn t) {
  constexpr int kPer = Elem<T>::kPerVec, kPieceLanes = kChunk / kPer;
  constexpr int kPitch = kChunk + kPer;  // elements; 16-byte rows, columns on all banks
  __shared__ float cs[kRows][kMostPairs], sn[kRows][kMostPairs];
  __shared__ int position[kRows];
  __shared__ __attribute__((aligned(16))) T tile[kWaves][kRows * kPitch];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  int bits = 0;
  const bool report = blockIdx.y == 0;
  if (report && blockIdx.x == 0 && L.row_offset != nullptr &&
      bad_offsets(L.row_offset, L.R, L.rows_capacity))
    bits = kErrLength;
  int r = blockIdx.x, group = 0, a = r, n = 1;
  if (L.row_offset != nullptr) {
    const int b = blockIdx.x;
    auto key = [&](int i) { return (L.row_offset[i] >> 4) + 2 * i; };
    r = last_not_above(L.R, b, key);
    if (r >= 0) {
      a = L.row_offset[r];
      const int end = L.row_offset[r + 1];
      n = a < 0 || end < a || end > L.rows_capacity ? 0 : end - a;
      group = b - key(r);
    } else {
      n = 0;
    }
  }
  int len = 0;
  if (n > 0) {
    len = L.kv_len[r];
    if (len < 0 || len > L.max_pages << L.page_shift) bits |= kErrLength, len = 0;
  }
  const int t0 = len - n, first = ((t0 >> 4) + group) * 16;  // tokens, of the request and of the group
  const int from_token = max(first, t0), rows = min(first + 16, len) - from_token;
  if (n == 0 || group < 0 || rows <= 0) {
    if (bits) flag_error(L.err, bits);
    return;
  }
  const int row0 = a + (from_token - t0), slot0 = from_token & 15;
  // one page holds the whole group
  int page = -1;
  if (first < 0) {
    bits |= kErrLength;
  } else {
    page = L.table[(int64_t)r * L.max_pages + (first >> L.page_shift)];
    if ((unsigned)page >= (unsigned)L.n_pages) bits |= kErrPage, page = -1;
  }
  if (bits && report) flag_error(L.err, bits);
  const int slot_in_page = first & ((1 << L.page_shift) - 1);
  const int slots = L.Hq + 2 * L.Hkv;
  const int s0 = (int)((int64_t)blockIdx.y * slots / gridDim.y);
  const int s1 = (int)((int64_t)(blockIdx.y + 1) * slots / gridDim.y);
  const int turned = L.Hq + (page >= 0 ? L.Hkv : 0);  // without a page the queries alone
  if (s0 < turned) {
    if (t.rot > 0) {
      if (tid < rows)
        position[tid] = L.positions != nullptr ? L.positions[row0 + tid] : from_token + tid;
      __syncthreads();
      turn_rows(t, rows, position, cs, sn);
      __syncthreads();
    }
    T *k_page = reinterpret_cast<T *>(L.k_pages) + (int64_t)max(page, 0) * L.k_page_stride +
                (int64_t)(slot_in_page + slot0) * L.D;
    walk(rows, min(s1, turned) - s0, items_of<T, kMode>(t), [&](int row, int slot, int it) {
      slot += s0;
      const int64_t at = row0 + row;
      const T *from;
      T *to;
      if (slot < L.Hq) {
        from = reinterpret_cast<const T *>(L.q) + at * L.q_stride + slot * L.D;
        to = reinterpret_cast<T *>(L.q_out) + at * L.qo_stride + slot * L.D;
      } else {
        const int h = slot - L.Hq;
        from = reinterpret_cast<const T *>(L.k_new) + at * L.kv_stride + h * L.D;
        to = k_page + ((int64_t)h << L.page_shift) * L.D + row * L.D;
      }
      turn_item<T, kMode>(t, it, from, to, cs[row], sn[row]);
    });
  }
  if (page < 0 || s1 <= L.Hq + L.Hkv) return;
  // values: a wave lays kChunk elements of a head along the 16 tokens through its own tile
  const int h0 = max(s0 - L.Hq - L.Hkv, 0), h1 = s1 - L.Hq - L.Hkv, chunks = L.D / kChunk;
  T *v_page = reinterpret_cast<T *>(L.v_pages) + (int64_t)page * L.v_page_stride + slot_in_page;
  const T *v_new = reinterpret_cast<const T *>(L.v_new) + (int64_t)row0 * L.kv_stride;
  T *mine = tile[wave];
  for (int i = h0 * chunks + wave; i < h1 * chunks; i += kWaves) {
    const int e0 = i * kChunk;  // of the row's Hkv * D
    wave_sync();
#pragma unroll
    for (int x = lane; x < kRows * kPieceLanes; x += kWave) {
      const int row = x / kPieceLanes, e = x % kPieceLanes * kPer;
      if (row < rows)
        *reinterpret_cast<u32x4 *>(mine + (slot0 + row) * kPitch + e) =
            *reinterpret_cast<const u32x4 *>(v_new + row * L.kv_stride + e0 + e);
    }
    wave_sync();
    if (rows == kRows) {
#pragma unroll
      for (int x = lane; x < kChunk * kRows / kPer; x += kWave) {
        const int e = x / (kRows / kPer), slot = x % (kRows / kPer) * kPer;
        T v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = mine[(slot + j) * kPitch + e];
        u32x4 out;
        __builtin_memcpy(&out, v, 16);
        *reinterpret_cast<u32x4 *>(v_page + ((int64_t)(e0 + e) << L.page_shift) + slot) = out;
      }
    } else {
#pragma unroll
      for (int x = lane; x < kChunk * kRows; x += kWave) {
        const int e = x / kRows, slot = x % kRows;
        if (slot >= slot0 && slot < slot0 + rows)
          v_page[((int64_t)(e0 + e) << L.page_shift) + slot] = mine[slot * kPitch + e];
      }
    }
  }
}

// ----------------------------------------------------------------- launches
namespace {

Turn turn_of(int rot, int D, float magnitude, float sign, const uint64_t *turns) {
  Turn t{turns, rot, D, 0, magnitude, sign};
  while (1 << t.pair_shift < rot / 2) ++t.pair_shift;
  return t;
}

Mode mode_of(int rot, bool interleaved, bool bf16) {
  if (rot == 0 || interleaved) return kInter;
  return rot / 2 % (bf16 ? 8 : 4) == 0 ? kPieces : kSingle;
}

}  // namespace

hipError_t launch_rotary(const RotaryLaunch &L, hipStream_t stream) {
  const Turn t = turn_of(L.rot, L.D, L.magnitude, L.back ? -1.0f : 1.0f, L.turns);
  const int block_rows = 4;
  const int blocks = (L.n_rows + block_rows - 1) / block_rows, slots = L.Hq + L.Hkv;
  const int want = (4 * kComputeUnits + blocks - 1) / blocks;
  const dim3 grid(blocks, want < slots ? want : slots);
  auto go = [&](auto type, auto mode) {
    using T = decltype(type);
    constexpr Mode kMode = decltype(mode)::value;
    DSPARK_LAUNCH("rotary", stream, (rotary_kernel<T, kMode>), grid, kBlock, L, t, block_rows);
  };
  const Mode mode = mode_of(L.rot, L.interleaved, L.bf16);
  auto with = [&](auto type) {
    if (mode == kPieces) go(type, std::integral_constant<Mode, kPieces>());
    else if (mode == kInter) go(type, std::integral_constant<Mode, kInter>());
    else go(type, std::integral_constant<Mode, kSingle>());
  };
  if (L.bf16) with(bf16_t());
  else with(float());
  return hipGetLastError();
}

hipError_t launch_append(const AppendLaunch &L, hipStream_t stream) {
  const Turn t = turn_of(L.rot, L.D, L.magnitude, 1.0f, L.turns);
  const int blocks = L.row_offset == nullptr ? L.R : L.rows_capacity / 16 + 2 * L.R;
  const int slots = L.Hq + 2 * L.Hkv;
  const int want = (8 * kComputeUnits + blocks - 1) / blocks;
  const dim3 grid(blocks, want < slots ? want : slots);
  auto go = [&](auto type, auto mode) {
    using T = decltype(type);
    constexpr Mode kMode = decltype(mode)::value;
    DSPARK_LAUNCH("cache_append", stream, (append_kernel<T, kMode>), grid, kBlock, L, t);
  };
  const Mode mode = mode_of(L.rot, L.interleaved, L.bf16);
  auto with = [&](auto type) {
    if (mode == kPieces) go(type, std::integral_constant<Mode, kPieces>());
    else if (mode == kInter) go(type, std::integral_constant<Mode, kInter>());
    else go(type, std::integral_constant<Mode, kSingle>());
  };
  if (L.bf16) with(bf16_t());
  else with(float());
  return hipGetLastError();
}

}  // namespace dspark
