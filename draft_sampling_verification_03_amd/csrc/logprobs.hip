// Log probabilities of given tokens, entropy and the top alternatives of logit
// rows, and their gradient.
//
// Forward, two launches.  logprob_chunk_kernel: one workgroup takes a chunk of
// one row and keeps it in registers (every load in flight at once), so the row
// is read from memory once; from the registers come the chunk's maximum, then
//   S = sum 2^u, E = sum 2^u u, u = (x - max) log2(e) / T   (no running rescale)
// and the chunk's k largest elements.  logprob_join_kernel: one workgroup a row
// joins the chunks by their maxima, and
//   log S, entropy = log S - E ln 2 / S, logp = (x_t - max) / T - log S.
//
// Top k of a chunk without sorting it: every wave finds the ceil(k / 4)-th
// largest of its lanes' maxima (the lanes hold different elements, so at least
// ceil(k / 4) elements of the wave reach it); the least of the four is a
// threshold that at least k elements of the chunk reach, and hardly more than
// that.  Those are collected and ranked by counting.
#include <limits.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kMaxCand = 1024;  // collected elements of a chunk or a row

// Order of the alternatives: larger value first, then smaller index.  A key
// holds the value's bits as an ordered integer above the index's complement;
// 0 is below every key.
__device__ __forceinline__ uint64_t alt_key(float x, int idx) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 counts as 0
  const uint32_t o = b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
  return ((uint64_t)o << 32) | (0xFFFFFFFFu - (uint32_t)idx);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o >> 31) ? (o ^ 0x80000000u) : ~o);
}
__device__ __forceinline__ int key_index(uint64_t k) { return (int)(0xFFFFFFFFu - (uint32_t)k); }

__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint64_t w = __shfl_xor((unsigned long long)v, o);
    v = w > v ? w : v;
  }
  return v;
}

// The row's request: the number of rho in [1, R) with row_offset[rho] <= row
// (the offsets do not decrease), by ballots over loads that are all in flight.
__device__ __forceinline__ int request_of_row(const int32_t *row_offset, int R, int row) {
  const int lane = threadIdx.x & (kWave - 1);
  int lo = 0;
  for (int t0 = 1; t0 < R; t0 += kWave) {
    const int t = t0 + lane;
    lo += __popcll(__ballot(t < R && row_offset[min(t, R)] <= row));
  }
  return lo;
}

// The token of a row: -1 none (also past the request's tokens).
__device__ __forceinline__ int token_of_row(const int32_t *tokens, const int32_t *row_offset, int R,
                                            int tok_stride, int row) {
  if (tokens == nullptr) return -1;
  if (row_offset == nullptr) return tokens[row];
  const int rho = request_of_row(row_offset, R, row);
  const int j = row - row_offset[rho];
  return j >= 0 && j < tok_stride ? tokens[(int64_t)rho * tok_stride + j] : -1;
}

__device__ __forceinline__ int rows_in_use(const int32_t *row_offset, int R, int n_rows) {
  return row_offset == nullptr ? n_rows : min(row_offset[R], n_rows);
}

// Ranks the n keys of buf (LDS, all different) by counting and writes the
// first k of them in order.
template <typename F>
__device__ __forceinline__ void rank_keys(const uint64_t *buf, int n, int k, F write) {
  for (int i = threadIdx.x; i < n; i += kBlock) {
    const uint64_t mine = buf[i];
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += buf[j] > mine;
    if (rank < k) write(rank, mine);
  }
}

struct ChunkParams {
  int n_rows, V, R, k, n_chunks, pieces_per_chunk;
  int64_t row_stride;
  float scale;  // log2(e) / T
  const void *X;
  const int32_t *row_offset;
  float4 *sums;    // [n_rows][n_chunks]: (max x, S, E, unused)
  uint64_t *keys;  // [n_rows][n_chunks][k], descending, 0 behind the last
};

}  // namespace

template <typename T, int VPT>
__global__ __launch_bounds__(kBlock) void logprob_chunk_kernel(ChunkParams p) {
  constexpr int kPer = Elem<T>::kPerVec;
  __shared__ float red[8];
  __shared__ uint64_t cand[kMaxCand];
  __shared__ int n_cand;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int row = blockIdx.x / p.n_chunks, c = blockIdx.x % p.n_chunks;
  if (row >= rows_in_use(p.row_offset, p.R, p.n_rows)) return;
  const int n_pieces = (p.V + kPer - 1) / kPer;
  const int p0 = c * p.pieces_per_chunk, p1 = min(p0 + p.pieces_per_chunk, n_pieces);
  const T *X = reinterpret_cast<const T *>(p.X) + (int64_t)row * p.row_stride;

  // the chunk in registers; a piece past its end reads the last one again
  u32x4 raw[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    raw[j] = ld_stream4(X + (int64_t)min(p0 + j * kBlock + tid, p1 - 1) * kPer);
  if (tid == 0) n_cand = 0;

  // element q of piece j; past the chunk or the vocabulary: -infinity
  auto value = [&](int j, int q, const float *x) __attribute__((always_inline)) {
    const int piece = p0 + j * kBlock + tid;
    return piece < p1 && piece * kPer + q < p.V ? x[q] : -INFINITY;
  };
  float pm[VPT], tm = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float x[kPer];
    unpack16(raw[j], (T *)nullptr, x);
    pm[j] = -INFINITY;
#pragma unroll
    for (int q = 0; q < kPer; ++q) pm[j] = fmaxf(pm[j], value(j, q, x));
    tm = fmaxf(tm, pm[j]);
  }

  // threshold of the k largest
  const int kw = (p.k + 3) / 4;
  float thr = tm;
  if (kw > 0) {
    float left = tm;
    uint64_t out = 0;  // lanes taken
    for (int i = 0; i < kw; ++i) {
      thr = wave_max(left);
      const uint64_t at = __ballot(left == thr) & ~out;
      if (at == 0) { thr = -INFINITY; break; }  // NaN lanes
      const uint64_t one = at & (~at + 1);
      out |= one;
      if (one >> lane & 1) left = -INFINITY;
    }
  }
  const float wm = wave_max(tm);
  if (lane == 0) { red[wave] = wm; red[4 + wave] = thr; }
  __syncthreads();
  const float mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  thr = fminf(fminf(red[4], red[5]), fminf(red[6], red[7]));

  float S = 0.0f, E = 0.0f;
  if (mx != -INFINITY) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float x[kPer];
      unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float u = (value(j, q, x) - mx) * p.scale;
        const float e = exp2_fast(u);
        S += e;
        E = fmaf(e, fmaxf(u, -1e4f), E);  // a masked logit has e = 0: its u only has to be finite
      }
    }
  } else {  // all masked, unless a NaN hides among them
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float x[kPer];
      unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float v = value(j, q, x);
        if (v != v) S = v;
      }
    }
  }
  const float Sw = wave_sum(S), Ew = wave_sum(E);
  if (p.k > 0) {
    // the finite elements that reach the threshold (masked ones are filled in by the join)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (pm[j] >= thr && pm[j] != -INFINITY) {
        float x[kPer];
        unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const float v = value(j, q, x);
          if (v >= thr && v != -INFINITY) {
            const int at = atomicAdd(&n_cand, 1);
            if (at < kMaxCand) cand[at] = alt_key(v, (p0 + j * kBlock + tid) * kPer + q);
          }
        }
      }
    }
  }
  __syncthreads();
  if (lane == 0) { red[wave] = Sw; red[4 + wave] = Ew; }
  uint64_t *keys = p.keys + ((int64_t)row * p.n_chunks + c) * p.k;
  const int n = n_cand;
  if (p.k > 0 && n <= kMaxCand) {
    rank_keys(cand, n, p.k, [&](int rank, uint64_t key) { keys[rank] = key; });
    for (int i = n + tid; i < p.k; i += kBlock) keys[i] = 0;
  } else if (p.k > 0) {
    // more equal or unevenly spread elements than fit: k rounds, each the
    // largest element of the registers below the one before
    uint64_t before = ~0ull;
    __syncthreads();
    for (int i = 0; i < p.k; ++i) {
      uint64_t best = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        float x[kPer];
        unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const float v = value(j, q, x);
          if (v == -INFINITY) continue;
          const uint64_t key = alt_key(v, (p0 + j * kBlock + tid) * kPer + q);
          if (key < before && key > best) best = key;
        }
      }
      best = wave_max_key(best);
      if (lane == 0) cand[wave] = best;
      __syncthreads();
      best = cand[0];
      for (int w = 1; w < kBlock / kWave; ++w) best = cand[w] > best ? cand[w] : best;
      before = best;
      if (tid == 0) keys[i] = best;
      __syncthreads();
    }
  }
  __syncthreads();
  if (tid == 0)
    p.sums[(int64_t)row * p.n_chunks + c] =
        make_float4(mx, ((red[0] + red[1]) + red[2]) + red[3], ((red[4] + red[5]) + red[6]) + red[7],
                    0.0f);
}

namespace {
struct JoinParams {
  int n_rows, V, R, k, n_chunks, tok_stride;
  int64_t row_stride;
  float invT, invT_low, scale;  // 1 / T and what its rounding left; log2(e) / T
  const void *X;
  const int32_t *tokens, *row_offset;
  const float4 *sums;
  const uint64_t *keys;
  float *logp, *entropy, *stats, *top_logp;
  int32_t *top_ids;
  int32_t *err;
};
}  // namespace

template <typename T>
__global__ __launch_bounds__(kBlock) void logprob_join_kernel(JoinParams p) {
  __shared__ float red[8];
  __shared__ uint64_t cand[kMaxCand];
  __shared__ uint64_t picked[64];
  __shared__ int n_cand;
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int row = blockIdx.x;
  const int used = rows_in_use(p.row_offset, p.R, p.n_rows);
  if (row == 0 && tid == 0 && p.row_offset != nullptr && p.row_offset[p.R] > p.n_rows)
    flag_error(p.err, kErrLength);
  if (row >= used) return;
  if (tid == 0) n_cand = 0;
  const float4 *sums = p.sums + (int64_t)row * p.n_chunks;
  float mx = -INFINITY;
  for (int c = tid; c < p.n_chunks; c += kBlock) mx = fmaxf(mx, sums[c].x);
  mx = block_max(mx, red);
  float S = 0.0f, E = 0.0f;
  for (int c = tid; c < p.n_chunks; c += kBlock) {
    const float4 s = sums[c];
    // a chunk of the type's lowest values: f is 0, and d only has to be finite
    const float d = fmaxf((s.x - mx) * p.scale, -1e4f), f = exp2_fast(d);
    if (s.y != 0.0f) {  // a chunk that is all masked has no sum
      S += s.y * f;
      E += f * (s.z + s.y * d);
    }
  }
  S = block_sum(S, red);
  E = block_sum(E, red);
  const bool ok = isfinite(mx) && isfinite(S) && S > 0.0f;
  const float logS = logf(S);
  const T *X = reinterpret_cast<const T *>(p.X) + (int64_t)row * p.row_stride;
  if (wave == 0) {
    const int tok = token_of_row(p.tokens, p.row_offset, p.R, p.tok_stride, row);
    if (lane == 0) {
      int bits = ok ? 0 : kErrNonFinite;
      if (p.logp != nullptr) {
        float lp = 0.0f;
        if (tok < -1 || tok >= p.V) {
          bits |= kErrToken;
          lp = NAN;
        } else if (tok >= 0) {
          const float d = Elem<T>::at(X, tok) - mx;
          lp = fmaf(d, p.invT, -logS);
        }
        p.logp[row] = ok ? lp : NAN;
      }
      if (p.entropy != nullptr) p.entropy[row] = ok ? logS - E * 0.6931471805599453f / S : NAN;
      if (p.stats != nullptr) {
        // S belongs to the exact max / T; the stored m is that rounded
        const float m = mx * p.invT;
        const float off = fmaf(mx, p.invT_low, fmaf(mx, p.invT, -m));
        p.stats[2 * (int64_t)row] = ok ? m : NAN;
        p.stats[2 * (int64_t)row + 1] = ok ? S + S * off : NAN;
      }
      if (bits) flag_error(p.err, bits);
    }
  }
  if (p.k == 0) return;

  // Threshold: the k-th largest of the chunks' q-th elements, q the least with
  // n_chunks q >= k ... for q = 1 the k-th largest head, else the least q-th one.
  const uint64_t *keys = p.keys + (int64_t)row * p.n_chunks * p.k;
  const int q = (p.k + p.n_chunks - 1) / p.n_chunks;
  uint64_t thr = 0;
  if (q > 1) {
    uint64_t low = ~0ull;
    for (int c = lane; c < p.n_chunks; c += kWave) {
      const uint64_t v = keys[(int64_t)c * p.k + q - 1];
      low = v < low ? v : low;
    }
    thr = ~wave_max_key(~low);
  } else {
    for (int c = tid; c < p.n_chunks && c < kMaxCand; c += kBlock) cand[c] = keys[(int64_t)c * p.k];
    if (tid == 0) picked[0] = 0;
    __syncthreads();
    // heads of all-masked chunks are 0 and equal: they leave picked[0] at 0
    rank_keys(cand, min(p.n_chunks, kMaxCand), p.k, [&](int rank, uint64_t key) {
      if (rank == p.k - 1) picked[0] = key;
    });
    __syncthreads();
    thr = picked[0];
  }
  __syncthreads();
  const int total = p.n_chunks * p.k;
  for (int i = tid; i < total; i += kBlock) {
    const uint64_t v = keys[i];
    if (v != 0 && v >= thr) {
      const int at = atomicAdd(&n_cand, 1);
      if (at < kMaxCand) cand[at] = v;
    }
  }
  __syncthreads();
  int n = n_cand;
  if (n <= kMaxCand) {
    rank_keys(cand, n, p.k, [&](int rank, uint64_t key) { picked[rank] = key; });
    n = min(n, p.k);
  } else {
    // unevenly spread chunks: k rounds over all keys
    uint64_t before = ~0ull;
    n = p.k;
    __syncthreads();
    for (int r = 0; r < p.k; ++r) {
      uint64_t best = 0;
      for (int i = tid; i < total; i += kBlock) {
        const uint64_t v = keys[i];
        if (v < before && v > best) best = v;
      }
      best = wave_max_key(best);
      if (lane == 0) cand[wave] = best;
      __syncthreads();
      best = cand[0];
      for (int w = 1; w < kBlock / kWave; ++w) best = cand[w] > best ? cand[w] : best;
      before = best;
      if (tid == 0) picked[r] = best;
      __syncthreads();
    }
  }
  __syncthreads();
  int32_t *ids = p.top_ids + (int64_t)row * p.k;
  float *tlp = p.top_logp + (int64_t)row * p.k;
  if (tid < n) {
    const uint64_t key = picked[tid];
    ids[tid] = ok ? key_index(key) : -1;
    tlp[tid] = ok ? fmaf(key_value(key) - mx, p.invT, -logS) : NAN;
  }
  // fewer than k unmasked: the lowest indices that are not among them follow.
  // n of the first k + n indices at most are taken, so k of them are not.
  if (n < p.k && wave == 0) {
    int at = n;
    for (int i0 = 0; i0 < p.k + n && at < p.k; i0 += kWave) {
      const int i = i0 + lane;
      bool is_free = i < p.V;
      for (int j = 0; j < n; ++j) is_free = is_free && key_index(picked[j]) != i;
      const uint64_t m = __ballot(is_free);
      const int mine = at + __popcll(m & ((1ull << lane) - 1));
      if (is_free && mine < p.k) {
        ids[mine] = ok ? i : -1;
        tlp[mine] = ok ? -INFINITY : NAN;
      }
      at += __popcll(m);
    }
  }
}

namespace {
struct GradParams {
  int n_rows, V, R, k, n_chunks, pieces_per_chunk, tok_stride;
  int64_t row_stride, dx_stride;
  float invT, invT_low;
  const void *X;
  const int32_t *tokens, *row_offset, *top_ids;
  const float *stats, *entropy, *g_logp, *g_entropy, *g_top;
  void *dX;
  int32_t *err;
};
__device__ __forceinline__ u32x4 pack16(const float *x, bf16_t *) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = (uint32_t)f32_to_bf16(x[2 * i]) | (uint32_t)f32_to_bf16(x[2 * i + 1]) << 16;
  return v;
}
__device__ __forceinline__ u32x4 pack16(const float *x, float *) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(x[i]);
  return v;
}
}  // namespace

// Gradient: one read of X and one write of dX, nothing kept between.  With
// d = x / T - m (two fused multiply-adds: the product's rounding would shift
// every probability) and p = 2^(d log2 e) / S an element's value is
//   -p (G + g_H (d - log S + H)) / T,  G the row's sum of incoming gradients,
// plus its own incoming gradients / T at the token and the alternatives.  Those
// k + 1 columns are looked up in a bit set of the chunk's 16-byte pieces, so a
// thread tests one bit per piece and almost never looks at the list.
template <typename T, int VPT>
__global__ __launch_bounds__(kBlock) void logprob_grad_kernel(GradParams p) {
  constexpr int kPer = Elem<T>::kPerVec;
  __shared__ int col[65];
  __shared__ float grad[65];
  __shared__ uint32_t marked[VPT * kBlock / 32];
  __shared__ float s_sum;
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const int row = blockIdx.x / p.n_chunks, c = blockIdx.x % p.n_chunks;
  const int used = rows_in_use(p.row_offset, p.R, p.n_rows);
  if (row == 0 && c == 0 && tid == 0 && p.row_offset != nullptr && p.row_offset[p.R] > p.n_rows)
    flag_error(p.err, kErrLength);
  if (row >= used) return;
  const int n_pieces = (p.V + kPer - 1) / kPer;
  const int p0 = c * p.pieces_per_chunk, p1 = min(p0 + p.pieces_per_chunk, n_pieces);
  const T *X = reinterpret_cast<const T *>(p.X) + (int64_t)row * p.row_stride;
  T *dX = reinterpret_cast<T *>(p.dX) + (int64_t)row * p.dx_stride;
  u32x4 raw[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j)
    raw[j] = ld_stream4(X + (int64_t)min(p0 + j * kBlock + tid, p1 - 1) * kPer);
  for (int i = tid; i < VPT * kBlock / 32; i += kBlock) marked[i] = 0;
  __syncthreads();
  if (tid < kWave) {
    int bits = 0;
    float sum = 0.0f;
    for (int i0 = 0; i0 <= p.k; i0 += kWave) {
      const int i = i0 + lane;  // 0: the token, i > 0: alternative i - 1
      int at = -1;
      float g = 0.0f;
      if (i0 == 0) {
        const int tok = p.g_logp == nullptr ? -1
                                            : token_of_row(p.tokens, p.row_offset, p.R, p.tok_stride, row);
        if (i == 0) {
          at = tok;
          if (tok < -1 || tok >= p.V) bits |= kErrToken;
          if (tok >= 0 && tok < p.V) g = p.g_logp[row];
        }
      }
      if (i > 0 && i <= p.k) {
        at = p.top_ids[(int64_t)row * p.k + i - 1];
        if (at < 0 || at >= p.V) bits |= kErrToken;
        else g = p.g_top[(int64_t)row * p.k + i - 1];
      }
      const bool valid = at >= 0 && at < p.V;
      sum += g;
      if (i <= p.k) {
        col[i] = valid ? at : -1;
        grad[i] = g;
        if (valid) {
          const int piece = at / kPer - p0;
          if (piece >= 0 && piece < p1 - p0) atomicOr(&marked[piece >> 5], 1u << (piece & 31));
        }
      }
    }
    sum = wave_sum(sum);
    if (lane == 0) s_sum = sum;
    const float S = p.stats[2 * (int64_t)row + 1], m = p.stats[2 * (int64_t)row];
    if (lane == 0 && c == 0 && !(isfinite(m) && isfinite(S) && S > 0.0f)) bits |= kErrNonFinite;
    if (bits) flag_error(p.err, bits);
  }
  __syncthreads();
  const float m = p.stats[2 * (int64_t)row], S = p.stats[2 * (int64_t)row + 1];
  const bool ok = isfinite(m) && isfinite(S) && S > 0.0f;
  const float gH = p.g_entropy != nullptr ? p.g_entropy[row] : 0.0f;
  const float H = p.g_entropy != nullptr ? p.entropy[row] : 0.0f;
  const float G = s_sum, logS = logf(S), r = -p.invT / S, base = G + gH * (H - logS);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int local = j * kBlock + tid, piece = p0 + local;
    if (piece >= p1) continue;
    float x[kPer], y[kPer];
    unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      // a masked logit has e = 0: its value and its d only have to be finite
      const float v = fmaxf(x[q], -1e30f);
      const float d = fmaf(v, p.invT_low, fmaf(v, p.invT, -m));
      const float e = exp2_fast(d * kLog2e);
      y[q] = e * r * fmaf(gH, fmaxf(d, -1e4f), base);
    }
    if (marked[local >> 5] >> (local & 31) & 1) {
      for (int i = 0; i <= p.k; ++i) {
        const int off = col[i] - piece * kPer;
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (off == q) y[q] += grad[i] * p.invT;
      }
    }
    if (!ok) {
#pragma unroll
      for (int q = 0; q < kPer; ++q) y[q] = 0.0f;
    }
    T *to = dX + (int64_t)piece * kPer;
    if ((piece + 1) * kPer <= p.V) {
      __builtin_nontemporal_store(pack16(y, (T *)nullptr), reinterpret_cast<u32x4 *>(to));
    } else {  // the last piece of an odd vocabulary
#pragma unroll
      for (int q = 0; q < kPer; ++q)
        if (piece * kPer + q < p.V) store_elem(to, q, y[q]);
    }
  }
}

namespace {

// Pieces per thread: the largest of 8, 4, 2 and 1 that still makes `want`
// workgroups; a call too small for that takes 1.
int pieces_per_thread(int n_rows, int V, int per, int want) {
  const int64_t pieces = (V + per - 1) / per;
  for (int vpt = 8; vpt > 1; vpt /= 2)
    if ((int64_t)n_rows * ((pieces + vpt * kBlock - 1) / (vpt * kBlock)) >= want) return vpt;
  return 1;
}
constexpr int kWant = 4 * kComputeUnits;

struct Split { int vpt, n_chunks, pieces_per_chunk; };
// chunks of equal size
Split split_of(int n_rows, int V, bool bf16) {
  const int per = bf16 ? 8 : 4, pieces = (V + per - 1) / per;
  Split s;
  s.vpt = pieces_per_thread(n_rows, V, per, kWant);
  s.n_chunks = (pieces + s.vpt * kBlock - 1) / (s.vpt * kBlock);
  s.pieces_per_chunk = (pieces + s.n_chunks - 1) / s.n_chunks;
  s.n_chunks = (pieces + s.pieces_per_chunk - 1) / s.pieces_per_chunk;
  return s;
}

}  // namespace

size_t logprobs_ws_bytes(int n_rows, int V, int k, bool bf16) {
  const Split s = split_of(n_rows, V, bf16);
  const size_t n = (size_t)n_rows * s.n_chunks;
  return kWsHeader + ws_align(n * 16) + ws_align(n * k * 8);
}

template <typename T, int VPT>
static void launch_chunk(const ChunkParams &c, hipStream_t stream) {
  DSPARK_LAUNCH("logprob_chunk", stream, (logprob_chunk_kernel<T, VPT>), (uint32_t)c.n_rows * c.n_chunks,
                kBlock, c);
}
template <typename T> static hipError_t launch_logprobs_t(const LogprobsLaunch &L, hipStream_t stream) {
  const Split s = split_of(L.n_rows, L.V, L.bf16);
  const size_t n = (size_t)L.n_rows * s.n_chunks;
  ChunkParams c{};
  c.n_rows = L.n_rows; c.V = L.V; c.R = L.R; c.k = L.k; c.n_chunks = s.n_chunks;
  c.pieces_per_chunk = s.pieces_per_chunk; c.row_stride = L.row_stride;
  c.scale = (float)(1.4426950408889634 / L.temp); c.X = L.X; c.row_offset = L.row_offset;
  c.sums = (float4 *)L.scratch;
  c.keys = (uint64_t *)((char *)L.scratch + ws_align(n * 16));
  switch (s.vpt) {
    case 8: launch_chunk<T, 8>(c, stream); break;
    case 4: launch_chunk<T, 4>(c, stream); break;
    case 2: launch_chunk<T, 2>(c, stream); break;
    default: launch_chunk<T, 1>(c, stream); break;
  }
  JoinParams j{};
  j.n_rows = L.n_rows; j.V = L.V; j.R = L.R; j.k = L.k; j.n_chunks = s.n_chunks;
  j.tok_stride = L.tok_stride; j.row_stride = L.row_stride; j.invT = (float)(1.0 / L.temp);
  j.invT_low = (float)(1.0 / L.temp - (double)j.invT); j.scale = c.scale; j.X = L.X;
  j.tokens = L.tokens; j.row_offset = L.row_offset; j.sums = c.sums; j.keys = c.keys;
  j.logp = L.logp; j.entropy = L.entropy; j.stats = L.stats; j.top_logp = L.top_logp;
  j.top_ids = L.top_ids; j.err = L.err;
  DSPARK_LAUNCH("logprob_join", stream, logprob_join_kernel<T>, L.n_rows, kBlock, j);
  return hipGetLastError();
}

hipError_t launch_logprobs(const LogprobsLaunch &L, hipStream_t stream) {
  return L.bf16 ? launch_logprobs_t<bf16_t>(L, stream) : launch_logprobs_t<float>(L, stream);
}

template <typename T, int VPT>
static void launch_grad(const GradParams &g, hipStream_t stream) {
  DSPARK_LAUNCH("logprob_grad", stream, (logprob_grad_kernel<T, VPT>), (uint32_t)g.n_rows * g.n_chunks,
                kBlock, g);
}
template <typename T>
static hipError_t launch_grad_t(const LogprobsGradLaunch &L, hipStream_t stream) {
  const Split s = split_of(L.n_rows, L.V, L.bf16);
  GradParams g{};
  g.n_rows = L.n_rows; g.V = L.V; g.R = L.R; g.k = L.k; g.n_chunks = s.n_chunks;
  g.pieces_per_chunk = s.pieces_per_chunk; g.tok_stride = L.tok_stride;
  g.row_stride = L.row_stride; g.dx_stride = L.dx_stride; g.invT = (float)(1.0 / L.temp);
  g.invT_low = (float)(1.0 / L.temp - (double)g.invT); g.X = L.X; g.tokens = L.tokens;
  g.row_offset = L.row_offset; g.top_ids = L.top_ids; g.stats = L.stats; g.entropy = L.entropy;
  g.g_logp = L.g_logp; g.g_entropy = L.g_entropy; g.g_top = L.g_top; g.dX = L.dX; g.err = L.err;
  switch (s.vpt) {
    case 8: launch_grad<T, 8>(g, stream); break;
    case 4: launch_grad<T, 4>(g, stream); break;
    case 2: launch_grad<T, 2>(g, stream); break;
    default: launch_grad<T, 1>(g, stream); break;
  }
  return hipGetLastError();
}

hipError_t launch_logprobs_backward(const LogprobsGradLaunch &L, hipStream_t stream) {
  return L.bf16 ? launch_grad_t<bf16_t>(L, stream) : launch_grad_t<float>(L, stream);
}

}  // namespace dspark
