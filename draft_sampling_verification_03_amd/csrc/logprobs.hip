// Log probabilities of given tokens, entropy and the top alternatives of logit
// rows, and their gradient.
//
// Forward, two launches.  logprob_chunk_kernel: one workgroup takes a chunk of
// one row and keeps it in registers (every load in flight at once), so the row
// is read from memory once; from the registers come the chunk's maximum, then
//   S = sum 2^u, E = sum 2^u u, u = (x - max) log2(e) / T   (no running rescale)
// and the maximum of every 128 bytes.  logprob_join_kernel: one workgroup a row
// joins the chunks by their maxima,
//   log S, entropy = log S - E ln 2 / S, logp = (x_t - max) / T - log S,
// and finds the alternatives among the 128-byte lines: a threshold that at least k
// of the lines' maxima reach (and hardly more), those lines read again, and their
// elements that reach it ranked by counting.  So the alternatives cost the pass
// over the row one comparison of maxima, and no element is looked at twice but
// those of some 40 lines.  Where more lines or elements reach it than are kept,
// the threshold is raised by halving the range of values: 504 rows of 1021 bf16,
// k = 64, 19 us against 68 for ranking all 1021 and 28 for sorting them.
//
// Bound: one read of the logits.  1152 rows of 151936 bf16 with 20 alternatives (350
// MB): chunks 66 us (5.3 TB/s), join 16; 224 of 129277 fp32, mostly masked, 8
// alternatives: 22 + 8 us.  A top k in every chunk, the plainer way, made the chunks
// 124 us.  One row: 3 + 8 us, all of it latency.
#include <limits.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

// Elements of a row that are ranked: counting is one step a key, so 256 take about
// as long as the halving that would thin them (k = 64, V = 8000 fp32: 14 us, with
// 128 here 18).
constexpr int kMaxCand = 256;
constexpr int kLine = 8;        // pieces of 16 bytes in a line
constexpr int kMaxLines = 128;  // lines of a row that are read again
constexpr int kHeld = 32;       // lines' maxima a thread: V = 262144 fp32 has 8192 lines

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

// Maximum of three; the instruction takes any values, where fmaxf spends one more
// on each operand that might be a signalling NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
// Maximum of a 16-byte piece.
__device__ __forceinline__ float piece_max(const u32x4 &v, bf16_t *) {
  float x[8];
  unpack16(v, (bf16_t *)nullptr, x);
  return max3(max3(x[0], x[1], x[2]), max3(x[3], x[4], x[5]), max3(x[6], x[7], -INFINITY));
}
__device__ __forceinline__ float piece_max(const u32x4 &v, float *) {
  return max3(__uint_as_float(v[0]), __uint_as_float(v[1]),
              max3(__uint_as_float(v[2]), __uint_as_float(v[3]), -INFINITY));
}
// Maximum over the eight lanes of a line.
__device__ __forceinline__ float eight_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true)));
  return fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true)));
}
// Two bf16 or one fp32 minus infinity.
__device__ __forceinline__ uint32_t masked_word(bf16_t *) { return 0xFF80FF80u; }
__device__ __forceinline__ uint32_t masked_word(float *) { return 0xFF800000u; }
// A piece whose elements from n on are masked.
template <typename T> __device__ __forceinline__ u32x4 keep_first(u32x4 v, int n) {
  constexpr int kIn = 4 / (int)sizeof(T);  // elements of a word
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - i * kIn;
    if (left <= 0) v[i] = masked_word((T *)nullptr);
    else if (left < kIn) v[i] = (v[i] & 0xFFFFu) | 0xFF800000u;
  }
  return v;
}

// The row's request: the number of rho in [1, R) with row_offset[rho] <= row
// (the offsets do not decrease), 64 of them a ballot.  All R are looked at, so a row
// costs R / 64 dependent steps: two for the 128 requests of a round.
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
#pragma unroll 8
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
  float4 *sums;   // [n_rows][n_chunks]: (max x, S, E, unused)
  float *lines;   // [n_rows][n_chunks][kBlock / kLine][VPT]: maximum of each line
};

}  // namespace

template <typename T, int VPT>
__global__ __launch_bounds__(kBlock) void logprob_chunk_kernel(ChunkParams p) {
  constexpr int kPer = Elem<T>::kPerVec;
  __shared__ float red[8];
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

  // past the chunk or the vocabulary: masked
  if (p1 - p0 < VPT * kBlock) {  // uniform
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      raw[j] = p0 + j * kBlock + tid < p1 ? raw[j] : u32x4(masked_word((T *)nullptr));
  }
  if (p1 == n_pieces && p.V % kPer != 0) {
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      if (p0 + j * kBlock + tid == p1 - 1) raw[j] = keep_first<T>(raw[j], p.V % kPer);
  }
  // maxima: of the pieces, of the lines (8 lanes), of the chunk
  float tm = -INFINITY, line = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    float m = piece_max(raw[j], (T *)nullptr);
    tm = fmaxf(tm, m);
    if (p.k > 0) {
      m = eight_max(m);
      if ((lane & (kLine - 1)) == j) line = m;  // lane j of the eight writes line j
    }
  }
  if (p.k > 0 && (lane & (kLine - 1)) < VPT)
    p.lines[((int64_t)row * p.n_chunks + c) * (kBlock / kLine * VPT) + tid / kLine * VPT +
            (lane & (kLine - 1))] = line;
  const float wm = wave_max(tm);
  if (lane == 0) red[wave] = wm;
  __syncthreads();
  const float mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));

  float S = 0.0f, E = 0.0f;
  if (mx != -INFINITY) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float x[kPer];
      unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const float u = (x[q] - mx) * p.scale, e = exp2_fast(u);
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
      for (int q = 0; q < kPer; ++q)
        if (x[q] != x[q]) S = x[q];
    }
  }
  const float Sw = wave_sum(S), Ew = wave_sum(E);
  __syncthreads();  // every wave has read the maxima
  if (lane == 0) { red[wave] = Sw; red[4 + wave] = Ew; }
  __syncthreads();
  if (tid == 0)
    p.sums[(int64_t)row * p.n_chunks + c] =
        make_float4(mx, ((red[0] + red[1]) + red[2]) + red[3], ((red[4] + red[5]) + red[6]) + red[7],
                    0.0f);
}

namespace {
struct JoinParams {
  int n_rows, V, R, k, n_chunks, pieces_per_chunk, vpt, tok_stride;
  int64_t row_stride;
  float invT, invT_low, scale;  // 1 / T and what its rounding left; log2(e) / T
  const void *X;
  const int32_t *tokens, *row_offset;
  const float4 *sums;
  const float *lines;
  float *logp, *entropy, *stats, *top_logp;
  int32_t *top_ids;
  int32_t *err;
};

// Sum over the workgroup of a count that is the same in all lanes of a wave; two
// halves of the scratch in turn, so that one barrier is enough.
__device__ __forceinline__ int block_count(int v, int *scratch, int &turn) {
  turn ^= 4;
  if ((threadIdx.x & (kWave - 1)) == 0) scratch[turn + threadIdx.x / kWave] = v;
  __syncthreads();
  return scratch[turn] + scratch[turn + 1] + scratch[turn + 2] + scratch[turn + 3];
}

// Floats as unsigned integers in the same order, and back.
__device__ __forceinline__ uint32_t ordered(float x) { return (uint32_t)(alt_key(x, 0) >> 32); }
__device__ __forceinline__ float from_ordered(uint32_t o) { return key_value((uint64_t)o << 32); }

}  // namespace

template <typename T>
__global__ __launch_bounds__(kBlock) void logprob_join_kernel(JoinParams p) {
  __shared__ float red[8];
  __shared__ uint64_t cand[kMaxCand];
  __shared__ uint64_t picked[64];
  __shared__ int list[kMaxLines];
  __shared__ int n_cand, n_list;
  __shared__ int counts[8];
  const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
  const int row = blockIdx.x;
  const int used = rows_in_use(p.row_offset, p.R, p.n_rows);
  if (row == 0 && tid == 0 && p.row_offset != nullptr && p.row_offset[p.R] > p.n_rows)
    flag_error(p.err, kErrLength);
  if (row >= used) return;
  if (tid == 0) n_cand = n_list = 0;
  const T *X = reinterpret_cast<const T *>(p.X) + (int64_t)row * p.row_stride;
  // everything that the row needs is asked for at once: a chunk's sums a thread,
  // the lines' maxima, the token and its logit
  constexpr int kPer = Elem<T>::kPerVec;
  const int n_pieces = (p.V + kPer - 1) / kPer;
  const int per_chunk = kBlock / kLine * p.vpt, n_lines = p.k > 0 ? p.n_chunks * per_chunk : 0;
  const float4 sum = tid < p.n_chunks ? p.sums[(int64_t)row * p.n_chunks + tid]
                                      : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
  float held[kHeld];
  const float *lines = p.lines + (int64_t)row * n_lines;
#pragma unroll
  for (int b = 0; b < kHeld; b += 8) {
#pragma unroll
    for (int i = b; i < b + 8; ++i) held[i] = -INFINITY;
    if (b * kBlock < n_lines) {  // uniform
#pragma unroll
      for (int i = b; i < b + 8; ++i) {
        const float m = lines[min(i * kBlock + tid, n_lines - 1)];
        held[i] = i * kBlock + tid < n_lines ? m : -INFINITY;
      }
    }
  }
  int tok = -1;
  float x_tok = 0.0f;
  if (wave == 0) {
    tok = token_of_row(p.tokens, p.row_offset, p.R, p.tok_stride, row);
    if (tok >= 0 && tok < p.V) x_tok = Elem<T>::at(X, tok);
  }
  const float mx = block_max(sum.x, red);
  float S = 0.0f, E = 0.0f;
  {
    // a chunk of the type's lowest values: f is 0, and d only has to be finite
    const float d = fmaxf((sum.x - mx) * p.scale, -1e4f), f = exp2_fast(d);
    if (sum.y != 0.0f) {  // a chunk that is all masked has no sum
      S = sum.y * f;
      E = f * (sum.z + sum.y * d);
    }
  }
  S = wave_sum(S);
  E = wave_sum(E);
  if (lane == 0) { red[wave] = S; red[4 + wave] = E; }
  __syncthreads();
  S = ((red[0] + red[1]) + red[2]) + red[3];
  E = ((red[4] + red[5]) + red[6]) + red[7];
  const bool ok = isfinite(mx) && isfinite(S) && S > 0.0f;
  const float logS = logf(S);
  if (tid == 0) {
    int bits = ok ? 0 : kErrNonFinite;
    if (p.logp != nullptr) {
      float lp = 0.0f;
      if (tok < -1 || tok >= p.V) {
        bits |= kErrToken;
        lp = NAN;
      } else if (tok >= 0) {
        lp = fmaf(x_tok - mx, p.invT, -logS);
      }
      p.logp[row] = ok ? lp : NAN;
    }
    if (p.entropy != nullptr) p.entropy[row] = ok ? logS - E * 0.6931471805599453f / S : NAN;
    if (p.stats != nullptr) {
      // S belongs to the exact max / T; the stored m is that rounded, which is much of
      // an exponent where logits are large
      const float m = mx * p.invT;
      const float off = fmaf(mx, p.invT_low, fmaf(mx, p.invT, -m));
      p.stats[2 * (int64_t)row] = ok ? m : NAN;
      p.stats[2 * (int64_t)row + 1] = ok ? S * expf(off) : NAN;
    }
    if (bits) flag_error(p.err, bits);
  }
  if (p.k == 0) return;

  // Threshold.  The lanes hold different lines, so with the ceil(k / 4)-th largest
  // of each wave's lanes at least k lines reach the least of the four.
  float left = -INFINITY, thr = -INFINITY;
#pragma unroll
  for (int b = 0; b < kHeld; b += 8) {
    if (b * kBlock >= n_lines) continue;  // uniform
#pragma unroll
    for (int i = b; i < b + 8; ++i) left = fmaxf(left, held[i]);
  }
  uint64_t out = 0;  // lanes taken
  for (int i = 0; i < (p.k + 3) / 4; ++i) {
    thr = wave_max(left);
    const uint64_t at = __ballot(left == thr) & ~out;
    if (at == 0) { thr = -INFINITY; break; }  // the row has a NaN
    const uint64_t one = at & (~at + 1);
    out |= one;
    if (one >> lane & 1) left = -INFINITY;
  }
  __syncthreads();  // the sums are read
  if (lane == 0) red[wave] = thr;
  __syncthreads();
  thr = fminf(fminf(red[0], red[1]), fminf(red[2], red[3]));
  // the lines that reach it (masked elements are filled in at the end)
  auto gather = [&](bool strictly) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kHeld; b += 8) {
      if (b * kBlock >= n_lines) continue;  // uniform
#pragma unroll
      for (int i = b; i < b + 8; ++i) {
        const float m = held[i];
        if (m != -INFINITY && (strictly ? m > thr : m >= thr)) {
          const int at = atomicAdd(&n_list, 1);
          if (at < kMaxLines) list[at] = i * kBlock + tid;
        }
      }
    }
    __syncthreads();
  };
  gather(false);
  int turn = 0;
  // Raises thr by halving the range of values until count(thr) is from k to most;
  // where equal values leave no such threshold, to the k-th largest, and false.
  // Where thr is the maximum already it counts not once, so it passes no barrier.
  auto halve = [&](auto count, int most) __attribute__((always_inline)) {
    uint32_t lo = ordered(thr), hi = ordered(mx);
    bool found = false;
    while (lo < hi && !found) {  // at least k reach lo, fewer than k pass hi
      const uint32_t mid = lo + (hi - lo + 1) / 2;
      const int n = count(from_ordered(mid));
      if (n >= p.k) lo = mid;
      else hi = mid - 1;
      found = n >= p.k && n <= most;
    }
    thr = from_ordered(lo);
    return found;
  };
  bool tied = false;  // more share the threshold than are read again or ranked
  if (n_list > kMaxLines) {
    // uneven rows
    auto lines_at = [&](float t) __attribute__((always_inline)) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) n += __popcll(__ballot(held[i] >= t));
      return block_count(n, counts, turn);
    };
    tied = !halve(lines_at, kMaxLines);
    __syncthreads();  // every wave has read n_list
    if (tid == 0) n_list = 0;
    __syncthreads();
    gather(tied);  // strictly: fewer than k
  }
  // their elements: eight threads a line, at most four pieces a thread
  const int n_here = n_list;
  constexpr int kRounds = kMaxLines * kLine / kBlock;
  u32x4 raw[kRounds];
  int first[kRounds];  // index of the piece's first element, V: none
#pragma unroll
  for (int j = 0; j < kRounds; ++j) {
    const int i = (j * kBlock + tid) / kLine;
    first[j] = p.V;
    raw[j] = u32x4(masked_word((T *)nullptr));
    if (i < n_here) {
      const int id = list[i], c = id / per_chunk, in = id % per_chunk;
      const int local = in % p.vpt * kBlock + in / p.vpt * kLine + (tid & (kLine - 1));
      const int piece = c * p.pieces_per_chunk + local;
      if (local < p.pieces_per_chunk && piece < n_pieces) {
        first[j] = piece * kPer;
        raw[j] = *reinterpret_cast<const u32x4 *>(X + (int64_t)piece * kPer);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kRounds; ++j)
    if (first[j] + kPer > p.V) raw[j] = keep_first<T>(raw[j], p.V - first[j]);
  auto collect = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kRounds; ++j) {
      if (j * kBlock / kLine >= n_here) continue;  // uniform
      float x[kPer];
      unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const bool take = x[q] != -INFINITY && (tied ? x[q] > thr : x[q] >= thr);
        const uint64_t takers = __ballot(take);
        if (takers == 0) continue;  // uniform
        int at = 0;
        if (lane == 0) at = atomicAdd(&n_cand, __popcll(takers));
        at = __shfl(at, 0) + __popcll(takers & ((1ull << lane) - 1));
        if (take && at < kMaxCand) cand[at] = alt_key(x[q], first[j] + q);
      }
    }
    __syncthreads();
  };
  collect();
  if (n_cand > kMaxCand) {
    // fewer lines than alternatives, or many large elements a line
    auto reach = [&](float t) __attribute__((always_inline)) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < kRounds; ++j) {
        if (j * kBlock / kLine >= n_here) continue;  // uniform
        float x[kPer];
        unpack16(raw[j], (T *)nullptr, x);
#pragma unroll
        for (int q = 0; q < kPer; ++q) n += __popcll(__ballot(x[q] >= t));
      }
      return block_count(n, counts, turn);
    };
    tied = !halve(reach, kMaxCand);
    __syncthreads();  // every wave has read n_cand
    if (tid == 0) n_cand = 0;
    __syncthreads();
    collect();
  }
  int n = n_cand;
  rank_keys(cand, n, p.k, [&](int rank, uint64_t key) { picked[rank] = key; });
  n = min(n, p.k);
  __syncthreads();
  int32_t *ids = p.top_ids + (int64_t)row * p.k;
  float *tlp = p.top_logp + (int64_t)row * p.k;
  if (tid < n) {
    const uint64_t key = picked[tid];
    ids[tid] = ok ? key_index(key) : -1;
    tlp[tid] = ok ? fmaf(key_value(key) - mx, p.invT, -logS) : NAN;
  }
  // Too few: elements of the value that so many share follow by index, then
  // masked ones; the row is read in order until there are enough.
  for (int pass = tied ? 0 : 1; pass < 2; ++pass) {
    const float fill = pass == 0 ? thr : -INFINITY;
    const float lp = ok ? fmaf(fill - mx, p.invT, -logS) : NAN;
    for (int t = 0; t < n_pieces && n < p.k; t += kBlock) {
      const int piece = t + tid;
      float x[kPer];
      int mine = 0;
      if (piece < n_pieces) {
        unpack16(*reinterpret_cast<const u32x4 *>(X + (int64_t)piece * kPer), (T *)nullptr, x);
#pragma unroll
        for (int q = 0; q < kPer; ++q) mine += piece * kPer + q < p.V && x[q] == fill;
      }
      float total;
      int at = n + (int)block_exclusive_scan((float)mine, red, &total);
      if (mine > 0) {
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (piece * kPer + q < p.V && x[q] == fill) {
            if (at < p.k) {
              ids[at] = ok ? piece * kPer + q : -1;
              tlp[at] = lp;
            }
            ++at;
          }
      }
      n += (int)total;
    }
  }
  // a row without statistics may have neither
  if (!ok) {
    for (int i = n + tid; i < p.k; i += kBlock) {
      ids[i] = -1;
      tlp[i] = NAN;
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
// thread tests one bit per piece and almost never looks at the list.  Bound: the
// bytes; 1088 rows of 151936 bf16 (661 MB read and written) take 136 us, 4.85 TB/s,
// where a plain copy reaches 5.1; 39 of 129277 fp32 with 10 alternatives 10 us.
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
      // A masked logit has e = 0 and its d only has to be finite.  Of -infinity the sum is
      // -infinity or (times an invT_low of 0 or below) NaN, and the maximum takes the
      // other operand for either; a row with a NaN has no statistics.
      const float d = fmaxf(fmaf(x[q], p.invT_low, fmaf(x[q], p.invT, -m)), -1e4f);
      const float e = exp2_fast(d * kLog2e);
      y[q] = e * r * fmaf(gH, d, base);
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

static size_t lines_of(const Split &s) { return (size_t)s.n_chunks * (kBlock / kLine) * s.vpt; }

size_t logprobs_ws_bytes(int n_rows, int V, int k, bool bf16) {
  const Split s = split_of(n_rows, V, bf16);
  return kWsHeader + ws_align((size_t)n_rows * s.n_chunks * 16) +
         (k > 0 ? ws_align((size_t)n_rows * lines_of(s) * 4) : 0);
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
  c.lines = (float *)((char *)L.scratch + ws_align(n * 16));
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
  j.tokens = L.tokens; j.row_offset = L.row_offset; j.sums = c.sums; j.lines = c.lines;
  j.pieces_per_chunk = s.pieces_per_chunk; j.vpt = s.vpt;
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
