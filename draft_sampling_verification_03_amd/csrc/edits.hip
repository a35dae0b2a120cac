// Edits of logit rows by their request's token history (penalties, biases, grammar
// masks) and their gradient; the histories' growth.
//
// A workgroup takes a chunk of the vocabulary and rows of one request.  What the history
// says of the chunk's tokens is counted in LDS, one word a token, by integer atomics
// (whose order does not matter):
//   bits 0..20   times generated
//   bit  21      in the prompt
//   bits 22..31  n_bias - i, i the first entry of the request's biases for the token; 0: none
// A thread owns the same 16 tokens of every row, so it keeps in a register which of them
// have a word at all, and it alone changes their words as the drafts before each row come
// to count: the rows need no barrier.  Nearly all of a row has no word and no mask, and
// passes through as it is; in place a line of it with neither is not even read.
//
// Bound: the rows in and out.  1152 rows of 151936 bf16, histories of up to 6000, a quarter
// masked (702 MB; counters: 380 MB fetched, 350 written): 151 us, 4.6 TB/s, of which 10 go
// to the counting and 10 to words, biases and drafts; the gradient of 544 rows of 129280
// (282 MB) 69 us; fp32 rows with histories of up to 120000 46 us, two thirds of them the
// counting (one LDS operation for 64 tokens, in each of the 16 chunks).  Masks in place, half
// of them dense, half sparse: 169 MB fetched and 172 written, for nearly every 128 bytes
// hold both kinds: 68 to 73 us (fp32: 117).  The 1152 rows in place 129 us (fp32: 162), the
// gradient 48.  One row: 7 us of latency.
#include <float.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kCountBits = 21, kBiasShift = 22;
constexpr uint32_t kCountMask = (1u << kCountBits) - 1, kPromptBit = 1u << kCountBits;
constexpr int kOwn = 16;  // tokens of a thread
// A part of a request's rows counts the history anew, so it has a row at least for so many
// of its tokens: histories of up to 120000 for 1 to 5 rows 61 us, 79 where every row was a part.
constexpr int kTokensARow = 4096;
constexpr int kRequestsX = 1 << 16;  // requests along the grid's first dimension

// The tokens [0, n) at p, spread over the workgroup in 16-byte pieces: load() brings the
// first of them on their way, each() calls f(token, index, mode) for all, -1 and what is
// wrong among them.  mode is a constant: whether the indexes of the wave's call are all
// below `border`, all from it on, or mixed.
enum Side { kBelow, kFrom, kMixed };
template <int kThreads, int kFlight> struct Tokens {
  const int32_t *p;
  int n, head, quads;
  int4 v[kFlight];
  __device__ __forceinline__ Tokens(const int32_t *at, int count) : p(at), n(count) {
    head = min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / 4);
    quads = (n - head) / 4;
  }
  __device__ __forceinline__ void load(int q0) {
    const int4 *mid = reinterpret_cast<const int4 *>(p + head);
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      const int q = q0 + i * kThreads;
      v[i] = make_int4(-1, -1, -1, -1);
      if (q < quads) v[i] = mid[q];
    }
  }
  __device__ __forceinline__ void load() { load(threadIdx.x); }
  template <typename F> __device__ __forceinline__ void each(int border, F f) {
    const int tid = threadIdx.x, tail = head + 4 * quads;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave) * kWave;
    auto quad = [&](const int4 &x, int at, auto mode) {
      f(x.x, at, mode);
      f(x.y, at + 1, mode);
      f(x.z, at + 2, mode);
      f(x.w, at + 3, mode);
    };
    for (int step = 0; step < quads; step += kFlight * kThreads) {
      if (step > 0) load(step + tid);
#pragma unroll
      for (int i = 0; i < kFlight; ++i) {
        const int q = step + i * kThreads, first = head + 4 * (q + wave), at = head + 4 * (q + tid);
        if (q + wave >= quads) break;
        if (first >= border) quad(v[i], at, std::integral_constant<Side, kFrom>());
        else if (first + 4 * kWave <= border) quad(v[i], at, std::integral_constant<Side, kBelow>());
        else quad(v[i], at, std::integral_constant<Side, kMixed>());
      }
    }
    const std::integral_constant<Side, kMixed> mixed;
    if (tid < head) f(p[tid], tid, mixed);
    if (tid < n - tail) f(p[tail + tid], tail + tid, mixed);
  }
};

// Element i of a piece, i known at compile time.
template <typename T> __device__ __forceinline__ float element(u32x4 v, int i) {
  if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
  else return __uint_as_float(v[i]);
}
template <typename T> __device__ __forceinline__ void set_element(u32x4 &v, int i, float x) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t h = __builtin_bit_cast(uint16_t, (__bf16)x);
    v[i / 2] = i & 1 ? h << 16 | (v[i / 2] & 0xFFFFu) : (v[i / 2] & 0xFFFF0000u) | h;
  } else {
    v[i] = __float_as_uint(x);
  }
}
// The piece with `none` (a whole dword of it) in the elements that `allowed` leaves out.
template <typename T> __device__ __forceinline__ u32x4 masked(u32x4 v, uint32_t allowed, uint32_t none) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t lo = allowed >> (2 * k) & 1 ? 0xFFFFu : 0;
      const uint32_t keep = lo | (allowed >> (2 * k + 1) & 1 ? 0xFFFF0000u : 0);
      v[k] = (v[k] & keep) | (none & ~keep);
    } else {
      v[k] = allowed >> k & 1 ? v[k] : none;
    }
  }
  return v;
}
// element i of a piece
template <typename T> __device__ __forceinline__ void store_piece(T *to, u32x4 v, int i) {
  if constexpr (sizeof(T) == 2) to[i].bits = __builtin_bit_cast(u16x8, v)[i];
  else to[i] = __builtin_bit_cast(floatx4, v)[i];
}

struct Rules {  // of one request
  float repetition, inverse, frequency, presence;
  const float *bias_end;  // entry n_bias of its biases
};

// x / r to within a little over half a step: the product with 1 / r, and what that is off
// by divided again.
__device__ __forceinline__ float divide(float x, const Rules &k) {
  const float q = x * k.inverse;
  const float better = __builtin_fmaf(__builtin_fmaf(-q, k.repetition, x), k.inverse, q);
  return __builtin_isfinite(q) ? better : q;
}
__device__ __forceinline__ float edited(float x, uint32_t w, const Rules &k) {
  if (w & (kCountMask | kPromptBit)) x = x > 0.0f ? divide(x, k) : x * k.repetition;
  const uint32_t n = w & kCountMask;
  x = x - k.frequency * (float)n;
  x = x - (n > 0 ? k.presence : 0.0f);
  if (w >> kBiasShift) x = x + *(k.bias_end - (w >> kBiasShift));
  return x;
}
__device__ __forceinline__ float edited_gradient(float g, float x, uint32_t w, const Rules &k) {
  if (w & (kCountMask | kPromptBit)) g = x > 0.0f ? divide(g, k) : g * k.repetition;
  return g;
}

// What a unit needs of its request, from as many arrays: a lane each, so that all of them
// are one load and one wait.
struct Request {
  int a, n;         // its rows [a, a + n)
  int len, prompt;  // its history
  Rules rules;
  int bits;
};
__device__ __forceinline__ Request request_of(const EditLaunch &L, int r) {
  const int lane = threadIdx.x & (kWave - 1);
  const int32_t *at = nullptr;
  auto from = [&](int i, const void *p, int add) {
    if (lane == i && p != nullptr) at = reinterpret_cast<const int32_t *>(p) + r + add;
  };
  from(0, L.row_offset, 0);
  from(1, L.row_offset, 1);
  from(2, L.hist_len, 0);
  from(3, L.prompt_len, 0);
  from(4, L.repetition, 0);
  from(5, L.frequency, 0);
  from(6, L.presence, 0);
  int v = lane == 4 ? __float_as_int(1.0f) : 0;
  if (at != nullptr) v = *at;
  auto get = [&](int i) { return __builtin_amdgcn_readlane(v, i); };
  Request q;
  q.a = r, q.n = 1, q.bits = 0;
  if (L.row_offset != nullptr) {
    q.a = get(0);
    const int b = get(1);
    const bool bad = q.a < 0 || b < q.a || b > L.n_rows;
    if (bad) q.bits |= kErrLength;
    q.n = bad ? 0 : b - q.a;
  }
  q.len = get(2), q.prompt = get(3);
  if (q.len < 0 || q.len > L.hist_stride) q.bits |= kErrLength, q.len = 0;
  if (q.prompt < 0 || q.prompt > q.len) q.bits |= kErrLength, q.prompt = 0;
  auto parameter = [&](int i, float lo, float hi, float none) {
    const float x = __int_as_float(get(i));
    if (x >= lo && x <= hi) return x;
    q.bits |= kErrNonFinite;
    return none;
  };
  q.rules.repetition = parameter(4, 1e-3f, 1e3f, 1.0f);
  q.rules.frequency = parameter(5, -FLT_MAX, FLT_MAX, 0.0f);
  q.rules.presence = parameter(6, -FLT_MAX, FLT_MAX, 0.0f);
  q.rules.inverse = 1.0f / q.rules.repetition;
  q.rules.bias_end = L.bias + ((int64_t)r + 1) * L.n_bias;
  return q;
}

}  // namespace

// A workgroup takes one (request, part of its rows, chunk), chunks innermost.  A chunk is
// not one stretch of the vocabulary but every so many of its spans, a span being what one
// load of a wave covers: the frequent tokens are the low ones, and this way every chunk
// has some of them to count and edit.  One unit and not several in turn: what the
// compiler would keep in registers from one to the next cost half of the waves.
// kCounts: whether histories, drafts or biases are given at all; kMask: whether masks are.
//
// The rows are a pipeline: row j + 1 is on its way while row j is edited and stored; in
// place, where the masks say what is to be read, those of row j + 2 too.  Its loads are
// all made, so that the compiler can count which of them a step waits for: where a piece
// is not wanted (past the vocabulary, in place where nothing changes) the lane reads the
// row's first piece, which all lanes share.
template <typename T, bool kGrad, bool kCounts, bool kMask, bool kInPlace, int kThreads>
__global__ __launch_bounds__(kThreads) void edit_kernel(EditLaunch L, unsigned chunks, unsigned parts) {
  constexpr int kPer = Elem<T>::kPerVec, kVecs = kOwn / kPer, kChunk = kThreads * kOwn;
  constexpr int kSpan = kWave * kPer;  // tokens that one load of a wave covers
  constexpr uint32_t kAll = (1u << kPer) - 1, kWhole = (1u << kOwn) - 1;
  constexpr bool kRaw = kGrad && kCounts;  // the raw logits too
  __shared__ __attribute__((aligned(16))) uint32_t word[kCounts ? kChunk : 4];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const bool raw_too = kRaw && L.repetition != nullptr;
  const T *source = reinterpret_cast<const T *>(kGrad ? L.G : L.X);
  const T *raw = raw_too ? reinterpret_cast<const T *>(L.X) : source;
  const int64_t stride = kGrad ? L.g_stride : L.row_stride, raw_stride = raw_too ? L.row_stride : stride;
  const unsigned chunk = blockIdx.x % chunks, unit = blockIdx.x / chunks;
  const unsigned r = unit / parts + blockIdx.y * kRequestsX;
  const int part = unit % parts;
  if (r >= (unsigned)L.R) return;
  const Request q = request_of(L, r);
  // every part counts the history anew, so a part has a row for so many of its tokens
  const int least = q.len / kTokensARow + 1, shared = min((int)parts, max(q.n / least, 1));
  const int a = q.a, j0 = part < shared ? (int)((int64_t)q.n * part / shared) : q.n;
  const int j1 = part < shared ? (int)((int64_t)q.n * (part + 1) / shared) : q.n;
  int bits = q.bits;
  if (j0 == j1) {
    if (bits && chunk == 0) flag_error(L.err, bits);
    return;
  }
  const int32_t *drafts = kCounts && L.drafts != nullptr ? L.drafts + (int64_t)r * L.gamma : nullptr;
  uint32_t has = 0;  // which of the thread's tokens have a word
  // vector u of the thread begins at token e(u); its bits are u * kPer on
  auto e = [&](int u) {
    return (int)(((u * (kThreads / kWave) + tid / kWave) * chunks + chunk) * kSpan) + lane * kPer;
  };
  // The chunk and word of a token: there are at most 1024 spans and 32 chunks, so span *
  // inverse / 65536 is off by less than 1024 / 65536 < 1 / chunks, and the quotient is right.
  const unsigned inverse = (65535 + chunks) / chunks;
  // change(word) where the token is this chunk's.
  auto with_word = [&](int v, auto change) __attribute__((always_inline)) {
    const unsigned span = (unsigned)v / kSpan, mine = __umul24(span, inverse) >> 16;
    if (__umul24(mine, chunks) + chunk == span && (unsigned)v < (unsigned)L.V)
      change(&word[mine * kSpan + (unsigned)v % kSpan]);
    // a token that is wrong is seen by every chunk and part; the first chunk reports it
    if (chunk == 0 && (unsigned)v + 1u > (unsigned)L.V) bits |= kErrToken;
  };
  // mask and draft of 64 rows, a row a lane (out of range: as they are found)
  int mask_of, draft_of;
  auto look_ahead = [&](int j) {
    const int row = j + lane;
    mask_of = draft_of = -1;
    if (kMask && row < j1) mask_of = L.mask_index != nullptr ? L.mask_index[a + row] : a + row;
    if (drafts != nullptr && row > j0 && row < j1 && row <= L.gamma) draft_of = drafts[row - 1];
  };
  auto check_ahead = [&]() {
    if (kMask && (mask_of < -1 || mask_of >= L.n_masks)) bits |= kErrLength, mask_of = -1;
    if (kCounts && draft_of != -1 && (unsigned)draft_of >= (unsigned)L.V) bits |= kErrToken, draft_of = -1;
  };
  struct Allowed { uint32_t v[kMask ? kVecs : 1]; };  // bytes of a mask as they come
  auto load_mask = [&](Allowed &o, int k) {
    if constexpr (kMask) {
      const int m = __builtin_amdgcn_readlane(mask_of, k);
      const uint8_t *mask = reinterpret_cast<const uint8_t *>(L.mask + (m < 0 ? 0 : m) * L.mask_stride);
#pragma unroll
      for (int u = 0; u < kVecs; ++u) o.v[u] = mask[e(u) < L.V ? e(u) / 8 : 0];
    }
  };
  auto bits_of = [&](const Allowed &o, int k) {
    if constexpr (!kMask) return kWhole;
    uint32_t all = 0;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) all |= (o.v[u] >> (e(u) & 7) & kAll) << (u * kPer);
    return __builtin_amdgcn_readlane(mask_of, k) < 0 ? kWhole : all;
  };
  // the thread's bit of row k's draft, 0 where another thread has it
  auto draft_bit = [&](int k) -> uint32_t {
    if (!kCounts || drafts == nullptr) return 0;
    const int v = __builtin_amdgcn_readlane(draft_of, k);  // in the vocabulary, or -1
    const unsigned span = (unsigned)v / kSpan, mine = __umul24(span, inverse) >> 16;
    if (v < 0 || mine * chunks + chunk != span) return 0;
    const unsigned at = mine * kSpan + (unsigned)v % kSpan;
    if (at / kPer % kThreads != (unsigned)tid) return 0;
    return 1u << (at / kPer / kThreads * kPer + at % kPer);
  };
  auto count = [&](uint32_t bit) {  // one of the thread's tokens is a draft before this row
    if constexpr (kCounts) {
      has |= bit;
      if (bit != 0) {
        const int i = __ffs(bit) - 1;
        word[(i / kPer * kThreads + tid) * kPer + i % kPer] += 1;
      }
    }
  };
  struct Row {
    u32x4 v[kVecs], raw[kRaw ? kVecs : 1];
    Allowed mask;
    uint32_t lines;  // in place, bit u: the line of vector u is written
  };
  // A piece that ends behind the row's last token is read whole: it is aligned, and so
  // within the page of memory that holds the token.
  auto load_piece = [&](const T *from, int u, bool wanted) {
    return *reinterpret_cast<const u32x4 *>(from + (wanted && e(u) < L.V ? e(u) : 0));
  };
  // In place the 128 bytes of eight lanes are written whole or not at all: in part they cost
  // more than the bytes they save (masks in place: 136 MB written in 84 us, 172 in 73).  A
  // vote of the whole wave, so never behind a condition of a lane; made once for a row, as
  // it is loaded, and kept until it is stored: what is stored is what was loaded.
  auto line_changes = [&](int u, uint32_t al, uint32_t mk) {
    constexpr int kLine = 8;
    const uint64_t change = __ballot(e(u) < L.V && (al != kAll || mk != 0));
    return (change >> (lane & (kWave - kLine)) & ((1u << kLine) - 1)) != 0;
  };
  auto load_row = [&](Row &o, int j, uint32_t allowed, uint32_t marked) {
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t al = allowed >> (u * kPer) & kAll, mk = marked >> (u * kPer) & kAll;
      const bool line = !kInPlace || line_changes(u, al, mk);
      if constexpr (kInPlace) o.lines = (u == 0 ? 0 : o.lines) | (line ? 1u << u : 0);
      o.v[u] = load_piece(source + (a + j) * stride, u, line && (!kInPlace || al != 0));
    }
  };
  auto load_raw = [&](Row &o, int j, uint32_t marked) {
    if constexpr (kRaw)
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        o.raw[u] = load_piece(raw + (a + j) * raw_stride, u, raw_too && (marked >> (u * kPer) & kAll) != 0);
  };
  auto finish = [&](const Row &in, int j, uint32_t allowed, uint32_t marked) {
    T *to = reinterpret_cast<T *>(L.out) + (a + j) * L.out_stride;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t al = allowed >> (u * kPer) & kAll, mk = marked >> (u * kPer) & kAll;
      u32x4 out = in.v[u];
      if constexpr (kCounts) {
        const uint32_t edit = !kGrad || raw_too ? mk & al : 0;
        if (edit != 0) {
          uint32_t w[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) w[i] = word[(u * kThreads + tid) * kPer + i];
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (edit >> i & 1) {
              float x = element<T>(out, i);
              if constexpr (kGrad) x = edited_gradient(x, element<T>(in.raw[u], i), w[i], q.rules);
              else x = edited(x, w[i], q.rules);
              set_element<T>(out, i, x);
            }
        }
      }
      if (kMask && al != kAll)
        out = masked<T>(out, al, kGrad ? 0 : sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u);
      const bool stored = !kInPlace || (in.lines >> u & 1);
      if (e(u) >= L.V || !stored) continue;
      if (e(u) + kPer <= L.V) {
        *reinterpret_cast<u32x4 *>(to + e(u)) = out;
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (e(u) + i < L.V) store_piece<T>(to + e(u), out, i);
      }
    }
  };

  // everything that does not wait for the words is on its way before them
  Tokens<kThreads, 4> past(L.history + (int64_t)r * L.hist_stride, q.len);
  Tokens<kThreads, 1> ids(L.bias_ids + (int64_t)r * L.n_bias, L.n_bias);
  Tokens<kThreads, 1> before(drafts, drafts != nullptr ? min(j0, L.gamma) : 0);
  Row even, odd;
  if (kCounts) ids.load();
  if (kCounts) past.load();
  if (kCounts) before.load();
  look_ahead(j0);
  if (!kInPlace) load_row(even, j0, 0, 0);
  if (kCounts) {
#pragma unroll
    for (int i = 0; i < kOwn / 4; ++i)
      reinterpret_cast<uint4 *>(word)[i * kThreads + tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (L.n_bias > 0) {
      ids.each(0, [&](int v, int i, auto) {
        with_word(v, [&](uint32_t *w) { atomicMax(w, (uint32_t)(L.n_bias - i) << kBiasShift); });
      });
      __syncthreads();
    }
    past.each(q.prompt, [&](int v, int i, auto mode) {
      with_word(v, [&](uint32_t *w) {
        if (mode == kBelow || (mode == kMixed && i < q.prompt)) atomicOr(w, kPromptBit);
        else atomicAdd(w, 1u);
      });
    });
    before.each(0, [&](int v, int, auto) { with_word(v, [&](uint32_t *w) { atomicAdd(w, 1u); }); });
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
      has |= (word[(i / kPer * kThreads + tid) * kPer + i % kPer] != 0 ? 1u : 0u) << i;
  }
  for (int jb = j0; jb < j1; jb += kWave) {
    const int last = min(j1 - jb, kWave) - 1;
    if (jb > j0) look_ahead(jb);
    check_ahead();
    count(draft_bit(0));
    Allowed ahead;         // in place: the masks of the row after next
    uint32_t al = kWhole;  // and what this row allows
    if constexpr (kInPlace) {
      Allowed first;
      load_mask(first, 0);
      load_mask(ahead, min(1, last));
      al = bits_of(first, 0);
      load_row(even, jb, al, has);
    } else {
      if (jb > j0) load_row(even, jb, 0, 0);
      load_mask(even.mask, 0);
    }
    load_raw(even, jb, has);
    auto step = [&](const Row &now, Row &next, int k) {
      const int k1 = min(k + 1, last);
      const uint32_t bit = k < last ? draft_bit(k1) : 0;
      uint32_t next_al = kWhole;
      if constexpr (kInPlace) {
        next_al = bits_of(ahead, k1);
        load_mask(ahead, min(k + 2, last));
      } else {
        load_mask(next.mask, k1);
      }
      load_row(next, jb + k1, next_al, has | bit);
      load_raw(next, jb + k1, has | bit);
      if constexpr (!kInPlace) al = bits_of(now.mask, k);
      finish(now, jb + k, al, has);
      count(bit);
      al = next_al;
    };
    for (int k = 0; k <= last; k += 2) {
      step(even, odd, k);
      if (k < last) step(odd, even, k + 1);
    }
  }
  // every chunk sees what is wrong; the first of them reports it
  if (bits && chunk == 0) flag_error(L.err, bits);
}

// One workgroup a request: 2 us for a round's tokens, but a prompt of 100000 takes 48 and one
// of a million 872.
__global__ __launch_bounds__(kBlock) void history_append_kernel(HistoryLaunch L) {
  const int r = blockIdx.x, tid = threadIdx.x;
  const int len = L.hist_len[r];
  int64_t from = (int64_t)r * L.width, n = L.width;
  bool bad = len < 0 || len > L.hist_stride;
  if (L.n_acc != nullptr) {
    const int acc = L.n_acc[r];
    bad = bad || acc < -1 || acc >= L.width;
    n = (int64_t)acc + 1;
  }
  if (L.row_offset != nullptr) {
    const int a = L.row_offset[r], b = L.row_offset[r + 1];
    bad = bad || a < 0 || b < a;
    if (L.n_acc != nullptr) {  // the rows that the round has
      bad = bad || n > (int64_t)b - a;
    } else {
      bad = bad || b > L.n_tokens;
      from = a;
      n = (int64_t)b - a;
    }
  }
  bad = bad || len + n > L.hist_stride;
  __syncthreads();  // every thread has the length before it changes
  if (bad) n = 0;
  if (tid == 0) {
    if (bad) flag_error(L.err, kErrLength);
    L.hist_len_out[r] = len + (int)n;
    if (n > 0 && L.prompt_len != nullptr) L.prompt_len[r] = len + (int)n;
  }
  int32_t *to = L.history + (int64_t)r * L.hist_stride + len;
  for (int64_t i = tid; i < n; i += kBlock) to[i] = L.tokens[from + i];
}

// ----------------------------------------------------------------- launches
hipError_t launch_edit(const EditLaunch &L, hipStream_t stream) {
  const bool counts = L.history != nullptr || L.drafts != nullptr || L.n_bias > 0;
  auto go = [&](auto type, auto grad, auto has_counts, auto has_mask, auto in_place) {
    using T = decltype(type);
    constexpr bool kGrad = decltype(grad)::value, kCounts = decltype(has_counts)::value;
    constexpr bool kMask = decltype(has_mask)::value, kInPlace = decltype(in_place)::value;
    // 256 threads count a history twice as often: 149 us for 152 (1152 rows of 151936,
    // histories of up to 6000), but 66 for 47 (histories of up to 120000); 1024: 170 and 54
    constexpr int kThreads = 512;
    const unsigned chunks = (L.V + kThreads * kOwn - 1) / (kThreads * kOwn);
    const unsigned along = L.R < kRequestsX ? L.R : kRequestsX, base = along * chunks;  // <= 2^21
    const unsigned most = (L.n_rows + L.R - 1) / L.R;
    // About 4 rows a part, 2 where there is nothing to count: requests have 1 to 17 rows,
    // and the last workgroups end together.  1152 rows: 9 a part 166 us, 4 152, 3 159, 2 175;
    // with nothing to count 147, 137, 131, 125.  Then enough to fill the chip, and no
    // more workgroups than a launch can have (2^32 threads).
    unsigned parts = (most + 1) / (kCounts || kInPlace ? 4 : 2);
    if (parts * base < 4 * kComputeUnits) parts = (4 * kComputeUnits + base - 1) / base;
    if (parts > (1u << 22) / base) parts = (1u << 22) / base;
    if (parts > most) parts = most;
    if (parts < 1) parts = 1;
    const dim3 grid(base * parts, (L.R + kRequestsX - 1) / kRequestsX);
    DSPARK_LAUNCH(kGrad ? "edit_logits_backward" : "edit_logits", stream,
                  (edit_kernel<T, kGrad, kCounts, kMask, kInPlace, kThreads>), grid, kThreads, L, chunks,
                  parts);
  };
  // run time to compile time, one condition after another
  auto on = [](bool b, auto f) {
    if (b) f(std::true_type());
    else f(std::false_type());
  };
  auto with = [&](auto type) {
    on(L.G != nullptr, [&](auto grad) {
      on(counts, [&](auto has_counts) {
        on(L.mask != nullptr, [&](auto has_mask) {
          on(L.out == (L.G != nullptr ? L.G : L.X),
             [&](auto in_place) { go(type, grad, has_counts, has_mask, in_place); });
        });
      });
    });
  };
  if (L.bf16) with(bf16_t());
  else with(float());
  return hipGetLastError();
}

hipError_t launch_history_append(const HistoryLaunch &L, hipStream_t stream) {
  DSPARK_LAUNCH("history_append", stream, history_append_kernel, L.R, kBlock, L);
  return hipGetLastError();
}

}  // namespace dspark
