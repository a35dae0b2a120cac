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
// passes through as it is; in place it is not even read.
#include <float.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kCountBits = 21, kBiasShift = 22;
constexpr uint32_t kCountMask = (1u << kCountBits) - 1, kPromptBit = 1u << kCountBits;
constexpr int kOwn = 16;  // tokens of a thread

// f(token, index) for the tokens [0, n) at p, spread over the workgroup; -1 is skipped,
// what lies outside the vocabulary sets *bits.  16-byte loads, four of them in flight.
template <int kThreads, typename F>
__device__ __forceinline__ void each_token(const int32_t *p, int n, int V, int *bits, F f) {
  auto one = [&](int v, int i) __attribute__((always_inline)) {
    if ((unsigned)v < (unsigned)V) f(v, i);
    else if (v != -1) *bits |= kErrToken;
  };
  const int tid = threadIdx.x;
  const int head = min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / 4);
  const int quads = (n - head) / 4, tail = head + 4 * quads;
  const int4 *mid = reinterpret_cast<const int4 *>(p + head);
  for (int q0 = tid; q0 < quads; q0 += 4 * kThreads) {
    int4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = q0 + i * kThreads;
      v[i] = q < quads ? mid[q] : make_int4(-1, -1, -1, -1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = head + 4 * (q0 + i * kThreads);
      one(v[i].x, at);
      one(v[i].y, at + 1);
      one(v[i].z, at + 2);
      one(v[i].w, at + 3);
    }
  }
  if (tid < head) one(p[tid], tid);
  if (tid < n - tail) one(p[tail + tid], tail + tid);
}

template <typename T> __device__ __forceinline__ void unpack(u32x4 v, float *x) {
  if constexpr (sizeof(T) == 2) {
    const u16x8 h = __builtin_bit_cast(u16x8, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = bf16_to_f32(h[i]);
  } else {
    const floatx4 f = __builtin_bit_cast(floatx4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f[i];
  }
}
template <typename T> __device__ __forceinline__ u32x4 pack(const float *x) {
  if constexpr (sizeof(T) == 2) {
    bf16x8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (__bf16)x[i];
    return __builtin_bit_cast(u32x4, h);
  } else {
    return __builtin_bit_cast(u32x4, floatx4{x[0], x[1], x[2], x[3]});
  }
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

// x / r, rounded once: the product with 1 / r and what it is off by, divided again.
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

__device__ __forceinline__ float parameter(const float *p, int r, float none, float lo, float hi,
                                           int *bits) {
  if (p == nullptr) return none;
  const float v = p[r];
  if (v >= lo && v <= hi) return v;
  *bits |= kErrNonFinite;
  return none;
}

}  // namespace

// Units of work: (request, part of its rows, chunk), chunks innermost.  kCounts: whether
// histories, drafts or biases are given at all.
//
// The rows are a pipeline: the mask bits of row j + 2 and the logits of row j + 1 are on
// their way while row j is edited and stored.
template <typename T, bool kGrad, bool kCounts, int kThreads>
__global__ __launch_bounds__(kThreads) void edit_kernel(EditLaunch L, unsigned chunks, unsigned parts) {
  constexpr int kPer = Elem<T>::kPerVec, kVecs = kOwn / kPer, kChunk = kThreads * kOwn;
  constexpr uint32_t kAll = (1u << kPer) - 1;
  __shared__ __attribute__((aligned(16))) uint32_t word[kCounts ? kChunk : 4];
  const int tid = threadIdx.x, lane = tid & (kWave - 1);
  const unsigned units = L.R * parts * chunks;
  const bool in_place = L.out == (kGrad ? L.G : L.X);
  const T *source = reinterpret_cast<const T *>(kGrad ? L.G : L.X);
  const int64_t stride = kGrad ? L.g_stride : L.row_stride;
  for (unsigned unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const unsigned rest = unit / chunks, r = rest / parts, part = rest % parts;
    const int chunk = unit % chunks, base = chunk * kChunk;
    int bits = 0, a = r, n = 1;
    if (L.row_offset != nullptr) {
      a = L.row_offset[r];
      const int b = L.row_offset[r + 1];
      const bool bad = a < 0 || b < a || b > L.n_rows;
      if (bad) bits |= kErrLength;
      n = bad ? 0 : b - a;
    }
    const int j0 = (int)((int64_t)n * part / parts), j1 = (int)((int64_t)n * (part + 1) / parts);
    Rules rules;
    rules.repetition = parameter(L.repetition, r, 1.0f, 1e-3f, 1e3f, &bits);
    rules.frequency = parameter(L.frequency, r, 0.0f, -FLT_MAX, FLT_MAX, &bits);
    rules.presence = parameter(L.presence, r, 0.0f, -FLT_MAX, FLT_MAX, &bits);
    rules.inverse = 1.0f / rules.repetition;
    rules.bias_end = L.n_bias > 0 ? L.bias + ((int64_t)r + 1) * L.n_bias : nullptr;
    int len = 0, prompt = 0;
    if (kCounts && L.history != nullptr) {
      len = L.hist_len[r];
      if (len < 0 || len > L.hist_stride) bits |= kErrLength, len = 0;
      prompt = L.prompt_len != nullptr ? L.prompt_len[r] : 0;
      if (prompt < 0 || prompt > len) bits |= kErrLength, prompt = 0;
    }
    const int32_t *drafts = kCounts && L.drafts != nullptr ? L.drafts + (int64_t)r * L.gamma : nullptr;
    uint32_t has = 0;  // which of the thread's tokens have a word, and the words
    uint32_t w[kCounts ? kOwn : 1];
    // vector u of the thread begins at token e(u); its bits are u * kPer on
    auto e = [&](int u) { return base + (u * kThreads + tid) * kPer; };
    // mask and draft of 64 rows, a row a lane
    int mask_of, draft_of;
    auto look_ahead = [&](int j) {
      const int row = j + lane;
      mask_of = draft_of = -1;
      if (L.mask != nullptr && row < j1) {
        const int m = L.mask_index != nullptr ? L.mask_index[a + row] : a + row;
        if (m >= 0 && m < L.n_masks) mask_of = m;
        else if (m != -1) bits |= kErrLength;
      }
      if (drafts != nullptr && row > j0 && row < j1 && row <= L.gamma) {
        const int v = drafts[row - 1];
        if ((unsigned)v < (unsigned)L.V) draft_of = v;
        else if (v != -1) bits |= kErrToken;
      }
    };
    // what row k of the 64 allows of the thread's tokens
    auto allowed_by = [&](int k) {
      uint32_t all = (1u << kOwn) - 1;
      const int m = __builtin_amdgcn_readlane(mask_of, k);
      if (m < 0) return all;
      const uint8_t *mask = reinterpret_cast<const uint8_t *>(L.mask + m * L.mask_stride);
      all = 0;
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
        if (e(u) < L.V) all |= ((uint32_t)mask[e(u) / 8] >> (e(u) & 7) & kAll) << (u * kPer);
      return all;
    };
    // the thread's bit of row k's draft, 0 where another thread has it
    auto draft_bit = [&](int k) -> uint32_t {
      if (drafts == nullptr) return 0;
      const int at = __builtin_amdgcn_readlane(draft_of, k) - base;  // of no draft negative
      if ((unsigned)at >= (unsigned)kChunk || at / kPer % kThreads != tid) return 0;
      return 1u << (at / kPer / kThreads * kPer + at % kPer);
    };
    struct Row {
      u32x4 v[kVecs], raw[kGrad && kCounts ? kVecs : 1];
    };
    auto fetch = [&](Row &o, int j, uint32_t allowed, uint32_t marked, bool every) {
      const int64_t row = a + j;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        // a piece that ends behind the row's last token is read whole: it is aligned, and
        // so within the page of memory that holds the token
        const uint32_t al = allowed >> (u * kPer) & kAll, mk = marked >> (u * kPer) & kAll;
        if (e(u) >= L.V) continue;
        if (every || (al != 0 && (al != kAll || mk != 0)))
          o.v[u] = *reinterpret_cast<const u32x4 *>(source + row * stride + e(u));
        if constexpr (kGrad && kCounts)
          if (mk != 0 && L.repetition != nullptr)
            o.raw[u] = *reinterpret_cast<const u32x4 *>(reinterpret_cast<const T *>(L.X) +
                                                        row * L.row_stride + e(u));
      }
    };
    auto finish = [&](const Row &in, int j, uint32_t allowed, uint32_t marked) {
      T *to = reinterpret_cast<T *>(L.out) + (int64_t)(a + j) * L.out_stride;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const uint32_t al = allowed >> (u * kPer) & kAll, mk = marked >> (u * kPer) & kAll;
        if (e(u) >= L.V || (in_place && al == kAll && mk == 0)) continue;
        u32x4 out = in.v[u];
        if (al != kAll || mk != 0) {
          float x[kPer];
          unpack<T>(in.v[u], x);
          if constexpr (kCounts) {
            float y[kPer];
            if constexpr (kGrad) unpack<T>(in.raw[u], y);
#pragma unroll
            for (int i = 0; i < kPer; ++i)
              if (mk >> i & 1) {
                if constexpr (!kGrad) x[i] = edited(x[i], w[u * kPer + i], rules);
                else if (L.repetition != nullptr) x[i] = edited_gradient(x[i], y[i], w[u * kPer + i], rules);
              }
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (!(al >> i & 1)) x[i] = kGrad ? 0.0f : -INFINITY;
          out = pack<T>(x);
        }
        if (e(u) + kPer <= L.V) {
          *reinterpret_cast<u32x4 *>(to + e(u)) = out;
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (e(u) + i < L.V) store_piece<T>(to + e(u), out, i);
        }
      }
    };

    Row now;
    look_ahead(j0);
    if (!in_place && j0 < j1) fetch(now, j0, 0, 0, true);
    if (kCounts && j0 < j1) {
      __syncthreads();  // the unit before is done with the words
#pragma unroll
      for (int i = 0; i < kOwn / 4; ++i)
        reinterpret_cast<uint4 *>(word)[i * kThreads + tid] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      auto here = [&](int v) { return (unsigned)(v - base) < (unsigned)kChunk; };
      if (L.n_bias > 0) {
        each_token<kThreads>(L.bias_ids + (int64_t)r * L.n_bias, L.n_bias, L.V, &bits, [&](int v, int i) {
          if (here(v)) atomicMax(&word[v - base], (uint32_t)(L.n_bias - i) << kBiasShift);
        });
        __syncthreads();
      }
      if (len > 0)
        each_token<kThreads>(L.history + (int64_t)r * L.hist_stride, len, L.V, &bits, [&](int v, int i) {
          if (!here(v)) return;
          if (i < prompt) atomicOr(&word[v - base], kPromptBit);
          else atomicAdd(&word[v - base], 1u);
        });
      if (drafts != nullptr)
        each_token<kThreads>(drafts, min(j0, L.gamma), L.V, &bits, [&](int v, int) {
          if (here(v)) atomicAdd(&word[v - base], 1u);
        });
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        w[i] = word[(i / kPer * kThreads + tid) * kPer + i % kPer];
        has |= (w[i] != 0 ? 1u : 0u) << i;
      }
    }
    for (int jb = j0; jb < j1; jb += kWave) {
      const int rows = min(j1 - jb, kWave);
      if (jb > j0) look_ahead(jb);
      uint32_t al = allowed_by(0), next_al = rows > 1 ? allowed_by(1) : 0;
      auto count = [&](uint32_t bit) {  // one of the thread's tokens is a draft before this row
        if constexpr (kCounts) {
          has |= bit;
          if (bit != 0) {
#pragma unroll
            for (int i = 0; i < kOwn; ++i) w[i] += bit >> i & 1;
          }
        }
      };
      count(draft_bit(0));
      if (in_place || jb > j0) fetch(now, jb, al, has, !in_place);
      else if constexpr (kGrad && kCounts) fetch(now, jb, 0, has, false);  // the raw logits
      for (int k = 0; k < rows; ++k) {
        Row next;
        uint32_t last_al = 0, bit = 0;
        if (k + 2 < rows) last_al = allowed_by(k + 2);
        if (k + 1 < rows) {
          bit = draft_bit(k + 1);
          fetch(next, jb + k + 1, next_al, has | bit, !in_place);
        }
        finish(now, jb + k, al, has);
        count(bit);
        now = next;
        al = next_al;
        next_al = last_al;
      }
    }
    // every chunk sees what is wrong; the first of them reports it
    if (bits && chunk == 0) flag_error(L.err, bits);
  }
}

// One workgroup a request.
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
  auto go = [&](auto type, auto grad, auto has_counts) {
    using T = decltype(type);
    constexpr bool kGrad = decltype(grad)::value, kCounts = decltype(has_counts)::value;
    constexpr int kThreads = kBlock;
    const unsigned chunks = (L.V + kThreads * kOwn - 1) / (kThreads * kOwn);
    const unsigned base = L.R * chunks;  // R <= 2^22, chunks <= 64
    const unsigned most = (L.n_rows + L.R - 1) / L.R;
    unsigned parts = (8 * kComputeUnits + base - 1) / base;
    if (parts > most) parts = most;
    const unsigned units = base * parts, grid = units < (1u << 20) ? units : 1u << 20;
    DSPARK_LAUNCH(kGrad ? "edit_logits_backward" : "edit_logits", stream,
                  (edit_kernel<T, kGrad, kCounts, kThreads>), grid, kThreads, L, chunks, parts);
  };
  auto with = [&](auto type) {
    const std::true_type yes;
    const std::false_type no;
    if (L.G != nullptr && counts) go(type, yes, yes);
    else if (L.G != nullptr) go(type, yes, no);
    else if (counts) go(type, no, yes);
    else go(type, no, no);
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
