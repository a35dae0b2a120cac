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
constexpr int kOwn = 16;                // tokens of a thread
constexpr int kChunk = kBlock * kOwn;   // tokens of a workgroup

template <typename T> struct Edit {
  static constexpr int kPer = Elem<T>::kPerVec, kVecs = kOwn / kPer;
  static constexpr uint32_t kAll = (1u << kPer) - 1;
};

// f(token, index) for the tokens [0, n) at p, spread over the workgroup; -1 is skipped,
// what lies outside the vocabulary sets *bits.
template <typename F>
__device__ __forceinline__ void each_token(const int32_t *p, int n, int V, int *bits, F f) {
  auto one = [&](int v, int i) __attribute__((always_inline)) {
    if ((unsigned)v < (unsigned)V) f(v, i);
    else if (v != -1) *bits |= kErrToken;
  };
  // 16-byte loads of the aligned middle
  const int head = min(n, (int)((16 - ((uintptr_t)p & 15)) & 15) / 4);
  const int quads = (n - head) / 4, tail = head + 4 * quads;
#pragma unroll 4
  for (int q = threadIdx.x; q < quads; q += kBlock) {
    const int4 v = *reinterpret_cast<const int4 *>(p + head + 4 * q);
    one(v.x, head + 4 * q);
    one(v.y, head + 4 * q + 1);
    one(v.z, head + 4 * q + 2);
    one(v.w, head + 4 * q + 3);
  }
  if ((int)threadIdx.x < head) one(p[threadIdx.x], threadIdx.x);
  if ((int)threadIdx.x < n - tail) one(p[tail + threadIdx.x], tail + threadIdx.x);
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

// Units of work: (request, part of its rows, chunk), chunks innermost.
template <typename T, bool kGrad>
__global__ __launch_bounds__(kBlock) void edit_kernel(EditLaunch L, int chunks, int parts) {
  using E = Edit<T>;
  constexpr int kPer = E::kPer, kVecs = E::kVecs;
  __shared__ __attribute__((aligned(16))) uint32_t word[kChunk];
  const int tid = threadIdx.x;
  const int64_t units = (int64_t)L.R * parts * chunks;
  const bool counts = L.history != nullptr || L.drafts != nullptr || L.n_bias > 0;
  const bool in_place = L.out == (kGrad ? L.G : L.X);
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int chunk = (int)(unit % chunks);
    const int64_t rest = unit / chunks;
    const int r = (int)(rest / parts), part = (int)(rest % parts);
    const bool report = chunk == 0 && part == 0;
    int bits = 0;
    int a = r, n = 1;
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
    if (L.history != nullptr) {
      len = L.hist_len[r];
      if (len < 0 || len > L.hist_stride) bits |= kErrLength, len = 0;
      prompt = L.prompt_len != nullptr ? L.prompt_len[r] : 0;
      if (prompt < 0 || prompt > len) bits |= kErrLength, prompt = 0;
    }
    const int base = chunk * kChunk;
    const int32_t *drafts = L.drafts != nullptr ? L.drafts + (int64_t)r * L.gamma : nullptr;
    uint32_t has[kVecs];  // which of the thread's tokens have a word
#pragma unroll
    for (int u = 0; u < kVecs; ++u) has[u] = 0;
    if (counts && j0 < j1) {
      __syncthreads();  // the unit before is done with the words
#pragma unroll
      for (int i = 0; i < kOwn / 4; ++i)
        reinterpret_cast<uint4 *>(word)[i * kBlock + tid] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      auto here = [&](int v) { return (unsigned)(v - base) < (unsigned)kChunk; };
      if (L.n_bias > 0) {
        each_token(L.bias_ids + (int64_t)r * L.n_bias, L.n_bias, L.V, &bits, [&](int v, int i) {
          if (here(v)) atomicMax(&word[v - base], (uint32_t)(L.n_bias - i) << kBiasShift);
        });
        __syncthreads();
      }
      if (len > 0)
        each_token(L.history + (int64_t)r * L.hist_stride, len, L.V, &bits, [&](int v, int i) {
          if (!here(v)) return;
          if (i < prompt) atomicOr(&word[v - base], kPromptBit);
          else atomicAdd(&word[v - base], 1u);
        });
      if (drafts != nullptr)
        each_token(drafts, min(j0, L.gamma), L.V, &bits, [&](int v, int) {
          if (here(v)) atomicAdd(&word[v - base], 1u);
        });
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kVecs; ++u)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (word[(u * kBlock + tid) * kPer + i] != 0) has[u] |= 1u << i;
    }
    for (int j = j0; j < j1; ++j) {
      const int64_t row = a + j;
      if (j > j0 && drafts != nullptr && j <= L.gamma) {
        const int v = drafts[j - 1];
        if ((unsigned)v >= (unsigned)L.V) {
          if (v != -1) bits |= kErrToken;
        } else if ((unsigned)(v - base) < (unsigned)kChunk) {
          const int at = (v - base) / kPer;  // its vector of the chunk
          if (at % kBlock == tid) {
            word[v - base] += 1;
#pragma unroll
            for (int u = 0; u < kVecs; ++u)
              if (at / kBlock == u) has[u] |= 1u << ((v - base) % kPer);
          }
        }
      }
      const uint8_t *mask = nullptr;
      if (L.mask != nullptr) {
        const int m = L.mask_index != nullptr ? L.mask_index[row] : (int)row;
        if (m >= 0 && m < L.n_masks) mask = reinterpret_cast<const uint8_t *>(L.mask + m * L.mask_stride);
        else if (m != -1) bits |= kErrLength;
      }
      const T *from = reinterpret_cast<const T *>(kGrad ? L.G : L.X) +
                      row * (kGrad ? L.g_stride : L.row_stride);
      const T *raw = reinterpret_cast<const T *>(L.X) + row * L.row_stride;
      T *to = reinterpret_cast<T *>(L.out) + row * L.out_stride;
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        const int e = base + (u * kBlock + tid) * kPer;
        if (e >= L.V) continue;
        uint32_t allowed = E::kAll;
        if (mask != nullptr) allowed = mask[e / 8] >> (e & 7) & E::kAll;
        const bool whole = e + kPer <= L.V;
        if (in_place && allowed == E::kAll && has[u] == 0) continue;
        float x[kPer];
        u32x4 v;
        if (allowed != 0 || !whole) {
          if (whole) {
            v = *reinterpret_cast<const u32x4 *>(from + e);
          } else {
            uint32_t bits16[4] = {0, 0, 0, 0};
            for (int i = 0; i < L.V - e; ++i)
              __builtin_memcpy((char *)bits16 + i * sizeof(T), from + e + i, sizeof(T));
            v = u32x4{bits16[0], bits16[1], bits16[2], bits16[3]};
          }
        }
        if (whole && allowed == E::kAll && has[u] == 0) {
          *reinterpret_cast<u32x4 *>(to + e) = v;
          continue;
        }
        const T *vs = reinterpret_cast<const T *>(&v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          x[i] = allowed != 0 ? Elem<T>::at(vs, i) : 0.0f;
          if (has[u] >> i & 1) {
            const uint32_t w = word[(u * kBlock + tid) * kPer + i];
            if constexpr (kGrad) {
              if (L.repetition != nullptr)
                x[i] = edited_gradient(x[i], Elem<T>::at(raw, e + i), w, rules);
            } else {
              x[i] = edited(x[i], w, rules);
            }
          }
          if (!(allowed >> i & 1)) x[i] = kGrad ? 0.0f : -INFINITY;
        }
        if (whole) {
          T o[kPer];
#pragma unroll
          for (int i = 0; i < kPer; ++i) store_elem(o, i, x[i]);
          u32x4 out;
          __builtin_memcpy(&out, o, 16);
          *reinterpret_cast<u32x4 *>(to + e) = out;
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (e + i < L.V) store_elem(to, e + i, x[i]);
        }
      }
    }
    // a mask or draft that is wrong is seen by every chunk; the first reports it
    if (bits && chunk == 0) flag_error(L.err, report ? bits : bits & (kErrToken | kErrLength));
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
  const int chunks = (L.V + kChunk - 1) / kChunk;
  const int64_t base = (int64_t)L.R * chunks;
  const int most = (L.n_rows + L.R - 1) / L.R;
  int64_t parts = (8 * kComputeUnits + base - 1) / base;
  if (parts > most) parts = most;
  const int64_t units = base * parts;
  const int grid = (int)(units < (1 << 20) ? units : 1 << 20);
  auto go = [&](auto type, auto grad) {
    using T = decltype(type);
    constexpr bool kGrad = decltype(grad)::value;
    DSPARK_LAUNCH(kGrad ? "edit_logits_backward" : "edit_logits", stream, (edit_kernel<T, kGrad>), grid,
                  kBlock, L, chunks, (int)parts);
  };
  const bool grad = L.G != nullptr;
  if (L.bf16 && grad) go(bf16_t(), std::true_type());
  else if (L.bf16) go(bf16_t(), std::false_type());
  else if (grad) go(float(), std::true_type());
  else go(float(), std::false_type());
  return hipGetLastError();
}

hipError_t launch_history_append(const HistoryLaunch &L, hipStream_t stream) {
  DSPARK_LAUNCH("history_append", stream, history_append_kernel, L.R, kBlock, L);
  return hipGetLastError();
}

}  // namespace dspark
