// Page operations of the paged key-value cache: fork, reserve (with copy on
// write), commit, release, compact.
//
// The free pages are those with refs = 0, and the lowest are taken first, so
// the state after a call does not depend on the order in which anything ran
// (reference counts change by integer atomics, which commute).
//
// fork, reserve and compact are two launches: a plan kernel whose first
// workgroup decides everything that needs an order (prefix sums over requests
// and pages: a few microseconds of latency, nothing to spread) while the other
// workgroups copy the state when it does not change in place; then a wide
// kernel that writes tables and counts and moves the pages.  commit and release
// need no order: one wave per request, after a copy of the state when it does not
// change in place.  Of a small state one workgroup does all of a fork, commit or
// release (by_one below).
//
// Bound: launches and the plan's latency (512 requests, 40000 pages: fork 3 + 3 us,
// reserve 14 + 5, commit 3; 4 requests, 512 pages: fork 4, reserve 6 + 3, commit 2), and for compact
// the bytes moved (783 MB of pages: 142 us, 5.5 TB/s read and written; in stretches of
// 16 KB a workgroup, all loads of one in flight before its stores).
#include <limits.h>

#include "common.h"
#include "kernels.h"
#include "trace.h"

namespace dspark {

namespace {

constexpr int kPlanBlock = 1024, kPlanWaves = kPlanBlock / kWave;
constexpr int kHead = 64;  // plan: [0] pages to move, [1] n_live

// the plan's pieces (see cache_plan_ints)
struct Plan {
  int32_t *head, *req, *page;
  int R, n_pages;
  __device__ Plan(const CacheState &s)
      : head(s.plan), req(s.plan + kHead), page(s.plan + kHead + 3 * (int64_t)s.R), R(s.R),
        n_pages(s.n_pages) {}
  __device__ int32_t *per_request(int i) const { return req + (int64_t)i * R; }
  __device__ int32_t *per_page(int i) const { return page + (int64_t)i * n_pages; }
};

__device__ __forceinline__ int pages_of(int len, int shift) {
  return (int)(((uint32_t)len + ((1u << shift) - 1)) >> shift);
}
__device__ __forceinline__ bool bad_length(const CacheState &s, int len) {
  return len < 0 || len > s.max_pages << s.page_shift;
}
__device__ __forceinline__ bool bad_page(const CacheState &s, int p) {
  return (unsigned)p >= (unsigned)s.n_pages;
}
__device__ __forceinline__ int ld_atomic(const int32_t *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// table and refs of a state that does not change in place, by the workgroups
// from 1 on (lens go with the plan)
__device__ __forceinline__ void copy_state(const CacheState &s, int block, int n_blocks) {
  const int64_t t = (int64_t)s.R * s.max_pages, stride = (int64_t)n_blocks * blockDim.x;
  const int64_t first = (int64_t)block * blockDim.x + threadIdx.x;
  for (int64_t i = first; i < t; i += stride) s.table[i] = s.table_in[i];
  for (int64_t i = first; i < s.n_pages; i += stride) s.refs[i] = s.refs_in[i];
}

// Exclusive prefix of v over a plan workgroup in thread order, and the total.
__device__ __forceinline__ int plan_scan(int v, int *scratch, int *total) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  int inc = v;
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) {
    const int t = __shfl_up(inc, o);
    if (lane >= o) inc += t;
  }
  __syncthreads();
  if (lane == kWave - 1) scratch[w] = inc;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlanWaves; ++i) {
    before += i < w ? scratch[i] : 0;
    all += scratch[i];
  }
  *total = all;
  return before + inc - v;
}

// The wave's stretch of the pages in steps of 4 pages a lane: f(first page of
// the lane, its 4 counts); past the last page a count reads as `past`.
template <typename F>
__device__ __forceinline__ void walk_refs(const int32_t *refs, int n_pages, int past, F f) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int64_t stretch = ((n_pages + kPlanWaves - 1) / kPlanWaves + 255) & ~255;
  const int64_t begin = w * stretch, end = min(begin + stretch, (int64_t)n_pages);
#pragma unroll 4
  for (int64_t b = begin; b < end; b += 4 * kWave) {
    const int64_t p = b + 4 * lane;
    int c[4];
    if (p + 3 < n_pages) {
      const int4 v = *reinterpret_cast<const int4 *>(refs + p);
      c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[i] = p + i < n_pages ? refs[p + i] : past;
    }
    f((int)p, c);
  }
}

// Position of each of the lane's marked pages in page order, from `at` on;
// returns `at` behind the wave's last.
__device__ __forceinline__ int place4(const bool *mark, int at, int *pos) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint64_t below = (1ull << lane) - 1;
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t m = __ballot(mark[i]);
    before += __popcll(m & below);
    all += __popcll(m);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    pos[i] = at + before;
    before += mark[i];
  }
  return at + all;
}

// Sum of one count per wave over the waves before this one, and over all.
__device__ __forceinline__ int before_wave(int count, int *scratch, int *total) {
  __syncthreads();
  if ((threadIdx.x & (kWave - 1)) == 0) scratch[threadIdx.x / kWave] = count;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPlanWaves; ++i) {
    before += i < (int)(threadIdx.x / kWave) ? scratch[i] : 0;
    all += scratch[i];
  }
  *total = all;
  return before;
}

// Copies the pages from(i) -> to(i), i < n, of both pools: the grid takes
// stretches of 16 KB, all loads of a stretch in flight before its stores.
template <typename From, typename To>
__device__ __forceinline__ void move_pages(const CachePools &pools, int n, From from, To to) {
  if (pools.k == nullptr) return;
  constexpr int kUnit = 4, kStretch = kBlock * kUnit;  // 16-byte pieces
  const int64_t pieces = (int64_t)(pools.page_bytes / 16);
  const int64_t per_page = (pieces + kStretch - 1) / kStretch;
  const int64_t total = 2 * per_page * n;
  for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
    const int64_t i = u / (2 * per_page), rest = u - i * 2 * per_page;
    char *pool = (char *)(rest < per_page ? pools.k : pools.v);
    const int64_t b = (rest < per_page ? rest : rest - per_page) * kStretch + threadIdx.x;
    const u32x4 *src = reinterpret_cast<const u32x4 *>(pool + (int64_t)from(i) * pools.page_bytes);
    u32x4 *dst = reinterpret_cast<u32x4 *>(pool + (int64_t)to(i) * pools.page_bytes);
    u32x4 v[kUnit];
#pragma unroll
    for (int j = 0; j < kUnit; ++j)
      v[j] = __builtin_nontemporal_load(src + min(b + j * kBlock, pieces - 1));
#pragma unroll
    for (int j = 0; j < kUnit; ++j)
      if (b + j * kBlock < pieces) __builtin_nontemporal_store(v[j], dst + b + j * kBlock);
  }
}

// Request r gives back its pages [from, to) (one wave).
__device__ __forceinline__ void give_back(const CacheState &s, int r, int from, int to) {
  const int lane = threadIdx.x & (kWave - 1);
  int32_t *row = s.table + (int64_t)r * s.max_pages;
  for (int i = from + lane; i < to; i += kWave) {
    const int p = row[i];
    row[i] = -1;
    if (bad_page(s, p)) flag_error(s.err, kErrPage);
    else atomicSub(&s.refs[p], 1);
  }
}

}  // namespace

// All of the state, lens too, by n_blocks workgroups.
namespace {
__device__ __forceinline__ void copy_all(const CacheState &s, int block, int n_blocks) {
  copy_state(s, block, n_blocks);
  for (int r = block * (int)blockDim.x + threadIdx.x; r < s.R; r += n_blocks * (int)blockDim.x)
    s.lens[r] = s.lens_in[r];
}
}  // namespace

__global__ __launch_bounds__(kPlanBlock) void cache_copy_kernel(CacheState s) {
  copy_all(s, blockIdx.x, gridDim.x);
}

// --------------------------------------------------------------------- fork
// Request dst becomes src's first `len` tokens, by threads [thread, ...) in steps.
namespace {
__device__ __forceinline__ void share_pages(const CacheState &s, int src, int dst, int len, int thread,
                                            int threads) {
  if (len <= 0) return;
  const int32_t *from = s.table + (int64_t)src * s.max_pages;
  int32_t *to = s.table + (int64_t)dst * s.max_pages;
  const int n = pages_of(len, s.page_shift);
  for (int j = thread; j < n; j += threads) {
    const int p = from[j];
    to[j] = p;
    if (bad_page(s, p)) flag_error(s.err, kErrPage);
    else atomicAdd(&s.refs[p], 1);
  }
}
}  // namespace

// Which pairs hold: of those with the same destination the first does.  Leaves
// each pair's length (-1: skipped) in the plan; where it is the only workgroup
// (`whole`), the pairs' pages follow at once.
__global__ __launch_bounds__(kPlanBlock) void cache_fork_plan_kernel(CacheState s, int n,
                                                                     const int32_t *src,
                                                                     const int32_t *dst, bool whole) {
  if (blockIdx.x > 0) {
    copy_state(s, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  if (whole && !s.in_place()) copy_state(s, 0, 1);
  const Plan plan(s);
  int32_t *owner = plan.per_request(0), *length = plan.per_request(1);
  const int tid = threadIdx.x;
  auto outside = [&](int r) { return (unsigned)r >= (unsigned)s.R; };
  for (int i = tid; i < n; i += kPlanBlock)
    if (!outside(dst[i])) owner[dst[i]] = INT_MAX;
  if (!s.in_place())
    for (int r = tid; r < s.R; r += kPlanBlock) s.lens[r] = s.lens_in[r];
  __threadfence_block();
  __syncthreads();
  for (int i = tid; i < n; i += kPlanBlock)
    if (!outside(dst[i]) && !outside(src[i])) atomicMin(&owner[dst[i]], i);
  __syncthreads();
  int bits = 0;
  for (int i = tid; i < n; i += kPlanBlock) {
    const int a = src[i], b = dst[i];
    int len = -1;
    if (!outside(a) && !outside(b) && ld_atomic(&owner[b]) == i && s.lens_in[b] == 0) {
      len = s.lens_in[a];
      if (bad_length(s, len)) len = -1;
    }
    if (len < 0) bits = kErrLength;
    length[i] = len;
  }
  __syncthreads();  // every length is read before one is written
  for (int i = tid; i < n; i += kPlanBlock)
    if (length[i] >= 0) s.lens[dst[i]] = length[i];
  if (bits) flag_error(s.err, bits);
  if (whole)  // the state is copied and every length known since the barriers above
    for (int i = tid / kWave; i < n; i += kPlanWaves)
      share_pages(s, src[i], dst[i], length[i], tid & (kWave - 1), kWave);
}

__global__ __launch_bounds__(kBlock) void cache_fork_kernel(CacheState s, const int32_t *src,
                                                            const int32_t *dst) {
  const int i = blockIdx.x;
  share_pages(s, src[i], dst[i], Plan(s).per_request(1)[i], threadIdx.x, kBlock);
}

// ------------------------------------------------------------------ reserve
// Per request: the page to copy (or -1) and where its new pages start in the
// list of free ones; the requests with a copy; the free pages themselves.
__global__ __launch_bounds__(kPlanBlock) void cache_reserve_plan_kernel(CacheState s,
                                                                        const int32_t *row_offset,
                                                                        int32_t *missing) {
  if (blockIdx.x > 0) {
    copy_state(s, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ int scratch[kPlanWaves], n_copies, is_bad;
  const Plan plan(s);
  int32_t *copied = plan.per_request(0), *start = plan.per_request(1), *copying = plan.per_request(2);
  int32_t *free_ids = plan.per_page(0), *writers = plan.per_page(1), *first = plan.per_page(2);
  const int tid = threadIdx.x, shift = s.page_shift, in_page = (1 << shift) - 1;
  if (tid == 0) n_copies = is_bad = 0;
  __syncthreads();
  int bits = 0;
  for (int r = tid; r < s.R; r += kPlanBlock) {
    const int len = s.lens_in[r];
    const int64_t n = (int64_t)row_offset[r + 1] - row_offset[r];
    int shared = -1;
    if (bad_length(s, len) || n < 0 || len + n > (int64_t)s.max_pages << shift) {
      bits |= kErrLength;
      is_bad = 1;
    } else if (n > 0 && (len & in_page) != 0) {
      const int tail = s.table_in[(int64_t)r * s.max_pages + (len >> shift)];
      if (bad_page(s, tail)) {
        bits |= kErrPage;
      } else if (s.refs_in[tail] > 1) {
        shared = tail;
        writers[tail] = 0;
        first[tail] = INT_MAX;
      }
    }
    copied[r] = shared;
  }
  __threadfence_block();
  __syncthreads();
  const bool bad = is_bad != 0;
  if (!bad) {
    for (int r = tid; r < s.R; r += kPlanBlock)
      if (copied[r] >= 0) {
        atomicAdd(&writers[copied[r]], 1);
        atomicMin(&first[copied[r]], r);
      }
  }
  __syncthreads();
  int total = 0;
  for (int r0 = 0; !bad && r0 < s.R; r0 += kPlanBlock) {
    const int r = r0 + tid;
    int need = 0;
    if (r < s.R) {
      const int len = s.lens_in[r], n = row_offset[r + 1] - row_offset[r], tail = copied[r];
      need = pages_of(len + n, shift) - pages_of(len, shift);
      if (tail >= 0) {
        if (ld_atomic(&writers[tail]) == s.refs_in[tail] && ld_atomic(&first[tail]) == r) {
          copied[r] = -1;  // every holder writes it: the first keeps it
        } else {
          ++need;
          copying[atomicAdd(&n_copies, 1)] = r;
        }
      }
    }
    int sum;
    const int at = plan_scan(need, scratch, &sum);
    if (r < s.R) start[r] = total + at;
    total += sum;
  }
  int n_free = 0;
  walk_refs(s.refs_in, s.n_pages, 1, [&](int p, const int *c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) n_free += __popcll(__ballot(c[i] == 0));
  });
  int all_free;
  int at = before_wave(n_free, scratch, &all_free);
  const bool go = !bad && total <= all_free;
  if (go) {
    walk_refs(s.refs_in, s.n_pages, 1, [&](int p, const int *c) {
      if (at >= total) return;  // uniform
      bool mark[4];
      int pos[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) mark[i] = c[i] == 0;
      at = place4(mark, at, pos);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (mark[i] && pos[i] < total) free_ids[pos[i]] = p + i;
    });
  }
  for (int r = tid; r < s.R; r += kPlanBlock)
    if (go || !s.in_place())
      s.lens[r] = s.lens_in[r] + (go ? row_offset[r + 1] - row_offset[r] : 0);
  // the round's other calls take these: of rows that found no room they do nothing
  for (int r = tid; r <= s.R; r += kPlanBlock) s.rows[r] = go ? row_offset[r] : 0;
  if (tid == 0) {
    plan.head[0] = go ? n_copies : -1;
    *missing = bad ? -1 : max(total - all_free, 0);
    if (!bad && !go) bits |= kErrNoPages;
  }
  if (bits) flag_error(s.err, bits);
}

__global__ __launch_bounds__(kBlock) void cache_reserve_kernel(CacheState s, CachePools pools,
                                                               const int32_t *row_offset) {
  const Plan plan(s);
  const int n_copies = plan.head[0];
  if (n_copies < 0) return;
  const int32_t *copied = plan.per_request(0), *start = plan.per_request(1);
  const int32_t *copying = plan.per_request(2), *free_ids = plan.per_page(0);
  const int lane = threadIdx.x & (kWave - 1), shift = s.page_shift;
  const int waves = gridDim.x * (kBlock / kWave);
  for (int r = blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave; r < s.R; r += waves) {
    const int n = row_offset[r + 1] - row_offset[r], len = s.lens[r] - n;
    const int have = pages_of(len, shift), want = pages_of(len + n, shift), tail = copied[r];
    int32_t *row = s.table + (int64_t)r * s.max_pages;
    int at = start[r];
    if (tail >= 0) {
      if (lane == 0) {
        const int p = free_ids[at];
        row[have - 1] = p;
        s.refs[p] = 1;
        atomicSub(&s.refs[tail], 1);
      }
      ++at;
    }
    for (int i = have + lane; i < want; i += kWave) {
      const int p = free_ids[at + i - have];
      row[i] = p;
      s.refs[p] = 1;
    }
  }
  move_pages(pools, n_copies, [&](int64_t i) { return copied[copying[i]]; },
             [&](int64_t i) { return free_ids[start[copying[i]]]; });
}

// ----------------------------------------------------------- commit, release
namespace {
// One wave: request r keeps n_acc + 1 of its rows.
__device__ __forceinline__ void commit_one(const CacheState &s, int r, const int32_t *row_offset,
                                           const int32_t *n_acc) {
  const int lane = threadIdx.x & (kWave - 1);
  const int len = s.lens[r];
  const int64_t n = (int64_t)row_offset[r + 1] - row_offset[r], keep = (int64_t)n_acc[r] + 1;
  if (bad_length(s, len) || n < 0 || n > len || keep < 0 || keep > n) {
    if (lane == 0) flag_error(s.err, kErrLength);
    return;
  }
  const int now = len - (int)(n - keep);
  if (lane == 0) s.lens[r] = now;
  give_back(s, r, pages_of(now, s.page_shift), pages_of(len, s.page_shift));
}

// One wave: request r leaves.
__device__ __forceinline__ void release_one(const CacheState &s, int r) {
  const int lane = threadIdx.x & (kWave - 1);
  if ((unsigned)r >= (unsigned)s.R) {
    if (lane == 0) flag_error(s.err, kErrLength);
    return;
  }
  int len = 0;
  if (lane == 0) len = atomicExch(&s.lens[r], 0);  // twice the same: the second finds 0
  len = __shfl(len, 0);
  if (bad_length(s, len)) {
    if (lane == 0) flag_error(s.err, kErrLength);
    return;
  }
  give_back(s, r, 0, pages_of(len, s.page_shift));
}

// The number of this wave among all of the grid, and how many they are.  Where a
// kernel is one workgroup that first copies the state, its waves see the copy.
__device__ __forceinline__ int wave_index(const CacheState &s, bool whole, int *waves) {
  if (whole) {
    copy_all(s, 0, 1);
    __threadfence_block();
    __syncthreads();
  }
  *waves = gridDim.x * (blockDim.x / kWave);
  return (blockIdx.x * blockDim.x + threadIdx.x) / kWave;
}
}  // namespace

__global__ __launch_bounds__(kPlanBlock) void cache_commit_kernel(CacheState s,
                                                                  const int32_t *row_offset,
                                                                  const int32_t *n_acc, bool whole) {
  int waves;
  for (int r = wave_index(s, whole, &waves); r < s.R; r += waves)
    commit_one(s, r, row_offset, n_acc);
}

__global__ __launch_bounds__(kPlanBlock) void cache_release_kernel(CacheState s, int n,
                                                                   const int32_t *which, bool whole) {
  int waves;
  for (int i = wave_index(s, whole, &waves); i < n; i += waves) release_one(s, which[i]);
}

// ------------------------------------------------------------------ compact
__global__ __launch_bounds__(kPlanBlock) void cache_compact_plan_kernel(CacheState s,
                                                                        int32_t *n_live_out) {
  if (blockIdx.x > 0) {
    copy_state(s, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ int scratch[kPlanWaves];
  const Plan plan(s);
  int32_t *holes = plan.per_page(0), *movers = plan.per_page(1), *moved_to = plan.per_page(2);
  int count = 0, n_live;
  walk_refs(s.refs_in, s.n_pages, 0, [&](int p, const int *c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) count += __popcll(__ballot(c[i] > 0));
  });
  before_wave(count, scratch, &n_live);
  int n_holes = 0, n_movers = 0;
  walk_refs(s.refs_in, s.n_pages, 0, [&](int p, const int *c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n_holes += __popcll(__ballot(p + i < n_live && c[i] <= 0));
      n_movers += __popcll(__ballot(p + i >= n_live && c[i] > 0));
    }
  });
  int moves;
  int hole_at = before_wave(n_holes, scratch, &moves);
  int mover_at = before_wave(n_movers, scratch, &moves);
  walk_refs(s.refs_in, s.n_pages, 0, [&](int p, const int *c) {
    bool hole[4], mover[4];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hole[i] = p + i < n_live && c[i] <= 0;
      mover[i] = p + i >= n_live && c[i] > 0;
      // a table entry that names a free page (its count does not hold) finds -1
      if (p + i >= n_live && p + i < s.n_pages && !mover[i]) moved_to[p + i] = -1;
    }
    hole_at = place4(hole, hole_at, pos);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (hole[i]) holes[pos[i]] = p + i;
    mover_at = place4(mover, mover_at, pos);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (mover[i]) movers[pos[i]] = p + i;
  });
  __threadfence_block();
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kPlanBlock) moved_to[movers[i]] = holes[i];
  if (!s.in_place())
    for (int r = threadIdx.x; r < s.R; r += kPlanBlock) s.lens[r] = s.lens_in[r];
  if (threadIdx.x == 0) {
    plan.head[0] = moves;
    plan.head[1] = n_live;
    *n_live_out = n_live;
  }
}

__global__ __launch_bounds__(kBlock) void cache_compact_kernel(CacheState s, CachePools pools) {
  const Plan plan(s);
  const int moves = plan.head[0], n_live = plan.head[1];
  const int32_t *holes = plan.per_page(0), *movers = plan.per_page(1), *moved_to = plan.per_page(2);
  const int lane = threadIdx.x & (kWave - 1);
  const int waves = gridDim.x * (kBlock / kWave);
  // also where nothing moves: what is wrong in the state is flagged all the same
  for (int r = blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave; r < s.R; r += waves) {
    const int len = s.lens[r];
    if (bad_length(s, len)) {
      if (lane == 0) flag_error(s.err, kErrLength);
      continue;
    }
    int32_t *row = s.table + (int64_t)r * s.max_pages;
    for (int i = lane; i < pages_of(len, s.page_shift); i += kWave) {
      const int p = row[i];
      const int to = bad_page(s, p) ? -1 : p < n_live ? p : moved_to[p];
      if (to < 0) flag_error(s.err, kErrPage);
      else if (to != p) row[i] = to;
    }
  }
  for (int i = blockIdx.x * kBlock + threadIdx.x; i < moves; i += gridDim.x * kBlock) {
    s.refs[holes[i]] = s.refs[movers[i]];
    s.refs[movers[i]] = 0;
  }
  move_pages(pools, moves, [&](int64_t i) { return movers[i]; }, [&](int64_t i) { return holes[i]; });
}

// ----------------------------------------------------------------- launches
namespace {
constexpr int kMoveBlocks = 4 * kComputeUnits;

// workgroups of a plan kernel: the plan's own, and copiers (4 entries a thread
// or more) when the state does not change in place
int plan_blocks(const CacheState &s) {
  if (s.in_place()) return 1;
  const int64_t n = ((int64_t)s.R * s.max_pages + s.n_pages) / (4 * kPlanBlock) + 1;
  return 1 + (int)(n < 2 * kComputeUnits ? n : 2 * kComputeUnits);
}
int wave_blocks(int n) { return (n + kBlock / kWave - 1) / (kBlock / kWave); }
void copy_out(const CacheState &s, hipStream_t stream) {
  DSPARK_LAUNCH("cache_copy", stream, cache_copy_kernel, plan_blocks(s) - 1, kPlanBlock, s);
}

// Whether one workgroup does an operation on n requests that is else two launches:
// up to 16 entries a thread to copy and as many of the requests' own.  It takes the
// device no longer (16 requests, 600 pages: copy and release 2.8 us, 3.6 as two
// launches) and the host 2.6 us less.  In place, commit and release are one launch
// anyway.
bool by_one(const CacheState &s, int n) {
  const int64_t most = 16 * kPlanBlock;
  return (s.in_place() || (int64_t)s.R * s.max_pages + s.n_pages <= most) &&
         (int64_t)n * s.max_pages <= most;
}
}  // namespace

hipError_t launch_cache_fork(const CacheState &S, int n, const int32_t *src, const int32_t *dst,
                             hipStream_t stream) {
  const bool whole = by_one(S, n);
  DSPARK_LAUNCH("cache_fork_plan", stream, cache_fork_plan_kernel, whole ? 1 : plan_blocks(S),
                kPlanBlock, S, n, src, dst, whole);
  if (!whole) DSPARK_LAUNCH("cache_fork", stream, cache_fork_kernel, n, kBlock, S, src, dst);
  return hipGetLastError();
}

hipError_t launch_cache_reserve(const CacheState &S, const CachePools &P, const int32_t *row_offset,
                                int32_t *missing, hipStream_t stream) {
  DSPARK_LAUNCH("cache_reserve_plan", stream, cache_reserve_plan_kernel, plan_blocks(S), kPlanBlock,
                S, row_offset, missing);
  DSPARK_LAUNCH("cache_reserve", stream, cache_reserve_kernel, kMoveBlocks, kBlock, S, P, row_offset);
  return hipGetLastError();
}

hipError_t launch_cache_commit(const CacheState &S, const int32_t *row_offset, const int32_t *n_acc,
                               hipStream_t stream) {
  const bool whole = !S.in_place() && by_one(S, S.R);
  if (!whole && !S.in_place()) copy_out(S, stream);
  DSPARK_LAUNCH("cache_commit", stream, cache_commit_kernel, whole ? 1 : wave_blocks(S.R),
                whole ? kPlanBlock : kBlock, S, row_offset, n_acc, whole);
  return hipGetLastError();
}

hipError_t launch_cache_release(const CacheState &S, int n, const int32_t *which, hipStream_t stream) {
  const bool whole = !S.in_place() && by_one(S, n);
  if (!whole && !S.in_place()) copy_out(S, stream);
  DSPARK_LAUNCH("cache_release", stream, cache_release_kernel, whole ? 1 : wave_blocks(n),
                whole ? kPlanBlock : kBlock, S, n, which, whole);
  return hipGetLastError();
}

hipError_t launch_cache_compact(const CacheState &S, const CachePools &P, int32_t *n_live,
                                hipStream_t stream) {
  DSPARK_LAUNCH("cache_compact_plan", stream, cache_compact_plan_kernel, plan_blocks(S), kPlanBlock,
                S, n_live);
  DSPARK_LAUNCH("cache_compact", stream, cache_compact_kernel, kMoveBlocks, kBlock, S, P);
  return hipGetLastError();
}

}  // namespace dspark
