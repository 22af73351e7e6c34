// kvpages.hip - the pages' own operations beside the pointer exchange (gfx950): a prompt's
// particles forked from its first one, sequences freed, the pool compacted, and the copy
// of the pages that a copy-on-write or compaction list names.
//
// All but the copy are integer work on the refcounted block-table state (SMC explainers,
// "system optimisation design": shared blocks, released by reference count) and are bound
// by the latency of a few launches (512 tables of 133 blocks, a pool of 24,576: fork 3.7 us,
// free 3.7 + 2.2 + 2.9 us, compact 4.5 + 4.6 + 4.7 us); the order of every list they leave is
// fixed by block ids alone, so the state does not depend on the order of the atomics.
#include "../../include/smcsd.h"
#include "device.hpp"
#include "internal.hpp"

namespace smcsd {

namespace {

constexpr int kPgBlock = 256;
// Consecutive blocks of a thread in the kernels over the pool.  A workgroup adds up the counts of
// all other workgroups' groups, which larger groups would make fewer, but 32 to a thread lose
// at every size measured: count and rank of 24,576 blocks 19 us against 7, of 8 million 226
// against 45 (a thread's neighbours are then 128 bytes away).  That sum grows with the square of
// the pool: 64 tables of 2000 blocks freed (half of them) and compacted take 20 and 25 us in a pool of
// 2^20 blocks, 39 and 71 of 2^23, 183 and 403 of 2^25, 431 and 1276 of 2^26, the largest.
constexpr int kPerThread = 4;

// Bit i: `is` holds for the count of block b0 + i (b0 a multiple of kPerThread).
template <typename F>
__device__ __forceinline__ uint32_t block_bits(const int32_t *rc, int64_t b0, int64_t P, F is) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; i += 4) {
    int32_t v[4] = {0, 0, 0, 0};
    if (b0 + i + 4 <= P) {
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = rc[b0 + i + c];
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (b0 + i + c < P) v[c] = rc[b0 + i + c];
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) m |= (b0 + i + c < P && is(v[c]) ? 1u : 0u) << (i + c);
  }
  return m;
}

// ---------------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------------
constexpr int kForkRows = 16;  // destination rows of one thread: one refcount change for all

// Thread = (prompt, slot, part of kForkRows particles): neighbouring threads take
// neighbouring slots, so every row is read and written in whole lines.
__global__ __launch_bounds__(kPgBlock) void k_fork(const int32_t *__restrict__ forked, int B, int N,
                                                   int32_t *__restrict__ T, int M,
                                                   int32_t *__restrict__ rc, int64_t P,
                                                   int32_t *__restrict__ status, int cols, int parts,
                                                   int64_t items) {
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int col = (int)(it % cols);
    const int64_t bp = it / cols;
    const int part = (int)(bp % parts), b = (int)(bp / parts);
    const int s = min(col * kPgBlock + (int)threadIdx.x, M - 1);
    int32_t *row0 = T + (int64_t)b * N * M + s;
    const int32_t id = row0[0];  // on its way before the prompt's flag is looked at
    if (forked[b] == 0 || col * kPgBlock + (int)threadIdx.x >= M || id == -1) continue;
    if (id < 0 || id >= P) {
      if (part == 0) atomicOr(status, SMCSD_ST_BAD_INPUT);
      continue;
    }
    const int n0 = 1 + part * kForkRows, n1 = min(N, n0 + kForkRows);
    int32_t old[kForkRows];  // all read before any is written: one wait instead of one a row
#pragma unroll
    for (int i = 0; i < kForkRows; ++i) old[i] = row0[(int64_t)min(n0 + i, n1 - 1) * M];
    int took = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kForkRows; ++i) {
      if (n0 + i >= n1) continue;
      if (old[i] == -1) {
        row0[(int64_t)(n0 + i) * M] = id;
        ++took;
      } else {
        bad = true;
      }
    }
    if (took) atomicAdd(&rc[id], took);
    if (bad) atomicOr(status, SMCSD_ST_BAD_INPUT);
  }
}

// ---------------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------------
// A block whose last reference went is marked in its own refcount until it is pushed.  In a
// corrupt state others take from the mark and give back (at most one each of the threads in
// flight, some 2^19): it lies 2^29 from the least number and 2^29 below what counts as marked.
constexpr int32_t kFreedMark = -(3 << 29);
__device__ __forceinline__ bool is_freed(int32_t r) { return r < INT32_MIN / 2; }

__global__ __launch_bounds__(kPgBlock) void k_free_drop(const int32_t *__restrict__ freed, int64_t S,
                                                        int32_t *__restrict__ T, int M,
                                                        int32_t *__restrict__ rc, int64_t P,
                                                        int32_t *__restrict__ status, int cols) {
  const int64_t items = S * cols;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t g = it / cols;
    const int s = (int)(it - g * cols) * kPgBlock + threadIdx.x;
    if (freed[g] == 0 || s >= M) continue;
    const int32_t id = T[g * M + s];
    if (id == -1) continue;
    T[g * M + s] = -1;
    if (id < 0 || id >= P) {
      atomicOr(status, SMCSD_ST_BAD_INPUT);
      continue;
    }
    const int32_t old = atomicSub(&rc[id], 1);
    if (old == 1) {
      atomicExch(&rc[id], kFreedMark);
    } else if (old <= 0) {
      atomicAdd(&rc[id], 1);
      atomicOr(status, SMCSD_ST_BAD_INPUT);
    }
  }
}

// Workgroup g counts group g's freed blocks; workgroup 0 keeps the old top for the push.
__global__ __launch_bounds__(kPgBlock) void k_free_count(const int32_t *__restrict__ rc, int64_t P,
                                                         const int32_t *__restrict__ free_top,
                                                         int32_t *__restrict__ gcount,
                                                         int32_t *__restrict__ old_top) {
  __shared__ int lds[kPgBlock / kWave];
  const int64_t b0 = ((int64_t)blockIdx.x * kPgBlock + threadIdx.x) * kPerThread;
  const int total = block_sum<int, kPgBlock>(__popc(block_bits(rc, b0, P, is_freed)), lds);
  if (threadIdx.x == 0) {
    gcount[blockIdx.x] = total;
    if (blockIdx.x == 0) *old_top = *free_top;
  }
}

// Workgroup g pushes group g's freed blocks: a block's place is the old top plus the number
// of freed blocks with higher ids (those of later groups, then those above it here).
__global__ __launch_bounds__(kPgBlock) void k_free_push(int32_t *__restrict__ rc, int64_t P, int groups,
                                                        const int32_t *__restrict__ gcount,
                                                        const int32_t *__restrict__ old_top,
                                                        int32_t *__restrict__ fl,
                                                        int32_t *__restrict__ free_top,
                                                        int32_t *__restrict__ status) {
  __shared__ int lds[kPgBlock / kWave];
  const int g = blockIdx.x;
  const int64_t b0 = ((int64_t)g * kPgBlock + threadIdx.x) * kPerThread;
  uint32_t m = block_bits(rc, b0, P, is_freed);
  const int mine = gcount[g];
  if (mine == 0 && g != 0) return;
  int later = 0;
  for (int i = g + 1 + threadIdx.x; i < groups; i += kPgBlock) later += gcount[i];
  later = block_sum<int, kPgBlock>(later, lds);
  const int32_t raw = *old_top;
  const int64_t top = raw < 0 ? 0 : (raw > P ? P : raw);
  if (g == 0 && threadIdx.x == 0) {
    const int64_t to = top + later + mine;
    if (raw != top || to > P) atomicOr(status, SMCSD_ST_BAD_INPUT);
    *free_top = (int32_t)(to > P ? P : to);
  }
  if (mine == 0) return;
  const int n = __popc(m);
  int total;
  const int below = block_exclusive_scan<int, kPgBlock>(n, lds, &total);
  int64_t at = top + later + (total - below - n);  // freed blocks above this thread's come first
  while (m) {
    const int i = 31 - __clz((int)m);
    m &= ~(1u << i);
    rc[b0 + i] = 0;
    if (at < P) fl[at] = (int32_t)(b0 + i);
    ++at;
  }
}

// ---------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------
// map[b]: where block b goes.  Live blocks below n stay; a live block above is mover
// number j counted from the highest id down (its place among all live blocks tells j at
// once, while the number of movers is only known where id n lies); others are dead.
constexpr int32_t kMapDead = -1, kMapStay = -2;

__device__ __forceinline__ bool is_live(int32_t r) { return r > 0; }

__global__ __launch_bounds__(kPgBlock) void k_compact_count(const int32_t *__restrict__ rc, int64_t P,
                                                            int32_t *__restrict__ gcount) {
  __shared__ int lds[kPgBlock / kWave];
  const int64_t b0 = ((int64_t)blockIdx.x * kPgBlock + threadIdx.x) * kPerThread;
  const int total = block_sum<int, kPgBlock>(__popc(block_bits(rc, b0, P, is_live)), lds);
  if (threadIdx.x == 0) gcount[blockIdx.x] = total;
}

struct CompactWs {
  int32_t *gcount, *meta, *map, *holes, *movers;  // meta: live blocks, moves
};

__global__ __launch_bounds__(kPgBlock) void k_compact_rank(int32_t *__restrict__ rc, int64_t P,
                                                           int groups, CompactWs w,
                                                           int32_t *__restrict__ move_count) {
  __shared__ int lds[kPgBlock / kWave];
  const int g = blockIdx.x;
  const int64_t b0 = ((int64_t)g * kPgBlock + threadIdx.x) * kPerThread;
  const uint32_t m = block_bits(rc, b0, P, is_live);
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < groups; i += kPgBlock) {
    const int c = w.gcount[i];
    all += c;
    before += i < g ? c : 0;
  }
  before = block_sum<int, kPgBlock>(before, lds);
  const int n = block_sum<int, kPgBlock>(all, lds);
  int total;
  before += block_exclusive_scan<int, kPgBlock>(__popc(m), lds, &total);
  if (g == 0 && threadIdx.x == 0) {
    w.meta[0] = n;
    if (n == P) w.meta[1] = *move_count = 0;
  }
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t b = b0 + i;
    if (b >= P) break;
    const int rank = before + __popc(m & ((1u << i) - 1));  // live blocks below b
    int32_t to = kMapDead;
    if ((m >> i) & 1) {
      to = b < n ? kMapStay : n - 1 - rank;
      if (b >= n) w.movers[n - 1 - rank] = (int32_t)b;
    } else {
      if (rc[b] < 0) rc[b] = 0;
      if (b < n) w.holes[b - rank] = (int32_t)b;
    }
    w.map[b] = to;
    if (b == n) w.meta[1] = *move_count = n - rank;  // the live blocks from id n on
  }
}

__global__ __launch_bounds__(kPgBlock) void k_compact_apply(int32_t *__restrict__ T, int64_t entries,
                                                            int block_size, int32_t *__restrict__ rc,
                                                            int64_t P, CompactWs w,
                                                            int32_t *__restrict__ fl,
                                                            int32_t *__restrict__ free_top,
                                                            int32_t *__restrict__ moves,
                                                            int32_t *__restrict__ status) {
  const int64_t n = w.meta[0], m = w.meta[1];
  const int64_t stride = (int64_t)gridDim.x * kPgBlock, t0 = (int64_t)blockIdx.x * kPgBlock + threadIdx.x;
  if (t0 == 0) *free_top = (int32_t)(P - n);
  for (int64_t i = t0; i < m; i += stride) {
    const int32_t src = w.movers[m - 1 - i], dst = w.holes[i];
    moves[3 * i] = src;
    moves[3 * i + 1] = dst;
    moves[3 * i + 2] = block_size;
    rc[dst] = rc[src];
    rc[src] = 0;
  }
  for (int64_t i = t0; i < P - n; i += stride) fl[i] = (int32_t)(P - 1 - i);
  bool bad = false;
  for (int64_t e = t0; e < entries; e += stride) {
    const int32_t id = T[e];
    if (id == -1) continue;
    if (id < 0 || id >= P) {
      bad = true;
      continue;
    }
    const int32_t to = w.map[id];
    if (to >= 0) T[e] = w.holes[m - 1 - to];
    if (to == kMapDead) {
      T[e] = -1;
      bad = true;
    }
  }
  if (bad) atomicOr(status, SMCSD_ST_BAD_INPUT);
}

// ---------------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------------
struct CopyCaches {
  char *p[SMCSD_KV_COPY_MAX_CACHES];
};

constexpr int kCopyUnroll = 4;
constexpr uint32_t kCopyWords = 1 << 20;

// Workgroup = one (entry, cache) at a time, over all segments, four words of a thread in flight.
// W: bytes moved at once.  Bound by memory: 1.6 GB of a compaction's moves take 320 us (5.0 TB/s
// read and written, the rate of a large copy); 67 MB of copy-on-write tails 26 us (2.6 TB/s, their
// pages lie scattered and each is a few KB).
template <typename W>
__global__ __launch_bounds__(kPgBlock) void k_copy(CopyCaches caches, int n_caches, int64_t block_stride,
                                                   int segments, int64_t segment_stride,
                                                   int64_t token_bytes, int block_size,
                                                   const int32_t *__restrict__ list,
                                                   const int32_t *__restrict__ count, int64_t capacity,
                                                   int64_t P, int32_t *__restrict__ status) {
  const int32_t raw = *count;
  const int64_t entries = raw < 0 ? 0 : (raw > capacity ? capacity : raw);
  if (raw != entries && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(status, SMCSD_ST_BAD_INPUT);
  const int64_t items = entries * n_caches;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t e = it / n_caches;
    const int c = (int)(it - e * n_caches);
    const int32_t src = list[3 * e], dst = list[3 * e + 1], tokens = list[3 * e + 2];
    if (dst == -1) continue;
    if (src < 0 || src >= P || dst < 0 || dst >= P || tokens < 0 || tokens > block_size) {
      if (c == 0 && threadIdx.x == 0) atomicOr(status, SMCSD_ST_BAD_INPUT);
      continue;
    }
    if (src == dst) continue;
    const char *from = caches.p[c] + src * block_stride;
    char *to = caches.p[c] + dst * block_stride;
    const uint32_t per = (uint32_t)(tokens * token_bytes / (int)sizeof(W));  // words of a segment
    if (per == 0) continue;
    // some segments at a time, few enough for 32-bit word numbers
    const int most = (int)max(1u, kCopyWords / per);
    for (int h0 = 0; h0 < segments; h0 += most) {
      const uint32_t words = per * (uint32_t)min(most, segments - h0);
      for (uint32_t i0 = threadIdx.x; i0 < words; i0 += kPgBlock * kCopyUnroll) {
        W v[kCopyUnroll];
        int64_t off[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
          const uint32_t i = i0 + u * kPgBlock;
          const uint32_t h = i / per;
          off[u] = (h0 + (int64_t)h) * segment_stride + (int64_t)(i - h * per) * (int)sizeof(W);
          if (i < words) v[u] = *reinterpret_cast<const W *>(from + off[u]);
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
          if (i0 + u * kPgBlock < words) *reinterpret_cast<W *>(to + off[u]) = v[u];
      }
    }
  }
}

inline int64_t groups_of(int64_t P) { return ceil_div(P, kPgBlock * kPerThread); }

}  // namespace

size_t kv_free_ws_bytes(int64_t P) { return align256(sizeof(int32_t) * (size_t)(groups_of(P) + 1)); }

size_t kv_compact_ws_bytes(int64_t P) {
  return align256(sizeof(int32_t) * (size_t)(groups_of(P) + 2)) + 3 * align256(sizeof(int32_t) * (size_t)P);
}

hipError_t launch_kv_fork(const int32_t *forked, int B, int N, int32_t *T, int M, int32_t *rc, int64_t P,
                          int32_t *status, hipStream_t stream) {
  const int cols = (int)ceil_div(M, kPgBlock), parts = (int)ceil_div(N - 1, kForkRows);
  const int64_t items = (int64_t)B * cols * parts;
  if (items == 0) return hipSuccess;  // N = 1: nothing to share
  hipLaunchKernelGGL(k_fork, dim3(grid_blocks(items, kPgBlock)), dim3(kPgBlock), 0, stream, forked, B, N, T,
                     M, rc, P, status, cols, parts, items);
  return hipGetLastError();
}

hipError_t launch_kv_free(const int32_t *freed, int64_t S, int32_t *T, int M, int32_t *rc, int32_t *fl,
                          int32_t *free_top, int64_t P, int32_t *status, char *ws, hipStream_t stream) {
  const int groups = (int)groups_of(P), cols = (int)ceil_div(M, kPgBlock);
  int32_t *gcount = reinterpret_cast<int32_t *>(ws), *old_top = gcount + groups;
  hipLaunchKernelGGL(k_free_drop, dim3(grid_blocks(S * cols, kPgBlock)), dim3(kPgBlock), 0, stream, freed, S,
                     T, M, rc, P, status, cols);
  hipLaunchKernelGGL(k_free_count, dim3(groups), dim3(kPgBlock), 0, stream, rc, P, free_top, gcount, old_top);
  hipLaunchKernelGGL(k_free_push, dim3(groups), dim3(kPgBlock), 0, stream, rc, P, groups, gcount, old_top, fl, free_top,
                     status);
  return hipGetLastError();
}

hipError_t launch_kv_compact(int32_t *T, int64_t S, int M, int block_size, int32_t *rc, int32_t *fl,
                             int32_t *free_top, int64_t P, int32_t *moves, int32_t *move_count,
                             int32_t *status, char *ws, hipStream_t stream) {
  const int groups = (int)groups_of(P);
  const size_t list = align256(sizeof(int32_t) * (size_t)P);
  char *lists = ws + align256(sizeof(int32_t) * (size_t)(groups + 2));
  CompactWs w;
  w.gcount = reinterpret_cast<int32_t *>(ws);
  w.meta = w.gcount + groups;
  w.map = reinterpret_cast<int32_t *>(lists);
  w.holes = reinterpret_cast<int32_t *>(lists + list);
  w.movers = reinterpret_cast<int32_t *>(lists + 2 * list);
  hipLaunchKernelGGL(k_compact_count, dim3(groups), dim3(kPgBlock), 0, stream, rc, P, w.gcount);
  hipLaunchKernelGGL(k_compact_rank, dim3(groups), dim3(kPgBlock), 0, stream, rc, P, groups, w, move_count);
  const int64_t most = std::max<int64_t>(S * M, P);
  hipLaunchKernelGGL(k_compact_apply, dim3(grid_blocks(ceil_div(most, kPgBlock), kPgBlock)), dim3(kPgBlock),
                     0, stream, T, S * M, block_size, rc, P, w, fl, free_top, moves, status);
  return hipGetLastError();
}

hipError_t launch_kv_copy(void *const *caches, int n_caches, int64_t block_stride, int segments,
                          int64_t segment_stride, int64_t token_bytes, int block_size, const int32_t *list,
                          const int32_t *count, int64_t capacity, int64_t P, int32_t *status,
                          hipStream_t stream) {
  CopyCaches cc{};
  uint64_t low = (uint64_t)block_stride | (uint64_t)segment_stride | (uint64_t)token_bytes;
  for (int i = 0; i < n_caches; ++i) {
    cc.p[i] = static_cast<char *>(caches[i]);
    low |= reinterpret_cast<uintptr_t>(caches[i]);
  }
  const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(capacity * n_caches, 2048)));
  if (low % 16 == 0)
    hipLaunchKernelGGL(k_copy<uint4>, grid, dim3(kPgBlock), 0, stream, cc, n_caches, block_stride, segments,
                       segment_stride, token_bytes, block_size, list, count, capacity, P, status);
  else if (low % 4 == 0)
    hipLaunchKernelGGL(k_copy<uint32_t>, grid, dim3(kPgBlock), 0, stream, cc, n_caches, block_stride, segments,
                       segment_stride, token_bytes, block_size, list, count, capacity, P, status);
  else
    hipLaunchKernelGGL(k_copy<uint8_t>, grid, dim3(kPgBlock), 0, stream, cc, n_caches, block_stride, segments,
                       segment_stride, token_bytes, block_size, list, count, capacity, P, status);
  return hipGetLastError();
}

}  // namespace smcsd
