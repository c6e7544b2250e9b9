/*
 * mk_kv.cu -- page ownership of the paged KV cache (include/mk_cache.h).
 *
 * Each call is two kernels.  kv_plan, one cluster of up to 16 CTAs, does the
 * bookkeeping: it checks the arguments, adds up the holders that pages gain and
 * lose in a copy of the counts, ranks the free pages, and only then -- behind
 * the last point where the call can be refused -- writes tables, lengths and
 * counts and lists the pages to copy.  Its phases are separated by the
 * cluster's hardware barrier, so there is no spin-wait.  kv_move, on every SM,
 * copies the listed pages in all pools.  It is launched as a programmatic
 * dependent and waits for the plan on the device.
 */
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <new>

#include "mk_cache.h"

namespace {

constexpr int kMaxCluster = 16;
constexpr int kPlanThreads = 1024; /* at most */
constexpr int kSeg = 128;          /* table entries of one warp's item: 4 independent loads a lane */
constexpr int kMoveThreads = 256;
constexpr int kMoveChunk = 4096;   /* bytes of one warp's copy: 8 16-byte loads in flight a lane */
constexpr int kMaxPools = 512;
constexpr int kSource = 1 << 30;   /* mark in the new counts: this page is copied by the call */
constexpr int kMaxRefs = 1 << 28;

enum { OP_COPY = 0, OP_FORK = 1, OP_RESIZE = 2, OP_COMPACT = 3 };

struct Ctrl {
  int32_t status;   /* first refused call's status; calls change nothing while it is set */
  int32_t call_err; /* of the call in progress */
  int32_t n_copy;   /* pages for kv_move */
  int32_t remap;    /* 1: kv_move also rewrites the tables through `map` */
};

struct Params {
  int32_t num_pages, page_size, n_seqs, max_pages, n_pools, n;
  int64_t page_bytes;
  int32_t *tables, *lens, *refs;
  const int32_t *a, *b;        /* the call's DEVICE arguments */
  int32_t *page_map;           /* compact: caller's, may be NULL */
  /* workspace */
  Ctrl *ctrl;
  int32_t *err_host;
  int32_t *new_refs, *claim, *fresh, *copy_src, *copy_dst; /* claim [max(pages, seqs)], else [pages] */
  int32_t *need, *first, *len0, *len1;                     /* [n_seqs] */
  int32_t *stage;                                          /* [n_seqs][max_pages] */
  char *const *pools;                                      /* [n_pools] */
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void dependents_may_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
/* Reads the same shared variable of another CTA of the cluster. */
__device__ __forceinline__ int peer_load(const int *mine, int rank) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(mine), far;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(far) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(far) : "memory");
  return v;
}

/* Sum of the CTAs' variable, and *before: of those with a lower rank.  By whole warps. */
__device__ __forceinline__ int peer_sum(const int *mine, int rank, int ctas, int *before) {
  const int lane = threadIdx.x & 31;
  const int v = lane < ctas ? peer_load(mine, lane) : 0;
  *before = __reduce_add_sync(0xffffffffu, lane < rank ? v : 0);
  return __reduce_add_sync(0xffffffffu, v);
}

/* Exclusive prefix sum over the block; *total is the block's sum. */
__device__ int block_scan(int v, int *sums, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = lane < (int)(blockDim.x >> 5) ? sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < (int)(blockDim.x >> 5)) sums[lane] = s;
  }
  __syncthreads();
  const int before = warp ? sums[warp - 1] : 0;
  *total = sums[(blockDim.x >> 5) - 1];
  __syncthreads();
  return before + x - v;
}

/* Of several wrong arguments the largest status is kept, whichever is met first. */
__device__ __forceinline__ void refuse(const Params &p, int code) {
  atomicMax(&p.ctrl->call_err, code);
}

/* A used table entry has to name a held page.  Returns it, or -1 (refused). */
__device__ __forceinline__ int held_page(const Params &p, int page) {
  if ((unsigned)page >= (unsigned)p.num_pages || __ldcg(p.refs + page) < 1) {
    refuse(p, MK_ERR_PAGE_OOB);
    return -1;
  }
  return page;
}

__device__ __forceinline__ void list_copy(const Params &p, int src, int dst) {
  const int k = atomicAdd(&p.ctrl->n_copy, 1);
  p.copy_src[k] = src;
  p.copy_dst[k] = dst;
}

/* What bounds it: latency.  A plan reads and writes some tens to hundreds of
 * KB; its time is its chain of dependent loads (argument, length, table entry,
 * count) and its 3 to 5 cluster barriers, so every phase spreads its entries
 * over all warps with several loads in flight a lane.  With the move of pages of 32 bytes, a
 * fork of one sequence to four takes 12 us; 64 forks of up to 1025 entries take 23 us onto
 * empty rows or onto rows that agree with their source already, 30 onto rows that held
 * another source's pages (a count up and one down for every page). */
template <int OP>
__global__ void __launch_bounds__(kPlanThreads) kv_plan(const Params p) {
  __shared__ int sums[32];
  __shared__ int my_count, my_holes;
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = blockIdx.x, ctas = gridDim.x, threads = blockDim.x; /* one cluster */
  const int gtid = rank * threads + tid, nthr = ctas * threads;
  const int gwarp = gtid >> 5, nwarp = nthr >> 5;
  const int P = p.page_size, M = p.max_pages, N = p.num_pages;

  wait_for_previous();
  dependents_may_launch();
  const int held_up = __ldcg(&p.ctrl->status); /* looked at behind the first barrier */

  /* ---- 0: clear what the call counts in */
  if (OP == OP_FORK || OP == OP_RESIZE) {
    for (int i = gtid; i < N; i += nthr) p.new_refs[i] = p.refs[i];
    for (int i = gtid; i < p.n_seqs; i += nthr) p.claim[i] = 0;
  } else if (OP == OP_COPY) {
    for (int i = gtid; i < N; i += nthr) p.claim[i] = 0;
  }
  if (gtid == 0) {
    p.ctrl->call_err = 0;
    p.ctrl->n_copy = 0;
    p.ctrl->remap = 0;
  }
  cluster_sync();
  if (held_up) return; /* the same for every thread: written at a call's end only */

  /* ---- 1: check the arguments and add up */
  if (OP == OP_COPY) {
    for (int i = gtid; i < p.n; i += nthr) {
      const int s = p.a[i], d = p.b[i];
      if ((unsigned)s >= (unsigned)N || (unsigned)d >= (unsigned)N)
        refuse(p, MK_ERR_PAGE_OOB);
      else if (s != d && atomicExch(p.claim + d, 1) != 0)
        refuse(p, MK_ERR_INVALID_ARG);
    }
  }
  const unsigned nseg = (M + kSeg - 1) / kSeg;
  const unsigned items = (unsigned)(OP == OP_COMPACT ? p.n_seqs : p.n) * nseg; /* below 2^31: see create */
  if (OP == OP_FORK || OP == OP_RESIZE) {
    for (unsigned it = gwarp; it < items; it += nwarp) {
      const int i = (int)(it / nseg), seg = (int)(it - (unsigned)i * nseg);
      const int s = p.a[i], d = OP == OP_FORK ? p.b[i] : s;
      if ((unsigned)s >= (unsigned)p.n_seqs || (unsigned)d >= (unsigned)p.n_seqs) {
        if (lane == 0) refuse(p, MK_ERR_INVALID_ARG);
        continue;
      }
      const int ls = p.lens[s];
      /* fork: dst goes from `ld` to `ls`; resize: the row goes from `ls` to `ln` */
      const int ld = OP == OP_FORK ? p.lens[d] : ls, ln = OP == OP_FORK ? ls : p.b[i];
      const long long cap = (long long)M * P;
      if (ls < 0 || ld < 0 || ln < 0 || ls > cap || ld > cap || ln > cap) {
        if (lane == 0) refuse(p, MK_ERR_PAGE_OOB);
        continue;
      }
      if (seg == 0 && lane == 0) {
        if (atomicExch(p.claim + d, 1) != 0) refuse(p, MK_ERR_INVALID_ARG);
        p.len0[i] = ld;
        p.len1[i] = ln;
      }
      const int us = ls / P + (ls % P != 0), ud = ld / P + (ld % P != 0);
      const int un = ln / P + (ln % P != 0);
      if (OP == OP_FORK) {
        const int full = ls / P;
        if (seg == 0 && lane == 0) p.need[i] = (s != d && ls % P) ? 1 : 0;
        if (s == d) continue;
        int v[kSeg / 32], w[kSeg / 32];
#pragma unroll
        for (int k = 0; k < kSeg / 32; ++k) {
          const int j = seg * kSeg + k * 32 + lane;
          v[k] = j < us ? p.tables[(size_t)s * M + j] : -1;
          w[k] = j < ud ? p.tables[(size_t)d * M + j] : -1;
        }
#pragma unroll
        for (int k = 0; k < kSeg / 32; ++k) {
          const int j = seg * kSeg + k * 32 + lane;
          if (j < us) v[k] = held_page(p, v[k]);
          if (j < ud) w[k] = held_page(p, w[k]);
          if (j < us && v[k] >= 0) p.stage[(size_t)i * M + j] = v[k];
          /* a beam that follows one of its own family keeps most of its pages */
          if (j < full && v[k] == w[k]) continue;
          if (j < us && v[k] >= 0) {
            if (j < full)
              atomicAdd(p.new_refs + v[k], 1);
            else
              atomicOr(p.new_refs + v[k], kSource);
          }
          if (j < ud && w[k] >= 0) atomicAdd(p.new_refs + w[k], -1);
        }
      } else {
        const int last = us - 1;
        const bool grows = ln > ls && ls % P != 0; /* the last page may need a copy */
#pragma unroll
        for (int k = 0; k < kSeg / 32; ++k) {
          const int j = seg * kSeg + k * 32 + lane;
          if (j >= un && j < us) {
            const int q = held_page(p, p.tables[(size_t)s * M + j]);
            if (q >= 0) atomicAdd(p.new_refs + q, -1);
          }
          if (grows && j == last) {
            const int q = held_page(p, p.tables[(size_t)s * M + j]);
            const bool cow = q >= 0 && __ldcg(p.refs + q) > 1;
            if (cow) {
              atomicAdd(p.new_refs + q, -1);
              atomicOr(p.new_refs + q, kSource);
            }
            p.need[i] = un - us + (cow ? 1 : 0);
          }
        }
        if (!grows && seg == 0 && lane == 0) p.need[i] = max(0, un - us);
      }
    }
  }
  int holes = 0, live = 0; /* of this CTA's range of pages */
  const int per = (N + ctas - 1) / ctas;
  const int lo = min(N, rank * per), hi = min(N, lo + per);
  if (OP == OP_COMPACT) {
    for (unsigned it = gwarp; it < items; it += nwarp) {
      const int s = (int)(it / nseg), seg = (int)(it - (unsigned)s * nseg);
      const int ls = p.lens[s];
      if (ls < 0 || ls > (long long)M * P) {
        if (lane == 0) refuse(p, MK_ERR_PAGE_OOB);
        continue;
      }
      const int us = ls / P + (ls % P != 0);
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k) {
        const int j = seg * kSeg + k * 32 + lane;
        if (j < us) held_page(p, p.tables[(size_t)s * M + j]);
      }
    }
    for (int i = lo + tid; i < hi; i += threads) {
      const int v = p.refs[i];
      live += v > 0;
      if (v < 0) refuse(p, MK_ERR_INVALID_ARG);
    }
    int total;
    block_scan(live, sums, &total);
    if (tid == 0) my_count = total;
  }
  cluster_sync();

  /* ---- 2: rank the free pages (fork, resize), the holes and movers (compact) */
  int wanted = 0, n_live = 0;
  if (OP == OP_COPY) {
    for (int i = gtid; i < p.n; i += nthr) {
      const int s = p.a[i], d = p.b[i];
      if ((unsigned)s < (unsigned)N && s != d && __ldcg(p.claim + s) != 0)
        refuse(p, MK_ERR_INVALID_ARG);
    }
  }
  if (OP == OP_FORK || OP == OP_RESIZE) {
    /* the first turn's loads are under way together */
    const int need0 = tid < p.n ? __ldcg(p.need + tid) : 0;
    const int refs0 = lo + tid < hi ? __ldcg(p.new_refs + lo + tid) : 1;
    /* need[] is complete unless phase 1 refused.  One answer for the block: others
     * may refuse while this phase runs. */
    const bool sound = __syncthreads_or(__ldcg(&p.ctrl->call_err) != 0) == 0;
    if (sound) {
      for (int i0 = 0; i0 < p.n; i0 += threads) {
        const int i = i0 + tid;
        const int raw = i0 == 0 ? need0 : i < p.n ? __ldcg(p.need + i) : 0;
        const int v = min(raw, N + 1); /* 1024 * 2^20: no overflow */
        int total;
        const int at = block_scan(v, sums, &total);
        if (rank == 0 && i < p.n) p.first[i] = wanted + at;
        wanted = min(wanted + total, N + 1);
      }
    }
    int count = 0;
    for (int i = lo + tid; i < hi; i += threads) {
      const int v = i == lo + tid ? refs0 : __ldcg(p.new_refs + i);
      count += v == 0;
      if (v < 0 || (v & ~kSource) > kMaxRefs) refuse(p, MK_ERR_INVALID_ARG);
    }
    int total;
    block_scan(count, sums, &total);
    if (tid == 0) my_count = total;
  }
  if (OP == OP_COMPACT) {
    int base; /* live pages in the ranges before */
    n_live = peer_sum(&my_count, rank, ctas, &base);
    for (int i0 = lo; i0 < hi; i0 += threads) {
      const int i = i0 + tid;
      const int v = i < hi && p.refs[i] > 0;
      int total;
      const int at = base + block_scan(v, sums, &total); /* live pages below i */
      base += total;
      if (i < hi) {
        if (v && i >= n_live) p.copy_src[at] = i; /* at counts from the live pages that stay */
        if (!v && i < n_live) {
          p.fresh[i - at] = i;
          ++holes;
        }
        p.claim[i] = !v ? -1 : i < n_live ? i : -2; /* -2: moves, written below */
      }
    }
    int total;
    block_scan(holes, sums, &total);
    if (tid == 0) my_holes = total;
  }
  cluster_sync();

  /* ---- 3: the last point where the call can be refused */
  int err = __ldcg(&p.ctrl->call_err);
  int before = 0, n_free = 0;
  int n_moves = 0;
  if (OP == OP_FORK || OP == OP_RESIZE) {
    n_free = peer_sum(&my_count, rank, ctas, &before);
    if (err == 0 && wanted > n_free) err = MK_ERR_NO_PAGES;
  }
  if (OP == OP_COMPACT) {
    int holes_before;
    n_moves = peer_sum(&my_holes, rank, ctas, &holes_before);
  }
  if (err != 0) {
    if (gtid == 0) {
      p.ctrl->status = err;
      p.ctrl->n_copy = 0;
      *(volatile int32_t *)p.err_host = err;
      __threadfence_system();
    }
    cluster_sync(); /* no CTA ends while a peer may read its counts */
    return;
  }

  /* ---- 4: commit */
  if (OP == OP_COPY) {
    for (int i = gtid; i < p.n; i += nthr)
      if (p.a[i] != p.b[i]) list_copy(p, p.a[i], p.b[i]);
  }
  if (OP == OP_COMPACT) {
    const int stay = n_live - n_moves;
    for (int k = gtid; k < n_moves; k += nthr) {
      const int src = __ldcg(p.copy_src + stay + k), dst = __ldcg(p.fresh + k);
      p.copy_dst[stay + k] = dst;
      p.claim[src] = dst;
      p.refs[dst] = __ldcg(p.refs + src);
      p.refs[src] = 0;
      if (p.page_map) p.page_map[src] = dst;
    }
    if (p.page_map)
      for (int i = lo + tid; i < hi; i += threads) {
        const int v = __ldcg(p.claim + i);
        if (i < n_live || v == -1) p.page_map[i] = v; /* a mover's entry is written above */
      }
    if (gtid == 0) {
      p.ctrl->n_copy = n_moves;
      p.ctrl->remap = 1 + stay; /* kv_move's list starts there */
    }
    cluster_sync(); /* no CTA ends while a peer may read its counts */
  }
  if (OP == OP_FORK || OP == OP_RESIZE) {
    if (wanted > 0 && before < wanted) {
      for (int i0 = lo; i0 < hi && before < wanted; i0 += threads) {
        const int i = i0 + tid;
        const int v = i < hi && __ldcg(p.new_refs + i) == 0;
        int total;
        const int at = before + block_scan(v, sums, &total);
        before += total;
        if (v && at < wanted) {
          p.fresh[at] = i;
          p.new_refs[i] = 1;
        }
      }
    }
    cluster_sync();
    for (int i = gtid; i < N; i += nthr) p.refs[i] = __ldcg(p.new_refs + i) & ~kSource;
    for (unsigned it = gwarp; it < items; it += nwarp) {
      const int i = (int)(it / nseg), seg = (int)(it - (unsigned)i * nseg);
      const int s = p.a[i], d = OP == OP_FORK ? p.b[i] : s;
      const int l0 = __ldcg(p.len0 + i), l1 = __ldcg(p.len1 + i);
      const int u0 = l0 / P + (l0 % P != 0), u1 = l1 / P + (l1 % P != 0);
      const int first = __ldcg(p.first + i), need = __ldcg(p.need + i);
      if (OP == OP_FORK && s == d) continue;
      const int full = l1 / P;
#pragma unroll
      for (int k = 0; k < kSeg / 32; ++k) {
        const int j = seg * kSeg + k * 32 + lane;
        int32_t *at = p.tables + (size_t)d * M + j;
        if (OP == OP_FORK) {
          if (j < u1) {
            const int from = __ldcg(p.stage + (size_t)i * M + j);
            if (j < full) {
              *at = from;
            } else {
              const int to = __ldcg(p.fresh + first);
              *at = to;
              list_copy(p, from, to);
            }
          } else if (j < u0) {
            *at = -1;
          }
        } else {
          const int cow = need - max(0, u1 - u0);
          if (j >= u1 && j < u0) *at = -1;
          if (j >= u0 && j < u1) *at = __ldcg(p.fresh + first + cow + j - u0);
          if (cow && j == u0 - 1) {
            const int to = __ldcg(p.fresh + first);
            list_copy(p, *at, to);
            *at = to;
          }
        }
      }
      if (seg == 0 && lane == 0) p.lens[d] = l1;
    }
  }
}

/* Copies pages src[i] over dst[i] in every pool: reads and writes of HBM, nothing else.
 * One warp copies 4 KB at a time with all of its 16-byte loads in flight before the first
 * store, both marked as read and written once.  1024 pages of 16 KB in 96 pools (3.2 GB read
 * and written): 507 us, 6.35 TB/s, 95 % of a plain copy's; 64 pages from 8 sources, 100 MB of
 * writes and few reads: 27 us.  2 KB at a time and six blocks an SM: 513 and 31 us. */
__device__ __forceinline__ void move_pages(const Params &p, unsigned n, const int32_t *src,
                                           const int32_t *dst) {
  const long long page_bytes = p.page_bytes;
  const int lane = threadIdx.x & 31;
  const unsigned warp = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
  const unsigned nwarp = gridDim.x * (kMoveThreads / 32);
  const unsigned per_page = (unsigned)((page_bytes + kMoveChunk - 1) / kMoveChunk);
  const unsigned per_copy = per_page * p.n_pools;
  unsigned c = warp / per_copy, r = warp - c * per_copy; /* this warp's copy, its chunk among all pools' */
  while (c < n) {
    const unsigned pool = r / per_page, chunk = r - pool * per_page;
    const long long s = __ldcg(src + c), d = __ldcg(dst + c);
    r += nwarp;
    const unsigned q = r / per_copy;
    c += q;
    r -= q * per_copy;
    if (s == d) continue;
    const long long off = (long long)chunk * kMoveChunk + lane * 16;
    char *base = p.pools[pool];
    const char *from = base + s * page_bytes + off;
    char *to = base + d * page_bytes + off;
    const long long left = page_bytes - off;
    uint4 v[kMoveChunk / 512];
#pragma unroll
    for (int k = 0; k < kMoveChunk / 512; ++k)
      if (k * 512 < left) v[k] = __ldcs((const uint4 *)(from + k * 512));
#pragma unroll
    for (int k = 0; k < kMoveChunk / 512; ++k)
      if (k * 512 < left) __stcs((uint4 *)(to + k * 512), v[k]);
  }
}

/* The plan's copies, and the tables through its map of pages. */
__global__ void __launch_bounds__(kMoveThreads, 4)
    kv_move(const __grid_constant__ Params p) {
  wait_for_previous();
  dependents_may_launch();
  const int remap = __ldcg(&p.ctrl->remap), base = remap > 0 ? remap - 1 : 0;
  move_pages(p, __ldcg(&p.ctrl->n_copy), p.copy_src + base, p.copy_dst + base);
  if (remap > 0) {
    const int lane = threadIdx.x & 31;
    const unsigned warp = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5;
    const unsigned nwarp = gridDim.x * (kMoveThreads / 32);
    const unsigned nseg = (p.max_pages + 31) / 32, items = p.n_seqs * nseg;
    for (unsigned it = warp; it < items; it += nwarp) {
      const unsigned s = it / nseg;
      const long long j = (long long)(it - s * nseg) * 32 + lane;
      const int l = p.lens[s];
      if (j < l / p.page_size + (l % p.page_size != 0)) {
        int32_t *at = p.tables + (size_t)s * p.max_pages + j;
        *at = __ldcg(p.claim + *at);
      }
    }
  }
}

/* mk_kv_copy_pages for up to kFewPairs pairs and 32 KB of page bits, in one kernel: every
 * block checks all pairs against its own bits, so that none waits for another. */
constexpr int kFewPairs = 4096, kFewPages = 1 << 18;
__global__ void __launch_bounds__(kMoveThreads, 4)
    kv_copy_few(const __grid_constant__ Params p) {
  extern __shared__ unsigned target[];
  const int tid = threadIdx.x;
  const unsigned N = p.num_pages;
  for (unsigned i = tid; i < (N + 31) / 32; i += kMoveThreads) target[i] = 0;
  wait_for_previous();
  dependents_may_launch();
  const int held_up = __ldcg(&p.ctrl->status); /* by an earlier refusal, or another block's of this call */
  __syncthreads();
  bool outside = false, twice = false;
  for (int i = tid; i < p.n; i += kMoveThreads) {
    const unsigned s = p.a[i], d = p.b[i];
    if (s >= N || d >= N)
      outside = true;
    else if (s != d)
      twice |= (atomicOr(target + d / 32, 1u << d % 32) >> d % 32) & 1;
  }
  outside = __syncthreads_or(outside);
  for (int i = tid; i < p.n; i += kMoveThreads) {
    const unsigned s = p.a[i];
    twice |= s < N && s != (unsigned)p.b[i] && (target[s / 32] >> s % 32 & 1);
  }
  twice = __syncthreads_or(twice);
  if (held_up) return;
  if (outside || twice) {
    if (blockIdx.x == 0 && tid == 0) {
      const int err = outside ? MK_ERR_PAGE_OOB : MK_ERR_INVALID_ARG;
      p.ctrl->status = err;
      *(volatile int32_t *)p.err_host = err;
      __threadfence_system();
    }
    return;
  }
  move_pages(p, p.n, p.a, p.b);
}

/* ---- keep: rows of a sequence's picked tokens move together ------------------- */

struct Keep {
  Params p; /* n sequences a[i] */
  const int32_t *starts, *offsets, *picks;
  int32_t n_picks, heads, row_chunks; /* kv heads of a page; 16-byte pieces of a token's row in one */
  int32_t units;                      /* such pieces of a token in all pools */
  unsigned warps;                     /* warps' shares of a sequence's pieces */
};

/* Whether the sequence and the range of picks of entry i can be looked at. */
__device__ __forceinline__ bool keep_sound(const Keep &a, int i, int s, int lo, int hi) {
  return (unsigned)s < (unsigned)a.p.n_seqs && lo >= 0 && hi >= lo && hi <= a.n_picks && (i > 0 || lo == 0);
}
/* The j-th pick of an entry that begins at place `start` in row s; `before` is the one before it.  x
 * and y of rows are the page and the place in it where the token lies, z and w where it goes; x is -1
 * where they cannot be told.  Returns a status, for all but the pages' holders. */
__device__ __forceinline__ int keep_pick(const Keep &a, int s, int start, int pick, int before, int j, int4 *rows) {
  const Params &p = a.p;
  const int P = p.page_size;
  const long long from = (long long)start + pick, cap = (long long)p.max_pages * P;
  *rows = make_int4(-1, 0, -1, 0);
  if (pick <= before) return MK_ERR_INVALID_ARG;
  if (start < 0 || from >= cap) return MK_ERR_PAGE_OOB;
  if (pick < j) return MK_OK; /* one before it is wrong, which its own check reports */
  const int32_t *row = p.tables + (size_t)s * p.max_pages;
  const int to = start + j, len = __ldcg(p.lens + s);
  const int src = __ldcg(row + (int)from / P), dst = __ldcg(row + to / P);
  if (len > cap || from >= len || (unsigned)src >= (unsigned)p.num_pages || (unsigned)dst >= (unsigned)p.num_pages)
    return MK_ERR_PAGE_OOB;
  *rows = make_int4(src, (int)from % P, dst, to % P);
  return MK_OK;
}
/* Both pages have to be held, and the one that a token moves to by nobody else. */
__device__ __forceinline__ int keep_holders(const Keep &a, const int4 &rows) {
  if (rows.x < 0) return MK_OK; /* reported already */
  const int to = __ldcg(a.p.refs + rows.z), from = __ldcg(a.p.refs + rows.x);
  if (to < 1 || from < 1) return MK_ERR_PAGE_OOB;
  return to > 1 && (rows.x != rows.z || rows.y != rows.w) ? MK_ERR_INVALID_ARG : MK_OK;
}

/* Where a token's row begins in a pool's head 0, in bytes: now (x, -1 where that cannot be told) and
 * afterwards (y). */
__device__ __forceinline__ longlong2 keep_bytes(const Keep &a, const int4 &rows) {
  const long long row_bytes = 16ll * a.row_chunks;
  return rows.x < 0 ? make_longlong2(-1, -1)
                    : make_longlong2(rows.x * a.p.page_bytes + rows.y * row_bytes,
                                     rows.z * a.p.page_bytes + rows.w * row_bytes);
}

/* A warp's 32 pieces of every picked token of one sequence.  A lane has the same 16 bytes of each,
 * and takes them in order, eight loads ahead of their stores: a token goes to a place at or before
 * its own and the picks rise, so no store touches what is still to be loaded.  `bytes_of` gives
 * keep_bytes of one pick to all lanes. */
struct Mover {
  char *base;
  bool mine;
  uint4 v[8];
  char *to[8];
  __device__ __forceinline__ Mover(const Keep &a, unsigned share) {
    const Params &p = a.p;
    const int unit = (int)share * 32 + (threadIdx.x & 31);
    mine = unit < a.units;
    const int per_pool = a.heads * a.row_chunks, pool = mine ? unit / per_pool : 0;
    const int rest = unit - pool * per_pool, head = rest / a.row_chunks;
    base = p.pools[pool] + (long long)head * p.page_size * (16ll * a.row_chunks) + (rest - head * a.row_chunks) * 16;
  }
  template <class F>
  __device__ __forceinline__ void load(int j0, int count, F bytes_of) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      to[k] = nullptr;
      if (j0 + k >= count) continue;
      const longlong2 at = bytes_of(j0 + k);
      if (!mine || at.x < 0 || at.x == at.y) continue;
      to[k] = base + at.y;
      v[k] = __ldcg((const uint4 *)(base + at.x));
    }
  }
  __device__ __forceinline__ void store() const {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (to[k]) __stcg((uint4 *)to[k], v[k]);
  }
};

/* Checks all picks, one cluster, and lets kv_keep_rows go on or not. */
__global__ void __launch_bounds__(kPlanThreads) kv_keep_plan(const __grid_constant__ Keep a) {
  const Params &p = a.p;
  const int lane = threadIdx.x & 31;
  const int gtid = blockIdx.x * blockDim.x + threadIdx.x, nthr = gridDim.x * blockDim.x;
  wait_for_previous();
  dependents_may_launch();
  const int held_up = __ldcg(&p.ctrl->status);
  for (int i = gtid; i < p.n_seqs; i += nthr) p.claim[i] = 0;
  if (gtid == 0) {
    p.ctrl->call_err = 0;
    p.ctrl->n_copy = 0;
    p.ctrl->remap = 0;
  }
  cluster_sync();
  if (held_up) return;
  for (int i = gtid; i < p.n; i += nthr) {
    const int s = __ldcg(p.a + i);
    if (!keep_sound(a, i, s, __ldcg(a.offsets + i), __ldcg(a.offsets + i + 1)) ||
        atomicExch(p.claim + s, 1) != 0)
      refuse(p, MK_ERR_INVALID_ARG);
  }
  cluster_sync();
  int err = __ldcg(&p.ctrl->call_err); /* the same for all: the next refusal comes behind a barrier */
  cluster_sync();
  if (err == 0) {
    for (int i = gtid >> 5; i < p.n; i += nthr >> 5) {
      const int s = __ldcg(p.a + i), lo = __ldcg(a.offsets + i), hi = __ldcg(a.offsets + i + 1);
      const int start = __ldcg(a.starts + i);
      for (int k = lo + lane; k < hi; k += 32) {
        int4 rows;
        int e = keep_pick(a, s, start, __ldcg(a.picks + k), k > lo ? __ldcg(a.picks + k - 1) : -1, k - lo, &rows);
        if (!e) e = keep_holders(a, rows);
        if (e) refuse(p, e);
      }
    }
    cluster_sync();
    err = __ldcg(&p.ctrl->call_err);
  }
  if (gtid == 0) {
    p.ctrl->n_copy = err == 0;
    if (err) {
      p.ctrl->status = err;
      *(volatile int32_t *)p.err_host = err;
      __threadfence_system();
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 4) kv_keep_rows(const __grid_constant__ Keep a) {
  wait_for_previous();
  dependents_may_launch();
  if (__ldcg(&a.p.ctrl->n_copy) == 0) return;
  const int lane = threadIdx.x & 31;
  const unsigned long long nwarp = gridDim.x * (kMoveThreads / 32), all = (unsigned long long)a.warps * a.p.n;
  for (unsigned long long w = (blockIdx.x * kMoveThreads + threadIdx.x) >> 5; w < all; w += nwarp) {
    const int i = (int)(w / a.warps);
    const int s = __ldcg(a.p.a + i), lo = __ldcg(a.offsets + i), n = __ldcg(a.offsets + i + 1) - lo;
    const int start = __ldcg(a.starts + i);
    longlong2 mine;
    auto bytes_of = [&](int j) {
      if (j % 32 == 0 && j + lane < n) {
        int4 rows;
        keep_pick(a, s, start, __ldcg(a.picks + lo + j + lane), -1, j + lane, &rows);
        mine = keep_bytes(a, rows);
      }
      return make_longlong2(__shfl_sync(0xffffffffu, mine.x, j & 31), __shfl_sync(0xffffffffu, mine.y, j & 31));
    };
    Mover m(a, (unsigned)(w - (unsigned long long)i * a.warps));
    for (int j0 = 0; j0 < n; j0 += 8) {
      m.load(j0, n, bytes_of);
      m.store();
    }
  }
}

/* Both in one kernel, for up to kFewKept sequences and kFewPicks picks: every block checks all of
 * them, so that none waits for another, and finds their rows on the way.  Three loads in a row
 * (picks, tables, and holders with the first rows under way) and two barriers stand before the first
 * store.  64 paths of up to 8 tokens in 96 pools, 44 MB read and written in rows of 256 bytes, take
 * 13.0 us, 4 paths in 16 pools 3.3 (14.4 with pages and places in the list instead of bytes; 17.2 in
 * blocks of 256 threads, four an SM and each with the same checks to make). */
constexpr int kFewKept = 1024, kFewPicks = 2048, kKeepThreads = 512;
constexpr int keep_few_bytes(int n, int n_picks, int n_seqs) {
  return n_picks * 16 + (3 * n + 1) * 4 + (n_seqs + 31) / 32 * 4;
}
__global__ void __launch_bounds__(kKeepThreads, 2) kv_keep_few(const __grid_constant__ Keep a) {
  extern __shared__ longlong2 bytes[]; /* keep_bytes [n_picks], offsets [n + 1], sequences, starts [n], a bit a row */
  const Params &p = a.p;
  const int tid = threadIdx.x, n = p.n;
  int *off = (int *)(bytes + a.n_picks), *seq = off + n + 1, *start = seq + n;
  unsigned *claim = (unsigned *)(start + n);
  __shared__ int s_flags; /* 1: entries, 2: picks out of range, 4: picks wrong */
  for (int i = tid; i < (p.n_seqs + 31) / 32; i += kKeepThreads) claim[i] = 0;
  if (tid == 0) s_flags = 0;
  wait_for_previous();
  dependents_may_launch();
  const int held_up = __ldcg(&p.ctrl->status); /* by an earlier refusal, or another block's of this call */
  int pick = tid < a.n_picks ? __ldcg(a.picks + tid) : 0;
  int before = tid && tid < a.n_picks ? __ldcg(a.picks + tid - 1) : -1;
  for (int i = tid; i <= n; i += kKeepThreads) {
    off[i] = __ldcg(a.offsets + i);
    if (i < n) {
      seq[i] = __ldcg(p.a + i);
      start[i] = __ldcg(a.starts + i);
    }
  }
  __syncthreads();
  int flags = 0;
  for (int i = tid; i < n; i += kKeepThreads) {
    const int s = seq[i];
    if (!keep_sound(a, i, s, off[i], off[i + 1]) || (atomicOr(claim + s / 32, 1u << s % 32) >> s % 32 & 1)) flags |= 1;
  }
  const int used = min(off[n], a.n_picks);
  int4 mine = make_int4(-1, 0, -1, 0); /* of this thread's first pick, whose holders are looked up below */
  for (int k = tid; k < used; k += kKeepThreads) {
    if (k != tid) {
      pick = __ldcg(a.picks + k);
      before = __ldcg(a.picks + k - 1);
    }
    int lo = 0, hi = n - 1; /* the last entry that begins at or before it, where offsets are in order */
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (off[m] <= k)
        lo = m;
      else
        hi = m - 1;
    }
    const int j = k - off[lo], s = seq[lo];
    bytes[k] = make_longlong2(-1, -1);
    if (j < 0 || (unsigned)s >= (unsigned)p.n_seqs) continue; /* an entry that is not sound */
    int4 rows;
    int e = keep_pick(a, s, start[lo], pick, j ? before : -1, j, &rows);
    bytes[k] = keep_bytes(a, rows);
    if (k == tid)
      mine = rows;
    else if (!e)
      e = keep_holders(a, rows);
    flags |= e == MK_ERR_PAGE_OOB ? 2 : e ? 4 : 0;
  }
  if (flags) atomicOr(&s_flags, flags);
  __syncthreads();
  const unsigned nwarp = gridDim.x * (kKeepThreads / 32), all = a.warps * n;
  unsigned w = (blockIdx.x * kKeepThreads + tid) >> 5;
  const bool sound = !(s_flags & 1) && w < all; /* its entries: else their rows are not in order */
  int i = sound ? (int)(w / a.warps) : 0, first = sound ? off[i] : 0, count = sound ? off[i + 1] - first : 0;
  Mover m(a, w - i * a.warps);
  auto bytes_of = [&](int j) { return bytes[first + j]; };
  m.load(0, count, bytes_of);
  const int e = keep_holders(a, mine);
  if (e) atomicOr(&s_flags, e == MK_ERR_PAGE_OOB ? 2 : 4);
  __syncthreads();
  if (held_up) return;
  if (s_flags) {
    if (blockIdx.x == 0 && tid == 0) {
      const int err = s_flags & 1 ? MK_ERR_INVALID_ARG : s_flags & 2 ? MK_ERR_PAGE_OOB : MK_ERR_INVALID_ARG;
      p.ctrl->status = err;
      *(volatile int32_t *)p.err_host = err;
      __threadfence_system();
    }
    return;
  }
  while (true) {
    m.store();
    for (int j0 = 8; j0 < count; j0 += 8) {
      m.load(j0, count, bytes_of);
      m.store();
    }
    w += nwarp;
    if (w >= all) break;
    i = (int)(w / a.warps);
    first = off[i];
    count = off[i + 1] - first;
    m = Mover(a, w - i * a.warps);
    m.load(0, count, bytes_of);
  }
}

/* Makes `dev` current for a scope: a handle may be called with another device
 * current. */
struct OnDevice {
  int was = 0;
  bool ok = true, changed = false;
  explicit OnDevice(int dev) {
    ok = cudaGetDevice(&was) == cudaSuccess;
    if (ok && was != dev) {
      ok = cudaSetDevice(dev) == cudaSuccess;
      changed = ok;
    }
  }
  ~OnDevice() {
    if (changed) cudaSetDevice(was);
  }
};

}  // namespace

struct mk_kv {
  mk_kv_desc d{};
  Params base{};
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0, max_cluster = kMaxCluster;
  uint8_t *ws = nullptr;
  int32_t *err_host = nullptr;
};

namespace {

template <int OP>
cudaError_t launch_plan(const mk_kv *kv, const Params &p) {
  /* 8 CTAs of 512 threads, or the largest cluster (16 CTAs) of 1024, which begins later and
   * has four times the warps for the rows' segments and the pages.  Both times, a fork of n
   * rows of 30 entries and their release: 128 rows over 4036 pages 20.9 and 26.3 us, 256 over
   * 8004 27.3 and 26.2, 384 over 11972 34.5 and 27.2; 16 rows of 1000 over 18024 25.5 and
   * 27.3, 32 over 34040 35.9 and 29.0; 4 rows of 8 over 16384 pages 23.0 and 24.4, over 32768
   * 27.1 and 25.7, over 65536 35.1 and 27.7. */
  const long long segs = (p.max_pages + kSeg - 1) / kSeg * (long long)(OP == OP_COMPACT ? p.n_seqs : p.n);
  const bool large = OP == OP_COPY || segs + p.num_pages / 128 > 288;
  const int ctas = large ? kv->max_cluster : std::min(8, kv->max_cluster);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(large ? kPlanThreads : kPlanThreads / 2);
  cfg.stream = kv->stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)ctas, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_plan<OP>, p);
}

/* The largest cluster of a plan that this device takes. */
template <class Kernel>
cudaError_t allow_clusters(Kernel plan, int *largest) {
  cudaError_t e = cudaFuncSetAttribute(plan, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kPlanThreads);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  for (; *largest > 1; *largest /= 2) {
    int n = 0;
    cfg.gridDim = dim3(*largest);
    at[0].val.clusterDim = {(unsigned)*largest, 1, 1};
    if (cudaOccupancyMaxActiveClusters(&n, plan, &cfg) == cudaSuccess && n > 0) break;
    cudaGetLastError(); /* a size too large is no error of the caller's */
  }
  return cudaSuccess;
}

typedef void (*MoveKernel)(Params);

/* max_copies bounds the pages that are copied. */
mk_status launch_move(mk_kv *kv, MoveKernel k, const Params &p, long long max_copies,
                      long long extra_warps, size_t smem) {
  const long long per_copy =
      (kv->d.page_bytes + kMoveChunk - 1) / kMoveChunk * (long long)kv->d.n_pools;
  const long long warps = std::max(max_copies * per_copy, extra_warps);
  const long long want = (warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::max(1LL, std::min(want, (long long)kv->n_sm * 4)));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = kv->stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

template <int OP>
mk_status submit(mk_kv *kv, const Params &p, long long max_copies, long long extra_warps) {
  OnDevice on(kv->dev);
  if (!on.ok) return MK_ERR_CUDA;
  if (OP == OP_COPY && p.n <= kFewPairs && p.num_pages <= kFewPages)
    return launch_move(kv, kv_copy_few, p, max_copies, 0, ((size_t)p.num_pages + 31) / 32 * 4);
  if (launch_plan<OP>(kv, p) != cudaSuccess) return MK_ERR_CUDA;
  return launch_move(kv, kv_move, p, max_copies, extra_warps, 0);
}

bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace

extern "C" {

mk_status mk_kv_create(const mk_kv_desc *d, void *stream, mk_kv **out) {
  if (!d || !out) return MK_ERR_INVALID_ARG;
  if (d->n_pools < 1 || d->num_pages < 1 || d->page_size < 1 || d->n_seqs < 1 ||
      d->max_pages_per_seq < 1 || d->page_bytes < 16 || d->page_bytes % 16)
    return MK_ERR_INVALID_ARG;
  if (d->n_pools > kMaxPools || d->num_pages > (1 << 20) || d->n_seqs > 65536 ||
      (int64_t)d->max_pages_per_seq * d->page_size > INT32_MAX ||
      d->page_bytes > ((int64_t)1 << 32) ||
      (int64_t)d->n_seqs * d->max_pages_per_seq > (int64_t)1 << 30)
    return MK_ERR_UNSUPPORTED;
  if (!d->pools || !d->page_tables || !d->seq_lens || !d->page_refs || !aligned4(d->page_tables) ||
      !aligned4(d->seq_lens) || !aligned4(d->page_refs))
    return MK_ERR_INVALID_ARG;
  for (int i = 0; i < d->n_pools; ++i)
    if (!d->pools[i] || ((uintptr_t)d->pools[i] & 15u)) return MK_ERR_INVALID_ARG;
  int dev = 0;
  cudaDeviceProp prop;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaGetDeviceProperties(&prop, dev) != cudaSuccess)
    return MK_ERR_NO_DEVICE;
  if (prop.major != 10 || prop.minor != 3) return MK_ERR_NO_DEVICE;

  mk_kv *kv = new (std::nothrow) mk_kv();
  if (!kv) return MK_ERR_CUDA;
  kv->d = *d;
  kv->d.pools = nullptr;
  kv->stream = (cudaStream_t)stream;
  kv->dev = dev;
  kv->n_sm = prop.multiProcessorCount;
  const size_t N = d->num_pages, S = d->n_seqs, M = d->max_pages_per_seq;
  size_t off = 0;
  auto take = [&](size_t ints) {
    const size_t o = off;
    off += (ints * 4 + 255) / 256 * 256;
    return o;
  };
  const size_t o_ctrl = take(sizeof(Ctrl) / 4), o_refs = take(N), o_claim = take(std::max(N, S)),
               o_fresh = take(N), o_src = take(N), o_dst = take(N), o_need = take(S),
               o_first = take(S), o_len0 = take(S), o_len1 = take(S), o_stage = take(S * M), o_pools = take(2 * (size_t)d->n_pools);
  cudaError_t e = allow_clusters(kv_plan<OP_COPY>, &kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters(kv_plan<OP_FORK>, &kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters(kv_plan<OP_RESIZE>, &kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters(kv_plan<OP_COMPACT>, &kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters(kv_keep_plan, &kv->max_cluster);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kv_keep_few, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             keep_few_bytes(kFewKept, kFewPicks, 65536));
  if (e == cudaSuccess) e = cudaMalloc(&kv->ws, off);
  if (e == cudaSuccess) e = cudaMemsetAsync(kv->ws, 0, off, kv->stream);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(kv->ws + o_pools, d->pools, sizeof(void *) * d->n_pools,
                        cudaMemcpyHostToDevice, kv->stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(kv->stream);
  if (e == cudaSuccess) e = cudaHostAlloc(&kv->err_host, 64, cudaHostAllocMapped);
  Params &p = kv->base;
  if (e == cudaSuccess) {
    std::memset(kv->err_host, 0, 64);
    e = cudaHostGetDevicePointer((void **)&p.err_host, kv->err_host, 0);
  }
  if (e != cudaSuccess) {
    mk_kv_destroy(kv);
    cudaGetLastError(); /* reported here: not to the caller's next launch as well */
    return MK_ERR_CUDA;
  }
  p.num_pages = d->num_pages;
  p.page_size = d->page_size;
  p.n_seqs = d->n_seqs;
  p.max_pages = d->max_pages_per_seq;
  p.n_pools = d->n_pools;
  p.page_bytes = d->page_bytes;
  p.pools = (char *const *)(kv->ws + o_pools);
  p.tables = d->page_tables;
  p.lens = d->seq_lens;
  p.refs = d->page_refs;
  p.ctrl = (Ctrl *)(kv->ws + o_ctrl);
  p.new_refs = (int32_t *)(kv->ws + o_refs);
  p.claim = (int32_t *)(kv->ws + o_claim);
  p.fresh = (int32_t *)(kv->ws + o_fresh);
  p.copy_src = (int32_t *)(kv->ws + o_src);
  p.copy_dst = (int32_t *)(kv->ws + o_dst);
  p.need = (int32_t *)(kv->ws + o_need);
  p.first = (int32_t *)(kv->ws + o_first);
  p.len0 = (int32_t *)(kv->ws + o_len0);
  p.len1 = (int32_t *)(kv->ws + o_len1);
  p.stage = (int32_t *)(kv->ws + o_stage);
  *out = kv;
  return MK_OK;
}

void mk_kv_destroy(mk_kv *kv) {
  if (!kv) return;
  {
    OnDevice on(kv->dev);
    cudaStreamSynchronize(kv->stream);
    if (kv->ws) cudaFree(kv->ws);
    if (kv->err_host) cudaFreeHost(kv->err_host);
  }
  delete kv;
}

mk_status mk_kv_copy_pages(mk_kv *kv, int32_t n, const int32_t *src, const int32_t *dst) {
  if (!kv || n < 0 || n > kv->d.num_pages) return MK_ERR_INVALID_ARG;
  if (n == 0) return MK_OK;
  if (!src || !dst || !aligned4(src) || !aligned4(dst)) return MK_ERR_INVALID_ARG;
  Params p = kv->base;
  p.n = n;
  p.a = src;
  p.b = dst;
  return submit<OP_COPY>(kv, p, n, 0);
}

mk_status mk_kv_fork(mk_kv *kv, int32_t n, const int32_t *src, const int32_t *dst) {
  if (!kv || n < 0 || n > kv->d.n_seqs) return MK_ERR_INVALID_ARG;
  if (n == 0) return MK_OK;
  if (!src || !dst || !aligned4(src) || !aligned4(dst)) return MK_ERR_INVALID_ARG;
  Params p = kv->base;
  p.n = n;
  p.a = src;
  p.b = dst;
  return submit<OP_FORK>(kv, p, n, 0);
}

mk_status mk_kv_resize(mk_kv *kv, int32_t n, const int32_t *seqs, const int32_t *new_lens) {
  if (!kv || n < 0 || n > kv->d.n_seqs) return MK_ERR_INVALID_ARG;
  if (n == 0) return MK_OK;
  if (!seqs || !new_lens || !aligned4(seqs) || !aligned4(new_lens)) return MK_ERR_INVALID_ARG;
  Params p = kv->base;
  p.n = n;
  p.a = seqs;
  p.b = new_lens;
  return submit<OP_RESIZE>(kv, p, n, 0);
}

mk_status mk_kv_compact(mk_kv *kv, int32_t *page_map) {
  if (!kv || !aligned4(page_map)) return MK_ERR_INVALID_ARG;
  Params p = kv->base;
  p.page_map = page_map;
  const long long rows = (long long)kv->d.n_seqs * ((kv->d.max_pages_per_seq + 31) / 32);
  return submit<OP_COMPACT>(kv, p, kv->d.num_pages / 2, rows);
}

mk_status mk_kv_keep(mk_kv *kv, int32_t n, const int32_t *seqs, const int32_t *starts,
                     const int32_t *offsets, int32_t n_picks, const int32_t *picks,
                     int32_t n_kv_heads) {
  if (!kv || n < 0 || n > kv->d.n_seqs || n_picks < 0 || n_kv_heads < 1) return MK_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)n_kv_heads * kv->d.page_size; /* of a page: tokens times heads */
  if (kv->d.page_bytes % rows || kv->d.page_bytes / rows % 16) return MK_ERR_INVALID_ARG;
  if (n == 0) return MK_OK;
  if (!seqs || !starts || !offsets || (n_picks && !picks) || !aligned4(seqs) || !aligned4(starts) ||
      !aligned4(offsets) || !aligned4(picks))
    return MK_ERR_INVALID_ARG;
  Keep a{};
  a.p = kv->base;
  a.p.n = n;
  a.p.a = seqs;
  a.starts = starts;
  a.offsets = offsets;
  a.picks = picks;
  a.n_picks = n_picks;
  a.heads = n_kv_heads;
  a.row_chunks = (int32_t)(kv->d.page_bytes / rows / 16);
  const int64_t units = (int64_t)kv->d.n_pools * a.heads * a.row_chunks;
  if (units > (1 << 24)) return MK_ERR_UNSUPPORTED; /* 256 MB a token */
  a.units = (int32_t)units;
  a.warps = (unsigned)((units + 31) / 32);
  OnDevice on(kv->dev);
  if (!on.ok) return MK_ERR_CUDA;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = kv->stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const long long warps = (long long)a.warps * n;
  const unsigned blocks = (unsigned)std::min((warps + kMoveThreads / 32 - 1) / (kMoveThreads / 32), (long long)kv->n_sm * 4);
  if (n <= kFewKept && n_picks <= kFewPicks) {
    cfg.gridDim = dim3((unsigned)std::min((warps + kKeepThreads / 32 - 1) / (kKeepThreads / 32), (long long)kv->n_sm * 2));
    cfg.blockDim = dim3(kKeepThreads);
    cfg.dynamicSmemBytes = keep_few_bytes(n, n_picks, kv->d.n_seqs);
    return cudaLaunchKernelEx(&cfg, kv_keep_few, a) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
  }
  cfg.gridDim = dim3(kv->max_cluster);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.numAttrs = 2;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim = {(unsigned)kv->max_cluster, 1, 1};
  if (cudaLaunchKernelEx(&cfg, kv_keep_plan, a) != cudaSuccess) return MK_ERR_CUDA;
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_keep_rows, a) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_kv_sync(mk_kv *kv) {
  if (!kv) return MK_ERR_INVALID_ARG;
  OnDevice on(kv->dev);
  if (!on.ok) return MK_ERR_CUDA;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(kv->stream, &cap) != cudaSuccess) return MK_ERR_CUDA;
  if (cap != cudaStreamCaptureStatusNone) return MK_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(kv->stream) != cudaSuccess) return MK_ERR_CUDA;
  const int32_t code = *(volatile int32_t *)kv->err_host;
  if (code == 0) return MK_OK;
  *(volatile int32_t *)kv->err_host = 0;
  if (cudaMemsetAsync(&kv->base.ctrl->status, 0, sizeof(int32_t), kv->stream) != cudaSuccess)
    return MK_ERR_CUDA;
  return code;
}

}  // extern "C"
