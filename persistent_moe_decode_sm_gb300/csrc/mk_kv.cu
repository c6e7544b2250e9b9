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

/* The largest cluster of kv_plan that this device takes. */
template <int OP>
cudaError_t allow_clusters(int *largest) {
  cudaError_t e = cudaFuncSetAttribute(kv_plan<OP>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    if (cudaOccupancyMaxActiveClusters(&n, kv_plan<OP>, &cfg) == cudaSuccess && n > 0) break;
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
  cudaError_t e = allow_clusters<OP_COPY>(&kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters<OP_FORK>(&kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters<OP_RESIZE>(&kv->max_cluster);
  if (e == cudaSuccess) e = allow_clusters<OP_COMPACT>(&kv->max_cluster);
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
