/*
 * mk_attn.cu -- attention of a batch over paged K and V whose leading pages
 * sequences share (include/mk_cache.h).
 *
 * The work is cut into tiles of 128 keys.  An item is a range of keys that a
 * set of query rows reads: a group's shared pages with all rows (query tokens x
 * heads of one kv head) of the group's sequences, 256 rows at a time, or one
 * sequence's own pages with that sequence's rows.  All items' tiles lie end to
 * end on one line, cut evenly over the SMs, so a CTA's share may begin and end
 * inside an item; every piece leaves a partial (maximum, sum, weighted sum) per
 * row, and attn_merge joins them.  The cut follows from the lengths on the
 * device: each CTA takes it itself, so that a captured call follows its batch.
 *
 * attn_tiles, one CTA per SM: a producer warp moves K and V tiles with TMA, one
 * box per page and 64 dims, into swizzled shared memory; one thread issues
 * S = Q K^T and O += P V on the tensor cores (tcgen05, 128 rows, accumulators in
 * TMEM); two warpgroups turn S into P, one row a thread, P going back to TMEM
 * as the A operand.  The two work on their own S, P and O, so that one's
 * softmax runs under the other's products: on two tiles of rows over the same
 * keys where an item has more than 128 rows, else on the even and odd key tiles
 * of the same rows, joined at the piece's end.
 */
#include <cuda.h> /* tensor-map types; the encoder is reached through the runtime */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "mk_cache.h"
#include "mk_plan.h"

namespace {

constexpr int kThreads = 320;      /* 8 softmax warps, the producer, the issuer */
constexpr int kTile = 128;         /* keys per tile; rows per row tile */
constexpr int kMaxSeqs = 1024;     /* of a call: the cut's tables are in shared memory */
constexpr uint64_t kWaitLimit = 2000000000ull; /* ns */
/* The running maximum moves only when a score exceeds it by this much (in powers
 * of two): P then stays below 2^8, exact in its relative precision, and the
 * accumulator is rescaled a few times per row rather than in most tiles. */
constexpr float kSlack = 8.0f;

struct Args {
  int32_t Hq, Hkv, G, P, num_pages, max_pages, n_seqs, n_tokens, n_groups, box_rows;
  const int32_t *tables, *lens, *off, *starts, *prefix;
  const __nv_bfloat16 *q;
  long long q_stride;
  __nv_bfloat16 *out;
  float *lse;
  float scale_log2; /* scale * log2(e) */
  int32_t *err_host;
  /* workspace */
  int32_t *sched;    /* the cut, for attn_merge: [0] bad, [1] groups' units, [2] all units, then
                      * [kMaxSeqs + 1] each: cumulated units of the groups, of the sequences,
                      * the groups' shared keys */
  float *part;       /* [2 * n_tokens * Hq + grid * 256][D] weighted sums */
  float2 *part_ml;   /* the same rows: maximum (in powers of two), sum */
};

template <int D>
struct Cfg {
  static constexpr int COLS = D < 64 ? D : 64;     /* dims of one swizzled row */
  static constexpr int NH = D / COLS;              /* such column blocks of a tile */
  static constexpr int ROWB = COLS * 2;            /* bytes of a row: the swizzle's width */
  static constexpr int BLOCK = kTile * ROWB;       /* bytes of one column block */
  static constexpr int TILE = BLOCK * NH;
  static constexpr int STAGES = D == 128 ? 2 : 4;  /* of K and of V: 128 or 64 KB in flight */
  static constexpr uint64_t SWIZZLE = D < 64 ? 4 : 2; /* matrix descriptors: 64, 128 bytes */
  static constexpr int SMEM = 1024 + TILE * (2 + 2 * STAGES);
};

struct Smem { /* behind the tiles */
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t sfull[2], pready[2], qready[2], oready[2], xfull, xfree, drain;
  uint32_t tmem;
  int abort;
  int sums[kThreads / 32];
  int total_g, total;
  float xm[kTile], xl[kTile];
  int32_t off[kMaxSeqs + 1], len[kMaxSeqs], start[kMaxSeqs], cum_s[kMaxSeqs + 1];
  int32_t gs[kMaxSeqs + 1], plen[kMaxSeqs], lead[kMaxSeqs], cum_g[kMaxSeqs + 1];
};

/* ---- PTX -------------------------------------------------------------------- */

__device__ __forceinline__ uint32_t saddr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint64_t *b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t *b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
/* Waits for a phase; false when another role gave up or the limit ran out. */
__device__ bool bar_wait(uint64_t *b, uint32_t parity, volatile int *abort) {
  const uint32_t a = saddr(b);
  uint64_t since = 0;
  for (int i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(a), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if ((i & 63) == 63) {
      const uint64_t t = now_ns();
      if (!since)
        since = t;
      else if (t - since > kWaitLimit) {
        *abort = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, volatile int *abort) {
  return __all_sync(0xffffffffu, bar_wait(b, parity, abort));
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                       uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(saddr(bar))
      : "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   saddr(bar))
               : "memory");
}
/* D (+)= A B with A and B in shared memory, or A in TMEM. */
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
#define R8(x, i) x(i), x(i + 1), x(i + 2), x(i + 3), x(i + 4), x(i + 5), x(i + 6), x(i + 7)
#define R32(x, i) R8(x, i), R8(x, i + 8), R8(x, i + 16), R8(x, i + 24)
/* 32 or 128 columns of this thread's TMEM lane.  The load and its wait are one
 * statement: between two, the compiler could move registers that have not landed. */
__device__ __forceinline__ void tmem_ld32(uint32_t at, float *v) {
#define OUT(i) "=f"(v[i])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R32(OUT, 0)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_ld128(uint32_t at, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
      "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
      "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
      "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
      "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R32(OUT, 0), R32(OUT, 32), R32(OUT, 64), R32(OUT, 96)
      : "r"(at)
      : "memory");
#undef OUT
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *v) {
#define IN(i) "r"(v[i])
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31};" ::R32(IN, 0),
      "r"(at)
      : "memory");
#undef IN
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
/* Shared-memory matrix descriptor: swizzled rows, `sbo` bytes from one group of
 * 8 rows to the next, `lbo` from one column block to the next (N-major only). */
__device__ __forceinline__ uint64_t mat_desc(uint32_t at, uint32_t lbo, uint32_t sbo, uint64_t swz) {
  return (uint64_t)((at & 0x3FFFF) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (swz << 61);
}
/* kind::f16 instruction: bf16 x bf16 -> fp32, M 128. */
__host__ __device__ constexpr uint32_t inst_desc(int n, bool b_n_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_n_major ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

/* ---- the cut ------------------------------------------------------------------ */

__host__ __device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

/* Tiles of block j (BT query tokens) of a sequence's own keys. */
__device__ __forceinline__ int own_tiles(int len, int T, int start, int BT, int j) {
  const int seen = min(len, len - T + min(T, (j + 1) * BT)); /* keys the block's last token sees */
  return seen > start ? div_up(seen - start, kTile) : 0;
}
/* The CTA that owns unit u of `total` cut over n CTAs: CTA c owns [c total / n, (c + 1) total / n). */
__device__ __forceinline__ int cta_of(int u, int total, int n) {
  return (int)((((long long)u + 1) * n - 1) / total);
}
/* Last i in [0, n) with a[i] <= x (a not decreasing, a[0] <= x). */
__device__ __forceinline__ int find(const int32_t *a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if (a[m] <= x)
      lo = m;
    else
      hi = m - 1;
  }
  return lo;
}

__device__ int cta_scan(int v, Smem *sm, int *total) { /* exclusive */
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm->sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sm->sums[w];
    all += sm->sums[w];
  }
  *total = all;
  __syncthreads();
  return before + x - v;
}

/* Loads and checks the batch and cuts it.  False (for the whole CTA, and every
 * CTA alike) if it is not sound. */
__device__ bool take_cut(const Args &a, Smem *sm) {
  const int tid = threadIdx.x;
  const int BT = 2 * (kTile / a.G);
  const long long cap = (long long)a.max_pages * a.P;
  bool bad = false;
  for (int i = tid; i <= a.n_seqs; i += kThreads) sm->off[i] = a.off ? a.off[i] : i;
  for (int i = tid; i < a.n_seqs; i += kThreads) {
    const int l = a.lens[i];
    bad |= l < 0 || l > cap;
    sm->len[i] = l;
  }
  for (int i = tid; i <= a.n_groups; i += kThreads) {
    sm->gs[i] = a.n_groups ? a.starts[i] : 0;
    if (i < a.n_groups) {
      const int l = a.prefix[i];
      bad |= l < 0;
      sm->plen[i] = l;
      sm->lead[i] = a.n_seqs;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.n_seqs; i += kThreads) bad |= sm->off[i + 1] < sm->off[i];
  if (tid == 0) bad |= sm->off[0] != 0 || sm->off[a.n_seqs] > a.n_tokens;
  for (int i = tid; i < a.n_groups; i += kThreads) bad |= sm->gs[i + 1] < sm->gs[i];
  if (tid == 0 && a.n_groups) bad |= sm->gs[0] != 0 || sm->gs[a.n_groups] != a.n_seqs;
  if (__syncthreads_or(bad)) return false;
  /* shared keys: whole pages that every sequence with something to read has; a
   * group of one reads them with its own */
  if (a.n_groups) {
    for (int i = tid; i < a.n_seqs; i += kThreads)
      if (sm->len[i] > 0 && sm->off[i + 1] > sm->off[i]) {
        const int g = find(sm->gs, a.n_groups + 1, i);
        atomicMin(&sm->plen[g], sm->len[i]);
        atomicMin(&sm->lead[g], i);
      }
    __syncthreads();
    for (int i = tid; i < a.n_groups; i += kThreads)
      sm->plen[i] = sm->gs[i + 1] - sm->lead[i] < 2 ? 0 : sm->plen[i] / a.P * a.P;
  }
  __syncthreads();
  int base = 0;
  for (int i0 = 0; i0 < a.n_groups; i0 += kThreads) {
    const int i = i0 + tid;
    int units = 0;
    if (i < a.n_groups) {
      const int tokens = sm->off[sm->gs[i + 1]] - sm->off[sm->gs[i]];
      units = a.Hkv * div_up(tokens, BT) * div_up(sm->plen[i], kTile);
    }
    int total;
    const int at = cta_scan(units, sm, &total);
    if (i < a.n_groups) sm->cum_g[i] = base + at;
    base += total;
  }
  const int total_g = base;
  for (int i0 = 0; i0 < a.n_seqs; i0 += kThreads) {
    const int i = i0 + tid;
    int units = 0;
    if (i < a.n_seqs) {
      const int T = sm->off[i + 1] - sm->off[i];
      const int start = a.n_groups ? sm->plen[find(sm->gs, a.n_groups + 1, i)] : 0;
      sm->start[i] = start;
      for (int j = 0; j * BT < T; ++j) units += own_tiles(sm->len[i], T, start, BT, j);
      units *= a.Hkv;
    }
    int total;
    const int at = cta_scan(units, sm, &total);
    if (i < a.n_seqs) sm->cum_s[i] = base + at;
    base += total;
  }
  if (tid == 0) {
    sm->cum_g[a.n_groups] = total_g;
    sm->cum_s[a.n_seqs] = base;
    sm->total_g = total_g;
    sm->total = base;
  }
  __syncthreads();
  return true;
}

/* One CTA's part of an item. */
struct Piece {
  int own;             /* 1: a sequence's own keys, 0: a group's shared ones */
  int seq;             /* whose table row names the pages */
  int kvh, tok0, ntok; /* query tokens of the item */
  int key0, kend;      /* the item's keys */
  int t0, t1, nt;      /* tiles of this piece, of the item */
};

__device__ Piece piece_at(const Args &a, const Smem *sm, int u, int u1) {
  const int BT = 2 * (kTile / a.G);
  Piece p;
  int j, r;
  if (u < sm->total_g) {
    const int g = find(sm->cum_g, a.n_groups, u);
    p.own = 0;
    p.seq = sm->lead[g];
    const int end = sm->off[sm->gs[g + 1]], first = sm->off[sm->gs[g]], n = div_up(end - first, BT);
    p.nt = div_up(sm->plen[g], kTile);
    r = u - sm->cum_g[g];
    const int item = r / p.nt;
    r -= item * p.nt;
    p.kvh = item / n;
    j = item - p.kvh * n;
    p.tok0 = first + j * BT;
    p.ntok = min(BT, end - p.tok0);
    p.key0 = 0;
    p.kend = sm->plen[g];
  } else {
    const int b = find(sm->cum_s, a.n_seqs, u);
    p.own = 1;
    p.seq = b;
    const int T = sm->off[b + 1] - sm->off[b], len = sm->len[b], start = sm->start[b];
    const int per = (sm->cum_s[b + 1] - sm->cum_s[b]) / a.Hkv;
    r = u - sm->cum_s[b];
    p.kvh = r / per;
    r -= p.kvh * per;
    for (j = 0;; ++j) {
      p.nt = own_tiles(len, T, start, BT, j);
      if (r < p.nt) break;
      r -= p.nt;
    }
    p.tok0 = sm->off[b] + j * BT;
    p.ntok = min(BT, T - j * BT);
    p.key0 = start;
    p.kend = min(len, len - T + min(T, (j + 1) * BT));
  }
  p.t0 = r;
  p.t1 = min(p.nt, r + (u1 - u));
  return p;
}

/* ---- the tiles ---------------------------------------------------------------- */

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ Args a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint8_t *qs = base, *ks = qs + 2 * C::TILE, *vs = ks + C::STAGES * C::TILE;
  Smem *sm = (Smem *)(vs + C::STAGES * C::TILE);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      bar_init(&sm->kfull[i], 1);
      bar_init(&sm->kempty[i], 1);
      bar_init(&sm->vfull[i], 1);
      bar_init(&sm->vempty[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(&sm->sfull[s], 1);
      bar_init(&sm->pready[s], 4);
      bar_init(&sm->qready[s], 4);
      bar_init(&sm->oready[s], 1);
    }
    bar_init(&sm->xfull, 4);
    bar_init(&sm->xfree, 4);
    bar_init(&sm->drain, 1);
    sm->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool sound = take_cut(a, sm);
  if (blockIdx.x == 0) {
    if (tid == 0) {
      a.sched[0] = !sound;
      a.sched[1] = sound ? sm->total_g : 0;
      a.sched[2] = sound ? sm->total : 0;
      if (!sound) *(volatile int32_t *)a.err_host = MK_ERR_INVALID_ARG;
    }
    if (sound) {
      int32_t *w = a.sched + 4;
      for (int i = tid; i <= a.n_groups; i += kThreads) {
        w[i] = sm->cum_g[i];
        if (i < a.n_groups) w[2 * (kMaxSeqs + 1) + i] = sm->plen[i];
      }
      for (int i = tid; i <= a.n_seqs; i += kThreads) w[kMaxSeqs + 1 + i] = sm->cum_s[i];
    }
  }
  if (!sound) return;
  const int total = sm->total, n_cta = gridDim.x;
  const int u_begin = (int)((long long)blockIdx.x * total / n_cta);
  const int u_end = (int)(((long long)blockIdx.x + 1) * total / n_cta);
  if (u_begin == u_end) return;

  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(&sm->tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  volatile int *abort = &sm->abort;
  const int TB = kTile / a.G; /* query tokens of a row tile */

  if (warp == 8) {
    /* ---- producer: K one tile ahead of V, the order in which the products need them */
    const int boxes = kTile / a.box_rows;
    const int box = lane % boxes, half = lane / boxes;
    const uint32_t box_bytes = a.box_rows * C::ROWB;
    int ik = 0, iv = 0;
    bool ok = true;
    for (int u = u_begin; ok && u < u_end;) {
      const Piece p = piece_at(a, sm, u, u_end);
      const int n = p.t1 - p.t0;
      u += n;
      const int32_t *row = a.tables + (size_t)p.seq * a.max_pages;
      for (int i = 0; ok && i <= n; ++i) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int t = kv == 0 ? i : i - 1;
          if (t < 0 || t >= n) continue;
          int &it = kv == 0 ? ik : iv;
          const int slot = it % C::STAGES;
          uint64_t *full = kv == 0 ? &sm->kfull[slot] : &sm->vfull[slot];
          uint64_t *empty = kv == 0 ? &sm->kempty[slot] : &sm->vempty[slot];
          const int key = p.key0 + (p.t0 + t) * kTile + box * a.box_rows;
          int page = -1;
          if (half < C::NH && key < p.kend) {
            page = __ldg(row + key / a.P);
            if ((unsigned)page >= (unsigned)a.num_pages) {
              page = -1;
              *(volatile int32_t *)a.err_host = MK_ERR_PAGE_OOB;
            }
          }
          ok = warp_wait(empty, ((it / C::STAGES) & 1) ^ 1, abort);
          if (!ok) break;
          const int loads = __popc(__ballot_sync(0xffffffffu, page >= 0));
          if (lane == 0) bar_expect(full, loads * box_bytes);
          __syncwarp();
          if (page >= 0)
            tma_2d(saddr((kv == 0 ? ks : vs) + slot * C::TILE + half * C::BLOCK +
                         box * box_bytes),
                   kv == 0 ? &kmap : &vmap, half * C::COLS,
                   (page * a.Hkv + p.kvh) * a.P + key % a.P, full);
          ++it;
        }
      }
    }
    if (!ok) { /* gave up: let the copies in flight land */
      for (int i = 0; i < C::STAGES; ++i) {
        volatile int none = 0;
        const int jk = ik - 1 - i, jv = iv - 1 - i;
        if (jk >= 0) warp_wait(&sm->kfull[jk % C::STAGES], (jk / C::STAGES) & 1, &none);
        if (jv >= 0) warp_wait(&sm->vfull[jv % C::STAGES], (jv / C::STAGES) & 1, &none);
      }
    }
  } else if (warp == 9) {
    /* ---- issuer: op j is tile j or j / 2 of the piece on stream j % 2 */
    if (lane == 0) {
      constexpr uint32_t id_qk = inst_desc(kTile, false), id_pv = inst_desc(D, true);
      int ik = 0, iv = 0, nq[2] = {0, 0}, np[2] = {0, 0};
      bool ok = true;
      for (int u = u_begin; ok && u < u_end;) {
        const Piece p = piece_at(a, sm, u, u_end);
        const int n = p.t1 - p.t0;
        u += n;
        const bool pair = p.ntok > TB;
        const int ops = pair ? 2 * n : n;
        for (int s = 0; ok && s < 2; ++s)
          if (s < ops) ok = bar_wait(&sm->qready[s], nq[s]++ & 1, abort);
        auto qk = [&](int j) {
          const int s = j & 1, it = ik + (pair ? j >> 1 : j), slot = it % C::STAGES;
          if (!bar_wait(&sm->kfull[slot], (it / C::STAGES) & 1, abort)) return false;
          tc_fence_after();
          const uint32_t q0 = saddr(qs + s * C::TILE), k0 = saddr(ks + slot * C::TILE);
#pragma unroll
          for (int h = 0; h < C::NH; ++h)
#pragma unroll
            for (int c = 0; c < C::COLS / 16; ++c)
              mma_ss(tmem + s * kTile,
                     mat_desc(q0 + h * C::BLOCK + c * 32, 16, 8 * C::ROWB, C::SWIZZLE),
                     mat_desc(k0 + h * C::BLOCK + c * 32, 16, 8 * C::ROWB, C::SWIZZLE), id_qk,
                     h + c > 0);
          tc_commit(&sm->sfull[s]);
          if (!pair || s == 1) tc_commit(&sm->kempty[slot]);
          return true;
        };
        for (int j = 0; ok && j < 2 && j < ops; ++j) ok = qk(j);
        for (int j = 0; ok && j < ops; ++j) {
          const int s = j & 1, t = pair ? j >> 1 : j, it = iv + t, slot = it % C::STAGES;
          ok = bar_wait(&sm->vfull[slot], (it / C::STAGES) & 1, abort) &&
               bar_wait(&sm->pready[s], np[s]++ & 1, abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v0 = saddr(vs + slot * C::TILE);
#pragma unroll
          for (int c = 0; c < kTile / 16; ++c)
            mma_ts(tmem + 2 * kTile + s * kTile, tmem + s * kTile + c * 8,
                   mat_desc(v0 + c * 16 * C::ROWB, C::BLOCK, 8 * C::ROWB, C::SWIZZLE), id_pv,
                   j > 1 || c > 0);
          if (!pair || s == 1) tc_commit(&sm->vempty[slot]);
          if (j + 2 < ops) ok = qk(j + 2);
        }
        for (int s = 0; ok && s < 2; ++s)
          if (s < ops) tc_commit(&sm->oready[s]);
        ik += n;
        iv += n;
      }
      if (!ok) { /* gave up: let the products in flight end */
        volatile int none = 0;
        tc_commit(&sm->drain);
        bar_wait(&sm->drain, 0, &none);
      }
    }
  } else {
    /* ---- softmax: stream s, one row a thread */
    const int s = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21; /* this warp's TMEM lanes */
    const uint32_t at_s = tmem + lanes + s * kTile, at_o = at_s + 2 * kTile;
    const float c2 = a.scale_log2;
    int ns = 0, no = 0, iv = 0, nx = 0;
    bool ok = true;
    for (int u = u_begin; ok && u < u_end;) {
      const Piece p = piece_at(a, sm, u, u_end);
      const int n = p.t1 - p.t0;
      u += n;
      const bool pair = p.ntok > TB;
      const int ops = pair ? 2 * n : n;
      if (s < ops) {
        const int tok0 = p.tok0 + (pair ? s * TB : 0);
        const int ntok = min(TB, p.tok0 + p.ntok - tok0);
        const int rows = ntok * a.G;
        /* Q rows into swizzled shared memory, zeros behind the last */
        uint8_t *qd = qs + s * C::TILE;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const int k = i * kTile + r, qr = k / (D / 8), ch = k % (D / 8);
          const int hb = ch / (C::COLS / 8), cc = ch % (C::COLS / 8);
          uint4 x = make_uint4(0, 0, 0, 0);
          if (qr < rows) {
            const int t = qr / a.G;
            x = __ldg((const uint4 *)(a.q + (tok0 + t) * a.q_stride +
                                      (long long)(p.kvh * a.G + qr - t * a.G) * D + ch * 8));
          }
          const int sw = D < 64 ? cc ^ ((qr >> 1) & 3) : cc ^ (qr & 7);
          *(uint4 *)(qd + hb * C::BLOCK + qr * C::ROWB + sw * 16) = x;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&sm->qready[s]);

        const bool valid = r < rows, busy = (warp & 3) * 32 < rows;
        const int tok = tok0 + (valid ? r / a.G : 0);
        const int head = p.kvh * a.G + (valid ? r % a.G : 0);
        const int b = p.own ? p.seq : find(sm->off, a.n_seqs + 1, tok);
        /* keys of the item that this row sees end here */
        const int limit = min(p.kend, sm->len[b] - (sm->off[b + 1] - tok) + 1);
        float m = -INFINITY, l = 0.0f; /* m in score units */
        for (int j = s; j < ops; j += 2) {
          const int t = pair ? j >> 1 : j;
          const int k0 = p.key0 + (p.t0 + t) * kTile;
          ok = warp_wait(&sm->sfull[s], ns++ & 1, abort);
          if (!ok) break;
          tc_fence_after();
          if (busy) {
            float x[kTile];
            tmem_ld128(at_s, x);
            if (!__all_sync(0xffffffffu, limit >= k0 + kTile)) {
#pragma unroll
              for (int i = 0; i < kTile; ++i) x[i] = k0 + i < limit ? x[i] : -INFINITY;
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < kTile; ++i) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (j < 2) {
              m = top;
            } else {
              const bool move = m == -INFINITY ? top > m : (top - m) * c2 > kSlack;
              if (__any_sync(0xffffffffu, move)) {
                /* the products into O so far are complete: they were issued before this S */
                const float to = move ? top : m;
                const float f = move ? exp2_approx((m - to) * c2) : 1.0f; /* m -inf: 0 */
#pragma unroll
                for (int i = 0; i < D; i += 32) {
                  float o[32];
                  tmem_ld32(at_o + i, o);
                  uint32_t w[32];
#pragma unroll
                  for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(o[k] * f);
                  tmem_st32(at_o + i, w);
                }
                l *= f;
                m = to;
              }
            }
            const float off = m == -INFINITY ? 0.0f : -m * c2;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[32];
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float e0 = exp2_approx(fmaf(x[h * 64 + 2 * k], c2, off));
                const float e1 = exp2_approx(fmaf(x[h * 64 + 2 * k + 1], c2, off));
                sum[k & 1] += e0;
                sum[2 + (k & 1)] += e1;
                w[k] = pack_bf16(e0, e1);
              }
              tmem_st32(at_s + h * 32, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_wait_st();
          }
          if (k0 + kTile > p.kend) {
            /* zero the V rows behind the last key: what lies there may be NaN */
            const int it = iv + t, slot = it % C::STAGES;
            ok = warp_wait(&sm->vfull[slot], (it / C::STAGES) & 1, abort);
            if (!ok) break;
            if (k0 + r >= p.kend) {
              uint8_t *vr = vs + slot * C::TILE + r * C::ROWB;
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                *(uint4 *)(vr + i / (C::COLS / 8) * C::BLOCK + i % (C::COLS / 8) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sm->pready[s]);
        }
        if (!ok) break;
        ok = warp_wait(&sm->oready[s], no++ & 1, abort);
        if (!ok) break;
        tc_fence_after();
        /* even and odd tiles of the same rows: the second stream hands over its part */
        const bool joins = !pair && n > 1;
        float *xo = (float *)qs; /* [D][128]: Q is read by now */
        if (joins && s == 1) {
          if (busy) {
#pragma unroll
            for (int i = 0; i < D; i += 32) {
              float o[32];
              tmem_ld32(at_o + i, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) xo[(i + k) * kTile + r] = o[k];
            }
            sm->xm[r] = m;
            sm->xl[r] = l;
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&sm->xfull);
          ok = warp_wait(&sm->xfree, nx++ & 1, abort); /* Q may be written again */
          if (!ok) break;
        } else {
          float f0 = 1.0f, f1 = 0.0f;
          if (joins) {
            ok = warp_wait(&sm->xfull, nx++ & 1, abort);
            if (!ok) break;
            const float m1 = sm->xm[r], mm = fmaxf(m, m1);
            if (mm != -INFINITY) {
              f0 = exp2_approx((m - mm) * c2);
              f1 = exp2_approx((m1 - mm) * c2);
            }
            l = l * f0 + sm->xl[r] * f1;
            m = mm;
          }
          const bool whole = p.own && p.key0 == 0 && n == p.nt; /* nothing to merge */
          const long long orow = (long long)tok * a.Hq + head;
          const long long prow =
              p.t0 == 0 ? (long long)p.own * a.n_tokens * a.Hq + orow
                        : 2ll * a.n_tokens * a.Hq + (long long)blockIdx.x * 2 * kTile +
                              (pair ? s * kTile : 0) + r;
          const float inv = l > 0.0f ? 1.0f / l : 0.0f;
          if (busy) {
#pragma unroll
            for (int i = 0; i < D; i += 32) {
              float o[32];
              tmem_ld32(at_o + i, o);
              if (joins) {
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = o[k] * f0 + xo[(i + k) * kTile + r] * f1;
              }
              if (valid && whole) {
                uint4 *d = (uint4 *)(a.out + orow * D + i);
#pragma unroll
                for (int k = 0; k < 32; k += 8)
                  d[k / 8] = make_uint4(pack_bf16(o[k] * inv, o[k + 1] * inv),
                                        pack_bf16(o[k + 2] * inv, o[k + 3] * inv),
                                        pack_bf16(o[k + 4] * inv, o[k + 5] * inv),
                                        pack_bf16(o[k + 6] * inv, o[k + 7] * inv));
              } else if (valid) {
                float4 *d = (float4 *)(a.part + prow * D + i);
#pragma unroll
                for (int k = 0; k < 32; k += 4)
                  d[k / 4] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
              }
            }
            if (valid && whole) {
              if (a.lse)
                a.lse[orow] = l > 0.0f ? (m * c2 + log2f(l)) * 0.69314718055994531f : -INFINITY;
            } else if (valid) {
              a.part_ml[prow] = make_float2(m == -INFINITY ? m : m * c2, l);
            }
          }
          if (joins) {
            /* no warp of either stream writes Q again before all have read */
            __syncwarp();
            if (lane == 0) bar_arrive(&sm->xfree);
            ok = warp_wait(&sm->xfree, (nx - 1) & 1, abort);
            if (!ok) break;
          }
        }
        tc_fence_before();
      }
      iv += n;
    }
  }
  __syncthreads();
  if (tid == 0 && *abort) *(volatile int32_t *)a.err_host = MK_ERR_DEVICE_TIMEOUT;
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

/* ---- the join ----------------------------------------------------------------- */

/* One warp per output row: M = max m_i, out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
 * Reads L2: the partials were written just before. */
template <int D>
__global__ void __launch_bounds__(256) attn_merge(const __grid_constant__ Args a, int n_cta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long orow = ((long long)blockIdx.x * 256 + threadIdx.x) >> 5;
  if (a.sched[0]) return;
  const int tok = (int)(orow / a.Hq), head = (int)(orow - (long long)tok * a.Hq);
  const int tokens = a.off ? a.off[a.n_seqs] : a.n_seqs;
  if (tok >= tokens) return;
  const int TB = kTile / a.G, BT = 2 * TB, total = a.sched[2];
  const int kvh = head / a.G, hg = head - kvh * a.G;
  const int32_t *cum_g = a.sched + 4, *cum_s = cum_g + kMaxSeqs + 1, *plens = cum_s + kMaxSeqs + 1;
  const int b = a.off ? find(a.off, a.n_seqs + 1, tok) : tok;
  const int first = a.off ? a.off[b] : b, T = a.off ? a.off[b + 1] - first : 1, len = a.lens[b];
  int plen = 0, n_shared = 0, n_own = 0;          /* pieces */
  int cs = 0, co = 0;                             /* their first CTAs */
  int rs = 0, ro = 0;                             /* the row's place in a CTA's own slots */
  if (a.n_groups) {
    const int g = find(a.starts, a.n_groups + 1, b);
    plen = plens[g];
    if (plen) {
      const int gtok = a.off ? a.off[a.starts[g]] : a.starts[g];
      const int gend = a.off ? a.off[a.starts[g + 1]] : a.starts[g + 1];
      const int nt = div_up(plen, kTile), nb = div_up(gend - gtok, BT), j = (tok - gtok) / BT;
      const int u = cum_g[g] + (kvh * nb + j) * nt, ti = tok - gtok - j * BT;
      cs = cta_of(u, total, n_cta);
      n_shared = cta_of(u + nt - 1, total, n_cta) - cs + 1;
      rs = ti / TB * kTile + ti % TB * a.G + hg;
    }
  }
  const int jb = (tok - first) / BT, nt_own = own_tiles(len, T, plen, BT, jb);
  if (nt_own) {
    int u = cum_s[b] + (cum_s[b + 1] - cum_s[b]) / a.Hkv * kvh;
    for (int j = 0; j < jb; ++j) u += own_tiles(len, T, plen, BT, j);
    const int ti = tok - first - jb * BT;
    co = cta_of(u, total, n_cta);
    n_own = cta_of(u + nt_own - 1, total, n_cta) - co + 1;
    ro = ti / TB * kTile + ti % TB * a.G + hg;
  }
  if (n_shared == 0 && n_own == 1) return; /* written by attn_tiles */
  const int n = n_shared + n_own;
  const long long dense = (long long)a.n_tokens * a.Hq;
  auto place = [&](int i) -> long long { /* partial row of piece i */
    const bool own = i >= n_shared;
    const int k = own ? i - n_shared : i;
    if (k == 0) return own ? dense + orow : orow;
    return 2 * dense + (long long)((own ? co : cs) + k) * 2 * kTile + (own ? ro : rs);
  };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, a.part_ml[place(i)].x);
#pragma unroll
  for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
  constexpr int N = D / 32; /* columns a lane */
  float o[N] = {}, l = 0.0f;
  if (M != -INFINITY) {
    for (int i0 = 0; i0 < n; i0 += 32) {
      float f = 0.0f;
      if (i0 + lane < n) {
        const float2 ml = a.part_ml[place(i0 + lane)];
        f = exp2_approx(ml.x - M);
        l += f * ml.y;
      }
      const int m = min(32, n - i0);
#pragma unroll 4
      for (int i = 0; i < m; ++i) {
        const float w = __shfl_sync(0xffffffffu, f, i);
        const float *src = a.part + place(i0 + i) * D + lane * N;
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = fmaf(w, src[k], o[k]);
      }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k) a.out[orow * D + lane * N + k] = __float2bfloat16_rn(o[k] * inv);
  if (a.lse && lane == 0)
    a.lse[orow] = l > 0.0f ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

/* Makes `dev` current for a scope. */
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

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace

struct mk_attn {
  mk_attn_desc d{};
  std::vector<CUtensorMap> maps; /* K and V of each layer */
  float scale_log2 = 0.0f;
  int box_rows = 0;
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0;
  uint8_t *ws = nullptr;
  size_t o_part = 0, o_ml = 0;
  int32_t *err_host = nullptr, *err_dev = nullptr;
};

namespace {

template <int D>
cudaError_t prepare() {
  return cudaFuncSetAttribute(attn_tiles<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<D>::SMEM + (int)sizeof(Smem));
}

template <int D>
cudaError_t launch(const mk_attn *at, int layer, const Args &a) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(at->n_sm);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM + sizeof(Smem);
  cfg.stream = at->stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  cudaError_t e =
      cudaLaunchKernelEx(&cfg, attn_tiles<D>, at->maps[2 * layer], at->maps[2 * layer + 1], a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(((long long)a.n_tokens * a.Hq + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, attn_merge<D>, a, at->n_sm);
}

}  // namespace

extern "C" {

mk_status mk_attn_create(const mk_attn_desc *d, void *stream, mk_attn **out) {
  if (!d || !out) return MK_ERR_INVALID_ARG;
  if (d->n_q_heads < 1 || d->n_kv_heads < 1 || d->head_dim < 1 || d->page_size < 1 ||
      d->num_pages < 1 || d->max_tokens < 1 || d->max_seqs < 1 ||
      d->max_groups < 0 || d->n_layers < 1 || d->n_q_heads % d->n_kv_heads ||
      !(d->scale >= 0.0f) || !std::isfinite(d->scale))
    return MK_ERR_INVALID_ARG;
  if ((d->head_dim != 32 && d->head_dim != 64 && d->head_dim != 128) || d->page_size % 16 ||
      d->page_size > 256 || d->n_q_heads / d->n_kv_heads > 64 || d->n_q_heads > 1024 ||
      d->max_tokens > (1 << 20) || d->max_seqs > kMaxSeqs || d->max_groups > kMaxSeqs ||
      (int64_t)d->num_pages * d->n_kv_heads * d->page_size > INT32_MAX)
    return MK_ERR_UNSUPPORTED;
  if (!d->k_caches || !d->v_caches) return MK_ERR_INVALID_ARG;
  for (int l = 0; l < d->n_layers; ++l)
    if (!d->k_caches[l] || !d->v_caches[l] || !aligned(d->k_caches[l], 16) ||
        !aligned(d->v_caches[l], 16))
      return MK_ERR_INVALID_ARG;
  int dev = 0;
  cudaDeviceProp prop;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaGetDeviceProperties(&prop, dev) != cudaSuccess)
    return MK_ERR_NO_DEVICE;
  if (prop.major != 10 || prop.minor != 3) return MK_ERR_NO_DEVICE;
  mk_attn *at = new (std::nothrow) mk_attn();
  if (!at) return MK_ERR_CUDA;
  at->d = *d;
  at->d.k_caches = at->d.v_caches = nullptr;
  const double scale = d->scale > 0.0f ? (double)d->scale : 1.0 / std::sqrt((double)d->head_dim);
  at->scale_log2 = (float)(scale * 1.4426950408889634);
  at->stream = (cudaStream_t)stream;
  at->dev = dev;
  at->n_sm = prop.multiProcessorCount;
  /* a box lies within a page: as many of a tile's rows as divide the page */
  at->box_rows = d->page_size & -d->page_size;
  if (at->box_rows > kTile) at->box_rows = kTile;
  mk_status st = MK_OK;
  try {
    at->maps.resize(2 * (size_t)d->n_layers);
    for (int l = 0; l < d->n_layers && st == MK_OK; ++l) {
      st = mk_encode_rows_map(d, d->k_caches[l], at->box_rows, &at->maps[2 * l]);
      if (st == MK_OK) st = mk_encode_rows_map(d, d->v_caches[l], at->box_rows, &at->maps[2 * l + 1]);
    }
  } catch (...) {
    st = MK_ERR_CUDA;
  }
  if (st != MK_OK) {
    delete at;
    return st;
  }
  const size_t rows = 2 * (size_t)d->max_tokens * d->n_q_heads + (size_t)at->n_sm * 2 * kTile;
  at->o_part = ((4 + 3 * (size_t)(kMaxSeqs + 1)) * 4 + 255) / 256 * 256;
  at->o_ml = at->o_part + rows * d->head_dim * 4;
  cudaError_t e = d->head_dim == 32 ? prepare<32>() : d->head_dim == 64 ? prepare<64>() : prepare<128>();
  if (e == cudaSuccess) e = cudaMalloc(&at->ws, at->o_ml + rows * sizeof(float2));
  if (e == cudaSuccess) e = cudaHostAlloc(&at->err_host, 64, cudaHostAllocMapped);
  if (e == cudaSuccess) {
    std::memset(at->err_host, 0, 64);
    e = cudaHostGetDevicePointer((void **)&at->err_dev, at->err_host, 0);
  }
  if (e != cudaSuccess) {
    mk_attn_destroy(at);
    return MK_ERR_CUDA;
  }
  *out = at;
  return MK_OK;
}

void mk_attn_destroy(mk_attn *at) {
  if (!at) return;
  {
    OnDevice on(at->dev);
    cudaStreamSynchronize(at->stream);
    if (at->ws) cudaFree(at->ws);
    if (at->err_host) cudaFreeHost(at->err_host);
  }
  delete at;
}

mk_status mk_prefix_attention(mk_attn *at, int32_t layer, const mk_attn_batch *b, const void *q,
                              int64_t q_token_stride, void *out, float *lse) {
  if (!at || !b) return MK_ERR_INVALID_ARG;
  const mk_attn_desc &d = at->d;
  if (layer < 0 || layer >= d.n_layers || b->n_seqs < 0 || b->n_tokens < 0 || b->n_groups < 0 ||
      b->max_pages_per_seq < 1)
    return MK_ERR_INVALID_ARG;
  if (b->n_seqs > d.max_seqs || b->n_tokens > d.max_tokens || b->n_groups > d.max_groups)
    return MK_ERR_BATCH;
  if ((int64_t)b->max_pages_per_seq * d.page_size > (1 << 30)) return MK_ERR_UNSUPPORTED;
  if (b->n_seqs == 0 || b->n_tokens == 0) return MK_OK;
  if (!b->page_tables || !b->seq_lens || !aligned(b->page_tables, 4) || !aligned(b->seq_lens, 4) ||
      !aligned(b->q_offsets, 4) || !aligned(b->group_starts, 4) || !aligned(b->prefix_lens, 4) ||
      (!b->q_offsets && b->n_tokens != b->n_seqs) ||
      (b->n_groups > 0 && (!b->group_starts || !b->prefix_lens)))
    return MK_ERR_INVALID_ARG;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      q_token_stride < (int64_t)d.n_q_heads * d.head_dim || q_token_stride % 8)
    return MK_ERR_INVALID_ARG;
  OnDevice on(at->dev);
  if (!on.ok) return MK_ERR_CUDA;
  Args a{};
  a.Hq = d.n_q_heads;
  a.Hkv = d.n_kv_heads;
  a.G = d.n_q_heads / d.n_kv_heads;
  a.P = d.page_size;
  a.num_pages = d.num_pages;
  a.max_pages = b->max_pages_per_seq;
  a.n_seqs = b->n_seqs;
  a.n_tokens = b->n_tokens;
  a.n_groups = b->n_groups;
  a.box_rows = at->box_rows;
  a.tables = b->page_tables;
  a.lens = b->seq_lens;
  a.off = b->q_offsets;
  a.starts = b->group_starts;
  a.prefix = b->prefix_lens;
  a.q = (const __nv_bfloat16 *)q;
  a.q_stride = q_token_stride;
  a.out = (__nv_bfloat16 *)out;
  a.lse = lse;
  a.scale_log2 = at->scale_log2;
  a.err_host = at->err_dev;
  a.sched = (int32_t *)at->ws;
  a.part = (float *)(at->ws + at->o_part);
  a.part_ml = (float2 *)(at->ws + at->o_ml);
  const cudaError_t e = d.head_dim == 32   ? launch<32>(at, layer, a)
                        : d.head_dim == 64 ? launch<64>(at, layer, a)
                                           : launch<128>(at, layer, a);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_attn_sync(mk_attn *at) {
  if (!at) return MK_ERR_INVALID_ARG;
  OnDevice on(at->dev);
  if (!on.ok) return MK_ERR_CUDA;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(at->stream, &cap) != cudaSuccess) return MK_ERR_CUDA;
  if (cap != cudaStreamCaptureStatusNone) return MK_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(at->stream) != cudaSuccess) return MK_ERR_CUDA;
  const int32_t code = *(volatile int32_t *)at->err_host;
  *(volatile int32_t *)at->err_host = 0;
  return code;
}

}  // extern "C"
