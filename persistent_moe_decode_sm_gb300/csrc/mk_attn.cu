/*
 * mk_attn.cu -- attention of a batch over paged K and V whose leading pages
 * sequences share (include/mk_cache.h).
 *
 * The work is cut into tiles of 128 keys.  An item is a range of keys that a
 * set of query rows reads: a group's shared pages with the rows (query tokens x
 * heads of one kv head) of the group's sequences, or one sequence's own pages
 * with that sequence's rows.  Items of more than 128 rows (up to 256: pairs), then
 * items of at most 128 rows (singles) lie end to end on a line, each as long as
 * its tiles and a fixed cost, and the line is cut evenly over the SMs.  An SM's
 * share may begin and end inside an item; every piece leaves a partial (maximum,
 * sum, weighted sum) per row, and attn_merge joins them.  The cut follows from
 * the lengths on the device: each CTA takes it itself, so that a captured call
 * follows its batch.
 *
 * attn_tiles, one CTA per SM: producer warps move K and V tiles with TMA, one box
 * per page and 64 dims, into swizzled shared memory; issuing warps start S = Q K^T
 * and O += P V on the tensor cores (tcgen05, 128 rows, accumulators in TMEM); two
 * warpgroups, the streams, turn S into P, one row a thread, P going back to TMEM
 * as the A operand.  A pair's two row tiles run on the two streams over the same
 * K and V; of the CTA's singles each stream has its own half.  Either way one
 * stream's softmax runs under the other's products.
 */
#include <cuda.h> /* tensor-map types; the encoder is reached through the runtime */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "mk_attn_cut.h"
#include "mk_cache.h"
#include "mk_plan.h"

namespace {

using namespace mk_cut;

constexpr int kThreads = 384;      /* two softmax warpgroups, two producers, two issuers */
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88; /* 256 * 208 + 128 * 88 = 384 * 168 */
constexpr int kQueue = 4;          /* pieces that a producer is ahead of its stream */
constexpr int kMaxSeqs = 1024, kMaxGroups = 512; /* of a call: the cut's tables are in shared memory */
constexpr unsigned long long kWaitLimit = 2000000000ull; /* ns: of a call unless set, and of the last waits */
/* The reference that a row's P are taken against moves only when a score exceeds it by
 * this much (in powers of two): P then stays below 2^8, its relative precision in bf16
 * is the same, and the accumulator is rescaled a few times a row instead of in most tiles. */
constexpr float kSlack = 8.0f;
struct Args {
  int32_t Hq, Hkv, G, P, num_pages, max_pages, n_seqs, n_tokens, n_groups, box_rows;
  const int32_t *tables, *lens, *off, *starts, *prefix;
  __nv_bfloat16 *out;
  float *lse;
  float scale_log2; /* scale * log2(e) */
  const uint32_t *tree; /* [n_tokens][tree_words] bits of the sequence's tokens that a token sees, or NULL */
  int32_t tree_words, max_query; /* max_query: tokens of a sequence */
  const __nv_bfloat16 *q, *k_pool, *v_pool; /* for redo_rows: the tiles have tensor maps */
  int64_t q_stride;
  int32_t TB;       /* query tokens of a row tile: 128 / G */
  uint32_t inv_g;   /* ceil(2^16 / G): r * inv_g >> 16 is r / G for r < 128 */
  unsigned long long inv_p; /* ceil(2^38 / P): k * inv_p >> 38 is k / P for k < 2^30 */
  int32_t *err_host;
  unsigned long long wait_limit; /* ns */
  int32_t poison;    /* test hook: stream 0's issuer waits for what never comes */
  /* workspace */
  int32_t *bad;      /* the batch is not sound */
  int32_t *error;    /* the first since mk_attn_sync took one, 0: none */
  int4 *where;       /* [2][n_tokens][Hkv], zero between calls: where a token's partials are, of
                      * the shared keys and of its own.  x: pieces + 1, 1: written already, 0:
                      * none; y: the first piece's worker; z: the token's first row in worker 0's
                      * place; w: rows from a worker's place to the next */
  float *part;       /* [2 * n_tokens * Hq + 4 * SMs * 128][D] weighted sums */
  float2 *part_ml;   /* the same rows: maximum (in powers of two), sum; of a tree's rows that need
                      * no join too, there with the sum only where the result is not finite, else -1 */
};

__device__ __forceinline__ void report(const Args &a, int code) {
  if (atomicCAS(a.error, 0, code) == 0) *(volatile int32_t *)a.err_host = code;
}

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

/* One worker's part of an item. */
struct Piece {
  int line;            /* 0: a pair, 1: a single */
  int own;             /* 1: a sequence's own keys, 0: a group's shared ones */
  int seq;             /* whose table row names the pages */
  int kvh, tok0, ntok; /* query tokens of the item */
  int key0, kend;      /* the item's keys */
  int t0, n, nt;       /* first tile and tiles of this piece (0: no more), tiles of the item */
  int begin;           /* the item's first place */
};

/* A wait that runs out of time ends the CTA's work: every role looks here while it waits. */
struct Stop {
  int abort;
  unsigned long long limit; /* ns */
};

struct Smem { /* behind the tiles */
  uint64_t kfull[4], kempty[4], vfull[4], vempty[4];
  uint64_t sfull[2], pready[2][2], oready[2], drain[2];
  uint64_t turn[2];                           /* of a pair's softmaxes */
  uint64_t q_full[2], q_free[2];              /* Q of a stream's piece */
  uint64_t qfull[2][kQueue], qempty[2][kQueue]; /* the queue's */
  Piece queue[2][kQueue];
  uint32_t tmem;
  Stop stop;
  int fills[2][4], q_fills[2];                /* uses begun of each K and V slot, of each Q */
  unsigned long long sums[2][kThreads / 32];
  int total, pairs;   /* length of the line, of its pairs */
  int32_t off[kMaxSeqs + 1], len[kMaxSeqs];
  int32_t cum_s[2][kMaxSeqs + 1], cum_g[2][kMaxGroups + 1]; /* beginnings: pairs, singles */
  int32_t plen[kMaxGroups], lead[kMaxGroups]; /* a group's prefix, its first sequence that reads */
  uint16_t gs[kMaxGroups + 1];                /* a group's first sequence */
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
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(saddr(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
/* Waits for a phase; false when another role gave up or the limit ran out. */
__device__ __forceinline__ bool bar_wait(uint64_t *b, uint32_t parity, Stop *stop) {
  uint64_t since = 0;
  for (int i = 0;; ++i) {
    if (__all_sync(0xffffffffu, bar_try(b, parity))) return true;
    if (__any_sync(0xffffffffu, *(volatile int *)&stop->abort != 0)) return false;
    if ((i & 63) == 63) {
      const uint64_t t = now_ns();
      if (!since)
        since = t;
      else if (t - since > stop->limit)
        *(volatile int *)&stop->abort = 1;
    }
  }
}
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, Stop *stop) {
  return __all_sync(0xffffffffu, bar_try(b, parity)) || bar_wait(b, parity, stop);
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                       uint64_t *bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.u32 e, %5, 0;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(saddr(bar)), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                       uint64_t *bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.u32 e, %6, 0;\n"
      " @e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];\n}\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(saddr(bar)), "r"(lead)
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
/* The issuing warp runs its code as a whole, so that addresses and descriptors stay in
 * uniform registers; `lead` is 1 in the one lane whose instruction counts.  (One lane
 * alone in a branch issued a product in 100 cycles, more than the product takes.) */
__device__ __forceinline__ uint32_t elect_lead() {
  uint32_t p;
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(p));
  return p;
}
__device__ __forceinline__ void tc_commit(uint64_t *bar, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.u32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          saddr(bar)),
      "r"(lead)
      : "memory");
}
/* D (+)= A B with A and B in shared memory, or A in TMEM. */
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc, uint32_t lead) {
  asm volatile(
      "{\n .reg .pred p, e;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 e, %5, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
#define R8(x, i) x(i), x(i + 1), x(i + 2), x(i + 3), x(i + 4), x(i + 5), x(i + 6), x(i + 7)
#define R32(x, i) R8(x, i), R8(x, i + 8), R8(x, i + 16), R8(x, i + 24)
/* 16, 32, 64 or 128 columns of this thread's TMEM lane.  The load and its wait are one
 * statement: between two, the compiler could move registers that have not landed. */
#define OUT(i) "=f"(v[i])
__device__ __forceinline__ void tmem_ld16(uint32_t at, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R8(OUT, 0), R8(OUT, 8)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t at, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R32(OUT, 0)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t at, float *v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : R32(OUT, 0), R32(OUT, 32)
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
#define IN(i) "r"(v[i])
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15};" ::R8(IN, 0),
      R8(IN, 8), "r"(at)
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
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return __ffma2_rn(a, b, c);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
/* What the two bf16 of w leave of e (exact in fp32), rounded to bf16.  The products take the
 * bf16 halves as they are: with two unpacking instructions a pair instead, 4800 tokens of 32
 * heads over 32768 keys took 3.18 ms, so 2.89. */
__device__ __forceinline__ uint32_t rest_bf16(uint32_t w, float2 e) {
  float x, y;
  asm("{\n .reg .b16 l, h, m;\n mov.b32 {l, h}, %2;\n mov.b16 m, 0xBF80;\n"
      " fma.rn.f32.bf16 %0, l, m, %3;\n fma.rn.f32.bf16 %1, h, m, %4;\n}"
      : "=f"(x), "=f"(y) : "r"(w), "f"(e.x), "f"(e.y));
  return pack_bf16(x, y);
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

/* Last i in [0, n) with a[i] <= x (a not decreasing, a[0] <= x). */
template <class T>
__device__ __forceinline__ int find(const T *a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int m = (lo + hi + 1) >> 1;
    if ((int)a[m] <= x)
      lo = m;
    else
      hi = m - 1;
  }
  return lo;
}
/* The last i in [0, n) that `holds` (it holds for 0 and up to some i), by a whole warp: 32
 * places a round, so one or two rounds in most cases. */
template <class F>
__device__ __forceinline__ int warp_last(int n, F holds) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5, i = lane * step;
    const unsigned yes = __ballot_sync(0xffffffffu, i < n && holds(lo + i));
    const int k = 31 - __clz(yes | 1u);
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}
/* find by a whole warp. */
template <class T>
__device__ __forceinline__ int warp_find(const T *a, int n, int x) {
  return warp_last(n, [&](int i) { return (int)a[i] <= x; });
}

/* A group's shared keys: whole pages that every one of its sequences with something
 * to read has; a group of one reads them with its own. */
__device__ __forceinline__ int shared_keys(const Args &a, const Smem *sm, int g) {
  if ((int)sm->gs[g + 1] - sm->lead[g] < 2) return 0;
  return (int)(((unsigned long long)sm->plen[g] * a.inv_p) >> 38) * a.P;
}
__device__ __forceinline__ unsigned long long two(int pairs, int singles) {
  return (unsigned long long)(unsigned)pairs << 32 | (unsigned)singles;
}

/* Loads and checks the batch and cuts it.  False (for the whole CTA, and every
 * CTA alike) if it is not sound.  Most of its time goes to fetching its own
 * instructions and to its chain of loads, so it is short code with few barriers
 * rather than fast code: 384 entries a turn, one turn for most batches. */
__device__ bool take_cut(const Args &a, Smem *sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ns = a.n_seqs, ng = a.n_groups, TB = a.TB;
  const int turns = (max(ns, ng) + kThreads) / kThreads; /* ns + 1 offsets */
  bool bad = false;
#pragma unroll 1
  for (int k = 0; k < turns; ++k) {
    const int i = tid + k * kThreads;
    int l = 0, o = i, o1 = i + 1, g = 0, g1 = 0, p = 0;
    if (i < ns) l = a.lens[i];
    if (a.off && i <= ns) {
      o = a.off[i];
      if (i < ns) o1 = a.off[i + 1];
    }
    if (ng && i <= ng) {
      g = a.starts[i];
      if (i < ng) {
        g1 = a.starts[i + 1];
        p = a.prefix[i];
      }
    }
    if (i < ns) {
      bad |= l < 0 || l > (long long)a.max_pages * a.P || o1 < o || o1 - o > a.max_query;
      sm->len[i] = l;
    }
    if (i <= ns) {
      bad |= (i == 0 && o != 0) || (i == ns && o > a.n_tokens);
      sm->off[i] = o;
    }
    if (i <= ng) {
      bad |= (i == 0 && g != 0) || (i == ng && ng && g != ns) || (i < ng && (g1 < g || p < 0));
      sm->gs[i] = (uint16_t)g;
    }
    if (i < ng) {
      sm->plen[i] = p;
      sm->lead[i] = ns;
    }
  }
  if (__syncthreads_or(bad)) return false;
  if (ng) {
#pragma unroll 1
    for (int i = tid; i < ns; i += kThreads)
      if (sm->len[i] > 0 && sm->off[i + 1] > sm->off[i]) {
        const int g = find(sm->gs, ng + 1, i);
        atomicMin(&sm->plen[g], sm->len[i]);
        atomicMin(&sm->lead[g], i);
      }
    __syncthreads();
  }
  /* lengths of the groups' and of the sequences' items, pairs and singles, summed up */
  unsigned long long base_g = 0, base_s = 0;
#pragma unroll 1
  for (int k = 0; k < turns; ++k) {
    const int i = tid + k * kThreads;
    unsigned long long vg = 0, vs = 0;
    if (i < ng) {
      const int T = sm->off[sm->gs[i + 1]] - sm->off[sm->gs[i]];
      const int nt = key_tiles(0, shared_keys(a, sm, i)), nb = pair_blocks(T, TB);
      vg = two(nb * a.Hkv * item_cost(0, nt), has_single(T, TB, nb) ? a.Hkv * item_cost(1, nt) : 0);
    }
    if (i < ns) {
      const int T = sm->off[i + 1] - sm->off[i], len = sm->len[i];
      const int start = ng ? shared_keys(a, sm, find(sm->gs, ng + 1, i)) : 0;
      const int nb = pair_blocks(T, TB);
      const int pairs = nb ? pairs_before(start, len, T, TB, nb) : 0;
      int singles = 0;
      if (has_single(T, TB, nb)) singles = item_cost(1, key_tiles(start, block_end(len, T, TB, nb)));
      vs = two(pairs * a.Hkv, singles * a.Hkv);
    }
    unsigned long long xg = vg, xs = vs;
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
      const unsigned long long yg = __shfl_up_sync(0xffffffffu, xg, o);
      const unsigned long long ys = __shfl_up_sync(0xffffffffu, xs, o);
      if (lane >= o) {
        xg += yg;
        xs += ys;
      }
    }
    if (lane == 31) {
      sm->sums[0][warp] = xg;
      sm->sums[1][warp] = xs;
    }
    __syncthreads();
    xg += base_g - vg;
    xs += base_s - vs;
#pragma unroll 4
    for (int w = 0; w < kThreads / 32; ++w) {
      const unsigned long long g = sm->sums[0][w], q = sm->sums[1][w];
      if (w < warp) {
        xg += g;
        xs += q;
      }
      base_g += g;
      base_s += q;
    }
    if (i <= ng) {
      sm->cum_g[0][i] = (int)(xg >> 32);
      sm->cum_g[1][i] = (int)xg;
    }
    if (i <= ns) { /* behind the groups': added by the reader */
      sm->cum_s[0][i] = (int)(xs >> 32);
      sm->cum_s[1][i] = (int)xs;
    }
    __syncthreads();
  }
  if (tid == 0) {
    sm->pairs = (int)(base_g >> 32) + (int)(base_s >> 32);
    sm->total = sm->pairs + (int)base_g + (int)base_s;
  }
  __syncthreads();
  return true;
}

/* The piece at place x of the pairs (line 0) or the singles (1), x < end; x moves
 * behind it.  A share that ends within an item's fixed cost has no tile of it: n is
 * 0.  By a whole warp. */
__device__ __forceinline__ Piece next_piece(const Args &a, const Smem *sm, int line, int &x, int end) {
  const int TB = a.TB, ng = a.n_groups;
  const int in_groups = sm->cum_g[line][ng];
  Piece p;
  p.line = line;
  p.own = x >= in_groups;
  int j, begin, first, T; /* the item's block, its place; the block's tokens */
  if (!p.own) {
    const int g = warp_find(sm->cum_g[line], ng, x);
    first = sm->off[sm->gs[g]];
    T = sm->off[sm->gs[g + 1]] - first;
    p.seq = sm->lead[g];
    p.key0 = 0;
    p.kend = shared_keys(a, sm, g);
    p.nt = key_tiles(0, p.kend);
    const int nb = pair_blocks(T, TB);
    begin = sm->cum_g[line][g];
    const int cost = item_cost(line, p.nt), item = (x - begin) / cost;
    begin += item * cost;
    p.kvh = line == 0 ? item / nb : item;
    j = line == 0 ? item - p.kvh * nb : nb;
  } else {
    const int b = warp_find(sm->cum_s[line], a.n_seqs, x - in_groups);
    const int len = sm->len[b];
    first = sm->off[b];
    T = sm->off[b + 1] - first;
    p.seq = b;
    p.key0 = ng ? shared_keys(a, sm, warp_find(sm->gs, ng + 1, b)) : 0;
    begin = in_groups + sm->cum_s[line][b];
    const int per = (sm->cum_s[line][b + 1] - sm->cum_s[line][b]) / a.Hkv;
    p.kvh = (x - begin) / per;
    begin += p.kvh * per;
    const int nb = pair_blocks(T, TB);
    j = nb;
    if (line == 0) {
      j = warp_last(nb, [&](int i) { return pairs_before(p.key0, len, T, TB, i) <= x - begin; });
      begin += pairs_before(p.key0, len, T, TB, j);
    }
    p.kend = block_end(len, T, TB, j);
    p.nt = key_tiles(p.key0, p.kend);
  }
  p.tok0 = first + j * 2 * TB;
  p.ntok = min(2 * TB, T - j * 2 * TB);
  const Range r = piece_range(line, begin, p.nt, x, end);
  p.t0 = r.t0;
  p.n = r.n;
  x = r.next;
  p.begin = begin;
  return p;
}

/* An item's first piece tells attn_merge where the item's partials are.  By a whole
 * warp, a token a lane. */
__device__ __forceinline__ void tell_merge(const Args &a, const Smem *sm, const Piece &p) {
  const int total = sm->total, pairs = sm->pairs, n = active_ctas(total, gridDim.x);
  int w[2];
#pragma unroll 1
  for (int k = 0; k < 2; ++k) { /* the workers of the item's first tile and its last */
    const int x = p.begin + fixed_cost(p.line) + (k ? (p.nt - 1) * tile_cost(p.line) : 0);
    w[k] = worker_of(p.line, x, total, pairs, n);
  }
  const bool whole = p.own && p.key0 == 0 && p.n == p.nt;
  const int pieces = w[1] - w[0] + 1;
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < p.ntok; i += 32) {
    const int tile = i >= a.TB;
    const int row = (p.line ? 2 * (int)gridDim.x * kTile : tile * kTile) + (i - tile * a.TB) * a.G;
    a.where[((long long)p.own * a.n_tokens + p.tok0 + i) * a.Hkv + p.kvh] =
        make_int4(whole ? 1 : pieces + 1, w[0], row, p.line ? kTile : 2 * kTile);
  }
}

/* Word i of what query token `tok` of a tree sees of its sequence's tokens; of the keys before
 * them (i < 0) it sees all. */
__device__ __forceinline__ uint32_t tree_word(const Args &a, int tok, int i) {
  if (i < 0) return 0xffffffffu;
  return i < a.tree_words ? __ldcg(a.tree + (size_t)tok * a.tree_words + i) : 0;
}
/* The 32 keys from `key` on as bits, from the two words that hold them; none from `limit` on. */
__device__ __forceinline__ uint32_t tree_keys(uint32_t lo, uint32_t hi, int key, int base, int limit) {
  const uint32_t w = __funnelshift_r(lo, hi, (key - base) & 31);
  const int d = limit - key;
  return d >= 32 ? w : d <= 0 ? 0 : w & ((1u << d) - 1);
}

/* ---- the tiles ---------------------------------------------------------------- */

/* S = Q K^T of a tile; half h of O (+)= P V: P's keys 64 h .. 64 h + 63, and what their
 * rounding left, 64 columns further on. */
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t s, uint64_t q, uint64_t k, uint32_t lead) {
  using C = Cfg<D>;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    const int o = (c / (C::COLS / 16) * C::BLOCK + c % (C::COLS / 16) * 32) >> 4;
    mma_ss(s, q + o, k + o, inst_desc(kTile, false), c > 0, lead);
  }
}
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t p, uint64_t v, int h, bool acc,
                                         uint32_t lead) {
  using C = Cfg<D>;
  p += h * (kTile / 4);
  v += h * ((kTile / 2 * C::ROWB) >> 4);
#pragma unroll
  for (int c = 0; c < kTile / 32; ++c)
    mma_ts(o, p + c * 8, v + ((c * 16 * C::ROWB) >> 4), inst_desc(D, true), acc || h > 0 || c > 0,
           lead);
#pragma unroll
  for (int c = 0; c < kTile / 32; ++c)
    mma_ts(o, p + kTile / 2 + c * 8, v + ((c * 16 * C::ROWB) >> 4), inst_desc(D, true), 1, lead);
}

/* Loads tile t of a piece, as far as its keys go: a box per page (or part of one) and
 * 64 dims.  Lane i looks up the page of box i, a tile ahead. */
template <int D>
struct Loader {
  using C = Cfg<D>;
  const Args &a;
  int lane, boxes, page;
  uint32_t lead;
  __device__ Loader(const Args &a_, int lane_) : a(a_), lane(lane_) {
    boxes = kTile / a.box_rows;
    page = -1;
    lead = elect_lead();
  }
  __device__ __forceinline__ int page_of(int k) const {
    return (int)(((unsigned long long)k * a.inv_p) >> 38);
  }
  __device__ __forceinline__ void look_up(const Piece &p, int t) {
    const int k = p.key0 + (p.t0 + t) * kTile + lane * a.box_rows;
    page = -1;
    if (t < p.n && lane < boxes && k < p.kend)
      /* through L2: the grid before this one may have written the tables while this one started */
      page = __ldcg(a.tables + (size_t)p.seq * a.max_pages + page_of(k));
  }
  __device__ __forceinline__ void load(const Piece &p, int t, int pg, const CUtensorMap *map,
                                       uint8_t *tile, uint64_t *full, int *fills) {
    const int k0 = p.key0 + (p.t0 + t) * kTile;
    const int k = k0 + lane * a.box_rows;
    const bool mine = lane < boxes && k < p.kend;
    const bool good = mine && (unsigned)pg < (unsigned)a.num_pages;
    if (mine && !good) report(a, MK_ERR_PAGE_OOB);
    const unsigned set = __ballot_sync(0xffffffffu, good);
    const int y = (pg * a.Hkv + p.kvh) * a.P + k - page_of(k) * a.P;
    const uint32_t bytes = a.box_rows * C::ROWB;
    if (lead) {
      atomicAdd(fills, 1);
      bar_expect(full, __popc(set) * bytes * C::NH);
    }
    __syncwarp();
    uint32_t dst = saddr(tile);
#pragma unroll 4
    for (int i = 0; i < boxes; ++i, dst += bytes) {
      const int yi = __shfl_sync(0xffffffffu, y, i);
      const uint32_t go = (set >> i & 1) ? lead : 0;
#pragma unroll
      for (int h = 0; h < C::NH; ++h) tma_2d(dst + h * C::BLOCK, map, h * C::COLS, yi, full, go);
    }
  }
};

/* o_r = sum_j p_rj v_j, l_r = sum_j p_rj, p_rj = 2^(c q_r.k_j - m_r) over a piece's tiles of
 * 128 keys.  Of one tile the tensor cores have 512 cycles for S = Q K^T and 1024 for O += P V,
 * a row tile's 4 warps 550 for the exponentials and 2000 in all, and 64 KB of K and V take
 * an SM 2800 at its share of HBM.  So singles are bound by HBM where the cache is not in L2
 * (16 sequences in two groups over 131072 and 32768 shared keys, 352 MB: 80 us with the join,
 * 4.4 TB/s), pairs by the chain S, P, O of a stream, of which the other stream hides a part
 * (4800 tokens of 32 heads over 32768 keys: 2.8 ms, 0.92 PFLOP/s and half as much again for
 * the second product of P, tensor cores 76 % active), and small calls by their first
 * instructions: the cut, 2.6 us, the first tile 6 us after the start.
 * TREE: among its sequence's tokens a row sees those that its bits name (one at or before itself);
 * only tiles with such keys look at them, and the words are fetched while S is under way (8 trees of
 * 33 to 62 tokens over 6700 to 8200 keys: 74.4 us, the same batch without bits 74.5). */
template <int D, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
               const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args a) {
  using C = Cfg<D>;
  constexpr int R = C::STAGES / 2; /* K (and V) slots of a stream; pairs use all of both */
  extern __shared__ uint8_t raw[];
  uint8_t *base = (uint8_t *)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint8_t *qs = base, *ks = qs + 2 * C::TILE, *vs = ks + C::STAGES * C::TILE;
  Smem *sm = (Smem *)(vs + C::STAGES * C::TILE);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0); /* uniform for the compiler too */

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      bar_init(&sm->kfull[i], 1);
      bar_init(&sm->kempty[i], 2);
      bar_init(&sm->vfull[i], 1);
      bar_init(&sm->vempty[i], 2);
    }
    for (int s = 0; s < 2; ++s) {
      bar_init(&sm->sfull[s], 1);
      bar_init(&sm->pready[s][0], 4);
      bar_init(&sm->pready[s][1], 4);
      bar_init(&sm->q_full[s], 1);
      bar_init(&sm->q_free[s], 4);
      bar_init(&sm->oready[s], 1);
      bar_init(&sm->turn[s], 4);
      bar_init(&sm->drain[s], 1);
      for (int i = 0; i < kQueue; ++i) {
        bar_init(&sm->qfull[s][i], 1);
        bar_init(&sm->qempty[s][i], 5); /* the issuer, four softmax warps */
      }
    }
    sm->stop.abort = 0;
    sm->stop.limit = a.wait_limit;
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < C::STAGES; ++k) sm->fills[i][k] = 0;
      sm->q_fills[i] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 10) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     saddr(&sm->tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const bool sound = take_cut(a, sm);
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  Stop *stop = &sm->stop;
  const long long n_cta = gridDim.x;
  const int TB = a.TB;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const int s = warp & 1;
    if (warp < 10) {
      /* ---- producer of stream s.  It also takes the stream's pieces, some ahead: first the
       * CTA's share of the pairs, the same for both, then the stream's share of the singles.
       * Of the pairs stream 0's loads K and stream 1's loads V, into all slots; of the singles
       * each loads both of its stream, K before V, the order in which the products need them. */
      Loader<D> ld(a, lane);
      int x = 0, end = 0, x1 = 0, end1 = 0; /* this stream's share of the pairs, the singles */
      if (sound) {
        const int total = sm->total, pairs = sm->pairs, n = active_ctas(total, gridDim.x);
        if ((int)blockIdx.x < n) {
          const Share mine = share_of(blockIdx.x, s, total, pairs, n);
          x = mine.x;
          end = mine.end;
          x1 = mine.x1;
          end1 = mine.end1;
        }
      }
      uint32_t armed_k = 0, armed_v = 0; /* parities of each slot's next use */
      bool ok = true;
      int line = 0, it = 0, ring = 0, q_uses = 0;
      for (int put = 0; ok; ++put) {
        Piece p;
        p.n = 0;
        while (p.n == 0 && line < 2) {
          if (x < end) {
            p = next_piece(a, sm, line, x, end);
          } else if (++line == 1) {
            x = x1;
            end = end1;
            for (int i = 0; i < C::STAGES; ++i) /* uses of each slot so far */
              armed_k |= (uint32_t)(((it + C::STAGES - 1 - i) / C::STAGES) & 1) << i;
            armed_v = armed_k;
          }
        }
        const int qslot = put % kQueue;
        ok = warp_wait(&sm->qempty[s][qslot], ((put / kQueue) & 1) ^ 1, stop);
        if (!ok) break;
        if (lane == 0) {
          sm->queue[s][qslot] = p;
          bar_arrive(&sm->qfull[s][qslot]);
        }
        __syncwarp();
        if (p.n == 0) break;
        ld.look_up(p, 0);
        const int q_tok = p.tok0 + (line == 0 ? s * TB : 0);
#pragma unroll 1
        for (int t = 0; ok && t < p.n; ++t) {
          const int page = ld.page;
          ld.look_up(p, t + 1);
          const int slot = line == 0 ? it % C::STAGES : s * R + ring;
#pragma unroll 1
          for (int kv = line == 0 ? s : 0; kv <= (line == 0 ? s : 1); ++kv) {
            const uint32_t par = line == 0 ? it / C::STAGES : (kv ? armed_v : armed_k) >> slot;
            ok = warp_wait(kv ? &sm->vempty[slot] : &sm->kempty[slot], (par & 1) ^ 1, stop);
            if (!ok) break;
            ld.load(p, t, page, kv ? &vmap : &kmap, (kv ? vs : ks) + slot * C::TILE,
                    kv ? &sm->vfull[slot] : &sm->kfull[slot], &sm->fills[kv][slot]);
            if (line == 1) (kv ? armed_v : armed_k) ^= 1u << slot;
            if (t == 0 && (line == 0 || kv == 0)) {
              /* Q: [tokens][heads of the group][64 dims], the rows' order.  Rows behind the
               * last token are other rows of Q or zeros, and are not looked at. */
              ok = warp_wait(&sm->q_free[s], (q_uses & 1) ^ 1, stop);
              if (!ok) break;
              ++q_uses;
              if (ld.lead) {
                ++sm->q_fills[s];
                bar_expect(&sm->q_full[s], C::NH * C::ROWB * TB * a.G);
              }
              __syncwarp();
#pragma unroll
              for (int h = 0; h < C::NH; ++h)
                tma_3d(saddr(qs + s * C::TILE + h * C::BLOCK), &qmap, h * C::COLS, p.kvh * a.G, q_tok,
                       &sm->q_full[s], ld.lead);
            }
          }
          if (!ok) break;
          if (t == 0 && p.t0 == 0 && (line == 1 || s == 0)) tell_merge(a, sm, p);
          if (line == 0)
            ++it;
          else
            ring = ring + 1 == R ? 0 : ring + 1;
        }
      }
    } else {
      /* ---- issuer of stream s: S = Q K^T of a tile, then O += P V of its halves as P comes.
       * The other stream's issuer fills the tensor cores meanwhile. */
      const uint32_t lead = elect_lead();
      const uint32_t at_s = tmem + s * kTile, at_o = at_s + 2 * kTile;
      const uint64_t q0 = mat_desc(saddr(qs), 16, 8 * C::ROWB, C::SWIZZLE);
      const uint64_t k0 = mat_desc(saddr(ks), 16, 8 * C::ROWB, C::SWIZZLE);
      const uint64_t v0 = mat_desc(saddr(vs), C::BLOCK, 8 * C::ROWB, C::SWIZZLE);
      bool ok = !(a.poison && s == 0) || warp_wait(&sm->drain[s], 0, stop);
      int it = 0, ring = 0;
      uint32_t par = 0, q_par = 0, p_par = 0; /* singles: parities of the stream's slots */
      bool singles = false;
      for (int got = 0; ok; ++got) {
        const int qslot = got % kQueue;
        ok = warp_wait(&sm->qfull[s][qslot], (got / kQueue) & 1, stop);
        if (!ok) break;
        const int n = sm->queue[s][qslot].n, line = sm->queue[s][qslot].line;
        __syncwarp();
        if (lane == 0) bar_arrive(&sm->qempty[s][qslot]);
        if (n == 0) break;
        if (line == 1 && !singles) {
          singles = true;
          for (int i = 0; i < C::STAGES; ++i)
            par |= (uint32_t)(((it + C::STAGES - 1 - i) / C::STAGES) & 1) << i;
        }
        ok = warp_wait(&sm->q_full[s], q_par, stop);
        if (!ok) break;
        q_par ^= 1;
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
          const int slot = line == 0 ? it % C::STAGES : s * R + ring;
          const uint32_t parity = (line == 0 ? it / C::STAGES : par >> slot) & 1;
          const uint32_t o = (uint32_t)slot * (C::TILE >> 4);
          ok = warp_wait(&sm->kfull[slot], parity, stop);
          if (!ok) break;
          tc_fence_after();
          issue_qk<D>(at_s, q0 + (uint32_t)s * (C::TILE >> 4), k0 + o, lead);
          tc_commit(&sm->sfull[s], lead);
          tc_commit(&sm->kempty[slot], lead);
          if (line == 1) tc_commit(&sm->kempty[slot], lead); /* a pair's two readers count one each */
          ok = warp_wait(&sm->vfull[slot], parity, stop);
          for (int h = 0; ok && h < 2; ++h) {
            ok = warp_wait(&sm->pready[s][h], p_par, stop);
            tc_fence_after();
            if (ok) issue_pv<D>(at_o, at_s, v0 + o, h, t > 0, lead);
          }
          if (!ok) break;
          p_par ^= 1;
          if (t == n - 1) tc_commit(&sm->oready[s], lead);
          tc_commit(&sm->vempty[slot], lead);
          if (line == 1) {
            tc_commit(&sm->vempty[slot], lead);
            par ^= 1u << slot;
            ring = ring + 1 == R ? 0 : ring + 1;
          } else {
            ++it;
          }
        }
        if (!ok) break;
      }
      /* The products, and what their commits write into shared memory, end here in any case. */
      Stop last{0, kWaitLimit};
      tc_commit(&sm->drain[s], lead);
      if (!warp_wait(&sm->drain[s], 0, &last)) *(volatile int *)&stop->abort = 1;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    /* ---- softmax: stream s, one row a thread */
    const int s = warp >> 2, r = tid & (kTile - 1), w0 = (warp & 3) * 32;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21; /* this warp's TMEM lanes */
    const uint32_t at_s = tmem + lanes + s * kTile, at_o = at_s + 2 * kTile;
    uint8_t *qd = qs + s * C::TILE + w0 * C::ROWB; /* this warp's rows of Q */
    const float c2 = a.scale_log2;
    uint32_t s_par = 0, o_par = 0;
    int it = 0, ring = 0;   /* pair tiles; this stream's slot */
    uint32_t v_par = 0;     /* parities of this stream's slots, set behind the pairs */
    int got = 0;
    bool ok = true;
    for (; ok; ++got) {
      const int qslot = got % kQueue;
      ok = warp_wait(&sm->qfull[s][qslot], (got / kQueue) & 1, stop);
      if (!ok) break;
      const Piece c = sm->queue[s][qslot];
      __syncwarp();
      if (lane == 0) bar_arrive(&sm->qempty[s][qslot]);
      if (c.n == 0) break;
      const bool pair = c.line == 0;
      if (!pair && v_par >> 31 == 0) {
        v_par = 1u << 31;
        for (int i = 0; i < C::STAGES; ++i)
          v_par |= (uint32_t)(((it + C::STAGES - 1 - i) / C::STAGES) & 1) << i;
      }
      const int ctok0 = c.tok0 + (pair ? s * TB : 0);
      const int crows = min(TB, c.tok0 + c.ntok - ctok0) * a.G;
      const bool valid = r < crows, busy = w0 < crows;
      const int rt = valid ? (r * a.inv_g) >> 16 : 0, tok = ctok0 + rt;
      const int b = c.own ? c.seq : a.off ? find(sm->off, a.n_seqs + 1, tok) : tok;
      /* keys of the item that this row sees end here */
      const int limit = min(c.kend, sm->len[b] - (sm->off[b + 1] - tok) + 1);
      const int base = TREE ? sm->len[b] - (sm->off[b + 1] - sm->off[b]) : 0; /* the tokens' first place */
      /* below it every row of the warp sees all */
      const int warp_limit = __reduce_min_sync(0xffffffffu, TREE ? min(limit, base) : limit);
      float m = -INFINITY, l = 0.0f; /* m in score units */
#pragma unroll 1
      for (int t = 0; t < c.n; ++t) {
        const int k0 = c.key0 + (c.t0 + t) * kTile;
        uint32_t seen[TREE ? kTile / 32 : 1];
        if (TREE && busy && warp_limit < k0 + kTile) {
          uint32_t lo = tree_word(a, tok, (k0 - base) >> 5);
#pragma unroll
          for (int i = 0; i < kTile / 32; ++i) {
            const uint32_t hi = tree_word(a, tok, ((k0 - base) >> 5) + i + 1);
            seen[TREE ? i : 0] = tree_keys(lo, hi, k0 + 32 * i, base, limit);
            lo = hi;
          }
        }
        ok = warp_wait(&sm->sfull[s], s_par, stop);
        if (!ok) break;
        s_par ^= 1;
        tc_fence_after();
        if (pair && it + s > 0) {
          /* The streams of a pair take turns, stream 0's tile before stream 1's: side by
           * side they would share the exponential unit and then leave it, and the tensor
           * cores, idle together (4800 tokens over 32768 keys: 3.27 ms, so 2.89). */
          ok = warp_wait(&sm->turn[s], (it - 1 + s) & 1, stop);
          if (!ok) break;
        }
        const int slot = pair ? it % C::STAGES : s * R + ring;
        if (k0 + kTile > c.kend) {
          /* zero the V rows behind the last key: what lies there may be NaN */
          ok = warp_wait(&sm->vfull[slot], pair ? (it / C::STAGES) & 1 : (v_par >> slot) & 1,
                         stop);
          if (!ok) break;
          if (k0 + r >= c.kend) {
            uint8_t *vr = vs + slot * C::TILE + r * C::ROWB;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *(uint4 *)(vr + i / (C::COLS / 8) * C::BLOCK + i % (C::COLS / 8) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_async_smem();
        }
        if (pair) {
          ++it;
        } else {
          v_par ^= 1u << slot;
          ring = ring + 1 == R ? 0 : ring + 1;
        }
        if (!busy) {
          __syncwarp();
          if (lane == 0) {
            bar_arrive(&sm->pready[s][0]);
            bar_arrive(&sm->pready[s][1]);
            if (pair) bar_arrive(&sm->turn[1 - s]);
          }
          continue;
        }
        float x[kTile];
        tmem_ld128(at_s, x);
        if (TREE && warp_limit < k0 + kTile) {
#pragma unroll
          for (int i = 0; i < kTile; ++i) x[i] = seen[TREE ? i / 32 : 0] >> i % 32 & 1 ? x[i] : -INFINITY;
        } else if (warp_limit < k0 + kTile) {
          const int d = limit - k0;
#pragma unroll
          for (int i = 0; i < kTile; ++i) x[i] = i < d ? x[i] : -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 4; i < kTile; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = i + k + 4 < kTile ? fmaxf(mx[k], fmaxf(x[i + k], x[i + k + 4]))
                                      : fmaxf(mx[k], x[i + k]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (t == 0) {
          m = top;
        } else {
          const bool move = m == -INFINITY ? top > m : (top - m) * c2 > kSlack;
          if (__any_sync(0xffffffffu, move)) {
            /* the products into O so far are complete: they were issued before this S */
            const float now = move ? top : m;
            const float f = move ? exp2_approx((m - now) * c2) : 1.0f; /* m -inf: 0 */
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              float o[16];
              tmem_ld16(at_o + i, o);
              uint32_t w[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * f);
              tmem_st16(at_o + i, w);
            }
            l *= f;
            m = now;
          }
        }
        const float off = m == -INFINITY ? 0.0f : -m * c2;
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        /* P in quarters; the product of the first half starts under the second.  A quarter's
         * store lands while the next is computed.  P goes into the product as a bf16 value and
         * the bf16 rounding of what that leaves, so it is good to 2^-17, as in the decode step
         * (bf16 alone moves a result by about as much as the result's own rounding does).  The
         * second product and its operand cost 64 samples of one prompt 13 % (36 us, with them
         * 41), 16 sequences over long prefixes 7 % (75, 80), 4800 tokens over 32768 keys a third
         * (2.12 ms, 2.83). */
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t w[16], rest[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 e = fma2(make_float2(x[h * 32 + 2 * k], x[h * 32 + 2 * k + 1]),
                            make_float2(c2, c2), make_float2(off, off));
            e.x = exp2_approx(e.x);
            e.y = exp2_approx(e.y);
            sum[k & 1] = add2(sum[k & 1], e);
            w[k] = pack_bf16(e.x, e.y);
            rest[k] = rest_bf16(w[k], e);
          }
          if (h != 2) {
            tmem_st16(at_s + h * 16, w);
            tmem_st16(at_s + kTile / 2 + h * 16, rest);
          }
          if (h >= 2) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              bar_arrive(&sm->pready[s][h - 2]);
              if (h == 2 && pair) bar_arrive(&sm->turn[1 - s]); /* behind h 3: 2.89 ms for 2.85 */
            }
          }
          if (h == 2) {
            tmem_st16(at_s + h * 16, w);
            tmem_st16(at_s + kTile / 2 + h * 16, rest);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      }
      if (!ok) break;
      ok = warp_wait(&sm->oready[s], o_par, stop);
      if (!ok) break;
      o_par ^= 1;
      tc_fence_after();
      if (busy) {
        /* the lane again, so that addresses made of it are not kept across the pieces */
        int ln = lane;
        asm volatile("" : "+r"(ln));
        /* rows of O through this warp's part of Q (read by now), so that a row's
         * columns are written together */
        const bool whole = c.own && c.key0 == 0 && c.n == c.nt; /* nothing to merge */
        const int row0 = ctok0 * a.Hq + c.kvh * a.G;    /* output row of (token, head) 0 */
        const long long dense = (long long)a.n_tokens * a.Hq;
        const long long extra =
            2 * dense + (pair ? 2ll * blockIdx.x + s : 2ll * n_cta + 2ll * blockIdx.x + s) * kTile;
        constexpr int W = D / 2, CR = C::ROWB / 16; /* columns staged at a time; float4 of a swizzled row */
        constexpr int RL = W / 4, RI = 32 / RL;     /* lanes of a row, rows at a time */
        const int ch = ln % RL, mine = min(32, crows - w0); /* rows of this warp */
        float *to = a.part + (c.t0 ? extra : c.own * dense + row0) * D + ch * 4;
        const float f = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l; /* NaN stays NaN */
        float odd = 0.0f; /* NaN if a column is not finite */
#pragma unroll 1
        for (int i0 = 0; i0 < D; i0 += W) {
          float o[W];
          if (W == 64)
            tmem_ld64(at_o + i0, o);
          else if (W == 32)
            tmem_ld32(at_o + i0, o);
          else
            tmem_ld16(at_o + i0, o);
          if (TREE && whole) {
#pragma unroll
            for (int k = 0; k < W; ++k) odd = fmaf(o[k], 0.0f, odd);
          }
#pragma unroll
          for (int k = 0; k < W / 4; ++k)
            *(float4 *)(qd + k / CR * C::BLOCK + ln * C::ROWB + ((k % CR) ^ (ln & (CR - 1))) * 16) =
                make_float4(o[4 * k] * f, o[4 * k + 1] * f, o[4 * k + 2] * f, o[4 * k + 3] * f);
          __syncwarp();
#pragma unroll 4
          for (int row = ln / RL; row < mine; row += RI) {
            const int rr = w0 + row, qt = (rr * a.inv_g) >> 16;
            const float4 v = *(const float4 *)(qd + ch / CR * C::BLOCK + row * C::ROWB +
                                               ((ch % CR) ^ (row & (CR - 1))) * 16);
            const int at = c.t0 ? rr : qt * a.Hq + (rr - qt * a.G); /* row behind `to` */
            if (whole)
              *(uint2 *)(a.out + (long long)(row0 + at) * D + ch * 4 + i0) =
                  make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            else
              *(float4 *)(to + (long long)at * D + i0) = v;
          }
          __syncwarp();
        }
        const long long orow = row0 + (long long)rt * a.Hq + (r - rt * a.G);
        if (valid && whole) {
          if (a.lse)
            a.lse[orow] = l == 0.0f ? -INFINITY : (m * c2 + log2f(l)) * 0.69314718055994531f;
          if (TREE)
            a.part_ml[dense + orow] = make_float2(m == -INFINITY ? m : m * c2, odd == odd || l != l ? -1.0f : l);
        } else if (valid) {
          a.part_ml[c.t0 ? extra + r : c.own * dense + orow] =
              make_float2(l != l ? 0.0f : m == -INFINITY ? m : m * c2, l); /* NaN goes by l */
        }
      }
      tc_fence_before();
      fence_async_smem(); /* this warp's part of Q may be loaded over */
      __syncwarp();
      if (lane == 0) bar_arrive(&sm->q_free[s]);
    }
  }
  if (blockIdx.x == 0 && tid == 0) {
    *a.bad = !sound;
    if (!sound) report(a, MK_ERR_INVALID_ARG);
  }
  __syncthreads();
  if (warp == 10) {
    if (*(volatile int *)&stop->abort) {
      /* Somebody gave up, so nobody may have waited for the last copy into each slot.  Shared
       * memory stays until they have landed. */
      if (lane == 0) report(a, MK_ERR_DEVICE_TIMEOUT);
      Stop last{0, kWaitLimit};
      for (int i = 0; i < 2; ++i)
        if (sm->q_fills[i]) warp_wait(&sm->q_full[i], (sm->q_fills[i] - 1) & 1, &last);
      for (int i = 0; i < C::STAGES; ++i) {
        if (sm->fills[0][i]) warp_wait(&sm->kfull[i], (sm->fills[0][i] - 1) & 1, &last);
        if (sm->fills[1][i]) warp_wait(&sm->vfull[i], (sm->fills[1][i] - 1) & 1, &last);
      }
    }
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

/* ---- the join ----------------------------------------------------------------- */

/* Rows of a tree's results that are not finite, once more: the products with V take weights of 0 for the
 * keys that a row does not see, and 0 times what lies there may be NaN.  By the block that has heads h0 to
 * h1 of a token: columns where a hidden value is not finite are summed again over what the token sees, for
 * the heads whose sum ml.y is not -1, against the maximum and sum of the row, which V does not reach.
 * Other columns are what the definition gives.  Rare, and slow, since it reads a row's keys again: a value
 * that is not finite in each of 8 trees of 40 tokens over 8000 keys makes the call take 3.6 ms (78 us), of 2
 * over 106000 keys 22.5 ms (190 us).  Where all is finite, knowing so costs 16 trees behind two prompts
 * 0.8 us of 82. */
template <int D>
__device__ __noinline__ void redo_rows(const Args &a, int tok, int kvh, int h0, int h1, const float2 *ml) {
  constexpr int N = D / 32, C = D / 8; /* columns a lane, 16-byte pieces of a row */
  __shared__ uint4 s_q[8][C], s_k[32][C + 1], s_v[32][C];
  __shared__ bool s_seen[32], s_again[D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int b = tok;
  if (a.off) { /* the last sequence that begins at or before it */
    int hi = a.n_seqs - 1;
    for (b = 0; b < hi;) {
      const int m = (b + hi + 1) >> 1;
      if (__ldcg(a.off + m) <= tok)
        b = m;
      else
        hi = m - 1;
    }
  }
  const int first = a.off ? __ldcg(a.off + b) : b, end = a.off ? __ldcg(a.off + b + 1) : b + 1;
  const int len = __ldcg(a.lens + b), base = len - (end - first), limit = len - (end - tok) + 1;
  auto sees = [&](int key) -> bool {
    if (key < base || key >= limit) return key < limit;
    const int u = key - base;
    return __ldcg(a.tree + (size_t)tok * a.tree_words + (u >> 5)) >> (u & 31) & 1;
  };
  auto row_of = [&](int key) -> long long { /* in the pools, -1 for a page that is out of range */
    const int page = __ldcg(a.tables + (size_t)b * a.max_pages + key / a.P);
    if ((unsigned)page >= (unsigned)a.num_pages) return -1;
    return (((long long)page * a.Hkv + kvh) * a.P + key % a.P) * D;
  };
  bool again = false;
  if (tid < D) {
    for (int key = max(base, 0); key < len; ++key) {
      const long long at = sees(key) ? -1 : row_of(key);
      if (at >= 0) again |= (__ldcg((const unsigned short *)a.v_pool + at + tid) & 0x7f80) == 0x7f80;
    }
    s_again[tid] = again;
  }
  if (!__syncthreads_or(again)) return;
  for (int hg0 = h0; hg0 < h1; hg0 += 8) {
    const int hg = hg0 + warp, hq = kvh * a.G + hg;
    const bool mine = hg < h1 && ml[hg - h0].y >= 0.0f;
    if (!__syncthreads_or(mine)) continue;
    const float M = mine ? ml[hg - h0].x : -INFINITY;
    if (mine && lane < C) s_q[warp][lane] = __ldcg((const uint4 *)(a.q + tok * a.q_stride + hq * D) + lane);
    float o[N] = {};
    for (int key0 = 0; key0 < limit; key0 += 32) {
      __syncthreads();
      for (int i = tid; i < 32 * C; i += 256) {
        const int j = i / C, c = i % C, key = key0 + j;
        const long long at = key < limit && sees(key) ? row_of(key) : -1;
        s_k[j][c] = at < 0 ? make_uint4(0, 0, 0, 0) : __ldcg((const uint4 *)(a.k_pool + at) + c);
        s_v[j][c] = at < 0 ? make_uint4(0, 0, 0, 0) : __ldcg((const uint4 *)(a.v_pool + at) + c);
        if (c == 0) s_seen[j] = at >= 0;
      }
      __syncthreads();
      if (M == -INFINITY) continue;
      float x = 0.0f;
#pragma unroll 4
      for (int c = 0; c < C; ++c) {
        const uint4 q = s_q[warp][c], k = s_k[lane][c];
        const uint32_t qs[4] = {q.x, q.y, q.z, q.w}, ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x = fmaf(__uint_as_float(qs[i] << 16), __uint_as_float(ks[i] << 16), x);
          x = fmaf(__uint_as_float(qs[i] & 0xffff0000u), __uint_as_float(ks[i] & 0xffff0000u), x);
        }
      }
      const float p = s_seen[lane] ? exp2_approx(fmaf(x, a.scale_log2, -M)) : 0.0f;
#pragma unroll 4
      for (int j = 0; j < 32; ++j) {
        const float w = __shfl_sync(0xffffffffu, p, j);
        const unsigned short *v = (const unsigned short *)s_v[j] + lane * N;
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = fmaf(w, __uint_as_float((uint32_t)v[k] << 16), o[k]);
      }
    }
    if (!mine) continue;
    const float l = ml[hg - h0].y, inv = l == 0.0f ? 0.0f : 1.0f / l;
    __nv_bfloat16 *dst = a.out + ((size_t)tok * a.Hq + hq) * D + lane * N;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (s_again[lane * N + k]) dst[k] = __float2bfloat16_rn(o[k] * inv);
  }
}

/* M = max m_i, out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i over a row's pieces.  A
 * block has a token and kv head, or some heads of its group (`blocks` blocks, a cluster,
 * share it) where there are too few for all SMs; its warps take the heads, several a head
 * where there are fewer than eight.  Reads L2: the partials were written just before.
 * What bounds it is its chain of three loads (where, maxima and sums, weighted sums), so
 * 32 pieces' maxima and four pieces' sums are in flight together (with eight, and 80
 * registers, fewer blocks fit an SM: 64 samples of one prompt 42 us, so 38); where blocks are
 * MANY, more of them an SM instead. */
template <int D, bool MANY, bool TREE>
__global__ void __launch_bounds__(256, MANY ? 7 : 4) attn_merge(const __grid_constant__ Args a, int n_cta, int blocks) {
  __shared__ float sums[8][D];
  __shared__ float2 odd_ml[TREE ? 64 : 1]; /* of heads whose results are not finite: for redo_rows */
  bool any_odd = false;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = blockIdx.x / blocks, rank = blockIdx.x - unit * blocks, units = a.n_tokens * a.Hkv;
  const int tok = unit / a.Hkv, kvh = unit - tok * a.Hkv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int bad = *a.bad, tokens = a.off ? a.off[a.n_seqs] : a.n_seqs;
  const int4 ws = a.where[unit], wo = a.where[units + unit];
  if (bad || tok >= tokens) return;
  /* read by all: cleared for the next call */
  __syncthreads();
  if (blocks > 1)
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
  if (rank == 0 && threadIdx.x < 2) a.where[threadIdx.x * units + unit] = make_int4(0, 0, 0, 0);
  const int heads = (a.G + blocks - 1) / blocks, h0 = rank * heads, h1 = min(a.G, h0 + heads);
  if (wo.x == 1) { /* written by attn_tiles */
    if (TREE) {
      const int hg = h0 + threadIdx.x;
      bool odd = false;
      if (hg < h1) {
        odd_ml[threadIdx.x] = a.part_ml[(size_t)(a.n_tokens + tok) * a.Hq + kvh * a.G + hg];
        odd = odd_ml[threadIdx.x].y >= 0.0f;
      }
      if (__syncthreads_or(odd)) redo_rows<D>(a, tok, kvh, h0, h1, odd_ml);
    }
    return;
  }
  const int n_shared = ws.x ? ws.x - 1 : 0, n = n_shared + (wo.x ? wo.x - 1 : 0);
  int split = 8; /* warps a head */
  while (split > 1 && 8 / split < heads) split >>= 1;
  const int part = warp % split, at_once = 8 / split;
  const uint32_t dense = (uint32_t)a.n_tokens * a.Hq; /* rows: below 2^32 by the limits of create */
  for (int hg0 = h0; hg0 < h1; hg0 += at_once) {
    const int hg = min(hg0 + warp / split, a.G - 1);
    const bool mine = hg0 + warp / split < h1;
    const uint32_t orow = (uint32_t)tok * a.Hq + kvh * a.G + hg;
    const uint32_t at_s = 2 * dense + ws.y * ws.w + ws.z + hg;
    const uint32_t at_o = 2 * dense + wo.y * wo.w + wo.z + hg;
    auto place = [&](int i) -> uint32_t { /* partial row of piece i */
      const int k = i - n_shared;
      if (k < 0) return i ? at_s + i * ws.w : orow;
      return k ? at_o + k * wo.w : dense + orow;
    };
    constexpr int N = D / 32; /* columns a lane */
    float o[N] = {}, l = 0.0f, M = -INFINITY;
    if (mine)
      for (int i = lane; i < n; i += 32) M = fmaxf(M, a.part_ml[place(i)].x);
#pragma unroll
    for (int w = 16; w; w >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, w));
    if (M != -INFINITY) {
      for (int i0 = 0; i0 < n; i0 += 32) {
        float f = 0.0f;
        uint32_t row = 0;
        if (i0 + lane < n) {
          row = place(i0 + lane);
          const float2 ml = a.part_ml[row];
          f = exp2_approx(ml.x - M);
          l += f * ml.y;
        }
        const int m = min(32, n - i0);
#pragma unroll(MANY ? 2 : 4)
        for (int i = part; i < m; i += split) {
          const float w = __shfl_sync(0xffffffffu, f, i);
          const float *src = a.part + (size_t)__shfl_sync(0xffffffffu, row, i) * D + lane * N;
          float v[N];
          if (N == 4)
            *(float4 *)v = *(const float4 *)src;
          else if (N == 2)
            *(float2 *)v = *(const float2 *)src;
          else
            v[0] = src[0];
#pragma unroll
          for (int k = 0; k < N; ++k) o[k] = fmaf(w, v[k], o[k]);
        }
      }
#pragma unroll
      for (int w = 16; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
    }
    if (split > 1) { /* the warps' sums, in order */
#pragma unroll
      for (int k = 0; k < N; ++k) sums[warp][k * 32 + lane] = o[k];
      __syncthreads();
      if (part == 0)
        for (int w = 1; w < split; ++w)
#pragma unroll
          for (int k = 0; k < N; ++k) o[k] += sums[warp + w][k * 32 + lane];
      __syncthreads();
    }
    if (!mine || part) continue;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l; /* NaN stays NaN */
    __nv_bfloat16 *dst = a.out + (size_t)orow * D + lane * N;
    if (N == 4) {
      *(uint2 *)dst =
          make_uint2(pack_bf16(o[0] * inv, o[1 % N] * inv), pack_bf16(o[2 % N] * inv, o[3 % N] * inv));
    } else if (N == 2) {
      *(uint32_t *)dst = pack_bf16(o[0] * inv, o[1 % N] * inv);
    } else {
      *dst = __float2bfloat16_rn(o[0] * inv);
    }
    if (a.lse && lane == 0)
      a.lse[orow] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
    if (TREE) {
      float odd = 0.0f; /* NaN if a column is not finite; where the sum is NaN, so is the row */
#pragma unroll
      for (int k = 0; k < N; ++k) odd = fmaf(o[k], 0.0f, odd);
      const bool again = __any_sync(0xffffffffu, odd != odd) && l == l;
      if (lane == 0) odd_ml[hg - h0] = make_float2(M, again ? l : -1.0f);
      any_odd |= again;
    }
  }
  if (TREE && __syncthreads_or(any_odd)) redo_rows<D>(a, tok, kvh, h0, h1, odd_ml);
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
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  return (uintptr_t)a < (uintptr_t)b + (uint64_t)nb && (uintptr_t)b < (uintptr_t)a + (uint64_t)na;
}

}  // namespace

struct mk_attn {
  mk_attn_desc d{};
  std::vector<CUtensorMap> maps;    /* K and V of each layer */
  std::vector<const void *> pools; /* the same */
  float scale_log2 = 0.0f;
  int box_rows = 0;
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0;
  unsigned long long wait_limit = kWaitLimit;
  bool poison = false; /* the next call */
  uint8_t *ws = nullptr;
  size_t o_where = 0, o_part = 0, o_ml = 0;
  int32_t *err_host = nullptr, *err_dev = nullptr;
};

namespace {

template <int D>
cudaError_t prepare() {
  static_assert(Cfg<D>::SMEM + sizeof(Smem) <= 232448, "shared memory of a CTA");
  constexpr int smem = Cfg<D>::SMEM + (int)sizeof(Smem);
  const cudaError_t e =
      cudaFuncSetAttribute(attn_tiles<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attn_tiles<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int D>
cudaError_t launch(const mk_attn *at, int layer, const CUtensorMap &qmap, const Args &a) {
  cudaLaunchAttribute pdl[2];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(at->n_sm);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D>::SMEM + sizeof(Smem);
  cfg.stream = at->stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const CUtensorMap &kmap = at->maps[2 * layer], &vmap = at->maps[2 * layer + 1];
  const cudaError_t e = a.tree ? cudaLaunchKernelEx(&cfg, attn_tiles<D, true>, qmap, kmap, vmap, a)
                               : cudaLaunchKernelEx(&cfg, attn_tiles<D, false>, qmap, kmap, vmap, a);
  if (e != cudaSuccess) return e;
  int blocks = 1;
  while (2 * blocks <= a.G && blocks < 8 && a.n_tokens * a.Hkv * blocks < 2 * at->n_sm) blocks *= 2;
  pdl[1].id = cudaLaunchAttributeClusterDimension;
  pdl[1].val.clusterDim = {(unsigned)blocks, 1, 1};
  cfg.numAttrs = 2;
  cfg.gridDim = dim3((unsigned)a.n_tokens * a.Hkv * blocks);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  const bool many = a.n_tokens * a.Hkv >= 16 * at->n_sm;
  return a.tree ? cudaLaunchKernelEx(&cfg, many ? attn_merge<D, true, true> : attn_merge<D, false, true>, a, at->n_sm, blocks)
                : cudaLaunchKernelEx(&cfg, many ? attn_merge<D, true, false> : attn_merge<D, false, false>, a, at->n_sm, blocks);
}

}  // namespace

extern "C" {

mk_status mk_attn_create(const mk_attn_desc *d, void *stream, mk_attn **out) {
  if (!d || !out) return MK_ERR_INVALID_ARG;
  if (d->n_q_heads < 1 || d->n_kv_heads < 1 || d->head_dim < 1 || d->page_size < 1 ||
      d->num_pages < 1 || d->max_tokens < 1 || d->max_seqs < 1 ||
      d->max_groups < 0 || d->n_layers < 1 || d->n_q_heads % d->n_kv_heads ||
      !(d->scale >= 0.0f))
    return MK_ERR_INVALID_ARG;
  /* of the scores, for powers of two */
  const double scale = d->scale > 0.0f ? (double)d->scale : 1.0 / std::sqrt((double)d->head_dim);
  const float scale_log2 = (float)(scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return MK_ERR_INVALID_ARG;
  if ((d->head_dim != 32 && d->head_dim != 64 && d->head_dim != 128) || d->page_size % 16 ||
      d->page_size > 256 || d->n_q_heads / d->n_kv_heads > 64 || d->n_q_heads > 1024 ||
      d->max_tokens > (1 << 20) || d->max_seqs > kMaxSeqs || d->max_groups > kMaxGroups ||
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
  at->scale_log2 = scale_log2;
  at->stream = (cudaStream_t)stream;
  at->dev = dev;
  at->n_sm = prop.multiProcessorCount;
  /* a box lies within a page: as many of a tile's rows as divide the page */
  at->box_rows = d->page_size & -d->page_size;
  if (at->box_rows > kTile) at->box_rows = kTile;
  mk_status st = MK_OK;
  try {
    at->maps.resize(2 * (size_t)d->n_layers);
    for (int l = 0; l < d->n_layers; ++l) {
      at->pools.push_back(d->k_caches[l]);
      at->pools.push_back(d->v_caches[l]);
    }
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
  const size_t rows = 2 * (size_t)d->max_tokens * d->n_q_heads + (size_t)at->n_sm * 4 * kTile;
  at->o_where = 256;
  at->o_part = at->o_where + (2 * (size_t)d->max_tokens * d->n_kv_heads * sizeof(int4) + 255) / 256 * 256;
  at->o_ml = at->o_part + rows * d->head_dim * 4;
  cudaError_t e = d->head_dim == 32 ? prepare<32>() : d->head_dim == 64 ? prepare<64>() : prepare<128>();
  if (e == cudaSuccess) e = cudaMalloc(&at->ws, at->o_ml + rows * sizeof(float2));
  if (e == cudaSuccess) e = cudaMemsetAsync(at->ws, 0, at->o_part, at->stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(at->stream);
  if (e == cudaSuccess) e = cudaHostAlloc(&at->err_host, 64, cudaHostAllocMapped);
  if (e == cudaSuccess) {
    std::memset(at->err_host, 0, 64);
    e = cudaHostGetDevicePointer((void **)&at->err_dev, at->err_host, 0);
  }
  if (e != cudaSuccess) {
    mk_attn_destroy(at);
    cudaGetLastError(); /* reported here: not to the caller's next launch as well */
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

static mk_status attend(mk_attn *at, int32_t layer, const mk_attn_batch *b, const uint32_t *tree,
                        int32_t tree_words, const void *q, int64_t q_token_stride, void *out,
                        float *lse) {
  if (!at || !b) return MK_ERR_INVALID_ARG;
  const mk_attn_desc &d = at->d;
  if (layer < 0 || layer >= d.n_layers || b->n_seqs < 0 || b->n_tokens < 0 || b->n_groups < 0 ||
      b->max_pages_per_seq < 1)
    return MK_ERR_INVALID_ARG;
  if (b->n_seqs > d.max_seqs || b->n_tokens > d.max_tokens || b->n_groups > d.max_groups)
    return MK_ERR_BATCH;
  const int64_t cap = (int64_t)b->max_pages_per_seq * d.page_size;
  if (cap > (1 << 30)) return MK_ERR_UNSUPPORTED;
  /* the line of items is measured in 32 bits */
  const int64_t block = 2 * (kTile / (d.n_q_heads / d.n_kv_heads));
  if ((2 * (b->n_tokens / block) + b->n_seqs + b->n_groups) * d.n_kv_heads *
          ((cap / kTile + 1) * kPairTile + kPairItem) > (1 << 30))
    return MK_ERR_UNSUPPORTED;
  if (b->n_seqs == 0 || b->n_tokens == 0) return MK_OK;
  if (!b->page_tables || !b->seq_lens || !aligned(b->page_tables, 4) || !aligned(b->seq_lens, 4) ||
      !aligned(b->q_offsets, 4) || !aligned(b->group_starts, 4) || !aligned(b->prefix_lens, 4) ||
      (!b->q_offsets && b->n_tokens != b->n_seqs) ||
      (b->n_groups > 0 && (!b->group_starts || !b->prefix_lens)))
    return MK_ERR_INVALID_ARG;
  if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) ||
      q_token_stride < (int64_t)d.n_q_heads * d.head_dim || q_token_stride % 8 ||
      q_token_stride >= (int64_t)1 << 39 /* of a tensor map, in elements */)
    return MK_ERR_INVALID_ARG;
  /* a piece writes its rows while another still reads queries */
  const int64_t row = (int64_t)d.n_q_heads * d.head_dim * 2;
  const int64_t q_bytes = (b->n_tokens - 1) * q_token_stride * 2 + row;
  const int64_t lse_bytes = (int64_t)b->n_tokens * d.n_q_heads * 4;
  if (overlap(q, q_bytes, out, b->n_tokens * row) ||
      (lse && (overlap(q, q_bytes, lse, lse_bytes) || overlap(out, b->n_tokens * row, lse, lse_bytes))))
    return MK_ERR_INVALID_ARG;
  const int64_t tree_bytes = (int64_t)b->n_tokens * tree_words * 4;
  if (tree && (overlap(tree, tree_bytes, out, b->n_tokens * row) ||
               (lse && overlap(tree, tree_bytes, lse, lse_bytes))))
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
  a.out = (__nv_bfloat16 *)out;
  a.lse = lse;
  a.scale_log2 = at->scale_log2;
  a.tree = tree;
  a.tree_words = tree_words;
  a.max_query = tree ? 32 * tree_words : INT32_MAX;
  a.q = (const __nv_bfloat16 *)q;
  a.q_stride = q_token_stride;
  a.k_pool = (const __nv_bfloat16 *)at->pools[2 * layer];
  a.v_pool = (const __nv_bfloat16 *)at->pools[2 * layer + 1];
  a.TB = kTile / a.G;
  a.inv_g = (65536 + a.G - 1) / a.G;
  a.inv_p = ((1ull << 38) + a.P - 1) / a.P;
  a.err_host = at->err_dev;
  a.wait_limit = at->wait_limit;
  a.poison = at->poison;
  a.bad = (int32_t *)at->ws;
  a.error = (int32_t *)at->ws + 1;
  a.where = (int4 *)(at->ws + at->o_where);
  a.part = (float *)(at->ws + at->o_part);
  a.part_ml = (float2 *)(at->ws + at->o_ml);
  CUtensorMap qmap;
  const mk_status st = mk_encode_q_map(&d, q, b->n_tokens, q_token_stride, a.TB, &qmap);
  if (st != MK_OK) return st;
  const cudaError_t e = d.head_dim == 32   ? launch<32>(at, layer, qmap, a)
                        : d.head_dim == 64 ? launch<64>(at, layer, qmap, a)
                                           : launch<128>(at, layer, qmap, a);
  if (e != cudaSuccess) return MK_ERR_CUDA;
  at->poison = false;
  return MK_OK;
}

mk_status mk_prefix_attention(mk_attn *at, int32_t layer, const mk_attn_batch *b, const void *q,
                              int64_t q_token_stride, void *out, float *lse) {
  return attend(at, layer, b, nullptr, 0, q, q_token_stride, out, lse);
}

mk_status mk_tree_attention(mk_attn *at, int32_t layer, const mk_attn_batch *b,
                            const uint32_t *tree, int32_t tree_words, const void *q,
                            int64_t q_token_stride, void *out, float *lse) {
  if (tree_words < 1 || tree_words > (1 << 20) / 32 || !aligned(tree, 4)) return MK_ERR_INVALID_ARG;
  if (!tree && b && b->n_seqs > 0 && b->n_tokens > 0) return MK_ERR_INVALID_ARG;
  return attend(at, layer, b, tree, tree_words, q, q_token_stride, out, lse);
}

mk_status mk_attn_set_wait_limit_ns(mk_attn *at, uint64_t ns) {
  if (!at || ns == 0) return MK_ERR_INVALID_ARG;
  at->wait_limit = ns;
  return MK_OK;
}

mk_status mk_attn_debug_poison_wait(mk_attn *at) {
  if (!at) return MK_ERR_INVALID_ARG;
  at->poison = true;
  return MK_OK;
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
  if (code == 0) return MK_OK;
  *(volatile int32_t *)at->err_host = 0;
  if (cudaMemsetAsync((int32_t *)at->ws + 1, 0, sizeof(int32_t), at->stream) != cudaSuccess)
    return MK_ERR_CUDA;
  return code;
}

}  // extern "C"
