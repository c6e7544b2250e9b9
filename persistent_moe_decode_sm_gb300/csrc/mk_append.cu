/*
 * mk_append.cu -- keys and values of a batch's tokens normed, rotated and written to the pages of
 * their sequences, queries normed and rotated beside them (include/mk_cache.h).
 *
 * A warp takes a token, or some of a token's heads where there are few tokens: 32 lanes of 8 dims
 * hold 256 / head_dim heads at a time, so a lane has the same dims of every head, and turns its
 * cosines and sines once for all of them.  A token's sequence, place, page and position are looked
 * up while the one before it is under way.
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "mk_cache.h"
#include "mk_device.h"

namespace {

using namespace mk_dev;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxSeqs = 1024; /* of a call: offsets and lengths are in shared memory */
constexpr int kBatch = 4;      /* steps whose loads are in flight together */
constexpr int kBlocks = 3;     /* of an SM */

/* Which of a head's dims a lane holds, as four pairs (a, b): PAIR_HALVES 4 dims and the 4 half the
 * rotary part further on (rotary_dim a multiple of 8), PAIR_NEIGHBOURS 8 dims in a row, PAIR_ANY any
 * halves, to which 8 dims in a row are exchanged through shared memory (25400 tokens with 100 of 128
 * dims turned and norms: 130 us, loaded and stored one by one 319).  A lane turns an angle once for all
 * heads of its part of a token. */
enum { PAIR_HALVES = 0, PAIR_NEIGHBOURS = 1, PAIR_ANY = 2 };

struct Args {
  int32_t Hq, Hkv, P, M, num_pages, n_seqs, n_tokens, R;
  int32_t q_steps, kv_steps, parts, steps; /* warp's steps of a token's q, of k or v; parts of a token; steps a part */
  const int32_t *tables, *lens, *off, *positions;
  const uint64_t *turns; /* [64] turns a position of each pair, in 2^-64; 0 behind the rotary part */
  const __nv_bfloat16 *q, *k, *v, *q_norm, *k_norm;
  __nv_bfloat16 *q_out, *k_pool, *v_pool;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  float magnitude, eps;
  Errors err;
};

/* cos and sin of 2 pi position F / 2^64: the product mod 1 is exact; of its first 32 bits the
 * nearest quarter turn is taken off in integers, and the rest, within pi / 4, goes through the Taylor
 * series (next terms: x^11 / 11! below 2e-9, x^12 / 12! below 2e-10). */
__device__ __forceinline__ void turn(uint32_t position, uint64_t F, float *c, float *s) {
  const uint32_t u = (uint32_t)((F * position) >> 32), quarter = (u + (1u << 29)) >> 30;
  const float x = (float)(int32_t)(u - (quarter << 30)) * 1.46291807927e-9f; /* 2 pi / 2^32 */
  const float y = x * x;
  float sn = fmaf(y, 2.755731922e-6f, -1.984126984e-4f); /* 1 / 9!, 1 / 7! */
  sn = fmaf(sn, y, 8.333333333e-3f);
  sn = fmaf(sn, y, -1.666666667e-1f);
  sn = fmaf(sn * y, x, x);
  float cs = fmaf(y, -2.755731922e-7f, 2.480158730e-5f); /* 1 / 10!, 1 / 8! */
  cs = fmaf(cs, y, -1.388888889e-3f);
  cs = fmaf(cs, y, 4.166666667e-2f);
  cs = fmaf(cs, y, -0.5f);
  cs = fmaf(cs, y, 1.0f);
  const bool swap = quarter & 1;
  const float a = swap ? sn : cs, b = swap ? cs : sn;
  *c = ((quarter + 1) & 2) ? -a : a; /* quarters 1 and 2 */
  *s = (quarter & 2) ? -b : b;       /* quarters 2 and 3 */
}

__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

/* A lane's 8 dims of a head of D. */
template <int D, int PAIR>
struct Dims {
  int l, half, oa, ob; /* lane of the head; first dims of the two pieces */
  __device__ Dims(int lane, int R) : l(lane % (D / 8)), half(R >> 1) {
    const bool turns = 8 * l < R;
    oa = PAIR == PAIR_HALVES && turns ? 4 * l : 8 * l;
    ob = PAIR == PAIR_HALVES && turns ? 4 * l + half : 8 * l + 4;
  }
  /* the dims of pair k; pairs behind the rotary part are neighbours */
  __device__ __forceinline__ int a(int k) const {
    const int p = 4 * l + k;
    if (PAIR == PAIR_HALVES) return oa + k;
    return PAIR == PAIR_ANY && p < half ? p : 2 * p;
  }
  __device__ __forceinline__ int b(int k) const {
    const int p = 4 * l + k;
    if (PAIR == PAIR_HALVES) return ob + k;
    return PAIR == PAIR_ANY && p < half ? p + half : 2 * p + 1;
  }
  __device__ __forceinline__ bool turns(int k) const {
    return PAIR == PAIR_HALVES ? 8 * l < 2 * half : 4 * l + k < half;
  }
  __device__ __forceinline__ uint4 load(const __nv_bfloat16 *head) const {
    if constexpr (PAIR == PAIR_NEIGHBOURS) return __ldcg((const uint4 *)(head + oa));
    if constexpr (PAIR == PAIR_HALVES) {
      const uint2 x = __ldcg((const uint2 *)(head + oa)), y = __ldcg((const uint2 *)(head + ob));
      return make_uint4(x.x, x.y, y.x, y.y);
    }
    if constexpr (PAIR == PAIR_ANY) return __ldcg((const uint4 *)(head + 8 * l)); /* not pairs yet */
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *head, const uint4 &v) const {
    if (PAIR == PAIR_HALVES) {
      *(uint2 *)(head + oa) = make_uint2(v.x, v.y);
      *(uint2 *)(head + ob) = make_uint2(v.z, v.w);
    } else {
      *(uint4 *)(head + 8 * l) = v;
    }
  }
  /* PAIR_ANY: 8 dims in a row to pairs and back, by whole warps, through `mine`, the head's place in
   * shared memory. */
  __device__ __forceinline__ uint4 to_pairs(const uint4 &v, unsigned short *mine) const {
    __syncwarp();
    *(uint4 *)(mine + 8 * l) = v;
    __syncwarp();
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = mine[a(k)] | (uint32_t)mine[b(k)] << 16;
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ uint4 from_pairs(const uint4 &v, unsigned short *mine) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      mine[a(k)] = (unsigned short)w[k];
      mine[b(k)] = (unsigned short)(w[k] >> 16);
    }
    __syncwarp();
    return *(const uint4 *)(mine + 8 * l);
  }
  __device__ __forceinline__ void unpack(const uint4 &v, float *xa, float *xb) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (PAIR == PAIR_HALVES) {
        xa[k] = k & 1 ? high(w[k / 2]) : low(w[k / 2]);
        xb[k] = k & 1 ? high(w[2 + k / 2]) : low(w[2 + k / 2]);
      } else {
        xa[k] = low(w[k]);
        xb[k] = high(w[k]);
      }
    }
  }
  __device__ __forceinline__ uint4 packed(const float *xa, const float *xb) const {
    if (PAIR == PAIR_HALVES)
      return make_uint4(pack(xa[0], xa[1]), pack(xa[2], xa[3]), pack(xb[0], xb[1]), pack(xb[2], xb[3]));
    return make_uint4(pack(xa[0], xb[0]), pack(xa[1], xb[1]), pack(xa[2], xb[2]), pack(xa[3], xb[3]));
  }
};

/* NORM_SOME: heads whose mean square is below 2^121, with an eps that keeps the root's argument away from
 * 2^-126; NORM_ANY, taken where eps is below 2^-100: heads of any size.  It looks at each mean, which costs
 * 25400 tokens 2.5 us (90.9, so 88.4). */
enum { NORM_NONE = 0, NORM_SOME = 1, NORM_ANY = 2 };

/* A lane's part of what is done to a head: a' = f (a ca + b sb), b' = f (b cb + a sa), with f the
 * norm's factor, and the gains in the rest. */
template <int D, int PAIR, int NORM>
struct Turn {
  float ca[4], cb[4], sa[4], sb[4];
  float eps;
  bool normed;
  __device__ __forceinline__ void set(const Dims<D, PAIR> &dims, const float *cs, const float *sn, const uint4 &gain,
                                      bool normed_, float eps_) {
    float ga[4] = {1.0f, 1.0f, 1.0f, 1.0f}, gb[4] = {1.0f, 1.0f, 1.0f, 1.0f};
    if (NORM) dims.unpack(gain, ga, gb);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      ca[k] = cs[k] * ga[k];
      cb[k] = cs[k] * gb[k];
      sa[k] = sn[k] * ga[k];
      sb[k] = -sn[k] * gb[k];
    }
    normed = normed_;
    eps = eps_;
  }
  /* of a head, which D / 8 lanes hold */
  __device__ __forceinline__ static float mean_square(const float *xa, const float *xb) {
    float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      ss = __ffma2_rn(make_float2(xa[j], xa[j + 1]), make_float2(xa[j], xa[j + 1]), ss);
      ss = __ffma2_rn(make_float2(xb[j], xb[j + 1]), make_float2(xb[j], xb[j + 1]), ss);
    }
    float f = ss.x + ss.y;
#pragma unroll
    for (int o = 1; o < D / 8; o *= 2) f += __shfl_xor_sync(0xffffffffu, f, o);
    return f * (1.0f / D);
  }
  __device__ __forceinline__ uint4 operator()(const Dims<D, PAIR> &dims, const uint4 &v) const {
    float xa[4], xb[4], f = 1.0f;
    dims.unpack(v, xa, xb);
    if (NORM && normed) {
      const float mean = mean_square(xa, xb) + eps;
      f = rsqrtf(mean);
      if (NORM == NORM_ANY) {
        /* squares near the ends of 32 bits: the head times a power of two, and eps times its square */
        const bool few = mean < 0x1p-100f, many = !(mean < 0x1p100f);
        if (__any_sync(0xffffffffu, few || many)) {
          const float s = few ? 0x1p100f : many ? 0x1p-68f : 1.0f;
#pragma unroll
          for (int j = 0; j < 4; ++j) xa[j] *= s, xb[j] *= s;
          f = rsqrtf(mean_square(xa, xb) + eps * s * s);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const float2 a = make_float2(xa[j], xa[j + 1]), b = make_float2(xb[j], xb[j + 1]);
      float2 y0 = __fmul2_rn(a, make_float2(ca[j], ca[j + 1])), y1 = __fmul2_rn(b, make_float2(cb[j], cb[j + 1]));
      /* an infinity beside a dim that does not turn stays there */
      if (PAIR == PAIR_HALVES) {
        if (dims.turns(0)) {
          y0 = __ffma2_rn(b, make_float2(sb[j], sb[j + 1]), y0);
          y1 = __ffma2_rn(a, make_float2(sa[j], sa[j + 1]), y1);
        }
      } else {
        if (dims.turns(j)) y0.x = fmaf(b.x, sb[j], y0.x), y1.x = fmaf(a.x, sa[j], y1.x);
        if (dims.turns(j + 1)) y0.y = fmaf(b.y, sb[j + 1], y0.y), y1.y = fmaf(a.y, sa[j + 1], y1.y);
      }
      if (NORM) {
        y0 = __fmul2_rn(y0, make_float2(f, f));
        y1 = __fmul2_rn(y1, make_float2(f, f));
      }
      xa[j] = y0.x, xa[j + 1] = y0.y;
      xb[j] = y1.x, xb[j + 1] = y1.y;
    }
    return dims.packed(xa, xb);
  }
};

/* n steps of a warp over heads that lie src_step and dst_step apart; this lane has a head in the
 * first `mine` of them. */
template <int D, int PAIR, class F>
__device__ __forceinline__ void heads(const Dims<D, PAIR> &dims, int n, int mine, const __nv_bfloat16 *src, int src_step,
                                      __nv_bfloat16 *dst, long long dst_step, F f) {
#pragma unroll 1
  for (; n > 0; n -= kBatch, mine -= kBatch) {
    uint4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      v[k] = make_uint4(0, 0, 0, 0);
      if (k < mine) v[k] = dims.load(src + k * src_step);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (k >= n) break;
      v[k] = f(v[k]);
      if (k < mine) dims.store(dst + k * dst_step, v[k]);
    }
    src += kBatch * src_step;
    dst += kBatch * dst_step;
  }
}

/* A token's place, position and page; the last two may be on their way. */
struct Where {
  int place, position, page;
};

/* q' and k' = turn(norm(x)), v, each row read and written once.  25400 tokens of 32 + 2 x 4 heads of 128
 * with norms, 520 MB, take 88 us, 5.9 TB/s, 87 % of a plain copy, with 24 warps an SM (102 with 16, 104
 * with 32; copies to shared memory several steps ahead instead of loads to registers: 94).  Eight
 * single tokens take 2.9 us, a chain of loads: offsets and lengths, tables and positions, rows. */
template <int D, int PAIR, int NORM>
__global__ void __launch_bounds__(kThreads, kBlocks) append_tokens(const __grid_constant__ Args a) {
  constexpr int LPH = D / 8, HPW = 32 / LPH; /* lanes of a head, heads of a warp's step */
  __shared__ int s_off[kMaxSeqs + 1], s_len[kMaxSeqs];
  __shared__ __align__(16) unsigned short s_pairs[PAIR == PAIR_ANY ? kWarps : 1][PAIR == PAIR_ANY ? 256 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hl = lane / LPH;
  const Dims<D, PAIR> dims(lane, a.R);

  /* From here on what the grid before wrote is read, through L2: its blocks may have left older
   * lines in this SM's L1. */
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  bool bad = false;
  for (int i = tid; i <= a.n_seqs; i += kThreads) {
    const int o = a.off ? __ldcg(a.off + i) : i;
    bad |= (i == 0 && o != 0) || (i == a.n_seqs && o > a.n_tokens);
    s_off[i] = o;
    if (i < a.n_seqs) {
      const int next = a.off ? __ldcg(a.off + i + 1) : i + 1, l = __ldcg(a.lens + i);
      bad |= next < o || l < 0 || l > (long long)a.M * a.P;
      s_len[i] = l;
    }
  }
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  unsigned short *const s_head = s_pairs[PAIR == PAIR_ANY ? warp : 0] + hl * D;
  auto in_pairs = [&](const uint4 &v) { return PAIR == PAIR_ANY ? dims.to_pairs(v, s_head) : v; };
  auto in_rows = [&](const uint4 &v) { return PAIR == PAIR_ANY ? dims.from_pairs(v, s_head) : v; };
  const uint4 gq = NORM && a.q_norm ? in_pairs(dims.load(a.q_norm)) : ones;
  const uint4 gk = NORM && a.k_norm ? in_pairs(dims.load(a.k_norm)) : ones;
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && tid == 0) report(a.err, MK_ERR_INVALID_ARG);
    return;
  }
  const unsigned items = (unsigned)s_off[a.n_seqs] * a.parts;
  auto look_up = [&](unsigned item) {
    Where w{-1, 0, -1};
    if (item >= items) return w;
    const int tok = (int)(item / a.parts);
    int lo = 0, hi = a.n_seqs - 1; /* the last sequence that begins at or before it */
    if (a.off) {
      while (lo < hi) {
        const int m = (lo + hi + 1) >> 1;
        if (s_off[m] <= tok)
          lo = m;
        else
          hi = m - 1;
      }
    } else {
      lo = tok;
    }
    w.place = s_len[lo] - (s_off[lo + 1] - tok);
    w.position = a.positions ? __ldcg(a.positions + tok) : w.place;
    if (w.place >= 0) w.page = __ldcg(a.tables + (size_t)lo * a.M + w.place / a.P);
    return w;
  };
  unsigned item = blockIdx.x * kWarps + warp;
  Where next = look_up(item);
  for (; item < items; item += gridDim.x * kWarps) {
    const int tok = (int)(item / a.parts), part = (int)(item - (unsigned)tok * a.parts);
    const int first = part * a.steps, last = first + a.steps; /* of the steps of q, then k, then v */
    const Where w = next;
    next = look_up(item + gridDim.x * kWarps);
    if (w.place < 0) continue;
    if (w.position < 0) {
      if (lane == 0) report(a.err, MK_ERR_INVALID_ARG);
      continue;
    }
    Turn<D, PAIR, NORM> turned;
    float cs[4], sn[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      turn((uint32_t)w.position, __ldg(a.turns + 4 * dims.l + k), &cs[k], &sn[k]);
      cs[k] = dims.turns(k) ? cs[k] * a.magnitude : 1.0f;
      sn[k] *= a.magnitude;
    }
    auto share = [&](int before, int all, int n_heads, int *i0, int *mine) { /* this item's of `all` steps */
      *i0 = max(0, first - before);
      const int n = min(all, last - before) - *i0;
      *mine = min(n, (n_heads - hl + HPW - 1) / HPW - *i0);
      return n;
    };
    int i0, mine, n = share(0, a.q_steps, a.Hq, &i0, &mine);
    if (n > 0) {
      turned.set(dims, cs, sn, gq, NORM && a.q_norm, a.eps);
      const int h = i0 * HPW + hl;
      heads<D, PAIR>(dims, n, mine, a.q + tok * a.q_stride + h * D, HPW * D, a.q_out + tok * a.q_out_stride + h * D,
                     HPW * D, [&](const uint4 &v) { return in_rows(turned(dims, in_pairs(v))); });
    }
    if (last <= a.q_steps) continue;
    if ((unsigned)w.page >= (unsigned)a.num_pages) {
      if (lane == 0) report(a.err, MK_ERR_PAGE_OOB);
      continue;
    }
    const long long row = (long long)a.P * D; /* from a head of a page to the next */
    const long long at = (long long)w.page * a.Hkv * row + (long long)(w.place % a.P) * D;
    n = share(a.q_steps, a.kv_steps, a.Hkv, &i0, &mine);
    if (n > 0) {
      turned.set(dims, cs, sn, gk, NORM && a.k_norm, a.eps);
      const int h = i0 * HPW + hl;
      heads<D, PAIR>(dims, n, mine, a.k + tok * a.k_stride + h * D, HPW * D, a.k_pool + at + h * row, HPW * row,
                     [&](const uint4 &v) { return in_rows(turned(dims, in_pairs(v))); });
    }
    n = share(a.q_steps + a.kv_steps, a.kv_steps, a.Hkv, &i0, &mine);
    if (n > 0) {
      const int h = i0 * HPW + hl;
      heads<D, PAIR>(dims, n, mine, a.v + tok * a.v_stride + h * D, HPW * D, a.v_pool + at + h * row, HPW * row,
                     [&](const uint4 &v) { return v; });
    }
  }
}

}  // namespace

struct mk_append {
  mk_append_desc d{};
  std::vector<void *> k, v; /* pools of each layer */
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0, pair = 0;
  uint8_t *ws = nullptr; /* the error word, then the turns */
  Errors err{};
  int32_t *err_host = nullptr;
};

namespace {

template <int D, int PAIR>
cudaError_t launch(const cudaLaunchConfig_t &cfg, const Args &a) {
  if (!a.q_norm && !a.k_norm) return cudaLaunchKernelEx(&cfg, append_tokens<D, PAIR, NORM_NONE>, a);
  return a.eps < 0x1p-100f ? cudaLaunchKernelEx(&cfg, append_tokens<D, PAIR, NORM_ANY>, a)
                           : cudaLaunchKernelEx(&cfg, append_tokens<D, PAIR, NORM_SOME>, a);
}
template <int D>
cudaError_t launch(const mk_append *app, const cudaLaunchConfig_t &cfg, const Args &a) {
  return app->pair == PAIR_HALVES       ? launch<D, PAIR_HALVES>(cfg, a)
         : app->pair == PAIR_NEIGHBOURS ? launch<D, PAIR_NEIGHBOURS>(cfg, a)
                                        : launch<D, PAIR_ANY>(cfg, a);
}

}  // namespace

extern "C" {

mk_status mk_append_create(const mk_append_desc *d, void *stream, mk_append **out) {
  if (!d || !out) return MK_ERR_INVALID_ARG;
  if (d->n_q_heads < 0 || d->n_kv_heads < 1 || d->head_dim < 1 || d->page_size < 1 ||
      d->num_pages < 1 || d->n_layers < 1 || d->rotary_dim < 0 || d->rotary_dim % 2 ||
      d->rotary_dim > d->head_dim || !(d->magnitude >= 0.0f) || !std::isfinite(d->magnitude) ||
      !(d->norm_eps >= 0.0f) || !std::isfinite(d->norm_eps))
    return MK_ERR_INVALID_ARG;
  if ((d->head_dim != 32 && d->head_dim != 64 && d->head_dim != 128) || d->n_q_heads > 1024 ||
      d->n_kv_heads > 1024)
    return MK_ERR_UNSUPPORTED;
  if (!d->k_caches || !d->v_caches) return MK_ERR_INVALID_ARG;
  for (int l = 0; l < d->n_layers; ++l)
    if (!d->k_caches[l] || !d->v_caches[l] || !aligned(d->k_caches[l], 16) ||
        !aligned(d->v_caches[l], 16))
      return MK_ERR_INVALID_ARG;
  if (d->rotary_dim && !d->frequencies && !(d->rope_base > 0.0f && std::isfinite(d->rope_base)))
    return MK_ERR_INVALID_ARG;
  for (int i = 0; d->frequencies && i < d->rotary_dim / 2; ++i)
    if (!std::isfinite(d->frequencies[i])) return MK_ERR_INVALID_ARG;
  int dev = 0, n_sm = 0;
  if (!this_device(&dev, &n_sm)) return MK_ERR_NO_DEVICE;
  mk_append *app = new (std::nothrow) mk_append();
  if (!app) return MK_ERR_CUDA;
  app->d = *d;
  app->d.k_caches = app->d.v_caches = nullptr;
  app->d.frequencies = nullptr;
  if (app->d.magnitude == 0.0f) app->d.magnitude = 1.0f;
  app->stream = (cudaStream_t)stream;
  app->dev = dev;
  app->n_sm = n_sm;
  app->pair = d->interleaved || !d->rotary_dim ? PAIR_NEIGHBOURS : d->rotary_dim % 8 ? PAIR_ANY : PAIR_HALVES;
  uint64_t turns[64] = {};
  try {
    app->k.assign(d->k_caches, d->k_caches + d->n_layers);
    app->v.assign(d->v_caches, d->v_caches + d->n_layers);
  } catch (...) {
    delete app;
    return MK_ERR_CUDA;
  }
  for (int i = 0; i < d->rotary_dim / 2; ++i) {
    const double f = d->frequencies ? d->frequencies[i] : std::pow((double)d->rope_base, -2.0 * i / d->rotary_dim);
    const long double t = (long double)f / 6.283185307179586476925286766559L, part = t - std::floor(t);
    turns[i] = part < 1.0L ? (uint64_t)std::ldexp(part, 64) : 0;
  }
  cudaError_t e = cudaMalloc(&app->ws, 64 + sizeof(turns));
  if (e == cudaSuccess) e = cudaMemsetAsync(app->ws, 0, 64, app->stream);
  if (e == cudaSuccess)
    e = cudaMemcpyAsync(app->ws + 64, turns, sizeof(turns), cudaMemcpyHostToDevice, app->stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(app->stream);
  if (e == cudaSuccess) e = cudaHostAlloc(&app->err_host, 64, cudaHostAllocMapped);
  if (e == cudaSuccess) {
    std::memset(app->err_host, 0, 64);
    app->err.first = (int32_t *)app->ws;
    e = cudaHostGetDevicePointer((void **)&app->err.host, app->err_host, 0);
  }
  if (e != cudaSuccess) {
    mk_append_destroy(app);
    cudaGetLastError(); /* reported here: not to the caller's next launch as well */
    return MK_ERR_CUDA;
  }
  *out = app;
  return MK_OK;
}

void mk_append_destroy(mk_append *app) {
  if (!app) return;
  {
    OnDevice on(app->dev);
    cudaStreamSynchronize(app->stream);
    if (app->ws) cudaFree(app->ws);
    if (app->err_host) cudaFreeHost(app->err_host);
  }
  delete app;
}

mk_status mk_append_tokens(mk_append *app, int32_t layer, const mk_attn_batch *b,
                           const mk_append_rows *r) {
  if (!app || !b || !r) return MK_ERR_INVALID_ARG;
  const mk_append_desc &d = app->d;
  if (layer < 0 || layer >= d.n_layers || b->n_seqs < 0 || b->n_tokens < 0 || b->max_pages_per_seq < 1)
    return MK_ERR_INVALID_ARG;
  if (b->n_seqs > kMaxSeqs) return MK_ERR_BATCH;
  if ((int64_t)b->max_pages_per_seq * d.page_size > INT32_MAX) return MK_ERR_UNSUPPORTED;
  const int64_t wq = (int64_t)d.n_q_heads * d.head_dim, wkv = (int64_t)d.n_kv_heads * d.head_dim;
  const bool with_q = r->q != nullptr;
  /* items are counted in 32 bits: heads a token, one a warp at least */
  if ((int64_t)b->n_tokens * (d.n_q_heads + 2 * d.n_kv_heads) > INT32_MAX) return MK_ERR_UNSUPPORTED;
  if (b->n_seqs == 0 || b->n_tokens == 0) return MK_OK;
  if (!b->page_tables || !b->seq_lens || !aligned(b->page_tables, 4) || !aligned(b->seq_lens, 4) ||
      !aligned(b->q_offsets, 4) || (!b->q_offsets && b->n_tokens != b->n_seqs) ||
      !aligned(r->positions, 4))
    return MK_ERR_INVALID_ARG;
  if (with_q != (r->q_out != nullptr) || (with_q && d.n_q_heads == 0) || !r->k || !r->v ||
      !aligned(r->q, 16) || !aligned(r->k, 16) || !aligned(r->v, 16) || !aligned(r->q_out, 16) ||
      !aligned(r->q_norm, 16) || !aligned(r->k_norm, 16))
    return MK_ERR_INVALID_ARG;
  const int64_t longest = (int64_t)1 << 39; /* of a stride: offsets stay within 63 bits */
  if (r->k_stride < wkv || r->v_stride < wkv || r->k_stride % 8 || r->v_stride % 8 ||
      r->k_stride >= longest || r->v_stride >= longest ||
      (with_q && (r->q_stride < wq || r->q_out_stride < wq || r->q_stride % 8 || r->q_out_stride % 8 ||
                  r->q_stride >= longest || r->q_out_stride >= longest)))
    return MK_ERR_INVALID_ARG;
  if (with_q) {
    const int64_t n = b->n_tokens, so = 2 * r->q_out_stride;
    const bool in_place = r->q == r->q_out && (n == 1 || r->q_stride == r->q_out_stride);
    if ((!in_place && rows_meet(r->q, 2 * r->q_stride, 2 * wq, r->q_out, so, 2 * wq, n)) ||
        rows_meet(r->k, 2 * r->k_stride, 2 * wkv, r->q_out, so, 2 * wq, n) ||
        rows_meet(r->v, 2 * r->v_stride, 2 * wkv, r->q_out, so, 2 * wq, n))
      return MK_ERR_INVALID_ARG;
  }
  OnDevice on(app->dev);
  if (!on.ok) return MK_ERR_CUDA;
  Args a{};
  a.Hq = with_q ? d.n_q_heads : 0;
  a.Hkv = d.n_kv_heads;
  a.P = d.page_size;
  a.M = b->max_pages_per_seq;
  a.num_pages = d.num_pages;
  a.n_seqs = b->n_seqs;
  a.n_tokens = b->n_tokens;
  a.R = d.rotary_dim;
  a.tables = b->page_tables;
  a.lens = b->seq_lens;
  a.off = b->q_offsets;
  a.positions = r->positions;
  a.turns = (const uint64_t *)(app->ws + 64);
  a.q = (const __nv_bfloat16 *)r->q;
  a.k = (const __nv_bfloat16 *)r->k;
  a.v = (const __nv_bfloat16 *)r->v;
  a.q_norm = with_q ? (const __nv_bfloat16 *)r->q_norm : nullptr;
  a.k_norm = (const __nv_bfloat16 *)r->k_norm;
  a.q_out = (__nv_bfloat16 *)r->q_out;
  a.k_pool = (__nv_bfloat16 *)app->k[layer];
  a.v_pool = (__nv_bfloat16 *)app->v[layer];
  a.q_stride = r->q_stride;
  a.k_stride = r->k_stride;
  a.v_stride = r->v_stride;
  a.q_out_stride = r->q_out_stride;
  a.magnitude = d.magnitude;
  a.eps = d.norm_eps;
  a.err = app->err;
  /* parts of a token: as many as make 4 warps an SM, each of one step at least (1160 tokens of 16 + 2 x 4
   * heads of 64: 3.9 us whole, 4.6 in parts for 8 warps an SM) */
  const int heads = 256 / d.head_dim; /* of a step */
  a.q_steps = (a.Hq + heads - 1) / heads;
  a.kv_steps = (a.Hkv + heads - 1) / heads;
  const int steps = a.q_steps + 2 * a.kv_steps;
  const int64_t want = ((int64_t)app->n_sm * 4 + b->n_tokens - 1) / b->n_tokens;
  a.steps = (int)std::max<int64_t>(1, steps / std::min<int64_t>(steps, want));
  a.parts = (steps + a.steps - 1) / a.steps;
  const int64_t blocks = ((int64_t)b->n_tokens * a.parts + kWarps - 1) / kWarps;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(blocks, app->n_sm * kBlocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = app->stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = d.head_dim == 32   ? launch<32>(app, cfg, a)
                        : d.head_dim == 64 ? launch<64>(app, cfg, a)
                                           : launch<128>(app, cfg, a);
  return e == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_append_sync(mk_append *app) {
  return app ? take_error(app->dev, app->stream, app->err, app->err_host) : MK_ERR_INVALID_ARG;
}

}  // extern "C"
