/*
 * mk_append.cu -- keys and values of a batch's tokens normed, rotated and written to the pages of
 * their sequences, queries normed and rotated beside them (include/mk_cache.h).
 *
 * A warp takes a token, or some of a token's heads where there are few tokens: 32 lanes of 8 dims
 * hold 256 / head_dim heads at a time, so a lane has the same dims of every head, and turns its
 * cosines and sines once for all of them.  The token's sequence, place, page and angle are looked
 * up while its first heads are on their way.
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
constexpr int kBatch = 4;      /* 16-byte loads in flight a lane */

/* How a dim finds its partner: in the same lane, in a lane some way on, or anywhere. */
enum { PAIR_INSIDE = 0, PAIR_LANES = 1, PAIR_ANY = 2 };

struct Args {
  int32_t Hq, Hkv, P, M, num_pages, n_seqs, n_tokens, R;
  int32_t rows, parts, steps; /* heads of a token (q, k, v); parts of a token; steps a part */
  const int32_t *tables, *lens, *off, *positions;
  const uint64_t *turns; /* [R / 2] turns a position, in 2^-64 */
  const __nv_bfloat16 *q, *k, *v, *q_norm, *k_norm;
  __nv_bfloat16 *q_out, *k_pool, *v_pool;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  float magnitude, eps;
  Errors err;
};

/* cos and sin of 2 pi position F / 2^64: the product mod 1 is exact, the nearest quarter turn is
 * taken off in integers, and the rest, within pi / 4, goes through the Taylor series (next terms:
 * x^11 / 11! below 2e-9, x^12 / 12! below 2e-10). */
__device__ __forceinline__ void turn(uint32_t position, uint64_t F, float *c, float *s) {
  const uint64_t u = F * position;
  const uint64_t quarter = (u + (1ull << 61)) >> 62;
  const float x = __ll2float_rn((long long)(u - (quarter << 62))) * 3.4061215800304e-19f; /* 2 pi / 2^64 */
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

__device__ __forceinline__ void unpack8(const uint4 &w, float *x) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(v[i] << 16);
    x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float *x) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

template <int D, int PAIR>
__global__ void __launch_bounds__(kThreads) append_tokens(const __grid_constant__ Args a) {
  constexpr int LPH = D / 8, HPW = 32 / LPH; /* lanes of a head, heads of a warp's step */
  __shared__ int s_off[kMaxSeqs + 1], s_len[kMaxSeqs];
  __shared__ float s_any[PAIR == PAIR_ANY ? kWarps : 1][PAIR == PAIR_ANY ? 32 * 8 : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int hl = lane / LPH, d0 = lane % LPH * 8, half = a.R >> 1;

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
  if (__syncthreads_or(bad)) {
    if (blockIdx.x == 0 && tid == 0) report(a.err, MK_ERR_INVALID_ARG);
    return;
  }
  const int tokens = s_off[a.n_seqs];
  const unsigned items = (unsigned)tokens * a.parts;
  for (unsigned item = blockIdx.x * kWarps + warp; item < items; item += gridDim.x * kWarps) {
    const int tok = (int)(item / a.parts), part = (int)(item - (unsigned)tok * a.parts);
    const int row0 = part * a.steps * HPW, row1 = min(a.rows, row0 + a.steps * HPW);
    auto source = [&](int r) -> const uint4 * {
      const __nv_bfloat16 *p = r < a.Hq           ? a.q + tok * a.q_stride + r * D
                               : r < a.Hq + a.Hkv ? a.k + tok * a.k_stride + (r - a.Hq) * D
                                                  : a.v + tok * a.v_stride + (r - a.Hq - a.Hkv) * D;
      return (const uint4 *)(p + d0);
    };
    uint4 raw[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = row0 + k * HPW + hl;
      raw[k] = make_uint4(0, 0, 0, 0);
      if (r < row1) raw[k] = __ldcg(source(r));
    }
    /* whose token it is, its place and page */
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
    const int place = s_len[lo] - (s_off[lo + 1] - tok);
    const int position = a.positions ? __ldcg(a.positions + tok) : place;
    if (place < 0) continue;
    if (position < 0) {
      if (lane == 0) report(a.err, MK_ERR_INVALID_ARG);
      continue;
    }
    long long at = -1; /* first element of the token's first K or V head in the pools */
    if (row1 > a.Hq) {
      const int page = __ldcg(a.tables + (size_t)lo * a.M + place / a.P);
      if ((unsigned)page < (unsigned)a.num_pages)
        at = ((long long)page * a.Hkv * a.P + place % a.P) * D;
      else if (lane == 0)
        report(a.err, MK_ERR_PAGE_OOB);
    }
    /* this lane's cosines, and sines with the sign of their dim; 1 and 0 behind the rotary part */
    constexpr int NP = PAIR == PAIR_INSIDE ? 4 : 8;
    float cs[NP], sn[NP];
    if (row0 < a.Hq + a.Hkv) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int d = PAIR == PAIR_INSIDE ? d0 + 2 * i : d0 + i;
        cs[i] = 1.0f;
        sn[i] = 0.0f;
        if (d < a.R) {
          const int pair = PAIR == PAIR_INSIDE ? d >> 1 : d < half ? d : d - half;
          turn((uint32_t)position, a.turns[pair], &cs[i], &sn[i]);
          cs[i] *= a.magnitude;
          sn[i] *= PAIR != PAIR_INSIDE && d < half ? -a.magnitude : a.magnitude;
        }
      }
    }
    for (int r0 = row0; r0 < row1; r0 += kBatch * HPW) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = r0 + k * HPW + hl;
        if (r0 + k * HPW >= row1) break;
        const bool is_q = r < a.Hq, turned = r < a.Hq + a.Hkv;
        uint4 w = raw[k];
        if (r0 + k * HPW < a.Hq + a.Hkv) { /* by whole warps: some of its heads are */
          float x[8], y[8];
          unpack8(w, x);
          const __nv_bfloat16 *gain = is_q ? a.q_norm : a.k_norm;
          if (a.q_norm || a.k_norm) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = 1; o < LPH; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (gain && turned) {
              float g[8];
              unpack8(*(const uint4 *)(gain + d0), g);
              const float f = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = x[i] * f * g[i];
            }
          }
          if (PAIR == PAIR_INSIDE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool on = d0 + 2 * i < a.R;
              y[2 * i] = on ? __fmul_rn(x[2 * i], cs[i]) - __fmul_rn(x[2 * i + 1], sn[i]) : x[2 * i];
              y[2 * i + 1] = on ? __fmul_rn(x[2 * i + 1], cs[i]) + __fmul_rn(x[2 * i], sn[i]) : x[2 * i + 1];
            }
          } else if (PAIR == PAIR_LANES) {
            const int dist = half >> 3, l = lane % LPH;
            const int from = lane + (l < dist ? dist : l < 2 * dist ? -dist : 0);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p = __shfl_sync(0xffffffffu, x[i], from);
              y[i] = d0 < a.R ? __fmul_rn(x[i], cs[i]) + __fmul_rn(p, sn[i]) : x[i];
            }
          } else {
            float *mine = s_any[warp] + hl * D;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[d0 + i] = x[i];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int d = d0 + i;
              y[i] = x[i];
              if (d < a.R)
                y[i] = __fmul_rn(x[i], cs[i]) + __fmul_rn(mine[d < half ? d + half : d - half], sn[i]);
            }
          }
          if (turned) w = pack8(y);
        }
        if (r >= row1) continue;
        if (is_q)
          *(uint4 *)(a.q_out + tok * a.q_out_stride + r * D + d0) = w;
        else if (at >= 0)
          *(uint4 *)((turned ? a.k_pool : a.v_pool) + at +
                     (long long)(turned ? r - a.Hq : r - a.Hq - a.Hkv) * a.P * D + d0) = w;
      }
      if (r0 + kBatch * HPW < row1) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int r = r0 + (kBatch + k) * HPW + hl;
          if (r < row1) raw[k] = __ldcg(source(r));
        }
      }
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

template <int D>
cudaError_t launch(const mk_append *app, const cudaLaunchConfig_t &cfg, const Args &a) {
  return app->pair == PAIR_INSIDE  ? cudaLaunchKernelEx(&cfg, append_tokens<D, PAIR_INSIDE>, a)
         : app->pair == PAIR_LANES ? cudaLaunchKernelEx(&cfg, append_tokens<D, PAIR_LANES>, a)
                                   : cudaLaunchKernelEx(&cfg, append_tokens<D, PAIR_ANY>, a);
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
  app->pair = d->interleaved || !d->rotary_dim ? PAIR_INSIDE : d->rotary_dim % 16 ? PAIR_ANY : PAIR_LANES;
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
  a.rows = a.Hq + 2 * a.Hkv;
  a.tables = b->page_tables;
  a.lens = b->seq_lens;
  a.off = b->q_offsets;
  a.positions = r->positions;
  a.turns = (const uint64_t *)(app->ws + 64);
  a.q = (const __nv_bfloat16 *)r->q;
  a.k = (const __nv_bfloat16 *)r->k;
  a.v = (const __nv_bfloat16 *)r->v;
  a.q_norm = (const __nv_bfloat16 *)r->q_norm;
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
  /* parts of a token: as many as make 8 warps an SM, each of one step at least */
  const int steps = (a.rows + 256 / d.head_dim - 1) / (256 / d.head_dim);
  const int64_t want = ((int64_t)app->n_sm * 8 + b->n_tokens - 1) / b->n_tokens;
  a.steps = (int)std::max<int64_t>(1, steps / std::min<int64_t>(steps, want));
  a.parts = (steps + a.steps - 1) / a.steps;
  const int64_t blocks = ((int64_t)b->n_tokens * a.parts + kWarps - 1) / kWarps;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(blocks, app->n_sm * 4));
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
