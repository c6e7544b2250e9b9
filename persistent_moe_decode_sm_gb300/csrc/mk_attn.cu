/*
 * mk_attn.cu -- attention of a batch over paged K and V whose leading pages
 * sequences share (include/mk_cache.h).
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <vector>

#include "mk_cache.h"

namespace {

struct Args {
  int32_t Hq, Hkv, D, P, num_pages, max_pages, n_seqs, n_tokens, n_groups;
  const int32_t *tables, *lens, *off, *starts, *prefix;
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride;
  __nv_bfloat16 *out;
  float *lse;
  float scale;
  int32_t *err_host;
};

/* One warp per query token and head, one key at a time. */
__global__ void attn_rows(const Args a) {
  const int lane = threadIdx.x & 31;
  const long long row = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (row >= (long long)a.n_tokens * a.Hq) return;
  const int tok = (int)(row / a.Hq), head = (int)(row % a.Hq), kvh = head / (a.Hq / a.Hkv);
  bool bad = false;
  int b = -1, last = 0;
  if (a.off) {
    if (a.off[0] != 0) bad = true;
    for (int i = 0; i < a.n_seqs; ++i) {
      if (a.off[i + 1] < a.off[i] || a.off[i + 1] > a.n_tokens) bad = true;
      if (tok >= a.off[i] && tok < a.off[i + 1]) {
        b = i;
        last = a.off[i + 1];
      }
    }
  } else {
    b = tok;
    last = tok + 1;
  }
  for (int i = 0; i < a.n_seqs; ++i)
    if (a.lens[i] < 0 || a.lens[i] > (long long)a.max_pages * a.P) bad = true;
  if (a.n_groups) {
    if (a.starts[0] != 0 || a.starts[a.n_groups] != a.n_seqs) bad = true;
    for (int i = 0; i < a.n_groups; ++i)
      if (a.starts[i + 1] < a.starts[i] || a.prefix[i] < 0) bad = true;
  }
  if (bad) {
    *(volatile int32_t *)a.err_host = MK_ERR_INVALID_ARG;
    return;
  }
  if (b < 0) return;
  const int vis = a.lens[b] - (last - tok) + 1;
  const int n = a.D / 32;
  float q[4] = {}, o[4] = {}, m = -INFINITY, l = 0.0f;
  for (int i = 0; i < n; ++i)
    q[i] = __bfloat162float(a.q[tok * a.q_stride + (long long)head * a.D + i * 32 + lane]) * a.scale;
  for (int j = 0; j < vis; ++j) {
    const int page = a.tables[(size_t)b * a.max_pages + j / a.P];
    if ((unsigned)page >= (unsigned)a.num_pages) {
      *(volatile int32_t *)a.err_host = MK_ERR_PAGE_OOB;
      continue;
    }
    const size_t at = (((size_t)page * a.Hkv + kvh) * a.P + j % a.P) * a.D + lane;
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += q[i] * __bfloat162float(a.k[at + i * 32]);
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const float mn = fmaxf(m, s), c = expf(m - mn), p = expf(s - mn);
    for (int i = 0; i < n; ++i) o[i] = o[i] * c + p * __bfloat162float(a.v[at + i * 32]);
    l = l * c + p;
    m = mn;
  }
  for (int i = 0; i < n; ++i)
    a.out[row * a.D + i * 32 + lane] = __float2bfloat16(l > 0.0f ? o[i] / l : 0.0f);
  if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
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
  std::vector<const void *> k, v;
  float scale = 0.0f;
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0;
  int32_t *err_host = nullptr, *err_dev = nullptr;
};

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
      d->max_tokens > (1 << 20) || d->max_seqs > 1024 || d->max_groups > 1024 ||
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
  try {
    at->k.assign(d->k_caches, d->k_caches + d->n_layers);
    at->v.assign(d->v_caches, d->v_caches + d->n_layers);
  } catch (...) {
    delete at;
    return MK_ERR_CUDA;
  }
  at->d.k_caches = at->d.v_caches = nullptr;
  at->scale = d->scale > 0.0f ? d->scale : (float)(1.0 / std::sqrt((double)d->head_dim));
  at->stream = (cudaStream_t)stream;
  at->dev = dev;
  at->n_sm = prop.multiProcessorCount;
  cudaError_t e = cudaHostAlloc(&at->err_host, 64, cudaHostAllocMapped);
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
  a.D = d.head_dim;
  a.P = d.page_size;
  a.num_pages = d.num_pages;
  a.max_pages = b->max_pages_per_seq;
  a.n_seqs = b->n_seqs;
  a.n_tokens = b->n_tokens;
  a.n_groups = b->n_groups;
  a.starts = b->group_starts;
  a.prefix = b->prefix_lens;
  a.tables = b->page_tables;
  a.lens = b->seq_lens;
  a.off = b->q_offsets;
  a.q = (const __nv_bfloat16 *)q;
  a.k = (const __nv_bfloat16 *)at->k[layer];
  a.v = (const __nv_bfloat16 *)at->v[layer];
  a.q_stride = q_token_stride;
  a.out = (__nv_bfloat16 *)out;
  a.lse = lse;
  a.scale = at->scale;
  a.err_host = at->err_dev;
  const long long rows = (long long)b->n_tokens * d.n_q_heads;
  attn_rows<<<(unsigned)((rows + 7) / 8), 256, 0, at->stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MK_OK : MK_ERR_CUDA;
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
