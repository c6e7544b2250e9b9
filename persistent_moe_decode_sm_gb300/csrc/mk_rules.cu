/*
 * mk_rules.cu -- penalties, biases and masks on logits, and the greedy token under them
 * (include/mk_rules.h).
 *
 * The work is cut into items of one row and one slice of the vocabulary.  A block takes items of
 * one slice after another, rows in order, and keeps a word for each token of the slice in shared
 * memory: how often the token was generated, whether the prompt has it, whether it has a bias.
 * The words of a history are counted once for all rows in a row that share it (the tokens of a
 * drafted tree); a row's path and biases are put in before its logits pass by, and taken out again.
 */
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "mk_device.h"
#include "mk_rules.h"

namespace {

using namespace mk_dev;

constexpr int kThreads = 256;
constexpr int kSlice = 8192, kLeast = 1024; /* tokens of a slice: at most, at least */
constexpr int kMost = 1 << 24;              /* vocabulary, rows */
constexpr uint32_t kPrompt = 1u << 31, kBias = 1u << 30, kCount = kBias - 1;

struct Args {
  mk_rules_batch b;
  int32_t vocab, slice, slices;
  const void *logits;
  int64_t row_stride;
  float *out;
  int32_t *out_tokens;
  unsigned long long *best; /* [max_rows] of the slices so far, 0 between calls */
  int32_t *done;            /* [max_rows] slices so far, 0 between calls */
  Errors err;
};

__device__ __forceinline__ float4 load4(const float *p) { return __ldcg((const float4 *)p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
  const uint2 w = __ldcg((const uint2 *)p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float load1(const float *p) { return __ldcg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) {
  const unsigned short w = __ldcg((const unsigned short *)p);
  return __uint_as_float((uint32_t)w << 16);
}

/* A row's arguments, the same in every thread. */
struct Row {
  int begin, end, prompt, path0, path1, bias0, bias1, mask;
  float rep, pres, freq;
};
__device__ __forceinline__ bool load_row(const mk_rules_batch &b, int row, Row *r) {
  *r = Row{0, 0, 0, 0, 0, 0, 0, -1, 1.0f, 0.0f, 0.0f};
  if (b.ranges) {
    r->begin = __ldcg(b.ranges + 2 * (size_t)row);
    r->end = __ldcg(b.ranges + 2 * (size_t)row + 1);
    if (b.prompt_lens) r->prompt = __ldcg(b.prompt_lens + row);
  }
  if (b.path_offsets) {
    r->path0 = __ldcg(b.path_offsets + row);
    r->path1 = __ldcg(b.path_offsets + row + 1);
  }
  if (b.bias_offsets) {
    r->bias0 = __ldcg(b.bias_offsets + row);
    r->bias1 = __ldcg(b.bias_offsets + row + 1);
  }
  if (b.repetition) r->rep = __ldcg(b.repetition + row);
  if (b.presence) r->pres = __ldcg(b.presence + row);
  if (b.frequency) r->freq = __ldcg(b.frequency + row);
  if (b.allowed) r->mask = b.allowed_rows ? __ldcg(b.allowed_rows + row) : row;
  return r->begin >= 0 && r->end >= r->begin && r->end <= b.n_tokens && r->prompt >= 0 &&
         r->path0 >= 0 && r->path1 >= r->path0 && r->path1 <= b.n_path && r->bias0 >= 0 &&
         r->bias1 >= r->bias0 && r->bias1 <= b.n_bias && r->mask < b.n_masks && r->rep > 0.0f;
}

__device__ __forceinline__ float ruled(float x, uint32_t word, const float *bias, bool may, const Row &r) {
  if (word) {
    if (word & ~kBias) {
      x = x > 0.0f ? __fdiv_rn(x, r.rep) : __fmul_rn(x, r.rep);
      const uint32_t c = word & kCount;
      if (c) {
        x = __fsub_rn(x, __fmul_rn(r.freq, (float)c));
        x = __fsub_rn(x, r.pres);
      }
    }
    if (word & kBias) x = __fadd_rn(x, *bias);
  }
  return may ? x : -INFINITY;
}

/* The row's best so far: x in an order that integers keep (-0 as 0), then the lowest id. */
__device__ __forceinline__ unsigned long long best_key(float x, int id) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (unsigned long long)(u ^ (uint32_t)((int32_t)u >> 31 | 0x80000000)) << 32 | (uint32_t)~id;
}

template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads, 3) apply_rules(const __grid_constant__ Args a) {
  extern __shared__ uint4 shared[];
  __shared__ unsigned long long s_best;
  uint32_t *words = (uint32_t *)shared;
  float *biases = (float *)(words + a.slice);
  const mk_rules_batch &b = a.b;
  const int tid = threadIdx.x, lane = tid & 31;
  const bool counts = b.ranges || b.path_offsets || b.bias_offsets;
  if (tid == 0) s_best = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long total = (long long)a.slices * b.n_rows;
  const long long first = total * blockIdx.x / gridDim.x, last = total * (blockIdx.x + 1) / gridDim.x;
  int at_slice = -1, at_begin = 0, at_end = 0, at_prompt = 0; /* whose words are there */
  for (long long item = first; item < last; ++item) {
    const int slice = (int)(item / b.n_rows), row = (int)(item - (long long)slice * b.n_rows);
    const int v0 = slice * a.slice, nv = min(a.slice, a.vocab - v0);
    Row r;
    if (!load_row(b, row, &r)) {
      if (tid == 0) report(a.err, MK_ERR_INVALID_ARG);
      continue;
    }
    bool wrong = false;
    if (counts) {
      if (slice != at_slice || r.begin != at_begin || r.end != at_end || r.prompt != at_prompt) {
        __syncthreads();
        for (int i = tid; i < a.slice / 4; i += kThreads) shared[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        for (int i = r.begin + tid; i < r.end; i += kThreads) {
          const unsigned t = (unsigned)(__ldcg(b.tokens + i) - v0);
          if (t < (unsigned)nv) {
            if (i - r.begin < r.prompt)
              atomicOr(words + t, kPrompt);
            else
              atomicAdd(words + t, 1u);
          }
        }
        at_slice = slice;
        at_begin = r.begin;
        at_end = r.end;
        at_prompt = r.prompt;
      }
      for (int i = r.path0 + tid; i < r.path1; i += kThreads) {
        const unsigned t = (unsigned)(__ldcg(b.path_tokens + i) - v0);
        if (t < (unsigned)nv) atomicAdd(words + t, 1u);
      }
      for (int i = r.bias0 + tid; i < r.bias1; i += kThreads) {
        const int id = __ldcg(b.bias_tokens + i);
        wrong |= (unsigned)id >= (unsigned)a.vocab || (i > r.bias0 && __ldcg(b.bias_tokens + i - 1) >= id);
        const unsigned t = (unsigned)(id - v0);
        if (t < (unsigned)nv) {
          atomicOr(words + t, kBias);
          biases[t] = __ldcg(b.bias + i);
        }
      }
      wrong = __syncthreads_or(wrong);
      if (wrong && tid == 0) report(a.err, MK_ERR_INVALID_ARG);
    }
    if (!wrong) {
      const T *src = (const T *)a.logits + row * a.row_stride + v0;
      float *dst = a.out ? a.out + (long long)row * a.vocab + v0 : nullptr;
      const uint32_t *mask =
          r.mask >= 0 ? b.allowed + (size_t)r.mask * ((a.vocab + 31) / 32) + v0 / 32 : nullptr;
      float top = -INFINITY;
      int at = -1;
      if (VEC) {
        for (int i = 4 * tid; i + 3 < nv; i += 4 * kThreads) {
          const float4 x = load4(src + i);
          const uint32_t may = mask ? __ldcg(mask + i / 32) >> (i & 31) : 15u;
          const uint4 w = counts ? shared[i / 4] : make_uint4(0, 0, 0, 0);
          float4 y;
          y.x = ruled(x.x, w.x, biases + i, may & 1, r);
          y.y = ruled(x.y, w.y, biases + i + 1, may & 2, r);
          y.z = ruled(x.z, w.z, biases + i + 2, may & 4, r);
          y.w = ruled(x.w, w.w, biases + i + 3, may & 8, r);
          if (dst) __stcs((float4 *)(dst + i), y);
          if (y.x > top) top = y.x, at = i;
          if (y.y > top) top = y.y, at = i + 1;
          if (y.z > top) top = y.z, at = i + 2;
          if (y.w > top) top = y.w, at = i + 3;
        }
      }
      for (int i = (VEC ? nv & ~3 : 0) + tid; i < nv; i += kThreads) {
        const bool may = !mask || (__ldcg(mask + i / 32) >> (i & 31) & 1);
        const float y = ruled(load1(src + i), counts ? words[i] : 0, biases + i, may, r);
        if (dst) __stcs(dst + i, y);
        if (y > top) top = y, at = i;
      }
      if (a.out_tokens) {
        unsigned long long key = at < 0 ? 0 : best_key(top, v0 + at);
#pragma unroll
        for (int o = 16; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        if (lane == 0 && key) atomicMax(&s_best, key);
      }
    }
    if (a.out_tokens || counts) __syncthreads();
    if (!wrong && a.out_tokens && tid == 0) {
      unsigned long long key = s_best;
      s_best = 0;
      bool mine = true; /* the row's last slice writes its token */
      if (a.slices > 1) {
        if (key) atomicMax(a.best + row, key);
        __threadfence();
        mine = atomicAdd(a.done + row, 1) == a.slices - 1;
        if (mine) {
          __threadfence();
          key = atomicExch(a.best + row, 0ull);
          a.done[row] = 0;
        }
      }
      if (mine) a.out_tokens[row] = key ? (int32_t)~(uint32_t)key : -1;
    }
    if (counts) { /* the row's own words out again */
      for (int i = r.path0 + tid; i < r.path1; i += kThreads) {
        const unsigned t = (unsigned)(__ldcg(b.path_tokens + i) - v0);
        if (t < (unsigned)nv) atomicSub(words + t, 1u);
      }
      for (int i = r.bias0 + tid; i < r.bias1; i += kThreads) {
        const unsigned t = (unsigned)(__ldcg(b.bias_tokens + i) - v0);
        if (t < (unsigned)nv) atomicAnd(words + t, ~kBias);
      }
    }
    if (a.out_tokens || counts) __syncthreads();
  }
}

}  // namespace

struct mk_rules {
  int32_t vocab = 0, max_rows = 0;
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0;
  uint8_t *ws = nullptr; /* the error word; best and done of each row */
  Errors err{};
  int32_t *err_host = nullptr;
};

namespace {

typedef void (*Kernel)(Args);
constexpr Kernel kKernels[2][2] = {{apply_rules<float, false>, apply_rules<float, true>},
                                   {apply_rules<__nv_bfloat16, false>, apply_rules<__nv_bfloat16, true>}};

}  // namespace

extern "C" {

mk_status mk_rules_create(int32_t vocab, int32_t max_rows, void *stream, mk_rules **out) {
  if (!out || vocab < 1 || max_rows < 1) return MK_ERR_INVALID_ARG;
  if (vocab > kMost || max_rows > kMost) return MK_ERR_UNSUPPORTED;
  int dev = 0, n_sm = 0;
  if (!this_device(&dev, &n_sm)) return MK_ERR_NO_DEVICE;
  mk_rules *m = new (std::nothrow) mk_rules();
  if (!m) return MK_ERR_CUDA;
  m->vocab = vocab;
  m->max_rows = max_rows;
  m->stream = (cudaStream_t)stream;
  m->dev = dev;
  m->n_sm = n_sm;
  const size_t bytes = 64 + 16 * (size_t)max_rows;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i)
    e = cudaFuncSetAttribute(kKernels[i / 2][i % 2], cudaFuncAttributeMaxDynamicSharedMemorySize, kSlice * 8);
  if (e == cudaSuccess) e = cudaMalloc(&m->ws, bytes);
  if (e == cudaSuccess) e = cudaMemsetAsync(m->ws, 0, bytes, m->stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(m->stream);
  if (e == cudaSuccess) e = cudaHostAlloc(&m->err_host, 64, cudaHostAllocMapped);
  if (e == cudaSuccess) {
    std::memset(m->err_host, 0, 64);
    m->err.first = (int32_t *)m->ws;
    e = cudaHostGetDevicePointer((void **)&m->err.host, m->err_host, 0);
  }
  if (e != cudaSuccess) {
    mk_rules_destroy(m);
    cudaGetLastError(); /* reported here: not to the caller's next launch as well */
    return MK_ERR_CUDA;
  }
  *out = m;
  return MK_OK;
}

void mk_rules_destroy(mk_rules *m) {
  if (!m) return;
  {
    OnDevice on(m->dev);
    cudaStreamSynchronize(m->stream);
    if (m->ws) cudaFree(m->ws);
    if (m->err_host) cudaFreeHost(m->err_host);
  }
  delete m;
}

mk_status mk_rules_apply(mk_rules *m, const mk_rules_batch *b, const void *logits, int32_t is_bf16,
                         int64_t row_stride, float *out, int32_t *out_tokens) {
  if (!m || !b || b->n_rows < 0 || b->n_tokens < 0 || b->n_path < 0 || b->n_bias < 0 || b->n_masks < 0)
    return MK_ERR_INVALID_ARG;
  if (b->n_rows > m->max_rows) return MK_ERR_BATCH;
  if (b->n_tokens > kCount / 2 || b->n_path > kCount / 2) return MK_ERR_UNSUPPORTED; /* a word's count */
  if (b->n_rows == 0) return MK_OK;
  const void *four[] = {b->tokens, b->ranges, b->prompt_lens, b->path_offsets, b->path_tokens, b->repetition,
                        b->presence, b->frequency, b->bias_offsets, b->bias_tokens, b->bias, b->allowed,
                        b->allowed_rows, out, out_tokens};
  for (const void *p : four)
    if (!aligned(p, 4)) return MK_ERR_INVALID_ARG;
  if ((b->ranges && b->n_tokens && !b->tokens) || (b->path_offsets && b->n_path && !b->path_tokens) ||
      (b->bias_offsets && b->n_bias && (!b->bias_tokens || !b->bias)) || (b->prompt_lens && !b->ranges) ||
      (b->allowed_rows && !b->allowed) || (b->allowed && !b->allowed_rows && b->n_masks < b->n_rows))
    return MK_ERR_INVALID_ARG;
  const int64_t size = is_bf16 ? 2 : 4, V = m->vocab;
  if (!logits || (!out && !out_tokens) || !aligned(logits, (unsigned)size) || row_stride < V ||
      row_stride >= (int64_t)1 << 39)
    return MK_ERR_INVALID_ARG;
  const bool in_place = out == logits && !is_bf16 && row_stride == V;
  if (out && !in_place && rows_meet(logits, row_stride * size, V * size, out, V * 4, V * 4, b->n_rows))
    return MK_ERR_INVALID_ARG;
  OnDevice on(m->dev);
  if (!on.ok) return MK_ERR_CUDA;
  Args a{};
  a.b = *b;
  if (!b->allowed) a.b.n_masks = 1; /* row masks are not looked at */
  a.vocab = m->vocab;
  a.logits = logits;
  a.row_stride = row_stride;
  a.out = out;
  a.out_tokens = out_tokens;
  a.err = m->err;
  a.best = (unsigned long long *)(m->ws + 64);
  a.done = (int32_t *)(m->ws + 64 + 8 * (size_t)m->max_rows);
  /* slices: as large as leaves every SM an item */
  a.slice = kSlice;
  while (a.slice > kLeast && (V + a.slice - 1) / a.slice * b->n_rows < m->n_sm) a.slice /= 2;
  a.slices = (int32_t)((V + a.slice - 1) / a.slice);
  const bool vec = row_stride % 4 == 0 && aligned(logits, 4 * (unsigned)size) &&
                   (!out || (V % 4 == 0 && aligned(out, 16)));
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((int64_t)a.slices * b->n_rows, m->n_sm * 3));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)a.slice * 8;
  cfg.stream = m->stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kKernels[is_bf16 ? 1 : 0][vec], a) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_rules_sync(mk_rules *m) {
  return m ? take_error(m->dev, m->stream, m->err, m->err_host) : MK_ERR_INVALID_ARG;
}

}  // extern "C"
