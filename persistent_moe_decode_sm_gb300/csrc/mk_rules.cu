/*
 * mk_rules.cu -- penalties, biases and masks on logits, and the greedy token under them
 * (include/mk_rules.h).
 *
 * The work is cut into items of one row and one slice of the vocabulary.  A block takes items of
 * one slice after another, rows in order, and keeps a word for each token of the slice in shared
 * memory: how often the token was generated, whether the prompt has it, whether it has a bias.
 * The words of a history are counted once for all rows in a row that share it (the tokens of a
 * drafted tree); a row's path and biases are put in before its logits pass by, and taken out again.
 *
 * What bounds it: 384 bf16 rows of 152064 (350 MB) take 107 us, 3.3 TB/s, of which the copy with
 * the greedy token is 69 (writes to DRAM, about 70 instructions for 128 tokens, a row's beginning and
 * end) and masks, words and their rules the rest.  With rules in line, where a token's word
 * is met, most warps run them for one lane: 132 us; but a list takes its time to make, so where rows
 * are few they are in line: 8 rows 13.4 us (with a list 15.7), one row of 32000 5.5 (8.0), both a chain of
 * loads, each for the next: arguments, histories, the rows' best.
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

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kSlice = 8192, kLeast = 1024; /* tokens of a slice: at most, at least */
constexpr int kMost = 1 << 24;              /* vocabulary, rows */
/* Blocks an SM: without vectors the registers of four spill (256 rows of 50257: 47 us, with four 68). */
constexpr int blocks_of(bool vec) { return vec ? 4 : 3; }
constexpr unsigned long long kWrong = 1; /* the key of a row that is not written: below that of any value */
constexpr uint32_t kPrompt = 1u << 31, kBias = 1u << 30, kCount = kBias - 1;

struct Args {
  mk_rules_batch b;
  int32_t vocab, slice, slices;
  int32_t behind_step; /* out_tokens holds the step's own tokens, which a wrong row must not keep */
  const void *logits;
  int64_t row_stride;
  float *out;
  int32_t *out_tokens;
  unsigned long long *best; /* [max_rows] of the slices so far, 0 between calls */
  int32_t *done;            /* blocks that are done, 0 between calls */
  Errors err;
};

/* Four tokens' logits as they lie in memory; none beyond `n` are looked at. */
template <class T>
struct Four;
template <>
struct Four<float> {
  float4 v;
  __device__ __forceinline__ void load(const float *p) { v = __ldcg((const float4 *)p); }
  __device__ __forceinline__ void load(const float *p, int step, int n) {
    v.x = n > 0 ? __ldcg(p) : 0.0f;
    v.y = n > step ? __ldcg(p + step) : 0.0f;
    v.z = n > 2 * step ? __ldcg(p + 2 * step) : 0.0f;
    v.w = n > 3 * step ? __ldcg(p + 3 * step) : 0.0f;
  }
  __device__ __forceinline__ float4 get() const { return v; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { v = __ldcg((const uint2 *)p); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *q, int step, int n) {
    const unsigned short *p = (const unsigned short *)q;
    const uint32_t a = n > 0 ? __ldcg(p) : 0, b = n > step ? __ldcg(p + step) : 0;
    const uint32_t c = n > 2 * step ? __ldcg(p + 2 * step) : 0, d = n > 3 * step ? __ldcg(p + 3 * step) : 0;
    v = make_uint2(a | b << 16, c | d << 16);
  }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
};

__device__ __forceinline__ float load1(const float *p) { return __ldcg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) {
  return __uint_as_float((uint32_t)__ldcg((const unsigned short *)p) << 16);
}

/* A row's arguments.  A lane of one warp loads each. */
struct Row {
  int begin, end, prompt, path0, path1, bias0, bias1, mask;
  float rep, pres, freq;
  int sound; /* whether they can be used */
};
constexpr int kRowWords = 11;
struct RowLoader {
  const int32_t *at;
  int stride, otherwise;
  __device__ RowLoader(const mk_rules_batch &b, int lane) : at(nullptr), stride(1), otherwise(0) {
    switch (lane) {
      case 0: at = b.ranges, stride = 2; break;
      case 1: at = b.ranges ? b.ranges + 1 : nullptr, stride = 2; break;
      case 2: at = b.prompt_lens; break;
      case 3: at = b.path_offsets; break;
      case 4: at = b.path_offsets ? b.path_offsets + 1 : nullptr; break;
      case 5: at = b.bias_offsets; break;
      case 6: at = b.bias_offsets ? b.bias_offsets + 1 : nullptr; break;
      case 7: at = b.allowed_rows, otherwise = -1; break;
      case 8: at = (const int32_t *)b.repetition, otherwise = 0x3f800000; break;
      case 9: at = (const int32_t *)b.presence; break;
      case 10: at = (const int32_t *)b.frequency; break;
    }
    if (lane == 7 && b.allowed && !b.allowed_rows) otherwise = -2; /* the row's own */
  }
  __device__ __forceinline__ int operator()(int row) const {
    return at ? __ldcg(at + (size_t)row * stride) : otherwise == -2 ? row : otherwise;
  }
};
__device__ __forceinline__ bool sound(const mk_rules_batch &b, const Row &r) {
  return r.begin >= 0 && r.end >= r.begin && r.end <= b.n_tokens && r.prompt >= 0 && r.path0 >= 0 &&
         r.path1 >= r.path0 && r.path1 <= b.n_path && r.bias0 >= 0 && r.bias1 >= r.bias0 &&
         r.bias1 <= b.n_bias && r.mask < b.n_masks && r.rep > 0.0f;
}

/* The row's best so far: x in an order that integers keep (-0 as 0), then the lowest id. */
__device__ __forceinline__ unsigned long long best_key(float x, int id) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (unsigned long long)(u ^ (uint32_t)((int32_t)u >> 31 | 0x80000000)) << 32 | (uint32_t)~id;
}

/* A row's penalties on one logit.  The quotient is x / r rounded once: r's rounded reciprocal, and
 * the remainder of the first quotient in fused arithmetic (Markstein, "Computation of elementary
 * functions on the IBM RISC System/6000 processor", 1990), which holds where nothing comes near
 * the ends of the range; there the division itself is called. */
struct Penalty {
  float rep, inverse, pres, freq;
  bool tame;
  __device__ explicit Penalty(const Row &r) {
    rep = r.rep;
    inverse = __frcp_rn(r.rep);
    pres = r.pres;
    freq = r.freq;
    tame = r.rep > 0x1p-30f && r.rep < 0x1p30f;
  }
  __device__ __forceinline__ float operator()(float x, uint32_t word) const {
    const float q = x * inverse, d = fmaf(fmaf(-q, rep, x), inverse, q), size = fabsf(x);
    float y = x > 0.0f ? d : __fmul_rn(x, rep);
    if (x > 0.0f && !(tame && size > 0x1p-60f && size < 0x1p60f)) y = __fdiv_rn(x, rep);
    const uint32_t c = word & kCount;
    const float z = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, (float)c)), pres);
    y = c ? z : y;
    return word & ~kBias ? y : x;
  }
};

/* An id's place in a slice that begins at v0; any id, so in unsigned numbers. */
__device__ __forceinline__ int less(int id, int v0) { return (int)((unsigned)id - (unsigned)v0); }

/* A block's slice: a word for each token, and (LIST) which tokens have one, and those tokens: the
 * history's in order, then the row's own. */
struct Words {
  uint32_t *word, *marked; /* [slice], [slice / 32] bits */
  uint16_t *list;          /* [slice] */
  __device__ Words(void *at, int slice)
      : word((uint32_t *)at), marked(word + slice), list((uint16_t *)(marked + slice / 32)) {}
  __device__ __forceinline__ void mark(int t, uint32_t before, int *length) const {
    if (before) return;
    list[atomicAdd(length, 1)] = (uint16_t)t;
    atomicOr(marked + t / 32, 1u << t % 32);
  }
};
static_assert(kSlice / 32 <= kThreads, "a thread lists one word of the bits");
constexpr size_t words_bytes(int slice) { return (size_t)slice * 6 + slice / 8; }

/* A thread's tokens of a slice, four to each chunk of 1024: in a row (VEC), or one of each 32 of its
 * warp's 128.  They are
 * masked and copied; those with a word, few as a rule, get their rules behind that, densely, from
 * the list, or (not LIST) right there.  What a row needs next is loaded while the row before it is under way: its arguments and
 * logits, then its path, biases and mask. */
template <class T, bool VEC, int AHEAD, bool LIST>
__global__ void __launch_bounds__(kThreads, blocks_of(VEC)) apply_rules(const __grid_constant__ Args a) {
  constexpr int STEP = VEC ? 1 : 32, CHUNK = 4 * kThreads; /* AHEAD chunks' logits are under way */
  extern __shared__ uint4 shared[];
  __shared__ unsigned long long s_best;
  __shared__ int s_length, s_history; /* of the list, and of its part that rows share */
  __shared__ __align__(16) Row s_row[2];
  __shared__ int s_id[kThreads]; /* the row's first biases */
  __shared__ float s_bias[kThreads];
  const Words ws(shared, a.slice);
  const mk_rules_batch &b = a.b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, mine = VEC ? 4 * tid : warp * 128 + lane;
  const int mine_mask = VEC ? mine : warp * 128 + (lane & 3) * 32; /* the first token of this thread's word of a mask */
  const bool counts = b.ranges || b.path_offsets || b.bias_offsets;
  const RowLoader loader(b, warp == kWarps - 1 ? lane : 32);
  if (tid == 0) {
    s_best = 0;
    s_length = 0;
  }
  auto clear = [&] {
    for (int i = tid; i < a.slice / 4; i += kThreads) ((uint4 *)ws.word)[i] = make_uint4(0, 0, 0, 0);
    if (LIST)
      for (int i = tid; i < a.slice / 32; i += kThreads) ws.marked[i] = 0;
  };
  if (counts) clear(); /* the grid before may still be running */
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  /* Two stretches of the items, slice by slice and row by row: text is made of few tokens, and those
   * have low ids, so a block has as much of the first slices as of the last. */
  const long long total = (long long)a.slices * b.n_rows, halves = 2ll * gridDim.x;
  const long long lo = total * blockIdx.x / halves, lo_end = total * (blockIdx.x + 1) / halves;
  const long long hi = total * (halves - 1 - blockIdx.x) / halves, hi_end = total * (halves - blockIdx.x) / halves;
  const int n_lo = (int)(lo_end - lo), n_items = n_lo + (int)(hi_end - hi);
  if (n_items) {
    const long long first = n_lo ? lo : hi;
    int slice = (int)(first / b.n_rows), row = (int)(first - (long long)slice * b.n_rows);
    const int mask_words = (a.vocab + 31) / 32;
    Four<T> raw[AHEAD];
    const T *ahead; /* where the next chunks' logits lie, and how many tokens are left from there */
    int ahead_left;
    auto begin = [&](int slice, int row) {
      const int i = slice * a.slice + mine;
      ahead = (const T *)a.logits + row * a.row_stride + i;
      ahead_left = min(a.slice, a.vocab - slice * a.slice) - mine;
    };
    auto fetch = [&](int k) {
      if (!VEC)
        raw[k].load(ahead + k * CHUNK, STEP, ahead_left - k * CHUNK);
      else if (ahead_left > k * CHUNK)
        raw[k].load(ahead + k * CHUNK);
    };
    auto go_on = [&] {
      ahead += AHEAD * CHUNK;
      ahead_left -= AHEAD * CHUNK;
    };
    auto put_row = [&](Row &to, int word) { /* by one warp */
      if (lane < kRowWords) ((int *)&to)[lane] = word;
      __syncwarp();
      if (lane == 0) to.sound = sound(b, to);
    };
    if (warp == kWarps - 1) put_row(s_row[0], lane < kRowWords ? loader(row) : 0);
    begin(slice, row);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) fetch(k);
    go_on();
    __syncthreads();
    int path_id = -1, bias_id = -1, bias_before = -1;
    float bias = 0.0f;
    uint32_t may[AHEAD];
    auto fetch_mask = [&](int k, const uint32_t *at, int left) {
      may[k] = at && left > k * CHUNK ? __ldcg(at + k * (CHUNK / 32)) : 0xffffffffu;
    };
    const uint32_t *mask = nullptr; /* this thread's word of the row's next chunk */
    auto fetch_own = [&](const Row &r, bool is_sound, int slice) {
      mask = nullptr;
      path_id = bias_id = bias_before = -1;
      if (!is_sound) return;
      if (r.path0 + tid < r.path1) path_id = __ldcg(b.path_tokens + r.path0 + tid);
      if (r.bias0 + tid < r.bias1) {
        bias_id = __ldcg(b.bias_tokens + r.bias0 + tid);
        bias = __ldcg(b.bias + r.bias0 + tid);
        if (tid) bias_before = __ldcg(b.bias_tokens + r.bias0 + tid - 1);
      }
      const int s0 = slice * a.slice;
      if (r.mask >= 0) mask = b.allowed + (size_t)r.mask * mask_words + (s0 + mine_mask) / 32;
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) fetch_mask(k, mask, min(a.slice, a.vocab - s0) - mine_mask);
    };
    Row r = s_row[0];
    bool is_sound = r.sound;
    fetch_own(r, is_sound, slice);
    int at_slice = -1, at_begin = 0, at_end = 0, at_prompt = 0; /* whose words are there */
#pragma unroll 1
    for (int n = 0; n < n_items; ++n) {
      const int v0 = slice * a.slice, nv = min(a.slice, a.vocab - v0);
      const bool more = n + 1 < n_items;
      int next_slice = slice, next_row = row + 1;
      if (n + 1 == n_lo) {
        next_slice = (int)(hi / b.n_rows);
        next_row = (int)(hi - (long long)next_slice * b.n_rows);
      } else if (next_row == b.n_rows) {
        next_row = 0;
        ++next_slice;
      }
      int next_word = 0;
      if (more && warp == kWarps - 1 && lane < kRowWords) next_word = loader(next_row);
      const bool readable = is_sound;
      bool wrong = !is_sound;
      const int n_bias = r.bias1 - r.bias0;
      int own_path = -1, own_bias = -1; /* this thread's first words of the row's own */
      auto add = [&](int t, uint32_t count, uint32_t flag) {
        const uint32_t before = flag ? atomicOr(ws.word + t, flag) : atomicAdd(ws.word + t, count);
        if (LIST) ws.mark(t, before, &s_length);
      };
      if (counts && is_sound) {
        if (slice != at_slice || r.begin != at_begin || r.end != at_end || r.prompt != at_prompt) {
          if (at_slice >= 0) {
            clear();
            __syncthreads();
          }
          for (int i0 = r.begin + tid; i0 < r.end; i0 += 8 * kThreads) {
            int t[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) t[k] = i0 + k * kThreads < r.end ? less(__ldcg(b.tokens + i0 + k * kThreads), v0) : -1;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if ((unsigned)t[k] >= (unsigned)nv) continue;
              if (i0 + k * kThreads - r.begin < r.prompt)
                atomicOr(ws.word + t[k], kPrompt);
              else
                atomicAdd(ws.word + t[k], 1u);
              if (LIST) atomicOr(ws.marked + t[k] / 32, 1u << t[k] % 32);
            }
          }
          if (LIST) {
            __syncthreads();
            /* the list, in order: a thread has one word of the bits */
            uint32_t bits = tid < a.slice / 32 ? ws.marked[tid] : 0;
            const int mine = __popc(bits);
            int before = mine;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
              const int y = __shfl_up_sync(0xffffffffu, before, o);
              if (lane >= o) before += y;
            }
            if (lane == 31) s_id[warp] = before;
            __syncthreads();
            int to = before - mine, all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              if (w < warp) to += s_id[w];
              all += s_id[w];
            }
            for (; bits; bits &= bits - 1) ws.list[to++] = (uint16_t)(tid * 32 + __ffs(bits) - 1);
            if (tid == 0) s_length = s_history = all;
            __syncthreads();
          }
          at_slice = slice;
          at_begin = r.begin;
          at_end = r.end;
          at_prompt = r.prompt;
        }
        if (path_id >= v0 && path_id - v0 < nv) {
          own_path = path_id - v0;
          add(own_path, 1, 0);
        }
        if (tid < n_bias) {
          wrong = (unsigned)bias_id >= (unsigned)a.vocab || bias_before >= bias_id;
          s_id[tid] = bias_id;
          s_bias[tid] = bias;
          if (bias_id >= v0 && bias_id - v0 < nv) {
            own_bias = bias_id - v0;
            add(own_bias, 0, kBias);
          }
        }
        for (int i = r.path0 + tid + kThreads; i < r.path1; i += kThreads) {
          const int t = less(__ldcg(b.path_tokens + i), v0);
          if ((unsigned)t < (unsigned)nv) add(t, 1, 0);
        }
        for (int i = r.bias0 + tid + kThreads; i < r.bias1; i += kThreads) {
          const int id = __ldcg(b.bias_tokens + i), t = less(id, v0);
          wrong |= (unsigned)id >= (unsigned)a.vocab || __ldcg(b.bias_tokens + i - 1) >= id;
          if ((unsigned)t < (unsigned)nv) add(t, 0, kBias);
        }
        wrong = __syncthreads_or(wrong);
      }
      if (wrong && tid == 0) report(a.err, MK_ERR_INVALID_ARG);
      const int length = LIST && counts && is_sound ? s_length : 0;
      const Penalty penalty(r);
      auto ruled = [&](float x, uint32_t word, int id) {
        float y = penalty(x, word);
        if (word & kBias) {
          int at = 0, e = n_bias - 1; /* the last bias token at or below id: id itself */
          while (at < e) {
            const int m = (at + e + 1) >> 1;
            if ((m < kThreads ? s_id[m] : __ldcg(b.bias_tokens + r.bias0 + m)) <= id)
              at = m;
            else
              e = m - 1;
          }
          y = __fadd_rn(y, at < kThreads ? s_bias[at] : __ldcg(b.bias + r.bias0 + at));
        }
        return y;
      };
      const T *src = (const T *)a.logits + row * a.row_stride + v0;
      float *dst = a.out ? a.out + (long long)row * a.vocab + v0 : nullptr;
      const uint32_t *masks = r.mask >= 0 && !wrong ? b.allowed + (size_t)r.mask * mask_words + v0 / 32 : nullptr;
      float top = -INFINITY;
      int at = -1;
      const uint32_t *marked = ws.marked + mine / 32;
      float *to = dst + mine;
      int left = wrong ? 0 : nv - mine; /* of this thread's tokens */
#pragma unroll 1
      for (int c0 = 0; c0 < a.slice; c0 += AHEAD * CHUNK) {
        const bool ends = c0 + AHEAD * CHUNK == a.slice;
        if (ends) {
          ahead_left = 0;
          if (more) begin(next_slice, next_row);
        }
        if (mask) mask += AHEAD * (CHUNK / 32);
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
          const float4 x = raw[k].get();
          uint32_t ok = may[k] >> (mine & 31), rest = 15; /* may follow; has no word */
          if (!VEC) {
            ok = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) ok |= (__shfl_sync(0xffffffffu, may[k], j) >> lane & 1) << j;
          }
          fetch(k);
          if (!ends) fetch_mask(k, mask, left + mine - mine_mask - AHEAD * CHUNK);
          if (left <= k * CHUNK) continue;
          if (VEC) {
            if (length) rest = ~marked[k * (CHUNK / 32)] >> (mine & 31);
          } else {
            uint32_t m[4] = {};
            if (length) *(uint4 *)m = *(const uint4 *)(ws.marked + (c0 + k * CHUNK) / 32 + warp * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (left <= k * CHUNK + j * STEP || (m[j] >> lane & 1)) rest &= ~(1u << j);
          }
          float y[4] = {x.x, x.y, x.z, x.w}, z[4];
          if (!LIST && counts) {
            uint32_t w[4];
            if (VEC) {
              *(uint4 *)w = *(const uint4 *)(ws.word + c0 + k * CHUNK + mine);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) w[j] = rest >> j & 1 ? ws.word[c0 + k * CHUNK + mine + j * STEP] : 0;
            }
            uint32_t todo = (w[0] ? 1 : 0) | (w[1] ? 2 : 0) | (w[2] ? 4 : 0) | (w[3] ? 8 : 0);
#pragma unroll 1
            for (; todo; todo &= todo - 1) { /* one or two of the four, as a rule */
              const int j = __ffs(todo) - 1;
              const float z = ruled(j == 0 ? y[0] : j == 1 ? y[1] : j == 2 ? y[2] : y[3],
                                    j == 0 ? w[0] : j == 1 ? w[1] : j == 2 ? w[2] : w[3],
                                    v0 + c0 + k * CHUNK + mine + j * STEP);
              y[0] = j == 0 ? z : y[0];
              y[1] = j == 1 ? z : y[1];
              y[2] = j == 2 ? z : y[2];
              y[3] = j == 3 ? z : y[3];
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (!(ok >> j & 1)) y[j] = -INFINITY;
            z[j] = rest >> j & 1 ? y[j] : -INFINITY;
          }
          if (dst) {
            if (VEC) {
              __stcs((float4 *)(to + k * CHUNK), make_float4(y[0], y[1], y[2], y[3]));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (left > k * CHUNK + j * STEP) __stcs(to + k * CHUNK + j * STEP, y[j]);
            }
          }
          const float m = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])); /* NaN only if all are */
          const int here = c0 + k * CHUNK + (z[0] == m ? 0 : z[1] == m ? STEP : z[2] == m ? 2 * STEP : 3 * STEP);
          at = m > top ? here : at;
          top = fmaxf(top, m);
        }
        go_on();
        marked += AHEAD * (CHUNK / 32);
        to += AHEAD * CHUNK;
        left -= AHEAD * CHUNK;
      }
      unsigned long long key = at >= 0 ? best_key(top, v0 + mine + at) : 0;
      if (more && warp == kWarps - 1) put_row(s_row[(n + 1) & 1], next_word);
      if (length) {
#pragma unroll 1
        for (int k0 = 0; k0 < length; k0 += 4 * kThreads) {
          int t[4];
          float x[4];
          uint32_t may[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = k0 + j * kThreads + tid;
            t[j] = k < length && !wrong ? ws.list[k] : -1;
            if (t[j] >= 0) {
              x[j] = load1(src + t[j]);
              may[j] = masks ? __ldcg(masks + t[j] / 32) : 0xffffffffu;
            }
          }
          /* over what was copied; in place it is the logit still, or masked for good */
          if (k0 == 0) __syncthreads();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (t[j] < 0) continue;
            float y = ruled(x[j], ws.word[t[j]], v0 + t[j]);
            if (!(may[j] >> t[j] % 32 & 1)) y = -INFINITY;
            if (dst) __stcs(dst + t[j], y);
            if (y > -INFINITY) key = max(key, best_key(y, v0 + t[j]));
          }
        }
      }
      if (a.out_tokens) {
        /* the largest value, then the lowest id that has it (the complement of a key's second half) */
        const uint32_t value = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32));
        const uint32_t id = __reduce_max_sync(0xffffffffu, (uint32_t)(key >> 32) == value ? (uint32_t)key : 0);
        if (lane == 0 && value) atomicMax(&s_best, (unsigned long long)value << 32 | id);
      }
      __syncthreads();
      if (a.out_tokens && tid == 0) {
        /* nothing waits for this: the last block takes the rows' best */
        const unsigned long long best = wrong ? kWrong : s_best;
        s_best = 0;
        if (best) atomicMax(a.best + row, best);
      }
      if (counts && readable) { /* the row's own words out again */
        if (own_path >= 0) atomicSub(ws.word + own_path, 1u);
        if (own_bias >= 0) atomicAnd(ws.word + own_bias, ~kBias);
        for (int i = r.path0 + tid + kThreads; i < r.path1; i += kThreads) {
          const unsigned t = less(__ldcg(b.path_tokens + i), v0);
          if (t < (unsigned)nv) atomicSub(ws.word + t, 1u);
        }
        for (int i = r.bias0 + tid + kThreads; i < r.bias1; i += kThreads) {
          const unsigned t = less(__ldcg(b.bias_tokens + i), v0);
          if (t < (unsigned)nv) atomicAnd(ws.word + t, ~kBias);
        }
        if (LIST) {
          for (int k = s_history + tid; k < length; k += kThreads)
            atomicAnd(ws.marked + ws.list[k] / 32, ~(1u << ws.list[k] % 32));
          if (tid == 0) s_length = s_history;
        }
      }
      if (more) {
        r = s_row[(n + 1) & 1];
        is_sound = r.sound;
        fetch_own(r, is_sound, next_slice);
      }
      __syncthreads();
      slice = next_slice;
      row = next_row;
    }
  }
  if (!a.out_tokens) return;
  if (tid == 0) { /* behind this thread's best, and before the others' are read */
    int before;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(before) : "l"(a.done) : "memory");
    s_length = before == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!s_length) return;
  for (int i0 = tid; i0 < b.n_rows; i0 += 8 * kThreads) {
    unsigned long long key[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * kThreads;
      key[k] = i < b.n_rows ? __ldcg(a.best + i) : kWrong;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * kThreads;
      if (i < b.n_rows) a.best[i] = 0;
      if (key[k] != kWrong)
        a.out_tokens[i] = key[k] ? (int32_t)~(uint32_t)key[k] : -1;
      else if (a.behind_step && i < b.n_rows)
        a.out_tokens[i] = -1;
    }
  }
  if (tid == 0) *a.done = 0;
}

}  // namespace

struct mk_rules {
  int32_t vocab = 0, max_rows = 0;
  cudaStream_t stream = nullptr;
  int dev = 0, n_sm = 0;
  uint8_t *ws = nullptr; /* the error word, the blocks done; best of each row */
  Errors err{};
  int32_t *err_host = nullptr;
};

namespace {

typedef void (*Kernel)(Args);
template <class T, bool VEC>
Kernel of_slice(int slice, bool list) {
  /* AHEAD divides a slice's chunks.  With a list, four chunks of fp32 are more registers than there are
   * (256 rows of 152064: 108 us, so 98); four of bf16 are as many as two of those (384 rows 107, 114). */
  return list                    ? apply_rules<T, VEC, VEC && sizeof(T) == 4 ? 2 : 4, true>
         : slice >= 4 * kLeast   ? apply_rules<T, VEC, 4, false>
         : slice == 2 * kLeast   ? apply_rules<T, VEC, 2, false>
                                 : apply_rules<T, VEC, 1, false>;
}
Kernel kernel_of(bool bf16, bool vec, int slice, bool list) {
  return bf16 ? vec ? of_slice<__nv_bfloat16, true>(slice, list) : of_slice<__nv_bfloat16, false>(slice, list)
         : vec ? of_slice<float, true>(slice, list) : of_slice<float, false>(slice, list);
}

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
  const size_t bytes = 64 + 8 * (size_t)max_rows;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 4 && e == cudaSuccess; ++i)
    e = cudaFuncSetAttribute(kernel_of(i / 2, i % 2, kSlice, true), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)words_bytes(kSlice));
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

mk_status mk_rules_check(const mk_rules *m, const mk_rules_batch *b, const void *logits, int32_t is_bf16,
                         int64_t row_stride, const float *out, const int32_t *out_tokens) {
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
      (b->allowed_rows && b->n_masks && !b->allowed) || (b->allowed && !b->allowed_rows && b->n_masks < b->n_rows))
    return MK_ERR_INVALID_ARG;
  const int64_t size = is_bf16 ? 2 : 4, V = m->vocab;
  if (!logits || (!out && !out_tokens) || !aligned(logits, (unsigned)size) || row_stride < V ||
      row_stride >= (int64_t)1 << 39)
    return MK_ERR_INVALID_ARG;
  const bool in_place = out == logits && !is_bf16 && row_stride == V;
  if (out && !in_place && rows_meet(logits, row_stride * size, V * size, out, V * 4, V * 4, b->n_rows))
    return MK_ERR_INVALID_ARG;
  return MK_OK;
}

static mk_status apply(mk_rules *m, const mk_rules_batch *b, const void *logits, int32_t is_bf16,
                       int64_t row_stride, float *out, int32_t *out_tokens, bool behind_step) {
  const mk_status refused = mk_rules_check(m, b, logits, is_bf16, row_stride, out, out_tokens);
  if (refused != MK_OK) return refused;
  if (b->n_rows == 0) return MK_OK;
  const int64_t size = is_bf16 ? 2 : 4, V = m->vocab;
  OnDevice on(m->dev);
  if (!on.ok) return MK_ERR_CUDA;
  Args a{};
  a.b = *b;
  if (!b->allowed && !b->allowed_rows) a.b.n_masks = 1; /* row masks are not looked at */
  a.vocab = m->vocab;
  a.logits = logits;
  a.row_stride = row_stride;
  a.out = out;
  a.out_tokens = out_tokens;
  a.behind_step = behind_step;
  a.err = m->err;
  a.best = (unsigned long long *)(m->ws + 64);
  a.done = (int32_t *)(m->ws + 32);
  /* slices: no larger than the vocabulary takes, and as large as leaves an SM two items (8 rows of
   * 152064: 13.4 us, with one 16.2, with four 15.6; large slices cost a row less: 384 rows 107 us, with
   * 4096 tokens a slice 144).  Lists where rows are many, but not in the smallest slices, where most
   * tokens have a word (2048 rows of 1000: a list cost the kernel half as much again when it was one of
   * 47 us, 69; now 35). */
  a.slice = kSlice;
  while (a.slice > kLeast && a.slice / 2 >= V) a.slice /= 2;
  auto items = [&] { return (V + a.slice - 1) / a.slice * b->n_rows; };
  const bool list = a.slice >= 4 * kLeast && items() >= 2 * m->n_sm;
  while (a.slice > kLeast && items() < 2 * m->n_sm) a.slice /= 2;
  a.slices = (int32_t)((V + a.slice - 1) / a.slice);
  const bool vec = V % 4 == 0 && row_stride % 4 == 0 && aligned(logits, 4 * (unsigned)size) && aligned(out, 16);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((int64_t)a.slices * b->n_rows, m->n_sm * blocks_of(vec)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = list ? words_bytes(a.slice) : (size_t)a.slice * 4;
  cfg.stream = m->stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel_of(is_bf16 != 0, vec, a.slice, list), a) == cudaSuccess ? MK_OK : MK_ERR_CUDA;
}

mk_status mk_rules_apply(mk_rules *m, const mk_rules_batch *b, const void *logits, int32_t is_bf16,
                         int64_t row_stride, float *out, int32_t *out_tokens) {
  return apply(m, b, logits, is_bf16, row_stride, out, out_tokens, false);
}

mk_status mk_rules_follow(mk_rules *m, const mk_rules_batch *b, float *logits, int32_t *out_tokens) {
  if (!m || (b && b->n_rows > 0 && !out_tokens)) return MK_ERR_INVALID_ARG;
  return apply(m, b, logits, 0, m->vocab, logits, out_tokens, true);
}

mk_status mk_rules_sync(mk_rules *m) {
  return m ? take_error(m->dev, m->stream, m->err, m->err_host) : MK_ERR_INVALID_ARG;
}

}  // extern "C"
