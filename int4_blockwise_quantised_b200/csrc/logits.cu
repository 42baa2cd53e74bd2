// vv_logits_process: repetition / frequency / presence penalties, biases and a grammar's bit mask
// on a batch of logits, with the greedy token of each row ("vibevoice-asr-bitnet-onnx": greedy
// decode with stop tokens; this is what a transcript's caller puts between lm_head and argmax).
//
//   seen:  x <- x > 0 ? x / r : x * r        n > 0: x <- (x - f n) - p
//   bias:  x <- x + w                        bit 0: x <- -inf
//
// One pass over the logits.  A CTA owns a slice of consecutive tokens of one row; it asks for the
// row's first ids and biases, then for its logits, all into registers, and looks through the row's
// whole history for what falls into its slice: one bit per token in shared memory says whether it
// occurs, and only the counters of generated tokens are ever touched.  Equal ids of a warp are
// counted by one lane (match) and a set bit is not set again, so thousands of equal ids (a
// prompt's audio span) do not serialise on one address.  The greedy token goes through one 64-bit
// maximum per row: (order-preserving bits of x, inverted token), whose result does not depend on
// the order of arrival and picks the lowest token on ties; the last CTA of a row writes it and
// leaves the workspace zero.
//
// 8 bytes per logit (fp32), history and mask a few per cent: 64 rows of 152064 take 12.4 us at the
// copy's rate, here 26.1 (3.1 TB/s): 19.5 without any rule (copy and maximum, 7.6 M instructions), 1.1 for
// the mask, 1.5 for 300 biases a row, 4 for the 4785 ids of a row, which every slice looks through (2.4 M
// of 12.3 M instructions).  What bounds it is the chain of a CTA (ids and logits, marks, counts, dense
// pass, named tokens, each behind a barrier); one row is a chain of latencies (6.3 us).  In fp16 or bf16
// it takes 23.1 us.  Rows that do not begin on 16 bytes move element by element: 64 rows of 152063 take
// 29 us in fp32, 44 in fp16.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vv_device.cuh"
#include "vv_internal.h"

namespace vv {
namespace {


struct RowBest {
  unsigned long long key;  // 0: nothing above -inf so far
  unsigned arrived;
  unsigned pad;
};

struct LogitsArgs {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;
  vv_logits_rules r;
  int32_t* argmax;
  RowBest* ws;
  int V;
  bool packed;  // counts and biases share a word
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Bits of x in an order-preserving unsigned form (-0 counts as +0); > 0 for every x above -inf.
__device__ __forceinline__ unsigned ordered_bits(float x) {
  const unsigned u = __float_as_uint(x + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// A load that stays where it is written (the compiler moves plain ones down to their use).
__device__ __forceinline__ unsigned load_now(const int32_t* p) {
  unsigned v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

template <typename T, int kThreads, int kPer>  // kPer: logits per thread, in registers
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logits_process_kernel(const __grid_constant__ LogitsArgs a) {
  constexpr int kSlice = kThreads * kPer;  // tokens of a row per CTA
  constexpr int VEC = 16 / sizeof(T);   // elements of a 16-byte load
  constexpr int NV = kPer / VEC;        // such loads per thread
  extern __shared__ __align__(16) unsigned char lsm[];
  __shared__ unsigned long long warp_key[kThreads / 32];
  constexpr int kNear = 512 / kThreads;  // biases of a thread in registers
  __shared__ float bias_val[kNear * kThreads];
  const bool history = a.r.tokens != nullptr, biased = a.r.bias_ids != nullptr;
  // per token of the run: how often it was generated, and which of the row's biases it has; in one
  // word when both fit 16 bits (history and biases of at most 65535 entries)
  unsigned* count = reinterpret_cast<unsigned*>(lsm);                                         // [kSlice]
  unsigned* bias = reinterpret_cast<unsigned*>(lsm + (history && !a.packed ? kSlice * 4 : 0));  // [kSlice]
  const int bias_shift = a.packed ? 16 : 0;
  const unsigned count_mask = a.packed ? 0xffffu : 0xffffffffu;
  __shared__ __align__(16) unsigned bits[kSlice / 32][4];  // a bit per token: seen, said, has a bias; allowed
  constexpr int kSeen = 0, kSaid = 1, kBias = 2;
  const int b = blockIdx.y, v0 = blockIdx.x * kSlice, tid = threadIdx.x;
  const int nv = min(kSlice, a.V - v0);
  const T* in = static_cast<const T*>(a.in) + (int64_t)b * a.in_stride + v0;
  T* out = static_cast<T*>(a.out) + (int64_t)b * a.out_stride + v0;
  // rows of odd length or stride are not 16-byte aligned: those rows move element by element
  const bool wide = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;

  // what is needed first is asked for first: the row's scalars, its first ids (whatever its length:
  // the row is max_tokens wide), its mask, then the logits
  const float rep = history && a.r.repetition ? a.r.repetition[b] : 1.f;
  const float freq = history && a.r.frequency ? a.r.frequency[b] : 0.f;
  const float pres = history && a.r.presence ? a.r.presence[b] : 0.f;
  const uint32_t* mask = a.r.mask ? a.r.mask + (int64_t)b * a.r.mask_stride : nullptr;
  const int32_t* tok = history ? a.r.tokens + (int64_t)b * a.r.tokens_stride : nullptr;
  const int width = history ? a.r.max_tokens : 0;
  // ids of a thread in registers: one round trip to memory for most rows, and the second pass over
  // them (the counting) needs none.  Ten are what 64 registers a thread (two CTAs of 512) leave room
  // for beside 24 logits, 5120 of a row together; a longer history is read twice (64 rows: 26.8 us for
  // 5119 ids, 27.6 for 5121, 32.0 for 9421)
  constexpr int kMany = 5120 / kThreads;
  unsigned t[kMany];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kMany; ++j) {
      const int i = j0 + j * kThreads + tid;
      t[j] = (unsigned)v0 - 1u;  // outside the run
      if (i < width) t[j] = load_now(tok + i);
    }
#pragma unroll
    for (int j = 0; j < kMany; ++j) t[j] -= (unsigned)v0;
  };
  fetch(0);
  bool bad = false;
  int plen = 0, len = 0, i0 = 0, i1 = 0;
  if (history) {
    const int raw = a.r.token_lens[b], raw_p = a.r.prompt_lens ? a.r.prompt_lens[b] : 0;
    len = min(max(raw, 0), a.r.max_tokens);
    plen = min(max(raw_p, 0), len);
    bad = raw != len || raw_p < 0 || raw_p > a.r.max_tokens;
  }
  if (biased) {
    const int raw0 = a.r.bias_offsets[b], raw1 = a.r.bias_offsets[b + 1];
    i0 = min(max(raw0, 0), a.r.n_bias);
    i1 = min(max(raw1, i0), a.r.n_bias);
    bad = bad || raw0 != i0 || raw1 != i1;
  }
  // the row's first biases
  unsigned near_id[kNear];
  float near_val[kNear];
#pragma unroll
  for (int k = 0; k < kNear; ++k) {
    const int i = i0 + k * kThreads + tid;
    near_id[k] = (unsigned)v0 - 1u;  // outside the run
    near_val[k] = 0.f;
    if (i < i1) {
      near_id[k] = load_now(a.r.bias_ids + i);
      near_val[k] = __uint_as_float(load_now(reinterpret_cast<const int32_t*>(a.r.bias_vals + i)));
    }
  }
  static_assert(kSlice / 32 <= kThreads, "at most a word of the mask per thread");
  const bool has_word = kSlice / 32 == kThreads || tid < kSlice / 32;
  const int left = has_word ? nv - tid * 32 : 0;
  // tokens past the row's end are barred like masked ones
  unsigned allowed = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1 : 0u;
  if (mask && left > 0) allowed &= mask[(v0 >> 5) + tid];
  const bool vec = wide && nv % VEC == 0;
  __align__(16) T x[kPer];
  if (vec) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = (j * kThreads + tid) * VEC;
      *reinterpret_cast<uint4*>(&x[j * VEC]) = e0 < nv ? *reinterpret_cast<const uint4*>(in + e0) : make_uint4(0, 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e0 = (j * kThreads + tid) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[j * VEC + e] = e0 + e < nv ? in[e0 + e] : from_f32<T>(0.f);
    }
  }

  if (bad && tid == 0 && blockIdx.x == 0) set_device_error(VV_ERR_RANGE);
  // which tokens of the run the history and the biases name: one bit each, so that nothing else has
  // to be cleared, and logits without any are only masked and copied
  if (has_word) *reinterpret_cast<uint4*>(bits[tid]) = make_uint4(0, 0, 0, allowed);
  __syncthreads();
  if (history || biased) {
    // a prompt may hold one id thousands of times: the bit is looked at before it is set
    auto mark = [&](int which, unsigned d) {
      volatile unsigned* word = &bits[d >> 5][which];
      if (!((*word >> (d & 31)) & 1)) atomicOr(&bits[d >> 5][which], 1u << (d & 31));
    };
    constexpr int kGroup = kMany % 4 == 0 ? 4 : 5;
    static_assert(kMany % kGroup == 0, "whole groups");
    constexpr int kRound = kMany * kThreads;
    for (int j0 = 0; j0 < len; j0 += kRound) {
      if (j0 > 0) fetch(j0);
#pragma unroll
      for (int g = 0; g < kMany; g += kGroup) {
        if (j0 + g * kThreads >= len) break;
        // mostly none of the group falls into the run
        unsigned least = t[g];
#pragma unroll
        for (int j = g + 1; j < g + kGroup; ++j) least = min(least, t[j]);
        if (least >= (unsigned)nv) continue;
#pragma unroll
        for (int j = g; j < g + kGroup; ++j) {
          const int i = j0 + j * kThreads + tid;
          if (t[j] >= (unsigned)nv || i >= len) continue;
          if (i < plen) {
            mark(kSeen, t[j]);
          } else {
            mark(kSaid, t[j]);
            count[t[j]] = 0;
          }
        }
      }
    }
    // f(entry, token of the run): the biases that fall into it
    auto each_bias = [&](auto&& f) {
#pragma unroll
      for (int k = 0; k < kNear; ++k) {
        const unsigned d = near_id[k] - (unsigned)v0;
        if (d < (unsigned)nv) f(k * kThreads + tid, d);
      }
      for (int i = i0 + kNear * kThreads + tid; i < i1; i += kThreads) {
        const unsigned d = (unsigned)a.r.bias_ids[i] - (unsigned)v0;
        if (d < (unsigned)nv) f(i - i0, d);
      }
    };
#pragma unroll
    for (int k = 0; k < kNear; ++k) bias_val[k * kThreads + tid] = near_val[k];
    each_bias([&](int, unsigned d) {
      mark(kBias, d);
      bias[d] = 0;
    });
    __syncthreads();
    // an id named twice keeps its last value: the entry of the largest index wins
    each_bias([&](int k, unsigned d) { atomicMax(&bias[d], (unsigned)k << bias_shift); });
    if (bias_shift) __syncthreads();
    for (int j0 = plen / kRound * kRound; j0 < len; j0 += kRound) {
      if (len > kRound) fetch(j0);
#pragma unroll
      for (int j = 0; j < kMany; ++j) {
        if (j0 + (j + 1) * kThreads <= plen || j0 + j * kThreads >= len) continue;  // the prompt's, or none
        const int i = j0 + j * kThreads + tid;
        const unsigned d = t[j] < (unsigned)nv && i >= plen && i < len ? t[j] : 0xffffffffu;
        if (!__any_sync(0xffffffffu, d != 0xffffffffu)) continue;
        const unsigned same = __match_any_sync(0xffffffffu, d);
        if (d != 0xffffffffu && (tid & 31) == __ffs(same) - 1) atomicAdd(&count[d], __popc(same));
      }
    }
    __syncthreads();
  }

  // All logits: copied, barred ones as -inf.  The best of those without a rule of their own: strictly
  // larger only, so the lowest token of equals (a thread's tokens ascend).
  float best = -INFINITY;
  int best_at = 0;
  constexpr unsigned kAll = (1u << VEC) - 1;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = (j * kThreads + tid) * VEC;  // its VEC (4 or 8) bits lie in one word
    const uint4 word = *reinterpret_cast<const uint4*>(bits[e0 >> 5]);
    const unsigned named = (word.x | word.y | word.z) >> (e0 & 31), barred = ~(word.w >> (e0 & 31));
    float y[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) y[e] = to_f32<T>(x[j * VEC + e]);
    if ((named | barred) & kAll) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if ((barred >> e) & 1) x[j * VEC + e] = from_f32<T>(-INFINITY);
        if (((named | barred) >> e) & 1) y[e] = -INFINITY;
      }
    }
    if (vec) {
      if (e0 < nv) *reinterpret_cast<uint4*>(out + e0) = *reinterpret_cast<const uint4*>(&x[j * VEC]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e0 + e < nv) out[e0 + e] = x[j * VEC + e];
    }
    float top = y[0];
#pragma unroll
    for (int e = 1; e < VEC; ++e) top = fmaxf(top, y[e]);  // NaN only where all are
    if (top > best) {
      best = top;
#pragma unroll
      for (int e = VEC - 1; e >= 0; --e)
        if (y[e] == top) best_at = v0 + e0 + e;
    }
  }
  // The few that the history or a bias names, a word of 32 tokens per thread; their logits stand
  // unchanged where they were read (in place: as the copy just written).
  if (history || biased) {
    __syncthreads();
    const uint4 word = has_word ? *reinterpret_cast<const uint4*>(bits[tid]) : make_uint4(0, 0, 0, 0);
    for (unsigned rest = (word.x | word.y | word.z) & word.w; rest; rest &= rest - 1) {
      const unsigned bit = rest & -rest;
      const int d = tid * 32 + __ffs(rest) - 1;
      float y = to_f32<T>(in[d]);
      if ((word.x | word.y) & bit) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
      if (word.y & bit) y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, (float)(count[d] & count_mask))), pres);
      if (word.z & bit) {
        const unsigned k = bias[d] >> bias_shift;
        y = __fadd_rn(y, k < kNear * kThreads ? bias_val[k] : a.r.bias_vals[i0 + k]);
      }
      out[d] = from_f32<T>(y);
      if (y > best || (y == best && v0 + d < best_at)) {
        best = y;
        best_at = v0 + d;
      }
    }
  }
  if (!a.argmax) return;
  // the warp's best: the largest value, then the lowest of its tokens
  const unsigned mine = best > -INFINITY ? ordered_bits(best) : 0u;
  const unsigned top = __reduce_max_sync(0xffffffffu, mine);
  const unsigned at = __reduce_min_sync(0xffffffffu, mine == top ? (unsigned)best_at : 0xffffffffu);
  unsigned long long key = top ? ((unsigned long long)top << 32) | (0xffffffffu - at) : 0ull;
  if ((tid & 31) == 0) warp_key[tid >> 5] = key;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kThreads / 32; ++w) key = warp_key[w] > key ? warp_key[w] : key;
    RowBest* row = a.ws + b;
    if (gridDim.x > 1) {
      if (key) atomicMax(&row->key, key);
      __threadfence();
      if (atomicAdd(&row->arrived, 1u) != gridDim.x - 1) return;
      __threadfence();
      key = atomicExch(&row->key, 0ull);
      row->arrived = 0;
    }
    a.argmax[b] = key ? (int)(0xffffffffu - (unsigned)key) : -1;
  }
}

template <typename T, int THREADS, int PER>
cudaError_t launch_slices(const LogitsArgs& a, int B, cudaStream_t s) {
  constexpr int kSlice = THREADS * PER;
  const size_t smem = (a.r.tokens ? kSlice * 4 : 0) + (a.r.bias_ids && !a.packed ? kSlice * 4 : 0);
  const cudaError_t e = allow_smem<logits_process_kernel<T, THREADS, PER>>(kSlice * 8);
  if (e != cudaSuccess) return e;
  logits_process_kernel<T, THREADS, PER><<<dim3((a.V + kSlice - 1) / kSlice, B), THREADS, smem, s>>>(a);
  return cudaGetLastError();
}

// Every CTA reads its row's whole history, so a slice is 12288 tokens (64 rows of 152064 with 4785
// ids: 25.8 us; slices of 8192 / 4096 / 16384 tokens: 26.9-29.8 / 38 / 25.4 us, eight rows 8.9 / 9.5 / 10.3
// where these take 9.2); a few rows take slices of 2048 while these are at
// most two CTAs per SM: 1 / 2 / 4 / 8 such rows take 7.5 / 9.1 / 8.4 / 10.0 us in large slices and 6.6 /
// 8.3 / 8.6 / 11.6 us in small ones.
template <typename T>
cudaError_t launch_logits(const LogitsArgs& a, int B, cudaStream_t s) {
  const int64_t small = (int64_t)B * ((a.V + 2047) / 2048);
  return small <= 2 * sm_count() ? launch_slices<T, 256, 8>(a, B, s) : launch_slices<T, 512, 24>(a, B, s);
}

}  // namespace
}  // namespace vv

extern "C" size_t vv_logits_process_workspace_size(int32_t B) {
  return B >= 1 && B <= 65535 ? (size_t)B * sizeof(vv::RowBest) : 0;
}

extern "C" vv_status vv_logits_process(const void* logits, int64_t logits_stride, int32_t dtype,
                                       int32_t B, int64_t V, const vv_logits_rules* rules,
                                       void* out, int64_t out_stride, int32_t* argmax, void* ws,
                                       size_t ws_bytes, vv_stream stream) {
  VV_CHECK_ARG(logits && rules && out, "vv_logits_process: null pointer");
  VV_CHECK_ARG(dtype == VV_F32 || dtype == VV_F16 || dtype == VV_BF16,
               "vv_logits_process: dtype %d", dtype);
  VV_CHECK_SHAPE(B >= 1 && B <= 65535 && V >= 1 && V < (int64_t(1) << 30),
                 "vv_logits_process: B=%d V=%lld", B, (long long)V);
  VV_CHECK_SHAPE(B == 1 || (logits_stride >= V && out_stride >= V),
                 "vv_logits_process: rows overlap (strides %lld and %lld, V=%lld)",
                 (long long)logits_stride, (long long)out_stride, (long long)V);
  const vv_logits_rules& r = *rules;
  const int64_t size = dtype == VV_F32 ? 4 : 2;
  VV_CHECK_ARG(((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & (size - 1)) == 0,
               "vv_logits_process: logits and out must be aligned to their elements");
  const char *x = static_cast<const char*>(logits), *y = static_cast<const char*>(out);
  const int64_t nx = ((B - 1) * logits_stride + V) * size, ny = ((B - 1) * out_stride + V) * size;
  VV_CHECK_ARG((x == y && (B == 1 || logits_stride == out_stride)) || x + nx <= y || y + ny <= x,
               "vv_logits_process: out must be the logits themselves (same stride) or not overlap "
               "them");
  if (r.tokens) {
    VV_CHECK_ARG(r.token_lens, "vv_logits_process: tokens without token_lens");
    VV_CHECK_SHAPE(r.max_tokens >= 0 && r.max_tokens < (1 << 24) &&
                       (B == 1 || r.tokens_stride >= r.max_tokens),
                   "vv_logits_process: max_tokens=%d tokens_stride=%lld", r.max_tokens,
                   (long long)r.tokens_stride);
  }
  if (r.bias_ids)
    VV_CHECK_ARG(r.bias_vals && r.bias_offsets && r.n_bias >= 0,
                 "vv_logits_process: biases need ids, values, offsets and n_bias >= 0");
  const int words = (int)((V + 31) / 32);
  if (r.mask)
    VV_CHECK_SHAPE(B == 1 || r.mask_stride >= words, "vv_logits_process: mask_stride=%lld (%d words)",
                   (long long)r.mask_stride, words);
  if (argmax) {
    VV_CHECK_ARG(ws && vv::aligned16(ws), "vv_logits_process: workspace null or misaligned");
    const size_t need = vv_logits_process_workspace_size(B);
    if (ws_bytes < need)
      return vv::set_error(VV_ERR_CAPACITY, "vv_logits_process: workspace %zu < %zu", ws_bytes,
                           need);
  }
  vv::LogitsArgs a = {};
  a.in = logits;
  a.out = out;
  a.in_stride = logits_stride;
  a.out_stride = out_stride;
  a.r = r;
  a.argmax = argmax;
  a.ws = static_cast<vv::RowBest*>(ws);
  a.V = (int)V;
  a.packed = r.tokens && r.bias_ids && r.max_tokens < 65536 && r.n_bias < 65536;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == VV_F32   ? vv::launch_logits<float>(a, B, s)
                  : dtype == VV_F16 ? vv::launch_logits<__half>(a, B, s)
                                    : vv::launch_logits<__nv_bfloat16>(a, B, s);
  return vv::cuda_check(e, "vv_logits_process launch");
}
