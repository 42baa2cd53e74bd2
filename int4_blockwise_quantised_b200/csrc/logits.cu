// vv_logits_process: repetition / frequency / presence penalties, biases and a grammar's bit mask
// on a batch of logits, with the greedy token of each row ("vibevoice-asr-bitnet-onnx": greedy
// decode with stop tokens; this is what a transcript's caller puts between lm_head and argmax).
//
//   seen:  x <- x > 0 ? x / r : x * r        n > 0: x <- (x - f n) - p
//   bias:  x <- x + w                        bit 0: x <- -inf
//
// One pass over the logits.  A CTA owns a run of kSlice consecutive tokens of one row; it issues
// the loads of its logits into registers first and, while they are on their way, reads the row's
// whole history, keeping what falls into its run: one bit per token in shared memory says whether
// it occurs, and only the counters of generated tokens are ever touched.  Equal ids of a warp are
// counted by one lane (match) and a set bit is not set again, so thousands of equal ids (a
// prompt's audio span) do not serialise on one address.  The greedy token goes through one 64-bit
// maximum per row: (order-preserving bits of x, inverted token), whose result does not depend on
// the order of arrival and picks the lowest token on ties; the last CTA of a row writes it and
// leaves the workspace zero.
//
// Bound by HBM: 8 bytes per logit (fp32), the history and mask are a few per cent.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "vv_device.cuh"
#include "vv_internal.h"

namespace vv {
namespace {

constexpr int kLogitThreads = 512;
constexpr int kPer = 16;                        // logits per thread, in registers
constexpr int kSlice = kLogitThreads * kPer;    // 8192 tokens of a row per CTA

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
  int V, words;
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

template <typename T>
__global__ void __launch_bounds__(kLogitThreads, 3) logits_process_kernel(const __grid_constant__ LogitsArgs a) {
  constexpr int VEC = 16 / sizeof(T);   // elements of a 16-byte load
  constexpr int NV = kPer / VEC;        // such loads per thread
  extern __shared__ __align__(16) unsigned char lsm[];
  __shared__ unsigned long long warp_key[kLogitThreads / 32];
  const bool history = a.r.tokens != nullptr, biased = a.r.bias_ids != nullptr;
  unsigned* count = reinterpret_cast<unsigned*>(lsm);                              // [kSlice]
  unsigned* bias = reinterpret_cast<unsigned*>(lsm + (history ? kSlice * 4 : 0));  // [kSlice]
  __shared__ unsigned bits[3][kSlice / 32];
  constexpr int kSeen = 0, kSaid = 1, kBias = 2;
  const int b = blockIdx.y, v0 = blockIdx.x * kSlice, tid = threadIdx.x;
  const int nv = min(kSlice, a.V - v0);
  const T* in = static_cast<const T*>(a.in) + (int64_t)b * a.in_stride + v0;
  T* out = static_cast<T*>(a.out) + (int64_t)b * a.out_stride + v0;
  // rows of odd length or stride are not 16-byte aligned: those rows move element by element
  const bool wide = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;

  __align__(16) T x[kPer];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = (j * kLogitThreads + tid) * VEC;
    if (wide && e0 + VEC <= nv) {
      *reinterpret_cast<uint4*>(&x[j * VEC]) = *reinterpret_cast<const uint4*>(in + e0);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e0 + e < nv) x[j * VEC + e] = in[e0 + e];
    }
  }

  const float rep = history && a.r.repetition ? a.r.repetition[b] : 1.f;
  const float freq = history && a.r.frequency ? a.r.frequency[b] : 0.f;
  const float pres = history && a.r.presence ? a.r.presence[b] : 0.f;
  const uint32_t* mask = a.r.mask ? a.r.mask + (int64_t)b * a.r.mask_stride : nullptr;
  unsigned allow[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    // the first of VEC (4 or 8) tokens is a multiple of it: their bits lie in one word
    const int e0 = v0 + (j * kLogitThreads + tid) * VEC;
    allow[j] = mask && e0 < a.V ? mask[e0 >> 5] >> (e0 & 31) : 0xffffffffu;
  }

  // which tokens of the run the history and the biases name: one bit each, so that nothing else has
  // to be cleared, and a run of logits without any is only masked and copied
  bool bad = false;
  int plen = 0, len = 0, i0 = 0, i1 = 0;
  const int32_t* tok = nullptr;
  if (history) {
    const int raw = a.r.token_lens[b], raw_p = a.r.prompt_lens ? a.r.prompt_lens[b] : 0;
    len = min(max(raw, 0), a.r.max_tokens);
    plen = min(max(raw_p, 0), len);
    bad = raw != len || raw_p < 0 || raw_p > a.r.max_tokens;
    tok = a.r.tokens + (int64_t)b * a.r.tokens_stride;
  }
  if (biased) {
    const int raw0 = a.r.bias_offsets[b], raw1 = a.r.bias_offsets[b + 1];
    i0 = min(max(raw0, 0), a.r.n_bias);
    i1 = min(max(raw1, i0), a.r.n_bias);
    bad = bad || raw0 != i0 || raw1 != i1;
  }
  if (bad && tid == 0 && blockIdx.x == 0) set_device_error(VV_ERR_RANGE);
  if (history || biased) {
    for (int i = tid; i < 3 * kSlice / 32; i += kLogitThreads) (&bits[0][0])[i] = 0;
    __syncthreads();
    // a prompt may hold one id thousands of times: the bit is looked at before it is set
    auto mark = [&](int which, unsigned d) {
      volatile unsigned* word = &bits[which][d >> 5];
      if (!((*word >> (d & 31)) & 1)) atomicOr(&bits[which][d >> 5], 1u << (d & 31));
    };
    constexpr int kMany = 4;  // ids of a thread on their way at once
    for (int j0 = 0; j0 < len; j0 += kMany * kLogitThreads) {
      unsigned t[kMany];
#pragma unroll
      for (int j = 0; j < kMany; ++j) {
        const int i = j0 + j * kLogitThreads + tid;
        t[j] = i < len ? (unsigned)tok[i] - (unsigned)v0 : 0xffffffffu;
      }
#pragma unroll
      for (int j = 0; j < kMany; ++j) {
        if (t[j] >= (unsigned)nv) continue;
        if (j0 + j * kLogitThreads + tid < plen) {
          mark(kSeen, t[j]);
        } else {
          mark(kSaid, t[j]);
          count[t[j]] = 0;
        }
      }
    }
    for (int i = i0 + tid; i < i1; i += kLogitThreads) {
      const unsigned d = (unsigned)a.r.bias_ids[i] - (unsigned)v0;
      if (d < (unsigned)nv) {
        mark(kBias, d);
        bias[d] = 0;
      }
    }
    __syncthreads();
    for (int j0 = plen; j0 < len; j0 += kLogitThreads) {  // whole warps, for the match
      const int i = j0 + tid;
      unsigned d = i < len ? (unsigned)tok[i] - (unsigned)v0 : 0xffffffffu;
      if (d >= (unsigned)nv) d = 0xffffffffu;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d != 0xffffffffu && (tid & 31) == __ffs(same) - 1) atomicAdd(&count[d], __popc(same));
    }
    // an id named twice keeps its last value: the entry of the largest index wins
    for (int i = i0 + tid; i < i1; i += kLogitThreads) {
      const unsigned d = (unsigned)a.r.bias_ids[i] - (unsigned)v0;
      if (d < (unsigned)nv) atomicMax(&bias[d], (unsigned)i);
    }
    __syncthreads();
  }

  unsigned long long best = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e0 = (j * kLogitThreads + tid) * VEC;
    if (e0 >= nv) continue;
    const unsigned allowed = allow[j];
    unsigned seen = 0, said = 0, named = 0;
    if (history || biased) {
      seen = bits[kSeen][e0 >> 5] >> (e0 & 31);
      said = bits[kSaid][e0 >> 5] >> (e0 & 31);
      named = bits[kBias][e0 >> 5] >> (e0 & 31);
    }
    const bool any = ((seen | said | named) & ((1u << VEC) - 1)) != 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int i = e0 + e;
      if (i >= nv) break;
      float y = to_f32<T>(x[j * VEC + e]);
      if (any) {
        if (((seen | said) >> e) & 1) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
        if ((said >> e) & 1) y = __fsub_rn(__fsub_rn(y, __fmul_rn(freq, (float)count[i])), pres);
        if ((named >> e) & 1) y = __fadd_rn(y, a.r.bias_vals[bias[i]]);
      }
      if (!((allowed >> e) & 1)) y = -INFINITY;
      x[j * VEC + e] = from_f32<T>(y);
      if (y > -INFINITY) {
        const unsigned long long key = ((unsigned long long)ordered_bits(y) << 32) | (0xffffffffu - (unsigned)(v0 + i));
        best = key > best ? key : best;
      }
    }
    if (wide && e0 + VEC <= nv) {
      *reinterpret_cast<uint4*>(out + e0) = *reinterpret_cast<const uint4*>(&x[j * VEC]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e0 + e < nv) out[e0 + e] = x[j * VEC + e];
    }
  }
  if (!a.argmax) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
    best = other > best ? other : best;
  }
  if ((tid & 31) == 0) warp_key[tid >> 5] = best;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kLogitThreads / 32; ++w) best = warp_key[w] > best ? warp_key[w] : best;
    RowBest* row = a.ws + b;
    if (gridDim.x > 1) {
      if (best) atomicMax(&row->key, best);
      __threadfence();
      if (atomicAdd(&row->arrived, 1u) != gridDim.x - 1) return;
      __threadfence();
      best = atomicExch(&row->key, 0ull);
      row->arrived = 0;
    }
    a.argmax[b] = best ? (int)(0xffffffffu - (unsigned)best) : -1;
  }
}

template <typename T>
cudaError_t launch_logits(const LogitsArgs& a, int B, cudaStream_t s) {
  const size_t smem = (a.r.tokens ? kSlice * 4 : 0) + (a.r.bias_ids ? kSlice * 4 : 0);
  cudaError_t e = cudaFuncSetAttribute(logits_process_kernel<T>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSlice * 8);
  if (e != cudaSuccess) return e;
  logits_process_kernel<T><<<dim3((a.V + kSlice - 1) / kSlice, B), kLogitThreads, smem, s>>>(a);
  return cudaGetLastError();
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
  a.words = words;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = dtype == VV_F32   ? vv::launch_logits<float>(a, B, s)
                  : dtype == VV_F16 ? vv::launch_logits<__half>(a, B, s)
                                    : vv::launch_logits<__nv_bfloat16>(a, B, s);
  return vv::cuda_check(e, "vv_logits_process launch");
}
