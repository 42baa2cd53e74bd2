// vv_gqa_prefix_attn: grouped-query attention of one token per sequence over a prompt that all
// sequences share and the pages that each sequence owns ("vibevoice-asr-bitnet-onnx":
// decoder_step attention; "VibeVoice-1.5B — Current Status": several contexts stepped alongside
// each other).
//
//   out[b, h] = sum_t p_t V_t / sum_t p_t,  p_t = exp(scale q . K_t),  t over prompt ++ own pages
//
// Softmax over the union of two key sets splits exactly: with (m, l, o) the maximum, the sum of
// exp(s - m) and the weighted sum of values of each part, the union's are M = max(m_i),
// L = sum l_i e^(m_i - M), O = sum o_i e^(m_i - M).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "attn_shared.h"
#include "vv_device.cuh"
#include "vv_internal.h"

namespace vv {
namespace {

constexpr int D = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------------- own pages
//
// One CTA = one sequence, one key-value head, one of `splits` parts of the keys; its four warps
// take chunks of 16 keys in turn, each through a ring of its own (cp.async, no CTA barrier in the
// loop), so a page may end anywhere at a multiple of 16 and a warp waits for its own loads only.
// The group's query heads (at most 16) are the rows of m16n8k16 products: S = Q K^T with the
// chunk's keys as columns, O += P V with P straight from S's registers.  Decode attention reads
// each key once for at most 16 query rows: 64 floating operations per byte at most, far below
// what the warp-level matrix instruction sustains (about 250 per byte of HBM traffic), so the
// loads are what counts and not the tensor path; a 128-row tile of the 5th-generation one would
// be empty by 7/8 here.
// Rows past the end of a sequence are filled with zeros by the copy itself (whatever a page holds
// there, NaN included, never reaches the sums) and their scores are set to -inf.
constexpr int kOwnWarps = 4;
constexpr int kOwnThreads = kOwnWarps * 32;
constexpr int kOwnStages = 3;
constexpr int kChunk = 16;                            // keys per chunk
constexpr int kChunkBytes = kChunk * D * 2;           // K or V of a chunk
constexpr int kStageBytes = 2 * kChunkBytes;
constexpr int kMinChunks = 16;                        // least chunks of a split
constexpr int kMinShared = 128;                       // least prompt with a kernel of its own

struct SharedAttnArgs {
  const void* q;
  const void* kpre;
  const void* vpre;
  const void* kp;
  const void* vp;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  float* part;       // [B][Hkv][splits][G][kPartRow]: this kernel's parts
  unsigned* arrived; // [B][Hkv]
  const float* pre_part;  // [Hkv][pre_splits][B * G][kPartRow]: the shared prompt's
  int pre_splits;    // 0: the prompt's keys, if any, are read here (kpre, vpre, P)
  int64_t q_stride, out_stride, pre_head, pre_token, page_stride, head_stride, token_stride;
  int B, Hkv, G, P, ps, pages, max_blocks, splits;
  float c;  // scale * log2(e)
};

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// 16 bytes global -> shared; `bytes` = 0 writes zeros and reads nothing
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {  // -inf -> 0; its error is far below a half step of T
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__global__ void __launch_bounds__(kOwnThreads) own_attn_kernel(const __grid_constant__ SharedAttnArgs a) {
  extern __shared__ __align__(128) unsigned char osm[];
  __shared__ int s_last;
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.G;
  const int raw_len = a.lens[b];
  if (raw_len < 0) {  // padding row
    pdl_wait();
    return;
  }
  const int cap = (int)min((int64_t)a.max_blocks * a.ps, (int64_t)0x7fffffff);
  const int len = min(raw_len, cap);
  if (raw_len > cap && tid == 0 && split == 0 && g == 0) set_device_error(VV_ERR_CAPACITY);

  // chunks: the prompt's first, then the sequence's own
  const int npre = a.pre_splits ? 0 : (a.P + kChunk - 1) / kChunk;
  const int nch = npre + (len + kChunk - 1) / kChunk;
  const int per = max((nch + a.splits - 1) / a.splits, kMinChunks);
  const int active = max((nch + per - 1) / per, 1);
  if (split >= active) {
    pdl_wait();
    return;
  }
  const int c0 = split * per, c1 = min(c0 + per, nch);

  const T* kpre = static_cast<const T*>(a.kpre) + (int64_t)g * a.pre_head;
  const T* vpre = static_cast<const T*>(a.vpre) + (int64_t)g * a.pre_head;
  const T* kp = static_cast<const T*>(a.kp) + (int64_t)g * a.head_stride;
  const T* vp = static_cast<const T*>(a.vp) + (int64_t)g * a.head_stride;
  const int32_t* tbl = a.table + (int64_t)b * a.max_blocks;
  const uint32_t ring = smem_u32(osm) + warp * (kOwnStages * kStageBytes);

  // the group's queries as A fragments, 8 steps of 16 dimensions; rows past G are zero
  uint32_t qf[8][4];
  {
    const int r = lane >> 2, kc = (lane & 3) * 2;
    const T* q0 = static_cast<const T*>(a.q) + (int64_t)b * a.q_stride + (int64_t)g * G * D;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = r + (e & 1) * 8, col = s * 16 + kc + (e >> 1) * 8;
        qf[s][e] = row < G ? *reinterpret_cast<const uint32_t*>(q0 + row * D + col) : 0u;
      }
    }
  }

  // page of own chunk c (-1: none); the lookup runs a chunk ahead of the copy that uses it
  auto page_of = [&](int c) {
    if (c < npre || c >= c1) return 0;
    return tbl[(c - npre) * kChunk / a.ps];
  };
  // copies chunk c into ring slot st; returns the number of its keys
  auto issue = [&](int c, int st, int page) {
    const T *ks, *vs;
    int64_t step;
    int keys;
    if (c < npre) {
      keys = min(a.P - c * kChunk, kChunk);
      ks = kpre + (int64_t)c * kChunk * a.pre_token;
      vs = vpre + (int64_t)c * kChunk * a.pre_token;
      step = a.pre_token;
    } else {
      const int p0 = (c - npre) * kChunk;
      keys = min(len - p0, kChunk);
      if (page < 0 || page >= a.pages) {
        keys = 0;
        page = 0;
        if (lane == 0) set_device_error(VV_ERR_RANGE);
      }
      const int64_t at = (int64_t)page * a.page_stride + (int64_t)(p0 % a.ps) * a.token_stride;
      ks = kp + at;
      vs = vp + at;
      step = a.token_stride;
    }
    const uint32_t dst = ring + st * kStageBytes;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = i * 2 + (lane >> 4), c16 = lane & 15;
      const uint32_t n = row < keys ? 16u : 0u;
      const int64_t off = (row < keys ? row : 0) * step + c16 * 8;
      const uint32_t d = dst + row * 256 + ((c16 ^ (row & 7)) << 4);
      cp16(d, ks + off, n);
      cp16(d + kChunkBytes, vs + off, n);
    }
    return keys;
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };

  float o[16][4];
#pragma unroll
  for (int n = 0; n < 16; ++n) {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  }
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  int keys[kOwnStages];
  int c_issue = c0 + warp;
  int page = page_of(c_issue);
#pragma unroll
  for (int s = 0; s < kOwnStages - 1; ++s) {
    const int next = page_of(c_issue + kOwnWarps);
    keys[s] = c_issue < c1 ? issue(c_issue, s, page) : 0;
    commit();
    page = next;
    c_issue += kOwnWarps;
  }
  int st = 0, st_in = kOwnStages - 1;
  for (int ch = c0 + warp; ch < c1; ch += kOwnWarps) {
    const int next = page_of(c_issue + kOwnWarps);
    int k_in = 0;
    if (c_issue < c1) k_in = issue(c_issue, st_in, page);
    commit();
    page = next;
    c_issue += kOwnWarps;
#pragma unroll
    for (int s = 0; s < kOwnStages; ++s)
      if (s == st_in) keys[s] = k_in;
    asm volatile("cp.async.wait_group %0;" ::"n"(kOwnStages - 1) : "memory");
    __syncwarp();
    int n_keys = 0;
#pragma unroll
    for (int s = 0; s < kOwnStages; ++s)
      if (s == st) n_keys = keys[s];
    const uint32_t kt = ring + st * kStageBytes, vt = kt + kChunkBytes;

    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
    {
      const int row = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        uint32_t r[4];
        ldsm4(r, kt + row * 256 + (((s * 2 + half) ^ (row & 7)) << 4));
        mma16816<T>(s0, qf[s], r[0], r[1]);
        mma16816<T>(s1, qf[s], r[2], r[3]);
      }
    }
    // s0: keys 2 (lane % 4) + {0, 1} of rows lane / 4 and lane / 4 + 8; s1: the same, keys + 8
    const int col = (lane & 3) * 2;
    float x[2][4];
    x[0][0] = col < n_keys ? s0[0] * a.c : -INFINITY;
    x[0][1] = col + 1 < n_keys ? s0[1] * a.c : -INFINITY;
    x[0][2] = col + 8 < n_keys ? s1[0] * a.c : -INFINITY;
    x[0][3] = col + 9 < n_keys ? s1[1] * a.c : -INFINITY;
    x[1][0] = col < n_keys ? s0[2] * a.c : -INFINITY;
    x[1][1] = col + 1 < n_keys ? s0[3] * a.c : -INFINITY;
    x[1][2] = col + 8 < n_keys ? s1[2] * a.c : -INFINITY;
    x[1][3] = col + 9 < n_keys ? s1[3] * a.c : -INFINITY;
    float corr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[h], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;  // nothing above -inf yet: all weights 0
      corr[h] = exp2_fast(m[h] - ref);
      m[h] = mn;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[h][e] = exp2_fast(x[h][e] - ref);
      l[h] = l[h] * corr[h] + ((x[h][0] + x[h][1]) + (x[h][2] + x[h][3]));
    }
    if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        o[n][0] *= corr[0];
        o[n][1] *= corr[0];
        o[n][2] *= corr[1];
        o[n][3] *= corr[1];
      }
    }
    const uint32_t p[4] = {pack_pair<T>(x[0][0], x[0][1]), pack_pair<T>(x[1][0], x[1][1]),
                           pack_pair<T>(x[0][2], x[0][3]), pack_pair<T>(x[1][2], x[1][3])};
    {
      const int row = lane & 15, half = lane >> 4;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t r[4];
        ldsm4t(r, vt + row * 256 + (((n * 2 + half) ^ (row & 7)) << 4));
        mma16816<T>(o[2 * n], p, r[0], r[1]);
        mma16816<T>(o[2 * n + 1], p, r[2], r[3]);
      }
    }
    __syncwarp();
    st = st + 1 == kOwnStages ? 0 : st + 1;
    st_in = st_in + 1 == kOwnStages ? 0 : st_in + 1;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // the warps' partials meet in shared memory (over the rings)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  float* sp = reinterpret_cast<float*>(osm);  // [warps][G][kPartRow]
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = (lane >> 2) + h * 8;
    if (row < G) {
      float* d = sp + (warp * G + row) * kPartRow;
#pragma unroll
      for (int n = 0; n < 16; ++n)
        *reinterpret_cast<float2*>(d + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
      if ((lane & 3) == 0) {
        d[D] = m[h];
        d[D + 1] = l[h];
      }
    }
  }
  __syncthreads();
  // A warp joins a row at a time, four dimensions a lane.  Of each set of parts the maxima and sums
  // are read 32 at a time, one a lane, then the rows one after the other: two round trips to L2
  // for up to 32 parts.
  struct Joined {
    float m, l;
    float4 o;
  };
  auto absorb = [&](Joined& r, const float* parts, int n, int64_t stride) {
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int cnt = min(n - i0, 32);
      const float* base = parts + i0 * stride;
      const float2 ml = lane < cnt ? *reinterpret_cast<const float2*>(base + lane * stride + D)
                                   : make_float2(-INFINITY, 0.f);
      const float mn = fmaxf(r.m, warp_max(ml.x)), ref = mn == -INFINITY ? 0.f : mn;
      const float w0 = exp2_fast(r.m - ref), w = exp2_fast(ml.x - ref);
      r.m = mn;
      r.l = r.l * w0 + warp_sum(lane < cnt ? w * ml.y : 0.f);
      r.o = make_float4(r.o.x * w0, r.o.y * w0, r.o.z * w0, r.o.w * w0);
#pragma unroll 4
      for (int i = 0; i < cnt; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float4 v = *reinterpret_cast<const float4*>(base + i * stride + lane * 4);
        r.o = make_float4(fmaf(wi, v.x, r.o.x), fmaf(wi, v.y, r.o.y), fmaf(wi, v.z, r.o.z), fmaf(wi, v.w, r.o.w));
      }
    }
  };
  const int64_t item = (int64_t)b * a.Hkv + g;
  float* part = a.part + item * a.splits * G * kPartRow;
  if (active > 1) {
    for (int row = warp; row < G; row += kOwnWarps) {
      Joined r = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      absorb(r, sp + row * kPartRow, kOwnWarps, (int64_t)G * kPartRow);
      float* d = part + ((int64_t)split * G + row) * kPartRow;
      *reinterpret_cast<float4*>(d + lane * 4) = r.o;
      if (lane == 0) *reinterpret_cast<float2*>(d + D) = make_float2(r.m, r.l);
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) s_last = atomicAdd(&a.arrived[item], 1u) == (unsigned)(active - 1);
    __syncthreads();
    if (!s_last) {
      pdl_wait();
      return;
    }
    __threadfence();
    if (tid == 0) a.arrived[item] = 0;
  }
  pdl_wait();  // the prompt's parts are complete
  for (int row = warp; row < G; row += kOwnWarps) {
    Joined r = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (active > 1)
      absorb(r, part + row * kPartRow, active, (int64_t)G * kPartRow);
    else
      absorb(r, sp + row * kPartRow, kOwnWarps, (int64_t)G * kPartRow);
    const int64_t rows = (int64_t)a.B * G;
    absorb(r, a.pre_part + ((int64_t)g * a.pre_splits * rows + (int64_t)b * G + row) * kPartRow, a.pre_splits, rows * kPartRow);
    const int h = g * G + row;
    // l is 0 where no key has a weight; a NaN score makes l NaN and goes on to the result
    const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
    T* dst = static_cast<T*>(a.out) + (int64_t)b * a.out_stride + h * D + lane * 4;
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_pair<T>(r.o.x * inv, r.o.y * inv), pack_pair<T>(r.o.z * inv, r.o.w * inv));
    if (a.lse && lane == 0)
      a.lse[(int64_t)b * a.Hkv * G + h] = r.l == 0.f ? -INFINITY : (r.m + log2f(r.l)) * kLn2;
  }
}

// Parts per (sequence, head): enough CTAs for two per SM, none with fewer than kMinChunks chunks.
int own_splits(int B, int Hkv, int64_t keys) {
  const int64_t want = std::max<int64_t>(1, 2 * sm_count() / std::max<int64_t>(1, (int64_t)B * Hkv));
  const int64_t most = std::max<int64_t>(1, (keys + kChunk * kMinChunks - 1) / (kChunk * kMinChunks));
  return (int)std::min<int64_t>({want, most, 64});
}

struct Plan {
  int splits, pre_splits, pre_per;
  size_t part, pre_part, total;  // byte offsets in the workspace; the arrival counters come first
};
Plan plan_of(int B, int Hkv, int G, int P, int64_t max_own) {
  Plan p = {};
  // One sequence shares nothing, and a prompt of a few chunks costs less to read again than a
  // second kernel: there the prompt's keys are the first chunks of every sequence.
  const bool shared = B > 1 && P >= kMinShared;
  if (shared) prefix_tc_split(B * G, Hkv, P, &p.pre_splits, &p.pre_per);
  p.splits = own_splits(B, Hkv, max_own + (shared ? 0 : P));
  const size_t row = kPartRow * sizeof(float);
  p.part = ((size_t)B * Hkv * 4 + 255) / 256 * 256;
  p.pre_part = p.part + (p.splits > 1 ? (size_t)B * Hkv * p.splits * G * row : 0);
  p.total = p.pre_part + (size_t)p.pre_splits * B * Hkv * G * row;
  return p;
}

template <typename T>
cudaError_t launch_own(const SharedAttnArgs& a, cudaStream_t s) {
  const size_t smem = std::max<size_t>(kOwnWarps * kOwnStages * kStageBytes,
                                       (size_t)kOwnWarps * a.G * kPartRow * 4);
  cudaError_t e = cudaFuncSetAttribute(own_attn_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  return launch(own_attn_kernel<T>, dim3(a.splits, a.Hkv, a.B), dim3(kOwnThreads), smem, s,
                a.pre_splits > 0, a);
}

bool sizes_ok(int B, int Hq, int Hkv, int D_, int P) {
  return D_ == 128 && B >= 1 && B <= 65535 && Hkv >= 1 && Hkv <= 1024 && Hq >= Hkv &&
         Hq % Hkv == 0 && Hq / Hkv <= 16 && P >= 0 && P < (1 << 24);
}

}  // namespace
}  // namespace vv

extern "C" size_t vv_gqa_prefix_attn_workspace_size(int32_t B, int32_t Hq, int32_t Hkv, int32_t D_,
                                                    int32_t prefix_len, int64_t max_own) {
  if (!vv::sizes_ok(B, Hq, Hkv, D_, prefix_len) || max_own < 0) return 0;
  return vv::plan_of(B, Hkv, Hq / Hkv, prefix_len, max_own).total;
}

extern "C" vv_status vv_gqa_prefix_attn(const void* q, int64_t q_stride, int32_t B, int32_t Hq,
                                        int32_t Hkv, int32_t D_, const void* k_prefix,
                                        const void* v_prefix, int64_t prefix_head_stride,
                                        int64_t prefix_token_stride, int32_t prefix_len,
                                        const vv_paged_kv* kv, const int32_t* block_tables,
                                        int32_t max_blocks, const int32_t* own_lens, float scale,
                                        void* out, int64_t out_stride, float* lse, void* ws,
                                        size_t ws_bytes, vv_stream stream) {
  VV_CHECK_ARG(q && kv && block_tables && own_lens && out && ws, "vv_gqa_prefix_attn: null pointer");
  VV_CHECK_SHAPE(vv::sizes_ok(B, Hq, Hkv, D_, prefix_len),
                 "vv_gqa_prefix_attn: B=%d Hq=%d Hkv=%d D=%d prefix_len=%d", B, Hq, Hkv, D_,
                 prefix_len);
  vv_status st = vv::check_paged_kv(kv, Hkv, D_, "vv_gqa_prefix_attn");
  if (st != VV_OK) return st;
  VV_CHECK_ARG(vv::aligned16(q) && vv::aligned16(k_prefix) && vv::aligned16(v_prefix) &&
                   vv::aligned16(out) && vv::aligned16(ws),
               "vv_gqa_prefix_attn: pointers must be 16-byte aligned");
  VV_CHECK_SHAPE(max_blocks >= 1, "vv_gqa_prefix_attn: max_blocks=%d", max_blocks);
  VV_CHECK_SHAPE(q_stride % 8 == 0 && q_stride >= 0 && out_stride % 8 == 0 &&
                     (B == 1 || out_stride >= (int64_t)Hq * D_),
                 "vv_gqa_prefix_attn: row strides must be multiples of 8 elements and output rows "
                 "must not overlap");
  if (prefix_len > 0) {
    VV_CHECK_ARG(k_prefix && v_prefix, "vv_gqa_prefix_attn: prefix_len %d without a prefix",
                 prefix_len);
    VV_CHECK_SHAPE(prefix_token_stride >= D_ && prefix_token_stride % 8 == 0 &&
                       (Hkv == 1 || prefix_head_stride >= D_) && prefix_head_stride % 8 == 0 &&
                       prefix_token_stride < (int64_t(1) << 38) &&
                       prefix_head_stride < (int64_t(1) << 38),
                   "vv_gqa_prefix_attn: prefix strides %lld, %lld (multiples of 8 elements)",
                   (long long)prefix_head_stride, (long long)prefix_token_stride);
  }
  VV_CHECK_ARG(scale > 0.f && std::isfinite(scale), "vv_gqa_prefix_attn: scale %g", scale);
  const int G = Hq / Hkv;
  const vv::Plan p = vv::plan_of(B, Hkv, G, prefix_len, (int64_t)max_blocks * kv->page_size);
  if (ws_bytes < p.total)
    return vv::set_error(VV_ERR_CAPACITY, "vv_gqa_prefix_attn: workspace %zu < %zu", ws_bytes,
                         p.total);
  vv::SharedAttnArgs a = {};
  a.q = q;
  a.kpre = k_prefix;
  a.vpre = v_prefix;
  a.kp = kv->k;
  a.vp = kv->v;
  a.table = block_tables;
  a.lens = own_lens;
  a.out = out;
  a.lse = lse;
  a.arrived = static_cast<unsigned*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part);
  a.pre_part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.pre_part);
  a.pre_splits = p.pre_splits;
  a.q_stride = q_stride;
  a.out_stride = out_stride;
  a.pre_head = prefix_head_stride;
  a.pre_token = prefix_token_stride;
  a.page_stride = kv->page_stride;
  a.head_stride = kv->head_stride;
  a.token_stride = kv->token_stride;
  a.B = B;
  a.Hkv = Hkv;
  a.G = G;
  a.P = prefix_len;
  a.ps = kv->page_size;
  a.pages = kv->pages;
  a.max_blocks = max_blocks;
  a.splits = p.splits;
  a.c = scale * vv::kLog2e;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.pre_splits) {
    vv::PrefixTcArgs t = {};
    t.q = q;
    t.k = k_prefix;
    t.v = v_prefix;
    t.part = const_cast<float*>(a.pre_part);
    t.q_stride = q_stride;
    t.head = prefix_head_stride;
    t.token = prefix_token_stride;
    t.B = B;
    t.Hkv = Hkv;
    t.G = G;
    t.P = prefix_len;
    t.splits = p.pre_splits;
    t.per = p.pre_per;
    t.c = a.c;
    t.dtype = kv->dtype;
    VV_CUDA(vv::launch_prefix_tc(t, s));
  }
  const cudaError_t e = kv->dtype == VV_F16 ? vv::launch_own<__half>(a, s) : vv::launch_own<__nv_bfloat16>(a, s);
  return vv::cuda_check(e, "vv_gqa_prefix_attn launch");
}
