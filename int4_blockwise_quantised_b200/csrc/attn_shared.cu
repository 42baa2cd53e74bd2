// vv_gqa_prefix_attn: grouped-query attention of one token per sequence over a prompt that all
// sequences share and the pages that each sequence owns ("vibevoice-asr-bitnet-onnx":
// decoder_step attention; "VibeVoice-1.5B — Current Status": several contexts stepped alongside
// each other).
//
//   out[b, h] = sum_t p_t V_t / sum_t p_t,  p_t = exp(scale q . K_t),  t over prompt ++ own pages
//
// Softmax over the union of key sets splits exactly: with (m, l, o) the maximum, the sum of
// exp(s - m) and the weighted sum of values of each part, the union's are M = max(m_i),
// L = sum l_i e^(m_i - M), O = sum o_i e^(m_i - M).  So three kernels, each launched while the one
// before it still runs (programmatic launch): the sequences' own pages, the shared prompt for all
// sequences together (attn_shared_tc.cu, nothing to do with the first; it ends after it), and the
// join of all parts, a warp per output row.  Joining at the end of the first two took longer (17.4 us
// for 16 sequences on a prompt of 4530, 12.8 with the join apart): a few CTAs hold several heads, and a
// head's parts are a dozen dependent reads.
//
// Measured: 2 x (1024 + at most 64) keys, 12 / 2 heads: 8.4 us; 16 x (4530 + 257): 12.8 us; 48 x (32768 +
// 1024), 28 / 4 heads: 46 us (23 GFLOP, 125 MB); 23 x 4785 without a prompt: 23.9 us (92 MB, 3.9 TB/s).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attn_shared.h"
#include "attn_tc.cuh"
#include "pack16.cuh"
#include "vv_device.cuh"
#include "vv_internal.h"

namespace vv {
namespace {

constexpr int D = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------------------------- own pages
//
// All keys of all sequences and key-value heads form one list of 16-key chunks, ordered by
// sequence, head and position; the CTAs (one per SM) take equal runs of it, found from the lengths
// on the device, so ragged batches load every SM alike (each head counts kEnd chunks more, what it
// costs to begin and end one).  A head, or the part of it that lies in a run, ends as partial rows
// (o, m, l) in the workspace; the join kernel puts them together.
//
// One warp walks the run ahead of the others: eight lanes look up eight chunks' pages at a time
// and copy their rows (TMA, 128-byte swizzle) into a ring of 21 chunks, 168 KB on their way per
// SM; it runs across the ends of heads, so neither a new sequence's length and table nor the
// joining of the last one leaves HBM idle.  Seven warps take the chunks in turn, each waiting for
// its own chunk alone.
// The group's query heads (at most 16) are the rows of m16n8k16 products: S = Q K^T with the keys
// as columns, O += P V with P straight from S's registers.  Decode attention reads each key once
// for at most 16 query rows, 64 floating operations per byte at most, far below what the
// warp-level matrix instruction sustains, so the loads are what counts and not the tensor path; a
// 128-row tile of the 5th-generation one would be empty by 7/8 here.
// What a page holds behind a sequence's last key (NaN included) is kept out: those scores are set
// to -inf and those rows of V to zero before the products.
constexpr int kOwnWarps = 7;                          // consumers; one more warp copies
constexpr int kOwnThreads = (kOwnWarps + 1) * 32;
constexpr int kChunk = 16;                            // keys
constexpr int kHalfBytes = kChunk * 128;              // 64 of the 128 dimensions of a chunk
constexpr int kStageBytes = 4 * kHalfBytes;           // K then V
constexpr int kOwnStages = 3 * kOwnWarps;              // a multiple: a stage has one consumer, which
                                                      // sees each of its phases (a parity wait
                                                      // must not be two phases behind)
static_assert(kOwnStages % kOwnWarps == 0, "a stage belongs to one consumer warp");
constexpr int kBatch = 8;                             // chunks copied at a time
static_assert(kBatch <= kOwnStages, "a batch never waits for itself");
constexpr int kEnd = 10;                              // a head's beginning and end, in chunks
constexpr int kMinRun = 4 + kEnd;                     // least places of a run: a short head alone
constexpr int kMinShared = 128;                       // least prompt with a kernel of its own
constexpr int kOwnSmem = kOwnStages * kStageBytes + kOwnWarps * 8 * kPartRow * 4 + 1024;

struct SharedAttnArgs {
  const void* q;
  const int32_t* table;
  const int32_t* lens;
  float* part;       // [B][Hkv][G][kPartRow]: heads that lie in one run
  float* run_part;   // [CTAs][2][G][kPartRow]: a run's first head (begun in an earlier run), its last
  int2* where;       // [B][Hkv]: the run that the head begins in, runs that share it
  bool shared;       // the prompt has a kernel of its own; else its keys, if any, are read here
  int64_t q_stride;
  int B, Hkv, G, P, ps, pages, max_blocks;
  float c;  // scale * log2(e)
};

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
// Copies a chunk of K or of V: both halves of 64 dimensions, 16 rows each.
__device__ __forceinline__ void tma_chunk(uint32_t dst, const CUtensorMap* tm, int token, int head, int page,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3, %2, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(token), "r"(head), "r"(page), "r"(smem_u32(bar))
      : "memory");
}

struct OwnMaps {
  CUtensorMap k, v;        // pages: dims {64, page_size, 2, Hkv, pages}, box {64, 16, 2, 1, 1}
  CUtensorMap kpre, vpre;  // prompt: dims {64, P, 2, Hkv, 1}, the same box; rows past P read as zeros
};

// `total` places in n runs, the first `more` of them a place longer.
struct Runs {
  int64_t len;
  int more;
  __device__ Runs(int64_t total, int n) {
    if (total <= 0x7fffffff) {  // 32-bit division is much shorter
      len = (unsigned)total / (unsigned)n;
      more = (int)((unsigned)total % (unsigned)n);
    } else {
      len = total / n;
      more = (int)(total % n);
    }
  }
  __device__ int64_t begin(int c) const { return c * len + min(c, more); }
  __device__ int of(int64_t x) const {  // the run that holds place x
    const int64_t longer = more * (len + 1);
    return x < longer ? (int)(x / (len + 1)) : more + (int)((x - longer) / len);
  }
};

// Where a warp is in its CTA's run: chunk t of `chunks` of head g of sequence b.
struct Walker {
  int b, g, t, chunks, len;
};
// A row's joined parts, four dimensions a lane.
struct Joined {
  float m, l;
  float4 o;
};

// Joins n parts of a row into r; part(k) points to part k: o[128], m, l.  The maxima and sums of KB
// parts are read one a lane and their rows together, one round trip to memory a batch.
template <int KB, typename F>
__device__ __forceinline__ void absorb(Joined& r, int n, int lane, F&& part) {
  for (int k0 = 0; k0 < n; k0 += KB) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (lane < KB && k0 + lane < n) ml = *reinterpret_cast<const float2*>(part(k0 + lane) + D);
    float4 v[KB];
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + k < n) v[k] = *reinterpret_cast<const float4*>(part(k0 + k) + lane * 4);
    }
    const float mn = fmaxf(r.m, warp_max(ml.x)), ref = mn == -INFINITY ? 0.f : mn;
    const float w0 = tc::ex2_approx(r.m - ref), w = tc::ex2_approx(ml.x - ref);
    r.m = mn;
    r.l = r.l * w0 + warp_sum(w * ml.y);
    r.o = make_float4(r.o.x * w0, r.o.y * w0, r.o.z * w0, r.o.w * w0);
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      r.o = make_float4(fmaf(wk, v[k].x, r.o.x), fmaf(wk, v[k].y, r.o.y), fmaf(wk, v[k].z, r.o.z), fmaf(wk, v[k].w, r.o.w));
    }
  }
}

template <typename T, bool WIDE>  // WIDE: 9 to 16 query heads per key-value head
__global__ void __launch_bounds__(kOwnThreads, 1)
    own_attn_kernel(const __grid_constant__ OwnMaps mp, const __grid_constant__ SharedAttnArgs a) {
  extern __shared__ __align__(1024) unsigned char osm_raw[];
  unsigned char* osm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(osm_raw) + 1023) & ~uintptr_t(1023));
  float* sp = reinterpret_cast<float*>(osm + kOwnStages * kStageBytes);  // [warps][8 rows][kPartRow]
  __shared__ __align__(8) uint64_t full[kOwnStages], empty[kOwnStages];
  __shared__ int64_t warp_sum_s[kOwnThreads / 32];
  __shared__ Walker s_first;
  __shared__ int s_bad[kOwnStages];  // the chunk's page does not exist
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, G = a.G;
  pdl_launch_dependents();  // the next kernels need nothing of this one until their end
  const int cap = (int)min((int64_t)a.max_blocks * a.ps, (int64_t)0x7fffffff);
  const int npre = a.shared ? 0 : (a.P + kChunk - 1) / kChunk;
  if (tid == kOwnWarps * 32) {
    tc::prefetch_map(&mp.k);
    tc::prefetch_map(&mp.v);
  }
  if (tid < kOwnStages) {
    mbar_init(&full[tid], 1);
    mbar_init(&empty[tid], 1);
    fence_mbar_init();
  }
  // chunks of a sequence, per head: a sequence without keys has one empty chunk (its rows are
  // written by whoever holds it), a padding row none
  // (unsigned: a length may be 2^31 - 1)
  auto chunks_of = [&](int len) { return len < 0 ? 0 : max(npre + (int)(((unsigned)min(len, cap) + kChunk - 1) / kChunk), 1); };
  auto places_of = [&](int chunks) { return chunks ? (int64_t)chunks + kEnd : 0; };
  const int per = (a.B + kOwnThreads - 1) / kOwnThreads;
  const int b_lo = min(tid * per, a.B), b_hi = min(b_lo + per, a.B);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) mine += places_of(chunks_of(a.lens[b]));
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += u;
  }
  if (lane == 31) warp_sum_s[warp] = scan;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kOwnThreads / 32; ++w) {
    if (w < warp) before += warp_sum_s[w];
    total += warp_sum_s[w];
  }
  before = (before + scan - mine) * a.Hkv;  // places before this thread's sequences
  total *= a.Hkv;
  // runs: all CTAs, or fewer when the list is short
  const int n_run = (int)min((int64_t)gridDim.x, max(total / kMinRun, (int64_t)1));
  const int cta = blockIdx.x;
  if (total == 0 || cta >= n_run) return;
  const Runs runs(total, n_run);
  const int64_t x0 = runs.begin(cta), x1 = runs.begin(cta + 1);
  if (before <= x0 && x0 < before + mine * a.Hkv) {
    int64_t at = before;
    for (int b = b_lo;; ++b) {
      const int len = a.lens[b], chunks = chunks_of(len);
      const int64_t places = places_of(chunks);
      if (x0 < at + places * a.Hkv) {
        int g = 0;
        for (at += places; at <= x0; at += places) ++g;
        s_first = {b, g, (int)(x0 - (at - places)), chunks, len};
        break;
      }
      at += places * a.Hkv;
    }
  }
  __syncthreads();
  // the parts of heads in this run: f(walker, place of chunk walker.t, chunks here, chunks before)
  auto for_each_head = [&](auto&& f) {
    Walker w = s_first;
    int64_t x = x0;
    int c = 0;
    while (true) {
      if (w.t < w.chunks) {
        const int n = (int)min((int64_t)(w.chunks - w.t), x1 - x);
        f(w, x, n, c);
        c += n;
      }
      x += places_of(w.chunks) - w.t;
      if (x >= x1) return;
      w.t = 0;
      if (++w.g == a.Hkv) {
        w.g = 0;
        do {
          w.len = a.lens[++w.b];
          w.chunks = chunks_of(w.len);
        } while (w.chunks == 0);
      }
    }
  };

  if (warp == kOwnWarps) {
    for_each_head([&](const Walker& w, int64_t, int n, int c) {
      if (w.t == 0 && w.g == 0 && w.len > cap && lane == 0) set_device_error(VV_ERR_CAPACITY);
      const int n_own = min(w.len, cap);
      // lane's chunk of the batch that begins with chunk i: its page, -1 where there is nothing to copy
      auto page_of = [&](int i) {
        const int t = w.t + i + lane;
        if (lane >= kBatch || i + lane >= n) return -1;
        if (t < npre) return 0;
        const int p0 = (t - npre) * kChunk;
        if (p0 >= n_own) return -1;
        int page = a.table[(int64_t)w.b * a.max_blocks + p0 / a.ps];
        if (page < 0 || page >= a.pages) {
          set_device_error(VV_ERR_RANGE);
          page = -2;
        }
        return page;
      };
      int page = page_of(0);
      for (int i = 0; i < n; i += kBatch) {
        const int next = page_of(i + kBatch);  // looked up while this batch waits and is copied
        if (lane < kBatch && i + lane < n) {
          const int t = w.t + i + lane, at = c + i + lane, st = at % kOwnStages, used = at / kOwnStages;
          // the stage's chunk before was copied by an earlier batch: this wait ends by itself
          if (used > 0) wait_phase(&empty[st], (used - 1) & 1);
          s_bad[st] = page == -2;
          mbar_arrive_expect_tx(&full[st], page >= 0 ? kStageBytes : 0);
          if (page >= 0) {
            const bool pre = t < npre;
            const int p0 = (pre ? t : t - npre) * kChunk, tok = pre ? p0 : p0 % a.ps;
            const uint32_t s0 = smem_u32(osm + st * kStageBytes);
            tma_chunk(s0, pre ? &mp.kpre : &mp.k, tok, w.g, page, &full[st]);
            tma_chunk(s0 + 2 * kHalfBytes, pre ? &mp.vpre : &mp.v, tok, w.g, page, &full[st]);
          }
        }
        __syncwarp();
        page = next;
      }
    });
    return;
  }

  auto consumers_sync = [] { asm volatile("bar.sync 1, %0;" ::"n"(kOwnWarps * 32) : "memory"); };
  for_each_head([&](const Walker& w, int64_t x, int n, int c) {
    // the group's queries as A fragments, 8 steps of 16 dimensions; rows past G are zero
    uint32_t qf[8][4];
    {
      const int r = lane >> 2, kc = (lane & 3) * 2;
      const T* q0 = static_cast<const T*>(a.q) + (int64_t)w.b * a.q_stride + (int64_t)w.g * G * D;
#pragma unroll
      for (int s = 0; s < 8; ++s) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = r + (e & 1) * 8, col = s * 16 + kc + (e >> 1) * 8;
          qf[s][e] = (WIDE || !(e & 1)) && row < G ? *reinterpret_cast<const uint32_t*>(q0 + row * D + col) : 0u;
        }
      }
    }
    // fp16 weights are taken 2^14 larger than relative to the maximum, so that those down to 2^-28 keep
    // all their bits; the reference carries it, and the join divides it out.  (2^15 would leave no room
    // below fp16's 65504 for the rounding of a reference in the millions.)
    constexpr float kHeadroom = std::is_same<T, __half>::value ? 14.f : 0.f;
    float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    }
    for (int i = (warp + kOwnWarps - c % kOwnWarps) % kOwnWarps; i < n; i += kOwnWarps) {
      const int st = (c + i) % kOwnStages, t = w.t + i;
      int n_keys = min(t < npre ? a.P - t * kChunk : min(w.len, cap) - (t - npre) * kChunk, kChunk);
      wait_phase(&full[st], ((c + i) / kOwnStages) & 1);
      if (s_bad[st]) n_keys = 0;
      if (n_keys > 0) {
        const uint32_t kt = smem_u32(osm + st * kStageBytes), vt = kt + 2 * kHalfBytes;
        if (n_keys < kChunk) {
          // zero what the page holds behind the last key, 16 bytes a lane
          for (int z = lane + n_keys * 8; z < kChunk * 8; z += 32) {
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + z * 16), "r"(0) : "memory");
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + kHalfBytes + z * 16), "r"(0) : "memory");
          }
          __syncwarp();
        }
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        {
          const int row = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            uint32_t r[4];
            ldsm4(r, kt + (s >> 2) * kHalfBytes + row * 128 + ((((s & 3) * 2 + half) ^ (row & 7)) << 4));
            mma16816<T>(sc[0], qf[s], r[0], r[1]);
            mma16816<T>(sc[1], qf[s], r[2], r[3]);
          }
        }
        // sc[0]: keys 2 (lane % 4) + {0, 1} of rows lane / 4 and lane / 4 + 8; sc[1]: the same, keys + 8
        if (n_keys < kChunk) {
          const int col = (lane & 3) * 2;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (col + (e & 1) >= n_keys) sc[0][e] = -INFINITY;
            if (col + (e & 1) + 8 >= n_keys) sc[1][e] = -INFINITY;
          }
        }
        float corr[2] = {1.f, 1.f};
        uint32_t p[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
          float mx = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float mn = fmaxf(m[h], fmaf(mx, a.c, -kHeadroom));
          const float ref = mn == -INFINITY ? 0.f : mn;  // nothing above -inf yet: all weights 0
          corr[h] = tc::ex2_approx(m[h] - ref);
          m[h] = mn;
          const float w0 = tc::ex2_approx(fmaf(sc[0][2 * h], a.c, -ref)), w1 = tc::ex2_approx(fmaf(sc[0][2 * h + 1], a.c, -ref));
          const float w2 = tc::ex2_approx(fmaf(sc[1][2 * h], a.c, -ref)), w3 = tc::ex2_approx(fmaf(sc[1][2 * h + 1], a.c, -ref));
          l[h] = l[h] * corr[h] + ((w0 + w1) + (w2 + w3));
          p[h] = pack2<T>(w0, w1);
          p[h + 2] = pack2<T>(w2, w3);
        }
        if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            o[k][0] *= corr[0];
            o[k][1] *= corr[0];
            o[k][2] *= corr[1];
            o[k][3] *= corr[1];
          }
        }
        {
          const int row = lane & 15, half = lane >> 4;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t r[4];
            ldsm4t(r, vt + (k >> 2) * kHalfBytes + row * 128 + ((((k & 3) * 2 + half) ^ (row & 7)) << 4));
            mma16816<T>(o[2 * k], p, r[0], r[1]);
            mma16816<T>(o[2 * k + 1], p, r[2], r[3]);
          }
        }
        if (n_keys < kChunk) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the next copy
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }

    // ---- the head ends here, or goes on in the next run: its rows, joined over the warps through
    // shared memory (eight at a time, a row per warp), to where the join kernel looks for them
    const int64_t h0 = x - w.t, h1 = h0 + w.chunks, head = (int64_t)w.b * a.Hkv + w.g;
    const bool begun = h0 >= x0, whole = begun && h1 <= x1;
    if (begun && tid == 0) a.where[head] = make_int2(cta, whole ? 1 : runs.of(h1 - 1) - cta + 1);
    float* to = (whole ? a.part + head * G * kPartRow : a.run_part + ((int64_t)cta * 2 + (begun ? 1 : 0)) * G * kPartRow);
#pragma unroll
    for (int h = 0; h < (WIDE ? 2 : 1); ++h) {
      float* d = sp + (warp * 8 + (lane >> 2)) * kPartRow;
#pragma unroll
      for (int k = 0; k < 16; ++k)
        *reinterpret_cast<float2*>(d + k * 8 + (lane & 3) * 2) = make_float2(o[k][2 * h], o[k][2 * h + 1]);
      if ((lane & 3) == 0) *reinterpret_cast<float2*>(d + D) = make_float2(m[h], l[h]);
      consumers_sync();
      for (int row = warp; row < min(G - 8 * h, 8); row += kOwnWarps) {
        Joined r = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        absorb<kOwnWarps>(r, kOwnWarps, lane, [&](int k) { return sp + (k * 8 + row) * kPartRow; });
        float* at = to + (8 * h + row) * kPartRow;
        *reinterpret_cast<float4*>(at + lane * 4) = r.o;
        if (lane == 0) *reinterpret_cast<float2*>(at + D) = make_float2(r.m, r.l);
      }
      consumers_sync();  // the join buffer is free again
    }
  });
}

// --------------------------------------------------------------------------------------- join
//
// A warp per output row: where its own parts lie, then all parts (own and the prompt's) together,
// four dimensions a lane; two dependent reads of memory, whatever the number of parts up to 16.
struct JoinArgs {
  const float* part;
  const float* run_part;
  const int2* where;
  const float* pre_part;  // [Hkv][pre_splits][B * G][kPartRow]
  const int32_t* lens;
  void* out;
  float* lse;
  int64_t out_stride;
  int B, Hkv, G, pre_splits;
};
constexpr int kJoinWarps = 4;

template <typename T, int KB>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ JoinArgs a) {
  const int lane = threadIdx.x & 31, Hq = a.Hkv * a.G;
  const int64_t row = (int64_t)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  const int b = (int)(row / Hq), h = (int)(row - (int64_t)b * Hq), g = h / a.G, i = h - g * a.G;
  const bool live = row < (int64_t)a.B * Hq && a.lens[min(b, a.B - 1)] >= 0;  // not a padding row
  pdl_wait();
  if (!live) return;
  const int64_t head = (int64_t)b * a.Hkv + g, all = (int64_t)a.B * a.G;
  const int2 at = a.where[head];
  const float* pre = a.pre_part + ((int64_t)g * a.pre_splits * all + (int64_t)b * a.G + i) * kPartRow;
  Joined r = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  absorb<KB>(r, at.y + a.pre_splits, lane, [&](int k) {
    if (k >= at.y) return pre + (k - at.y) * all * kPartRow;
    if (at.y == 1) return a.part + (head * a.G + i) * kPartRow;
    // the set that the first run ended with, then the sets that the runs after it began with
    return a.run_part + ((2 * (int64_t)(at.x + k) + (k == 0)) * a.G + i) * kPartRow;
  });
  // l is 0 where no key has a weight; a NaN score makes l NaN and goes on to the result
  const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
  T* dst = static_cast<T*>(a.out) + (int64_t)b * a.out_stride + h * D + lane * 4;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(r.o.x * inv, r.o.y * inv), pack2<T>(r.o.z * inv, r.o.w * inv));
  if (a.lse && lane == 0) a.lse[(int64_t)b * Hq + h] = r.l == 0.f ? -INFINITY : (r.m + log2f(r.l)) * kLn2;
}

struct Plan {
  int ctas, pre_splits, pre_per;
  size_t run_part, part, pre_part, total;  // byte offsets in the workspace; `where` comes first
};
// Chunks of a sequence and key-value head: own pages (no more than a length can name) and P prompt keys.
int64_t chunk_count(int64_t max_own, int P) {
  const int64_t own = std::min<int64_t>(max_own, int64_t(1) << 31);
  return std::max<int64_t>((own + kChunk - 1) / kChunk + (P + kChunk - 1) / kChunk, 1);
}
void lay_out(Plan& p, int B, int Hkv, int G, int64_t chunks, int64_t pre_rows) {
  const size_t row = kPartRow * sizeof(float), set = G * row, heads = (size_t)B * Hkv;
  p.ctas = (int)std::min<int64_t>(sm_count(), chunks * B * Hkv);
  p.run_part = (heads * sizeof(int2) + 255) / 256 * 256;
  p.part = p.run_part + p.ctas * 2 * set;
  p.pre_part = p.part + heads * set;
  p.total = p.pre_part + pre_rows * row;
}
// One sequence shares nothing, and a prompt of a few chunks costs less to read again than a
// second kernel: there the prompt's keys are the first chunks of every sequence.
bool prompt_apart(int B, int P) { return B > 1 && P >= kMinShared; }
Plan plan_of(int B, int Hkv, int G, int P, int64_t max_own) {
  Plan p = {};
  const bool shared = prompt_apart(B, P);
  if (shared) prefix_tc_split(B * G, Hkv, P, &p.pre_splits, &p.pre_per);
  lay_out(p, B, Hkv, G, chunk_count(max_own, shared ? 0 : P), (int64_t)p.pre_splits * B * Hkv * G);
  return p;
}
// What no plan of at most B sequences, P prompt keys and max_own keys of their own exceeds.  A plan's
// own need is not enough for that: the prompt is cut into fewer parts as the rows of queries grow
// (28 / 4 heads on 32768 keys: 37 parts for 18 sequences, 12 for 48), and into 31 for 3968 keys
// where it is 16 for 4096.
size_t most_bytes(int B, int Hkv, int G, int P, int64_t max_own) {
  Plan p = {};
  lay_out(p, B, Hkv, G, chunk_count(max_own, P), prompt_apart(B, P) ? prefix_tc_most_rows(B * G, Hkv, P) : 0);
  return p.total;
}

// Tensor map of rows of D elements, the two halves of a row as a dimension of their own so that
// one copy fills both swizzled halves of a chunk: dims {64, tokens, 2, heads, pages}, box
// {64, 16, 2, 1, 1}.
bool page_map(CUtensorMap* tm, const void* base, int dtype, int64_t tokens, int64_t heads, int64_t pages,
              int64_t token_stride, int64_t head_stride, int64_t page_stride) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[5] = {64, (cuuint64_t)tokens, 2, (cuuint64_t)heads, (cuuint64_t)pages};
  // the stride of a dimension of one element is never used, but has to be a valid one
  cuuint64_t strides[4] = {(cuuint64_t)token_stride * 2, 128, (cuuint64_t)(heads > 1 ? head_stride : token_stride) * 2,
                           (cuuint64_t)(pages > 1 ? page_stride : token_stride) * 2};
  cuuint32_t box[5] = {64, kChunk, 2, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(tm, dtype == VV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
            const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, bool WIDE>
cudaError_t launch_all(const OwnMaps& mp, const SharedAttnArgs& a, const PrefixTcArgs* t, const JoinArgs& j, int ctas,
                       cudaStream_t s) {
  cudaError_t e = allow_smem<own_attn_kernel<T, WIDE>>(kOwnSmem);
  if (e != cudaSuccess) return e;
  e = launch(own_attn_kernel<T, WIDE>, dim3(ctas), dim3(kOwnThreads), kOwnSmem, s, false, mp, a);
  if (e != cudaSuccess) return e;
  if (t) {
    e = launch_prefix_tc(*t, s);
    if (e != cudaSuccess) return e;
  }
  const int64_t rows = (int64_t)j.B * j.Hkv * j.G;
  const dim3 grid((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), block(kJoinWarps * 32);
  // A row's parts, the prompt's and most often one or two of its own, in one batch of reads where
  // they fit: 12.6 us for 16 x 4530 keys (18 + 1 parts) in batches of 24, 13.4 us in batches of 16;
  // without a prompt 24 slots are idle registers (24.3 us where 8 take 23.5).
  const int parts = j.pre_splits + 2;
  return parts <= 8    ? launch(join_kernel<T, 8>, grid, block, 0, s, true, j)
         : parts <= 16 ? launch(join_kernel<T, 16>, grid, block, 0, s, true, j)
                       : launch(join_kernel<T, 24>, grid, block, 0, s, true, j);
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
  return vv::most_bytes(B, Hkv, Hq / Hkv, prefix_len, max_own);
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
  a.table = block_tables;
  a.lens = own_lens;
  char* base = static_cast<char*>(ws);
  a.where = reinterpret_cast<int2*>(base);
  a.run_part = reinterpret_cast<float*>(base + p.run_part);
  a.part = reinterpret_cast<float*>(base + p.part);
  a.shared = p.pre_splits > 0;
  float* pre_part = reinterpret_cast<float*>(base + p.pre_part);
  a.q_stride = q_stride;
  a.B = B;
  a.Hkv = Hkv;
  a.G = G;
  a.P = prefix_len;
  a.ps = kv->page_size;
  a.pages = kv->pages;
  a.max_blocks = max_blocks;
  a.c = scale * vv::kLog2e;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  vv::PrefixTcArgs t = {};
  const vv::PrefixTcArgs* pre = p.pre_splits ? &t : nullptr;
  if (pre) {
    t.q = q;
    t.k = k_prefix;
    t.v = v_prefix;
    t.part = pre_part;
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
  }
  vv::OwnMaps mp = {};
  bool ok = vv::page_map(&mp.k, kv->k, kv->dtype, kv->page_size, Hkv, kv->pages, kv->token_stride, kv->head_stride, kv->page_stride) &&
            vv::page_map(&mp.v, kv->v, kv->dtype, kv->page_size, Hkv, kv->pages, kv->token_stride, kv->head_stride, kv->page_stride);
  if (ok && prefix_len > 0 && !p.pre_splits)
    ok = vv::page_map(&mp.kpre, k_prefix, kv->dtype, prefix_len, Hkv, 1, prefix_token_stride, prefix_head_stride, 0) &&
         vv::page_map(&mp.vpre, v_prefix, kv->dtype, prefix_len, Hkv, 1, prefix_token_stride, prefix_head_stride, 0);
  if (!ok) return vv::set_error(VV_ERR_CUDA, "vv_gqa_prefix_attn: tensor map encoding failed");
  const vv::JoinArgs j = {a.part, a.run_part, a.where, pre_part, own_lens, out, lse, out_stride, B, Hkv, G, p.pre_splits};
  const bool f16 = kv->dtype == VV_F16, wide = G > 8;
  const cudaError_t e = f16 ? (wide ? vv::launch_all<__half, true>(mp, a, pre, j, p.ctas, s) : vv::launch_all<__half, false>(mp, a, pre, j, p.ctas, s))
                            : (wide ? vv::launch_all<__nv_bfloat16, true>(mp, a, pre, j, p.ctas, s)
                                    : vv::launch_all<__nv_bfloat16, false>(mp, a, pre, j, p.ctas, s));
  return vv::cuda_check(e, "vv_gqa_prefix_attn launch");
}
