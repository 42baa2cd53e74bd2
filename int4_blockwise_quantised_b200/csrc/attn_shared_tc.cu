// The shared prompt's part of vv_gqa_prefix_attn: all sequences' queries against the same keys,
// each key read once per 128 query rows.
//
//   S = scale Q K^T,  P = 2^(S log2e - m),  o = P V,  l = sum P     per row of Q
//
// The rows of one key-value head (sequence x query head of the group) fill the 128 lanes of
// tensor memory: 64 sequences of 7 heads are 3.5 tiles, where one sequence alone would fill 5% of
// one.  One CTA = one tile of 128 rows, one key-value head, one part of the keys, on the
// 5th-generation tensor cores:
//   warp 0      : copies of the K tiles (128 keys, 128-byte swizzle) into a three-stage ring, a
//                 stage free again once the S product that read it is done;
//   warp 2      : the V tiles into a two-stage ring;
//   warp 1      : tensor memory (2 x S, 2 x P, O: 512 columns) and the products S_j = Q K_j^T;
//   warp 3      : the products O += P_j V_j (P_j from tensor memory, V read MN-major straight from
//                 the row-major tile); waits and commits of one kind of product then pass while the
//                 other kind keeps the tensor core busy;
//   warps 4..7, 8..11: softmax of the even and of the odd blocks, one thread per row.
// A thread takes its row's 128 scores of a block into registers, which frees the S buffer at once:
// S_{j+2} is queued ahead of P_j V_j, so the tensor core never waits for exponentials that it does
// not need, and a group's next scores are there when it has stored its weights.  A maximum needs
// no exchange inside a block; the two groups hand the row's running maximum on from block to block
// through shared memory (a one-way named barrier per 32 rows), so that one O serves both.  While
// one group's exponentials run (128 a row and block: 1024 cycles of the special-function units)
// the other loads, finds its maximum and stores.  O is rescaled only when a block's maximum
// exceeds the running one by more than 2^8: weights stay below 2^8, and the same reference divides
// them out.  fp16 weights are taken 2^6 larger still (at most 2^14), so that those down to 2^-20 of the
// largest keep all their bits and smaller ones are off by at most 2^-31 of it.
// The weights are rounded to the element type because the tensor cores multiply 16-bit operands;
// their sum l is taken before that rounding.  The tile's partial rows (o, m, l) go to the workspace
// in fp32; the join kernel puts the parts together.
// 48 sequences x 28 heads on 32768 keys, 22 blocks of 128 keys a CTA: a block takes 1449 cycles (what twice
// the prompt takes more), where its products take 1024 and its exponentials 1024 of the special-function
// units; at the 1.5 GHz that the SMs run at under it, 0.93 to 0.98 us, 21 us and 1.07 PFLOP/s for the
// loop.  Start and end are 12900 cycles more.
// Every mbarrier wait is bounded; tensor memory is released before the CTA exits.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "attn_shared.h"
#include "attn_tc.cuh"
#include "pack16.cuh"
#include "vv_device.cuh"
#include "vv_internal.h"

namespace vv {
namespace {

using namespace tc;

constexpr int D = 128;
constexpr int BM = 128;   // query rows per CTA
constexpr int BN = 128;   // keys per block
constexpr int kThreads = 384;
constexpr int kKStages = 3, kVStages = 2;  // V_j, P_j and S_j share the index j & 1
constexpr int kTiles = 1 + kKStages + kVStages;
constexpr float kRescale = 8.0f;
template <typename T>
constexpr float kHeadroom = std::is_same<T, __half>::value ? 6.0f : 0.0f;
constexpr uint32_t kBarBytes = 256;
constexpr int kOutRow = 132;  // floats per row of the output stage (conflict-free float4 columns)
constexpr size_t kSmem = kTiles * kTile + kBarBytes + 2 * BM * 4 + 2 * BM * 8 + 1024;
static_assert(BM * kOutRow * 4 <= (kKStages + kVStages) * kTile, "the output stage lies over the rings");

// instruction descriptor (kind::f16, D f32, M = N = 128): A and B fp16 (0) or bf16 (1)
template <typename T>
constexpr uint32_t idesc(bool b_mn) {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(BN >> 3) << 17) |
         ((uint32_t)(BM >> 4) << 24);
}

struct KvMaps {
  CUtensorMap k, v;  // dims {D, P, Hkv}, box {64, 128, 1}; rows past P read as zeros
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ KvMaps mp, const __grid_constant__ PrefixTcArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* sQ = smem;
  unsigned char* sK = smem + kTile;
  unsigned char* sV = smem + (1 + kKStages) * kTile;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kTiles * kTile);
  uint64_t* k_full = bars;                  // [kKStages]
  uint64_t* k_empty = k_full + kKStages;    // [kKStages]
  uint64_t* v_full = k_empty + kKStages;    // [kVStages]
  uint64_t* s_full = v_full + kVStages;     // [2]
  uint64_t* s_free = s_full + 2;            // [2] scores are in registers
  uint64_t* p_full = s_free + 2;            // [2]
  uint64_t* pv_done = p_full + 2;           // [2] also frees the V stage
  uint64_t* o_done = pv_done + 2;           // all products: one phase, waited for by both groups
  uint64_t* v_go = o_done + 1;              // the first K tile is here: one phase
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_go + 1);
  float(*m_row)[BM] = reinterpret_cast<float(*)[BM]>(smem + kTiles * kTile + kBarBytes);  // [2][BM]
  float2(*ml)[BM] = reinterpret_cast<float2(*)[BM]>(smem + kTiles * kTile + kBarBytes + 2 * BM * 4);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rows = a.B * a.G;
  const int r0 = blockIdx.x * BM, split = blockIdx.y, g = blockIdx.z;
  const int blocks = (a.P + BN - 1) / BN;
  const int j0 = split * a.per, n = min(a.per, blocks - j0);  // n >= 1 by the launch's grid

  pdl_launch_dependents();  // the join waits for this kernel's end by itself
  auto load_k = [&](int j) {
    const int st = j % kKStages;
    unsigned char* kt = sK + st * kTile;
    mbar_arrive_expect_tx(&k_full[st], kTile);
    tma_load_3d(kt, &mp.k, 0, (j0 + j) * BN, g, &k_full[st]);
    tma_load_3d(kt + kAtom, &mp.k, 64, (j0 + j) * BN, g, &k_full[st]);
  };
  auto load_v = [&](int j) {
    const int st = j % kVStages;
    unsigned char* vt = sV + st * kTile;
    mbar_arrive_expect_tx(&v_full[st], kTile);
    tma_load_3d(vt, &mp.v, 0, (j0 + j) * BN, g, &v_full[st]);
    tma_load_3d(vt + kAtom, &mp.v, 64, (j0 + j) * BN, g, &v_full[st]);
  };
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < kVStages; ++i) mbar_init(&v_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(o_done, 1);
    mbar_init(v_go, 1);
    fence_mbar_init();
    load_k(0);  // on its way before the rest of the CTA is ready
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Q: two threads per row, 64 dimensions each, into the swizzled K-major atoms; rows past the
  // last are zero
  if (tid >= 128) {
    const int r = (tid - 128) >> 1, half = tid & 1, row = r0 + r;
    uint4 v[8];
    if (row < rows) {
      const int b = row / a.G, h = row - b * a.G;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const T*>(a.q) + (int64_t)b * a.q_stride + (int64_t)(g * a.G + h) * D + half * 64);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = src[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = make_uint4(0, 0, 0, 0);
    }
    unsigned char* dst = sQ + half * kAtom + r * 128;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + ((i ^ (r & 7)) << 4)) = v[i];
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the tensor core reads it
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  auto tS = [tmem](int i) { return tmem + (uint32_t)(i * 128); };
  auto tP = [tmem](int i) { return tmem + 256u + (uint32_t)(i * 64); };
  const uint32_t tO = tmem + 384u;

  if (warp == 0) {
    if (lane == 0) {
      // all CTAs begin at once: the others' first tiles come before this one's second
      auto first_tile = [&] {
        wait_phase(&k_full[0], 0);
        mbar_arrive(v_go);
      };
      for (int j = 1; j < n; ++j) {
        if (j >= kKStages) wait_phase(&k_empty[j % kKStages], (j / kKStages - 1) & 1);
        if (j == 2) first_tile();
        load_k(j);
      }
      if (n <= 2) first_tile();
    }
    __syncwarp();
  } else if (warp == 2) {
    if (lane == 0) {
      wait_phase(v_go, 0);
      for (int j = 0; j < n; ++j) {
        if (j >= kVStages) wait_phase(&pv_done[j & 1], ((j >> 1) - 1) & 1);
        load_v(j);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t qa = smem_u32(sQ);
    constexpr uint32_t kIdS = idesc<T>(false);
    auto issue_s = [&](int j) {
      const int st = j % kKStages, sb = j & 1;
      wait_phase(&k_full[st], (j / kKStages) & 1);
      tc_after();
      const uint32_t kb = smem_u32(sK + st * kTile);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (uint32_t)(k >> 2) * kAtom + (uint32_t)(k & 3) * 32;
        mma_ss_elect(tS(sb), desc_k_sw128(qa + off), desc_k_sw128(kb + off), kIdS, k > 0 ? 1u : 0u);
      }
      mma_commit_elect(&s_full[sb]);
      mma_commit_elect(&k_empty[st]);
    };
    issue_s(0);
    if (n > 1) issue_s(1);
    for (int j = 2; j < n; ++j) {
      wait_phase(&s_free[j & 1], ((j >> 1) - 1) & 1);
      issue_s(j);
    }
  } else if (warp == 3) {
    constexpr uint32_t kIdPV = idesc<T>(true);
    for (int j = 0; j < n; ++j) {
      const int sb = j & 1;
      wait_phase(&v_full[sb], (j >> 1) & 1);
      wait_phase(&p_full[sb], (j >> 1) & 1);
      tc_after();
      const uint32_t vb = smem_u32(sV + sb * kTile);
#pragma unroll
      for (int k = 0; k < BN / 16; ++k)
        mma_ts_elect(tO, tP(sb) + (uint32_t)(k * 8), desc_mn_sw128(vb + (uint32_t)k * 2048), kIdPV,
                     (j > 0 || k > 0) ? 1u : 0u);
      mma_commit_elect(&pv_done[sb]);
    }
    mma_commit_elect(o_done);
  } else if (warp >= 4) {
    const int s = (warp - 4) >> 2, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float c = a.c;
    float m_mine = -INFINITY, l = 0.f;  // l: this group's blocks, relative to m_mine
    for (int j = s; j < n; j += 2) {
      wait_phase(&s_full[s], (j >> 1) & 1);
      tc_after();
      uint32_t sr[4][32];
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) tmem_ld32(tS(s) + lane_off + (uint32_t)(cc * 32), sr[cc]);
      tmem_wait_ld();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[s]);
      const int left = a.P - (j0 + j) * BN;  // keys of this block
      if (left < BN) {
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
#pragma unroll
          for (int t = 0; t < 32; ++t)
            if (cc * 32 + t >= left) sr[cc][t] = __float_as_uint(-INFINITY);
        }
      }
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int cc = 0; cc < 4; ++cc) {
#pragma unroll
        for (int t = 0; t < 32; ++t) m4[t & 3] = fmaxf(m4[t & 3], __uint_as_float(sr[cc][t]));
      }
      const float mb = fmaf(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])), c, -kHeadroom<T>);
      // the running reference after block j - 1, from the other group's warp of the same rows
      float m_prev = -INFINITY;
      if (j > 0) {
        asm volatile("bar.sync %0, 64;" ::"r"(2 + quarter * 2 + (s ^ 1)) : "memory");
        m_prev = m_row[s ^ 1][r];
      }
      const bool move = mb > m_prev + kRescale;
      const float m_new = move ? mb : m_prev;
      if (j + 1 < n) {
        m_row[s][r] = m_new;
        asm volatile("bar.arrive %0, 64;" ::"r"(2 + quarter * 2 + s) : "memory");
      }
      // P_{j-2} has been read.  Its product also comes after that of block j - 3, so the other
      // group's barrier is in the phase of block j - 1 from here until P_j is handed over: the
      // rescaling below can wait for that phase by its parity
      if (j > 1) wait_phase(&pv_done[s], ((j >> 1) - 1) & 1);
      if (j > 0 && __any_sync(0xffffffffu, move)) {
        const float corr = move ? ex2_approx(m_prev - m_new) : 1.f;
        wait_phase(&pv_done[s ^ 1], ((j - 1) >> 1) & 1);  // O holds the blocks before
        tc_after();
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {  // 16 columns at a time: the scores stay in registers
          uint32_t o[16];
          tmem_ld16(tO + lane_off + (uint32_t)(cc * 16), o);
          tmem_wait_ld();
#pragma unroll
          for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * corr);
          tmem_st16(tO + lane_off + (uint32_t)(cc * 16), o);
        }
      }
      const float ref = m_new == -INFINITY ? 0.f : m_new;  // nothing above -inf yet: weights 0
      l *= ex2_approx(m_mine - ref);
      m_mine = m_new;
      float ls0 = 0.f, ls1 = 0.f;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t pp[32];
#pragma unroll
        for (int t = 0; t < 64; t += 2) {
          const float e0 = ex2_approx(fmaf(__uint_as_float(sr[hh * 2 + (t >> 5)][t & 31]), c, -ref));
          const float e1 = ex2_approx(fmaf(__uint_as_float(sr[hh * 2 + (t >> 5)][(t & 31) + 1]), c, -ref));
          ls0 += e0;
          ls1 += e1;
          pp[t >> 1] = pack2<T>(e0, e1);
        }
        tmem_st32(tP(s) + lane_off + (uint32_t)(hh * 32), pp);
      }
      l += ls0 + ls1;
      tmem_wait_st();
      tc_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s]);
    }
    // ---- the tile's partial rows: o through shared memory (the rings are idle by then) so that a
    // warp stores whole rows
    ml[s][r] = make_float2(m_mine, l);
    wait_phase(o_done, 0);
    tc_after();
    float* stage = reinterpret_cast<float*>(sK);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int cc = s * 2 + i;
      uint32_t o[32];
      tmem_ld32(tO + lane_off + (uint32_t)(cc * 32), o);
      tmem_wait_ld();
#pragma unroll
      for (int t = 0; t < 32; t += 4)
        *reinterpret_cast<uint4*>(stage + r * kOutRow + cc * 32 + t) = make_uint4(o[t], o[t + 1], o[t + 2], o[t + 3]);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float* dst = a.part + (((int64_t)g * a.splits + split) * rows + r0) * kPartRow;
    const int mine = (warp - 4) * 16, left = min(16, rows - r0 - mine);
#pragma unroll 4
    for (int i = 0; i < left; ++i)
      *reinterpret_cast<float4*>(dst + (int64_t)(mine + i) * kPartRow + lane * 4) =
          *reinterpret_cast<const float4*>(stage + (mine + i) * kOutRow + lane * 4);
    if (s == 0 && r0 + r < rows) {
      // the reference of the last block is the row's; l of each group relative to it
      const float2 other = ml[1][r];
      const float M = (n - 1) & 1 ? other.x : m_mine, ref = M == -INFINITY ? 0.f : M;
      *reinterpret_cast<float2*>(dst + (int64_t)r * kPartRow + D) =
          make_float2(M, l * ex2_approx(m_mine - ref) + other.y * ex2_approx(other.x - ref));
    }
  }
  tc_before();
  __syncthreads();
  pdl_wait();  // the join reads the own pages' parts too: it may only start after both kernels
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <typename T>
cudaError_t launch_t(const KvMaps& mp, const PrefixTcArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem<prefix_tc_kernel<T>>(kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.B * a.G + BM - 1) / BM, a.splits, a.Hkv);
  return launch(prefix_tc_kernel<T>, grid, dim3(kThreads), kSmem, s, true, mp, a);
}

// Most parts that the keys are cut into: enough for a CTA per SM, and at least 8.
int64_t most_splits(int64_t tiles) { return std::max<int64_t>(8, sm_count() / tiles); }

}  // namespace

void prefix_tc_split(int rows, int Hkv, int P, int* splits, int* per) {
  // Cost in blocks of 128 keys (about 0.8 us each): waves x (a part's blocks + 4 for its start and
  // end), and one for each further 32 parts that the join has to read.
  const int64_t tiles = (int64_t)((rows + BM - 1) / BM) * Hkv, sms = sm_count();
  const int blocks = (P + BN - 1) / BN;
  int64_t best = INT64_MAX;
  const int most = (int)std::min<int64_t>(blocks, most_splits(tiles));
  for (int s = 1; s <= most; ++s) {
    const int p = (blocks + s - 1) / s, used = (blocks + p - 1) / p;
    const int64_t cost = (tiles * used + sms - 1) / sms * (p + 4) + used / 32;
    if (cost < best) {
      best = cost;
      *splits = used;
      *per = p;
    }
  }
}

int64_t prefix_tc_most_rows(int rows, int Hkv, int P) {
  // The parts fall as the tiles grow, so the most rows of parts are those of some number of full tiles.
  const int64_t blocks = (P + BN - 1) / BN;
  int64_t most = 0;
  for (int64_t t = 1; t <= (rows + BM - 1) / BM; ++t)
    most = std::max(most, std::min<int64_t>(rows, t * BM) * std::min(blocks, most_splits(t * Hkv)));
  return most * Hkv;
}

cudaError_t launch_prefix_tc(const PrefixTcArgs& a, cudaStream_t s) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  KvMaps mp;
  for (int t = 0; t < 2; ++t) {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.P, (cuuint64_t)a.Hkv};
    cuuint64_t strides[2] = {(cuuint64_t)a.token * 2,
                             (cuuint64_t)(a.Hkv > 1 ? a.head : a.token) * 2};
    cuuint32_t box[3] = {64, BN, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    if (fn(t == 0 ? &mp.k : &mp.v,
           a.dtype == VV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
           3, const_cast<void*>(t == 0 ? a.k : a.v), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  return a.dtype == VV_F16 ? launch_t<__half>(mp, a, s) : launch_t<__nv_bfloat16>(mp, a, s);
}

}  // namespace vv
