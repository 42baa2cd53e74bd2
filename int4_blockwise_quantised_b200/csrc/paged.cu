// Bookkeeping and key/value writes of a paged cache: vv_paged_plan and vv_qk_rope_append.
//
// Both belong to a batch that continues one shared prompt ("VibeVoice-1.5B — Current Status":
// several contexts stepped alongside each other over the same weights): every sequence keeps its
// own keys and values in pages of a common pool, vv_paged_plan hands out the pages and says
// where each new token goes, vv_qk_rope_append puts it there.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pack16.cuh"
#include "vv_device.cuh"
#include "vv_internal.h"

namespace vv {
namespace {

// ------------------------------------------------------------------------------------- plan
//
//   after_b = len_b + new_b          old_b = ceil(len_b / ps)     need_b = ceil(after_b / ps)
//   table[b, old_b + j] = free[cursor + sum_{i<b} (need_i - old_i) + j]
//   token j of request b: own index i = len_b + j, slot = table[b, i / ps] * ps + i % ps,
//   position = prefix + i, row offsets[b] + j
//
// One launch and no communication between CTAs: each CTA scans all B requests itself (their
// lengths are a few KB, in L2 after the first CTA), keeps the exclusive sums of tokens and pages
// in shared memory and then takes its share of the requests, of the new pages and of the tokens;
// a token or page finds its request by bisection in those sums.  A step of a small batch is one
// CTA: what it costs is the latency of load, scan, bisection and store, not bytes (5.0 us for 32
// requests, 5.9 for 301; 4096 requests with 778k tokens, 9.5 MB: 12.4 us).
constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 16384;  // three int32 per request in shared memory (192 KB)

struct PlanArgs {
  const int32_t* lens;
  const int32_t* news;
  const int32_t* free_pages;
  const int32_t* cursor;
  int32_t* table;
  int32_t* lens_out;
  int32_t* offsets;
  int64_t* slots;
  int32_t* positions;
  int32_t* cursor_out;
  int B, prefix, ps, n_free, pool, max_blocks, max_tokens;
  unsigned magic;  // x / ps = umulhi(x, magic) >> shift for 0 <= x < 2^31 (ps = 1: magic 0)
  int shift;
};

// x + y for 0 <= x, y < 2^31, held at 2^31 - 1 (associative, so a scan may use it): lengths come
// from the caller's device memory, and a sum past 32 bits has to end as a recorded error.
__device__ __forceinline__ int add_sat(int x, int y) {
  return (int)min((unsigned)x + (unsigned)y, 0x7fffffffu);
}

// Largest b in [0, n) with sums[b] <= x (sums ascending, sums[0] = 0).
__device__ __forceinline__ int find_request(const int32_t* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PlanArgs a) {
  extern __shared__ int32_t plan_smem[];
  const int pitch = (a.B + 4) & ~3;
  int32_t* len_s = plan_smem;              // [B] tokens before the step
  int32_t* tok0 = plan_smem + pitch;       // [B + 1] exclusive sum of new tokens
  int32_t* page0 = plan_smem + 2 * pitch;  // [B] exclusive sum of new pages
  __shared__ int2 warp_sum_s[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto block_of = [&](int i) { return a.magic ? (int)(__umulhi((unsigned)i, a.magic) >> a.shift) : i; };  // i / ps
  auto pages_of = [&](int n) { return n ? block_of(n - 1) + 1 : 0; };                                      // ceil(n / ps)
  constexpr int kWarps = kPlanThreads / 32;
  const int cursor = a.cursor ? *a.cursor : 0;

  // a warp scans a run of requests, four neighbours a lane; then the warps' totals are scanned
  const int run = (a.B + kWarps * 128 - 1) / (kWarps * 128) * 128;
  const int b0 = min(warp * run, a.B), b1 = min(b0 + run, a.B);
  bool bad = false;
  int st = 0, sp = 0;  // the warp's sums so far
  for (int base = b0; base < b1; base += 128) {
    const int b = base + lane * 4;
    int len[4], add[4], fresh[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      len[i] = b + i < b1 ? a.lens[b + i] : 0;
      add[i] = b + i < b1 ? a.news[b + i] : 0;
    }
    int nt = 0, np = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fresh[i] = 0;
      if (len[i] < 0 || add[i] < 0 || (int64_t)len[i] + add[i] + a.prefix > 0x7fffffff) {
        bad = bad || len[i] >= 0 || add[i] != 0;  // appends nothing; a padding row that wants nothing is no error
        add[i] = 0;
      } else {
        fresh[i] = pages_of(len[i] + add[i]) - pages_of(len[i]);
      }
      nt = add_sat(nt, add[i]);
      np = add_sat(np, fresh[i]);
    }
    int it = nt, ip = np;  // inclusive over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ut = __shfl_up_sync(0xffffffffu, it, o), up = __shfl_up_sync(0xffffffffu, ip, o);
      if (lane >= o) {
        it = add_sat(it, ut);
        ip = add_sat(ip, up);
      }
    }
    const int et = __shfl_up_sync(0xffffffffu, it, 1), ep = __shfl_up_sync(0xffffffffu, ip, 1);
    int4 tok, pg;
    tok.x = add_sat(st, lane ? et : 0);
    pg.x = add_sat(sp, lane ? ep : 0);
    tok.y = add_sat(tok.x, add[0]);
    pg.y = add_sat(pg.x, fresh[0]);
    tok.z = add_sat(tok.y, add[1]);
    pg.z = add_sat(pg.y, fresh[1]);
    tok.w = add_sat(tok.z, add[2]);
    pg.w = add_sat(pg.z, fresh[2]);
    if (b < b1) {  // entries past B fall into the padding
      *reinterpret_cast<int4*>(len_s + b) = make_int4(len[0], len[1], len[2], len[3]);
      *reinterpret_cast<int4*>(tok0 + b) = tok;
      *reinterpret_cast<int4*>(page0 + b) = pg;
    }
    st = add_sat(st, __shfl_sync(0xffffffffu, it, 31));
    sp = add_sat(sp, __shfl_sync(0xffffffffu, ip, 31));
  }
  if (lane == 0) warp_sum_s[warp] = make_int2(st, sp);
  __syncthreads();
  int2 ws = lane < kWarps ? warp_sum_s[lane] : make_int2(0, 0);
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1) {
    const int ut = __shfl_up_sync(0xffffffffu, ws.x, o), up = __shfl_up_sync(0xffffffffu, ws.y, o);
    if (lane >= o) ws = make_int2(add_sat(ws.x, ut), add_sat(ws.y, up));
  }
  const int all_tok = __shfl_sync(0xffffffffu, ws.x, kWarps - 1);
  const int all_page = __shfl_sync(0xffffffffu, ws.y, kWarps - 1);
  const int t0 = __shfl_sync(0xffffffffu, ws.x, max(warp - 1, 0)), p0 = __shfl_sync(0xffffffffu, ws.y, max(warp - 1, 0));
  if (warp > 0) {
    for (int b = b0 + lane; b < b1; b += 32) {
      tok0[b] = add_sat(tok0[b], t0);
      page0[b] = add_sat(page0[b], p0);
    }
  }
  if (tid == 0) tok0[a.B] = all_tok;
  __syncthreads();

  int error = bad || cursor < 0 ? VV_ERR_RANGE : 0;
  const int gtid = blockIdx.x * kPlanThreads + tid, gsize = gridDim.x * kPlanThreads;
  const int n_tok = min(all_tok, a.max_tokens);
  if (all_tok > a.max_tokens) error = VV_ERR_CAPACITY;
  if (gtid == 0) {
    const int64_t end = (int64_t)cursor + all_page;
    if (end > a.n_free) error = VV_ERR_CAPACITY;
    *a.cursor_out = (int32_t)min(end, (int64_t)0x7fffffff);
  }
  for (int b = gtid; b <= a.B; b += gsize) {
    a.offsets[b] = min(tok0[b], n_tok);
    if (b < a.B) a.lens_out[b] = len_s[b] + (tok0[b + 1] - tok0[b]);
  }
  // the page of fresh index p (over all requests), -1 when the list has run out or names no page
  auto fresh_page = [&](int p) {
    const int64_t at = (int64_t)p + cursor;
    if (cursor < 0 || at >= a.n_free) return -1;
    const int page = a.free_pages[at];
    return page >= 0 && page < a.pool ? page : -1;
  };
  for (int64_t p = gtid; p < all_page; p += gsize) {
    const int b = find_request(page0, a.B, (int)p);
    const int block = pages_of(len_s[b]) + ((int)p - page0[b]);
    if (block >= a.max_blocks) {  // past the table: on to the next request's pages
      error = VV_ERR_CAPACITY;
      if (b + 1 == a.B) break;
      p += (page0[b + 1] - p - 1) / gsize * gsize;
      continue;
    }
    const int page = fresh_page((int)p);
    a.table[(int64_t)b * a.max_blocks + block] = page;
    if (page < 0 && error == 0) error = p + cursor >= a.n_free ? VV_ERR_CAPACITY : VV_ERR_RANGE;
  }
  // tokens, four in a row per thread: one bisection, then a walk
  for (int64_t t4 = (int64_t)gtid * 4; t4 < a.max_tokens; t4 += (int64_t)gsize * 4) {
    int64_t slot[4];
    int pos[4];
    int b = -1, end = -1, first = 0, blk = -1, page = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = (int)t4 + e;
      slot[e] = -1;
      pos[e] = 0;
      if (t >= n_tok) continue;
      if (t >= end) {
        if (b < 0)
          b = find_request(tok0, a.B, t);
        else
          do ++b;
          while (tok0[b + 1] <= t);
        end = tok0[b + 1];
        first = len_s[b] - tok0[b];
        blk = -1;
      }
      const int i = first + t;
      const int block = block_of(i);
      if (block != blk) {
        blk = block;
        const int old = pages_of(len_s[b]);
        page = -1;
        if (block >= a.max_blocks) {
          if (error == 0) error = VV_ERR_CAPACITY;
        } else if (block >= old) {
          page = fresh_page(page0[b] + (block - old));
        } else {
          page = a.table[(int64_t)b * a.max_blocks + block];
          if (page < 0 || page >= a.pool) {
            page = -1;
            if (error == 0) error = VV_ERR_RANGE;
          }
        }
      }
      if (page >= 0) slot[e] = (int64_t)page * a.ps + (i - block * a.ps);
      pos[e] = a.prefix + i;
    }
    if (t4 + 4 <= a.max_tokens) {
      longlong2* so = reinterpret_cast<longlong2*>(a.slots + t4);
      so[0] = make_longlong2(slot[0], slot[1]);
      so[1] = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + t4) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 3; ++e) {
        if (t4 + e < a.max_tokens) {
          a.slots[t4 + e] = slot[e];
          a.positions[t4 + e] = pos[e];
        }
      }
    }
  }
  if (error) set_device_error(error);
}

// ------------------------------------------------------------------------------ rope append
//
//   x <- x / sqrt(mean(x^2) + eps) * gain            (query and key heads, when gains are given)
//   (x_i, x_{i+64}) <- (x_i c - x_{i+64} s, x_{i+64} c + x_i s),  angle = pos * theta^(-2i/128)
//
// Bound by HBM: every head row is read once and written once (512 bytes for 128 elements): 50001
// tokens of 28 + 4 + 4 heads take 154 us in a replayed graph (6.0 TB/s), 159 to 167 among eager calls;
// with norms the instructions count too, 161 us, and 22.0 us for 4530 such tokens (3.8 TB/s); 16 tokens of
// 12 + 2 + 2 heads take 3.0 us.
// A unit is one token's heads, or a part of them; a warp works alone on its units and has the next
// one or two on their way (cp.async.bulk into a ring of its own, a token's heads of one kind are
// contiguous), whatever its registers and without a barrier between warps.  Half a warp turns one
// head row; a lane holds four elements and their partners, so that each is read and converted once.
// A token's angles are found once per unit, two a lane: the quarter turns pos * theta^(-2i/128) * 2 / pi
// reduced to [-1/2, 1/2] in 64 bits (in 32 bits a position of 10^6 would lose the angle's second
// digit), then sine and cosine of the remainder in 32 bits.
constexpr int kHeadDim = 128;
constexpr int kRopeHeads = 18;  // most heads of a unit, 4.5 KB
// With norms a row takes half as many instructions again: eight warps per CTA (two CTAs per SM) and one
// unit on its way beside the one in work.  Without, as many warps ask memory for more than it gives
// in good order: 50001 tokens of 28 + 4 + 4 heads take 171 us with eight, 170 with six, 154 with five
// and 161 with four; with norms 161 with eight, 188 with six and 225 with five.
template <bool GAINS>
struct RopeShape {
  static constexpr int kWarps = GAINS ? 8 : 5;
  static constexpr int kStages = GAINS ? 2 : 3;
};

struct RopeArgs {
  const char* q;
  const char* k;
  const char* v;
  char* q_out;
  char* kp;
  char* vp;
  const void* q_gain;
  const void* k_gain;
  const int32_t* pos;
  const int64_t* slots;
  int64_t q_stride, k_stride, v_stride, qo_stride;        // bytes
  int64_t page_stride, head_stride, token_stride;         // bytes
  int64_t n_slots;
  int T, Hq, Hkv, ps;
  int heads, parts;  // heads per unit; units per token
  float eps;
  double quarters[kHeadDim / 2];  // quarter turns a position: theta^(-2i/D) 2 / pi
};

// Two fp32 numbers in one register pair: sm_100 multiplies and adds both in one instruction.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ f32x2 pair(float2 x) { return pair(x.x, x.y); }
__device__ __forceinline__ float2 unpair(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Sine and cosine of z quarter turns, |z| <= 1/2: polynomials in w = z^2, interpolated at four Chebyshev
// nodes of [0, 1/4] to sin(pi z / 2) / z and (cos(pi z / 2) - 1) / w.  Right to 2^-22.8 of the value,
// however small it is; the hardware's fast sine is off by up to 2^-21, a third of the sine by which
// the slowest pair of theta 10^6 turns the token at position 1.
__device__ __forceinline__ void sincos2(f32x2 z, f32x2& sn, f32x2& cn) {
  auto both = [](float x) { return pair(x, x); };
  const f32x2 w = mul2(z, z);
  const f32x2 p = fma2(fma2(fma2(both(-0.00460214913f), w, both(0.0796802193f)), w, both(-0.645963490f)), w, both(1.57079637f));
  const f32x2 q = fma2(fma2(fma2(both(9.06739908e-4f), w, both(-0.0208615288f)), w, both(0.253669411f)), w, both(-1.23370051f));
  sn = mul2(p, z);
  cn = fma2(q, w, both(1.f));
}
// (cosine, sine) of n quarter turns more, n a whole number: its last two bits, where 2^52 + 2^51 puts them
__device__ __forceinline__ float2 quadrant(double n, float c, float s) {
  const unsigned q = (unsigned)__double2loint(n + 6755399441055744.0);
  const unsigned x = __float_as_uint(q & 1 ? s : c), y = __float_as_uint(q & 1 ? c : s);
  return make_float2(__uint_as_float(x ^ ((q + 1) << 30 & 0x80000000u)), __uint_as_float(y ^ (q << 30 & 0x80000000u)));
}

template <typename T, bool GAINS>
__global__ void __launch_bounds__(RopeShape<GAINS>::kWarps * 32, 2)
    qk_rope_append_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int kRow = kHeadDim * 2, kRopeWarps = RopeShape<GAINS>::kWarps, kRopeStages = RopeShape<GAINS>::kStages;
  extern __shared__ __align__(128) unsigned char ring_all[];
  __shared__ __align__(8) uint64_t full_all[kRopeWarps][kRopeStages];
  __shared__ __align__(16) float2 cs_all[kRopeWarps][kHeadDim / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_heads = a.Hq + 2 * a.Hkv, unit_bytes = a.heads * kRow;
  unsigned char* ring = ring_all + warp * (kRopeStages * unit_bytes);
  uint64_t* full = full_all[warp];
  float2* cs = cs_all[warp];
  if (lane == 0) {
    for (int i = 0; i < kRopeStages; ++i) mbar_init(&full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int64_t units = (int64_t)a.T * a.parts, step = (int64_t)gridDim.x * kRopeWarps;
  const int64_t u0 = (int64_t)blockIdx.x * kRopeWarps + warp;
  // lane p copies the unit's queries (p = 0), keys or values
  const char* src = lane == 0 ? a.q : lane == 1 ? a.k : a.v;
  const int64_t stride = lane == 0 ? a.q_stride : lane == 1 ? a.k_stride : a.v_stride;
  const int lo = lane == 0 ? 0 : a.Hq + (lane - 1) * a.Hkv, hi = lane == 0 ? a.Hq : lo + a.Hkv;
  auto copy = [&](int64_t u, int st) {
    if (u >= units) return;
    const int t = (int)(u / a.parts), h0 = (int)(u - (int64_t)t * a.parts) * a.heads, nh = min(a.heads, n_heads - h0);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], nh * kRow);
    __syncwarp();
    const int from = max(lo, h0), to = min(hi, h0 + nh);
    if (lane < 3 && from < to)
      bulk_g2s(ring + st * unit_bytes + (from - h0) * kRow, src + t * stride + (from - lo) * kRow, (to - from) * kRow,
               &full[st]);
  };
#pragma unroll
  for (int i = 0; i < kRopeStages; ++i) copy(u0 + i * step, i);

  const int c = lane & 15;  // elements 4c .. 4c + 3 of a row and their partners; 16-byte piece of a value row
  const double f0 = a.quarters[lane], f1 = a.quarters[lane + 32];
  int pos = 0;
  int64_t slot = -1;
  if (u0 < units) {
    pos = a.pos[u0 / a.parts];
    slot = a.slots[u0 / a.parts];
  }
  int st = 0;
  uint32_t round = 0;
  for (int64_t u = u0; u < units; u += step) {
    const int t = (int)(u / a.parts), h0 = (int)(u - (int64_t)t * a.parts) * a.heads, nh = min(a.heads, n_heads - h0);
    {
      const double x0 = (double)pos * f0, x1 = (double)pos * f1, n0 = rint(x0), n1 = rint(x1);
      f32x2 sn, cn;
      sincos2(pair((float)(x0 - n0), (float)(x1 - n1)), sn, cn);
      const float2 s = unpair(sn), c = unpair(cn);
      cs[lane] = quadrant(n0, c.x, s.x);
      cs[lane + 32] = quadrant(n1, c.y, s.y);
    }
    int64_t at = -1;  // byte offset of the token's cell in the pool
    if (slot >= a.n_slots) {
      if (lane == 0) set_device_error(VV_ERR_RANGE);
    } else if (slot >= 0) {
      const int page = (int)slot / a.ps;
      at = page * a.page_stride + ((int)slot - page * a.ps) * a.token_stride;
    }
    if (u + step < units) {  // the next unit's
      pos = a.pos[(u + step) / a.parts];
      slot = a.slots[(u + step) / a.parts];
    }
    __syncwarp();
    // (x, y) <- (x cx + y sx, y cy + x sy): the cosines and sines times the gains, two pairs a word
    f32x2 cx[2], sx[2], cy[2], sy[2];
    auto factors = [&](const void* gain) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 f = *reinterpret_cast<const float4*>(&cs[c * 4 + 2 * j]);
        float2 g = make_float2(1.f, 1.f), h = g;
        if (GAINS && gain) {
          g = unpack2<T>(static_cast<const uint32_t*>(gain)[c * 2 + j]);
          h = unpack2<T>(static_cast<const uint32_t*>(gain)[32 + c * 2 + j]);
        }
        cx[j] = pair(f.x * g.x, f.z * g.y);
        sx[j] = pair(-f.y * h.x, -f.w * h.y);
        cy[j] = pair(f.x * h.x, f.z * h.y);
        sy[j] = pair(f.y * g.x, f.w * g.y);
      }
    };
    // rows from .. to - 1 of the unit, two at a time, row r to dst(r)
    // (two iterations at once send memory the same requests in bursts: 2% slower without norms)
    auto turn = [&](int from, int to, bool norm, auto&& dst) {
      const unsigned char* in = ring + st * unit_bytes + c * 8;
#pragma unroll 1
      for (int r0 = from; r0 < to; r0 += 2) {
        const int r = min(r0 + (lane >> 4), to - 1);  // an odd last row is done twice
        const uint2 xw = *reinterpret_cast<const uint2*>(in + r * kRow);
        const uint2 yw = *reinterpret_cast<const uint2*>(in + r * kRow + kRow / 2);
        const f32x2 x[2] = {pair(unpack2<T>(xw.x)), pair(unpack2<T>(xw.y))};
        const f32x2 y[2] = {pair(unpack2<T>(yw.x)), pair(unpack2<T>(yw.y))};
        f32x2 u[2], v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          u[j] = fma2(x[j], cx[j], mul2(y[j], sx[j]));
          v[j] = fma2(y[j], cy[j], mul2(x[j], sy[j]));
        }
        if (GAINS && norm) {
          const float2 s2 = unpair(fma2(y[1], y[1], fma2(y[0], y[0], fma2(x[1], x[1], mul2(x[0], x[0])))));
          float ss = s2.x + s2.y;
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(ss * (1.f / kHeadDim) + a.eps);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            u[j] = mul2(u[j], pair(inv, inv));
            v[j] = mul2(v[j], pair(inv, inv));
          }
        }
        char* to_row = dst(r);
        *reinterpret_cast<uint2*>(to_row) = make_uint2(pack2<T>(unpair(u[0])), pack2<T>(unpair(u[1])));
        *reinterpret_cast<uint2*>(to_row + kRow / 2) = make_uint2(pack2<T>(unpair(v[0])), pack2<T>(unpair(v[1])));
      }
    };
    const int q_end = min(max(a.Hq - h0, 0), nh), k_end = min(max(a.Hq + a.Hkv - h0, 0), nh);
    if (q_end > 0 || (k_end > 0 && at >= 0)) factors(q_end > 0 ? a.q_gain : a.k_gain);
    wait_phase(&full[st], round & 1);
    char* q_out = a.q_out + t * a.qo_stride + h0 * kRow + c * 8;
    char* k_out = a.kp + at + (h0 - a.Hq) * a.head_stride + c * 8;
    if (!GAINS && at >= 0) {
      // the same factors for queries and keys: one loop
      turn(0, k_end, false, [&](int r) { return r < q_end ? q_out + r * kRow : k_out + r * a.head_stride; });
    } else {
      if (q_end > 0) turn(0, q_end, a.q_gain != nullptr, [&](int r) { return q_out + r * kRow; });
      if (at >= 0 && k_end > q_end) {
        if (q_end > 0) factors(a.k_gain);
        turn(q_end, k_end, a.k_gain != nullptr, [&](int r) { return k_out + r * a.head_stride; });
      }
    }
    if (at >= 0) {
#pragma unroll 2
      for (int r = k_end + (lane >> 4); r < nh; r += 2)
        *reinterpret_cast<uint4*>(a.vp + at + (h0 + r - a.Hq - a.Hkv) * a.head_stride + c * 16) =
            *reinterpret_cast<const uint4*>(ring + st * unit_bytes + r * kRow + c * 16);
    }
    __syncwarp();
    copy(u + kRopeStages * step, st);
    if (++st == kRopeStages) {
      st = 0;
      ++round;
    }
  }
}

template <typename T, bool GAINS>
cudaError_t launch_rope(const RopeArgs& a, int grid, size_t smem, cudaStream_t s) {
  using Shape = RopeShape<GAINS>;
  const cudaError_t e = allow_smem<qk_rope_append_kernel<T, GAINS>>(Shape::kWarps * Shape::kStages * kRopeHeads * 256);
  if (e != cudaSuccess) return e;
  qk_rope_append_kernel<T, GAINS><<<grid, Shape::kWarps * 32, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace vv

extern "C" vv_status vv_paged_plan(const int32_t* lens, const int32_t* new_lens, int32_t B,
                                   int32_t prefix_len, int32_t page_size, int32_t pages,
                                   const int32_t* free_pages, int32_t n_free,
                                   const int32_t* cursor, int32_t* block_tables,
                                   int32_t max_blocks, int32_t* lens_out, int32_t* offsets,
                                   int64_t* slots, int32_t* positions, int32_t max_tokens,
                                   int32_t* cursor_out, vv_stream stream) {
  VV_CHECK_ARG(lens && new_lens && block_tables && lens_out && offsets && slots && positions &&
                   cursor_out && (free_pages || n_free == 0),
               "vv_paged_plan: null pointer");
  VV_CHECK_ARG(vv::aligned16(slots) && vv::aligned16(positions),
               "vv_paged_plan: slots and positions must be 16-byte aligned");
  VV_CHECK_SHAPE(B >= 1 && B <= vv::kPlanMaxB, "vv_paged_plan: B=%d (1..%d)", B, vv::kPlanMaxB);
  VV_CHECK_SHAPE(page_size >= 1 && pages >= 1 && (int64_t)pages * page_size < (int64_t(1) << 31),
                 "vv_paged_plan: %d pages of %d tokens", pages, page_size);
  VV_CHECK_SHAPE(prefix_len >= 0 && n_free >= 0 && max_blocks >= 1 && max_tokens >= 1 &&
                     max_tokens <= 0x7ffffff0,
                 "vv_paged_plan: prefix_len=%d n_free=%d max_blocks=%d max_tokens=%d", prefix_len,
                 n_free, max_blocks, max_tokens);
  // every CTA reads the inputs for itself while others already write the outputs
  struct Span {
    const void* at;
    size_t bytes;
    bool meets(const Span& o) const {
      const char *x = static_cast<const char*>(at), *y = static_cast<const char*>(o.at);
      return x && y && x < y + o.bytes && y < x + bytes;
    }
  };
  const size_t nb = (size_t)B * 4, nt = (size_t)max_tokens;
  const Span in[] = {{lens, nb}, {new_lens, nb}, {free_pages, (size_t)n_free * 4}, {cursor, 4}};
  const Span outs[] = {{block_tables, nb * max_blocks}, {lens_out, nb},   {offsets, nb + 4},
                       {slots, nt * 8},                 {positions, nt * 4}, {cursor_out, 4}};
  for (const Span& o : outs) {
    for (const Span& i : in)
      VV_CHECK_ARG(!o.meets(i), "vv_paged_plan: an output overlaps lens, new_lens, free_pages or cursor");
    for (const Span* p = outs; p != &o; ++p) VV_CHECK_ARG(!o.meets(*p), "vv_paged_plan: two outputs overlap");
  }
  // division by page_size as a product: with l = ceil(log2 page_size), m = floor(2^(31 + l) / page_size)
  // + 1 is off by less than 2^l / 2^(31 + l) relative, too little to matter below 2^31
  unsigned magic = 0;
  int shift = 0;
  if (page_size > 1) {
    while ((int64_t(1) << shift) < page_size) ++shift;
    magic = (unsigned)((uint64_t(1) << (31 + shift)) / (unsigned)page_size + 1);
    shift -= 1;  // of the upper word of the product
  }
  vv::PlanArgs a = {lens,  new_lens,   free_pages, cursor, block_tables, lens_out,
                    offsets, slots, positions, cursor_out, B, prefix_len,
                    page_size, n_free, pages, max_blocks, max_tokens, magic, shift};
  const size_t smem = (size_t)((B + 4) & ~3) * 12;
  VV_CUDA(vv::allow_smem<vv::paged_plan_kernel>((vv::kPlanMaxB + 4) * 12));
  // one CTA per 2048 tokens, at most one per SM, since each repeats the scan: 12.2 us for 4096
  // requests with 778k tokens, 16.4 us with three per SM
  const int64_t per = vv::kPlanThreads * 4;
  const int grid = (int)std::min<int64_t>(vv::sm_count(), ((int64_t)max_tokens + per - 1) / per);
  vv::paged_plan_kernel<<<grid, vv::kPlanThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return vv::cuda_check(cudaGetLastError(), "vv_paged_plan launch");
}

extern "C" vv_status vv_qk_rope_append(const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const void* v, int64_t v_stride,
                                       int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                       const void* q_gain, const void* k_gain, float eps,
                                       const int32_t* positions, float theta,
                                       const int64_t* slots, const vv_paged_kv* kv, void* q_out,
                                       int64_t q_out_stride, vv_stream stream) {
  VV_CHECK_ARG(q && k && v && positions && slots && kv && q_out, "vv_qk_rope_append: null pointer");
  vv_status st = vv::check_paged_kv(kv, Hkv, D, "vv_qk_rope_append");
  if (st != VV_OK) return st;
  VV_CHECK_ARG(vv::aligned16(q) && vv::aligned16(k) && vv::aligned16(v) && vv::aligned16(q_out) &&
                   vv::aligned16(q_gain) && vv::aligned16(k_gain),
               "vv_qk_rope_append: pointers must be 16-byte aligned");
  VV_CHECK_SHAPE(T >= 1 && T < (int64_t(1) << 31), "vv_qk_rope_append: T=%lld", (long long)T);
  VV_CHECK_SHAPE(Hq >= 1 && Hq <= 1024, "vv_qk_rope_append: Hq=%d", Hq);
  VV_CHECK_SHAPE(q_stride % 8 == 0 && k_stride % 8 == 0 && v_stride % 8 == 0 &&
                     q_out_stride % 8 == 0 && q_stride >= 0 && k_stride >= 0 && v_stride >= 0 &&
                     (T == 1 || q_out_stride >= (int64_t)Hq * D),
                 "vv_qk_rope_append: row strides must be multiples of 8 elements and output rows "
                 "must not overlap");
  VV_CHECK_ARG(theta > 0.f && std::isfinite(theta) && eps >= 0.f && std::isfinite(eps),
               "vv_qk_rope_append: theta=%g eps=%g", theta, eps);
  // in place (same rows) or apart: a warp reads a whole head row before it writes it
  const char* q0 = static_cast<const char*>(q);
  const char* o0 = static_cast<const char*>(q_out);
  const int64_t q_bytes = ((T - 1) * q_stride + (int64_t)Hq * D) * 2;
  const int64_t o_bytes = ((T - 1) * q_out_stride + (int64_t)Hq * D) * 2;
  VV_CHECK_ARG((q0 == o0 && (T == 1 || q_stride == q_out_stride)) || q0 + q_bytes <= o0 ||
                   o0 + o_bytes <= q0,
               "vv_qk_rope_append: q_out must be q itself (same stride) or not overlap it");
  // keys and values are read by other warps while q_out's rows are written: apart, or between its rows
  // (parts of one fused buffer: the same stride)
  auto meets = [&](const void* p, int64_t stride) {
    const char* x = static_cast<const char*>(p);
    const int64_t row = (int64_t)Hkv * D * 2, out_row = (int64_t)Hq * D * 2, s = stride * 2;
    if (x + (T - 1) * s + row <= o0 || o0 + o_bytes <= x) return false;
    if (T == 1 || stride != q_out_stride) return true;
    const int64_t d = ((x - o0) % s + s) % s;  // from a row of q_out to the next row of p
    return d < out_row || d + row > s;
  };
  VV_CHECK_ARG(!meets(k, k_stride) && !meets(v, v_stride), "vv_qk_rope_append: q_out must not overlap k and v");
  vv::RopeArgs a;
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.q_out = static_cast<char*>(q_out);
  a.kp = static_cast<char*>(kv->k);
  a.vp = static_cast<char*>(kv->v);
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.pos = positions;
  a.slots = slots;
  a.q_stride = q_stride * 2;
  a.k_stride = k_stride * 2;
  a.v_stride = v_stride * 2;
  a.qo_stride = q_out_stride * 2;
  a.page_stride = kv->page_stride * 2;
  a.head_stride = kv->head_stride * 2;
  a.token_stride = kv->token_stride * 2;
  a.n_slots = (int64_t)kv->pages * kv->page_size;
  a.T = (int)T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.ps = kv->page_size;
  a.eps = eps;
  a.quarters[0] = 2.0 / 3.14159265358979323846;
  for (int n = 1; n < D / 2; n *= 2) {  // theta^(-2 i / D) from the powers of i's bits
    const double f = std::pow((double)theta, -2.0 * n / D);
    for (int i = 0; i < n; ++i) a.quarters[n + i] = a.quarters[i] * f;
  }
  // a token in as few units of at most 18 heads as there are warps for, in smaller ones (an even
  // number of heads, two rows at a time) when tokens are few
  const int heads = Hq + 2 * Hkv;
  const bool gains = q_gain || k_gain;
  const int cta_warps = gains ? vv::RopeShape<true>::kWarps : vv::RopeShape<false>::kWarps;
  const int stages = gains ? vv::RopeShape<true>::kStages : vv::RopeShape<false>::kStages;
  const int64_t warps = 2 * vv::sm_count() * cta_warps;
  int64_t parts = (heads + vv::kRopeHeads - 1) / vv::kRopeHeads;
  parts = std::max(parts, std::min<int64_t>((heads + 1) / 2, warps / T));
  a.heads = (int)((heads + parts - 1) / parts + 1) / 2 * 2;
  a.parts = (heads + a.heads - 1) / a.heads;
  const int64_t units = T * a.parts;
  const int grid = (int)std::min<int64_t>((units + cta_warps - 1) / cta_warps, 2 * vv::sm_count());
  const size_t smem = (size_t)cta_warps * stages * a.heads * D * 2;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f16 = kv->dtype == VV_F16;
  const cudaError_t e = f16 ? (gains ? vv::launch_rope<__half, true>(a, grid, smem, s) : vv::launch_rope<__half, false>(a, grid, smem, s))
                            : (gains ? vv::launch_rope<__nv_bfloat16, true>(a, grid, smem, s)
                                     : vv::launch_rope<__nv_bfloat16, false>(a, grid, smem, s));
  return vv::cuda_check(e, "vv_qk_rope_append launch");
}
