// Shared-prefix attention (internal): the two kernels behind vv_gqa_prefix_attn.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace vv {

constexpr int kPartRow = 132;  // floats of a partial row: o[128] (not normalised), m (log2), l, pad

// The shared prompt: every row (sequence, query head of the group) of a key-value head against
// the same keys.
struct PrefixTcArgs {
  const void* q;        // [B, Hq, D], rows q_stride apart
  const void* k;        // [Hkv, P, D] with strides `head`, `token` (elements)
  const void* v;
  float* part;          // [Hkv][splits][B * G][kPartRow]
  int64_t q_stride, head, token;
  int B, Hkv, G, P;
  int splits, per;      // parts of the keys, 128-key blocks per part
  float c;              // scale * log2(e)
  int dtype;            // VV_F16 / VV_BF16
};
// Parts of the prompt's keys (and 128-key blocks per part) for `rows` rows per key-value head.
void prefix_tc_split(int rows, int Hkv, int P, int* splits, int* per);
// Upper bound of splits x rows x Hkv over all smaller numbers of rows and prompts.
int64_t prefix_tc_most_rows(int rows, int Hkv, int P);
cudaError_t launch_prefix_tc(const PrefixTcArgs& a, cudaStream_t s);

}  // namespace vv
