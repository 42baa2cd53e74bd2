"""More GPU tests of the operators of a batch that continues one shared prompt: calls that their documentation
allows and that once went wrong.  Tolerances as derived in test_gpu_paged_batch."""

import math

import numpy as np
import pytest
import torch

from oracle import batch as obatch
from test_gpu_paged_batch import BF16, F16, attn_case, attn_check, attn_run, host, i32, pools, rope_bound, u_of, values, vv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 6])
def test_rope_append_in_place_within_a_fused_projection(vv, T):  # noqa: F811
    hq, hkv = 4, 2
    fused, fh = values((T, hq + 2 * hkv, 128), F16, 11)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    kv, kp, vp = pools(vv, 2, hkv, 16, F16, 12)
    pos, slots = 100 + np.arange(T), np.arange(T)[::-1].copy()
    out = vv.vv_qk_rope_append(q, k, v, i32(pos), torch.tensor(slots).cuda(), kv, 1e6, out=q)
    vv.vv_sync_status()
    assert out.data_ptr() == fused.data_ptr() and np.array_equal(host(fused)[:, hq:], fh[:, hq:])
    yq, yk, yv = obatch.qk_rope_append(fh[:, :hq], fh[:, hq:hq + hkv], fh[:, hq + hkv:], pos, slots, kp, vp, 1e6)
    assert np.all(np.abs(host(q) - yq) <= rope_bound(yq, fh[:, :hq], F16))
    assert np.array_equal(host(kv.v), yv)
    with pytest.raises(vv.VVError) as e:  # a head further on: over the first key head
        vv.vv_qk_rope_append(q, k, v, i32(pos), torch.tensor(slots).cuda(), kv, 1e6, out=fused[:, 1:1 + hq])
    assert e.value.code == vv.VV_ERR_INVALID_ARG


def test_prefix_attn_of_as_many_keys_as_a_length_can_name(vv):  # noqa: F811
    """2^31 - 1 keys, all of one page whose keys are equal: their mean is its value, their number in lse."""
    k, v = (torch.full((1, 1, 16, 128), x, dtype=F16, device="cuda") for x in (0.25, 3.0))
    kv, n = vv.PagedKV(k, v), 2 ** 31 - 1
    q = torch.full((1, 1, 128), 0.5, dtype=F16, device="cuda")
    table = torch.zeros((1, 2 ** 27), dtype=torch.int32, device="cuda")
    ws = torch.empty(vv.vv_gqa_prefix_attn_workspace_size(1, 1, 1, 128, 0, 2 ** 31), dtype=torch.uint8, device="cuda")
    lse = torch.empty((1, 1), device="cuda")
    out = vv.vv_gqa_prefix_attn(q, None, None, kv, table, i32([n]), 0.125, ws, lse=lse)
    vv.vv_sync_status()
    assert torch.all(out == 3.0)
    assert abs(lse.item() - (0.5 * 0.25 * 128 * 0.125 + math.log(n))) <= 1e-5  # 23.5 in fp32 steps
