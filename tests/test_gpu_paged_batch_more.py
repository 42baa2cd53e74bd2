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


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("B,P,n", [(1, 0, 16 * 3000), (3, 18 * 6 * 128, 0), (2, 4096, 16 * 500), (1, 20000, 0)])
def test_prefix_attn_weights_far_below_the_largest(vv, dtype, B, P, n):  # noqa: F811
    """Every 16th key takes all but e^-17.5 of a key's weight and has a value of zero: the result is what the
    others carry together.  fp16 weights below 2^-20 of the largest are off by 2^-31 of it at most, larger ones
    by half a step."""
    hkv, hq = 8, 16
    k16 = torch.zeros((16, 128), device="cuda")
    k16[1:, 0] = -17.5
    v16 = torch.full((16, 128), 1000.0, device="cuda")
    v16[0] = 0
    page = lambda x: x.expand(1, hkv, 16, 128).to(dtype).contiguous()  # noqa: E731
    kv = vv.PagedKV(page(k16), page(v16))
    pre = [x.repeat(P // 16, 1).expand(hkv, P, 128).to(dtype).contiguous() if P else None for x in (k16, v16)]
    q = torch.zeros((B, hq, 128), dtype=dtype, device="cuda")
    q[:, :, 0] = math.sqrt(128)
    table = torch.zeros((B, max(1, n // 16)), dtype=torch.int32, device="cuda")
    ws = torch.empty(vv.vv_gqa_prefix_attn_workspace_size(B, hq, hkv, 128, P, 16 * table.shape[1]), dtype=torch.uint8, device="cuda")
    lse = torch.empty((B, hq), device="cuda")
    scale = 1 / math.sqrt(128)
    out = vv.vv_gqa_prefix_attn(q, *pre, kv, table, i32([n] * B), scale, ws, lse=lse)
    vv.vv_sync_status()
    w = math.exp(-17.5 * q[0, 0, 0].item() * scale)
    y, total = 1000 * 15 * w / (1 + 15 * w), 1 + 15 * w
    u = u_of(dtype)
    bound = 2 * u * y + 2.0 ** -19 * y + (1000 * 15 * 2.0 ** -31 + 2.0 ** -25 if dtype == F16 else 0.0)
    assert np.max(np.abs(host(out) - y)) <= bound, (out.flatten()[:4].tolist(), y, bound)
    assert np.max(np.abs(host(lse) - math.log((P + n) / 16 * total))) <= 1e-5


@pytest.mark.parametrize("B,P,n", [(1, 0, 500), (4, 1500, 40)])
def test_prefix_attn_scores_of_millions(vv, B, P, n):  # noqa: F811
    """One key takes all, whatever the score's size in fp32: no weight passes the type's largest value."""
    c = attn_case(vv, B, 12, 2, P, [n] * B, 16, F16, seed=31)
    for t in (c["kpre"], c["kv"].k):
        if t is not None:
            t[..., 0] = torch.randperm(t[..., 0].numel(), device="cuda").view(t[..., 0].shape).to(F16) * 8
    c["q"][:, :, 0] = 2000.0
    c["q"][:, 1::2, 0] *= -1
    c["qh"], c["kph"] = host(c["q"]), host(c["kv"].k)
    c["kpreh"] = host(c["kpre"]) if P else None
    out, lse = attn_run(vv, c)
    vv.vv_sync_status()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("gains", [False, True])
def test_rope_append_small_angles(vv, dtype, gains):  # noqa: F811
    """Where a partner is zero the rotated value is x cos or x sin alone, and its error one rounding: the
    angle (reduced in fp64) is off by 2^-24 of itself, up to 2 pi 2^-26 where it is reduced, a sine and
    cosine by 2 of their last places (2^-24 below 1), products and a norm by 2^-20 of the value."""
    T, hq, hkv, theta = 64, 4, 2, 1e6
    x, xh = values((T, hq + 2 * hkv, 128), dtype, 21)
    x[:, ::2, 64:] = 0
    x[:, 1::2, :64] = 0
    xh = host(x)
    g, gh = values((128,), dtype, 22) if gains else (None, None)
    kv, kp, vp = pools(vv, T // 16, hkv, 16, dtype, 23)
    pos = np.concatenate([np.arange(-8, 24), 10 ** np.arange(8), 1000 + np.arange(24)])
    slots = np.arange(T)
    out = vv.vv_qk_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], i32(pos), torch.tensor(slots).cuda(), kv,
                               theta, q_gain=g, k_gain=g)
    vv.vv_sync_status()
    yq, yk, _ = obatch.qk_rope_append(xh[:, :hq], xh[:, hq:hq + hkv], xh[:, hq + hkv:], pos, slots, kp, vp, theta, gh, gh)
    angle = np.abs(pos[:, None].astype(np.float64) * theta ** (-2.0 * np.arange(64) / 128))
    angle = np.minimum(np.concatenate([angle, angle], -1), 1.0)[:, None]

    def bound(y, heads):
        n = obatch.ops.rmsnorm(heads, gh, 1e-6) if gains else heads
        a = np.abs(n) + np.abs(np.roll(n, 64, axis=-1))
        return (u_of(dtype) + 2.0 ** -20) * np.abs(y) + 2.0 ** -22 * a * angle + (2.0 ** -25 if dtype == F16 else 0.0)

    assert np.all(np.abs(host(out) - yq) <= bound(yq, xh[:, :hq]))
    cells = lambda pages: pages.swapaxes(1, 2).reshape(T, hkv, 128)  # noqa: E731
    got, want = cells(host(kv.k)), cells(yk)
    assert np.all(np.abs(got - want) <= bound(want, xh[:, hq:hq + hkv]))


@pytest.mark.parametrize("theta", [1e-9, 0.5, 3.4e38])
def test_rope_append_any_theta_rotates(vv, theta):  # noqa: F811
    """Angles beyond what 64 bits resolve still turn by some angle: a pair keeps its length."""
    x, xh = values((40, 3, 128), F16, 41)
    kv, _, _ = pools(vv, 3, 1, 16, F16, 42)
    pos = [0, 1, -1, 2 ** 31 - 1, -2 ** 31] * 8
    out = vv.vv_qk_rope_append(x[:, :1], x[:, 1:2], x[:, 2:], i32(pos), torch.arange(40, device="cuda"), kv, theta)
    vv.vv_sync_status()
    length = lambda y: np.hypot(y[..., :64], y[..., 64:])  # noqa: E731
    assert np.all(np.abs(length(host(out)) - length(xh[:, :1])) <= 2 * u_of(F16) * length(xh[:, :1]) + 2.0 ** -24)


def test_logits_argmax_that_is_neither_true_nor_false(vv):  # noqa: F811
    x = torch.zeros((2, 100), device="cuda")
    ws = torch.zeros(vv.vv_logits_process_workspace_size(2), dtype=torch.uint8, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        vv.vv_logits_process(x, ws, argmax=torch.ones(2))
    assert vv.vv_logits_process(x, ws, argmax=torch.ones(1))[1].tolist() == [0, 0]


def test_prefix_attn_smaller_batches_on_the_largest_ones_workspace(vv):  # noqa: F811
    """Sequences finish and a shorter prompt follows: the workspace of the largest call still serves, with the
    bits of a workspace of the call's own."""
    B, P, width = 16, 4096, 20
    ws = torch.empty(vv.vv_gqa_prefix_attn_workspace_size(B, 12, 2, 128, P, width * 16), dtype=torch.uint8, device="cuda")
    for b, p in ((16, 4096), (16, 3968), (11, 4096), (11, 2000), (2, 4096), (2, 130), (1, 4096), (3, 0)):
        c = attn_case(vv, b, 12, 2, p, [(17 * i) % 300 for i in range(b)], 16, F16, seed=b + p, max_blocks=width)
        out, lse = attn_run(vv, c, ws)
        own, own_lse = attn_run(vv, c)
        vv.vv_sync_status()
        assert torch.equal(out, own) and torch.equal(lse, own_lse)
        if p <= 2000:
            attn_check(c, out, lse)


@pytest.mark.parametrize("B,hq,hkv,P", [(65535, 1, 1, 200), (65535, 4, 1, 0), (3, 1024, 1024, 300), (1, 16384, 1024, 130)])
def test_prefix_attn_largest_batches_and_head_counts(vv, B, hq, hkv, P):  # noqa: F811
    """Rows at both ends of the range and between, against the formula in 64 bits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(B + hq)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda").to(F16)  # noqa: E731
    q, kv = normal(B, hq, 128), vv.PagedKV(normal(5, hkv, 16, 128), normal(5, hkv, 16, 128))
    pre = [normal(hkv, P, 128) if P else None for _ in range(2)]
    lens = torch.randint(-1, 40, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0], lens[-1] = 39, 17
    tables = torch.randint(0, 5, (B, 3), generator=g, device="cuda", dtype=torch.int32)
    ws = torch.empty(vv.vv_gqa_prefix_attn_workspace_size(B, hq, hkv, 128, P, 48), dtype=torch.uint8, device="cuda")
    lse = torch.full((B, hq), 77.0, device="cuda")
    out = vv.vv_gqa_prefix_attn(q, *pre, kv, tables, lens, 1 / math.sqrt(128), ws, lse=lse)
    vv.vv_sync_status()
    u = u_of(F16)
    for b in sorted({0, 1, 127, 128, B // 2, B - 1} & set(range(B))):
        n = int(lens[b])
        for h in sorted({0, hq // 2, hq - 1}):
            if n < 0:
                assert lse[b, h] == 77.0
                continue
            keys, vals = (torch.cat(([p[h * hkv // hq]] if P else []) + [x[int(t), h * hkv // hq] for t in tables[b]])[: P + n].double()
                          for p, x in zip(pre, (kv.k, kv.v)))
            if P + n == 0:
                assert torch.all(out[b, h] == 0) and torch.isneginf(lse[b, h])
                continue
            s = keys @ q[b, h].double() / math.sqrt(128)
            w = torch.softmax(s, 0)
            y, mean = w @ vals, w @ vals.abs()
            # as in test_gpu_paged_batch: one rounding of the result, one of each weight, scores in fp32
            assert torch.all((out[b, h].double() - y).abs() <= u * y.abs() + (u + 2.0 ** -13) * mean + 2.0 ** -24)
            assert abs(lse[b, h].item() - torch.logsumexp(s, 0).item()) <= 1e-4
