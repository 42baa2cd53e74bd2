"""Argument checks of the batch operators, before anything reaches a GPU (CPU only): through the C
ABI with addresses that are never dereferenced, and through the binding with CPU tensors."""

import ctypes

import pytest
import torch

vv = pytest.importorskip("int4_blockwise_quantised_b200._vv")

BASE = 1 << 20
A, S, C = vv.VV_ERR_INVALID_ARG, vv.VV_ERR_SHAPE, vv.VV_ERR_CAPACITY


def addr(i):
    """Addresses far apart, 16-byte aligned."""
    return BASE + (i << 32)


def call(fn, args, **change):
    args = dict(args, **change)
    return getattr(vv.lib, fn)(*args.values())


PLAN = dict(lens=addr(0), new=addr(1), B=4, prefix=0, ps=16, pages=10, free=addr(2), n_free=5,
            cursor=None, table=addr(3), max_blocks=3, lens_out=addr(4), offsets=addr(5),
            slots=addr(6), positions=addr(7), max_tokens=8, cursor_out=addr(8), stream=None)


@pytest.mark.parametrize("code,change", [
    (A, dict(lens=None)), (A, dict(table=None)), (A, dict(free=None)), (A, dict(cursor_out=None)),
    (A, dict(slots=addr(6) + 8)), (A, dict(positions=addr(7) + 4)), (S, dict(B=0)),
    (S, dict(B=16385)), (S, dict(ps=0)), (S, dict(pages=0)), (S, dict(pages=1 << 28)),
    (S, dict(prefix=-1)), (S, dict(n_free=-1)), (S, dict(max_blocks=0)), (S, dict(max_tokens=0)),
    (A, dict(lens_out=addr(0))), (A, dict(lens_out=addr(1) + 8)),
    (A, dict(cursor=addr(8), cursor_out=addr(8)))])
def test_plan_refuses(code, change):
    assert call("vv_paged_plan", PLAN, **change) == code, (change, vv.last_error())


def pool(**change):
    f = dict(k=addr(20), v=addr(21), page_stride=2 * 16 * 128, head_stride=16 * 128,
             token_stride=128, pages=8, page_size=16, dtype=vv.VV_F16)
    f.update(change)
    return ctypes.byref(vv.vv_paged_kv(*f.values()))


BAD_POOLS = [
    (A, dict(k=None)), (A, dict(v=addr(21) + 8)), (A, dict(dtype=vv.VV_F32)), (S, dict(pages=0)),
    (S, dict(page_size=0)), (S, dict(page_size=24)), (S, dict(page_size=8)),
    (S, dict(page_size=16, pages=1 << 27)), (S, dict(token_stride=64)), (S, dict(token_stride=132)),
    (S, dict(page_stride=-4096)), (S, dict(head_stride=100))]

ROPE = dict(q=addr(0), qs=512, k=addr(1), ks=256, v=addr(2), vs=256, T=3, Hq=4, Hkv=2, D=128,
            qg=None, kg=None, eps=1e-6, pos=addr(3), theta=1e6, slots=addr(4), kv=pool(),
            out=addr(5), os=512, stream=None)


@pytest.mark.parametrize("code,change", [
    (A, dict(q=None)), (A, dict(slots=None)), (A, dict(out=None)), (A, dict(kv=None)),
    (A, dict(k=addr(1) + 2)), (A, dict(qg=addr(9) + 2)), (S, dict(T=0)), (S, dict(T=1 << 31)),
    (S, dict(Hq=0)), (S, dict(Hkv=0)), (S, dict(D=64)), (S, dict(qs=516)), (S, dict(os=256)),
    (S, dict(vs=-256)), (A, dict(theta=0.0)), (A, dict(theta=float("inf"))), (A, dict(eps=-1.0)),
    (A, dict(eps=float("nan"))), (A, dict(out=addr(0), os=520)), (A, dict(out=addr(0) + 256))])
def test_rope_append_refuses(code, change):
    assert call("vv_qk_rope_append", ROPE, **change) == code, (change, vv.last_error())


@pytest.mark.parametrize("code,change", BAD_POOLS)
def test_bad_pools_are_refused(code, change):
    assert call("vv_qk_rope_append", ROPE, kv=pool(**change)) == code, (change, vv.last_error())
    assert call("vv_gqa_prefix_attn", ATTN, kv=pool(**change)) == code, (change, vv.last_error())


ATTN = dict(q=addr(0), qs=512, B=3, Hq=4, Hkv=2, D=128, kp=addr(1), vp=addr(2), ph=100 * 128,
            pt=128, P=100, kv=pool(), table=addr(3), max_blocks=4, lens=addr(4), scale=0.1,
            out=addr(5), os=512, lse=None, ws=addr(6), n=1 << 30, stream=None)


@pytest.mark.parametrize("code,change", [
    (A, dict(q=None)), (A, dict(table=None)), (A, dict(lens=None)), (A, dict(ws=None)),
    (A, dict(kp=None)), (A, dict(vp=addr(2) + 8)), (A, dict(out=addr(5) + 2)), (S, dict(B=0)),
    (S, dict(B=65536)), (S, dict(Hq=5)), (S, dict(Hq=34)), (S, dict(Hkv=0)), (S, dict(D=64)),
    (S, dict(P=-1)), (S, dict(P=1 << 24)), (S, dict(pt=64)), (S, dict(pt=132)), (S, dict(ph=-8)),
    (S, dict(qs=516)), (S, dict(os=256)), (S, dict(max_blocks=0)), (A, dict(scale=0.0)),
    (A, dict(scale=-1.0)), (A, dict(scale=float("nan"))), (A, dict(scale=float("inf"))),
    (C, dict(n=8))])
def test_prefix_attn_refuses(code, change):
    assert call("vv_gqa_prefix_attn", ATTN, **change) == code, (change, vv.last_error())


def test_workspace_sizes():
    size = vv.vv_gqa_prefix_attn_workspace_size
    assert size(3, 4, 2, 128, 100, 64) > 0
    for bad in ((0, 4, 2, 128, 100, 64), (3, 5, 2, 128, 100, 64), (3, 4, 2, 64, 100, 64),
                (3, 4, 2, 128, -1, 64), (3, 4, 2, 128, 100, -1)):
        assert size(*bad) == 0
    assert vv.vv_logits_process_workspace_size(7) > 0 and vv.vv_logits_process_workspace_size(0) == 0


def rules(**change):
    f = dict(tokens=addr(30), tokens_stride=50, token_lens=addr(31), prompt_lens=None,
             max_tokens=50, repetition=None, frequency=None, presence=None, bias_ids=addr(32),
             bias_vals=addr(33), bias_offsets=addr(34), n_bias=3, mask=addr(35), mask_stride=32)
    f.update(change)
    return ctypes.byref(vv.vv_logits_rules(*f.values()))


LOGITS = dict(x=addr(0), xs=1000, dtype=vv.VV_F32, B=2, V=1000, rules=rules(), out=addr(1), os=1000,
              argmax=addr(2), ws=addr(3), n=1 << 20, stream=None)


@pytest.mark.parametrize("code,change", [
    (A, dict(x=None)), (A, dict(out=None)), (A, dict(rules=None)), (A, dict(dtype=3)),
    (A, dict(x=addr(0) + 2)), (S, dict(B=0)), (S, dict(B=65536)), (S, dict(V=0)),
    (S, dict(V=1 << 30)), (S, dict(xs=999)), (S, dict(os=999)), (A, dict(out=addr(0), os=1001)),
    (A, dict(out=addr(0) + 400)), (A, dict(ws=None)), (A, dict(ws=addr(3) + 8)), (C, dict(n=16)),
    (A, dict(rules=rules(token_lens=None))), (S, dict(rules=rules(max_tokens=1 << 24))),
    (S, dict(rules=rules(tokens_stride=49))), (A, dict(rules=rules(bias_vals=None))),
    (A, dict(rules=rules(bias_offsets=None))), (A, dict(rules=rules(n_bias=-1))),
    (S, dict(rules=rules(mask_stride=31)))])
def test_logits_process_refuses(code, change):
    assert call("vv_logits_process", LOGITS, **change) == code, (change, vv.last_error())


def test_binding_refuses_cpu_tensors_and_bad_pools():
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(vv.VVError) as e:
        vv.vv_paged_plan(i32, i32, torch.zeros(4, 2, dtype=torch.int32), i32, 16, 8, 4)
    assert e.value.code == A and "CUDA" in str(e.value)
    with pytest.raises(vv.VVError):
        vv.vv_logits_process(torch.zeros(2, 8))
    kv = torch.zeros(2, 1, 16, 128, dtype=torch.float16)
    with pytest.raises(vv.VVError):
        vv.PagedKV(kv, kv)  # not on a GPU
    with pytest.raises(vv.VVError):
        vv.PagedKV(kv.float(), kv.float())
    with pytest.raises(vv.VVError):
        vv.PagedKV(kv, kv[:1])
    with pytest.raises(vv.VVError):
        vv.PagedKV(kv.transpose(2, 3), kv.transpose(2, 3))
