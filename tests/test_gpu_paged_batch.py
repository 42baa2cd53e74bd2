"""GPU parity of the operators of a batch that continues one shared prompt, against oracle.batch.

Tolerances are per element and derived from the arithmetic, with u = finfo(type).eps / 2 (half a
step of the stored type, relative):
  vv_paged_plan       integers: equal.
  vv_qk_rope_append   one rounding u |y|, plus the fp32 arithmetic before it: the angle is reduced
                      in fp64 and rounded once (2^-24 of at most half a turn: 2e-7), sine and
                      cosine are off by a few 2^-24, a norm by a few 2^-24 more: 2^-19 of
                      |x_i| + |x_{i+64}| covers all of it.
  vv_gqa_prefix_attn  one rounding u |out|; every weight rounded once, u sum p|v| / L; scores in
                      fp32 (128 products of which the largest sums here are below 64 in the log2
                      domain: relative error of a weight below 2^-13); fp16 weights below 2^-14
                      are off by up to 2^-25 absolute each, n of them against a total of at least
                      L.
  vv_logits_process   fp32 operations, each rounded once: at most 6 of them, 2^-24 relative to
                      values of at most `big`; then u |x|.  Greedy tokens equal where the winner's
                      lead is larger than that.
"""

import math

import numpy as np
import pytest
import torch

import synth
from helpers import TOL, normwise
from oracle import batch as obatch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def vv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from int4_blockwise_quantised_b200 import _vv

    return _vv


def u_of(dtype):
    return torch.finfo(dtype).eps / 2


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def values(shape, dtype, seed, std=1.0):
    """A device tensor of `dtype` and the same values in float64."""
    t = torch.from_numpy(synth.normal_f32(shape, std, seed)).to(dtype)
    return t.cuda(), t.double().numpy()


def host(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------------- plan
def plan_case(B, max_len, max_new, ps, seed, spare=3):
    r = synth.rng(seed)
    lens = r.integers(0, max_len + 1, B)
    new = r.integers(0, max_new + 1, B)
    old, need = -(-lens // ps), -(-(lens + new) // ps)
    pages = int(need.sum()) + 7
    order = r.permutation(pages)
    tables = np.full((B, max(int(need.max()), 1) + spare), -1)
    at = 0
    for b in range(B):
        tables[b, : old[b]] = order[at:at + old[b]]
        at += old[b]
    return lens, new, tables, order[at:], pages, int(new.sum())


PLANS = [(1, 0, 1, 16, 0, 0), (1, 40, 3, 16, 7, 3), (3, 100, 1, 16, 4530, 0), (33, 5, 0, 16, 0, 5),
         (64, 300, 40, 48, 1, 2), (500, 64, 9, 1, 0, 0), (513, 2000, 6, 128, 0, 1),
         (1025, 17, 5, 16, 3, 0), (16384, 3, 3, 16, 0, 9), (2, 10, 9000, 32, 0, 1)]


@pytest.mark.parametrize("B,max_len,max_new,ps,prefix,cursor", PLANS)
def test_plan(vv, B, max_len, max_new, ps, prefix, cursor):
    lens, new, tables, free, pages, total = plan_case(B, max_len, max_new, ps, B + ps)
    free = np.concatenate([np.full(cursor, 0), free])
    tokens = total + 1 + B % 7
    t = i32(tables)
    p = vv.vv_paged_plan(i32(lens), i32(new), t, i32(free), ps, pages, tokens, prefix_len=prefix,
                         cursor=i32([cursor]) if cursor else None)
    vv.vv_sync_status()
    after, offsets, slots, pos, want, cur = obatch.paged_plan(lens, new, tables, free, ps, tokens,
                                                              prefix, cursor)
    assert np.array_equal(p.lens.cpu().numpy(), after)
    assert np.array_equal(p.offsets.cpu().numpy(), offsets)
    assert np.array_equal(p.slots.cpu().numpy(), slots)
    assert np.array_equal(p.positions.cpu().numpy(), pos)
    assert np.array_equal(t.cpu().numpy(), want)
    assert p.cursor.item() == cur


def plan_error(vv, code, lens, new, tables, free, ps, pages, tokens, prefix=0):
    t = i32(tables)
    p = vv.vv_paged_plan(i32(lens), i32(new), t, i32(free), ps, pages, tokens, prefix_len=prefix)
    with pytest.raises(vv.VVError) as e:
        vv.vv_sync_status()
    assert e.value.code == code
    vv.vv_sync_status()  # cleared
    return p, t.cpu().numpy()


def test_plan_records_errors_and_stays_in_bounds(vv):
    T = [[5, -1], [6, -1], [-1, -1]]
    # a negative length appends nothing, the others are planned
    p, t = plan_error(vv, vv.VV_ERR_RANGE, [-3, 15, 0], [1, 2, 1], T, [1, 2, 3], 16, 8, 4)
    assert p.slots.cpu().tolist() == [6 * 16 + 15, 16, 32, -1] and t.tolist() == [[5, -1], [6, 1], [2, -1]]
    p, t = plan_error(vv, vv.VV_ERR_RANGE, [0, 15, 0], [-1, 2, 1], T, [1, 2, 3], 16, 8, 4)
    assert p.lens.cpu().tolist() == [0, 17, 1]
    # positions past 2^31 - 1; sums past 2^31
    big = 2 ** 31 - 1
    plan_error(vv, vv.VV_ERR_RANGE, [big, 1, 0], [1, 0, 0], T, [1], 16, 8, 4)
    plan_error(vv, vv.VV_ERR_RANGE, [big - 5, 1, 0], [1, 0, 0], T, [1], 16, 8, 4, prefix=10)
    p, t = plan_error(vv, vv.VV_ERR_CAPACITY, [0, 0, 0], [big, big, big], T, [1, 2], 1 << 20, 8, 9)
    assert p.offsets.cpu().tolist() == [0, 9, 9, 9] and p.slots.cpu().tolist()[0] == 1 << 20
    # the list runs out: -1, and the tokens without a page have slot -1
    p, t = plan_error(vv, vv.VV_ERR_CAPACITY, [16, 0, 0], [1, 1, 1], [[5, -1], [-1, -1], [-1, -1]],
                      [1, 2], 16, 8, 4)
    assert t.tolist() == [[5, 1], [2, -1], [-1, -1]]
    assert p.slots.cpu().tolist() == [16, 32, -1, -1] and p.cursor.item() == 3
    # a table too short
    p, t = plan_error(vv, vv.VV_ERR_CAPACITY, [30, 0, 0], [5, 1, 0], [[5, 4], [-1, -1], [-1, -1]],
                      [1, 2], 16, 8, 6)
    assert p.slots.cpu().tolist() == [4 * 16 + 14, 4 * 16 + 15, -1, -1, -1, 32] and t[1, 0] == 2
    # more tokens than rows
    p, t = plan_error(vv, vv.VV_ERR_CAPACITY, [0, 0, 0], [3, 3, 3], T, [1, 2, 3], 16, 8, 4)
    assert p.slots.cpu().tolist() == [16, 17, 18, 32] and p.offsets.cpu().tolist() == [0, 3, 4, 4]
    # page numbers outside the pool, from the list and from the table
    p, t = plan_error(vv, vv.VV_ERR_RANGE, [0, 15, 0], [1, 0, 1], T, [99, 3], 16, 8, 2)
    assert t.tolist() == [[-1, -1], [6, -1], [3, -1]] and p.slots.cpu().tolist() == [-1, 48]
    p, t = plan_error(vv, vv.VV_ERR_RANGE, [3, 15, 0], [1, 1, 0], [[-7, -1], [6, -1], [-1, -1]], [], 16, 8, 2)
    assert p.slots.cpu().tolist() == [-1, 6 * 16 + 15]


def test_plan_padding_rows_and_pages_past_a_table(vv):
    # padding rows at either end and between keep their mark, and take nothing
    t = i32([[-1, -1], [5, -1], [-1, -1], [6, -1], [-1, -1]])
    p = vv.vv_paged_plan(i32([-1, 16, -2 ** 31, 15, -7]), i32([0, 1, 0, 2, 0]), t, i32([1, 2, 3]), 16, 8, 5, prefix_len=9)
    vv.vv_sync_status()
    assert p.lens.tolist() == [-1, 17, -2 ** 31, 17, -7] and p.offsets.tolist() == [0, 0, 1, 1, 3, 3]
    assert p.slots.tolist() == [16, 6 * 16 + 15, 32, -1, -1] and p.positions.tolist() == [25, 24, 25, 0, 0]
    assert t.tolist() == [[-1, -1], [5, 1], [-1, -1], [6, 2], [-1, -1]] and p.cursor.item() == 2
    # thousands of pages past a table's end, before, between and after requests that fit
    n = 5000
    T = [[-1, -1], [-1, 7], [-1, -1], [-1, -1]]
    p, t = plan_error(vv, vv.VV_ERR_CAPACITY, [0, 0, 0, 0], [n, 1, n, 2], T, np.arange(2 * n + 3) % 8, 1, 8, 2 * n + 3)
    assert p.cursor.item() == 2 * n + 3
    assert t.tolist() == [[0, 1], [n % 8, 7], [(n + 1) % 8, (n + 2) % 8], [(2 * n + 1) % 8, (2 * n + 2) % 8]]
    want = np.full(2 * n + 3, -1)
    want[[0, 1, n, n + 1, n + 2, 2 * n + 1, 2 * n + 2]] = [0, 1, n % 8, (n + 1) % 8, (n + 2) % 8, (2 * n + 1) % 8, (2 * n + 2) % 8]
    assert np.array_equal(p.slots.cpu().numpy(), want)
    # as many as 31 bits hold end as an error, soon
    big = 2 ** 31 - 1
    p, t = plan_error(vv, vv.VV_ERR_CAPACITY, [0, 0, 2, 0], [big, 1, big - 2, 0], T, [1, 2, 3, 4], 1, 8, 4)
    assert t[0].tolist() == [1, 2] and p.slots.tolist() == [1, 2, -1, -1]


# ------------------------------------------------------------------------------ rope append
def pools(vv, pages, hkv, ps, dtype, seed, tokens_first=False):
    shape = (pages, ps, hkv, 128) if tokens_first else (pages, hkv, ps, 128)
    (k, kh), (v, vh) = values(shape, dtype, seed), values(shape, dtype, seed + 1)
    if tokens_first:
        k, v, kh, vh = k.transpose(1, 2), v.transpose(1, 2), kh.swapaxes(1, 2), vh.swapaxes(1, 2)
    return vv.PagedKV(k, v), kh, vh


def rope_bound(y, x, dtype):
    a = np.abs(x) + np.abs(np.roll(x, 64, axis=-1))
    return u_of(dtype) * np.abs(y) + 2.0 ** -19 * a + 2.0 ** -25  # last: subnormal fp16


ROPES = [(1, 4, 2, F16, False, 16, False, 100), (2, 7, 1, BF16, True, 16, False, 5),
         (7, 12, 2, F16, True, 32, True, 999000), (33, 28, 4, BF16, False, 64, True, 0),
         (130, 5, 5, F16, True, 48, False, -70), (16, 1, 1, BF16, True, 16, True, 2 ** 31 - 20),
         (700, 3, 1, F16, False, 16, True, 4000)]


@pytest.mark.parametrize("T,hq,hkv,dtype,gains,ps,tokens_first,first", ROPES)
def test_rope_append(vv, T, hq, hkv, dtype, gains, ps, tokens_first, first):
    fused, fh = values((T, hq + 2 * hkv, 128), dtype, T + hq)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    qh, kh, vh = fh[:, :hq], fh[:, hq:hq + hkv], fh[:, hq + hkv:]
    gq, gqh = values((128,), dtype, 1) if gains else (None, None)
    gk, gkh = values((128,), dtype, 2) if gains else (None, None)
    pages = -(-T // ps) + 2
    kv, kp, vp = pools(vv, pages, hkv, ps, dtype, 50, tokens_first)
    slots = synth.rng(T).permutation(pages * ps)[:T]
    if T > 5:
        slots[::5] = -1
    pos = first + np.arange(T)
    before = fused.clone()
    out = vv.vv_qk_rope_append(q, k, v, i32(pos), torch.tensor(slots).cuda(), kv, 1e6, q_gain=gq,
                               k_gain=gk, eps=1e-6)
    vv.vv_sync_status()
    assert torch.equal(fused, before)
    yq, yk, yv = obatch.qk_rope_append(qh, kh, vh, pos, slots, kp, vp, 1e6, gqh, gkh, 1e-6)
    nq = obatch.ops.rmsnorm(qh, gqh, 1e-6) if gains else qh
    assert np.all(np.abs(host(out) - yq) <= rope_bound(yq, nq, dtype))
    assert np.array_equal(host(kv.v), yv)
    x = np.array(kp)  # per cell: the unrotated values behind it
    nk = obatch.ops.rmsnorm(kh, gkh, 1e-6) if gains else kh
    for t in np.nonzero(slots >= 0)[0]:
        x[slots[t] // ps, :, slots[t] % ps] = nk[t]
    got = host(kv.k)
    untouched = np.ones((pages, ps), bool)
    untouched[slots[slots >= 0] // ps, slots[slots >= 0] % ps] = False
    assert np.array_equal(got.swapaxes(1, 2)[untouched], kp.swapaxes(1, 2)[untouched])
    assert np.all(np.abs(got - yk) <= rope_bound(yk, x, dtype))


def test_rope_append_one_gain_in_place_and_bad_slot(vv):
    T, hq, hkv = 5, 4, 2
    q, qh = values((T, hq, 128), F16, 1)
    k, kh = values((T, hkv, 128), F16, 2)
    g, gh = values((128,), F16, 3)
    kv, kp, vp = pools(vv, 2, hkv, 16, F16, 4)
    slots = torch.tensor([3, 32, 0, 2 ** 40, 31]).cuda()  # 32 slots in the pool
    pos = np.array([3, -4, 5, 6, 7])
    out = vv.vv_qk_rope_append(q, k, k, i32(pos), slots, kv, 1e4, q_gain=g, out=q)
    assert out.data_ptr() == q.data_ptr()
    with pytest.raises(vv.VVError) as e:
        vv.vv_sync_status()
    assert e.value.code == vv.VV_ERR_RANGE
    yq, yk, yv = obatch.qk_rope_append(qh, kh, kh, pos, [3, -1, 0, -1, 31], kp, vp, 1e4, q_gain=gh)
    assert np.all(np.abs(host(q) - yq) <= rope_bound(yq, obatch.ops.rmsnorm(qh, gh, 1e-6), F16))
    assert np.array_equal(host(kv.v), yv)
    assert np.max(np.abs(host(kv.k) - yk)) <= 2 ** -8


# ------------------------------------------------------------------------------- attention
def attn_case(vv, B, hq, hkv, P, lens, ps, dtype, seed=0, tokens_first=False, std=1.5, max_blocks=None):
    c = {}
    c["q"], c["qh"] = values((B, hq, 128), dtype, seed + 1, std)
    c["kpre"], c["kpreh"] = values((hkv, P, 128), dtype, seed + 2) if P else (None, None)
    c["vpre"], c["vpreh"] = values((hkv, P, 128), dtype, seed + 3) if P else (None, None)
    blocks = [-(-max(n, 0) // ps) for n in lens]
    pages = sum(blocks) + 2
    c["kv"], c["kph"], c["vph"] = pools(vv, pages, hkv, ps, dtype, seed + 4, tokens_first)
    order = synth.rng(seed).permutation(pages)
    c["tables"] = np.full((B, max_blocks or max(max(blocks), 1)), -1)
    at = 0
    for b in range(B):
        c["tables"][b, : blocks[b]] = order[at:at + blocks[b]]
        at += blocks[b]
    c["lens"], c["scale"] = list(lens), 1 / math.sqrt(128)
    return c


def attn_ws(vv, c, P=None):
    B, hq, _ = c["q"].shape
    n = vv.vv_gqa_prefix_attn_workspace_size(
        B, hq, c["kv"].heads, 128, (0 if c["kpre"] is None else c["kpre"].shape[1]) if P is None else P,
        c["tables"].shape[1] * c["kv"].page_size)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


def attn_run(vv, c, ws=None, **kw):
    B, hq, _ = c["q"].shape
    lse = torch.full((B, hq), 77.0, device="cuda")
    out = vv.vv_gqa_prefix_attn(c["q"], c["kpre"], c["vpre"], c["kv"], i32(c["tables"]),
                                i32(c["lens"]), c["scale"], attn_ws(vv, c) if ws is None else ws,
                                lse=lse, **kw)
    return out, lse


def attn_check(c, out, lse):
    dtype, P = out.dtype, 0 if c["kpre"] is None else c["kpre"].shape[1]
    y, ylse, mean, total = obatch.prefix_attention(
        c["qh"], c["kpreh"], c["vpreh"], c["kph"], c["vph"], c["tables"], c["lens"], c["scale"])
    u, n = u_of(dtype), P + max(c["lens"])
    bound = u * np.abs(y) + (u + 2.0 ** -13) * mean + 2.0 ** -24
    if dtype == F16:
        bound = bound + n * 2.0 ** -25 * 4 / total[..., None]
    got, glse = host(out), host(lse)
    for b, own in enumerate(c["lens"]):
        if own < 0:
            continue
        err = np.abs(got[b] - y[b])
        assert np.all(err <= bound[b]), (b, float(np.max(err / bound[b])))
        if P + own == 0:
            assert np.all(got[b] == 0) and np.all(np.isneginf(glse[b]))
        else:
            assert np.max(np.abs(glse[b] - ylse[b])) <= 1e-4
    return got


ATTNS = [  # B, Hq, Hkv, P, own lengths, page size, type
    (1, 4, 2, 0, [1], 16, F16), (1, 4, 2, 1, [0], 16, BF16), (2, 12, 2, 1024, [64, 3], 16, F16),
    (3, 4, 2, 0, [0, 17, 16], 16, F16), (5, 7, 1, 37, [0, 1, 15, 33, 100], 32, BF16),
    (2, 8, 8, 130, [129, 5], 16, F16), (3, 16, 1, 500, [700, 0, 41], 48, BF16),
    (4, 28, 4, 127, [200, 1, 0, 64], 64, F16), (23, 12, 2, 128, list(range(0, 46, 2)), 16, F16),
    (30, 28, 4, 300, [7 * i % 90 for i in range(30)], 128, BF16), (1, 7, 1, 0, [4785], 16, F16),
    (2, 4, 2, 4530, [300, 9], 16, BF16), (40, 6, 2, 900, [i % 5 for i in range(40)], 16, F16),
    (3, 4, 4, 15, [2100, 1500, 16], 16, F16), (150, 2, 2, 257, [i % 3 for i in range(150)], 16, BF16)]


@pytest.mark.parametrize("case", range(len(ATTNS)))
@pytest.mark.parametrize("tokens_first", [False, True])
def test_prefix_attn(vv, case, tokens_first):
    B, hq, hkv, P, lens, ps, dtype = ATTNS[case]
    c = attn_case(vv, B, hq, hkv, P, lens, ps, dtype, seed=100 * case, tokens_first=tokens_first)
    out, lse = attn_run(vv, c)
    vv.vv_sync_status()
    attn_check(c, out, lse)


def test_prefix_attn_extremes_of_scores(vv):
    """Scores of some hundreds (one key takes all), a maximum that keeps rising, equal keys."""
    for kind in ("sharp", "rising", "equal"):
        c = attn_case(vv, 3, 12, 2, 700, [300, 0, 40], 16, F16, seed=9)
        if kind == "sharp":
            c["scale"] = 4.0
        elif kind == "rising":
            ramp = torch.linspace(0.05, 3, 700, device="cuda")[None, :, None]
            base = c["q"][0, 0].float()[None, None, :]
            k = (ramp * base * 0.2).expand(2, 700, 128).to(F16).contiguous()
            c["kpre"], c["kpreh"] = k, host(k)
        else:
            c["kpre"] = c["kpre"][:, :1].expand(2, 700, 128).contiguous()
            c["kpreh"] = host(c["kpre"])
        out, lse = attn_run(vv, c)
        vv.vv_sync_status()
        y, ylse, mean, _ = obatch.prefix_attention(c["qh"], c["kpreh"], c["vpreh"], c["kph"], c["vph"],
                                                   c["tables"], c["lens"], c["scale"])
        # scores up to a few hundred: fp32 products and sums are off by some 2^-24 of them
        big = np.abs(ylse).max() + 20
        assert np.all(np.abs(host(out) - y) <= u_of(F16) * np.abs(y) + (u_of(F16) + big * 2.0 ** -19) * mean + 2.0 ** -14)
        assert np.max(np.abs(host(lse) - ylse)) <= big * 2.0 ** -19


def test_prefix_attn_ignores_what_lies_outside(vv):
    """NaN behind a sequence's last key, in foreign pages and past the prompt changes no bit, nor do
    table entries that no length reaches; a padding row is left alone."""
    for P in (0, 200, 1000):
        lens = [5, 0, 333, -1, 64, 18]
        c = attn_case(vv, 6, 12, 2, P, lens, 16, F16, seed=P, max_blocks=40)
        if P:  # the prompt is a slice of a longer cache
            big = [torch.zeros((2, P + 50, 128), dtype=F16, device="cuda") for _ in range(2)]
            for t, name in zip(big, ("kpre", "vpre")):
                t[:, :P] = c[name]
                c[name] = t[:, :P]
        out, lse = attn_run(vv, c)
        attn_check(c, out, lse)
        live = torch.zeros((c["kv"].pages, 16), dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            for t in range(max(n, 0)):
                live[int(c["tables"][b, t // 16]), t % 16] = True
        for pool in (c["kv"].k, c["kv"].v):
            pool.masked_fill_(~live[:, None, :, None], float("nan"))
        if P:
            for t in big:
                t[:, P:] = float("nan")
        for b, n in enumerate(lens):
            c["tables"][b, -(-max(n, 0) // 16):] = 2 ** 30
        c["q"][3] = float("nan")
        mark = torch.full_like(out, 3.0)
        out2, lse2 = attn_run(vv, c, out=mark)
        vv.vv_sync_status()
        keep = [0, 1, 2, 4, 5]
        assert torch.equal(out2[keep], out[keep]) and torch.equal(lse2[keep], lse[keep])
        assert torch.all(out2[3] == 3.0) and torch.all(lse2[3] == 77.0)


def test_prefix_attn_nan_and_inf_inside(vv):
    """A NaN among a row's own keys makes that sequence NaN and no other; a score of -inf is a
    masked key; only such scores give zeros."""
    for P in (0, 300):
        c = attn_case(vv, 3, 12, 2, P, [40, 30, 20], 16, F16, seed=3)
        page = int(c["tables"][1, 1])
        c["kv"].k[page, 0, 3] = float("nan")
        out, lse = attn_run(vv, c)
        assert torch.isnan(out[1, :6]).all() and torch.isnan(lse[1, :6]).all()
        assert torch.isfinite(out[[0, 2]]).all() and torch.isfinite(out[1, 6:]).all()
        c["q"].fill_(1.0)
        c["kv"].k[page, 0, 3] = 0.0
        c["kv"].k[page, 0, 3, 0] = -float("inf")
        a, _ = attn_run(vv, c)
        c["qh"], c["kph"] = host(c["q"]), host(c["kv"].k)
        y = obatch.prefix_attention(c["qh"], c["kpreh"], c["vpreh"], c["kph"], c["vph"],
                                    c["tables"], c["lens"], c["scale"])[0]
        assert np.max(np.abs(host(a) - y)) <= 2 ** -8
    c = attn_case(vv, 1, 4, 2, 0, [20], 16, F16)
    c["q"].fill_(1.0)
    c["kv"].k[..., 0] = -float("inf")
    out, lse = attn_run(vv, c)
    assert torch.all(out == 0) and torch.isneginf(lse).all()


def test_prefix_attn_bad_pages_and_long_lengths(vv):
    c = attn_case(vv, 2, 4, 2, 100, [40, 40], 16, F16, seed=8)
    good = c["tables"].copy()
    for bad in (-1, c["kv"].pages, 2 ** 31 - 1, -2 ** 31):
        c["tables"] = good.copy()
        c["tables"][0, 1] = bad
        out, lse = attn_run(vv, c)
        with pytest.raises(vv.VVError) as e:
            vv.vv_sync_status()
        assert e.value.code == vv.VV_ERR_RANGE
        # its 16 keys are left out: the same as the sequence without them
        d = dict(c, lens=[24, 40], tables=good.copy())
        d["tables"][0] = [good[0, 0], good[0, 2], -1]
        attn_check(d, out, lse)
    c["tables"] = good
    out, _ = attn_run(vv, dict(c, lens=[48, 40]))
    vv.vv_sync_status()
    out2, _ = attn_run(vv, dict(c, lens=[2 ** 31 - 1, 40]))
    with pytest.raises(vv.VVError) as e:
        vv.vv_sync_status()
    assert e.value.code == vv.VV_ERR_CAPACITY
    assert torch.equal(out, out2)


def test_prefix_attn_strided_rows_and_prefix(vv):
    """q inside a fused projection, out inside a wider buffer, the prompt as [P, Hkv, D]."""
    B, hq, hkv, P = 9, 28, 4, 333
    c = attn_case(vv, B, hq, hkv, P, [11 * i for i in range(B)], 16, BF16, seed=5)
    want, lse0 = attn_run(vv, c)
    fused = torch.full((B, hq + 2 * hkv, 128), float("nan"), dtype=BF16, device="cuda")
    fused[:, :hq] = c["q"]
    wide = torch.full((B, hq + 3, 128), 5.0, dtype=BF16, device="cuda")
    c["q"] = fused[:, :hq]
    c["kpre"] = c["kpre"].transpose(0, 1).contiguous().transpose(0, 1)
    c["vpre"] = c["vpre"].transpose(0, 1).contiguous().transpose(0, 1)
    out, lse = attn_run(vv, c, out=wide[:, :hq])
    vv.vv_sync_status()
    assert torch.equal(out, want) and torch.equal(lse, lse0) and torch.all(wide[:, hq:] == 5.0)


def test_prefix_attn_workspace_is_left_ready_and_results_repeat(vv):
    c = attn_case(vv, 3, 12, 2, 2000, [900, 10, 500], 16, F16, seed=2)
    d = attn_case(vv, 3, 12, 2, 70, [1, 0, 600], 16, F16, seed=4, max_blocks=57)
    ws = torch.zeros(max(attn_ws(vv, c).numel(), attn_ws(vv, d).numel()), dtype=torch.uint8, device="cuda")
    a, la = attn_run(vv, c, ws)
    b, lb = attn_run(vv, d, ws)
    for _ in range(3):
        a2, la2 = attn_run(vv, c, ws)
        b2, lb2 = attn_run(vv, d, ws)
        assert torch.equal(a, a2) and torch.equal(b, b2) and torch.equal(la, la2) and torch.equal(lb, lb2)
    attn_check(c, a, la)
    attn_check(d, b, lb)


@pytest.mark.parametrize("hq,hkv,P", [(9, 1, 20), (22, 2, 300), (16, 1, 128), (13, 1, 127)])
def test_prefix_attn_wide_groups_and_any_workspace(vv, hq, hkv, P):
    """9 to 16 query heads per key-value head, on a workspace of NaN; the result may take q's place."""
    c = attn_case(vv, 4, hq, hkv, P, [70, 0, -1, 17], 16, F16, seed=hq)
    ws = torch.full((attn_ws(vv, c).numel(),), 0xff, dtype=torch.uint8, device="cuda")
    out, lse = attn_run(vv, c, ws)
    vv.vv_sync_status()
    attn_check(c, out, lse)
    q = c["q"]
    c["q"] = q.clone()
    attn_run(vv, c, ws, out=c["q"])
    live = [0, 1, 3]
    assert torch.equal(c["q"][live], out[live]) and torch.equal(c["q"][2], q[2])


def test_prefix_attn_two_streams_and_two_threads(vv):
    """Calls on workspaces of their own may run at once, from two host threads too."""
    from threading import Thread

    cs = [attn_case(vv, 12, 12, 2, 1500, [40 * i for i in range(12)], 16, F16, seed=1),
          attn_case(vv, 3, 28, 4, 60, [700, 2, 90], 32, BF16, seed=2)]
    wss, want = [attn_ws(vv, c) for c in cs], [attn_run(vv, c) for c in cs]
    tabs = [(i32(c["tables"]), i32(c["lens"])) for c in cs]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        c, s = cs[i], torch.cuda.Stream()
        for _ in range(20):
            got[i].append(vv.vv_gqa_prefix_attn(c["q"], c["kpre"], c["vpre"], c["kv"], *tabs[i], c["scale"], wss[i], stream=s))
        s.synchronize()

    threads = [Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    vv.vv_sync_status()
    for i in range(2):
        assert len(got[i]) == 20 and all(torch.equal(o, want[i][0]) for o in got[i])


# ---------------------------------------------------------------------------------- logits
def logits_case(B, V, W, dtype, seed, bias=0, mask=False, penalties=True, prompt=None):
    r = synth.rng(seed)
    c = {}
    c["x"], c["xh"] = values((B, V), dtype, seed, 3.0)
    if W:
        c["tok"] = r.integers(0, max(1, V // 3), (B, W))
        c["tok"][:, ::7] = r.integers(-3, V + 3, (B, len(range(0, W, 7))))  # some outside [0, V)
        if W > 40:
            c["tok"][:, 10:35] = V - 1
        c["n"] = r.integers(0, W + 1, B)
        c["n"][0] = W
        c["p"] = np.minimum(r.integers(0, W + 1, B), c["n"]) if prompt is None else np.full(B, prompt)
    if W and penalties:
        c["rep"] = (1 + r.random(B)).astype(np.float32)
        c["freq"], c["pres"] = (r.standard_normal(B).astype(np.float32) for _ in range(2))
    if bias:
        c["off"] = np.concatenate([[0], np.cumsum(r.integers(0, bias + 1, B))])
        n = int(c["off"][-1])
        c["ids"] = r.integers(-2, V + 2, n)  # repeats, and some outside
        c["vals"] = r.standard_normal(n).astype(np.float32) * 3
    if mask:
        c["ok"] = r.random((B, V)) < r.random((B, 1))
        if B > 2:
            c["ok"][1] = False
    return c


def words_of(ok):
    B, V = ok.shape
    full = np.ones((B, -(-V // 32) * 32), bool)  # bits past V are set: they must not matter
    full[:, :V] = ok
    return torch.from_numpy(np.packbits(full, axis=1, bitorder="little").view(np.int32).copy()).cuda()


def logits_run(vv, c, **kw):
    f = lambda k: torch.tensor(c[k], device="cuda") if k in c else None  # noqa: E731
    n = lambda k: i32(c[k]) if k in c else None  # noqa: E731
    ws = torch.zeros(vv.vv_logits_process_workspace_size(c["x"].shape[0]), dtype=torch.uint8, device="cuda")
    r = vv.vv_logits_process(
        c["x"], ws, tokens=n("tok"), token_lens=n("n"), prompt_lens=n("p"), repetition=f("rep"),
        frequency=f("freq"), presence=f("pres"), bias_ids=n("ids"), bias_vals=f("vals"),
        bias_offsets=n("off"), mask=words_of(c["ok"]) if "ok" in c else None, **kw)
    vv.vv_sync_status()
    assert not ws.any()
    return r


def logits_check(c, out, idx):
    B = c["x"].shape[0]
    bias = None
    if "ids" in c:
        bias = [{int(c["ids"][i]): c["vals"][i] for i in range(c["off"][b], c["off"][b + 1])} for b in range(B)]
    y, want = obatch.logits_process(c["xh"], c.get("tok"), c.get("n"), c.get("p"), c.get("rep"),
                                    c.get("freq"), c.get("pres"), bias, c.get("ok"))
    dtype, got = out.dtype, host(out)
    big = np.abs(c["xh"]).max() * 2 + 3 * (c["tok"].shape[1] if "tok" in c else 0) + 30
    fp32 = 6 * 2.0 ** -24 * big
    inf = np.isneginf(y)
    assert np.array_equal(np.isneginf(got), inf)
    fin = ~inf
    u = 0.0 if dtype == F32 else u_of(dtype)
    got, y_fin = got[fin], y[fin]
    assert np.all(np.abs(got - y_fin) <= u * np.abs(y_fin) + (1 + u) * fp32)
    sure = np.sort(np.where(np.isnan(y), -np.inf, y), axis=1)[:, ::-1]
    for b in range(B):
        i = int(idx[b])
        if want[b] < 0 or (y.shape[1] > 1 and sure[b, 0] - sure[b, 1] > 2 * fp32):
            assert i == want[b]
        else:
            assert y[b, i] >= sure[b, 0] - 2 * fp32


LOGITS = [(1, 1, 0, F32, 0, False), (1, 1000, 5, F32, 0, False), (2, 1001, 100, F32, 9, True),
          (3, 8192, 64, BF16, 0, True), (5, 8193, 700, F16, 30, True), (2, 151936, 300, F32, 40, False),
          (7, 33001, 0, F32, 12, True), (65, 2049, 33, BF16, 3, False), (4, 20000, 3000, F32, 500, True),
          (2, 9001, 70000, F32, 2000, True), (2, 300, 6000, F16, 70000, False)]


@pytest.mark.parametrize("B,V,W,dtype,bias,mask", LOGITS)
def test_logits_process(vv, B, V, W, dtype, bias, mask):
    c = logits_case(B, V, W, dtype, V + W, bias, mask)
    out, idx = logits_run(vv, c)
    logits_check(c, out, idx)
    x = c["x"].clone()
    c["x"] = x
    same, idx2 = logits_run(vv, c, out=x)  # in place
    assert same.data_ptr() == x.data_ptr() and torch.equal(same, out) and torch.equal(idx, idx2)


# rows enough for the larger slices
MANY = [(40, 28672, 50, F16, 3, True), (150, 8193, 100, F16, 9, True), (60, 16384, 3000, F32, 200, True), (112, 8192, 64, BF16, 0, True),
        (45, 20481, 70000, F32, 30, False), (90, 10000, 6000, BF16, 800, True), (230, 2049, 0, F32, 4, False)]


@pytest.mark.parametrize("B,V,W,dtype,bias,mask", MANY)
def test_logits_process_many_rows(vv, B, V, W, dtype, bias, mask):
    c = logits_case(B, V, W, dtype, V + W, bias, mask)
    out, idx = logits_run(vv, c)
    logits_check(c, out, idx)
    x = c["x"].clone()
    same, idx2 = logits_run(vv, dict(c, x=x), out=x)  # in place
    assert torch.equal(same, out) and torch.equal(idx, idx2)


def test_logits_process_edges(vv):
    V = 20000
    # nothing but a copy and the greedy token; lowest of a tie, across slices and at -0 / +0
    x = torch.zeros((3, V), device="cuda")
    x[0, [9000, 19999, 400]] = 2.0
    x[1] = -0.0
    x[1, 12000] = 0.0
    x[2] = -float("inf")
    out, idx = logits_run(vv, {"x": x})
    assert torch.equal(out, x) and idx.tolist() == [400, 0, -1]
    # NaN is copied and never chosen; +inf is
    x = torch.full((2, V), float("nan"), device="cuda")
    x[0, 15000] = -3.0
    x[1, 17000] = float("inf")
    out, idx = logits_run(vv, {"x": x})
    assert idx.tolist() == [15000, 17000] and torch.equal(out.isnan(), x.isnan())
    # masked NaN and inf become -inf; the type's lowest value is an ordinary logit
    x = torch.full((1, V), torch.finfo(F32).min, device="cuda")
    x[0, 5], x[0, 6] = float("nan"), float("inf")
    ok = np.ones((1, V), bool)
    ok[0, [0, 5, 6]] = False
    out, idx = logits_run(vv, {"x": x, "ok": ok})
    assert idx.item() == 1 and torch.isneginf(out[0, [0, 5, 6]]).all() and out[0, 7] == torch.finfo(F32).min
    # a history of one id throughout: prompt ids count once, generated ones each time
    for plen, n in ((4530, 0), (0, 4530), (4000, 530)):
        c = {"x": torch.ones((1, V), device="cuda"), "tok": np.full((1, 4530), 16000), "n": np.array([4530]),
             "p": np.array([plen]), "rep": np.array([2.0], np.float32), "freq": np.array([0.5], np.float32),
             "pres": np.array([3.0], np.float32)}
        out, _ = logits_run(vv, c)
        assert out[0, 16000].item() == 0.5 - (0.5 * n + 3.0 if n else 0.0)
        assert torch.count_nonzero(out != 1).item() == 1


def test_logits_process_strides_and_lengths_out_of_range(vv):
    B, V = 4, 5003
    c = logits_case(B, V, 50, F32, 3, bias=20, mask=True)
    want, idx = logits_run(vv, c)
    wide = torch.full((B, V + 5), 9.0, device="cuda")
    wide[:, 1:V + 1] = c["x"]
    dst = torch.full((B, V + 2), 4.0, device="cuda")
    d = dict(c, x=wide[:, 1:V + 1])
    out, idx2 = logits_run(vv, d, out=dst[:, 1:V + 1])
    assert torch.equal(out, want) and torch.equal(idx, idx2)
    assert torch.all(dst[:, 0] == 4) and torch.all(dst[:, -1] == 4) and torch.all(wide[:, -1] == 9)
    for key, at, bad in (("n", 1, 51), ("n", 2, -1), ("p", 1, -1), ("p", 2, 99), ("off", 0, -1),
                         ("off", 4, 10 ** 6), ("off", 1, 2 ** 31 - 1)):
        e = dict(c)
        e[key] = c[key].copy()
        e[key][at] = bad
        with pytest.raises(vv.VVError) as err:
            logits_run(vv, e)
        assert err.value.code == vv.VV_ERR_RANGE, (key, at, bad)
    again, _ = logits_run(vv, c)
    assert torch.equal(again, want)
    out, none = vv.vv_logits_process(c["x"], argmax=False)
    assert none is None and torch.equal(out, c["x"])


# ------------------------------------------------------------------- streams, graphs, refusals
def test_other_streams_and_replayed_graphs(vv):
    """All four on a side stream, then captured: a replay reads the lengths of the moment."""
    B, hq, hkv, P, ps, W = 6, 12, 2, 500, 16, 64
    lens = i32([0, 15, 31, 5, 16, 40])
    c = attn_case(vv, B, hq, hkv, P, [60] * B, ps, F16, seed=21)
    kv, tables = c["kv"], torch.full((B, 5), -1, dtype=torch.int32, device="cuda")
    start = np.full((B, 5), -1)
    free = np.arange(kv.pages)
    at = 0
    for b, n in enumerate(lens.tolist()):
        k = -(-n // ps)
        start[b, :k] = free[at:at + k]
        at += k
    free_t, ones = i32(free[at:]), i32([1] * B)
    qkv, _ = values((B, hq + 2 * hkv, 128), F16, 33)
    lg = logits_case(B, 9000, W, F32, 1, mask=True)
    tok, n, p, bits = i32(lg["tok"]), i32(lg["n"]), i32(lg["p"]), words_of(lg["ok"])
    rep = torch.tensor(lg["rep"], device="cuda")
    aws = torch.zeros(vv.vv_gqa_prefix_attn_workspace_size(B, hq, hkv, 128, P, 80), dtype=torch.uint8, device="cuda")
    lws = torch.zeros(vv.vv_logits_process_workspace_size(B), dtype=torch.uint8, device="cuda")
    kv0 = kv.k.clone(), kv.v.clone()

    def step(stream=None):
        plan = vv.vv_paged_plan(lens, ones, tables, free_t, ps, kv.pages, B + 2, prefix_len=P, stream=stream)
        q = vv.vv_qk_rope_append(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], plan.positions[:B],
                                 plan.slots[:B], kv, 1e6, stream=stream)
        o = vv.vv_gqa_prefix_attn(q, c["kpre"], c["vpre"], kv, tables, plan.lens, c["scale"], aws, stream=stream)
        x, i = vv.vv_logits_process(lg["x"], lws, tokens=tok, token_lens=n, prompt_lens=p, repetition=rep,
                                    mask=bits, stream=stream)
        return plan, q, o, x, i

    def reset(ls):
        lens.copy_(i32(ls))
        tables.copy_(i32(start))
        kv.k.copy_(kv0[0])
        kv.v.copy_(kv0[1])
        torch.cuda.synchronize()

    first = lens.tolist()
    reset(first)
    eager = [t.clone() for t in (lambda r: [*r[0], *r[1:]])(step())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    reset(first)
    got = step(side)
    side.synchronize()
    for a, b in zip(eager, [*got[0], *got[1:]]):
        assert torch.equal(a, b)
    reset(first)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = step()
        captured = [*r[0], *r[1:]]
    for ls in (first, [0, 14, 30, 5, 15, 33], first):
        reset(ls)
        want = [t.clone() for t in (lambda r: [*r[0], *r[1:]])(step())]
        reset(ls)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, captured):
            assert torch.equal(a, b)
    vv.vv_sync_status()


def test_binding_refuses(vv):
    c = attn_case(vv, 3, 4, 2, 40, [5, 6, 7], 16, F16)
    ws, t, n = attn_ws(vv, c), i32(c["tables"]), i32(c["lens"])
    run = lambda **k: vv.vv_gqa_prefix_attn(**dict(dict(  # noqa: E731
        q=c["q"], k_prefix=c["kpre"], v_prefix=c["vpre"], kv=c["kv"], block_tables=t, lens=n, scale=0.1, ws=ws), **k))
    run()
    for bad in (dict(q=c["q"].bfloat16()), dict(q=c["q"][:, :, :64]), dict(q=c["q"].cpu()), dict(q=c["q"][0]),
                dict(k_prefix=None), dict(k_prefix=c["kpre"][:, :39]), dict(k_prefix=c["kpre"].float()),
                dict(v_prefix=c["vpre"].transpose(0, 1).contiguous().transpose(0, 1)),
                dict(block_tables=t.long()), dict(block_tables=t[:2]), dict(lens=n[:2]), dict(lens=n.cpu()),
                dict(ws=ws[:8]), dict(out=torch.empty(2, 4, 128, dtype=F16, device="cuda")),
                dict(lse=torch.empty(3, 4, dtype=F16, device="cuda")), dict(scale=0.0)):
        with pytest.raises(vv.VVError):
            run(**bad)
    q, k = c["q"], c["q"][:, :2]
    pos, slots = i32([0, 1, 2]), torch.arange(3, device="cuda")
    for bad in (dict(q=q[:, :, ::2]), dict(k=c["q"]), dict(v=k[:2]), dict(positions=slots), dict(slots=pos),
                dict(q_gain=torch.ones(64, dtype=F16, device="cuda")), dict(q_gain=torch.ones(128, device="cuda")),
                dict(out=q[:2]), dict(theta=-1.0)):
        with pytest.raises(vv.VVError):
            vv.vv_qk_rope_append(**dict(dict(q=q, k=k, v=k, positions=pos, slots=slots, kv=c["kv"], theta=1e4), **bad))
    x = torch.zeros((2, 100), device="cuda")
    lws = torch.zeros(vv.vv_logits_process_workspace_size(2), dtype=torch.uint8, device="cuda")
    for bad in (dict(ws=None), dict(ws=lws[:16]), dict(logits=x.double()), dict(logits=x[0]), dict(repetition=x[0, :2]),
                dict(tokens=i32([[1], [2]])), dict(mask=i32([[1], [2]])), dict(bias_ids=i32([1])),
                dict(out=torch.zeros((2, 99), device="cuda")), dict(out=torch.zeros((2, 100), dtype=F16, device="cuda"))):
        with pytest.raises(vv.VVError):
            vv.vv_logits_process(**dict(dict(logits=x, ws=lws), **bad))
    torch.cuda.synchronize()


# ------------------------------------------------------------------------- all of them together
def test_forked_transcripts_match_the_decoder(vv):
    """Three sequences fork from one prompt that a decoder prefilled; each step runs plan, append,
    attention and logits around the packed projections.  Every step's logits against the oracle's
    decoder_step of each sequence on its own (the decoder's contract tolerance)."""
    from helpers import gpu_model, ocfg, oracle_model
    from int4_blockwise_quantised_b200.model import Decoder
    from oracle import decoder as odec

    shape = synth.SHAPE_TINY
    L, hq, hkv, S, B, steps, ps = shape.layers, shape.n_q, shape.n_kv, 37, 3, 20, 16
    cfg, W, model = ocfg(shape), oracle_model(shape, "sym"), gpu_model(shape, "sym")
    ids = synth.rng(5).integers(0, shape.vocab, S).astype(np.int32)
    dec = Decoder(model, 64, max_prefill=64)
    dec.init(i32(ids), i32(np.arange(S)))
    dec.sync_status()
    caches = [([dec.k_cache[l, 0, :, :S].cpu().numpy() for l in range(L)],
               [dec.v_cache[l, 0, :, :S].cpu().numpy() for l in range(L)]) for _ in range(B)]

    kvs = [vv.PagedKV(*(torch.full((9, hkv, ps, 128), float("nan"), dtype=F16, device="cuda") for _ in range(2)))
           for _ in range(L)]
    tables = torch.full((B, 3), -1, dtype=torch.int32, device="cuda")
    free = i32(synth.rng(6).permutation(9))
    lens, cursor, ones = i32([0] * B), i32([0]), i32([1] * B)
    aws = torch.zeros(vv.vv_gqa_prefix_attn_workspace_size(B, hq, hkv, 128, S, 3 * ps), dtype=torch.uint8, device="cuda")
    lws = torch.zeros(vv.vv_logits_process_workspace_size(B), dtype=torch.uint8, device="cuda")
    said = torch.zeros((B, S + steps + 1), dtype=torch.int32, device="cuda")
    said[:, :S] = i32(ids)
    said[:, S] = i32([3, 500, 999])
    rep = torch.full((B,), 1.3, device="cuda")

    def norm(x, g):
        return (x / torch.sqrt((x * x).mean(-1, keepdim=True) + shape.eps) * g.float()).to(F16)

    for s in range(steps):
        token = said[:, S + s]
        plan = vv.vv_paged_plan(lens, ones, tables, free, ps, 9, B, prefix_len=S, cursor=cursor)
        lens, cursor = plan.lens, plan.cursor
        x = model.embed[token.long()].float()
        for l, lw in enumerate(model.layers):
            h = norm(x, lw["input_norm"])
            q, k, v = (vv.vv_matmul_nbits(h, *lw[m], lw[bias]).view(B, -1, 128)
                       for m, bias in (("wq", "bq"), ("wk", "bk"), ("wv", "bv")))
            q = vv.vv_qk_rope_append(q, k, v, plan.positions, plan.slots, kvs[l], shape.theta, out=q)
            o = vv.vv_gqa_prefix_attn(q, dec.k_cache[l, 0, :, :S], dec.v_cache[l, 0, :, :S], kvs[l], tables,
                                      lens, 1 / math.sqrt(128), aws)
            x = x + vv.vv_matmul_nbits(o.view(B, -1), *lw["wo"]).float()
            h = norm(x, lw["post_norm"])
            gate, up = (vv.vv_matmul_nbits(h, *lw[m]).float() for m in ("wgate", "wup"))
            x = x + vv.vv_matmul_nbits((torch.nn.functional.silu(gate) * up).to(F16), *lw["wdown"]).float()
        logits = norm(x, model.final_norm).float() @ model.lm_head.float().T
        out, idx = vv.vv_logits_process(logits, lws, tokens=said, token_lens=i32([S + s + 1] * B),
                                        prompt_lens=i32([S] * B), repetition=rep)
        vv.vv_sync_status()
        for b in range(B):
            kc, vc = caches[b]
            ora = odec.decoder_step(cfg, W, model.embed[int(token[b])].cpu().numpy(), S + s, kc, vc)
            assert normwise(host(logits[b]), ora["logits"]) <= TOL
            for l in range(L):
                kc[l] = np.concatenate([kc[l], ora["k_new"][l][:, None, :]], axis=1)
                vc[l] = np.concatenate([vc[l], ora["v_new"][l][:, None, :]], axis=1)
        y, want = obatch.logits_process(host(logits), said.cpu().numpy(), [S + s + 1] * B, [S] * B, [rep[0].item()] * B)
        assert idx.tolist() == want.tolist()
        said[:, S + s + 1] = idx
    assert cursor.item() == B * 2 and lens.tolist() == [steps] * B
