"""The batch operators past the first pass of their pipelined loops: rings filled again, buffers used
again, maxima that move, warps with several units.  Each case states what it reaches, computed from
the launch rules and the SM count, and checks it; tolerances as derived in test_gpu_paged_batch.
"""

import math

import numpy as np
import pytest
import torch

import synth
from oracle import batch as obatch
from test_gpu_paged_batch import BF16, F16, host, i32, plan_case, rope_bound, u_of, values, vv  # noqa: F401

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------------------- attention
CHUNK, END = 16, 10  # keys of an own chunk; what a head counts beside its chunks
STAGES, BLOCK = 21, 128  # of the own pages' ring; keys of a block of the prompt


def prompt_split(rows, hkv, P):
    """(parts, blocks per part) of a shared prompt, the launch rule of the prompt's kernel."""
    tiles, blocks = -(-rows // BLOCK) * hkv, -(-P // BLOCK)
    best = None
    for s in range(1, min(blocks, max(8, sms() // tiles)) + 1):
        per = -(-blocks // s)
        used = -(-blocks // per)
        cost = -(-tiles * used // sms()) * (per + 4) + used // 32
        if best is None or cost < best[0]:
            best = (cost, used, per)
    return best[1:]


def own_run(B, hkv, P, lens):
    """Places (chunks, and END a head) of a CTA's run of own chunks."""
    npre = 0 if B > 1 and P >= BLOCK else -(-P // CHUNK)
    places = hkv * sum(max(npre + -(-n // CHUNK), 1) + END for n in lens if n >= 0)
    return places // min(sms(), max(1, places // (4 + END)))


def case(vv, B, hq, hkv, P, lens, ps, dtype, seed, pages=60):  # noqa: F811
    """Long lengths over a small pool (a page may stand in a table many times) and a prompt tiled from
    some thousand positions: little data, many keys."""
    c = {"lens": list(lens), "scale": 1 / math.sqrt(128), "P": P}
    c["q"], c["qh"] = values((B, hq, 128), dtype, seed, 1.5)
    n = min(P, 1500)
    for i, name in enumerate(("kpre", "vpre")):
        c[name] = c[name + "h"] = None
        if P:
            base, _ = values((hkv, n, 128), dtype, seed + 1 + i)
            c[name] = base.repeat(1, -(-P // n), 1)[:, :P].contiguous()
            c[name + "h"] = host(c[name])
    (k, c["kph"]), (v, c["vph"]) = (values((pages, hkv, ps, 128), dtype, seed + 3 + i) for i in range(2))
    c["kv"] = vv.PagedKV(k, v)
    width = max(1, max(-(-max(x, 0) // ps) for x in lens))
    c["tables"] = synth.rng(seed).integers(0, pages, (B, width))
    return c


def run(vv, c, **kw):  # noqa: F811
    B, hq, _ = c["q"].shape
    n = vv.vv_gqa_prefix_attn_workspace_size(B, hq, c["kv"].heads, 128, c["P"], c["tables"].shape[1] * c["kv"].page_size)
    lse = torch.full((B, hq), 77.0, device="cuda")
    out = vv.vv_gqa_prefix_attn(c["q"], c["kpre"], c["vpre"], c["kv"], i32(c["tables"]), i32(c["lens"]), c["scale"],
                                torch.full((n,), 255, dtype=torch.uint8, device="cuda"), lse=lse, **kw)
    vv.vv_sync_status()
    return out, lse


def check(c, out, lse, rows=None):
    """The sequences `rows` (all) against the definition in 64 bits.  A weight is off by its rounding u,
    by the score's error (128 products in fp32, 2^-20 of the sum of their magnitudes with room for the
    tensor core's alignment) and, in fp16, by 2^-25 of the largest weight at most, n times."""
    rows = list(range(len(c["lens"]))) if rows is None else rows
    y, ylse, mean, total = obatch.prefix_attention(
        c["qh"][rows], c["kpreh"], c["vpreh"], c["kph"], c["vph"], c["tables"][rows], [c["lens"][b] for b in rows], c["scale"])
    big = 0.0
    for k in (c["kpreh"], c["kph"]):
        if k is not None:
            big = max(big, np.abs(c["qh"]).sum(-1).max() * np.abs(k).max() * c["scale"])
    u, n = u_of(out.dtype), c["P"] + max(c["lens"])
    score = big * 2.0 ** -20
    bound = u * np.abs(y) + (u + score) * mean + 2.0 ** -24
    if out.dtype == F16:
        bound = bound + n * 2.0 ** -25 * np.abs(c["vph"]).max() / total[..., None]
    got, glse = host(out)[rows], host(lse)[rows]
    for i, b in enumerate(rows):
        if c["lens"][b] < 0:
            continue
        err = np.abs(got[i] - y[i])
        assert np.all(err <= bound[i]), (b, float(np.max(err / bound[i])))
        if c["P"] + c["lens"][b] == 0:
            assert np.all(np.isneginf(glse[i]))
        else:
            assert np.max(np.abs(glse[i] - ylse[i])) <= 1e-4 + score


OWN = [  # B, Hq, Hkv, P, own lengths, page size, type
    (8, 4, 2, 0, [20000, 0, 13001, 17, 17345, 11000, 19999, 6], 16, F16),
    (5, 16, 1, 100, [60000, 31, 39997, 0, 55000], 64, BF16),
    (1, 7, 1, 120001, [30011], 32, F16),
    (9, 28, 4, 400, [6000, 9001, 128, -1, 8000, 9, 9400, 6333, 2], 16, BF16)]


@pytest.mark.parametrize("i", range(len(OWN)))
def test_own_pages_ring_is_filled_again(vv, i):  # noqa: F811
    B, hq, hkv, P, lens, ps, dtype = OWN[i]
    assert own_run(B, hkv, P, lens) > 2 * STAGES + 2 * END  # every stage twice, some three times
    c = case(vv, B, hq, hkv, P, lens, ps, dtype, 300 + 10 * i)
    out, lse = run(vv, c)
    check(c, out, lse)


PROMPTS = [  # B, Hq, Hkv, P, own lengths, type, sequences that are compared, blocks a part at least
    (3, 8, 8, 90 * 128, [5, 0, 40], F16, None, 5),
    (20, 28, 4, 90 * 128 + 77, [7 * i for i in range(20)], BF16, [0, 3, 11, 19], 6),
    (150, 8, 8, 60 * 128 - 1, [i % 3 for i in range(150)], F16, [0, 64, 127, 128, 149], 7),
    (48, 28, 4, 32768, [i for i in range(48)], BF16, [0, 47], 22)]


@pytest.mark.parametrize("i", range(len(PROMPTS)))
def test_prompt_of_many_blocks(vv, i):  # noqa: F811
    B, hq, hkv, P, lens, dtype, rows, blocks = PROMPTS[i]
    assert prompt_split(B * hq // hkv, hkv, P)[1] >= blocks
    c = case(vv, B, hq, hkv, P, lens, 16, dtype, 400 + 10 * i)
    out, lse = run(vv, c)
    check(c, out, lse, rows)
    for _ in range(3):  # the same bits whatever the order in which parts end
        again = run(vv, c)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


# The score of a block's best key, in nats, block by block within a part of six: a step of more than
# 8 ln 2 = 5.5 moves the running maximum of every row that it holds for.
LEVELS = {"every block": [0, 7, 14, 21, 28, 35], "odd blocks": [0, 7, 0, 14, 0, 21], "even blocks": [0, -9, 7, 0, 14, 2],
          "two in a row": [0, 0, 8, 16, 16, 5], "below the step": [0, 5, 5.5, 9, 11, 16], "the last": [0, 0, 0, 0, 0, 9],
          "falling": [35, 28, 21, 14, 7, 0]}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", LEVELS)
def test_prompt_whose_maximum_moves_between_blocks(vv, kind, dtype):  # noqa: F811
    """Half of the rows see the levels as written, the others a fraction or the opposite of them."""
    B, hq, hkv, per = 33, 28, 4, 6
    P = 18 * per * BLOCK - 50
    assert prompt_split(B * hq // hkv, hkv, P) == (18, per)
    c = case(vv, B, hq, hkv, P, [3 * i for i in range(B)], 16, dtype, 500 + len(kind))
    along = torch.zeros(128, device="cuda")
    along[::2] = 1.0
    level = torch.tensor(LEVELS[kind], device="cuda")[torch.arange(P, device="cuda") // BLOCK % per]
    # the keys' part along the direction gives the level; their other half stays random
    c["kpre"] = (c["kpre"].float() * (1 - along) * 0.5 + level[None, :, None] * along / 64 * math.sqrt(128)).to(dtype)
    share = torch.tensor([1.0, 1.0, 0.3, -1.0], device="cuda")[torch.arange(B * hq, device="cuda") % 4].view(B, hq, 1)
    c["q"] = (c["q"].float() * (1 - along) * 0.5 + share * along).to(dtype)
    c["kpreh"], c["qh"] = host(c["kpre"]), host(c["q"])
    out, lse = run(vv, c)
    check(c, out, lse, [0, 9, 18, 32])
    again = run(vv, c)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


# ------------------------------------------------------------------------------ rope append
# T, Hq, Hkv, gains: CTAs of 5 warps and rings of 3 units without norms, 8 and 2 with them
UNITS = [(12001, 1, 1, False), (12001, 1, 1, True), (6007, 17, 1, False), (6007, 17, 1, True), (40001, 1, 1, False)]


@pytest.mark.parametrize("T,hq,hkv,gains", UNITS)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_rope_append_with_several_units_a_warp(vv, T, hq, hkv, gains, dtype):  # noqa: F811
    warps, stages = (8, 2) if gains else (5, 3)
    parts = -(-(hq + 2 * hkv) // 18)
    assert T > 2 * sms() * warps  # tokens are not cut further
    assert T * parts // (2 * sms() * warps) >= 2 * stages + 1
    fused, fh = values((T, hq + 2 * hkv, 128), dtype, T + hq)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    qh, kh, vh = fh[:, :hq], fh[:, hq:hq + hkv], fh[:, hq + hkv:]
    (gq, gqh), (gk, gkh) = (values((128,), dtype, 1), values((128,), dtype, 2)) if gains else ((None, None),) * 2
    pages = -(-T // 32) + 1
    pool = [torch.full((pages, hkv, 32, 128), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    slots = synth.rng(T).permutation(pages * 32)[:T]
    slots[::11] = -1
    pos = synth.rng(T + 1).integers(-10 ** 6, 10 ** 6, T)
    out = vv.vv_qk_rope_append(q, k, v, i32(pos), torch.tensor(slots).cuda(), vv.PagedKV(*pool), 1e6, q_gain=gq, k_gain=gk)
    vv.vv_sync_status()
    seven = np.full((pages, hkv, 32, 128), 7.0)
    yq, yk, yv = obatch.qk_rope_append(qh, kh, vh, pos, slots, seven, seven, 1e6, gqh, gkh)
    nq, nk = (obatch.ops.rmsnorm(qh, gqh, 1e-6), obatch.ops.rmsnorm(kh, gkh, 1e-6)) if gains else (qh, kh)
    assert np.all(np.abs(host(out) - yq) <= rope_bound(yq, nq, dtype))
    assert np.array_equal(host(pool[1]), yv)
    at = slots >= 0
    cell = slots[at] // 32, slots[at] % 32
    got = host(pool[0]).swapaxes(1, 2)
    want = yk.swapaxes(1, 2)
    assert np.all(np.abs(got[cell] - want[cell]) <= rope_bound(want[cell], nk[at], dtype))
    rest = np.ones((pages, 32), bool)
    rest[cell] = False
    assert np.all(got[rest] == 7.0)


# ------------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("B,max_len,max_new,ps,prefix", [(4096, 129, 380, 32, 1024), (60, 3000, 20000, 1, 0)])
def test_plan_of_more_tokens_than_one_pass(vv, B, max_len, max_new, ps, prefix):  # noqa: F811
    lens, new, tables, free, pages, total = plan_case(B, max_len, max_new, ps, B)
    assert total > sms() * 512 * 4 + 2048
    t = i32(tables)
    p = vv.vv_paged_plan(i32(lens), i32(new), t, i32(free), ps, pages, total + 3, prefix_len=prefix)
    vv.vv_sync_status()
    after, offsets, slots, pos, want, cur = obatch.paged_plan(lens, new, tables, free, ps, total + 3, prefix)
    for got, y in ((p.lens, after), (p.offsets, offsets), (p.slots, slots), (p.positions, pos), (t, want)):
        assert np.array_equal(got.cpu().numpy(), y)
    assert p.cursor.item() == cur
