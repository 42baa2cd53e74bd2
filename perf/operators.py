"""The operators of a batch that continues one shared prompt, as cases to measure.

Several candidate transcripts of one recording, or several questions about it, decode together
from one prefilled prompt.  A step of such a batch goes through four operators:

  plan    block tables, slot map, positions and row offsets of the step's tokens, from the
          requests' lengths and a list of free pages (vv_paged_plan)
  rope    RMS norm of every query and key head (where the model has such gains), rotate-half
          positions, and the write of keys and values into their pages (vv_qk_rope_append)
  attn    grouped-query attention of one token per sequence over the prompt that all share and
          the sequence's own pages (vv_gqa_prefix_attn)
  logits  penalties for repeated tokens, biases and a grammar's bit mask on the logits, and the
          greedy token of each row (vv_logits_process)

Head counts, vocabularies and context lengths are those of the repository's own backbones:
12 query / 2 key-value heads and 151936 tokens (1.5B), 28 / 4 and 152064 (7B), 7 / 1 (0.5B),
head dimension 128, prompts of 1024, 4096, 4530 and 32768 positions.

With `own` false everything here is elementary torch in 32 bits (angles in 64).
"""

import math
import random

import torch

own = False

D = 128
THETA = 1.0e6
EPS = 1.0e-6
SPEECH_PAD = 151648  # the id that fills the audio span of a prompt
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one step of a running batch: every request appends one token
        {"name": "plan-step", "op": "plan", "B": 32, "max_len": 512, "max_new": 1, "long": 0,
         "page": 16, "prefix": 4530},
        # steps and newly admitted prompts in one batch, ragged
        {"name": "plan-mixed", "op": "plan", "B": 301, "max_len": 2048, "max_new": 9, "long": 4530,
         "page": 64, "prefix": 0},
        # a whole queue admitted at once
        {"name": "plan-admit", "op": "plan", "B": 4096, "max_len": 129, "max_new": 380, "long": 0,
         "page": 32, "prefix": 1024},
        # one decode step of the 1.5B model: 16 tokens, no gains
        {"name": "rope-step", "op": "rope", "T": 16, "Hq": 12, "Hkv": 2, "type": "f16",
         "gains": False, "page": 16, "fused": True, "far": 4786},
        # one recording's prompt, 7B heads, head norms
        {"name": "rope-prompt", "op": "rope", "T": 4530, "Hq": 28, "Hkv": 4, "type": "bf16",
         "gains": True, "page": 64, "fused": True, "far": 4530},
        # several prompts packed one behind the other, odd length, far positions
        {"name": "rope-packed", "op": "rope", "T": 50001, "Hq": 28, "Hkv": 4, "type": "f16",
         "gains": False, "page": 32, "fused": False, "far": 1000000},
        # a pair of sequences on a short prompt: latency counts
        {"name": "attn-pair", "op": "attn", "B": 2, "Hq": 12, "Hkv": 2, "P": 1024, "own": 64,
         "page": 16, "type": "f16", "lse": False},
        # 16 transcripts of a ten-minute recording, 1.5B
        {"name": "attn-recording", "op": "attn", "B": 16, "Hq": 12, "Hkv": 2, "P": 4530,
         "own": 257, "page": 16, "type": "f16", "lse": False},
        # 48 sequences on a 32k document, 7B
        {"name": "attn-document", "op": "attn", "B": 48, "Hq": 28, "Hkv": 4, "P": 32768,
         "own": 1024, "page": 64, "type": "bf16", "lse": True},
        # nothing shared: ragged sequences in pages alone
        {"name": "attn-apart", "op": "attn", "B": 23, "Hq": 28, "Hkv": 4, "P": 0, "own": 4785,
         "page": 32, "type": "f16", "lse": False},
        # one row with a short history
        {"name": "logits-one", "op": "logits", "B": 1, "V": 151936, "prompt": 30, "out": 270,
         "bias": 0, "mask": False, "type": "f32"},
        # a batch with the recording's prompt as history, biases and a grammar
        {"name": "logits-batch", "op": "logits", "B": 64, "V": 152064, "prompt": 4530, "out": 255,
         "bias": 300, "mask": True, "type": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((12, 2), (28, 4), (7, 1), (4, 2))


def draw(rng):
    op = rng.choice(("plan", "rope", "attn", "attn", "logits"))
    if op == "plan":
        b = _log(rng, 1, 4096)
        new = rng.choice((1, _log(rng, 2, max(2, min(2000, 700000 // b)))))
        return {"op": op, "B": b, "max_len": _log(rng, 1, 2048), "max_new": new,
                "long": rng.choice((0, _log(rng, 100, 4530))) if b <= 512 else 0,
                "page": rng.choice((16, 32, 48, 64, 128)), "prefix": rng.choice((0, _log(rng, 1, 32768)))}
    if op == "rope":
        hq, hkv = rng.choice(HEADS)
        return {"op": op, "T": _log(rng, 1, 50000 * 28 // max(hq, 28)), "Hq": hq, "Hkv": hkv,
                "type": rng.choice(("f16", "bf16")), "gains": rng.random() < 0.5,
                "page": rng.choice((16, 32, 64)), "fused": rng.random() < 0.5,
                "far": _log(rng, 1000, 1000000)}
    if op == "attn":
        hq, hkv = rng.choice(HEADS + ((8, 8), (8, 1)))
        b = _log(rng, 1, 48)
        p = rng.choice((0, _log(rng, 1, 32768), _log(rng, 1, 32768)))
        return {"op": op, "B": b, "Hq": hq, "Hkv": hkv, "P": p,
                "own": _log(rng, 1, 4785 if p == 0 else 1024), "page": rng.choice((16, 32, 64, 128)),
                "type": rng.choice(("f16", "bf16")), "lse": rng.random() < 0.5}
    return {"op": op, "B": _log(rng, 1, 64), "V": rng.choice((151936, 152064, 32000 + rng.randrange(1000), 1000)),
            "prompt": rng.choice((0, _log(rng, 1, 4530))), "out": _log(rng, 1, 2000),
            "bias": rng.choice((0, _log(rng, 1, 300))), "mask": rng.random() < 0.5,
            "type": rng.choice(("f32", "f32", "f16", "bf16"))}


# ------------------------------------------------------------------------------------ inputs
# Lengths belong to the case (work() needs them); values come from the seed.
def _plan_lens(c):
    r = random.Random(c["B"] * 7919 + c["max_len"] * 31 + c["max_new"])
    lens = [r.randint(0, c["max_len"]) for _ in range(c["B"])]
    if c["max_new"] == 1:
        new = [1] * c["B"]
    else:
        new = [r.randint(0, c["max_new"]) for _ in range(c["B"])]
    if c["long"]:
        for b in range(0, c["B"], 13):  # a newly admitted prompt
            lens[b], new[b] = 0, r.randint(c["long"] // 2 + 1, c["long"])
    return lens, new


def _own_lens(c):
    r = random.Random(c["B"] * 104729 + c["own"])
    lens = [r.randint(1, c["own"]) for _ in range(c["B"])]
    lens[r.randrange(c["B"])] = c["own"]
    if c["B"] > 4:
        lens[r.randrange(c["B"])] = 0  # a sequence that has just been forked from the prompt
    return lens


def _out_lens(c):
    r = random.Random(c["B"] * 65537 + c["out"])
    return [r.randint(c["out"] // 2, c["out"]) for _ in range(c["B"])]


def _ceil(a, b):
    return -(-a // b)


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case)
    del case

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    def perm(n):
        return torch.randperm(n, generator=g, device=dev).to(torch.int32)

    if s["op"] == "plan":
        lens, new = _plan_lens(s)
        page = s["page"]
        old = [_ceil(n, page) for n in lens]
        need = [_ceil(a + b, page) for a, b in zip(lens, new)]
        used, total = sum(old), sum(need)
        s["pool"] = total + 17
        pages = perm(s["pool"])
        s["max_blocks"] = max(max(need), 1) + 3
        table = torch.full((s["B"], s["max_blocks"]), -1, dtype=torch.int32, device=dev)
        held = torch.arange(s["max_blocks"], device=dev)[None, :] < _i32(old, dev)[:, None]
        table[held] = pages[:used]
        s["table"], s["free"] = table, pages[used:].contiguous()
        s["lens"], s["new"] = _i32(lens, dev), _i32(new, dev)
        s["tokens"] = max(sum(new), 1) + sum(new) % 5  # a few padding rows behind the last token
    elif s["op"] == "rope":
        t, hq, hkv, ty = s["T"], s["Hq"], s["Hkv"], TYPES[s["type"]]
        if s["fused"]:  # one projection's output, read in place through its row stride
            qkv = normal(t, hq + 2 * hkv, D, dtype=ty)
            s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        else:
            s["q"], s["k"], s["v"] = (normal(t, h, D, dtype=ty) for h in (hq, hkv, hkv))
        s["gq"] = (1 + normal(D, std=0.2)).to(ty) if s["gains"] else None
        s["gk"] = (1 + normal(D, std=0.2)).to(ty) if s["gains"] else None
        first = torch.randint(0, max(1, s["far"] - t), (1,), generator=g, device=dev)
        s["pos"] = (first + torch.arange(t, device=dev)).to(torch.int32)
        pages = _ceil(t, s["page"]) + 2
        at = perm(pages)[torch.arange(t, device=dev) // s["page"]].long()
        s["slots"] = at * s["page"] + torch.arange(t, device=dev) % s["page"]
        if t > 20:
            s["slots"][t - 3:] = -1  # padding rows of a fixed-size batch
        s["kp"], s["vp"] = (normal(pages, hkv, s["page"], D, dtype=ty) for _ in range(2))
        if own:
            from int4_blockwise_quantised_b200 import _vv
            s["kv"] = _vv.PagedKV(s["kp"], s["vp"])
    elif s["op"] == "attn":
        b, hq, hkv, ty, page = s["B"], s["Hq"], s["Hkv"], TYPES[s["type"]], s["page"]
        lens = _own_lens(s)
        blocks = [_ceil(n, page) for n in lens]
        pages = sum(blocks) + 5
        s["q"] = normal(b, hq, D, dtype=ty, std=1.5)
        s["kpre"], s["vpre"] = (normal(hkv, s["P"], D, dtype=ty) if s["P"] else None for _ in range(2))
        s["kp"], s["vp"] = (normal(pages, hkv, page, D, dtype=ty) for _ in range(2))
        s["max_blocks"] = _ceil(s["own"], page) + 1
        table = torch.full((b, s["max_blocks"]), -1, dtype=torch.int32, device=dev)
        held = torch.arange(s["max_blocks"], device=dev)[None, :] < _i32(blocks, dev)[:, None]
        table[held] = perm(pages)[: sum(blocks)]
        s["table"], s["lens"], s["scale"] = table, _i32(lens, dev), 1 / math.sqrt(D)
        if own:
            from int4_blockwise_quantised_b200 import _vv
            s["kv"] = _vv.PagedKV(s["kp"], s["vp"])
            n = _vv.vv_gqa_prefix_attn_workspace_size(b, hq, hkv, D, s["P"], s["max_blocks"] * page)
            s["ws"] = torch.zeros(n, dtype=torch.uint8, device=dev)
    else:
        b, v = s["B"], s["V"]
        s["logits"] = normal(b, v, dtype=TYPES[s["type"]], std=3.0)
        outs = _out_lens(s)
        width = s["prompt"] + s["out"]
        # text ids crowd towards the low end, the prompt's audio span is one id
        tok = (v * torch.rand((b, width), generator=g, device=dev).pow(3)).long().clamp_(max=v - 1)
        if s["prompt"] > 30:
            tok[:, 20:s["prompt"] - 10] = min(SPEECH_PAD, v - 1)
        s["tok"] = tok.to(torch.int32)
        s["prompt_lens"] = torch.full((b,), s["prompt"], dtype=torch.int32, device=dev)
        s["tok_lens"] = s["prompt_lens"] + _i32(outs, dev)
        s["rep"] = 1.05 + 0.3 * torch.rand(b, generator=g, device=dev)
        s["freq"] = 0.5 * torch.rand(b, generator=g, device=dev)
        s["pres"] = 0.5 * torch.rand(b, generator=g, device=dev)
        n = s["bias"]
        s["bias_ids"] = s["bias_vals"] = s["bias_offsets"] = s["bits"] = None
        if n:  # every row its own ids, none twice in a row
            start = torch.randint(0, v, (b, 1), generator=g, device=dev)
            ids = (start + 7919 * torch.arange(n, device=dev)[None, :]) % v
            s["bias_ids"] = ids.to(torch.int32).reshape(-1)
            s["bias_vals"] = normal(b * n, std=4.0)
            s["bias_offsets"] = (n * torch.arange(b + 1, device=dev)).to(torch.int32)
        if s["mask"]:  # a grammar allows few ids in some rows, most in others, none in a dead end
            share = torch.tensor([0.002, 0.9, 0.3], device=dev)[torch.arange(b, device=dev) % 3]
            bits = torch.rand((b, _ceil(v, 32) * 32), generator=g, device=dev) < share[:, None]
            if b > 3:
                bits[2] = False
            weights = 1 << torch.arange(32, device=dev)
            words = (bits.view(b, -1, 32).long() * weights).sum(-1)
            s["bits"] = (words - ((words >> 31) << 32)).to(torch.int32)
        if own:
            from int4_blockwise_quantised_b200 import _vv
            s["ws"] = torch.zeros(_vv.vv_logits_process_workspace_size(b), dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------------------------------- run
def run(s):
    if own:
        return RUN_OWN[s["op"]](s)
    return RUN_PLAIN[s["op"]](s)


def _own_plan(s):
    from int4_blockwise_quantised_b200 import _vv
    p = _vv.vv_paged_plan(s["lens"], s["new"], s["table"], s["free"], s["page"], s["pool"],
                          s["tokens"], prefix_len=s["prefix"])
    return {"lens": p.lens, "offsets": p.offsets, "slots": p.slots, "positions": p.positions,
            "used": p.cursor, "table": s["table"]}


def _own_rope(s):
    from int4_blockwise_quantised_b200 import _vv
    q = _vv.vv_qk_rope_append(s["q"], s["k"], s["v"], s["pos"], s["slots"], s["kv"], THETA,
                              q_gain=s["gq"], k_gain=s["gk"], eps=EPS)
    return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}


def _own_attn(s):
    from int4_blockwise_quantised_b200 import _vv
    lse = torch.empty((s["B"], s["Hq"]), dtype=torch.float32, device=s["q"].device) if s["lse"] else None
    o = _vv.vv_gqa_prefix_attn(s["q"], s["kpre"], s["vpre"], s["kv"], s["table"], s["lens"],
                               s["scale"], s["ws"], lse=lse)
    return {"out": o, "lse": lse} if s["lse"] else {"out": o}


def _own_logits(s):
    from int4_blockwise_quantised_b200 import _vv
    out, idx = _vv.vv_logits_process(
        s["logits"], s["ws"], tokens=s["tok"], token_lens=s["tok_lens"], prompt_lens=s["prompt_lens"],
        repetition=s["rep"], frequency=s["freq"], presence=s["pres"], bias_ids=s["bias_ids"],
        bias_vals=s["bias_vals"], bias_offsets=s["bias_offsets"], mask=s["bits"])
    return {"logits": out, "argmax": idx}


RUN_OWN = {"plan": _own_plan, "rope": _own_rope, "attn": _own_attn, "logits": _own_logits}


def _plain_plan(s):
    lens, new, page, dev = s["lens"].long(), s["new"].long(), s["page"], s["lens"].device
    after = lens + new
    old, need = (lens + page - 1) // page, (after + page - 1) // page
    fresh = torch.cumsum(need - old, 0)
    base = fresh - (need - old)
    j = torch.arange(s["max_blocks"], device=dev)[None, :]
    is_new = (j >= old[:, None]) & (j < need[:, None])
    take = (base[:, None] + j - old[:, None]).clamp(0, s["free"].numel() - 1)
    s["table"] = torch.where(is_new, s["free"][take], s["table"])
    ends = torch.cumsum(new, 0)
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), ends])
    t = torch.arange(s["tokens"], device=dev)
    b = torch.searchsorted(ends, t, right=True).clamp(max=s["B"] - 1)
    real = t < ends[-1]
    at = lens[b] + t - offsets[b]
    block = (at // page).clamp(0, s["max_blocks"] - 1)
    slots = torch.where(real, s["table"][b, block].long() * page + at % page, -1)
    positions = torch.where(real, s["prefix"] + at, 0)
    return {"lens": after.to(torch.int32), "offsets": offsets.to(torch.int32), "slots": slots,
            "positions": positions.to(torch.int32), "used": fresh[-1:].to(torch.int32),
            "table": s["table"]}


def _plain_rotated(x, gain, pos):
    x = x.float()
    if gain is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * gain.float()
    i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    angle = pos.double()[:, None] * THETA ** (-2.0 * i / D)
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    a, b = x[..., : D // 2], x[..., D // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _plain_rope(s):
    ty, page = TYPES[s["type"]], s["page"]
    q = _plain_rotated(s["q"], s["gq"], s["pos"]).to(ty)
    k = _plain_rotated(s["k"], s["gk"], s["pos"]).to(ty)
    keep = s["slots"] >= 0
    at = s["slots"][keep]
    s["kp"][at // page, :, at % page] = k[keep]
    s["vp"][at // page, :, at % page] = s["v"][keep]
    return {"q": q, "k_pages": s["kp"], "v_pages": s["vp"]}


def _plain_attn(s):
    b, hq, hkv, page = s["B"], s["Hq"], s["Hkv"], s["page"]
    grp, width = hq // hkv, s["max_blocks"] * s["page"]
    q = s["q"].float().view(b, hkv, grp, D) * s["scale"]
    at = s["table"].long().clamp(min=0)

    def rows(pool):  # [b, hkv, width, D]
        return pool[at].permute(0, 2, 1, 3, 4).reshape(b, hkv, width, D).float()

    live = torch.arange(width, device=q.device)[None, :] < s["lens"][:, None]
    scores = torch.matmul(q, rows(s["kp"]).transpose(-1, -2))
    scores = torch.where(live[:, None, None, :], scores, -math.inf)
    if s["P"]:
        # the shared part as one product a key-value head: [hkv, b * grp, P]
        qs = q.permute(1, 0, 2, 3).reshape(hkv, b * grp, D)
        shared = torch.matmul(qs, s["kpre"].float().transpose(-1, -2))
        shared = shared.view(hkv, b, grp, s["P"]).permute(1, 0, 2, 3)
        scores = torch.cat([shared, scores], -1)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    own_p = p[..., s["P"]:]
    values = torch.where(live[:, None, :, None], rows(s["vp"]), 0.0)
    o = torch.matmul(own_p, values)
    if s["P"]:
        ps = p[..., : s["P"]].permute(1, 0, 2, 3).reshape(hkv, b * grp, s["P"])
        o = o + torch.matmul(ps, s["vpre"].float()).view(hkv, b, grp, D).permute(1, 0, 2, 3)
    o = torch.where(total > 0, o / total, 0.0).reshape(b, hq, D).to(TYPES[s["type"]])
    if not s["lse"]:
        return {"out": o}
    return {"out": o, "lse": (torch.log(total) + top).reshape(b, hq)}


def _plain_logits(s):
    b, v, dev = s["B"], s["V"], s["logits"].device
    x = s["logits"].float()
    tok, j = s["tok"].long(), torch.arange(s["tok"].shape[1], device=dev)[None, :]
    there = j < s["tok_lens"][:, None]
    said = there & (j >= s["prompt_lens"][:, None])
    seen = torch.zeros((b, v), dtype=torch.int32, device=dev).scatter_add_(1, tok, there.int()) > 0
    count = torch.zeros((b, v), dtype=torch.int32, device=dev).scatter_add_(1, tok, said.int())
    rep = s["rep"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = torch.where(count > 0, x - s["freq"][:, None] * count - s["pres"][:, None], x)
    if s["bias"]:
        row = torch.arange(b, device=dev).repeat_interleave(s["bias"])
        bias = torch.zeros((b, v), device=dev)
        bias[row, s["bias_ids"].long()] = s["bias_vals"]
        x = x + bias
    if s["mask"]:
        at = torch.arange(v, device=dev)
        allowed = (s["bits"][:, at >> 5] >> (at & 31)[None, :].int()) & 1
        x = torch.where(allowed > 0, x, -math.inf)
    best = torch.argmax(x, -1)
    none = x.gather(1, best[:, None])[:, 0] == -math.inf
    return {"logits": x.to(s["logits"].dtype), "argmax": torch.where(none, -1, best).to(torch.int32)}


RUN_PLAIN = {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn, "logits": _plain_logits}


# -------------------------------------------------------------------------------------- work
def work(c):
    if c["op"] == "plan":
        lens, new = _plan_lens(c)
        fresh = sum(_ceil(a + n, c["page"]) - _ceil(a, c["page"]) for a, n in zip(lens, new))
        # lengths in and out, offsets; free pages in, entries out; slot (8) and position (4) a token
        return {"bytes": 16 * c["B"] + 8 * fresh + 12 * sum(new), "flops": 4 * sum(new)}
    if c["op"] == "rope":
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": c["T"] * (heads * D * 2 * 2 + 12),
                "flops": c["T"] * (c["Hq"] + c["Hkv"]) * D * (7 if c["gains"] else 3)}
    if c["op"] == "attn":
        keys = sum(_own_lens(c))
        kv = 2 * 2 * D * c["Hkv"] * (c["P"] + keys)
        return {"bytes": kv + 2 * 2 * D * c["B"] * c["Hq"] + 4 * c["B"] * c["Hq"] * c["lse"],
                "flops": 4 * D * c["Hq"] * (c["B"] * c["P"] + keys)}
    size = 4 if c["type"] == "f32" else 2
    rows = c["B"] * c["V"]
    per_row = 4 * c["prompt"] + 8 * c["bias"] + (c["V"] / 8 if c["mask"] else 0)
    return {"bytes": 2 * size * rows + c["B"] * per_row + 4 * sum(_out_lens(c)), "flops": 3 * rows}


# ------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"plan": lambda s: None, "rope": _exact_rope, "attn": _exact_attn,
                "logits": _exact_logits}[s["op"]](s)


def _exact_rope(s):
    k_pages, v_pages = s["kp"].double(), s["vp"].double()
    exponent = torch.arange(0, D, 2, dtype=torch.float64, device=s["q"].device) / D
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=s["q"].device),
                       s["pos"].double().outer(THETA ** -exponent))

    def turned(x, gain):
        x = x.double()
        if gain is not None:
            x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * gain.double()
        z = torch.complex(x[..., : D // 2].contiguous(), x[..., D // 2:].contiguous()) * turn[:, None]
        return torch.cat((z.real, z.imag), -1)

    q, k = turned(s["q"], s["gq"]), turned(s["k"], s["gk"])
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    page, cell = s["slots"][rows] // s["page"], s["slots"][rows] % s["page"]
    k_pages.permute(0, 2, 1, 3)[page, cell] = k[rows]
    v_pages.permute(0, 2, 1, 3)[page, cell] = s["v"].double()[rows]
    return {"q": q, "k_pages": k_pages, "v_pages": v_pages}


def _exact_attn(s):
    grp, dev = s["Hq"] // s["Hkv"], s["q"].device
    out = torch.zeros((s["B"], s["Hq"], D), dtype=torch.float64, device=dev)
    lse = torch.full((s["B"], s["Hq"]), -math.inf, dtype=torch.float64, device=dev)
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, : _ceil(n, s["page"])].long()
        for h in range(s["Hkv"]):
            k = s["kp"][pages, h].reshape(-1, D)[:n].double()
            v = s["vp"][pages, h].reshape(-1, D)[:n].double()
            if s["P"]:
                k = torch.cat((s["kpre"][h].double(), k))
                v = torch.cat((s["vpre"][h].double(), v))
            if not len(k):
                continue
            at = slice(h * grp, (h + 1) * grp)
            x = s["q"][b, at].double() @ k.T * s["scale"]
            lse[b, at] = torch.logsumexp(x, -1)
            out[b, at] = torch.softmax(x, -1) @ v
    return {"out": out, "lse": lse} if s["lse"] else {"out": out}


def _exact_logits(s):
    v = s["V"]
    rows = []
    for b in range(s["B"]):
        x = s["logits"][b].double()
        whole = s["tok"][b, : int(s["tok_lens"][b])].long()
        heard = torch.bincount(whole, minlength=v) > 0
        said = torch.bincount(whole[int(s["prompt_lens"][b]):], minlength=v).double()
        r = s["rep"][b].double()
        x = torch.where(heard & (x > 0), x / r, torch.where(heard, x * r, x))
        x = x - s["freq"][b].double() * said - s["pres"][b].double() * (said > 0)
        if s["bias"]:
            part = slice(b * s["bias"], (b + 1) * s["bias"])
            x[s["bias_ids"][part].long()] += s["bias_vals"][part].double()
        if s["mask"]:
            word = s["bits"][b].long() & 0xFFFFFFFF
            bit = (word[:, None] >> torch.arange(32, device=x.device)) & 1
            x[bit.reshape(-1)[:v] == 0] = -math.inf
        rows.append(x)
    return {"logits": torch.stack(rows), "argmax": None}
