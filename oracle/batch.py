"""Float64 / integer definitions of the operators of a batch that continues one shared prompt.

Plain numpy loops over requests, tokens and rows; nothing here is shared with the CUDA path.
"""

import math

import numpy as np

from . import ops


def paged_plan(lens, new_lens, tables, free_pages, page_size, max_tokens, prefix_len=0, cursor=0):
    """Block tables, slots and positions of a step's new tokens, request by request.

    Returns (lens after, offsets [B + 1], slots [max_tokens], positions [max_tokens], tables,
    cursor after).  Inputs must be valid: pages enough, tables wide enough, tokens within
    max_tokens."""
    tables = np.array(tables, dtype=np.int64)
    slots = np.full(max_tokens, -1, dtype=np.int64)
    positions = np.zeros(max_tokens, dtype=np.int64)
    offsets = [0]
    after = []
    for b, (n, add) in enumerate(zip(lens, new_lens)):
        for j in range(int(add)):
            i = int(n) + j
            block, cell = divmod(i, page_size)
            if cell == 0:  # the first token of a page takes the next free one
                tables[b, block] = free_pages[cursor]
                cursor += 1
            slots[offsets[-1] + j] = int(tables[b, block]) * page_size + cell
            positions[offsets[-1] + j] = prefix_len + i
        offsets.append(offsets[-1] + int(add))
        after.append(int(n) + int(add))
    return np.array(after), np.array(offsets), slots, positions, tables, cursor


def qk_rope_append(q, k, v, positions, slots, k_pages, v_pages, theta, q_gain=None, k_gain=None,
                   eps=1e-6):
    """Returns (q rotated, k_pages, v_pages) in float64; pages [pages, Hkv, page_size, D]."""
    def turned(x, gain):
        x = np.asarray(x, np.float64)
        if gain is not None:
            x = ops.rmsnorm(x, gain, eps)
        return ops.rope(x, np.asarray(positions)[:, None], theta)

    qr, kr = turned(q, q_gain), turned(k, k_gain)
    kp, vp = np.array(k_pages, np.float64), np.array(v_pages, np.float64)
    ps = kp.shape[2]
    for t, slot in enumerate(slots):
        if slot >= 0:
            page, cell = divmod(int(slot), ps)
            kp[page, :, cell] = kr[t]
            vp[page, :, cell] = np.asarray(v[t], np.float64)
    return qr, kp, vp


def prefix_attention(q, k_prefix, v_prefix, k_pages, v_pages, tables, lens, scale):
    """Returns (out, lse, weighted mean of |v|, smallest sum of exp(score - max)) in float64.

    q [B, Hq, D]; prefix [Hkv, P, D]; pages [pages, Hkv, page_size, D].  A sequence without keys
    gives zeros and -inf.  The third value bounds what rounding the weights can do to `out`."""
    q = np.asarray(q, np.float64)
    B, Hq, D = q.shape
    Hkv, ps = k_pages.shape[1], k_pages.shape[2]
    G = Hq // Hkv
    out, mean_abs = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, total = np.full((B, Hq), -np.inf), np.ones((B, Hq))
    for b in range(B):
        n = max(int(lens[b]), 0)
        pages = [int(p) for p in tables[b][: -(-n // ps)]]
        for h in range(Hq):
            g = h // G
            ks = [np.asarray(k_prefix[g], np.float64)] if k_prefix is not None else []
            vs = [np.asarray(v_prefix[g], np.float64)] if v_prefix is not None else []
            for i, p in enumerate(pages):
                ks.append(np.asarray(k_pages[p, g, : n - i * ps], np.float64))
                vs.append(np.asarray(v_pages[p, g, : n - i * ps], np.float64))
            if not ks or sum(len(x) for x in ks) == 0:
                continue
            K, V = np.concatenate(ks), np.concatenate(vs)
            s = scale * (K @ q[b, h])
            m = s.max()
            if m == -np.inf:
                continue
            w = np.exp(s - m)
            total[b, h] = w.sum()
            out[b, h] = w @ V / w.sum()
            mean_abs[b, h] = w @ np.abs(V) / w.sum()
            lse[b, h] = m + math.log(w.sum())
    return out, lse, mean_abs, total


def logits_process(logits, tokens=None, token_lens=None, prompt_lens=None, repetition=None,
                   frequency=None, presence=None, bias=None, allowed=None):
    """Returns (processed logits float64 [B, V], greedy token per row, -1 where nothing is left).

    bias: per row a dict token -> value; allowed: bool [B, V] or None."""
    x = np.array(logits, dtype=np.float64)
    B, V = x.shape
    idx = np.full(B, -1)
    for b in range(B):
        if tokens is not None:
            n_prompt = 0 if prompt_lens is None else int(prompt_lens[b])
            said = {}
            row = [int(t) for t in tokens[b][: int(token_lens[b])]]
            for t in row[n_prompt:]:
                said[t] = said.get(t, 0) + 1
            for t in set(row):
                if not 0 <= t < V:
                    continue
                if repetition is not None:
                    r = float(repetition[b])
                    x[b, t] = x[b, t] / r if x[b, t] > 0 else x[b, t] * r
                if t in said:
                    x[b, t] -= said[t] * (0.0 if frequency is None else float(frequency[b]))
                    x[b, t] -= 0.0 if presence is None else float(presence[b])
        if bias is not None:
            for t, w in bias[b].items():
                if 0 <= t < V:
                    x[b, t] += float(w)
        if allowed is not None:
            x[b, ~allowed[b]] = -np.inf
        live = np.where(np.isnan(x[b]), -np.inf, x[b])
        if live.max() > -np.inf:
            idx[b] = int(np.argmax(live))
    return x, idx
