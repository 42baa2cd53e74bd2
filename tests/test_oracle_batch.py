"""Pins of oracle.batch (CPU only): hand-made cases and independent formulations."""

import numpy as np

import synth
from oracle import batch, ops


def test_plan_hand_made():
    # pages of 4; request 0 holds 3 tokens (page 7), 1 holds 4 (page 2), 2 is new, 3 appends none
    tables = np.array([[7, -1, -1], [2, -1, -1], [-1, -1, -1], [5, -1, -1]])
    after, offsets, slots, pos, t, cur = batch.paged_plan(
        [3, 4, 0, 2], [2, 1, 5, 0], tables, [9, 8, 6, 1, 0], 4, 10, prefix_len=100, cursor=1)
    assert after.tolist() == [5, 5, 5, 2] and offsets.tolist() == [0, 2, 3, 8, 8] and cur == 5
    assert t.tolist() == [[7, 8, -1], [2, 6, -1], [1, 0, -1], [5, -1, -1]]
    assert slots.tolist() == [31, 32, 24, 4, 5, 6, 7, 0, -1, -1]
    assert pos.tolist() == [103, 104, 104, 100, 101, 102, 103, 104, 0, 0]


def test_append_writes_only_the_named_cells():
    T, hq, hkv, D = 3, 4, 2, 8
    q, k, v = (synth.normal_f32((T, h, D), 1.0, i) for i, h in enumerate((hq, hkv, hkv)))
    kp = synth.normal_f32((2, hkv, 4, D), 1.0, 5)
    qr, k1, v1 = batch.qk_rope_append(q, k, v, [0, 3, 5], [6, -1, 1], kp, kp, 1e4)
    assert np.allclose(qr[0], q[0])  # position 0 turns nothing
    assert np.allclose(k1[1, :, 2], k[0]) and np.array_equal(v1[0, :, 1], v[2].astype(np.float64))
    changed = np.any(k1 != kp, axis=(1, 3))
    assert changed.tolist() == [[False, True, False, False], [False, False, True, False]]
    n = batch.qk_rope_append(q, k, v, [0, 3, 5], [6, -1, 1], kp, kp, 1e4, q_gain=np.full(D, 2.0),
                             eps=0.0)[0]
    assert np.allclose(np.mean(n * n, -1), 4.0)  # unit rms, doubled; a rotation keeps it


def test_prefix_attention_is_attention_over_the_joined_keys():
    B, hq, hkv, D, P, ps = 3, 4, 2, 8, 5, 4
    q = synth.normal_f32((B, hq, D), 1.0, 1)
    kpre, vpre = synth.normal_f32((hkv, P, D), 1.0, 2), synth.normal_f32((hkv, P, D), 1.0, 3)
    kp, vp = synth.normal_f32((6, hkv, ps, D), 1.0, 4), synth.normal_f32((6, hkv, ps, D), 1.0, 5)
    tables, lens = [[4, 1], [0, -1], [-1, -1]], [7, 2, 0]
    out, lse, _, _ = batch.prefix_attention(q, kpre, vpre, kp, vp, tables, lens, 0.3)
    for b in range(B):
        pages = tables[b][: -(-lens[b] // ps)]
        ks = np.concatenate([kpre] + [kp[p] for p in pages], axis=1)[:, : P + lens[b]]
        vs = np.concatenate([vpre] + [vp[p] for p in pages], axis=1)[:, : P + lens[b]]
        assert np.allclose(out[b], ops.gqa_decode_attention(q[b], ks, vs, 0.3))
        for h in range(hq):
            assert np.isclose(lse[b, h], np.log(np.sum(np.exp(0.3 * ks[h // 2] @ q[b, h]))))
    out, lse, _, _ = batch.prefix_attention(q, None, None, kp, vp, tables, lens, 0.3)
    assert np.all(out[2] == 0) and np.all(np.isneginf(lse[2]))


def test_logits_hand_made():
    x = [[2.0, -2.0, 4.0, 0.5, 1.0], [1.0, 3.0, 3.0, 0.0, -1.0]]
    tokens, lens, prompts = [[0, 1, 2, 2], [4, 9, -1, 0]], [4, 3], [2, 1]
    y, idx = batch.logits_process(x, tokens, lens, prompts, [2.0, 2.0], [0.5, 0.5], [0.25, 0.25],
                                  bias=[{3: 1.5}, {}],
                                  allowed=np.array([[1, 1, 1, 1, 0], [0, 0, 0, 0, 0]], bool))
    # row 0: 0 and 1 are the prompt's, 2 was generated twice: 4 / 2 - 2 * 0.5 - 0.25
    assert y[0].tolist() == [1.0, -4.0, 0.75, 2.0, -np.inf] and idx.tolist() == [3, -1]
    y, idx = batch.logits_process(x, tokens, lens, prompts, [2.0, 2.0])
    assert y[1].tolist() == [1.0, 3.0, 3.0, 0.0, -2.0] and idx[1] == 1  # lowest of a tie
