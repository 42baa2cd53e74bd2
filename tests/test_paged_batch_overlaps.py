"""Overlapping arguments of the batch operators are refused before anything reaches a GPU (CPU only):
their CTAs read the inputs for themselves while others already write the outputs."""

import pytest

from test_paged_batch_args import A, PLAN, ROPE, addr, call, vv

B, MAX_BLOCKS, TOKENS, N_FREE = (PLAN[k] for k in ("B", "max_blocks", "max_tokens", "n_free"))
IN = {"lens": 4 * B, "new": 4 * B, "free": 4 * N_FREE, "cursor": 4}
OUT = {"table": 4 * B * MAX_BLOCKS, "lens_out": 4 * B, "offsets": 4 * (B + 1), "slots": 8 * TOKENS,
       "positions": 4 * TOKENS, "cursor_out": 4}
ALIGN = {"slots": 16, "positions": 16}


def overlapping(x, nx, ny):
    """Offsets of x (nx bytes) from y's start at which both meet: in place, at y's last bytes, and
    before y with x's last bytes on its first ones."""
    step = ALIGN.get(x, 4)
    return sorted({0, (ny - 1) // step * step, -((nx - 1) // step * step)})


PAIRS = [(o, i) for o in OUT for i in IN] + [(o, p) for o in OUT for p in OUT if o < p]


@pytest.mark.parametrize("x,y", PAIRS)
def test_plan_refuses_every_overlap_with_an_output(x, y):
    sizes = {**IN, **OUT}
    base = dict(PLAN, cursor=addr(9))
    for d in overlapping(x, sizes[x], sizes[y]):
        assert call("vv_paged_plan", base, **{x: base[y] + d}) == A, (x, y, d)
        assert "overlap" in vv.last_error()[1], (x, y, d)


# q_out against k and v (bytes; rows of 4 query and 2 key-value heads are 1024 and 512 bytes long)
FUSED = dict(ROPE, q=addr(0), k=addr(0) + 1024, v=addr(0) + 1536, qs=1024, ks=1024, vs=1024, os=1024, out=addr(0))


@pytest.mark.parametrize("base,change", [
    (ROPE, dict(out=addr(1))), (ROPE, dict(out=addr(2))), (ROPE, dict(out=addr(1) + 3 * 512 - 16)),
    (ROPE, dict(out=addr(2) - 1024 * 2 - 1008)), (ROPE, dict(out=addr(1), T=1)),
    (FUSED, dict(k=addr(0) + 1008)), (FUSED, dict(v=addr(0) + 2048 - 496)), (FUSED, dict(v=addr(0) + 4096 - 496)),
    (FUSED, dict(k=addr(0) + 1024 - 2048 + 16, v=addr(0) + 512)), (FUSED, dict(k=addr(0) + 1024, ks=256))])
def test_rope_append_refuses_q_out_over_keys_or_values(base, change):
    assert call("vv_qk_rope_append", base, **change) == A, (change, vv.last_error())
    assert "k and v" in vv.last_error()[1]
