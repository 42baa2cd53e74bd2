"""The workspace of vv_gqa_prefix_attn, sized once for the largest batch, prompt and table, serves every
smaller one (CPU only)."""

import pytest

from test_paged_batch_args import vv

SIZE = vv.vv_gqa_prefix_attn_workspace_size
BATCHES = [1, 2, 3, 8, 16, 18, 21, 22, 37, 48, 64, 65, 128, 129, 500, 4096, 65535]
PROMPTS = [0, 1, 127, 128, 129, 1000, 2048, 3968, 4096, 4530, 32768, 100000, (1 << 24) - 1]
OWN = [0, 1, 16, 17, 257, 4800, 1 << 31, (1 << 31) * (1 << 31)]


@pytest.mark.parametrize("hq,hkv", [(12, 2), (28, 4), (7, 1), (16, 1), (8, 8), (1024, 1024)])
def test_workspace_grows_with_batch_prompt_and_table(hq, hkv):
    need = {(b, p, n): SIZE(b, hq, hkv, 128, p, n) for b in BATCHES for p in PROMPTS for n in OWN}
    assert all(0 < x < 1 << 46 for x in need.values())
    steps = [BATCHES, PROMPTS, OWN]
    for at in need:  # one step up in each argument is enough: the order is transitive
        for i, values in enumerate(steps):
            j = values.index(at[i]) + 1
            if j < len(values):
                up = at[:i] + (values[j],) + at[i + 1:]
                assert need[at] <= need[up], (at, up)


def test_workspace_of_any_length_of_table():
    assert SIZE(48, 28, 4, 128, 4096, (1 << 63) - 1) == SIZE(48, 28, 4, 128, 4096, 1 << 31)
