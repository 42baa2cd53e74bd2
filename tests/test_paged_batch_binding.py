"""Refusals of the batch operators' binding that need no GPU."""

from types import SimpleNamespace

import pytest
import torch

from test_paged_batch_args import A, vv


def test_something_else_than_a_tensor_on_a_stream_is_refused():
    stream = SimpleNamespace(device=torch.device("cuda", 0))
    i32 = torch.zeros(4, dtype=torch.int32)
    for call in (lambda x: vv.vv_paged_plan(x, i32, i32.view(4, 1), i32, 16, 8, 4, stream=stream),
                 lambda x: vv.vv_logits_process(x, stream=stream)):
        for x in (None, [1.0], i32):
            with pytest.raises(vv.VVError) as e:
                call(x)
            assert e.value.code == A
