"""Workspaces of calls on a stream of the caller's belong to that stream, whatever object names it."""
import pytest
import torch

import exact_headdim_attention_gb300 as pkg
from tests.gpu_util import device_ok
from tests.test_gpu_paged import close, decode_case, to_dev
from tests.test_gpu_rope import make

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


class Handle:
    """Another library's stream object."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


def allocated_on(stream):
    return [s for s in torch.cuda.memory_snapshot() if s["stream"] == stream.cuda_stream]


@pytest.mark.parametrize("wrap", [lambda s: s, Handle])
def test_workspaces_belong_to_the_callers_stream(wrap):
    args, ref = decode_case([3000, 1, 0, 800], 8, 2, 256, 16, BF, seed=18)
    q, k, pos, inv, qw, kw, (gq, gk) = make(40, 4, 2, 128, 128, BF, torch.float32)
    rows, grads = to_dev(q, k, pos, inv, qw, kw), to_dev(gq, gk)
    want = pkg.ffpa_qk_norm_rope_bwd(*grads, *rows)
    for call, check in ((lambda s: pkg.ffpa_decode_paged(*args, enable_gqa=True, stream=s), lambda o: close(o, ref[0], ref[2], "O")),
                        (lambda s: pkg.ffpa_qk_norm_rope_bwd(*grads, *rows, stream=s),
                         lambda o: all(torch.equal(a, b) for a, b in zip(o, want)) or pytest.fail("gradients differ"))):
        torch.cuda.empty_cache()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        assert not allocated_on(side)
        out = call(wrap(side))
        assert allocated_on(side)
        side.synchronize()
        check(out)
    device_ok()
