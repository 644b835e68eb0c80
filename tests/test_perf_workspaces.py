"""The measured calls of the dense block (perf/more_operators.py): a workspace for each shape and
stream, since calls that share one have to follow each other."""
import importlib

import pytest
import torch

from tests._gpu import m  # noqa: F401  (builds the library)

pytestmark = pytest.mark.gpu


def test_calls_on_two_streams_have_a_workspace_each():
    mo = importlib.import_module("perf.more_operators")
    here = lambda *shape: mo._ffn(*shape, torch.cuda.current_device(),
                                  torch.cuda.current_stream().cuda_stream)[1]
    case = dict(op="ffn", T=130, d=256, I=256, act=1, train=True, acc=True)
    states = [mo.prepare(case, i) for i in range(2)]
    want = [mo._run_own(s) for s in states]
    torch.cuda.synchronize()
    streams, got, ws = [torch.cuda.Stream() for _ in states], [], []
    for s, state in zip(streams, states):
        with torch.cuda.stream(s):
            got.append(mo._run_own(state))
            ws.append(here(130, 256, 256, 1))
            assert ws[-1] is here(130, 256, 256, 1)
    torch.cuda.synchronize()
    assert ws[0].data_ptr() != ws[1].data_ptr()
    for a, b in zip(got, want):
        assert all(torch.equal(a[k], b[k]) for k in b)
    for i in range(40):  # and it keeps no shape for good
        here(1 + i, 128, 128, 0)
    assert mo._ffn.cache_info().currsize <= 16
    mo._ffn.cache_clear()
