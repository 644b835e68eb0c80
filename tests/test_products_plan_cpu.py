"""The dense block's choice of kernels (csrc/ffn_plan.h), asked without a GPU: the sizes of the GPU
tests reach every kernel that any size does."""
import math
import random

from tests import _ffn_plan as F
from tests import test_gpu_ffn as G
from tests import test_gpu_ffn_tiles as GT


def _params(test):
    out = [()]
    for mark in reversed(test.pytestmark):
        if mark.name == "parametrize":
            rows = [r if isinstance(r, tuple) else (r,) for r in mark.args[1]]
            out = [{**dict(o), **dict(zip(mark.args[0].split(","), r))} for o in out for r in rows]
    return out


def _sizes():
    """The sizes of the tests that look at every element."""
    out = [(p["T"], p["d"], p["I"]) for t in (G.test_forward, G.test_backward, G.test_few_tokens,
                                              G.test_large_shapes_element_by_element)
           for p in _params(t)]
    return out + [size for size, *_ in GT.TILES]


def test_every_kernel_that_a_size_takes_is_tested():
    rng = random.Random(0)
    draw = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    reached, tested = set(), set()
    for _ in range(40000):
        reached |= set(F.plan(draw(1, 20000), 128 * draw(1, 64), 128 * draw(1, 64)).items())
    for size in _sizes():
        tested |= set(F.plan(*size).items())
    assert reached <= tested, reached - tested
    # and that is nearly all there are: the rows of dW1, 2I, are whole 256s, so that 256 x 128 tiles
    # are never more than 128 x 256 ones
    every = {(p, k) for p in F.PRODUCTS for k in range(5)}
    assert every - reached == {("dw1", F.WIDE)}


def test_tiles_end_within_rows_and_columns():
    ends = {(p, t): False for p in F.PRODUCTS for t in (F.TALL, F.WIDE)}
    for T, d, I in _sizes():
        m = dict(gate_up=T, down=T, dh=T, dx=T, dw2=d, dw1=2 * I)
        n = dict(gate_up=2 * I, down=d, dh=I, dx=d, dw2=I, dw1=d)
        for p, t in F.plan(T, d, I).items():
            if t == F.TALL:
                ends[p, t] |= m[p] % 256 != 0
            elif t == F.WIDE:
                ends[p, t] |= n[p] % 256 != 0 and m[p] % 128 != 0
    # the rows of dW1 and the columns of [g | u] are whole 256s; dW2's rows whole 128s
    never = {("dw1", F.TALL), ("dw1", F.WIDE), ("gate_up", F.WIDE), ("dw2", F.WIDE)}
    assert {k for k, v in ends.items() if not v} == never
