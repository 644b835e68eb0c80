"""The int8 operators and the dense block at the ends of the sizes they take. Zeros add exact zeros to
every sum and give exact zeros, so a few hundred columns among them have the bounds of a problem of
their own."""
import numpy as np
import pytest
import torch

from tests import _products as P64
from tests import test_gpu_ffn as G
from tests import test_gpu_int8 as I8
from tests._gpu import DEV, _announce, m
from tests.test_gpu_ffn import _float32  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("C", [2 ** 31 - 128, 2 ** 31 - 2048, 2 ** 31 - 1920, 2 ** 30])
def test_the_longest_quantised_row(C):
    """A step of the kernel's loop behind the last column is past 2^31."""
    _announce(f"[i8] a row of {C}")
    at = torch.tensor([0, 7, 2047, 2048, C // 2 + 5, C - 2049, C - 1900, C - 129, C - 1], device=DEV)
    v = torch.randn(len(at), generator=torch.Generator(DEV).manual_seed(3), device=DEV).to(BF16)
    v[-1] = 4.0  # the largest in the last column
    x = torch.zeros(1, C, dtype=BF16, device=DEV)
    x[0, at] = v
    q = torch.full((1, C), 99, dtype=torch.int8, device=DEV)
    s = torch.zeros(1, device=DEV)
    m.moe_i8_quantize_rows(x, 1, C, q, s)
    rq, rs = P64.quantize_rows(v.double().cpu().numpy()[None])
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q[0, at].cpu().numpy(), rq[0])
    q[0, at] = 0
    assert not q.any()


def _columns(n, seed):
    """About two hundred of n columns, the first and the last among them."""
    g = torch.Generator().manual_seed(seed)
    c = torch.cat([torch.arange(40), torch.randint(n, (100,), generator=g),
                   torch.arange(n // 2 - 20, n // 2 + 20), torch.arange(n - 40, n)])
    return c.unique().to(DEV)


def _place(small, rows, cols, R, C):
    big = torch.zeros(R, C, dtype=small.dtype, device=DEV)
    big[rows[:, None], cols] = small
    return big


def _take(big, rows, cols):
    """The values at rows x cols; the others are zeros."""
    small = big[rows[:, None], cols]
    big[rows[:, None], cols] = 0
    assert not big.any()
    return small


# 4 I d just below 2^31, by d and by I; a handful of tokens and more
@pytest.mark.parametrize("T,d,I", [(3, 4194176, 128), (300, 4194176, 128), (4, 128, 4194176),
                                   (33, 128, 4194176), (150, 128, 4194176)], ids=str)
def test_the_longest_rows_of_the_block(T, d, I):
    _announce(f"[ffn] {T} x {d} x {I}")
    t = torch.arange(T, device=DEV)
    cd, ci = (torch.arange(n, device=DEV) if n == 128 else _columns(n, 5) for n in (d, I))
    c2 = torch.cat([ci, I + ci])  # of [g | u]
    few = m.make_ffn(T, len(cd), len(ci), P64.SILU)
    c = m.make_ffn(T, d, I, P64.SILU)
    v = G._inputs(T, len(cd), len(ci), 31)
    where = dict(x=(t, cd, T, d), dy=(t, cd, T, d), y0=(t, cd, T, d), dx0=(t, cd, T, d),
                 w1=(c2, cd, 2 * I, d), dw10=(c2, cd, 2 * I, d), w2=(cd, ci, d, I),
                 dw20=(cd, ci, d, I))
    big = {k: _place(v[k], *w) for k, w in where.items()}
    H, A, y = G._forward(c, big, acc=True)
    dx, dw1, dw2 = G._backward(c, big, H, A, acc=True)
    Hs, As = _take(H, t, c2), _take(A, t, ci)
    G._check_forward(few, v, Hs, As, _take(y, t, cd), True)
    G._check_backward(few, v, Hs, As, _take(dx, t, cd), _take(dw1, c2, cd), _take(dw2, cd, ci), True)


# N K just below 2^31, by N and by K; few rows and many
@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("N,K", [(16776960, 128), (8388352, 256), (16128, (1 << 17) - 128)], ids=str)
@pytest.mark.parametrize("act", [None, P64.SILU])
def test_the_largest_int8_weights(M, N, K, act):
    """The last columns' bits are those of a call with the last weights alone."""
    assert N * K < 2 ** 31 and N % 256 == 0
    _announce(f"[i8] {M} rows, {N} x {K} act {act}")
    a, sa, b, sb = I8._case(M, 1, N, K, 41)
    if act is not None:
        sb[:, :N // 2] *= 3.0 / (74.0 * 74.0 * K ** 0.5)
    off = I8._offsets([M])
    out = I8._run(off, a, sa, b, sb, act)
    n = 128  # the last ones, or of both projections
    pick = lambda t: (t[:, -n:].clone() if act is None else
                      torch.cat([t[:, N // 2 - n:N // 2], t[:, -n:]], dim=1))
    last = I8._run(off, a, sa, pick(b), pick(sb), act)
    assert torch.equal(out[:, -n:], last) and torch.isfinite(out).all()
    I8._check(last, off, a, sa, pick(b), pick(sb), act)
