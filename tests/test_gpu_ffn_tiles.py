"""The dense block's products in the tiles that test_gpu_ffn.py's sizes do not reach, and at the ends
of the sizes it takes. Which kernel a size takes is asked of the library's rules
(tests/_ffn_plan.py); test_products_plan_cpu.py holds that every kernel a product can take is among
the sizes of the two files."""
import pytest
import torch

from tests import _ffn_plan as F
from tests import _products as P64
from tests import test_gpu_ffn as G
from tests._gpu import DEV, _announce, m
from tests.test_gpu_ffn import _float32  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# (T, d, I), activation, and what it is here for: a product in a tile, its rows and columns ending
# within one
TILES = [
    ((1140, 1792, 2688), 0, "gate_up", F.WIDE), ((260, 128, 5504), 1, "gate_up", F.WIDE),
    ((399, 128, 4224), 2, "gate_up", F.TALL), ((516, 6784, 128), 2, "down", F.WIDE),
    ((648, 5504, 128), 3, "down", F.TALL), ((531, 384, 5504), 0, "dh", F.WIDE),
    ((526, 4736, 256), 1, "dx", F.WIDE), ((890, 3712, 2048), 2, "dx", F.TALL),
    ((259, 384, 6784), 3, "dw2", F.WIDE), ((3042, 640, 3712), 1, "dw2", F.WIDE),
]


@pytest.mark.parametrize("size,act,product,tile", TILES, ids=str)
def test_tiles_element_by_element(size, act, product, tile):
    assert F.plan(*size)[product] == tile
    G.test_large_shapes_element_by_element(*size, act)


@pytest.mark.parametrize("size,act,product,tile", TILES, ids=str)
def test_bf16_gradients_are_the_fp32_ones_rounded(size, act, product, tile):
    """The same sums (and, adding, the same total) rounded once, whichever tile stores them."""
    _announce(f"[ffn tiles] bf16 gradients of {size}")
    c, cb = m.make_ffn(*size, act), m.make_ffn(*size, act, m.MOE_FLAG_BF16_DW)
    v = G._inputs(*size, 21)
    H, A, _ = G._forward(c, v)
    for acc in (False, True):
        for a, b in zip(G._backward(c, v, H, A, acc), G._backward(cb, v, H, A, acc)):
            assert torch.equal(a.to(BF16), b), acc


def _spread(small, rows, T):
    """`small`'s rows at `rows` of T rows of zeros."""
    big = torch.zeros(T, small.shape[1], dtype=small.dtype, device=DEV)
    big[rows] = small
    return big


def _rest_is_zero(big, rows):
    big[rows] = 0
    return not big.any()


@pytest.mark.parametrize("d,I", [(256, 128), (128, 128)], ids=str)
def test_the_most_tokens(d, I):
    """(T + 64) max(d, 2I) just below 2^31: rows whose bytes lie past 2^31 and up to 2^32, behind a
    token's row and (in the weight gradients) a step of K. Tokens of zeros add exact zeros to every
    sum, so a few thousand others have the bounds of a batch of their own."""
    T = (2 ** 31 - 1) // max(d, 2 * I) - 64
    _announce(f"[ffn] {T} x {d} x {I}")
    half = T // 2  # of both kinds of rows, byte 2^31 lies here
    rows = torch.cat([torch.arange(0, 70), torch.arange(half - 150, half + 150),
                      torch.arange(T - 201, T)]).to(DEV)
    n = len(rows)
    c, few = m.make_ffn(T, d, I, P64.SILU), m.make_ffn(n, d, I, P64.SILU)
    v = G._inputs(n, d, I, 23)
    big = {k: _spread(t, rows, T) if k in ("x", "dy", "y0", "dx0") else t for k, t in v.items()}
    H, A, y = G._forward(c, big, acc=True)
    dx, dw1, dw2 = G._backward(c, big, H, A, acc=True)
    del big
    Hs, As, ys, dxs = (t[rows] for t in (H, A, y, dx))
    for t in (H, A, y, dx):
        assert _rest_is_zero(t, rows)
    G._check_forward(few, v, Hs, As, ys, True)
    G._check_backward(few, v, Hs, As, dxs, dw1, dw2, True)


def test_the_largest_weights():
    """4 I d just below 2^31, for a handful of tokens."""
    G.test_large_shapes_element_by_element(5, 16384, 32640, P64.GELU)
