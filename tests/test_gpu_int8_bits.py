"""A row's bits in the int8 products, whichever kernel takes it: one expert's weights, given to every
expert, and rows of one batch in calls of other sizes. The kernels differ in tiles, in how they hold
the sums and in where they apply scales and gate; results must not. (test_gpu_int8.py compares each
with the 64-bit form.)"""
import pytest
import torch

from tests import _products as P64
from tests._gpu import DEV, _announce
from tests.test_gpu_int8 import _float32, _offsets, _run  # noqa: F401  (the fixture too)

pytestmark = pytest.mark.gpu

N = 4096  # 32 tiles of 128 weights an expert
MOST = 4200
# One expert, by rows: whole rounds of large tiles and a last one in quarters (4200), one uncut
# (2500), in halves (1500), in quarters (1000); 128-row streaming of 8 and 6 blocks (100, 80); every CU at
# the weights, 2 x 2 blocks (64, 40), 2 x 1 (32, 20) and one (16, 5, 1).
ONE = (2500, 1500, 1000, 100, 80, 64, 40, 32, 20, 16, 5, 1)
# Several, rows each: 128-row streaming of 2 and of 4 blocks, halves of large tiles that fill the card
# once (7 experts), 32-row streaming (20 experts: 640 tiles).
MANY = ([20, 3, 31, 10], [60, 33, 64, 47], [70, 0, 45, 129, 33, 60, 1], [16] * 20, [9, 16, 12, 16, 14] * 4)


@pytest.mark.parametrize("K", [512, 640])  # an even and an odd number of steps: tiles that flow or not
@pytest.mark.parametrize("act", [None, *P64.ACTS])
def test_bits_do_not_depend_on_the_kernel(K, act):
    g = torch.Generator(DEV).manual_seed(K)
    a = torch.randint(-128, 128, (MOST, K), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(-128, 128, (1, N, K), generator=g, device=DEV, dtype=torch.int8)
    sa = torch.rand(MOST, generator=g, device=DEV) + 0.1
    sb = torch.rand(1, N, generator=g, device=DEV) + 0.1
    if act is not None:  # gates of a size at which every activation bends
        sb[:, :N // 2] *= 3.0 / (74.0 * 74.0 * K ** 0.5)
    whole = _run(_offsets([MOST]), a, sa, b, sb, act)
    for n in ONE:
        _announce(f"[i8 bits] K {K} act {act}: {n} rows")
        part = _run(_offsets([n]), a[:n].contiguous(), sa[:n].contiguous(), b, sb, act)
        assert torch.equal(part, whole[:n]), n
    for counts in MANY:
        _announce(f"[i8 bits] K {K} act {act}: {counts}")
        E, M = len(counts), sum(counts)
        part = _run(_offsets(counts), a[:M].contiguous(), sa[:M].contiguous(),
                    b.expand(E, -1, -1).contiguous(), sb.expand(E, -1).contiguous(), act)
        assert torch.equal(part, whole[:M]), counts
