"""The int8 quantiser and products on the GPU against 64-bit plain forms (tests/_products.py). Codes
and scales must be equal. A product's sum is exact; its value takes three fp32 roundings (the sum to
fp32, two scales) and half a step of bf16."""
import numpy as np
import pytest
import torch

from tests import _products as P64
from tests._gpu import DEV, _announce, m

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _float32():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


def _quant(x):
    R, C = x.shape
    q = torch.full((R, C), 99, dtype=torch.int8, device=DEV)
    s = torch.full((R,), -7.0, device=DEV)
    m.moe_i8_quantize_rows(x, R, C, q, s)
    return q, s


def _same_rows(x):
    q, s = _quant(x.to(DEV))
    rq, rs = P64.quantize_rows(x.double().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("R,C", [(1, 128), (3, 384), (65, 512), (7, 640), (130, 1024), (5, 1152),
                                 (33, 2048), (257, 2176), (9, 4096), (6, 4224), (24, 7168),
                                 (3, 8192), (2, 8320), (2, 16384), (3, 16512), (1, 40960)])
def test_rows_are_quantised_exactly(R, C):
    _announce(f"[i8] rows {R} x {C}")
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C, generator=g) * 2.0 ** torch.randint(-10, 10, (R, C), generator=g)
    if R > 2:
        x[1] = 0.0
        x[2, C // 2:] *= 1e30
    x[0, -1] = -x[0].abs().max() * 1.5  # the largest in the last column
    _same_rows(x.to(BF16))


def test_ties_and_tiny_rows():
    """Every mantissa against every amax mantissa's neighbours of a tie; rows down to bf16's
    smallest, and up to its largest."""
    rows = []
    for b in (128, 129, 131, 170, 200, 254, 255):
        v = torch.tensor([a * 2.0 ** -s for s in range(9) for a in range(128, b + 1 if s == 0 else 256)])
        row = torch.zeros(2304)
        row[:v.numel()] = v * (1 - 2 * (torch.arange(v.numel()) % 2))
        row[-1] = b
        for e in (-140, -126, -118, -117, -116, -100, 0, 100, 119):
            rows.append((row.double() * 2.0 ** e).to(BF16))
    x = torch.stack(rows)
    assert torch.isfinite(x).all()
    _same_rows(x)


@pytest.mark.parametrize("C", [256, 4096, 7168, 16512])
def test_rows_with_values_that_are_not_finite(C):
    x = torch.randn(12, C, generator=torch.Generator().manual_seed(C)).to(BF16)
    for r, (c, v) in {1: (0, np.inf), 4: (C - 1, -np.inf), 7: (C // 2, np.nan)}.items():
        x[r, c] = v
    x.view(torch.int16)[9, 3] = -1  # a NaN of all ones
    _same_rows(x)


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32,
                        device=DEV)


def _case(M, E, N, K, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    a = torch.randint(-128, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
    b = torch.randint(-128, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    return a, torch.rand(M, generator=g, device=DEV) + 0.1, b, \
        torch.rand(E, N, generator=g, device=DEV) + 0.1


def _check(out, off, a, sa, b, sb, act=None):
    M = a.shape[0]
    v = P64.i8_product(off.cpu().numpy(), a.cpu().numpy(), sa.cpu().numpy(), b.cpu().numpy(),
                       sb.cpu().numpy(), M)
    e = 3 * P64.F32 * np.abs(v)
    if act is not None:
        (g, u), (eg, eu) = np.split(v, 2, axis=1), np.split(e, 2, axis=1)
        v, e = P64.act(act, g) * u, P64.gated_error(g, u, eg, eu)
    got = out.double().cpu().numpy()
    there = ~np.isnan(v).any(axis=1)
    tol = P64.BF16 * (np.abs(v) + e) + e
    np.testing.assert_array_less(np.abs(got - v)[there], tol[there] + 1e-37)
    assert (got[~there] == 77.0).all()  # rows of no expert stay


def _run(off, a, sa, b, sb, act=None):
    M, K = a.shape
    E, N = b.shape[:2]
    if act is None:
        out = torch.full((M, N), 77.0, dtype=BF16, device=DEV)
        m.moe_i8_gemm(off, M, E, N, K, a, sa, b, sb, out)
    else:
        out = torch.full((M, N // 2), 77.0, dtype=BF16, device=DEV)
        m.moe_i8_gemm_gated(off, M, E, N // 2, K, act, a, sa, b, sb, out)
    return out


LOADS = [
    ([1], 0, 0, 128, 128), ([5], 0, 0, 256, 384), ([16], 0, 3, 384, 256), ([17], 2, 0, 128, 1152),
    ([31, 0, 2], 0, 1, 256, 256), ([0, 0, 40], 0, 0, 128, 640), ([63, 64, 65], 1, 2, 256, 128),
    ([100, 0, 129, 7], 0, 5, 384, 256), ([256], 0, 0, 512, 256), ([257, 3], 0, 4, 256, 384),
    ([300, 700, 0, 1], 5, 9, 640, 128), ([1025], 0, 0, 256, 512), ([0, 0], 0, 3, 128, 128),
    ([2] * 40, 0, 0, 256, 256), ([1, 0, 0, 9] * 16, 0, 1, 128, 128),
]


@pytest.mark.parametrize("counts,first,tail,N,K", LOADS, ids=str)
@pytest.mark.parametrize("act", [None, *P64.ACTS])
def test_products(counts, first, tail, N, K, act):
    E, M = len(counts), first + sum(counts) + tail
    _announce(f"[i8] product {counts} +{first} +{tail} {N} x {K} act {act}")
    if act is not None:
        N *= 2  # I = N / 2 is a multiple of 128 too
    a, sa, b, sb = _case(M, E, N, K, N + K + M)
    if act is not None:  # gates of a size at which every activation bends
        sb[:, :N // 2] *= 3.0 / (74.0 * 74.0 * K ** 0.5)
    off = _offsets(counts, first)
    _check(_run(off, a, sa, b, sb, act), off, a, sa, b, sb, act)


# whole rounds of 256 x 256 tiles, and a last one uncut, in halves and in quarters; an even and an odd
# number of steps of K
@pytest.mark.parametrize("N", [3584, 4352, 4480, 4608])
@pytest.mark.parametrize("K", [256, 384, 1024])
@pytest.mark.parametrize("act", [None, P64.SILU, P64.GELU])
def test_many_rows_an_expert(N, K, act):
    counts, first, tail = [2100, 0, 3000, 5], 3, 9
    _announce(f"[i8] {counts} rows, {N} x {K} act {act}")
    E, M = len(counts), first + sum(counts) + tail
    N = N if act is None else N // 256 * 256
    a, sa, b, sb = _case(M, E, N, K, N + K)
    if act is not None:
        sb[:, :N // 2] *= 3.0 / (74.0 * 74.0 * K ** 0.5)
    off = _offsets(counts, first)
    out = _run(off, a, sa, b, sb, act)
    at = off.tolist()
    assert (out[:first] == 77).all() and (out[at[-1]:] == 77).all()
    for e in range(E):
        lo, hi = at[e], at[e + 1]
        # the sums are whole numbers below 2^53
        v = a[lo:hi].double() @ b[e].double().t().contiguous()
        v = v * sa[lo:hi, None].double() * sb[e].double()
        err = 3 * P64.F32 * v.abs()
        if act is not None:
            (g, u), (eg, eu) = v.split(N // 2, dim=1), err.split(N // 2, dim=1)
            F = torch.nn.functional
            v = (F.silu(g) if act == P64.SILU else F.gelu(g)) * u
            err = (1.2 * eg * u.abs() + g.abs() * eu + 1.2 * eg * eu
                   + P64.F32 * (24 + 8 * g.abs()) * (g * u).abs())  # P64.gated_error
        tol = P64.BF16 * (v.abs() + err) + err + 1e-37
        assert ((out[lo:hi].double() - v).abs() <= tol).all()


# a handful of experts and rows (every CU at the weights), and the two streaming tiles
@pytest.mark.parametrize("counts,N", [([1], 1024), ([16], 8192), ([9, 5], 4096), ([31], 2048),
                                      ([20, 33, 2], 1024), ([64], 8192), ([40], 128),
                                      ([16] * 18, 4096), ([3, 0, 14] * 7, 4096),
                                      ([100, 60, 128, 96] * 3, 1024)], ids=str)
@pytest.mark.parametrize("K", [128, 2048, 3968, 7168])
@pytest.mark.parametrize("act", [None, P64.GELU_TANH])
def test_few_rows_an_expert(counts, N, K, act):
    E, M = len(counts), sum(counts)
    if E * N * K > 3e8:
        K = 640
    if act is not None:
        N = max(N, 256)  # I = N / 2 is a multiple of 128 too
    _announce(f"[i8] {counts} rows, {N} x {K} act {act}")
    a, sa, b, sb = _case(M, E, N, K, N + K + E)
    if act is not None:
        sb[:, :N // 2] *= 3.0 / (74.0 * 74.0 * K ** 0.5)
    off = _offsets(counts)
    out = _run(off, a, sa, b, sb, act)
    at = off.tolist()
    for e in range(E):
        lo, hi = at[e], at[e + 1]
        v = a[lo:hi].double() @ b[e].double().t().contiguous()
        v = v * sa[lo:hi, None].double() * sb[e].double()
        err = 3 * P64.F32 * v.abs()
        if act is not None:
            (g, u), (eg, eu) = v.split(N // 2, dim=1), err.split(N // 2, dim=1)
            v = torch.nn.functional.gelu(g, approximate="tanh") * u
            err = (1.2 * eg * u.abs() + g.abs() * eu + 1.2 * eg * eu
                   + P64.F32 * (24 + 8 * g.abs()) * (g * u).abs())  # P64.gated_error
        tol = P64.BF16 * (v.abs() + err) + err + 1e-37
        assert ((out[lo:hi].double() - v).abs() <= tol).all()


# quarters of 256 x 256 tiles that fill the card just once: 192, 224 and 256 tiles of 128 rows of weights
@pytest.mark.parametrize("counts,N", [([70, 0, 120, 3, 200, 7], 4096), ([33] * 7, 4096),
                                      ([0, 300, 1, 128], 7168), ([50, 40, 0, 60, 35, 45, 129, 1], 4096)],
                         ids=str)
@pytest.mark.parametrize("K", [128, 256, 1664])
@pytest.mark.parametrize("act", [None, P64.GELU_TANH])
def test_few_large_tiles(counts, N, K, act):
    test_few_rows_an_expert(counts, N, K, act)


def test_sums_reach_the_ends_of_32_bits():
    K = (1 << 17) - 128
    a = torch.full((3, K), -128, dtype=torch.int8, device=DEV)
    a[1] = 127
    a[2, ::2] = 127
    b = torch.full((1, 128, K), -128, dtype=torch.int8, device=DEV)
    b[0, 1::2] = 127
    sa, sb = torch.ones(3, device=DEV), torch.ones(1, 128, device=DEV)
    off = _offsets([3])
    _check(_run(off, a, sa, b, sb), off, a, sa, b, sb)


def test_results_do_not_depend_on_the_batch():
    """A row's bits alone, in small batches and in large ones, and behind other experts."""
    K, N = 512, 768
    a, sa, b, sb = _case(1500, 2, N, K, 5)
    for act in (None, P64.SILU):
        sb2 = sb if act is None else sb * 1e-4
        whole = _run(_offsets([1500, 0]), a, sa, b, sb2, act)
        for n in (1, 7, 30, 60, 100, 250, 700):
            part = _run(_offsets([n, 0]), a[:n].contiguous(), sa[:n].contiguous(), b, sb2, act)
            assert torch.equal(part, whole[:n]), n


def test_offsets_outside_are_clamped():
    a, sa, b, sb = _case(40, 3, 256, 256, 9)
    off = torch.tensor([-5, 20, 30, 90], dtype=torch.int32, device=DEV)
    for act in (None, P64.RELU):
        sb2 = sb if act is None else sb * 1e-4
        _check(_run(off, a, sa, b, sb2, act), off, a, sa, b, sb2, act)


def test_scales_that_are_not_finite_stay_in_their_row_and_channel():
    a, sa, b, sb = _case(70, 2, 256, 256, 11)
    off = _offsets([30, 40])
    clean = _run(off, a, sa, b, sb)
    sa[3], sb[1, 130] = float("nan"), float("nan")
    out = _run(off, a, sa, b, sb)
    hit = torch.zeros(70, 256, dtype=torch.bool, device=DEV)
    hit[3] = True
    hit[30:, 130] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


def test_scales_and_offsets_at_any_multiple_of_four_bytes():
    a, sa, b, sb = _case(50, 1, 256, 256, 13)
    want = _run(_offsets([50]), a, sa, b, sb)
    shift = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)
    off = torch.cat([torch.zeros(1, dtype=torch.int32, device=DEV), _offsets([50])])[1:]
    assert torch.equal(_run(off, a, shift(sa), b, shift(sb)), want)


def test_offsets_past_32_bits():
    """More than 2^31 codes of rows, and of weights, against the last ones in a call of their own."""
    R, C, N = 310_000, 7168, 128
    _announce(f"[i8] {R} x {C} rows quantised and multiplied")
    g = torch.Generator(DEV).manual_seed(0)
    x = torch.randn(R, C, device=DEV, generator=g, dtype=BF16)
    q, s = _quant(x)
    q1, s1 = _quant(x[-40:].clone())
    del x
    assert torch.equal(q[-40:], q1) and torch.equal(s[-40:], s1)
    b = torch.randint(-128, 128, (1, N, C), device=DEV, generator=g, dtype=torch.int8)
    sb = torch.rand(1, N, device=DEV, generator=g)
    out = _run(_offsets([R]), q, s, b, sb)
    assert torch.equal(out[-40:], _run(_offsets([40]), q1, s1, b, sb))
    del q, out
    E = 2400
    with pytest.raises(m.MoeError):
        _run(_offsets([1] * E), q1, s1, b.expand(E, -1, -1), sb.expand(E, -1))
    E, N = 900, 384
    b = torch.randint(-128, 128, (E, N, C), device=DEV, generator=g, dtype=torch.int8)
    sb = torch.rand(E, N, device=DEV, generator=g)
    assert b.numel() > 2 ** 31
    out = _run(_offsets([0] * (E - 1) + [40]), q1, s1, b, sb)
    assert torch.equal(out, _run(_offsets([40]), q1, s1, b[-1:].clone(), sb[-1:].clone()))


def test_captured_and_on_another_stream():
    a, sa, b, sb = _case(300, 3, 256, 512, 17)
    off = _offsets([100, 0, 200])
    x = torch.randn(300, 512, device=DEV).to(BF16)
    want, wq = _run(off, a, sa, b, sb), _quant(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty(300, 256, dtype=BF16, device=DEV)
    m.moe_i8_gemm(off, 300, 3, 256, 512, a, sa, b, sb, out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    q, s = torch.empty_like(wq[0]), torch.empty_like(wq[1])
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        m.moe_i8_quantize_rows(x, 300, 512, q, s)
        m.moe_i8_gemm(off, 300, 3, 256, 512, q, s, b, sb, out)
    for i in range(3):
        out.zero_()
        q.zero_()
        x.copy_(x.roll(i, 0))
        g.replay()
        torch.cuda.synchronize()
        eq = _quant(x)
        assert torch.equal(q, eq[0]) and torch.equal(s, eq[1])
        assert torch.equal(out, _run(off, eq[0], eq[1], b, sb))


def test_tensors_the_binding_refuses():
    a, sa, b, sb = _case(20, 1, 128, 128, 3)
    off = _offsets([20])
    out = torch.zeros(20, 128, dtype=BF16, device=DEV)
    good = [off, 20, 1, 128, 128, a, sa, b, sb, out]
    for at, bad in ((0, off.long()), (5, a.view(torch.uint8)), (5, a.cpu()), (5, a[:19]),
                    (6, sa.half()), (7, b.transpose(1, 2)), (8, sb.double()), (9, out.float()),
                    (9, out[:, ::2])):
        args = list(good)
        args[at] = bad
        with pytest.raises(m.MoeError):
            m.moe_i8_gemm(*args)
    assert (out == 0).all()
