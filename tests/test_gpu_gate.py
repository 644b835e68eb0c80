"""The gate and the router gradients on the GPU against 64-bit plain forms (tests/_ops.py).

The choice must be equal, expert for expert. Tolerances count roundings: u = 2^-24 is half an
fp32 step, the device's expf is within one step (2 u), 2^-8 is half a bf16 step.
"""
import itertools
import math

import numpy as np
import pytest
import torch

from tests import _ops
from tests._gpu import DEV, _announce, m

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
inf = math.inf


@pytest.fixture(autouse=True)
def _float32():
    """The inputs below are fp32 where no type is named, whatever another test file set."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)



def _logits(T, E, seed, closed=0.0, ties=False):
    rng = np.random.default_rng(seed)
    l = rng.normal(scale=1.7, size=(T, E)).astype(np.float32)
    if ties:  # few distinct values: nearly every choice is between equals
        l = np.round(l).astype(np.float32)
    if closed:
        l[rng.random((T, E)) < closed] = -inf
    return l


def _select(l, k, gate, bias=None):
    T, E = l.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    b = None if bias is None else torch.tensor(bias, dtype=torch.float32, device=DEV)
    m.moe_gate_select(m.make_cfg(T, 256, E, k, 128), gate, torch.tensor(l, device=DEV), b, idx, w)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy()


def _check_select(l, k, score, bias=None, groups=1, topk_groups=1, group_score=0, renorm=True,
                  scale=1.0):
    g = m.make_gate(score, groups, topk_groups, group_score, renorm, scale)
    idx, w = _select(l, k, g, bias)
    ridx, rw = _ops.gate(l, k, score, bias, groups, topk_groups, group_score, renorm,
                         float(np.float32(scale)))
    np.testing.assert_array_equal(idx, ridx)
    # one rounding of a 64-bit value to fp32
    assert np.all(np.abs(w - rw) <= U * 1.0001 * np.abs(rw) + 2.0 ** -149)


SIZES = [(1, 1, 1), (1, 256, 8), (3, 3, 2), (7, 64, 64), (5, 65, 8), (70, 100, 7), (33, 256, 8),
         (9, 257, 16), (20, 509, 10), (6, 1000, 64), (4, 1024, 40)]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choice_and_weights_without_groups(T, E, k, score):
    _announce(f"[gate] T={T} E={E} k={k} score={score}")
    bias = np.random.default_rng(E).normal(scale=0.05, size=E).astype(np.float32)
    for b, renorm, (closed, ties) in itertools.product(
            (None, bias), (False, True), ((0, False), (0.3, False), (0.1, True))):
        _check_select(_logits(T, E, T + E, closed, ties), k, score, b, renorm=renorm, scale=2.5)


GROUPS = [(256, 8, 4, 8), (256, 8, 1, 8), (256, 8, 8, 8), (64, 64, 9, 8), (96, 3, 2, 6),
          (1024, 2, 1, 10), (1024, 512, 100, 12), (130, 65, 33, 20), (1022, 511, 3, 6),
          (6, 2, 1, 3), (40, 4, 3, 1), (768, 12, 5, 33), (1024, 1024, 50, 40)]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E,G,tg,k", GROUPS)
def test_choice_with_groups(E, G, tg, k, score):
    _announce(f"[gate] E={E} groups={G} topk_groups={tg} k={k} score={score}")
    bias = np.random.default_rng(G).normal(scale=0.05, size=E).astype(np.float32)
    for b, gsc, (closed, ties) in itertools.product(
            (None, bias), (0, 1), ((0, False), (0.5, False), (0.2, True))):
        _check_select(_logits(17, E, E + G, closed, ties), k, score, b, G, tg, gsc, True, 1.0)


@pytest.mark.parametrize("score", [0, 1])
def test_closed_rows_nan_and_infinities(score):
    _announce(f"[gate] closed rows, NaN, infinities, score={score}")
    l = _logits(12, 96, 5)
    l[0] = -inf                    # nothing open
    l[1, 1:] = -inf                # one open expert
    l[2, ::2] = np.nan             # NaN closes
    l[3] = np.nan
    l[4, 10:60] = -np.finfo(np.float32).max  # masked with the type's lowest value
    l[5] = -np.finfo(np.float32).max
    l[6, 7] = np.finfo(np.float32).max
    l[7, [3, 50]] = inf            # two share the row
    l[8] = 0.0
    l[8, 40] = -0.0                # equal to 0: index order
    l[9] = 60.0 + np.arange(96, dtype=np.float32)  # sigmoids that are 1 in 64 bits: by logit
    l[10] = -200.0 - np.arange(96, dtype=np.float32)[::-1]
    for renorm, (G, tg, gsc) in itertools.product(
            (False, True), ((1, 1, 0), (8, 3, 0), (8, 3, 1), (96, 20, 1))):
        rows = l if not (score == 1 and gsc == 1) else np.delete(l, [9], axis=0)
        _check_select(rows, 8, score, None, G, tg, gsc, renorm, 1.0)
    bias = np.linspace(0.2, -0.2, 96).astype(np.float32)
    _check_select(l, 8, score, bias, 8, 3, 1, True, 1.0)


def test_choice_between_scores_that_fp32_cannot_tell_apart():
    """Two experts whose choice scores differ by less than an fp32 step of them."""
    l = np.zeros((64, 32), np.float32)
    rng = np.random.default_rng(0)
    bias = np.full(32, -1.0, np.float32)
    a = rng.permuted(np.tile(np.arange(32), (64, 1)), axis=1)[:, :2]
    bias[:] = np.float32(0.75)
    for t in range(64):
        l[t] = -9.0
        l[t, a[t, 0]] = 12.0
        l[t, a[t, 1]] = np.nextafter(np.float32(12.0), np.float32(13.0))
    _check_select(l, 2, 1, bias)


def test_a_row_does_not_depend_on_its_batch():
    _announce("[gate] T=5000 against its rows one at a time")
    l = _logits(5000, 256, 9)
    g = m.make_gate(1, 8, 4, 1, True, 2.5)
    b = np.random.default_rng(1).normal(scale=0.05, size=256).astype(np.float32)
    idx, w = _select(l, 8, g, b)
    for t in (0, 1, 77, 2048, 4999):
        i1, w1 = _select(l[t:t + 1], 8, g, b)
        np.testing.assert_array_equal(i1[0], idx[t])
        np.testing.assert_array_equal(w1[0], w[t])


def _grad_bound(l, idx, dw, score, renorm, scale):
    """Roundings of moe_gate_backward's fp32 steps, per logit, times u (see the comments)."""
    T, E = l.shape
    k = idx.shape[1]
    s = _ops.scores(l, score)
    ok = (idx >= 0) & (idx < E)
    p = np.where(ok, np.take_along_axis(s, np.where(ok, idx, 0), 1), 0.0)
    g = np.where(ok, np.abs(scale * np.asarray(dw, np.float64)), 0.0)
    ga = np.zeros((T, E))
    for t, j in itertools.product(range(T), range(k)):
        if ok[t, j]:
            ga[t, idx[t, j]] += g[t, j]
    fin = np.where(np.isfinite(l), l, 0.0)
    A = np.abs(fin).max() * 2  # the largest |l - max|: each exp carries |l - max| u more
    if score == 1 and not renorm:
        return s * (1 - s) * ga * (12 + k)  # s, 1 - s: 4 each; the products and slots' sums
    S = p.sum(1, keepdims=True)
    if score == 1:
        # s 4, S 10, q 15, sum of g q 23, difference and division 12, s (1 - s) 10, slots k
        return np.divide(s * (1 - s) * (ga + (g * p).sum(1, keepdims=True) / np.where(S > 0, S, 1)),
                         np.where(S > 0, S, 1)) * (48 + k)
    if renorm:
        q = np.divide(s, np.where(S > 0, S, 1))
        gq = (g * p).sum(1, keepdims=True) / np.where(S > 0, S, 1)
        # and the reference's own sum, whose terms cancel only to 2^-52 of them off the choice
        ref64 = s * 2 * gq * (k + 8) * 2.0 ** -52
        return q * (ga + gq * (ga > 0) * k) * (4 * A + 36 + k) + ref64 / U
    # p: 2 A + E / 64 + 12; the sum of p g 8 more; the last product 2; slots k
    return s * (ga + (g * p).sum(1, keepdims=True)) * (4 * A + E / 32 + 34 + k)


@pytest.mark.parametrize("score,renorm", [(0, True), (0, False), (1, True), (1, False)])
@pytest.mark.parametrize("T,E,k", SIZES)
def test_gate_gradient(T, E, k, score, renorm):
    _announce(f"[gate bwd] T={T} E={E} k={k} score={score} renorm={renorm}")
    rng = np.random.default_rng(T * 3 + E)
    for closed in (0.0, 0.2):
        l = _logits(T, E, T + E, closed)
        idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        if k > 1:
            idx[0, 1] = idx[0, 0]    # one expert twice
        if T > 2:
            idx[1, k - 1] = -1       # slots that name none
            idx[2, 0] = E
        dw = rng.normal(size=(T, k)).astype(np.float32)
        ref = _ops.gate_backward(l, idx, dw, score, renorm, 2.5)
        tol = _grad_bound(l, idx, dw, score, renorm, 2.5) * U + 1e-37
        cfg, g = m.make_cfg(T, 256, E, k, 128), m.make_gate(score, 1, 1, 0, renorm, 2.5)
        args = [torch.tensor(v, device=DEV) for v in (l, idx, dw)]
        dl = torch.full((T, E), -7.0, device=DEV)
        m.moe_gate_backward(cfg, g, *args, dl, False)
        got = dl.cpu().numpy()
        worst = float(np.max(np.abs(got - ref) / tol))
        assert worst <= 1, worst
        # added to what is there: one rounding of the sum more
        base = torch.randn(T, E, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
        acc = base.clone()
        m.moe_gate_backward(cfg, g, *args, acc, True)
        assert torch.equal(acc, base + dl)


@pytest.mark.parametrize("shift", [-80.0, -95.0, -300.0, -600.0])
def test_gradient_of_scores_below_fp32(shift):
    """Every logit of a row far down: the sigmoids leave fp32, their shares of the sum do not."""
    T, E, k = 40, 24, 6
    _announce(f"[gate bwd] logits about {shift}")
    l = (_logits(T, E, 11) + np.float32(shift)).astype(np.float32)
    gate = m.make_gate(m.MOE_SCORE_SIGMOID, 1, 1, 0, True, 2.5)
    idx, w = _select(l, k, gate)
    assert np.all(np.abs(w.sum(1) - 2.5) < 1e-5)
    dw = np.random.default_rng(12).normal(size=(T, k)).astype(np.float32)
    dl = torch.full((T, E), -7.0, device=DEV)
    m.moe_gate_backward(m.make_cfg(T, 256, E, k, 128), gate,
                        *[torch.tensor(v, device=DEV) for v in (l, idx, dw)], dl, False)
    ref = _ops.gate_backward(l, idx, dw, 1, True, 2.5)
    tol = _grad_bound(l, idx, dw, 1, True, 2.5) * U + 1e-37
    assert np.all(np.abs(dl.cpu().numpy() - ref) <= tol)


ROUTER = [(1, 256, 1), (1, 256, 256), (5, 512, 3), (64, 256, 8), (127, 256, 129), (128, 512, 128),
          (200, 768, 509), (1000, 256, 64), (333, 1024, 1024),
          # few tiles of dWr and many tokens, on each side of the choices between its kernels
          (1023, 512, 37), (1024, 512, 37), (1025, 256, 1), (1500, 2048, 16), (1611, 2048, 130),
          (2047, 4096, 101), (2048, 4096, 101), (2500, 4352, 70), (5000, 256, 300)]


@pytest.mark.parametrize("T,d,E", ROUTER)
def test_router_gradients(T, d, E):
    _announce(f"[router bwd] T={T} d={d} E={E}")
    g = torch.Generator().manual_seed(T + d + E)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16)
    wr = (0.02 * torch.randn(E, d, generator=g)).to(torch.bfloat16)
    # magnitudes over several binades, and whole rows without a gradient
    dl = torch.randn(T, E, generator=g) * 2.0 ** torch.randint(-12, 4, (T, E), generator=g)
    if T > 2:
        dl[1] = 0.0
    dx0 = torch.randn(T, d, generator=g).to(torch.bfloat16)
    dw0 = torch.randn(E, d, generator=g)
    cfg = m.make_cfg(T, d, E, 1, 128)
    X, W, D = x.to(DEV), wr.to(DEV), dl.to(DEV)
    x64, w64, d64 = x.double(), wr.double(), dl.double()
    # fp32 sums of three exact products a term: an fp32 step (2^-23) for each addition
    # dx sums two products a term, of dl as two bf16 parts p + q: of a value in [1, 2) p = bf16(v)
    # leaves at most 2^-8, which lies in a binade with bf16 half steps of 2^-17 or less, so q leaves
    # 2^-17 of v. (3 E + 4 steps alone are less than that one error, 64 steps, up to E = 19.)
    e_dx = ((3 * E + 4) * 2.0 ** -23 + 2.0 ** -17) * (d64.abs() @ w64.abs())
    e_dw = (3 * T + 4) * 2.0 ** -23 * (d64.abs().t() @ x64.abs())
    for acc in (False, True):
        dx, dw = dx0.clone().to(DEV), dw0.clone().to(DEV)
        m.moe_router_backward(cfg, X, W, D, dx, dw, acc, acc)
        rx, rw = d64 @ w64, d64.t() @ x64
        if acc:
            rx, rw = rx + dx0.double(), rw + dw0.double()
        ex = (dx.cpu().double() - rx).abs()
        ew = (dw.cpu().double() - rw).abs()
        assert (ex <= 2.0 ** -8 * (rx.abs() + e_dx) + e_dx + 2.0 ** -23 * rx.abs()).all()
        assert (ew <= e_dw + 2.0 ** -23 * rw.abs()).all()
        # one gradient at a time, the other's buffer not there
        dx1, dw1 = dx0.clone().to(DEV), dw0.clone().to(DEV)
        m.moe_router_backward(cfg, X, W, D, dx1, None, acc, acc)
        m.moe_router_backward(cfg, X, W, D, None, dw1, acc, acc)
        assert torch.equal(dx1, dx) and torch.equal(dw1, dw)


@pytest.mark.parametrize("T,d,E", [(6, 256, 1), (130, 256, 5), (200, 512, 129), (300, 256, 509),
                                     (1100, 256, 5), (2050, 4096, 101)])
def test_a_value_that_is_not_finite_spoils_its_own_rows_only(T, d, E):
    """The last step of dx's reduction reads past a row's E logits, into the next token's."""
    _announce(f"[router bwd, NaN] T={T} d={d} E={E}")
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).to(DEV)
    wr = torch.randn(E, d, generator=g).to(torch.bfloat16).to(DEV)
    dl = torch.randn(T, E, generator=g).to(DEV)
    cfg = m.make_cfg(T, d, E, 1, 128)

    def run(dl):
        dx = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
        dw = torch.zeros(E, d, device=DEV)
        m.moe_router_backward(cfg, x, wr, dl, dx, dw, False, False)
        return dx, dw

    rx, rw = run(dl)
    t, e = T // 2, 0  # the columns that the token before it reads as well
    for bad in (math.nan, inf, -inf):
        spoiled = dl.clone()
        spoiled[t, e] = bad
        dx, dw = run(spoiled)
        assert dx[t].isnan().all() and dw[e].isnan().all()
        rows, experts = torch.arange(T, device=DEV) != t, torch.arange(E, device=DEV) != e
        assert torch.equal(dx[rows], rx[rows]) and torch.equal(dw[experts], rw[experts])


def test_more_than_two_to_the_32_bytes_of_logits():
    """Tokens whose byte offsets pass 32 bits, against the same tokens in a call of their own."""
    T, E, k, n = 1_200_000, 1000, 6, 50
    assert 4 * T * E > 2 ** 32
    _announce(f"[gate] T={T} E={E}: the last {n} tokens")
    g = torch.Generator(DEV).manual_seed(0)
    l = torch.randn(T, E, device=DEV, generator=g)
    gate = m.make_gate(m.MOE_SCORE_SOFTMAX, 1, 1, 0, False, 1.0)

    def run(l):
        T = l.shape[0]
        cfg = m.make_cfg(T, 256, E, k, 128)
        idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
        w = torch.empty(T, k, device=DEV)
        m.moe_gate_select(cfg, gate, l, None, idx, w)
        dl = torch.empty(T, E, device=DEV)
        m.moe_gate_backward(cfg, gate, l, idx, w, dl, False)
        x = torch.ones(T, 256, dtype=torch.bfloat16, device=DEV)
        wr = torch.ones(E, 256, dtype=torch.bfloat16, device=DEV)
        wr[::3] = 0.5
        dx = torch.empty(T, 256, dtype=torch.bfloat16, device=DEV)
        m.moe_router_backward(m.make_cfg(T, 256, E, 1, 128), x, wr, dl, dx, None, False, False)
        return [t[-n:].clone() for t in (idx, w, dl, dx)]

    for a, b in zip(run(l), run(l[-n:].clone())):
        assert torch.equal(a, b)


def test_gate_and_router_calls_refuse_tensors_the_library_cannot_check():
    cfg, g = m.make_cfg(8, 256, 16, 2, 128), m.make_gate()
    l = torch.zeros(8, 16, device=DEV)
    idx, w = torch.zeros(8, 2, dtype=torch.int32, device=DEV), torch.zeros(8, 2, device=DEV)
    bad = [(l.double(), None, idx, w), (l.t(), None, idx, w), (l[:4], None, idx, w),
           (l.cpu(), None, idx, w), (l, None, idx.long(), w), (l, w[0], idx, w)]
    for args in bad:
        with pytest.raises(m.MoeError) as e:
            m.moe_gate_select(cfg, g, *args)
        assert e.value.status == -1


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("G", [2, 8, 96])
def test_choice_by_sums_of_two_where_every_group_stays(G, score):
    """Scores that meet in 64 bits (saturated sigmoids, softmax terms that underflow) go to the
    lower index, though their logits differ: without a bias only one group, or GROUP_MAX, is
    chosen by the logits."""
    _announce(f"[gate] G={G}, all stay, sums of two, score={score}")
    l = _logits(7, 96, 21)
    l[0] = 60.0 + np.arange(96, dtype=np.float32)
    l[1] = -5.0
    l[1, [3, 9, 12]] = 40.0, 50.0, 45.0
    l[2] = -2000.0 + np.arange(96, dtype=np.float32)
    l[2, 5] = 0.0
    l[3, ::3] = -inf
    l[4, 10:] = -inf
    l[4, :10] = 100.0 - np.arange(10, dtype=np.float32)[::-1]
    for k, renorm in itertools.product((3, 8, 40), (False, True)):
        for gsc in (0, 1):
            _check_select(l, k, score, None, G, G, gsc, renorm, 1.0)


def test_softmax_scores_that_underflow_weigh_nothing():
    """A bias may choose experts whose exponentials underflow in 64 bits: their scores are 0, and
    so is their sum."""
    _announce("[gate] softmax scores below 64 bits, chosen by the bias")
    E, k = 40, 5
    l = _logits(4, E, 3)
    bias = np.zeros(E, np.float32)
    bias[10:10 + k] = 2.0
    l[0] = -800.0
    l[0, 0] = 0.0
    l[1] = -1e30
    l[1, 39] = 7.0
    # exp of these in steps of 2^-1074: 11.47, 4.22, 1.55, 0.53 and 0.21
    l[2] = -900.0
    l[2, 0] = 0.0
    l[2, 10:10 + k] = -742.0, -743.0, -744.0, -745.078125, -746.0
    for renorm, (G, tg) in itertools.product((False, True), ((1, 1), (4, 4), (4, 3))):
        _check_select(l, k, 0, bias, G, tg, 1, renorm, 2.5)
    idx, w = _select(l, k, m.make_gate(0, 1, 1, 0, True, 1.0), bias)
    assert sorted(idx[0]) == list(range(10, 15)) and not w[0].any() and not w[1].any()


@pytest.mark.parametrize("G,tg", [(8, 3), (48, 30), (96, 40)])
def test_saturated_sigmoids_between_groups(G, tg):
    """Sigmoids that are 1 in 64 bits: groups whose sums are equal go by their index, and so do
    the experts in them, whatever their logits."""
    _announce(f"[gate] G={G} topk_groups={tg}, saturated sigmoids")
    l = _logits(3, 96, 22)
    l[0] = 60.0 + np.arange(96, dtype=np.float32)
    l[1, ::5] = 38.0 + np.arange(20, dtype=np.float32)
    l[2] = 60.0 + np.arange(96, dtype=np.float32)
    l[2, :24] = -inf
    for gsc, renorm in itertools.product((0, 1), (False, True)):
        _check_select(l, 8, 1, None, G, tg, gsc, renorm, 1.0)
        _check_select(l, 8, 1, np.zeros(96, np.float32), G, tg, gsc, renorm, 1.0)
