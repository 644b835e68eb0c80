"""Host checks of the 8-bit integer products and the dense gated feed-forward block: every refusal
happens before anything is enqueued; and the plain forms the GPU tests compare with are pinned
against differences and exact arithmetic."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import _products as P64
from tests._util import ensure_built

m = ensure_built()
P = ctypes.c_void_p(1 << 20)
Q = ctypes.c_void_p(1 << 21)
ODD = ctypes.c_void_p((1 << 20) + 2)
ARG = m.MOE_ERR_INVALID_ARG


def _refuses(fn, good, at, bad):
    args = list(good)
    args[at] = bad
    assert fn(*args) == ARG, (fn.__name__, at, bad)


def test_quantize_rows_refuses():
    fn = m.lib().moe_i8_quantize_rows
    good = (P, 4, 256, P, P, None)
    for at, bads in ((0, (None, ODD)), (1, (-1, 1 << 24)), (2, (0, 64, 200, -128)),
                     (3, (None, ODD)), (4, (None, ODD))):
        for bad in bads:
            _refuses(fn, good, at, bad)
    assert fn(None, 0, 256, None, None, None) == 0  # no rows, no addresses


@pytest.mark.parametrize("gated", [False, True])
def test_products_refuse(gated):
    L = m.lib()
    if gated:
        fn, good = L.moe_i8_gemm_gated, [P, 4, 2, 128, 256, 0, P, P, P, P, P, None]
        for bad in (-1, 4):
            _refuses(fn, good, 5, bad)
    else:
        fn, good = L.moe_i8_gemm, [P, 4, 2, 128, 256, P, P, P, P, P, None]
    ptr = 6 if gated else 5
    for at in (0, ptr, ptr + 1, ptr + 2, ptr + 3, ptr + 4):
        _refuses(fn, good, at, None)
        _refuses(fn, good, at, ODD)
    for at, bads in ((1, (-1,)), (2, (0, 1025, -3)), (3, (0, 64, 130, -128, 1 << 30)),
                     (4, (0, 64, 130, 1 << 17, (1 << 17) + 128))):
        for bad in bads:
            _refuses(fn, good, at, bad)
    big = list(good)
    big[3], big[4] = 1 << 17, 1 << 14  # N K = 2^31
    assert fn(*big) == ARG
    for M, E in ((2 ** 31 - 1, 1), (2 ** 24, 1), (1, 1024)):  # more threads than a grid has
        big = list(good)
        big[1], big[2], big[3], big[4] = M, E, 1 << 20, 128
        assert fn(*big) == ARG
    empty = list(good)
    empty[1] = 0
    empty[ptr] = empty[ptr + 1] = empty[ptr + 4] = None
    assert fn(*empty) == 0


def test_ffn_refuses_shapes():
    for bad in (dict(T=0), dict(d=64), dict(d=200), dict(I=0), dict(I=130), dict(act=4),
                dict(act=-1), dict(flags=1), dict(flags=2), dict(flags=8),
                dict(T=1 << 20, d=2048), dict(T=1 << 20, I=1024, d=128),
                dict(T=2 ** 31 - 1), dict(d=1 << 15, I=1 << 14)):
        c = m.make_ffn(**{**dict(T=4, d=256, I=128), **bad})
        with pytest.raises(m.MoeError) as e:
            m.moe_ffn_query(c)
        assert e.value.status == ARG, bad
        r = ctypes.byref(c)
        assert m.lib().moe_ffn_forward(r, P, P, P, P, P, Q, 0, P, 1 << 40, None) == ARG
        assert m.lib().moe_ffn_backward(r, P, P, P, P, P, Q, ODD, P, P, 0, 0, P, 1 << 40,
                                        None) == ARG
    assert m.lib().moe_ffn_query(None, ctypes.byref(m.MoeFfnSizes())) == ARG
    assert m.lib().moe_ffn_query(ctypes.byref(m.make_ffn(4, 256, 128)), None) == ARG


def test_ffn_calls_refuse_pointers_and_short_workspaces():
    L = m.lib()
    c = m.make_ffn(4, 256, 128)
    n = m.moe_ffn_query(c).workspace
    r = ctypes.byref(c)
    fwd = [r, P, P, P, P, P, Q, 0, P, n, None]
    for at in (1, 2, 3, 4, 5, 6, 8):
        if at != 4:  # H may be NULL
            _refuses(L.moe_ffn_forward, fwd, at, None)
        _refuses(L.moe_ffn_forward, fwd, at, ODD)
    _refuses(L.moe_ffn_forward, fwd, 6, P)  # y is not x
    short = list(fwd)
    short[9] = n - 1
    assert L.moe_ffn_forward(*short) == -5
    bwd = [r, P, P, P, P, P, P, Q, P, P, 0, 0, P, n, None]
    for at in (1, 2, 3, 4, 5, 6, 7, 8, 9, 12):
        _refuses(L.moe_ffn_backward, bwd, at, None)
        _refuses(L.moe_ffn_backward, bwd, at, ODD)
    _refuses(L.moe_ffn_backward, bwd, 7, P)  # dx is neither x nor dy
    short = list(bwd)
    short[13] = n - 1
    assert L.moe_ffn_backward(*short) == -5


def test_codes_are_those_of_the_exact_quotient():
    """Every ratio of two bf16 mantissas, and smaller values: the 64-bit form rounds as exact
    fractions do, ties included."""
    ties = 0
    for b in (128, 129, 131, 170, 200, 254, 255):
        vals = [a * 2.0 ** -s for s in range(0, 9) for a in range(128, b + 1 if s == 0 else 256)]
        row = np.array([vals + [float(b)]])
        codes, scales = P64.quantize_rows(row)
        for v, c in zip(vals, codes[0]):
            q = Fraction(127) * Fraction(v) / b
            assert c == round(q)  # Fractions round half to even
            ties += (q * 2).denominator == 1 and q.denominator == 2
        assert scales[0] == np.float32(b) / np.float32(127)
    assert ties > 20


@pytest.mark.parametrize("a", P64.ACTS)
def test_ffn_gradients_against_differences(a):
    rng = np.random.default_rng(a)
    T, d, I, h = 5, 6, 4, 1e-5
    x, dy = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    w1, w2 = rng.standard_normal((2 * I, d)), rng.standard_normal((d, I))
    H, A, _ = P64.ffn_forward(x, w1, w2, a)
    assert np.abs(H).min() > 1e-3  # no ReLU corner within the step
    _, dx, dw1, dw2 = P64.ffn_backward(x, w1, w2, H, A, dy, a)

    def loss():
        _, A, _ = P64.ffn_forward(x, w1, w2, a)
        return float((A @ w2.T * dy).sum())

    for v, g in ((x, dx), (w1, dw1), (w2, dw2)):
        for i in np.ndindex(*v.shape):
            keep = v[i]
            v[i] = keep + h
            up = loss()
            v[i] = keep - h
            down = loss()
            v[i] = keep
            # the differences' own error: h^2 times a third derivative of order 10
            assert abs((up - down) / (2 * h) - g[i]) < 1e-6 * (1 + abs(g[i])), i


@pytest.mark.parametrize("a", P64.ACTS)
def test_activations_are_torchs(a):
    g = np.linspace(-9, 9, 2001)
    t = torch.tensor(g, requires_grad=True)
    F = torch.nn.functional
    y = [F.silu, F.gelu, lambda v: F.gelu(v, approximate="tanh"), F.relu][a](t)
    y.sum().backward()
    np.testing.assert_allclose(P64.act(a, g), y.detach().numpy(), rtol=1e-12, atol=1e-14)
    np.testing.assert_allclose(P64.act_grad(a, g), t.grad.numpy(), rtol=1e-9, atol=1e-12)


def test_int8_mode_sizes_and_refusals():
    T, d, E, k, I = 300, 512, 16, 3, 256
    c = m.make_cfg(T, d, E, k, I, m.MOE_PREC_INT8)
    s8, s = m.moe_query(c), m.moe_query(m.make_cfg(T, d, E, k, I))
    up = lambda v: (v + 255) // 256 * 256
    Tk = T * k
    assert s8.ring_slot == s.ring_slot and s8.saved == up(2 * Tk * I) and s8.saved_A == 0
    assert s8.wq == up(E * 2 * I * d) + up(4 * E * 2 * I) + up(E * d * I) + up(4 * E * d)
    assert s8.workspace - s.workspace == up(Tk * max(d, I)) + up(4 * Tk)
    for flag in (m.MOE_FLAG_PERSISTENT, m.MOE_FLAG_MXFP8_WGRAD, m.MOE_FLAG_BF16_DW):
        with pytest.raises(m.MoeError) as e:
            m.moe_query(m.make_cfg(T, d, E, k, I, m.MOE_PREC_INT8, flag))
        assert e.value.status == ARG
    for bad in ((4, 1 << 17, 1, 1, 128), (4, 256, 1, 1, 1 << 17), (1 << 20, 256, 32, 16, 128),
                (4, 256, 1024, 1, 1 << 14), (4, 1 << 14, 1024, 1, 128)):
        with pytest.raises(m.MoeError) as e:
            m.moe_query(m.make_cfg(*bad, m.MOE_PREC_INT8))
        assert e.value.status == ARG, bad
    L, r = m.lib(), ctypes.byref(c)
    assert L.moe_quantize_weights(r, P, P, P, s8.wq - 1, None) == -5
    fwd = lambda wq, n: L.moe_forward(r, P, s8.ring_slot, 0, P, P, P, P, P, wq, n, P, P, s8.saved,
                                      P, s8.workspace, None)
    assert fwd(None, 0) == ARG and fwd(P, s8.wq - 1) == -5
    assert L.moe_backward(r, P, s8.ring_slot, 0, P, P, P, P, P, None, P, P, P, s8.wq, P, s8.saved,
                          P, P, P, P, None, P, 0, P, s8.workspace, None) == -3
    assert L.moe_forward_fused(r, P, P, P, P, P, P, s8.ring_slot, 0, P, P, P, P, P, P, P, P,
                               s8.saved, P, s8.workspace, None) == -3


def test_layer_refusals(monkeypatch):
    from mixture_experts_layer_deterministic_amd import layer
    calls = []
    for name in ("moe_forward", "moe_backward", "moe_ffn_forward", "moe_ffn_backward"):
        monkeypatch.setattr(layer, name, lambda *a, n=name: calls.append(n))
    monkeypatch.setattr(layer, "_dev", lambda *a: calls.append("checks"))
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu", precision=m.MOE_PREC_INT8)
    assert L.dw1 is None and L.dw2 is None
    with pytest.raises(ValueError, match="no backward"):
        L.backward(None, x, x, x)
    with pytest.raises(ValueError, match="no H"):
        L.H()
    with pytest.raises(ValueError, match="other tokens"):
        layer.MoeLayer(4, 256, 8, 2, 128, device="cpu",
                       shared=layer.SharedExpert(5, 256, 128, device="cpu"))
    sh = layer.SharedExpert(4, 256, 128, device="cpu", train=False)
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu", shared=sh)
    for call in (lambda: L.forward(x, x), lambda: L.forward(x, x, x=x),
                 lambda: L.forward_fused(x, x, x, x), lambda: L.backward(None, x, x, x, x=x)):
        with pytest.raises(ValueError, match="needs x and shared_w"):
            call()
    with pytest.raises(ValueError, match="without train"):
        L.backward(None, x, x, x, x=x, shared_w=(x, x))
    with pytest.raises(ValueError, match="nothing for a backward"):
        sh.backward(x, x, x, x, x)
    assert not calls
    L.forward(x, x, x=x, shared_w=(x, x))
    assert calls == ["moe_forward", "moe_ffn_forward"]
    sh.H = x
    L.backward(None, x, x, x, x=x, shared_w=(x, x))
    assert calls[2:] == ["checks", "moe_backward", "moe_ffn_backward"]


def test_a_shared_expert_keeps_a_batch_of_its_own_saved(monkeypatch):
    """Batches with a saved of their own: the shared expert's H and A go with it, or it is refused."""
    from mixture_experts_layer_deterministic_amd import layer
    seen = []
    for name in ("moe_forward", "moe_forward_fused", "moe_backward", "_dev"):
        monkeypatch.setattr(layer, name, lambda *a, n=name: seen.append(n))
    monkeypatch.setattr(layer, "moe_ffn_forward", lambda c, x, w1, w2, H, A, *a: seen.append((H, A)))
    monkeypatch.setattr(layer, "moe_ffn_backward", lambda c, x, w1, w2, H, A, *a: seen.append((H, A)))
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    sh = layer.SharedExpert(4, 256, 128, device="cpu")
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu", shared=sh)
    w, saved, own = (x, x), torch.empty_like(L.saved), sh.new_saved()
    assert own[0].shape == sh.H.shape and own[1].shape == sh.A.shape and own[0] is not sh.H
    calls = (lambda **k: L.forward(x, x, x=x, shared_w=w, **k),
             lambda **k: L.forward_fused(x, x, x, x, shared_w=w, **k),
             lambda **k: L.backward(None, x, x, x, x=x, shared_w=w, **k))
    for call in calls:
        for half in (dict(saved=saved), dict(shared_saved=own)):
            with pytest.raises(ValueError, match="given together"):
                call(**half)
    assert not seen
    for call in calls:
        call()
        assert seen[-1][0] is sh.H and seen[-1][1] is sh.A
        call(saved=saved, shared_saved=own)
        assert seen[-1][0] is own[0] and seen[-1][1] is own[1]
    bare = layer.SharedExpert(4, 256, 128, device="cpu", train=False)
    assert bare.new_saved()[0] is None
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu", shared=bare)
    with pytest.raises(ValueError, match="without train"):
        L.backward(None, x, x, x, x=x, shared_w=w, saved=saved, shared_saved=bare.new_saved())
