"""The layer's own paths through the gate and the block-scaled FP8 products: MoeLayer with a gate,
MoeLayer in FP8 mode, and both at once, against plain 64-bit forms; captured and replayed; on other
streams; run twice.

Tolerances. Both sides round at the same points, so what differs is where a sum of another order
falls on the other side of a rounding: half a bf16 step (2^-8) of single elements, and of an FP8
code one step (2^-3 of the code at most) of the few whose bf16 value moved. Each such element
counts little in a norm over many: the layer's parity bar for every mode, 1e-2 for activations and
2e-2 for gradients in relative Frobenius norm, is ten times what 2^-9 of every element would be.
"""
import numpy as np
import pytest
import torch

import workload
from tests import _ops
from tests._gpu import DEV, MoeLayer, _announce, _np, m
from tests._util import TOL_ACT, TOL_GRAD, assert_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _float32():
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)


SHAPES = {
    "tiny": dict(T=256, d=256, E=8, k=2, I=512),
    "ragged": dict(T=77, d=512, E=16, k=3, I=128),
    "one_token": dict(T=1, d=256, E=8, k=4, I=256),
    "big_experts": dict(T=700, d=256, E=2, k=2, I=128),
    "empty_experts": dict(T=20, d=256, E=64, k=1, I=128),
}


def _inputs(shape, seed=0):
    return workload.make_inputs("tiny", seed=seed, device=DEV, **SHAPES[shape])


def _layer(shape, **over):
    s = SHAPES[shape]
    return MoeLayer(s["T"], s["d"], s["E"], s["k"], s["I"], device=DEV, **over)


def _step(L, inp):
    if L.wq is not None:
        L.quantize_weights(inp["W1"], inp["W2"])
    L.step(inp["X"], inp["Wr"], inp["W1"], inp["W2"], inp["dY"])
    torch.cuda.synchronize()
    return L


def _results(L):
    return [t.clone() for t in (L.topk_idx, L.topk_w, L.y, L.dx, L.dw1, L.dw2, L.dwr, L.d_topk_w)]


@pytest.mark.parametrize("shape", list(SHAPES))
def test_fp8_mode_against_its_plain_form(shape):
    _announce(f"[fp8 layer] {shape} {SHAPES[shape]}")
    inp = _inputs(shape)
    L = _layer(shape, precision=m.MOE_PREC_FP8)
    L.quantize_weights(inp["W1"], inp["W2"])
    L.route(inp["X"], inp["Wr"])
    L.permute(inp["X"])
    L.forward(inp["W1"], inp["W2"])
    L.backward(None, inp["W1"], inp["W2"], inp["dY"])
    torch.cuda.synchronize()
    X, W1, W2, dY = (_np(inp[n]).astype(np.float64) for n in ("X", "W1", "W2", "dY"))
    ref = _ops.fp8_layer(X, W1, W2, dY, _np(L.topk_idx), _np(L.topk_w))
    assert_grad("Y", _np(L.y), ref["Y"], TOL_ACT)
    assert_grad("dX", _np(L.dx), ref["dX"], TOL_ACT)
    assert_grad("dW1", _np(L.dw1), ref["dW1"], TOL_GRAD)
    assert_grad("dW2", _np(L.dw2), ref["dW2"], TOL_GRAD)
    assert_grad("d_topk_w", _np(L.d_topk_w), ref["dw"], TOL_GRAD)


def test_fp8_mode_is_near_the_bf16_mode():
    """Each E4M3 code is within 2^-4 of its value; a product of two, about 2^-4 in rms; through
    two products (and three on the way back) stay below 2^-2."""
    inp = _inputs("tiny")
    a = _results(_step(_layer("tiny"), inp))
    b = _results(_step(_layer("tiny", precision=m.MOE_PREC_FP8), inp))
    for x, y in zip(a[2:], b[2:]):
        assert float((x.double() - y.double()).norm() / x.double().norm()) < 0.25


GATES = {
    "sigmoid_groups": dict(score=m.MOE_SCORE_SIGMOID, groups=4, topk_groups=2,
                           group_score=m.MOE_GROUP_TOP2, renorm=True, scale=2.5),
    "softmax_dense": dict(score=m.MOE_SCORE_SOFTMAX, renorm=False, scale=1.5),
    "sigmoid": dict(score=m.MOE_SCORE_SIGMOID, renorm=False),
}


@pytest.mark.parametrize("gate", list(GATES))
@pytest.mark.parametrize("precision", [m.MOE_PREC_BF16, m.MOE_PREC_MXFP8, m.MOE_PREC_FP8])
def test_gated_layer(gate, precision):
    """The choice and weights from the layer's own logits; then the router's gradients from the
    layer's own d_topk_w, added to the experts' dx of the same routing, given from outside."""
    _announce(f"[gated layer] {gate} precision={precision}")
    spec, s = GATES[gate], SHAPES["tiny"]
    inp = _inputs("tiny", seed=1)
    bias = torch.linspace(-0.1, 0.1, s["E"], device=DEV)
    L = _step(_layer("tiny", precision=precision, gate=m.make_gate(**spec), gate_bias=bias), inp)
    full = dict(groups=1, topk_groups=1, group_score=0, renorm=True, scale=1.0)
    full.update(spec)
    idx, w = _ops.gate(_np(L.logits), s["k"], full["score"], _np(bias), full["groups"],
                       full["topk_groups"], full["group_score"], full["renorm"], full["scale"])
    np.testing.assert_array_equal(_np(L.topk_idx), idx)
    np.testing.assert_allclose(_np(L.topk_w), w, rtol=2.0 ** -23, atol=0)
    # the experts alone, on this routing
    G = _layer("tiny", precision=precision)
    if G.wq is not None:
        G.quantize_weights(inp["W1"], inp["W2"])
    G.set_routing(L.topk_idx, L.topk_w)
    G.step(inp["X"], None, inp["W1"], inp["W2"], inp["dY"])
    torch.cuda.synchronize()
    for a, b in ((G.y, L.y), (G.dw1, L.dw1), (G.dw2, L.dw2), (G.d_topk_w, L.d_topk_w)):
        assert torch.equal(a, b)
    dl = _ops.gate_backward(_np(L.logits), idx, _np(L.d_topk_w), full["score"], full["renorm"],
                            full["scale"])
    assert_grad("dlogits", _np(L.dlogits), dl, 1e-5)  # fp32 steps: a few 2^-24, cancellation
    dl = _np(L.dlogits).astype(np.float64)
    X, Wr = (_np(inp[n]).astype(np.float64) for n in ("X", "Wr"))
    dx = _np(G.dx).astype(np.float64) + dl @ Wr
    # dl enters dx with 17 bits; the sum is rounded to bf16 once
    tol = 2.0 ** -8 * np.abs(dx) + 2.0 ** -14 * (np.abs(dl) @ np.abs(Wr)) + 1e-30
    assert np.all(np.abs(_np(L.dx) - dx) <= tol)
    assert_grad("dWr", _np(L.dwr), dl.T @ X, 1e-5)


def test_gated_layer_accumulates_and_repeats():
    inp = _inputs("tiny", seed=2)
    gate = m.make_gate(m.MOE_SCORE_SIGMOID, 4, 2, m.MOE_GROUP_TOP2, True, 2.5)
    mk = lambda: _layer("tiny", precision=m.MOE_PREC_FP8, gate=gate)
    a, b = _results(_step(mk(), inp)), _results(_step(mk(), inp))
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    L = _step(mk(), inp)
    L.backward(inp["Wr"], inp["W1"], inp["W2"], inp["dY"], accumulate=True, x=inp["X"])
    torch.cuda.synchronize()
    assert torch.equal(L.dwr, a[6] + a[6]) and torch.equal(L.dx, a[3])
    assert torch.equal(L.dw1, a[4] + a[4])
    with pytest.raises(ValueError):
        L.backward(inp["Wr"], inp["W1"], inp["W2"], inp["dY"])  # no tokens
    with pytest.raises(ValueError):
        L.step(inp["X"], inp["Wr"], inp["W1"], inp["W2"], inp["dY"], fused=True)


def test_gated_fp8_step_captured_and_replayed_on_new_inputs():
    _announce("[gated fp8 layer] graph capture and replays")
    gate = m.make_gate(m.MOE_SCORE_SIGMOID, 4, 2, m.MOE_GROUP_TOP2, True, 2.5)
    inps = [_inputs("tiny", seed=s) for s in (3, 4, 5)]
    want = [_results(_step(_layer("tiny", precision=m.MOE_PREC_FP8, gate=gate), i)) for i in inps]
    L = _layer("tiny", precision=m.MOE_PREC_FP8, gate=gate)
    held = {n: t.clone() for n, t in inps[0].items() if torch.is_tensor(t)}

    def run():
        L.quantize_weights(held["W1"], held["W2"])
        L.step(held["X"], held["Wr"], held["W1"], held["W2"], held["dY"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for inp, ref in list(zip(inps, want)) * 2:
        for n in held:
            held[n].copy_(inp[n])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(_results(L), ref):
            assert torch.equal(x, y)


def test_two_layers_on_two_streams_do_not_disturb_each_other():
    gate = m.make_gate(m.MOE_SCORE_SIGMOID, 4, 2, m.MOE_GROUP_TOP2, True, 2.5)
    inps = [_inputs("tiny", seed=s) for s in (6, 7)]
    want = [_results(_step(_layer("tiny", precision=m.MOE_PREC_FP8, gate=gate), i)) for i in inps]
    Ls = [_layer("tiny", precision=m.MOE_PREC_FP8, gate=gate) for _ in inps]
    streams = [torch.cuda.Stream() for _ in inps]
    torch.cuda.synchronize()
    for _ in range(3):
        for L, inp, s in zip(Ls, inps, streams):
            L.quantize_weights(inp["W1"], inp["W2"], stream=s)
            L.step(inp["X"], inp["Wr"], inp["W1"], inp["W2"], inp["dY"], stream=s)
    torch.cuda.synchronize()
    for L, ref in zip(Ls, want):
        for x, y in zip(_results(L), ref):
            assert torch.equal(x, y)


def test_fp8_mode_skips_bad_expert_indices():
    """A row that names no expert is skipped, as in the other modes, and the rest is as without."""
    inp = _inputs("tiny", seed=8)
    L = _layer("tiny", precision=m.MOE_PREC_FP8)
    L.quantize_weights(inp["W1"], inp["W2"])
    L.route(inp["X"], inp["Wr"])
    idx, w = L.topk_idx.clone(), L.topk_w.clone()
    idx[5, 1], idx[200, 0] = -1, 99
    ref = _ops.fp8_layer(*(_np(inp[n]).astype(np.float64) for n in ("X", "W1", "W2", "dY")),
                         _np(idx), _np(w))
    L.row_src.fill_(2 ** 31 - 1)  # what the skipped rows leave unwritten
    L.set_routing(idx, w)
    L.step(inp["X"], None, inp["W1"], inp["W2"], inp["dY"])
    torch.cuda.synchronize()
    assert L.device_status() == m.MOE_DEVICE_BAD_EXPERT_INDEX
    assert_grad("Y", _np(L.y), ref["Y"], TOL_ACT)
    assert_grad("dX", _np(L.dx), ref["dX"], TOL_ACT)
    assert_grad("dW1", _np(L.dw1), ref["dW1"], TOL_GRAD)


def test_fp8_mode_keeps_what_is_not_finite():
    """A NaN or an infinity of a token, or of a gradient, comes out as NaN at that token (and not
    finite in its experts' weight gradients), and changes no other; a weight's at its expert."""
    s = SHAPES["tiny"]
    inp = _inputs("tiny", seed=9)
    g = torch.Generator().manual_seed(1)
    idx = torch.rand(s["T"], s["E"], generator=g).topk(s["k"], dim=1).indices.to(torch.int32)

    def step(X, W1, dY):
        L = _layer("tiny", precision=m.MOE_PREC_FP8)
        L.quantize_weights(W1, inp["W2"])
        L.set_routing(idx.to(DEV), torch.full((s["T"], s["k"]), 0.5, device=DEV))
        L.step(X, None, W1, inp["W2"], dY)
        torch.cuda.synchronize()
        return L

    clean = step(inp["X"], inp["W1"], inp["dY"])
    X, dY, W1 = inp["X"].clone(), inp["dY"].clone(), inp["W1"].clone()
    X[5, 17], X[100, 3], dY[30, 200] = float("nan"), float("inf"), -float("inf")
    L = step(X, inp["W1"], dY)
    t = torch.arange(s["T"], device=DEV)
    fwd = (t == 5) | (t == 100)
    bwd = fwd | (t == 30)
    for got, ref, bad in ((L.y, clean.y, fwd), (L.dx, clean.dx, bwd),
                          (L.d_topk_w, clean.d_topk_w, bwd)):
        assert got[bad].isnan().all() and torch.equal(got[~bad], ref[~bad])
    for e in range(s["E"]):
        hit = bool((idx[[5, 100, 30]] == e).any())
        for got, ref in ((L.dw1, clean.dw1), (L.dw2, clean.dw2)):
            assert bool(got[e].isfinite().all()) != hit
            assert hit or torch.equal(got[e], ref[e])
    W1[2, 40, 9] = float("nan")
    L = step(inp["X"], W1, inp["dY"])
    bad = (idx == 2).any(1).to(DEV)
    for got, ref in ((L.y, clean.y), (L.dx, clean.dx)):
        assert got[bad].isnan().all() and torch.equal(got[~bad], ref[~bad])


# Products that the shapes above leave out: 128-row tiles (256 column tiles and more, few rows an
# expert), and 32-row tiles (640 of them, nearly all with rows) with 128-row ones in the backward.
SHAPES["many_experts"] = dict(T=150, d=512, E=64, k=2, I=256)
SHAPES["wide"] = dict(T=128, d=256, E=64, k=2, I=640)


@pytest.mark.parametrize("bf16_dw", [False, True])
@pytest.mark.parametrize("shape", ["many_experts", "wide", "ragged"])
def test_fp8_mode_accumulates_in_either_gradient_type(shape, bf16_dw):
    """Both gradient types, written and then added to: the second backward doubles them (in bf16
    within a rounding of each, far below the bar)."""
    _announce(f"[fp8 layer] {shape} {SHAPES[shape]} bf16_dw={bf16_dw}")
    inp = _inputs(shape, seed=10)
    L = _layer(shape, precision=m.MOE_PREC_FP8, bf16_dw=bf16_dw)
    L.quantize_weights(inp["W1"], inp["W2"])
    L.route(inp["X"], inp["Wr"])
    L.permute(inp["X"])
    L.forward(inp["W1"], inp["W2"])
    ref = _ops.fp8_layer(*(_np(inp[n]).astype(np.float64) for n in ("X", "W1", "W2", "dY")),
                         _np(L.topk_idx), _np(L.topk_w))
    for times in (1, 2):
        L.backward(None, inp["W1"], inp["W2"], inp["dY"], accumulate=times == 2)
        torch.cuda.synchronize()
        assert L.dw1.dtype == L.dw2.dtype == (torch.bfloat16 if bf16_dw else torch.float32)
        assert_grad("dW1", _np(L.dw1), times * ref["dW1"], TOL_GRAD)
        assert_grad("dW2", _np(L.dw2), times * ref["dW2"], TOL_GRAD)
    assert_grad("Y", _np(L.y), ref["Y"], TOL_ACT)
    assert_grad("dX", _np(L.dx), ref["dX"], TOL_ACT)
    assert_grad("d_topk_w", _np(L.d_topk_w), ref["dw"], TOL_GRAD)


def test_gated_backward_refuses_tokens_before_it_adds_gradients():
    inp = _inputs("tiny", seed=11)
    L = _step(_layer("tiny", gate=m.make_gate(m.MOE_SCORE_SIGMOID)), inp)
    before = _results(L)
    for x, wr in ((inp["X"].float(), inp["Wr"]), (inp["X"][:9], inp["Wr"]),
                  (inp["X"], inp["Wr"].cpu()), (inp["X"], inp["Wr"].t())):
        with pytest.raises(m.MoeError):
            L.backward(wr, inp["W1"], inp["W2"], inp["dY"], accumulate=True, x=x)
    torch.cuda.synchronize()
    for a, b in zip(_results(L), before):
        assert torch.equal(a, b)
