"""The layer on the 8-bit integer products and with its shared expert: MoeLayer in INT8 mode against
64-bit plain forms step by step, a training step with a shared expert against the layer and the block
on their own, and both captured and replayed.

Tolerances of the INT8 mode follow tests/test_gpu_int8.py: A through the exact products of the codes,
O from the stored A's codes, y from the stored O by k fp32 multiply-adds. A shared expert's output and
gradient are added in fp32 to what the layer stored in bf16 and rounded once more: the sum is compared
with that of the two stored parts, off by half a step of the part that is not stored here and half a
step of the total."""
import numpy as np
import pytest
import torch

import workload
from mixture_experts_layer_deterministic_amd.layer import SharedExpert
from tests import _products as P64
from tests._gpu import DEV, MoeLayer, _announce, m

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


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


def _np(t):
    return t.double().cpu().numpy()


def _inputs(shape, seed=0):
    return workload.make_inputs("tiny", seed=seed, device=DEV, **SHAPES[shape])


def _layer(shape, **over):
    s = SHAPES[shape]
    return MoeLayer(s["T"], s["d"], s["E"], s["k"], s["I"], device=DEV, **over)


def _forward(L, inp, **kw):
    L.route(inp["X"], inp["Wr"])
    L.permute(inp["X"])
    L.forward(inp["W1"], inp["W2"], **kw)
    torch.cuda.synchronize()


def _quantised(W):
    E, N, K = W.shape
    q, s = P64.quantize_rows(_np(W).reshape(E * N, K))
    return q.reshape(E, N, K), s.reshape(E, N)


@pytest.mark.parametrize("shape", list(SHAPES))
@pytest.mark.parametrize("gate", [False, True])
def test_int8_layer_against_the_plain_form(shape, gate):
    _announce(f"[i8 layer] {shape} gate={gate}")
    inp = _inputs(shape)
    L = _layer(shape, precision=m.MOE_PREC_INT8,
               gate=m.make_gate(m.MOE_SCORE_SIGMOID, renorm=True, scale=2.5) if gate else None)
    L.quantize_weights(inp["W1"], inp["W2"])
    _forward(L, inp)
    T, d, k, I = L.T, L.d, L.k, L.I
    off, rows = L.offsets.cpu().numpy(), T * k
    xq, xs = P64.quantize_rows(_np(L.xp()))
    v = P64.i8_product(off, xq, xs, *_quantised(inp["W1"]), rows)
    (g, u), e = np.split(v, 2, axis=1), 3 * P64.F32
    a, ea = P64.act(P64.SILU, g) * u, P64.gated_error(g, u, e * np.abs(g), e * np.abs(u))
    A = _np(L.A())
    assert (np.abs(A - a) <= P64.BF16 * (np.abs(a) + ea) + ea + 1e-37).all()
    aq, as_ = P64.quantize_rows(A)
    o = P64.i8_product(off, aq, as_, *_quantised(inp["W2"]), rows)
    O = _np(L.O())
    assert (np.abs(O - o) <= (P64.BF16 + 4 * P64.F32) * np.abs(o) + 1e-37).all()
    w, at = _np(L.topk_w), L.tk_row.cpu().numpy().reshape(T, k)
    parts = w[:, :, None] * O[at]
    y, mag = parts.sum(axis=1), np.abs(parts).sum(axis=1)
    ey = k * P64.F32 * mag
    assert (np.abs(_np(L.y) - y) <= P64.BF16 * (np.abs(y) + ey) + ey + 1e-37).all()
    # and near the layer in bf16: a code is off by at most 1 / 254 of its row's largest value
    R = _layer(shape, gate=L.gate)
    _forward(R, inp)
    assert torch.equal(R.topk_idx, L.topk_idx)
    assert (R.y.double() - L.y.double()).norm() <= 4 / 127 * R.y.double().norm()


def test_int8_layer_leaves_out_bad_expert_indexes():
    inp = _inputs("ragged")
    L = _layer("ragged", precision=m.MOE_PREC_INT8)
    L.quantize_weights(inp["W1"], inp["W2"])
    _forward(L, inp)
    y = L.y.clone()
    idx, w = L.topk_idx.clone(), L.topk_w.clone()
    idx[5, 1], w[5, 1] = 99, 0.0
    L.set_routing(idx, w)
    L.permute(inp["X"])
    L.forward(inp["W1"], inp["W2"])
    torch.cuda.synchronize()
    assert L.device_status() == m.MOE_DEVICE_BAD_EXPERT_INDEX
    keep = torch.arange(L.T, device=DEV) != 5
    assert torch.equal(L.y[keep], y[keep])


def _shared_weights(d, I, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    r = lambda *s: (torch.randn(*s, generator=g, device=DEV) * s[1] ** -0.5).to(BF16)
    return r(2 * I, d), r(d, I)


def _sum_of(got, a, b):
    """got = bf16(a + v) for a v that b is the bf16 image of."""
    a, b = _np(a), _np(b)
    ev = P64.BF16 * np.abs(b) * (1 + P64.BF16)
    tol = ev + (P64.BF16 + P64.F32) * (np.abs(a + b) + ev) + 1e-37
    assert (np.abs(_np(got) - (a + b)) <= tol).all()


@pytest.mark.parametrize("shape", ["tiny", "ragged", "one_token"])
@pytest.mark.parametrize("mode", ["plain", "gated", "fused", "fp8", "bf16_dw"])
def test_training_step_with_a_shared_expert(shape, mode):
    _announce(f"[shared] {shape} {mode}")
    inp, s = _inputs(shape), SHAPES[shape]
    T, d, I = s["T"], s["d"], 384
    gate = m.make_gate(m.MOE_SCORE_SIGMOID, renorm=True) if mode == "gated" else None
    prec = m.MOE_PREC_FP8 if mode == "fp8" else m.MOE_PREC_BF16
    over = dict(gate=gate, precision=prec, bf16_dw=mode == "bf16_dw")
    block = SharedExpert(T, d, I, act=m.MOE_ACT_GELU, device=DEV, bf16_dw=mode == "bf16_dw")
    alone = SharedExpert(T, d, I, act=m.MOE_ACT_GELU, device=DEV, bf16_dw=mode == "bf16_dw")
    L, R = _layer(shape, shared=block, **over), _layer(shape, **over)
    sw = _shared_weights(d, I, 3)
    X, dY = inp["X"], inp["dY"]
    for layer, kw in ((L, dict(shared_w=sw)), (R, {})):
        if layer.wq is not None:
            layer.quantize_weights(inp["W1"], inp["W2"])
        layer.step(X, inp["Wr"], inp["W1"], inp["W2"], dY, fused=mode == "fused", **kw)
    y, dx = torch.empty(T, d, dtype=BF16, device=DEV), torch.empty(T, d, dtype=BF16, device=DEV)
    alone.forward(X, *sw, y)
    alone.backward(X, *sw, dY, dx)
    torch.cuda.synchronize()
    _sum_of(L.y, R.y, y)
    _sum_of(L.dx, R.dx, dx)
    # the experts' own gradients and the block's are what they are apart
    for a, b in ((L.dw1, R.dw1), (L.dw2, R.dw2), (L.dwr, R.dwr), (L.d_topk_w, R.d_topk_w),
                 (block.dw1, alone.dw1), (block.dw2, alone.dw2), (block.H, alone.H)):
        assert torch.equal(a, b)


def test_two_batches_on_their_way_with_a_shared_expert():
    """Two forwards, then their backwards in reverse, each with its own saved: what each batch gives
    alone, and the sums of both batches' weight gradients."""
    inp, s = _inputs("tiny"), SHAPES["tiny"]
    T, d, I = s["T"], s["d"], 384
    block = lambda: SharedExpert(T, d, I, device=DEV)
    sw = _shared_weights(d, I, 5)
    X = [inp["X"], inp["X"].flip(0).contiguous()]
    dY = [inp["dY"], inp["dY"].flip(1).contiguous()]
    one = [_layer("tiny", shared=block()) for _ in X]
    for L, x, dy in zip(one, X, dY):
        L.step(x, inp["Wr"], inp["W1"], inp["W2"], dy, shared_w=sw)
    both = _layer("tiny", shared=block(), ring_slots=2)
    saved = [(torch.empty_like(both.saved), both.shared.new_saved()) for _ in X]
    for i, x in enumerate(X):
        both.route(x, inp["Wr"])
        both.permute(x, i)
        both.forward(inp["W1"], inp["W2"], i, saved[i][0], x=x, shared_w=sw,
                     shared_saved=saved[i][1])
        assert torch.equal(both.y, one[i].y)
    for i in (1, 0):
        both.route(X[i], inp["Wr"])
        both.permute(X[i], i)
        both.backward(inp["Wr"], inp["W1"], inp["W2"], dY[i], i, i == 0, saved[i][0], x=X[i],
                      shared_w=sw, shared_saved=saved[i][1])
        assert torch.equal(both.dx, one[i].dx)
        if i == 1:
            for k in ("dw1", "dw2"):
                assert torch.equal(getattr(both.shared, k), getattr(one[1].shared, k))
    # the same T products in fp32 on both sides, off by T half steps of their magnitudes at most on
    # each, and one addition
    A, dy = saved[0][1][1], _np(dY[0])
    mag = np.abs(dy).T @ np.abs(_np(A)) + np.abs(_np(one[1].shared.dw2))
    want = _np(one[0].shared.dw2) + _np(one[1].shared.dw2)
    assert (np.abs(_np(both.shared.dw2) - want) <= 2 * (T + 1) * P64.F32 * mag).all()


def test_int8_layer_with_a_shared_expert_captured_and_replayed():
    """A serving step in one graph: route, permute, int8 experts and the shared expert, replayed with
    other tokens between eager calls."""
    inp = _inputs("ragged")
    s = SHAPES["ragged"]
    sw = _shared_weights(s["d"], 256, 4)
    make = lambda: _layer("ragged", precision=m.MOE_PREC_INT8, shared=SharedExpert(
        s["T"], s["d"], 256, device=DEV, train=False))
    L, R = make(), make()
    for layer in (L, R):
        layer.quantize_weights(inp["W1"], inp["W2"])
    X = inp["X"].clone()

    def step(layer, x):
        layer.route(x, inp["Wr"])
        layer.permute(x)
        layer.forward(inp["W1"], inp["W2"], x=x, shared_w=sw)

    step(L, X)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(L, X)
    for i in range(4):
        X.copy_(torch.roll(inp["X"], i, 0))
        L.y.zero_()
        g.replay()
        torch.cuda.synchronize()
        step(R, X.clone())
        torch.cuda.synchronize()
        assert torch.equal(L.y, R.y) and torch.isfinite(L.y.float()).all()


def test_a_refused_batch_leaves_every_gradient():
    """A second microbatch whose shared_saved is another size's: nothing is added to any gradient, and
    the corrected call gives what it gives without the refused one."""
    inp, s = _inputs("ragged"), SHAPES["ragged"]
    T, d, I = s["T"], s["d"], 384
    sw, outs = _shared_weights(d, I, 7), []
    for refuse in (False, True):
        L = _layer("ragged", shared=SharedExpert(T, d, I, device=DEV))
        L.step(inp["X"], inp["Wr"], inp["W1"], inp["W2"], inp["dY"], shared_w=sw)
        back = lambda x, w, own=None: L.backward(
            inp["Wr"], inp["W1"], inp["W2"], inp["dY"], 0, True, None if own is None else L.saved,
            x=x, shared_w=w, shared_saved=own)
        grads = (L.dw1, L.dw2, L.dwr, L.dx, L.shared.dw1, L.shared.dw2)
        before = [t.clone() for t in grads]
        if refuse:
            H, A = L.shared.new_saved()
            shifted = torch.empty(T * d + 8, dtype=BF16, device=DEV)[1:T * d + 1].view(T, d)
            for args in ((inp["X"], sw, (H[:-1], A)), (inp["X"], sw, (H, A[:, :256])),
                         (shifted, sw), (inp["X"], (sw[0], sw[1].t()))):
                with pytest.raises(m.MoeError):
                    back(*args)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(grads, before))
        back(inp["X"], sw)
        torch.cuda.synchronize()
        outs.append([t.clone() for t in grads])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_int8_layer_serves_without_the_bf16_weights():
    inp = _inputs("ragged")
    L = _layer("ragged", precision=m.MOE_PREC_INT8)
    L.quantize_weights(inp["W1"], inp["W2"])
    _forward(L, inp)
    want = L.y.clone()
    L.y.zero_()
    _forward(L, dict(inp, W1=None, W2=None))
    assert torch.equal(L.y, want)
