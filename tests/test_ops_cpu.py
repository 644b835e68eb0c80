"""Host checks of the gate, router-gradient and block-scaled FP8 calls: every refusal happens
before anything is enqueued; and the 64-bit plain forms the GPU tests compare with are pinned
against other forms of the same definitions."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import _ops
from tests._util import ensure_built

m = ensure_built()
P = ctypes.c_void_p(1 << 20)
CFG = m.make_cfg(64, 256, 8, 2, 128)


@pytest.fixture(autouse=True)
def _float32():
    """The inputs below are fp32 where no type is named, whatever another test file set."""
    before = torch.get_default_dtype()
    torch.set_default_dtype(torch.float32)
    yield
    torch.set_default_dtype(before)



def _ref(x):
    return ctypes.byref(x)


BAD_GATES = [
    dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=16),
    dict(groups=4, topk_groups=0), dict(groups=4, topk_groups=5),
    dict(groups=8, topk_groups=1),  # k = 2 of one expert
    dict(group_score=2), dict(renorm=2), dict(scale=math.inf), dict(scale=math.nan),
]


@pytest.mark.parametrize("bad", BAD_GATES, ids=str)
def test_gate_calls_refuse_a_bad_gate(bad):
    L = m.lib()
    g = m.make_gate(**bad)
    s = m.moe_query(CFG)
    assert L.moe_gate_select(_ref(CFG), _ref(g), P, P, P, P, None) == -1
    assert L.moe_route_gated(_ref(CFG), _ref(g), P, P, P, P, P, P, P, s.workspace, None) == -1
    assert L.moe_gate_backward(_ref(CFG), _ref(g), P, P, P, P, 0, None) == -1


def test_gate_calls_refuse_bad_pointers_and_shapes():
    L = m.lib()
    g = m.make_gate()
    odd = ctypes.c_void_p((1 << 20) + 2)
    s = m.moe_query(CFG)
    for bad in (None, odd):
        for at in range(4):
            if at == 1 and bad is None:
                continue  # no bias is a bias of zero
            args = [P, P, P, P]
            args[at] = bad
            assert L.moe_gate_select(_ref(CFG), _ref(g), *args, None) == -1
            if at != 1 or bad is odd:
                assert L.moe_gate_backward(_ref(CFG), _ref(g), *args, 0, None) == -1
    assert L.moe_gate_select(_ref(CFG), None, P, P, P, P, None) == -1
    assert L.moe_gate_select(None, _ref(g), P, P, P, P, None) == -1
    assert L.moe_route_gated(_ref(CFG), _ref(g), P, P, P, P, P, P, P, s.workspace - 1, None) == -5
    assert L.moe_route_gated(_ref(CFG), _ref(g), odd, P, P, P, P, P, P, s.workspace, None) == -1


def test_router_backward_refuses_bad_arguments():
    L = m.lib()
    odd = ctypes.c_void_p((1 << 20) + 8)
    Q = ctypes.c_void_p(1 << 21)
    call = lambda x, w, dl, dx, dwr: L.moe_router_backward(_ref(CFG), x, w, dl, dx, dwr, 0, 0, None)
    assert call(None, P, P, Q, P) == -1
    assert call(P, odd, P, Q, P) == -1
    assert call(P, P, None, Q, P) == -1
    assert call(P, P, P, None, None) == -1   # no gradient wanted
    assert call(P, P, P, odd, P) == -1
    assert call(P, P, P, P, P) == -1         # dx over x


def test_fp8_calls_refuse_bad_arguments():
    L = m.lib()
    odd = ctypes.c_void_p((1 << 20) + 8)
    for rows, cols in ((-1, 128), (4, 0), (4, 64), (4, 130), (2 ** 31 - 1, 1 << 20)):
        assert L.moe_fp8_quantize_rows(P, rows, cols, P, P, None) == -1
    assert L.moe_fp8_quantize_rows(odd, 4, 128, P, P, None) == -1
    assert L.moe_fp8_quantize_rows(P, 4, 128, P, None, None) == -1
    assert L.moe_fp8_quantize_rows(P, 0, 128, P, P, None) == 0  # nothing to do
    for E, N, K in ((0, 128, 128), (1025, 128, 128), (1, 64, 128), (1, 128, 0), (1, 192, 128),
                    (1, 1 << 16, 1 << 15)):
        assert L.moe_fp8_quantize_weights(P, E, N, K, P, P, P, P, None) == -1
        assert L.moe_fp8_gemm(P, 4, E, N, K, P, P, P, P, P, None) == -1
    assert L.moe_fp8_quantize_weights(P, 1, 128, 128, P, P, P, None, None) == -1
    assert L.moe_fp8_quantize_weights(P, 1, 128, 128, P, P, None, P, None) == -1
    assert L.moe_fp8_gemm(P, -1, 1, 128, 128, P, P, P, P, P, None) == -1
    for at in range(6):
        args = [P] * 6
        args[at] = None
        off, a, sa, b, sb, out = args
        assert L.moe_fp8_gemm(off, 4, 1, 128, 128, a, sa, b, sb, out, None) == -1
    assert L.moe_fp8_gemm(P, 4, 1, 128, 128, odd, P, P, P, P, None) == -1
    assert L.moe_fp8_gemm(P, 2 ** 31 - 1, 1, 1 << 17, 128, P, P, P, P, P, None) == -1  # the grid
    assert L.moe_fp8_gemm(P, 0, 1, 128, 128, P, P, P, P, P, None) == 0  # no rows


@pytest.mark.skipif(torch.cuda.device_count() != 0,
                    reason="checks the no-device path; on a GPU host the calls would launch")
def test_good_arguments_reach_the_device_check():
    L = m.lib()
    g = m.make_gate(m.MOE_SCORE_SIGMOID, 4, 2, m.MOE_GROUP_TOP2)
    s = m.moe_query(CFG)
    Q = ctypes.c_void_p(1 << 21)
    assert L.moe_gate_select(_ref(CFG), _ref(g), P, None, P, P, None) == -4
    assert L.moe_route_gated(_ref(CFG), _ref(g), P, P, P, P, P, P, P, s.workspace, None) == -4
    assert L.moe_gate_backward(_ref(CFG), _ref(g), P, P, P, P, 1, None) == -4
    assert L.moe_router_backward(_ref(CFG), P, P, P, Q, None, 0, 0, None) == -4
    assert L.moe_router_backward(_ref(CFG), P, P, P, None, P, 0, 1, None) == -4
    assert L.moe_fp8_quantize_rows(P, 1, 128, P, P, None) == -4
    assert L.moe_fp8_quantize_weights(P, 1, 128, 128, P, P, None, None, None) == -4
    assert L.moe_fp8_gemm(P, 1, 1, 128, 128, P, P, P, P, P, None) == -4


# the plain forms -----------------------------------------------------------------------------


def test_gate_form_against_torch_on_the_plain_gates():
    l = torch.randn(40, 24, generator=torch.Generator().manual_seed(0), dtype=torch.float64)
    idx, w = _ops.gate(l.numpy(), 5, _ops.SOFTMAX)
    p, i = torch.softmax(l, 1).topk(5, dim=1)
    np.testing.assert_array_equal(idx, i.numpy())
    np.testing.assert_allclose(w, (p / p.sum(1, keepdim=True)).numpy(), rtol=1e-12)
    idx, w = _ops.gate(l.numpy(), 5, _ops.SIGMOID, renorm=False, scale=2.5)
    np.testing.assert_array_equal(idx, i.numpy())
    np.testing.assert_allclose(w, 2.5 * torch.sigmoid(l).gather(1, i).numpy(), rtol=1e-12)


def test_gate_form_on_worked_rows():
    inf = math.inf
    # ties go to the lower index; a closed expert comes last, with weight 0
    idx, w = _ops.gate(np.array([[1.0, 2.0, 2.0, -inf]]), 4, _ops.SIGMOID, renorm=False)
    assert idx.tolist() == [[1, 2, 0, 3]] and w[0, 3] == 0.0
    # a row of closed experts only
    idx, w = _ops.gate(np.full((1, 4), -inf), 2, _ops.SOFTMAX)
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]
    # the bias moves the choice and not the weights
    idx, w = _ops.gate(np.zeros((1, 4)), 1, _ops.SIGMOID, bias=[0, 0, 0, 1e-9], renorm=False)
    assert idx.tolist() == [[3]] and w.tolist() == [[0.5]]
    # group sums: 1.2 + 1.1 beats 2 + 0.1
    l = np.log(np.array([[2.0, 0.1, 1.2, 1.1]]) / 4.4)
    idx, _ = _ops.gate(l, 2, _ops.SOFTMAX, groups=2, group_score=_ops.GROUP_TOP2)
    assert idx.tolist() == [[2, 3]]
    idx, _ = _ops.gate(l, 2, _ops.SOFTMAX, groups=2, group_score=_ops.GROUP_MAX)
    assert idx.tolist() == [[0, 1]]


@pytest.mark.parametrize("score", [_ops.SOFTMAX, _ops.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradient_form_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.normal(size=(3, 12))
    idx = np.stack([rng.permutation(12)[:4] for _ in range(3)])
    idx[1, 2] = idx[1, 0]  # one expert twice
    idx[2, 3] = -1         # and a slot that names none
    dw = rng.normal(size=(3, 4))
    got = _ops.gate_backward(l, idx, dw, score, renorm, 2.5)
    f = lambda x: (_ops.gate_weights(x, idx, score, renorm, 2.5) * dw).sum()
    h = 1e-6
    for t in range(3):
        for e in range(12):
            d = np.zeros_like(l)
            d[t, e] = h
            # central differences: h^2 |f'''| / 6 + eps |f| / h, below 1e-8 for values of order 1
            assert abs((f(l + d) - f(l - d)) / (2 * h) - got[t, e]) < 1e-8


def test_e4m3_form_against_torch():
    v = torch.cat([torch.linspace(-460, 460, 4001), torch.linspace(-0.05, 0.05, 4001)])
    want = v.clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(_ops.e4m3(v.numpy()), want)


def test_fp8_mode_sizes_and_refusals():
    T, d, E, k, I = 300, 512, 16, 3, 256
    s8 = m.moe_query(m.make_cfg(T, d, E, k, I, m.MOE_PREC_FP8))
    s = m.moe_query(m.make_cfg(T, d, E, k, I))
    up = lambda v: (v + 255) // 256 * 256
    Tk = T * k
    assert s8.ring_slot == s.ring_slot and s8.saved == s.saved  # bf16 tokens and activations
    n1, n2 = E * 2 * I * d, E * d * I
    assert s8.wq == 2 * (up(n1) + up(4 * n1 // 16384) + up(n2) + up(4 * n2 // 16384))
    f = max(d, 2 * I)
    assert s8.workspace - s.workspace == up(Tk * f) + up(4 * Tk * f // 128) + up(2 * Tk * I)
    assert m.moe_query(m.make_cfg(T, d, E, k, I, m.MOE_PREC_FP8, m.MOE_FLAG_BF16_DW)).wq == s8.wq
    for flag in (m.MOE_FLAG_PERSISTENT, m.MOE_FLAG_MXFP8_WGRAD):
        with pytest.raises(m.MoeError) as ei:
            m.moe_query(m.make_cfg(T, d, E, k, I, m.MOE_PREC_FP8, flag))
        assert ei.value.status == -1
    L = m.lib()
    c = m.make_cfg(T, d, E, k, I, m.MOE_PREC_FP8)
    assert L.moe_forward_fused(_ref(c), P, P, P, P, P, P, s8.ring_slot, 0, P, P, P, P, P, P, P, P,
                               s8.saved, P, s8.workspace, None) == -3
    assert L.moe_quantize_weights(_ref(c), P, P, P, s8.wq - 1, None) == -5
    assert L.moe_forward(_ref(c), P, s8.ring_slot, 0, P, P, P, P, P, None, 0, P, P, s8.saved, P,
                         s8.workspace, None) == -1


def test_gated_layer_refuses_router_gradients_of_a_given_routing():
    from mixture_experts_layer_deterministic_amd import layer
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu", gate=m.make_gate())
    L.set_routing(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="no logits"):
        L.backward(x, x, x, x, x=x)


def test_single_launch_forward_is_refused_by_a_gated_layer(monkeypatch):
    """It routes by the top-k softmax, so the gate's gradients would be taken at another choice."""
    from mixture_experts_layer_deterministic_amd import layer
    launched = []
    monkeypatch.setattr(layer, "moe_forward_fused", lambda *a: launched.append(a))
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu", gate=m.make_gate())
    with pytest.raises(ValueError, match="top-k softmax"):
        L.forward_fused(x, x, x, x)
    with pytest.raises(ValueError, match="top-k softmax"):
        L.step(x, x, x, x, x, fused=True)
    assert not launched
    # a layer without a gate routes by it, and then has logits
    L = layer.MoeLayer(4, 256, 8, 2, 128, device="cpu")
    L.set_routing(torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    L.forward_fused(x, x, x, x)
    assert len(launched) == 1 and not L.given


def test_fp8_calls_take_empty_rows():
    """What a share without tokens passes: empty tensors, whose address is 0."""
    L = m.lib()
    e = ctypes.c_void_p(torch.empty(0, 128).data_ptr())
    assert e.value is None
    assert L.moe_fp8_quantize_rows(e, 0, 128, e, e, None) == 0
    assert L.moe_fp8_gemm(P, 0, 2, 128, 128, e, e, P, P, e, None) == 0
    # what is not empty, and the shapes, are checked all the same
    assert L.moe_fp8_quantize_rows(e, 0, 130, e, e, None) == -1
    assert L.moe_fp8_gemm(None, 0, 2, 128, 128, e, e, P, P, e, None) == -1
    assert L.moe_fp8_gemm(P, 0, 2, 128, 128, e, e, None, P, e, None) == -1
    assert L.moe_fp8_gemm(P, 0, 2, 100, 128, e, e, P, P, e, None) == -1
    assert L.moe_fp8_quantize_rows(e, 1, 128, e, e, None) == -1
    assert L.moe_fp8_gemm(P, 1, 2, 128, 128, e, P, P, P, P, None) == -1


def test_quantize_rows_refuses_a_grid_of_more_threads_than_a_launch_takes():
    L = m.lib()
    for rows, cols in ((2 ** 29, 128), (2 ** 29 - 31, 512), (2 ** 28, 640), (2 ** 22, 2 ** 16)):
        assert L.moe_fp8_quantize_rows(P, rows, cols, P, P, None) == -1
    if torch.cuda.device_count() == 0:  # a GPU would run it
        assert L.moe_fp8_quantize_rows(P, 2 ** 29 - 32, 128, P, P, None) == -4
