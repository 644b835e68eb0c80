"""MoeLayer.backward with a shared expert or a gate: what a later call would refuse is refused before
the experts' gradients are written or added to, so that a corrected call counts a batch once. And
MoeLayer.step, where there is no backward, before it does anything."""
import pytest
import torch

from tests._util import ensure_built

m = ensure_built()
BF16 = torch.bfloat16
T, d, E, k, I, S = 4, 256, 8, 2, 128, 384  # S: the shared expert's I


@pytest.fixture
def calls(monkeypatch):
    """The layer's calls by name; its tensor checks as on a GPU, but for the device."""
    from mixture_experts_layer_deterministic_amd import layer
    seen = []
    for name in ("moe_forward", "moe_backward", "moe_ffn_forward", "moe_ffn_backward",
                 "moe_gate_backward", "moe_router_backward", "moe_route", "moe_route_gated",
                 "moe_permute", "moe_forward_fused"):
        monkeypatch.setattr(layer, name, lambda *a, n=name: seen.append(n))

    def dev(what, stream, *args):
        for t, dtype, n in args:
            if t is not None and (t.dtype is not dtype or t.numel() < n or not t.is_contiguous()):
                raise m.MoeError(m.MOE_ERR_INVALID_ARG, what)

    monkeypatch.setattr(layer, "_dev", dev)
    return seen


def _bf(*shape, **kw):
    return torch.zeros(*shape, dtype=BF16, **kw)


def _odd(*shape):
    """Dense, but two bytes behind a multiple of sixteen."""
    n = torch.Size(shape).numel()
    return _bf(n + 8)[1:n + 1].view(shape)


def _layer(train=True, **over):
    from mixture_experts_layer_deterministic_amd import layer
    sh = layer.SharedExpert(T, d, S, device="cpu", train=train)
    return layer.MoeLayer(T, d, E, k, I, device="cpu", shared=sh, **over), sh


def _backward(L, **over):
    a = dict(wr=None, dy=_bf(T, d), x=_bf(T, d), sw=(_bf(2 * S, d), _bf(d, S)), saved=None, own=None)
    a.update(over)
    L.backward(a["wr"], _bf(E, 2 * I, d), _bf(E, d, I), a["dy"], 0, True, a["saved"], x=a["x"],
               shared_w=a["sw"], shared_saved=a["own"])


def test_a_shared_experts_operands_are_refused_before_any_gradient(calls):
    L, sh = _layer()
    own = lambda H, A: dict(saved=L.saved.clone(), own=(H, A))
    w1, w2 = _bf(2 * S, d), _bf(d, S)
    bad = [
        own(_bf(T, 2 * S - 128), _bf(T, S)),     # another I's H
        own(_bf(T - 1, 2 * S), _bf(T, S)),       # another T's
        own(_bf(T, 2 * S), _bf(T, S - 128)),
        own(_bf(T, 2 * S), None),                # no A, no H
        own(None, _bf(T, S)),
        own(_bf(T, 2 * S).float(), _bf(T, S)),
        own(_odd(T, 2 * S), _bf(T, S)),
        own(_bf(T, 2 * S), _odd(T, S)),
        dict(sw=(None, w2)), dict(sw=(w1, None)), dict(sw=(w1[:-1], w2)), dict(sw=(w1, w2.t())),
        dict(sw=(_odd(2 * S, d), w2)), dict(sw=(w1, _odd(d, S))),
        dict(x=_odd(T, d)), dict(x=_bf(T, d).float()), dict(dy=_odd(T, d)),
        dict(x=L.dx), dict(dy=L.dx),
    ]
    for i, over in enumerate(bad):
        with pytest.raises((ValueError, m.MoeError)):
            _backward(L, **over)
        assert not calls, (i, calls)
    _backward(L)
    _backward(L, **own(*sh.new_saved()))
    assert calls == ["moe_backward", "moe_ffn_backward"] * 2


def test_a_block_made_without_train_has_no_gradients_to_add_to(calls):
    """Also where a training block's saved is given to it."""
    L, _ = _layer(train=False)
    _, trained = _layer()
    with pytest.raises(ValueError, match="without train"):
        _backward(L, saved=L.saved.clone(), own=trained.new_saved())
    assert not calls


def test_gradients_of_another_type_or_size_are_refused(calls):
    L, sh = _layer()
    good = sh.dw1
    for bad in (good.to(BF16), good[:-1]):
        sh.dw1 = bad
        with pytest.raises(m.MoeError):
            _backward(L)
    sh.dw1, good = good, sh.dw2
    sh.dw2 = good.t()
    with pytest.raises(m.MoeError):
        _backward(L)
    assert not calls


def test_a_gated_layers_tokens_are_refused_before_any_gradient(calls):
    from mixture_experts_layer_deterministic_amd import layer
    L = layer.MoeLayer(T, d, E, k, I, device="cpu", gate=m.make_gate(m.MOE_SCORE_SIGMOID))
    wr = _bf(E, d)
    for over in (dict(x=_odd(T, d)), dict(x=L.dx), dict(wr=_odd(E, d)), dict(wr=wr[:-1])):
        with pytest.raises(m.MoeError):
            _backward(L, **{**dict(wr=wr), **over})
        assert not calls
    _backward(L, wr=wr)
    assert calls == ["moe_backward", "moe_gate_backward", "moe_router_backward"]


@pytest.mark.parametrize("fused", [False, True])
def test_a_step_without_a_backward_does_nothing(calls, fused):
    """step is a forward and a backward: a layer for inference, or one whose shared expert was made
    without train, refuses it before it routes or permutes."""
    from mixture_experts_layer_deterministic_amd import layer
    x, wr, w1, w2 = _bf(T, d), _bf(E, d), _bf(E, 2 * I, d), _bf(E, d, I)
    L = layer.MoeLayer(T, d, E, k, I, device="cpu", precision=m.MOE_PREC_INT8)
    with pytest.raises(ValueError, match="no backward"):
        L.step(x, wr, w1, w2, x, fused=fused)
    sw = (_bf(2 * S, d), _bf(d, S))
    L, _ = _layer(train=False)
    with pytest.raises(ValueError, match="without train"):
        L.step(x, wr, w1, w2, x, fused=fused, shared_w=sw)
    L, _ = _layer()
    with pytest.raises(ValueError, match="needs x and shared_w"):
        L.step(x, wr, w1, w2, x, fused=fused)
    assert not calls
    L.step(x, wr, w1, w2, _bf(T, d), fused=fused, shared_w=sw)
    assert calls == (["moe_forward_fused"] if fused else
                     ["moe_route", "moe_permute", "moe_forward"]) + [
        "moe_ffn_forward", "moe_backward", "moe_ffn_backward"]
