"""The dense gated feed-forward block on the GPU against 64-bit plain forms (tests/_products.py).

Tolerances, element by element. A sum of n products in fp32 is off by at most n half steps (F32) of
the sum of their magnitudes, whatever its order. What is stored in bf16 is off by half a step more.
A is compared through its g and u (gated_error); y with the product of the stored A; dH is internal,
so its own error (its sum, its activation, its rounding) goes through the products with the
magnitudes of what it meets."""
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


def _np(t):
    return t.double().cpu().numpy()


def _inputs(T, d, I, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF16)
    return dict(x=r(T, d), w1=r(2 * I, d, std=1.5 * d ** -0.5), w2=r(d, I, std=I ** -0.5),
                dy=r(T, d, std=0.3), y0=r(T, d), dx0=r(T, d), dw10=r(2 * I, d), dw20=r(d, I))


def _ws(c):
    return torch.empty(m.moe_ffn_query(c).workspace, dtype=torch.uint8, device=DEV)


def _forward(c, v, keep=True, acc=False, ws=None):
    T, d, I = c.T, c.d, c.I
    H = torch.full((T, 2 * I), 55.0, dtype=BF16, device=DEV) if keep else None
    A = torch.full((T, I), 55.0, dtype=BF16, device=DEV)
    y = v["y0"].clone() if acc else torch.full((T, d), 55.0, dtype=BF16, device=DEV)
    m.moe_ffn_forward(c, v["x"], v["w1"], v["w2"], H, A, y, acc, _ws(c) if ws is None else ws)
    return H, A, y


def _backward(c, v, H, A, acc=False, ws=None):
    dt = BF16 if c.flags else torch.float32
    if acc:
        dx, dw1, dw2 = v["dx0"].clone(), v["dw10"].to(dt), v["dw20"].to(dt)
        dw1, dw2 = dw1.clone(), dw2.clone()
    else:
        new = lambda *s, dt: torch.full(s, 55.0, dtype=dt, device=DEV)
        dx, dw1 = new(c.T, c.d, dt=BF16), new(2 * c.I, c.d, dt=dt)
        dw2 = new(c.d, c.I, dt=dt)
    m.moe_ffn_backward(c, v["x"], v["w1"], v["w2"], H, A, v["dy"], dx, dw1, dw2, acc, acc,
                       _ws(c) if ws is None else ws)
    return dx, dw1, dw2


def _near(got, want, err, bf16=True):
    e = err + (P64.BF16 * (np.abs(want) + err) if bf16 else 0.0) + 1e-37
    d = np.abs(_np(got) - want)
    assert np.isfinite(d).all() and (d <= e).all(), float((d / e).max())


def _check_forward(c, v, H, A, y, acc):
    x, w1, w2 = _np(v["x"]), _np(v["w1"]), _np(v["w2"])
    h, a, mag = P64.ffn_forward(x, w1, w2, c.act)
    eh = P64.F32 * c.d * mag
    if H is not None:
        _near(H, h, eh)
    (g, u), (eg, eu) = np.split(h, 2, axis=1), np.split(eh, 2, axis=1)
    _near(A, a, P64.gated_error(g, u, eg, eu))
    As = _np(A)
    yw, ey = As @ w2.T, P64.F32 * c.I * (np.abs(As) @ np.abs(w2).T)
    if acc:
        yw = yw + _np(v["y0"])
        ey = ey + P64.F32 * (np.abs(yw) + ey)
    _near(y, yw, ey)


def _check_backward(c, v, H, A, dx, dw1, dw2, acc):
    x, w1, w2, dy, Hs, As = (_np(t) for t in (v["x"], v["w1"], v["w2"], v["dy"], H, A))
    dh, dxw, dw1w, dw2w = P64.ffn_backward(x, w1, w2, Hs, As, dy, c.act)
    g, u = np.split(Hs, 2, axis=1)
    da = dy @ w2
    eda = P64.F32 * c.d * (np.abs(dy) @ np.abs(w2))
    # act and act' are off by (24 + 8 |g|) F32 of max(|g|, 1.2), as in gated_error
    ea = P64.F32 * (24 + 8 * np.abs(g)) * np.maximum(np.abs(g), 1.2)
    f, fg = np.abs(P64.act(c.act, g)), np.abs(P64.act_grad(c.act, g))
    edh = np.concatenate([np.abs(u) * (eda * (fg + ea) + np.abs(da) * ea),
                          eda * (f + ea) + np.abs(da) * ea], axis=1)
    edh = edh + (P64.BF16 + 4 * P64.F32) * (np.abs(dh) + edh)  # its products, and its rounding
    top = np.abs(dh) + edh
    edx = edh @ np.abs(w1) + P64.F32 * 2 * c.I * (top @ np.abs(w1))
    edw1 = edh.T @ np.abs(x) + P64.F32 * c.T * (top.T @ np.abs(x))
    edw2 = P64.F32 * c.T * (np.abs(dy).T @ np.abs(As))
    if acc:
        dxw, dw1w, dw2w = dxw + _np(v["dx0"]), dw1w + _np(v["dw10"]), dw2w + _np(v["dw20"])
    edx = edx + P64.F32 * (np.abs(dxw) + edx)
    edw1, edw2 = (e + P64.F32 * (np.abs(w) + e) for e, w in ((edw1, dw1w), (edw2, dw2w)))
    _near(dx, dxw, edx)
    _near(dw1, dw1w, edw1, bool(c.flags))
    _near(dw2, dw2w, edw2, bool(c.flags))


SHAPES = [(1, 128, 128), (2, 256, 128), (5, 384, 256), (15, 128, 384), (16, 512, 128),
          (17, 256, 640), (33, 640, 128), (63, 256, 256), (64, 384, 384), (65, 128, 128),
          (100, 512, 256), (129, 384, 128), (200, 256, 896), (256, 256, 256), (257, 640, 384),
          (333, 1024, 256), (513, 384, 512), (777, 256, 128), (3001, 128, 128), (2500, 384, 256)]


@pytest.mark.parametrize("T,d,I", SHAPES, ids=str)
@pytest.mark.parametrize("act", P64.ACTS)
def test_forward(T, d, I, act):
    _announce(f"[ffn] forward {T} x {d} x {I} act {act}")
    c = m.make_ffn(T, d, I, act)
    v = _inputs(T, d, I, T + d + I + act)
    H, A, y = _forward(c, v)
    _check_forward(c, v, H, A, y, False)
    _, A2, y2 = _forward(c, v, keep=False)
    assert torch.equal(A, A2) and torch.equal(y, y2)
    H, A3, y3 = _forward(c, v, acc=True)
    assert torch.equal(A, A3)
    _check_forward(c, v, H, A3, y3, True)


# few tokens: 16 and 32 columns of y a workgroup, 16 to 64 tokens, and either product too long for it
@pytest.mark.parametrize("T", [1, 4, 5, 16, 17, 31, 32, 33, 50, 64])
@pytest.mark.parametrize("d,I", [(6144, 128), (6272, 384), (1024, 1920), (128, 4096), (128, 8320),
                                 (2048, 4224)])
def test_few_tokens(T, d, I):
    test_forward(T, d, I, P64.ACTS[(T + I) % len(P64.ACTS)])


@pytest.mark.parametrize("T,d,I", SHAPES, ids=str)
@pytest.mark.parametrize("act,bf16_dw,acc", [(0, 0, False), (1, 4, True), (2, 0, True),
                                             (3, 4, False)])
def test_backward(T, d, I, act, bf16_dw, acc):
    _announce(f"[ffn] backward {T} x {d} x {I} act {act} flags {bf16_dw} acc {acc}")
    c = m.make_ffn(T, d, I, act, bf16_dw)
    v = _inputs(T, d, I, 3 * T + d + I + act)
    H, A, _ = _forward(c, v)
    out = _backward(c, v, H, A, acc)
    _check_backward(c, v, H, A, *out, acc)
    again = _backward(c, v, H, A, acc)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


@pytest.mark.parametrize("T,d,I", [(16, 7168, 2048), (300, 4096, 1408), (2048, 7168, 2048)], ids=str)
def test_large_shapes_by_norm(T, d, I):
    """At the layer's own sizes, against fp32 products: every stored value is within 2^-8 of its own
    size, dH's rounding included, so norms differ by no more than twice that."""
    _announce(f"[ffn] {T} x {d} x {I}")
    c = m.make_ffn(T, d, I, P64.SILU, m.MOE_FLAG_BF16_DW)
    v = _inputs(T, d, I, 1)
    H, A, y = _forward(c, v)
    x, w1, w2, dy = (v[k].float() for k in ("x", "w1", "w2", "dy"))
    h = x @ w1.t()
    g, u = h.split(I, dim=1)
    a = torch.nn.functional.silu(g) * u
    g, u = H.float().split(I, dim=1)
    s = torch.sigmoid(g)
    da = dy @ w2
    dh = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], dim=1)
    want = dict(H=h, A=a, y=a @ w2.t(), dx=dh @ w1, dw1=dh.t() @ x, dw2=dy.t() @ A.float())
    got = dict(zip(("dx", "dw1", "dw2"), _backward(c, v, H, A)), H=H, A=A, y=y)
    for k, w in want.items():
        assert (got[k].float() - w).norm() <= 2 * P64.BF16 * w.norm(), k


ACT64 = {P64.SILU: torch.nn.functional.silu, P64.GELU: torch.nn.functional.gelu,
         P64.GELU_TANH: lambda g: torch.nn.functional.gelu(g, approximate="tanh"),
         P64.RELU: torch.nn.functional.relu}


# sizes at which the products take their other tile shapes, whole rounds and the odd ends of both
@pytest.mark.parametrize("T,d,I,act", [(4096, 256, 2048, 0), (2100, 4096, 2048, 1),
                                       (4000, 4096, 256, 2), (1777, 1024, 1408, 3),
                                       (1000, 2304, 1920, 0), (300, 4096, 4096, 2)], ids=str)
def test_large_shapes_element_by_element(T, d, I, act):
    """The bounds of _check_forward and _check_backward, in 64 bits on the GPU."""
    _announce(f"[ffn] elements of {T} x {d} x {I} act {act}")
    c = m.make_ffn(T, d, I, act)
    v = _inputs(T, d, I, 11)
    H, A, y = _forward(c, v, acc=True)
    dx, dw1, dw2 = _backward(c, v, H, A, acc=True)
    x, w1, w2, dy, y0, dx0, dw10, dw20 = (v[k].double() for k in (
        "x", "w1", "w2", "dy", "y0", "dx0", "dw10", "dw20"))
    mm = lambda a, b: a @ b.contiguous()
    F32, HALF = P64.F32, P64.BF16

    def near(got, want, err, bf16=True):
        e = err + (HALF * (want.abs() + err) if bf16 else 0.0) + 1e-37
        r = ((got.double() - want).abs() / e).max().item()
        assert r <= 1.0, r

    def gate(g, u):
        g, u = g.clone().requires_grad_(True), u.clone().requires_grad_(True)
        f = ACT64[act](g)
        df, = torch.autograd.grad(f.sum(), g)
        return f.detach(), df

    h, eh = mm(x, w1.t()), F32 * d * mm(x.abs(), w1.abs().t())
    near(H, h, eh)
    (g, u), (eg, eu) = h.split(I, dim=1), eh.split(I, dim=1)
    ea = 1.2 * eg * u.abs() + g.abs() * eu + 1.2 * eg * eu + F32 * (24 + 8 * g.abs()) * (g * u).abs()
    near(A, gate(g, u)[0] * u, ea)
    As = A.double()
    yw, ey = mm(As, w2.t()) + y0, F32 * I * mm(As.abs(), w2.abs().t())
    near(y, yw, ey + F32 * (yw.abs() + ey))
    g, u = H.double().split(I, dim=1)
    f, df = gate(g, u)
    da, eda = mm(dy, w2), F32 * d * mm(dy.abs(), w2.abs())
    ea = F32 * (24 + 8 * g.abs()) * g.abs().clamp(min=1.2)
    dh = torch.cat([da * u * df, da * f], dim=1)
    edh = torch.cat([u.abs() * (eda * (df.abs() + ea) + da.abs() * ea),
                     eda * (f.abs() + ea) + da.abs() * ea], dim=1)
    edh = edh + (HALF + 4 * F32) * (dh.abs() + edh)
    top = dh.abs() + edh
    for got, want, err in (
            (dx, mm(dh, w1) + dx0, mm(edh, w1.abs()) + F32 * 2 * I * mm(top, w1.abs())),
            (dw1, mm(dh.t(), x) + dw10, mm(edh.t(), x.abs()) + F32 * T * mm(top.t(), x.abs())),
            (dw2, mm(dy.t(), As) + dw20, F32 * T * mm(dy.abs().t(), As.abs()))):
        near(got, want, err + F32 * (want.abs() + err), got.dtype == BF16)


def test_values_that_are_not_finite_stay_in_their_rows():
    T, d, I = 150, 256, 256
    c = m.make_ffn(T, d, I)
    v = _inputs(T, d, I, 2)
    H, A, y = _forward(c, v)
    clean = _backward(c, v, H, A)
    v["x"][7, 3], v["x"][140, 200] = float("inf"), float("nan")
    H2, A2, y2 = _forward(c, v)
    bad = torch.zeros(T, dtype=torch.bool, device=DEV)
    bad[[7, 140]] = True
    for t, u in ((H, H2), (A, A2), (y, y2)):
        assert torch.equal(t[~bad], u[~bad]) and not torch.isfinite(u[bad].float()).any()
    v["dy"][9, 0] = float("nan")
    dx, _, _ = _backward(c, v, H, A)
    assert torch.isnan(dx[9].float()).all()
    keep = torch.arange(T, device=DEV) != 9
    assert torch.equal(dx[keep], clean[0][keep])


@pytest.mark.parametrize("act", P64.ACTS)
@pytest.mark.parametrize("T", [3, 150])
def test_gates_of_any_magnitude_have_a_derivative(T, act):
    """act' is 0 or 1 to the last bit from |g| = 200 on, also where g * g is past fp32's range."""
    d, I = 256, 256
    c = m.make_ffn(T, d, I, act)
    v = _inputs(T, d, I, 6)
    v["w1"][I:] = 0  # dx from the gate's gradients alone
    H, A, _ = _forward(c, v)
    H[:, :I:2], H[:, 1:I:2], H[:, I:] = 200.0, -200.0, 0.5
    dx, dw1, _ = _backward(c, v, H, A)
    assert torch.isfinite(dx.float()).all() and (dx != 0).any()
    for far in (1e5, 1e13, 1e20, 1e30):
        H[:, :I:2], H[:, 1:I:2] = far, -far
        dx2, dw12, _ = _backward(c, v, H, A)
        assert torch.equal(dx, dx2) and torch.equal(dw1[:I], dw12[:I]), far


def test_what_lies_behind_the_last_token_is_left():
    """Buffers longer than T rows: rows behind stay, and are not read (they hold NaN)."""
    T, d, I, more = 70, 256, 384, 40
    c = m.make_ffn(T, d, I)
    v = _inputs(T, d, I, 4)
    H, A, y = _forward(c, v)
    out = _backward(c, v, H, A)
    long = {k: torch.full((T + more, t.shape[1]), float("nan"), dtype=BF16, device=DEV)
            for k, t in (("x", v["x"]), ("dy", v["dy"]), ("H", H), ("A", A), ("y", y),
                         ("dx", out[0]))}
    for k in ("x", "dy"):
        long[k][:T] = v[k]
    ws = _ws(c)
    m.moe_ffn_forward(c, long["x"], v["w1"], v["w2"], long["H"], long["A"], long["y"], False, ws)
    dw1, dw2 = torch.empty_like(out[1]), torch.empty_like(out[2])
    m.moe_ffn_backward(c, long["x"], v["w1"], v["w2"], long["H"], long["A"], long["dy"], long["dx"],
                       dw1, dw2, False, False, ws)
    for k, t in (("H", H), ("A", A), ("y", y), ("dx", out[0])):
        assert torch.equal(long[k][:T], t) and torch.isnan(long[k][T:].float()).all(), k
    assert torch.equal(dw1, out[1]) and torch.equal(dw2, out[2])


def test_two_streams_and_captured_graphs():
    """Two calls at once with a workspace each, and both directions in one graph, replayed with other
    inputs between eager calls."""
    c = m.make_ffn(130, 256, 256, P64.GELU)
    v, w = _inputs(130, 256, 256, 5), _inputs(130, 256, 256, 6)
    want = [_forward(c, i) for i in (v, w)]
    grads = [_backward(c, i, H, A) for i, (H, A, _) in zip((v, w), want)]
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for s, i in zip(streams, (v, w)):
        with torch.cuda.stream(s):
            H, A, y = _forward(c, i)
            outs.append(((H, A, y), _backward(c, i, H, A)))
    torch.cuda.synchronize()
    for (f, b), wf, wb in zip(outs, want, grads):
        assert all(torch.equal(p, q) for p, q in zip(f + b, wf + wb))
    ws = _ws(c)
    buf = {k: t.clone() for k, t in v.items()}
    g = torch.cuda.CUDAGraph()
    H, A, y = (torch.empty_like(t) for t in want[0])
    dx, dw1, dw2 = (torch.empty_like(t) for t in grads[0])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        m.moe_ffn_forward(c, buf["x"], buf["w1"], buf["w2"], H, A, y, False, ws)
        m.moe_ffn_backward(c, buf["x"], buf["w1"], buf["w2"], H, A, buf["dy"], dx, dw1, dw2, False,
                           False, ws)
    for n in range(4):
        src, wf, wb = ((v, want[0], grads[0]), (w, want[1], grads[1]))[n % 2]
        for k in buf:
            buf[k].copy_(src[k])
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((H, A, y, dx, dw1, dw2), wf + wb)), n
        _forward(c, v, ws=ws)  # the workspace serves an eager call between replays
        torch.cuda.synchronize()


def test_results_do_not_depend_on_what_the_workspace_held():
    c = m.make_ffn(40, 512, 256)
    v = _inputs(40, 512, 256, 8)
    outs = []
    for fill in (0, 255):
        ws = _ws(c).fill_(fill)
        H, A, y = _forward(c, v, ws=ws)
        ws.fill_(fill)
        outs.append((H, A, y, *_backward(c, v, H, A, ws=ws)))
    assert all(torch.equal(p, q) for p, q in zip(*outs))


def test_tensors_the_binding_refuses():
    c = m.make_ffn(20, 128, 128)
    v = _inputs(20, 128, 128, 3)
    H, A, y = _forward(c, v)
    ws = _ws(c)
    good = [c, v["x"], v["w1"], v["w2"], H, A, y, False, ws]
    for at, bad in ((1, v["x"].float()), (1, v["x"][:19]), (2, v["w1"].t()), (3, v["w2"].cpu()),
                    (4, H.half()), (5, A[:, ::2]), (8, ws.view(torch.int16))):
        args = list(good)
        args[at] = bad
        with pytest.raises(m.MoeError):
            m.moe_ffn_forward(*args)
    with pytest.raises(m.MoeError):  # fp32 gradients where the flag says bf16
        cb = m.make_ffn(20, 128, 128, 0, m.MOE_FLAG_BF16_DW)
        m.moe_ffn_backward(cb, v["x"], v["w1"], v["w2"], H, A, v["dy"], torch.empty_like(y),
                           torch.empty(256, 128, device=DEV), torch.empty(128, 128, device=DEV),
                           False, False, ws)
