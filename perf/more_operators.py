"""What the layer's 8-bit integer operators and its dense gated feed-forward block are measured on.

Each case is one call of an operator on the layer's own shapes: the DeepSeek-V3-shaped layer
(T = 2048, d = 7168, E = 256, k = 8, I = 2048), the streaming layer (d = 4096, I = 1024), the local
expert slice (16384 rows over 8 experts, very uneven) and the small calls of serving. The
feed-forward block is the layer's shared expert, which every token passes beside its routed ones.
"""
import functools
import math

import torch

own = False

SILU, GELU, GELU_TANH, RELU = 0, 1, 2, 3


# ------------------------------------------------------------------------------------------
# Cases


def listed():
    return [
        # a serving step's tokens before the gate/up product: latency
        dict(name="i8_rows_decode", op="i8_rows", rows=24, cols=7168),
        # the permuted tokens of the DeepSeek-V3-shaped batch
        dict(name="i8_rows_dsv3", op="i8_rows", rows=16384, cols=7168),
        # the down weights of eight experts, a scale per output channel
        dict(name="i8_weights", op="i8_rows", rows=8 * 7168, cols=2048),
        # the down product of a few serving tokens on one expert-parallel share
        dict(name="i8_gemm_decode", op="i8_gemm", M=24, E=16, N=7168, K=2048, active=11, skew=0.0,
             tail=3),
        # the down product of the local expert slice: Zipf load, three experts empty
        dict(name="i8_gemm_slice", op="i8_gemm", M=16384, E=8, N=7168, K=2048, active=5, skew=1.2,
             tail=0),
        # the gated gate/up product of the DeepSeek-V3-shaped batch: about 64 rows an expert
        dict(name="i8_gated_dsv3", op="i8_gated", M=16384, E=256, I=2048, K=7168, active=256,
             skew=0.0, tail=0, act=SILU),
        # the gated gate/up product of the local expert slice
        dict(name="i8_gated_slice", op="i8_gated", M=16384, E=8, I=2048, K=7168, active=5,
             skew=1.2, tail=0, act=SILU),
        # the shared expert of a serving step
        dict(name="ffn_decode", op="ffn", T=16, d=7168, I=2048, act=SILU, train=False, acc=False),
        # the shared expert of the DeepSeek-V3-shaped training batch; H is kept for the backward
        dict(name="ffn_dsv3", op="ffn", T=2048, d=7168, I=2048, act=SILU, train=True, acc=False),
        # an odd prompt, another activation, added to the routed experts' output
        dict(name="ffn_odd", op="ffn", T=1777, d=4096, I=1408, act=GELU, train=False, acc=True),
        # the backward of ffn_dsv3
        dict(name="ffn_bwd_dsv3", op="ffn_bwd", T=2048, d=7168, I=2048, act=SILU, acc=False),
        # an odd microbatch of the streaming layer, added to the gradients of earlier ones
        dict(name="ffn_bwd_odd", op="ffn_bwd", T=333, d=4096, I=1024, act=GELU_TANH, acc=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["i8_rows", "i8_gemm", "i8_gemm", "i8_gated", "i8_gated", "ffn", "ffn", "ffn",
                     "ffn_bwd", "ffn_bwd", "ffn_bwd"])
    if op == "i8_rows":
        return dict(op=op, rows=_log_int(rng, 1, 16384), cols=128 * _log_int(rng, 1, 112))
    act = rng.choice([SILU, GELU, GELU_TANH, RELU])
    if op in ("i8_gemm", "i8_gated"):
        E = _log_int(rng, 1, 64)
        active = rng.randint(1, E)
        K, N = 128 * _log_int(rng, 1, 56), 128 * _log_int(rng, 1, 56 if op == "i8_gemm" else 16)
        M = min(_log_int(rng, active + 8, 16384), 16384 * 4096 * 7168 // (2 * N * K))
        c = dict(op=op, M=M, E=E, K=K, active=active, skew=rng.choice([0.0, 0.6, 1.2]),
                 tail=rng.choice([0, 0, 7]))
        return dict(c, N=N) if op == "i8_gemm" else dict(c, I=N, act=act)
    d, I = 128 * _log_int(rng, 2, 56), 128 * _log_int(rng, 1, 32)
    T = min(_log_int(rng, 1, 4096), 2048 * 2048 * 7168 * (1 if op == "ffn_bwd" else 2) // (d * I))
    c = dict(op=op, T=T, d=d, I=I, act=act, acc=rng.random() < 0.5)
    return dict(c, train=rng.random() < 0.5) if op == "ffn" else c


def work(case):
    op = case["op"]
    if op == "i8_rows":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + 4 * case["rows"], "flops": 0}
    if op in ("i8_gemm", "i8_gated"):
        M, K = case["M"] - case["tail"], case["K"]
        N, out = (case["N"], case["N"]) if op == "i8_gemm" else (2 * case["I"], case["I"])
        return {"bytes": M * K + 4 * M + case["active"] * (N * K + 4 * N) + 2 * M * out,
                "flops": 2 * M * N * K}
    T, d, I = case["T"], case["d"], case["I"]
    acc = 2 if case["acc"] else 1
    if op == "ffn":
        return {"bytes": 2 * (T * d + 3 * I * d + (3 if case["train"] else 1) * T * I
                              + acc * T * d), "flops": 6 * T * I * d}
    return {"bytes": 2 * (2 * T * d + 3 * I * d + 3 * T * I + acc * (T * d + 3 * I * d)),
            "flops": 12 * T * I * d}


# ------------------------------------------------------------------------------------------
# Inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _codes(x):
    """int8 codes of the rows of x, a scale each: the largest magnitude becomes 127."""
    v = x.double()
    amax = v.abs().amax(dim=-1, keepdim=True)
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    codes = torch.round(v * 127.0 / safe)  # v * 127 is exact: ties are ties, and go to even
    scales = torch.where(amax > 0, amax.float() / 127.0, torch.ones_like(amax).float())
    return codes.to(torch.int8), scales.squeeze(-1)


def _act(a, g):
    if a == SILU:
        return g / (1.0 + torch.exp(-g))
    if a == GELU:
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    if a == GELU_TANH:
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))
    return torch.where(g > 0, g, torch.zeros_like(g))


def _dact(a, g):
    if a == SILU:
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if a == GELU:
        return (0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
                + g * torch.exp(-0.5 * g * g) * math.sqrt(0.5 / math.pi))
    if a == GELU_TANH:
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)
    return torch.where(g > 0, torch.ones_like(g), torch.zeros_like(g))


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    s = dict(case)
    if op == "i8_rows":
        # activations: Gaussian with a few large columns
        x = torch.randn(case["rows"], case["cols"], generator=g, device="cuda")
        x *= 1 + 20 * (torch.rand(case["cols"], generator=g, device="cuda") < 0.005)
        s["x"] = x.to(torch.bfloat16)
    elif op in ("i8_gemm", "i8_gated"):
        M, E, K = case["M"], case["E"], case["K"]
        N = case["N"] if op == "i8_gemm" else 2 * case["I"]
        cpu = torch.Generator().manual_seed(seed * 7919 + 5)
        # the experts that get rows, their shares (rank^-skew) and the rows dealt over them
        chosen = torch.randperm(E, generator=cpu)[:case["active"]]
        share = torch.arange(1, case["active"] + 1, dtype=torch.float64) ** -case["skew"]
        rows = M - case["tail"] - case["active"]  # one row each, the rest by share
        dealt = torch.multinomial(share, max(rows, 1), replacement=True, generator=cpu)[:rows]
        counts = torch.zeros(E, dtype=torch.int64)
        counts[chosen] = 1 + torch.bincount(dealt, minlength=case["active"])
        s["cap"] = int(counts.max())
        used = counts.nonzero().view(-1)
        s["used"], s["used_at"] = used.cuda(), (counts > 0).cumsum(0).sub_(1).cuda()
        offsets = torch.zeros(E + 1, dtype=torch.int32)
        offsets[1:] = counts.cumsum(0)
        s["offsets"] = offsets.cuda()
        s["a"], s["sa"] = _codes(_randn(g, M, K))
        s["b"] = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
        s["sb"] = torch.empty(E, N, device="cuda")
        for e in range(E):  # gates and ups of a spread of about one
            s["b"][e], s["sb"][e] = _codes(_randn(g, N, K, std=K ** -0.5))
        # the caller's output: rows behind the last expert's stay as they are
        s["out"] = torch.zeros(M, N if op == "i8_gemm" else case["I"], device="cuda",
                               dtype=torch.bfloat16)
    else:
        T, d, I = case["T"], case["d"], case["I"]
        s["x"] = _randn(g, T, d)
        s["w1"] = _randn(g, 2 * I, d, std=d ** -0.5)  # the gate's rows, then the up projection's
        s["w2"] = _randn(g, d, I, std=I ** -0.5)
        if op == "ffn":
            s["y0"] = _randn(g, T, d) if case["acc"] else None  # the routed experts' output
        else:
            # what the forward kept: both projections and the hidden activations
            s["H"] = (s["x"].float() @ s["w1"].float().t()).to(torch.bfloat16)
            gate, up = s["H"].float().split(I, dim=1)
            s["A"] = (_act(case["act"], gate) * up).to(torch.bfloat16)
            s["dy"] = _randn(g, T, d, std=0.1)
            if case["acc"]:  # the routed experts' dx, and earlier microbatches' weight gradients
                s["dx0"] = _randn(g, T, d, std=0.1)
                s["dw10"], s["dw20"] = _randn(g, 2 * I, d), _randn(g, d, I)
    return s


# ------------------------------------------------------------------------------------------
# The plain forms


def _i8_rows_plain(s):
    codes, scales = _codes(s["x"])
    return {"codes": codes, "scales": scales}


def _product_plain(s):
    """The expert-grouped product's rows in fp32, before any rounding."""
    M, E, K, cap, n = s["M"], s["E"], s["K"], s["cap"], s["active"]
    rows, N = M - s["tail"], s["b"].shape[1]
    a = s["a"][:rows].float() * s["sa"][:rows, None]
    # the weights of the experts that have rows
    b = s["b"].index_select(0, s["used"]).float().mul_(s["sb"].index_select(0, s["used"])[..., None])
    # rows padded to the largest expert's, and back
    pos = torch.arange(rows, device=a.device)
    e = torch.bucketize(pos, s["offsets"][1:].long(), right=True)
    slot = s["used_at"][e] * cap + pos - s["offsets"][e]
    ap = a.new_zeros(n * cap, K).index_copy_(0, slot, a)
    return torch.bmm(ap.view(n, cap, K), b.transpose(1, 2)).view(n * cap, N).index_select(0, slot)


def _i8_gemm_plain(s):
    o = _product_plain(s)
    s["out"][:o.shape[0]] = o.to(torch.bfloat16)
    return {"out": s["out"]}


def _i8_gated_plain(s):
    g, u = _product_plain(s).split(s["I"], dim=1)
    s["out"][:g.shape[0]] = (_act(s["act"], g) * u).to(torch.bfloat16)
    return {"out": s["out"]}


def _ffn_plain(s):
    h = s["x"].float() @ s["w1"].float().t()
    gate, up = h.split(s["I"], dim=1)
    a = _act(s["act"], gate) * up
    y = a @ s["w2"].float().t()
    if s["acc"]:
        y = s["y0"].float() + y
    out = {"y": y.to(torch.bfloat16), "A": a.to(torch.bfloat16)}
    if s["train"]:
        out["H"] = h.to(torch.bfloat16)
    return out


def _ffn_bwd_plain(s):
    gate, up = s["H"].float().split(s["I"], dim=1)
    dy, w1 = s["dy"].float(), s["w1"].float()
    da = dy @ s["w2"].float()
    dh = torch.cat([da * up * _dact(s["act"], gate), da * _act(s["act"], gate)], dim=1)
    dx, dw1, dw2 = dh @ w1, dh.t() @ s["x"].float(), dy.t() @ s["A"].float()
    if s["acc"]:
        dx, dw1, dw2 = s["dx0"].float() + dx, s["dw10"].float() + dw1, s["dw20"].float() + dw2
    return {"dx": dx.to(torch.bfloat16), "dw1": dw1.to(torch.bfloat16),
            "dw2": dw2.to(torch.bfloat16)}


_PLAIN = {"i8_rows": _i8_rows_plain, "i8_gemm": _i8_gemm_plain, "i8_gated": _i8_gated_plain,
          "ffn": _ffn_plain, "ffn_bwd": _ffn_bwd_plain}


# ------------------------------------------------------------------------------------------
# The framework's calls


@functools.lru_cache(maxsize=16)
def _ffn(T, d, I, act, device, stream):
    """The block's shape and its workspace, which a program keeps as long as it keeps the shape, one
    for each device and stream: calls that share a workspace follow each other. Weight gradients
    are bf16, as dx is."""
    import mixture_experts_layer_deterministic_amd as m
    cfg = m.make_ffn(T, d, I, act, m.MOE_FLAG_BF16_DW)
    return cfg, torch.empty(m.moe_ffn_query(cfg).workspace, dtype=torch.uint8, device="cuda")


def _run_own(s):
    import mixture_experts_layer_deterministic_amd as m
    op = s["op"]
    if op == "i8_rows":
        codes = torch.empty(s["rows"], s["cols"], dtype=torch.int8, device="cuda")
        scales = torch.empty(s["rows"], device="cuda")
        m.moe_i8_quantize_rows(s["x"], s["rows"], s["cols"], codes, scales)
        return {"codes": codes, "scales": scales}
    if op == "i8_gemm":
        m.moe_i8_gemm(s["offsets"], s["M"], s["E"], s["N"], s["K"], s["a"], s["sa"], s["b"],
                      s["sb"], s["out"])
        return {"out": s["out"]}
    if op == "i8_gated":
        m.moe_i8_gemm_gated(s["offsets"], s["M"], s["E"], s["I"], s["K"], s["act"], s["a"],
                            s["sa"], s["b"], s["sb"], s["out"])
        return {"out": s["out"]}
    T, d, I = s["T"], s["d"], s["I"]
    cfg, ws = _ffn(T, d, I, s["act"], torch.cuda.current_device(),
                   torch.cuda.current_stream().cuda_stream)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    if op == "ffn":
        y = s["y0"].clone() if s["acc"] else torch.empty(T, d, **bf)
        out = {"y": y, "A": torch.empty(T, I, **bf)}
        if s["train"]:
            out["H"] = torch.empty(T, 2 * I, **bf)
        m.moe_ffn_forward(cfg, s["x"], s["w1"], s["w2"], out.get("H"), out["A"], y, s["acc"], ws)
        return out
    if s["acc"]:
        dx, dw1, dw2 = s["dx0"].clone(), s["dw10"].clone(), s["dw20"].clone()
    else:
        dx, dw1 = torch.empty(T, d, **bf), torch.empty(2 * I, d, **bf)
        dw2 = torch.empty(d, I, **bf)
    m.moe_ffn_backward(cfg, s["x"], s["w1"], s["w2"], s["H"], s["A"], s["dy"], dx, dw1, dw2,
                       s["acc"], s["acc"], ws)
    return {"dx": dx, "dw1": dw1, "dw2": dw2}


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits


def _gated64(act, g, u):
    """act(g) u and its two derivatives at each element, by autograd."""
    g, u = g.detach().requires_grad_(True), u.detach().requires_grad_(True)
    if act == SILU:
        f = g * torch.special.expit(g)
    elif act == GELU:
        f = g * torch.special.ndtr(g)
    elif act == GELU_TANH:
        z = math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3)
        f = g * torch.special.expit(z)
    else:
        f = torch.clamp(g, min=0.0)
    h = f * u
    dg, du = torch.autograd.grad(h.sum(), (g, u))
    return h.detach(), dg, du


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "i8_rows":
        return {"codes": None, "scales": torch.where(
            (s["x"] != 0).any(dim=1), s["x"].double().abs().amax(dim=1) / 127.0, 1.0)}
    if op in ("i8_gemm", "i8_gated"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        off = s["offsets"].tolist()
        for e in range(s["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                w = s["b"][e].double().t().contiguous() * s["sb"][e].double()
                p = s["sa"][lo:hi].double()[:, None] * (s["a"][lo:hi].double() @ w)
                if op == "i8_gated":
                    p = _gated64(s["act"], p[:, :s["I"]], p[:, s["I"]:])[0]
                out[lo:hi] = p
        return {"out": out}
    x, w1, w2, I = s["x"].double(), s["w1"].double(), s["w2"].double(), s["I"]
    if op == "ffn":
        h = x @ w1.t().contiguous()
        a = _gated64(s["act"], h[:, :I], h[:, I:])[0]
        y = a @ w2.t().contiguous()
        out = {"y": y + s["y0"].double() if s["acc"] else y, "A": a}
        if s["train"]:
            out["H"] = h
        return out
    _, dg, du = _gated64(s["act"], s["H"][:, :I].double(), s["H"][:, I:].double())
    dy = s["dy"].double()
    da = dy @ w2
    dh = torch.cat([da * dg, da * du], dim=1)
    out = {"dx": dh @ w1, "dw1": dh.t().contiguous() @ x,
           "dw2": dy.t().contiguous() @ s["A"].double()}
    if s["acc"]:
        for k, v in (("dx", "dx0"), ("dw1", "dw10"), ("dw2", "dw20")):
            out[k] = out[k] + s[v].double()
    return out
