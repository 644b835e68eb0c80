"""What the layer's gate, router-gradient and block-scaled 8-bit operators are measured on.

Each case is one call (or, for a quantiser, one call) of an operator on the layer's own shapes:
the DeepSeek-V3-shaped layer (T = 2048, d = 7168, E = 256, k = 8, I = 2048), the streaming layer
(microbatches of 2368 tokens, d = 4096, E = 512, k = 10, I = 1024), the local expert slice (16384
rows over 8 experts, very uneven) and the small calls of serving.
"""
import functools
import math

import torch

own = False

SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


# ------------------------------------------------------------------------------------------
# Cases


def listed():
    return [
        # one serving step's tokens through the DeepSeek-V3-shaped gate: latency
        dict(name="gate_decode", op="gate", T=16, E=256, k=8, score=SIGMOID, bias=True, groups=8,
             topk_groups=4, group_score=GROUP_TOP2, renorm=True, scale=2.5, closed=False),
        # the training batch of the DeepSeek-V3-shaped layer
        dict(name="gate_dsv3", op="gate", T=2048, E=256, k=8, score=SIGMOID, bias=True, groups=8,
             topk_groups=4, group_score=GROUP_TOP2, renorm=True, scale=2.5, closed=False),
        # a whole macrobatch of the streaming layer through a plain softmax gate
        dict(name="gate_stream", op="gate", T=18944, E=512, k=10, score=SOFTMAX, bias=False,
             groups=1, topk_groups=1, group_score=GROUP_MAX, renorm=False, scale=1.0, closed=False),
        # the backward of gate_dsv3: gradients at the selected experts only
        dict(name="gate_bwd_dsv3", op="gate_bwd", T=2048, E=256, k=8, score=SIGMOID, renorm=True,
             scale=2.5, closed=False),
        # the backward of gate_stream: every logit has a gradient
        dict(name="gate_bwd_stream", op="gate_bwd", T=18944, E=512, k=10, score=SOFTMAX,
             renorm=False, scale=1.0, closed=False),
        # router gradients of the DeepSeek-V3-shaped training batch
        dict(name="router_bwd_dsv3", op="router_bwd", T=2048, d=7168, E=256, sparse=8,
             accumulate=True),
        # an odd batch and an odd number of experts, every logit with a gradient
        dict(name="router_bwd_odd", op="router_bwd", T=1777, d=4096, E=509, sparse=0,
             accumulate=False),
        # the permuted tokens of the DeepSeek-V3-shaped batch, before the gate/up product
        dict(name="quant_rows", op="quant_rows", rows=16384, cols=7168),
        # gate/up weights of eight experts after an optimizer step, both orientations
        dict(name="quant_weights", op="quant_weights", E=8, N=4096, K=7168),
        # the down product of a few serving tokens on one expert-parallel share
        dict(name="gemm_decode", op="gemm", M=24, E=16, N=7168, K=2048, active=11, skew=0.0,
             tail=3),
        # the gate/up product of the DeepSeek-V3-shaped batch: about 64 rows an expert
        dict(name="gemm_dsv3", op="gemm", M=16384, E=256, N=4096, K=7168, active=256, skew=0.0,
             tail=0),
        # the gate/up product of the local expert slice: Zipf load, three experts empty
        dict(name="gemm_slice", op="gemm", M=16384, E=8, N=4096, K=7168, active=5, skew=1.2,
             tail=0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_gate(rng, T):
    groups = rng.choice([1, 1, 2, 4, 8, 16])
    E = groups * _log_int(rng, 4, 1024 // groups if groups > 1 else 512)
    E = min(E, 1024 // groups * groups)
    topk_groups = rng.randint(1, groups)
    k = rng.randint(1, min(16, topk_groups * (E // groups)))
    T = max(1, min(T, 18944 * 512 // E))
    score = rng.choice([SOFTMAX, SIGMOID])
    return dict(T=T, E=E, k=k, score=score, bias=rng.random() < 0.6, groups=groups,
                topk_groups=topk_groups, group_score=rng.choice([GROUP_MAX, GROUP_TOP2]),
                renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                closed=rng.random() < 0.3)


def draw(rng):
    op = rng.choice(["gate", "gate", "gate_bwd", "router_bwd", "quant_rows", "quant_weights",
                     "gemm", "gemm", "gemm"])
    if op == "gate":
        return dict(op=op, **_draw_gate(rng, _log_int(rng, 1, 18944)))
    if op == "gate_bwd":
        c = _draw_gate(rng, _log_int(rng, 1, 18944))
        return dict(op=op, T=c["T"], E=c["E"], k=c["k"], score=c["score"], renorm=c["renorm"],
                    scale=c["scale"], closed=c["closed"])
    if op == "router_bwd":
        E = _log_int(rng, 2, 512)
        return dict(op=op, T=_log_int(rng, 1, 2400), d=256 * _log_int(rng, 1, 28), E=E,
                    sparse=rng.choice([0, min(8, E)]), accumulate=rng.random() < 0.5)
    if op == "quant_rows":
        return dict(op=op, rows=_log_int(rng, 1, 16384), cols=128 * _log_int(rng, 1, 56))
    if op == "quant_weights":
        return dict(op=op, E=rng.randint(1, 8), N=128 * _log_int(rng, 1, 32),
                    K=128 * _log_int(rng, 1, 56))
    E = _log_int(rng, 1, 64)
    active = rng.randint(1, E)
    return dict(op=op, M=_log_int(rng, active + 8, 16384), E=E, N=128 * _log_int(rng, 1, 32),
                K=128 * _log_int(rng, 1, 56), active=active, skew=rng.choice([0.0, 0.6, 1.2]),
                tail=rng.choice([0, 0, 7]))


def work(case):
    op = case["op"]
    if op == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 0}
    if op == "gate_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        dense = case["score"] == SOFTMAX and not case["renorm"]
        return {"bytes": 4 * T * E + 8 * T * k + 4 * T * (E if dense else k), "flops": 0}
    if op == "router_bwd":
        T, d, E = case["T"], case["d"], case["E"]
        acc = 2 if case["accumulate"] else 1
        return {"bytes": 4 * T * E + 2 * T * d + 2 * E * d + acc * (2 * T * d + 4 * E * d),
                "flops": 4 * T * E * d}
    if op == "quant_rows":
        n = case["rows"] * case["cols"]
        return {"bytes": 3 * n + n // 32, "flops": 0}
    if op == "quant_weights":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": 4 * n + 8 * (n // 16384), "flops": 0}
    M, N, K = case["M"] - case["tail"], case["N"], case["K"]
    return {"bytes": M * K + M * K // 32 + case["active"] * (N * K + N * K // 4096)
            + 2 * M * N, "flops": 2 * M * N * K}


# ------------------------------------------------------------------------------------------
# Inputs


def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _logits(case, g):
    # router logits of Gaussian tokens: a spread of about 1.7
    l = _randn(g, case["T"], case["E"], std=1.7)
    if case["closed"]:  # experts that may not be chosen
        l.masked_fill_(torch.rand(l.shape, generator=g, device="cuda") < 0.1, -math.inf)
    return l


def _codes(w, block_rows):
    """E4M3 codes and fp32 scales of w [.., R, K], a scale per block of block_rows x 128."""
    *b, R, K = w.shape
    v = w.float().view(*b, R // block_rows, block_rows, K // 128, 128)
    amax = v.abs().amax(dim=(-3, -1), keepdim=True)
    one = torch.ones_like(amax)
    q = (v * torch.where(amax > 0, 448.0 / amax, one)).clamp_(-448.0, 448.0)
    s = torch.where(amax > 0, amax / 448.0, one)
    return (q.reshape(w.shape).to(torch.float8_e4m3fn),
            s.view(*b, R // block_rows, K // 128))


def prepare(case, seed):
    g = _generator(case, seed)
    op = case["op"]
    s = dict(case)
    if op == "gate":
        s["logits"] = _logits(case, g)
        s["b"] = _randn(g, case["E"], std=0.05) if case["bias"] else None
    elif op == "gate_bwd":
        s["logits"] = _logits(case, g)
        # the choice the forward made: the k largest logits
        s["idx"] = s["logits"].topk(case["k"], dim=1).indices.to(torch.int32)
        s["dw"] = _randn(g, case["T"], case["k"])
    elif op == "router_bwd":
        T, d, E = case["T"], case["d"], case["E"]
        s["x"] = _randn(g, T, d, dtype=torch.bfloat16)
        s["wr"] = _randn(g, E, d, std=0.02, dtype=torch.bfloat16)
        dl = _randn(g, T, E, std=0.1)
        if case["sparse"]:  # gradients at the selected experts only
            keep = torch.rand(T, E, generator=g, device="cuda").topk(case["sparse"], dim=1).indices
            dl = torch.zeros_like(dl).scatter_(1, keep, dl.gather(1, keep))
        s["dl"] = dl
        # what the experts' backward left in dx, and earlier microbatches in dwr
        s["dx0"] = _randn(g, T, d, dtype=torch.bfloat16)
        s["dwr0"] = _randn(g, E, d)
    elif op == "quant_rows":
        # activations: Gaussian with a few large columns
        x = _randn(g, case["rows"], case["cols"])
        x *= 1 + 20 * (torch.rand(case["cols"], generator=g, device="cuda") < 0.005)
        s["x"] = x.to(torch.bfloat16)
    elif op == "quant_weights":
        s["w"] = _randn(g, case["E"], case["N"], case["K"], std=0.02, dtype=torch.bfloat16)
    else:
        M, E, N, K = case["M"], case["E"], case["N"], case["K"]
        cpu = torch.Generator().manual_seed(seed * 7919 + 3)
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
        a, sa = _codes(_randn(g, M, K), 1)
        s["a"], s["sa"] = a, sa.t().contiguous()  # one row of scales per K block
        s["b"] = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["sb"] = torch.empty(E, N // 128, K // 128, device="cuda")
        for e in range(E):
            s["b"][e], s["sb"][e] = _codes(_randn(g, N, K, std=0.02), 128)
        # the caller's output: rows behind the last expert's stay as they are
        s["out"] = torch.zeros(M, N, device="cuda", dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------------------------------
# The plain forms


def _scores(l, score):
    """Scores in 64 bits; a closed expert (-inf) scores 0."""
    l = l.double()
    if score == SIGMOID:
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    z = e.sum(dim=1, keepdim=True)
    return torch.where(z > 0, e / z, torch.zeros_like(e))


def _gate_plain(s):
    l, k, G = s["logits"], s["k"], s["groups"]
    T, E = l.shape
    closed = l == -math.inf
    p = _scores(l, s["score"])
    # without a bias and without sums of scores the order of the scores is that of the logits
    by_logit = s["b"] is None and (G == 1 or s["group_score"] == GROUP_MAX)
    c = l.double() if by_logit else p if s["b"] is None else p + s["b"].double()
    c = c.masked_fill(closed, -math.inf)
    if G > 1:
        cg = c.view(T, G, E // G)
        if s["group_score"] == GROUP_MAX or E == G:
            gs = cg.amax(dim=2)
        else:
            top = cg.sort(dim=2, descending=True).values[..., :2]
            gs = top[..., 0] + torch.where(top[..., 1] == -math.inf, 0.0, top[..., 1])
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        usable = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, best, True)
        usable = usable.repeat_interleave(E // G, dim=1)
    else:
        usable = torch.ones_like(closed)
    # the usable experts first, each part by choice score, equal ones by index
    order = c.sort(dim=1, descending=True, stable=True).indices
    order = order.gather(1, usable.gather(1, order).int().sort(
        dim=1, descending=True, stable=True).indices)
    idx = order[:, :k]
    w = p.gather(1, idx)
    if s["renorm"]:
        z = w.sum(dim=1, keepdim=True)
        w = torch.where(z > 0, w / z, torch.zeros_like(w))
    return {"idx": idx.to(torch.int32), "w": (w * s["scale"]).float()}


def _gate_bwd_plain(s):
    l, idx, dw = s["logits"], s["idx"].long(), s["dw"]
    g = s["scale"] * dw
    if s["score"] == SIGMOID:
        p = 1.0 / (1.0 + torch.exp(-l.gather(1, idx)))
        if s["renorm"]:
            z = p.sum(dim=1, keepdim=True)
            z = torch.where(z > 0, z, torch.ones_like(z))
            g = (g - (g * p / z).sum(dim=1, keepdim=True)) / z
        return {"dlogits": torch.zeros_like(l).scatter_(1, idx, g * p * (1.0 - p))}
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    if s["renorm"]:
        q = e.gather(1, idx)
        z = q.sum(dim=1, keepdim=True)
        q = q / torch.where(z > 0, z, torch.ones_like(z))
        return {"dlogits": torch.zeros_like(l).scatter_(
            1, idx, q * (g - (g * q).sum(dim=1, keepdim=True)))}
    z = e.sum(dim=1, keepdim=True)
    p = e / torch.where(z > 0, z, torch.ones_like(z))
    dp = torch.zeros_like(l).scatter_(1, idx, g)
    return {"dlogits": p * (dp - (p * dp).sum(dim=1, keepdim=True))}


def _router_bwd_plain(s):
    dl = s["dl"]
    dx = dl @ s["wr"].float()
    dwr = dl.t() @ s["x"].float()
    if s["accumulate"]:
        dx, dwr = s["dx0"].float() + dx, s["dwr0"] + dwr
    return {"dx": dx.to(torch.bfloat16), "dwr": dwr}


def _quant_rows_plain(s):
    q, sc = _codes(s["x"], 1)
    return {"codes": q, "scales": sc.t().contiguous()}


def _quant_weights_plain(s):
    q, sc = _codes(s["w"], 128)
    return {"codes": q, "scales": sc, "codes_t": q.transpose(1, 2).contiguous(),
            "scales_t": sc.transpose(1, 2).contiguous()}


def _gemm_plain(s):
    M, N, K, cap, n = s["M"], s["N"], s["K"], s["cap"], s["active"]
    rows = M - s["tail"]
    a = (s["a"][:rows].float().view(rows, K // 128, 128) * s["sa"].t()[:rows, :, None]).view(rows, K)
    # the weights of the experts that have rows
    sb = s["sb"].index_select(0, s["used"])[:, :, None, :, None]
    b = s["b"].view(torch.uint8).index_select(0, s["used"]).view(torch.float8_e4m3fn).float()
    b = b.view(n, N // 128, 128, K // 128, 128).mul_(sb).view(n, N, K)
    # rows padded to the largest expert's, and back; rows behind the last expert's stay
    pos = torch.arange(rows, device=a.device)
    e = torch.bucketize(pos, s["offsets"][1:].long(), right=True)
    slot = s["used_at"][e] * cap + pos - s["offsets"][e]
    ap = a.new_zeros(n * cap, K).index_copy_(0, slot, a)
    o = torch.bmm(ap.view(n, cap, K), b.transpose(1, 2)).view(n * cap, N)
    s["out"][:rows] = o.index_select(0, slot).to(torch.bfloat16)
    return {"out": s["out"]}


_PLAIN = {"gate": _gate_plain, "gate_bwd": _gate_bwd_plain, "router_bwd": _router_bwd_plain,
          "quant_rows": _quant_rows_plain, "quant_weights": _quant_weights_plain,
          "gemm": _gemm_plain}


# ------------------------------------------------------------------------------------------
# The framework's calls


@functools.lru_cache(maxsize=None)
def _cfg(T, E, k, d):
    import mixture_experts_layer_deterministic_amd as m
    return m.make_cfg(T, d, E, k, 128)


@functools.lru_cache(maxsize=None)
def _gate(score, groups, topk_groups, group_score, renorm, scale):
    import mixture_experts_layer_deterministic_amd as m
    return m.make_gate(score, groups, topk_groups, group_score, renorm, scale)


def _run_own(s):
    import mixture_experts_layer_deterministic_amd as m
    op = s["op"]
    if op == "gate":
        T, E, k = s["T"], s["E"], s["k"]
        idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
        w = torch.empty(T, k, device="cuda")
        m.moe_gate_select(_cfg(T, E, k, 256),
                          _gate(s["score"], s["groups"], s["topk_groups"], s["group_score"],
                                s["renorm"], s["scale"]), s["logits"], s["b"], idx, w)
        return {"idx": idx, "w": w}
    if op == "gate_bwd":
        T, E, k = s["T"], s["E"], s["k"]
        dl = torch.empty(T, E, device="cuda")
        m.moe_gate_backward(_cfg(T, E, k, 256),
                            _gate(s["score"], 1, 1, GROUP_MAX, s["renorm"], s["scale"]),
                            s["logits"], s["idx"], s["dw"], dl, False)
        return {"dlogits": dl}
    if op == "router_bwd":
        acc = s["accumulate"]
        dx = s["dx0"].clone() if acc else torch.empty_like(s["dx0"])
        dwr = s["dwr0"].clone() if acc else torch.empty_like(s["dwr0"])
        m.moe_router_backward(_cfg(s["T"], s["E"], 1, s["d"]), s["x"], s["wr"], s["dl"], dx, dwr,
                              acc, acc)
        return {"dx": dx, "dwr": dwr}
    if op == "quant_rows":
        R, C = s["rows"], s["cols"]
        q = torch.empty(R, C, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty(C // 128, R, device="cuda")
        m.moe_fp8_quantize_rows(s["x"], R, C, q, sc)
        return {"codes": q, "scales": sc}
    if op == "quant_weights":
        E, N, K = s["E"], s["N"], s["K"]
        q = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
        qt = torch.empty(E, K, N, dtype=torch.float8_e4m3fn, device="cuda")
        sc = torch.empty(E, N // 128, K // 128, device="cuda")
        sct = torch.empty(E, K // 128, N // 128, device="cuda")
        m.moe_fp8_quantize_weights(s["w"], E, N, K, q, sc, qt, sct)
        return {"codes": q, "scales": sc, "codes_t": qt, "scales_t": sct}
    m.moe_fp8_gemm(s["offsets"], s["M"], s["E"], s["N"], s["K"], s["a"], s["sa"], s["b"], s["sb"],
                   s["out"])
    return {"out": s["out"]}


def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------------------
# The definitions in 64 bits


def _exact_gate(s):
    l = s["logits"].double()
    if s["score"] == SIGMOID:
        p = torch.sigmoid(l)
    else:
        p = torch.nan_to_num(torch.softmax(l, dim=1), nan=0.0)
    c = p if s["b"] is None else p + s["b"].double()
    if s["b"] is None and (s["groups"] == 1 or s["group_score"] == GROUP_MAX):
        c = l
    c = torch.where(l == -math.inf, -math.inf, c).cpu().numpy()
    # one expert after the other: the largest that is left, argmax gives the lowest index
    T, E = c.shape
    G = s["groups"]
    import numpy as np
    key = c.copy()
    if G > 1:
        part = np.sort(c.reshape(T, G, E // G), axis=2)[..., ::-1]
        gs = part[..., 0]
        if s["group_score"] == GROUP_TOP2 and E > G:
            gs = gs + np.where(np.isinf(part[..., 1]), 0.0, part[..., 1])
        take = np.argsort(-gs, axis=1, kind="stable")[:, :s["topk_groups"]]
        ok = np.zeros((T, G), bool)
        np.put_along_axis(ok, take, True, axis=1)
        ok = np.repeat(ok, E // G, axis=1)
    else:
        ok = np.ones((T, E), bool)
    # closed but usable experts come behind the open ones and before the unusable
    key = np.where(ok, np.where(np.isinf(key), -1e300, key), -np.inf)
    rows = np.arange(T)
    idx = np.empty((T, s["k"]), np.int64)
    for j in range(s["k"]):
        idx[:, j] = key.argmax(axis=1)
        key[rows, idx[:, j]] = -np.inf
    w = np.take_along_axis(p.cpu().numpy(), idx, axis=1)
    if s["renorm"]:
        z = w.sum(axis=1, keepdims=True)
        w = w / np.where(z > 0, z, 1.0)
    return {"idx": None, "w": w * s["scale"]}


def _exact_gate_bwd(s):
    l = s["logits"].double()
    closed = l == -math.inf
    # rows of closed experts only have no softmax: any finite row stands in, its gradient is 0
    dead = closed.all(dim=1, keepdim=True)
    l = torch.where(dead, torch.zeros_like(l), l).requires_grad_(True)
    idx = s["idx"].long()
    p = torch.sigmoid(l) if s["score"] == SIGMOID else torch.softmax(l, dim=1)
    w = p.gather(1, idx)
    if s["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    (s["scale"] * w * s["dw"].double()).sum().backward()
    return {"dlogits": torch.nan_to_num(l.grad, nan=0.0).masked_fill(closed, 0.0)}


def _exact_router_bwd(s):
    dl = s["dl"].double()
    dx, dwr = torch.matmul(dl, s["wr"].double()), torch.matmul(dl.t().contiguous(), s["x"].double())
    if s["accumulate"]:
        dx, dwr = dx + s["dx0"].double(), dwr + s["dwr0"].double()
    return {"dx": dx, "dwr": dwr}


def _e4m3(v):
    """v (64 bits) rounded to the nearest E4M3 value, ties to even, saturated at 448."""
    _, ex = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(ex - 1, min=-6) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_quant(w, block_rows):
    *b, R, K = w.shape
    v = w.double().reshape(*b, R // block_rows, block_rows, K // 128, 128)
    s = v.abs().amax(dim=(-3, -1), keepdim=True) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return _e4m3(v / s).view(w.shape), s.reshape(*b, R // block_rows, K // 128)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "gate":
        return _exact_gate(s)
    if op == "gate_bwd":
        return _exact_gate_bwd(s)
    if op == "router_bwd":
        return _exact_router_bwd(s)
    if op == "quant_rows":
        q, sc = _exact_quant(s["x"], 1)
        return {"codes": q, "scales": sc.t().contiguous()}
    if op == "quant_weights":
        q, sc = _exact_quant(s["w"], 128)
        return {"codes": q, "scales": sc, "codes_t": q.transpose(1, 2).contiguous(),
                "scales_t": sc.transpose(1, 2).contiguous()}
    if work(case)["flops"] > 3e11:
        return None  # over 20 seconds in 64 bits
    M, K, N = s["M"], s["K"], s["N"]
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    off = s["offsets"].tolist()
    sa = s["sa"].double().t().repeat_interleave(128, dim=1)
    a = s["a"].double() * sa
    for e in range(s["E"]):
        if off[e + 1] > off[e]:
            sb = s["sb"][e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
            w = (s["b"][e].double() * sb).t().contiguous()
            out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ w
    return {"out": out}
