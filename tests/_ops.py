"""Plain 64-bit forms of the gate, the router gradients and the block-scaled FP8 operators (numpy
only), written from their definitions, for the tests."""
import numpy as np

SOFTMAX, SIGMOID = 0, 1
GROUP_MAX, GROUP_TOP2 = 0, 1


def scores(l, score):
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, np.float64))
    if score == SIGMOID:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    out = np.zeros_like(l)
    for t, row in enumerate(l):
        m = row.max()
        if m == -np.inf:
            continue
        with np.errstate(invalid="ignore"):
            e = np.where(row == m, 1.0, np.exp(row - m))
        out[t] = e / e.sum()
    return out


def gate(l, k, score, bias=None, groups=1, topk_groups=1, group_score=GROUP_MAX, renorm=True,
         scale=1.0):
    """(idx, w) of every row, one choice after the other in Python's own order of sorting."""
    l = np.where(np.isnan(l), -np.inf, np.asarray(l, np.float64))
    T, E = l.shape
    s = scores(l, score)
    if bias is not None:
        c = s + np.asarray(bias, np.float64)
    elif groups > 1 and group_score == GROUP_TOP2:
        c = s
    else:
        c = l
    c = np.where(l == -np.inf, -np.inf, c)
    gs = E // groups
    idx = np.empty((T, k), np.int64)
    w = np.empty((T, k))
    for t in range(T):
        stay = range(groups)
        if groups > 1:
            val = []
            for g in range(groups):
                part = sorted(c[t, g * gs:(g + 1) * gs], reverse=True)
                v = part[0]
                if group_score == GROUP_TOP2 and gs > 1 and part[1] != -np.inf:
                    v += part[1]
                val.append(v)
            stay = sorted(range(groups), key=lambda g: (-val[g], g))[:topk_groups]
        cand = [e for g in stay for e in range(g * gs, (g + 1) * gs)]
        best = sorted(cand, key=lambda e: (-c[t, e], e))[:k]
        p = s[t, best]
        if renorm:
            p = p / p.sum() if p.sum() > 0 else np.zeros(k)
        idx[t], w[t] = best, scale * p
    return idx, w


def gate_weights(l, idx, score, renorm, scale):
    """The weights of a given choice (entries outside [0, E) weigh nothing)."""
    s = scores(l, score)
    E = l.shape[1]
    ok = (idx >= 0) & (idx < E)
    p = np.where(ok, np.take_along_axis(s, np.where(ok, idx, 0), axis=1), 0.0)
    if renorm:
        z = p.sum(axis=1, keepdims=True)
        p = np.where(z > 0, p / np.where(z > 0, z, 1.0), 0.0)
    return scale * p


def gate_backward(l, idx, dw, score, renorm, scale):
    """d <w, dw> / dl through the Jacobian of the weights, slot by slot."""
    l = np.asarray(l, np.float64)
    T, E = l.shape
    s = scores(l, score)
    out = np.zeros((T, E))
    for t in range(T):
        slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
        p = np.array([s[t, idx[t, j]] for j in slots])
        g = scale * np.array([float(dw[t, j]) for j in slots])
        if renorm:  # d/ds_i of sum_j g_j s_j / S
            S = p.sum()
            ds = (g - (g * p).sum() / S) / S if S > 0 else np.zeros(len(slots))
        else:
            ds = g
        dse = np.zeros(E)
        for i, j in enumerate(slots):
            dse[idx[t, j]] += ds[i]
        if score == SIGMOID:
            out[t] = dse * s[t] * (1 - s[t])
        else:
            out[t] = s[t] * (dse - (dse * s[t]).sum())
    return out


def e4m3(v):
    """v rounded to the nearest E4M3 value, ties to even, saturated at 448."""
    v = np.asarray(v, np.float64)
    ex = np.clip(np.frexp(v)[1] - 1, -6, None) - 3
    return np.clip(np.ldexp(np.rint(np.ldexp(v, -ex)), ex), -448.0, 448.0)


def quantize(x, block_rows):
    """(values the codes stand for before the scale, scales) in the operators' own arithmetic:
    fp32 scale amax / 448 and fp32 factor 448 / amax (amax at least 2^-110 unless 0), the product
    rounded to fp32, then to E4M3."""
    x = np.asarray(x, np.float32)
    *b, R, K = x.shape
    v = x.reshape(*b, R // block_rows, block_rows, K // 128, 128)
    amax = np.abs(v).max(axis=(-3, -1), keepdims=True)
    one = np.float32(1)
    safe = np.where(amax > 0, np.maximum(amax, np.float32(2.0 ** -110)), one)
    inv = np.where(amax > 0, np.float32(448) / safe, one)
    scale = np.where(amax > 0, safe / np.float32(448), one)
    return e4m3(v * inv).reshape(x.shape), scale.reshape(*b, R // block_rows, K // 128)


def fp8_gemm(offsets, a, sa, b, sb):
    """a [M, K], sa [K / 128, M], b [E, N, K], sb [E, N / 128, K / 128] as values; rows outside the
    experts' are NaN."""
    M, K = a.shape
    E, N, _ = b.shape
    out = np.full((M, N), np.nan)
    av = a * np.repeat(np.asarray(sa, np.float64).T, 128, axis=1)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        if hi > lo:
            w = b[e] * np.repeat(np.repeat(np.asarray(sb[e], np.float64), 128, 0), 128, 1)
            out[lo:hi] = av[lo:hi] @ w.T
    return out


# the layer in FP8 mode -----------------------------------------------------------------------


def bf16(x):
    """Rounded to bfloat16, nearest, ties to even."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(
        np.float64)


def _image(x, block_rows):
    """The values the quantised x stands for."""
    q, s = quantize(x, block_rows)
    *b, R, K = x.shape
    return (q.reshape(*b, R // block_rows, block_rows, K // 128, 128)
            * np.asarray(s, np.float64)[..., :, None, :, None]).reshape(x.shape)


def fp8_layer(X, W1, W2, dY, idx, w):
    """Forward and backward of the FP8 mode with a given routing, in 64 bits, rounded and quantised
    where the library stores: rows of experts in turn, each token's slots at the end."""
    T, k = idx.shape
    E, twoI, d = W1.shape
    I = twoI // 2
    out = dict(Y=np.zeros((T, d)), dX=np.zeros((T, d)), dW1=np.zeros(W1.shape),
               dW2=np.zeros(W2.shape), dw=np.zeros((T, k)))
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if not len(t):
            continue
        x, wt = X[t], w[t, j][:, None].astype(np.float64)
        q1, q2 = _image(W1[e], 128), _image(W2[e], 128)
        H = bf16(_image(x, 1) @ q1.T)
        g, u = H[:, :I], H[:, I:]
        s = 1.0 / (1.0 + np.exp(-g))
        A = bf16(g * s * u)
        O = bf16(_image(A, 1) @ q2.T)
        dap = bf16(_image(dY[t], 1) @ q2)
        out["dw"][t, j] = (dap * A).sum(1)
        da = wt * dap
        dH = bf16(np.concatenate([da * u * s * (1 + g * (1 - s)), da * g * s], axis=1))
        dXp = bf16(_image(dH, 1) @ q1)
        out["dW1"][e] = dH.T @ x
        out["dW2"][e] = bf16(wt * dY[t]).T @ A
        np.add.at(out["Y"], t, wt * O)
        np.add.at(out["dX"], t, dXp)
    return out
