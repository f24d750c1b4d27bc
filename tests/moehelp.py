"""Plain forms in 64 bits of the mixture-of-experts step and of the drawn token
(numpy, torch on the host), and inputs for their tests."""
import math

import numpy as np
import torch

from q8_quantized_gemv_gb300 import lk

U = 2.0 ** -24  # half a step of f32, relatively


# ---- routing -----------------------------------------------------------------------

def route_ref(logits, bias, score, n_group, top_group, group_sum, k, renorm, scale):
    """ids, weights and the smallest gap between two values that the choice
    went by (relative to their size; inf where it is exact)."""
    l = logits.astype(np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    M, E = l.shape
    ids, w = np.full((M, k), -1, np.int32), np.zeros((M, k))
    gap = math.inf
    for t in range(M):
        there = l[t] > -np.inf
        if not there.any():
            continue
        s = np.zeros(E)
        if score == "softmax":
            s[there] = np.exp(l[t][there] - l[t][there].max())
            s /= s.sum()
        else:
            s[there] = 1 / (1 + np.exp(-l[t][there]))
        b = np.zeros(E) if bias is None else bias.astype(np.float64)
        live = [i for i in range(E) if there[i] and np.isfinite(b[i])]
        c = {i: s[i] + b[i] if bias is not None else l[t][i] for i in live}
        if n_group > 1:
            per = E // n_group
            val = {}
            for g in range(n_group):
                v = sorted((s[i] if bias is None and group_sum == 2 else c[i] for i in live if i // per == g),
                           reverse=True)
                if v:
                    val[g] = math.fsum(v[:group_sum])
            order = sorted(val, key=lambda g: (-val[g], g))
            if len(order) > top_group and (bias is not None or group_sum == 2):
                x, y = val[order[top_group - 1]], val[order[top_group]]
                if x != y:
                    gap = min(gap, (x - y) / max(abs(x), abs(y), 1e-300))
            live = [i for i in live if i // per in order[:top_group]]
        order = sorted(live, key=lambda i: (-c[i], i))
        if bias is not None:
            for x, y in zip(order[:k], order[1:k + 1]):
                if c[x] != c[y]:
                    gap = min(gap, (c[x] - c[y]) / max(abs(c[x]), abs(c[y]), 1e-300))
        chosen = order[:k]
        if renorm and chosen:
            if score == "softmax":
                p = np.exp(l[t][chosen] - l[t][chosen].max())
            else:
                p = s[chosen]
            p = p / p.sum() if p.sum() > 0 else p
        else:
            p = s[chosen]
        ids[t, :len(chosen)] = chosen
        w[t, :len(chosen)] = scale * p
    return ids, w, gap


# ---- the experts' products -----------------------------------------------------------

def experts(E, rows, K, seed, dev):
    """A stack of Q8_0 matrices: (levels, scales)."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    q = torch.randint(-127, 128, (E, rows, K), generator=g, device=dev, dtype=torch.int8)
    s = torch.randn((E, rows, K // 32), generator=g, device=dev).mul_(0.02 / math.sqrt(K)).abs_().add_(1e-5)
    return q, s.to(torch.float16)


def value(q, s):
    """The values of levels and scales, in 64 bits."""
    return q.double() * s.double().repeat_interleave(32, -1)


def act_value(acts, mode):
    """The values that activation rows stand for, in 64 bits."""
    if mode == lk.LK_DEQUANT:
        return acts["x"].double()
    v = acts["xq"].double()
    if mode == lk.LK_TWOPASS:
        v = v + acts["xl"].double() / 128
    return v * acts["xs"].double().repeat_interleave(32, -1)


def dot_tol(mode, K):
    """|product - exact| over sum |w x|: Dequant's 1e-5; quantized, partial b mod 4
    takes K / 128 fused steps, each product of scales two roundings (TwoPass three),
    then two sums."""
    return 1e-5 if mode == lk.LK_DEQUANT else (K // 128 + 8) * U


def glu_ref(gate, up, acts, mode, ids, E):
    """h [M * k, F] in 64 bits, NaN for absent pairs, and its tolerance."""
    x = act_value(acts, mode)
    K, F = x.shape[1], gate[0].shape[1]
    h, tol = (torch.full((ids.numel(), F), math.nan, dtype=torch.float64, device=x.device) for _ in range(2))
    for p, e in enumerate(ids.flatten().tolist()):
        if not 0 <= e < E:
            continue
        row = x[p // ids.shape[1]]
        (g, ag), (u, au) = ((w @ row, w.abs() @ row.abs()) for w in (value(gate[0][e], gate[1][e]),
                                                                     value(up[0][e], up[1][e])))
        s = g * torch.sigmoid(g)
        h[p] = s * u
        eg, eu = (dot_tol(mode, K) * a + 2 * U * z.abs() for a, z in ((ag, g), (au, u)))
        # |silu'| <= 1.1; expf within 2 ulp and four roundings
        tol[p] = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 10 * U * (s * u).abs() + 1e-38
    return h, tol


def down_ref(down, acts, mode, ids, weights, E):
    """y [M, N] in 64 bits and its tolerance."""
    h = act_value(acts, mode)
    M, k = ids.shape
    N, F = down[0].shape[1:]
    y, tol, mag = (torch.zeros((M, N), dtype=torch.float64, device=h.device) for _ in range(3))
    for p, e in enumerate(ids.flatten().tolist()):
        if not 0 <= e < E:
            continue
        w, t = value(down[0][e], down[1][e]), p // k
        r = weights.flatten()[p].double()
        d = w @ h[p]
        y[t] += r * d
        tol[t] += r.abs() * (dot_tol(mode, F) * (w.abs() @ h[p].abs()) + 2 * U * d.abs())
        mag[t] += (r * d).abs()
    return y, tol + (k + 1) * U * mag + 1e-38


def quantize(x, mode):
    """Words and scales of rows x by lk_quantize_act, a batch of rows at a time."""
    n, K = x.shape
    d = {"xq": torch.zeros((n, K), dtype=torch.int8, device=x.device),
         "xs": torch.zeros((n, K // 32), dtype=torch.float32, device=x.device)}
    if mode == lk.LK_TWOPASS:
        d["xl"] = torch.zeros((n, K), dtype=torch.int8, device=x.device)
    for r in range(0, n, lk.LK_MAX_BATCH):
        s = slice(r, min(n, r + lk.LK_MAX_BATCH))
        lk.lk_quantize_act(x[s].contiguous(), mode, d["xq"][s], d["xl"][s] if "xl" in d else None, d["xs"][s])
    return d


def acts_of(x, mode):
    return {"x": x} if mode == lk.LK_DEQUANT else quantize(x, mode)


def as_h(acts):
    """Activation arguments under the names lk_moe_down_q8 gives them."""
    return {{"x": "h", "xq": "hq", "xl": "hl", "xs": "hs"}[n]: t for n, t in acts.items()}


# ---- the drawn token -----------------------------------------------------------------

def sample_ref(l, T, top_k, top_p, min_p, u):
    """(index, probability, margin) of one row: margin is how far, relatively,
    top_p and u are from the nearest border between tokens, and min_p from a
    token's weight."""
    l = l.astype(np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    order = np.lexsort((np.arange(l.size), -l))
    if l[order[0]] == -np.inf:
        return -1, 0.0, math.inf
    if not T > 0:
        return int(order[0]), 1.0, math.inf
    w = np.exp(np.maximum((l[order] - l[order[0]]) / T, -1e9))
    margin = math.inf
    if 0 < top_k < l.size:
        w = w[:top_k]
    if top_p < 1:
        c = np.cumsum(w)
        n = max(1, int(np.searchsorted(c, top_p * c[-1], "left")) + 1)
        margin = min(margin, float(np.abs(c[max(0, n - 2):n] - top_p * c[-1]).min() / c[-1]))
        w = w[:n]
    least = min(1.0, min_p)
    if least > 0:
        if least < 1:
            margin = min(margin, float(np.abs(w / least - 1).min()))
        w = w[w >= least]
    idx = np.sort(order[:w.size])
    at = np.argsort(order[:w.size])
    c = np.cumsum(w[at])
    i = min(int(np.searchsorted(c, max(0.0, u) * c[-1], "right")), int(np.nonzero(w[at])[0][-1]))
    if 0 < u < 1:
        # a border near u * total decides only if it lies above 0
        b = np.concatenate([[0.0], c[:-1]])[max(0, i):i + 1]
        near = [abs(float(c[i]) - u * c[-1])] + [abs(float(x) - u * c[-1]) for x in b if x > 0]
        margin = min(margin, min(near) / float(c[-1]))
    return int(idx[i]), float(w[at][i] / c[-1]), margin
