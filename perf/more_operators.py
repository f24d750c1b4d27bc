"""Measured cases of the steps of a mixture-of-experts decoder's token that
the dense one lacks: routing a row to its experts (lk_moe_route), the experts'
gate/up products with SwiGLU (lk_moe_glu_q8), their down products summed by
the routing weights (lk_moe_down_q8), and the next token drawn from the logits
(lk_sample).

``run`` computes them in plain torch operations, or, where ``own`` is set, by
the library's calls.  Expert matrices are Q8_0: int8 levels [experts, rows, K]
and one f16 scale per 32 values; a pair is one of the k experts of a row.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
MODES = ("dequant", "int8act", "twopass")


# ---- the cases ---------------------------------------------------------------------

def listed():
    return [
        # one decode token: the launch latency is all there is
        dict(name="route 1 of 128", op="route", M=1, E=128, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             group_sum=1, renorm=True, scale=1.0, masked=False),
        # a full decode batch, experts chosen within groups by biased scores
        dict(name="route 64 of 256 in groups", op="route", M=64, E=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, group_sum=2, renorm=True, scale=2.5, masked=False),
        # an odd number of experts, some switched off, padding rows
        dict(name="route 33 of 60 masked", op="route", M=33, E=60, k=4, score="softmax", bias=True, groups=1,
             top_groups=1, group_sum=1, renorm=False, scale=1.0, masked=True),
        # one decode token: eight experts' matrices streamed for one row
        dict(name="glu 1 row int8act", op="glu", mode="int8act", M=1, E=128, k=8, K=4096, F=1024, padding=False),
        # a full decode batch: most experts are touched, a few rows each
        dict(name="glu 64 rows int8act", op="glu", mode="int8act", M=64, E=128, k=8, K=4096, F=1024, padding=False),
        # a small ragged batch in two words, smaller experts, odd widths
        dict(name="glu 5 rows twopass", op="glu", mode="twopass", M=5, E=60, k=4, K=2048, F=1408, padding=True),
        # the same steps behind the gate/up products
        dict(name="down 1 row int8act", op="down", mode="int8act", M=1, E=128, k=8, K=1024, F=4096, padding=False),
        dict(name="down 64 rows int8act", op="down", mode="int8act", M=64, E=128, k=8, K=1024, F=4096, padding=False),
        # few large experts, f32 activations, a ragged batch
        dict(name="down 7 rows dequant", op="down", mode="dequant", M=7, E=8, k=2, K=2048, F=5120, padding=True),
        # one decode token: latency
        dict(name="sample 1 x 151936", op="sample", M=1, N=151936, T=0.7, top_k=40, top_p=0.9, min_p=0.05,
             mixed=False),
        # a full batch, the nucleus of a large vocabulary
        dict(name="sample 64 x 151936 top-p", op="sample", M=64, N=151936, T=1.0, top_k=0, top_p=0.95, min_p=0.0,
             mixed=False),
        # an odd vocabulary, every row with settings of its own
        dict(name="sample 17 x 32003 mixed", op="sample", M=17, N=32003, T=1.3, top_k=500, top_p=0.99, min_p=0.01,
             mixed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "glu", "down", "sample"])
    if op == "sample":
        return dict(op=op, M=_log(rng, 1, 64), N=_log(rng, 1000, 151936), T=round(rng.uniform(0.3, 2.0), 3),
                    top_k=rng.choice([0, 0, 1, _log(rng, 2, 2000)]), top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.999), 3)]),
                    min_p=rng.choice([0.0, round(rng.uniform(0.001, 0.2), 3)]), mixed=rng.random() < 0.4)
    E, M = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 256]), _log(rng, 1, 64)
    if op == "route":
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 4])
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, E // groups * top))
        return dict(op=op, M=M, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=top, group_sum=rng.choice([1, 2]), renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5]), masked=rng.random() < 0.3)
    mode, k = rng.choice(MODES), rng.randint(1, 8)
    if mode == "dequant":
        M = min(M, 8)
    # K: the products' length, F: the output rows of an expert (of the gate and the up matrix each)
    K, F = (_log(rng, 4, 40) * 128, _log(rng, 2, 16) * 128) if op == "glu" else (_log(rng, 2, 16) * 128, _log(rng, 4, 40) * 128)
    most = (1 << 30) // (K * F * (2 if op == "glu" else 1))
    return dict(op=op, mode=mode, M=M, E=max(8, min(E, most)), k=k, K=K, F=F, padding=rng.random() < 0.3)


def _ids(case):
    """The experts of every row, [M, k]: distinct in a row, some experts more
    popular than others; with `padding` every fifth row has none (-1)."""
    r = np.random.RandomState(case["M"] * 4099 + case["E"] * 17 + case["k"])
    score = 0.5 * r.randn(case["E"])[None] + r.gumbel(size=(case["M"], case["E"]))
    ids = np.argsort(-score, axis=1)[:, :case["k"]].astype(np.int32)
    if case["padding"]:
        ids[3::5] = -1
    return ids


def work(case):
    if case["op"] == "route":
        M, E, k = case["M"], case["E"], case["k"]
        return {"bytes": 4 * M * E + (4 * E if case["bias"] else 0) + 8 * M * k, "flops": 8 * M * E}
    if case["op"] == "sample":
        return {"bytes": 4 * case["M"] * case["N"] + 28 * case["M"], "flops": 6 * case["M"] * case["N"]}
    ids = _ids(case)
    pairs, touched = int((ids >= 0).sum()), len(np.unique(ids[ids >= 0]))
    K, F = case["K"], case["F"]
    act = {"dequant": 4.0, "int8act": 1.125, "twopass": 2.125}[case["mode"]] * K
    if case["op"] == "glu":
        rows = int((ids >= 0).any(1).sum())
        return {"bytes": touched * 2 * F * K * 1.0625 + rows * act + 4 * pairs * F + 4 * ids.size,
                "flops": 4.0 * pairs * F * K}
    return {"bytes": touched * F * K * 1.0625 + pairs * act + 4.0 * case["M"] * F + 8 * ids.size,
            "flops": 2.0 * pairs * F * K}


# ---- inputs ------------------------------------------------------------------------

def _matrix(g, E, N, K):
    """Q8_0 expert matrices: levels [E, N, K], scales [E, N, K / 32]."""
    q = torch.randint(-127, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    s = torch.randn((E, N, K // 32), generator=g, device=DEV).mul_(0.02 / math.sqrt(K)).abs_().add_(1e-5)
    return q, s.to(torch.float16)


def _words(x, mode):
    """x [rows, K] as activation words: (xq, xl or None, xs)."""
    b = x.view(x.shape[0], -1, 32)
    a = b.abs().amax(-1)
    if mode == "int8act":
        s = torch.where(a >= 127 * 2.0 ** -126, a / torch.full_like(a, 127.0), torch.ones_like(a))
        hi = torch.round(b / s[..., None])
        return hi.to(torch.int8).view(x.shape), None, s
    s = a.clamp(min=1e-30) / torch.full_like(a, 127.0)
    hi = torch.round(b / s[..., None]).clamp(-128, 127)
    res = (b.double() - hi.double() * s[..., None].double()).float()
    lo = torch.round(res / (s / 128)[..., None]).clamp(-128, 127)
    return hi.to(torch.int8).view(x.shape), lo.to(torch.int8).view(x.shape), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    M = case["M"]
    if case["op"] == "route":
        E = case["E"]
        s["logits"] = torch.randn((M, E), generator=g, device=DEV).mul_(1.5)
        s["b"] = 0.1 * torch.randn((E,), generator=g, device=DEV) if case["bias"] else None
        if case["masked"]:
            s["logits"][:, torch.randperm(E, generator=g, device=DEV)[:E // 8]] = -math.inf
            s["logits"][4::7] = -math.inf
        s["ids"] = torch.zeros((M, case["k"]), dtype=torch.int32, device=DEV)
        s["weights"] = torch.zeros((M, case["k"]), device=DEV)
        return s
    if case["op"] == "sample":
        N = case["N"]
        # a few likely tokens and a long tail, in no order of the vocabulary
        rank = torch.argsort(torch.rand((M, N), generator=g, device=DEV), -1).float().add_(1)
        s["logits"] = torch.randn((M, N), generator=g, device=DEV).sub_(1.1 * torch.log(rank)).add_(12)
        of = torch.rand((4, M), generator=g, device=DEV) if case["mixed"] else torch.ones((4, M), device=DEV)
        s["T"] = case["T"] * of[0]
        s["tk"] = (case["top_k"] * of[1]).ceil().to(torch.int32)
        s["tp"] = 1 - (1 - case["top_p"]) * of[2]
        s["mp"] = case["min_p"] * of[3]
        if case["mixed"]:
            s["T"][3::5] = 0
            s["tk"][1::3] = 0
            s["tp"][2::3] = 1
        s["u"] = torch.rand((M,), generator=g, device=DEV)
        s["idx"] = torch.zeros((M,), dtype=torch.int32, device=DEV)
        s["prob"] = torch.zeros((M,), device=DEV)
        return s
    E, K, F, k, mode = case["E"], case["K"], case["F"], case["k"], case["mode"]
    s["ids"] = torch.from_numpy(_ids(case)).to(DEV)
    if case["op"] == "glu":
        s["wg"], s["wsg"] = _matrix(g, E, F, K)
        s["wu"], s["wsu"] = _matrix(g, E, F, K)
        x = torch.randn((M, K), generator=g, device=DEV)
        x = torch.where(torch.rand((M, K), generator=g, device=DEV) < 0.01, x * 20, x)
        s["out"] = torch.zeros((M * k, F), device=DEV)
    else:
        s["wd"], s["wsd"] = _matrix(g, E, F, K)
        a, b = torch.randn((2, M * k, K), generator=g, device=DEV)
        x = a / (1 + torch.exp(-a)) * b
        s["weights"] = torch.softmax(torch.randn((M, k), generator=g, device=DEV), -1)
        s["out"] = torch.zeros((M, F), device=DEV)
    s["x"], s["xq"], s["xl"], s["xs"] = (x, None, None, None) if mode == "dequant" else (None, *_words(x, mode))
    if own:
        from q8_quantized_gemv_gb300 import lk
        s["experts"] = lk.Experts(gate=(s["wg"], s["wsg"]), up=(s["wu"], s["wsu"])) if case["op"] == "glu" else \
            lk.Experts(down=(s["wd"], s["wsd"]))
    return s


# ---- the calls and their plain forms -----------------------------------------------

def _run_route(s):
    if own:
        from q8_quantized_gemv_gb300 import lk
        lk.lk_moe_route(s["logits"], s["ids"], s["weights"], bias=s["b"], score=s["score"], n_group=s["groups"],
                        top_group=s["top_groups"], group_sum=s["group_sum"], renorm=s["renorm"], scale=s["scale"])
        return {"ids": s["ids"], "weights": s["weights"]}
    M, E, k = s["M"], s["E"], s["k"]
    l = s["logits"].double()
    out = l == -math.inf
    if s["score"] == "softmax":
        m = l.amax(-1, keepdim=True)
        e = torch.exp(l - torch.where(m > -math.inf, m, torch.zeros_like(m)))
        p = e / e.sum(-1, keepdim=True).clamp(min=1e-300)
    else:
        p = 1 / (1 + torch.exp(-l))
    # what the choice goes by: without a bias the order of the scores, which is that of the logits
    c = p + s["b"].double() if s["b"] is not None else p
    c = torch.where(out, torch.full_like(c, -math.inf), c)
    if s["groups"] > 1:
        # a group's value: its largest one or two, those that are not there as nothing
        top = torch.sort(c.view(M, s["groups"], -1), dim=-1, descending=True)[0]
        some = top[..., 0] > -math.inf
        top = top[..., :s["group_sum"]]
        val = torch.where(top > -math.inf, top, torch.zeros_like(top)).sum(-1)
        val = torch.where(some, val, torch.full_like(val, -math.inf))
        order = torch.sort(val, dim=-1, descending=True, stable=True)[1]
        rank = torch.argsort(order, -1)
        c = torch.where((rank < s["top_groups"]).repeat_interleave(E // s["groups"], 1), c, torch.full_like(c, -math.inf))
    v, i = torch.sort(c, dim=-1, descending=True, stable=True)
    there, i = v[:, :k] > -math.inf, i[:, :k]
    w = torch.where(there, p.gather(1, i), torch.zeros_like(v[:, :k]))
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return {"ids": torch.where(there, i, torch.full_like(i, -1)).to(torch.int32), "weights": (w * s["scale"]).float()}


def _value(q, sc):
    """Levels times their scales, in f32."""
    return (q.float().view(*sc.shape, 32) * sc.float()[..., None]).view(q.shape)


def _acts(s):
    if s["mode"] == "dequant":
        return s["x"]
    x = s["xq"].float()
    if s["mode"] == "twopass":
        x = x + s["xl"].float() / 128
    return (x.view(*s["xs"].shape, 32) * s["xs"][..., None]).view(s["xq"].shape)


def _products(s, w, ws, x, per_pair):
    """The products of every pair's expert with its row of x: [M * k, rows].
    Few pairs: their experts' matrices; many: all of them, each read once."""
    M, k, E = s["M"], s["k"], s["E"]
    ids = s["ids"].long().clamp(min=0).flatten()
    if M * k <= E:
        x = x if per_pair else x.repeat_interleave(k, 0)
        return torch.bmm(_value(w[ids], ws[ids]), x[..., None])[..., 0]
    y = torch.matmul(x, _value(w, ws).transpose(-1, -2))
    return y[ids, torch.arange(M * k, device=DEV) if per_pair else torch.arange(M, device=DEV).repeat_interleave(k)]


def _run_glu(s):
    if own:
        from q8_quantized_gemv_gb300 import lk
        lk.lk_moe_glu_q8(s["experts"], s["mode"], s["ids"], s["out"], x=s["x"], xq=s["xq"], xl=s["xl"], xs=s["xs"])
        return s["out"]
    x = _acts(s)
    g, u = _products(s, s["wg"], s["wsg"], x, False), _products(s, s["wu"], s["wsu"], x, False)
    h = g / (1 + torch.exp(-g)) * u
    return torch.where((s["ids"] >= 0).view(-1, 1), h, torch.zeros_like(h))


def _run_down(s):
    if own:
        from q8_quantized_gemv_gb300 import lk
        lk.lk_moe_down_q8(s["experts"], s["mode"], s["ids"], s["weights"], s["out"], h=s["x"], hq=s["xq"], hl=s["xl"],
                          hs=s["xs"])
        return s["out"]
    d = _products(s, s["wd"], s["wsd"], _acts(s), True).view(s["M"], s["k"], -1)
    w = torch.where(s["ids"] >= 0, s["weights"], torch.zeros_like(s["weights"]))
    return (w[..., None] * d).sum(1)


def _run_sample(s):
    if own:
        from q8_quantized_gemv_gb300 import lk
        lk.lk_sample(s["logits"], s["u"], s["idx"], prob=s["prob"], temperature=s["T"], top_k=s["tk"], top_p=s["tp"],
                     min_p=s["mp"])
        return {"idx": s["idx"], "prob": s["prob"]}
    l, N = s["logits"].double(), s["N"]
    m, first = l.max(-1, keepdim=True)[0], (s["logits"] == s["logits"].amax(-1, keepdim=True)).int().argmax(-1)
    T = s["T"].double()[:, None]
    cold = T <= 0
    e = torch.exp((l - m) / torch.where(cold, torch.ones_like(T), T))
    order = torch.sort(s["logits"], dim=-1, descending=True, stable=True)[1]
    z = e.gather(1, order)
    tk = s["tk"][:, None]
    tk = torch.where(tk > 0, tk, torch.full_like(tk, N))
    z = torch.where(torch.arange(N, device=DEV) < tk, z, torch.zeros_like(z))
    c = z.cumsum(-1)
    tp = s["tp"].double()[:, None]
    # a token stays while those before it have not reached the share
    keep = (c - z < tp * c[:, -1:]) | (tp >= 1)
    keep[:, 0] = True
    z = torch.where(keep & (z >= s["mp"].double()[:, None].clamp(max=1)), z, torch.zeros_like(z))
    kept = torch.zeros_like(z).scatter_(1, order, z)
    c = kept.cumsum(-1)
    idx = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(-1)
    prob = kept.gather(1, idx[:, None])[:, 0] / c[:, -1]
    idx = torch.where(cold[:, 0], first, idx)
    return {"idx": idx.to(torch.int32), "prob": torch.where(cold[:, 0], torch.ones_like(prob), prob).float()}


def run(state):
    return {"route": _run_route, "glu": _run_glu, "down": _run_down, "sample": _run_sample}[state["op"]](state)


# ---- the definitions in 64 bits ----------------------------------------------------

def _exact_route(case, s):
    l, b = s["logits"].cpu().numpy().astype(np.float64), None if s["b"] is None else s["b"].cpu().numpy().astype(np.float64)
    k, per = case["k"], case["E"] // case["groups"]
    ids, weights = np.full((case["M"], k), -1, np.int32), np.zeros((case["M"], k))
    for t in range(case["M"]):
        live = [i for i in range(case["E"]) if l[t, i] > -np.inf]
        if not live:
            continue
        p = {i: 1 / (1 + math.exp(-l[t, i])) for i in live}
        if case["score"] == "softmax":
            total = math.fsum(math.exp(l[t, j] - l[t].max()) for j in live)
            p = {i: math.exp(l[t, i] - l[t].max()) / total for i in live}
        by = {i: p[i] + (b[i] if b is not None else 0.0) for i in live}
        if case["groups"] > 1:
            worth = {}
            for i in live:
                worth.setdefault(i // per, []).append(by[i])
            worth = {n: math.fsum(sorted(v)[-case["group_sum"]:]) for n, v in worth.items()}
            best = sorted(worth, key=lambda n: (-worth[n], n))[:case["top_groups"]]
            live = [i for i in live if i // per in best]
        chosen = sorted(live, key=lambda i: (-by[i], i))[:k]
        over = math.fsum(p[i] for i in chosen) if case["renorm"] else 1.0
        for j, i in enumerate(chosen):
            ids[t, j], weights[t, j] = i, case["scale"] * p[i] / over
    return {"ids": ids, "weights": weights}


def _exact_sample(case, s):
    n = {a: s[a].cpu().numpy().astype(np.float64) for a in ("logits", "T", "tk", "tp", "mp", "u")}
    idx, prob = np.zeros(case["M"], np.int32), np.zeros(case["M"])
    for t in range(case["M"]):
        l = n["logits"][t]
        order = np.lexsort((np.arange(l.size), -l))
        if n["T"][t] <= 0:
            idx[t], prob[t] = order[0], 1.0
            continue
        w = np.exp((l[order] - l[order[0]]) / n["T"][t])
        if 0 < n["tk"][t] < l.size:
            w = w[:int(n["tk"][t])]
        if n["tp"][t] < 1:
            w = w[:max(1, int(np.searchsorted(np.cumsum(w), n["tp"][t] * w.sum(), "left")) + 1)]
        w = w[w >= min(1.0, n["mp"][t])]
        at = np.argsort(order[:w.size])
        c = np.cumsum(w[at])
        i = min(int(np.searchsorted(c, n["u"][t] * c[-1], "right")), w.size - 1)
        idx[t], prob[t] = order[:w.size][at][i], w[at][i] / c[-1]
    return {"idx": idx, "prob": prob}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    k, K, mode = case["k"], case["K"], case["mode"]

    def blocks(q, sc):
        return q.double().unflatten(-1, (K // 32, 32)) * sc.double().unsqueeze(-1)
    if mode == "dequant":
        x = s["x"].double()
    else:
        x = blocks(s["xq"], s["xs"])
        if mode == "twopass":
            x = x + blocks(s["xl"], s["xs"] / 128)
        x = x.flatten(-2)
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for t, row in enumerate(_ids(case)):
        for j, e in enumerate(row):
            if e < 0:
                continue
            if case["op"] == "glu":
                g, u = (blocks(s[w][e], s["ws" + w[1]][e]).flatten(-2).mv(x[t]) for w in ("wg", "wu"))
                out[t * k + j] = g * torch.sigmoid(g) * u
            else:
                out[t] += s["weights"][t, j].double() * blocks(s["wd"][e], s["wsd"][e]).flatten(-2).mv(x[t * k + j])
    return out
