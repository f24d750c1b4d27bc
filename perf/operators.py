"""Measured cases of the attention step of a decoder: the rotated append of
new keys and values to a paged cache (lk_kv_append), the attention that reads
the cache (lk_attn), and its form for a batch that shares a long prefix
(lk_attn_shared).

``run`` computes them in plain torch operations, or, where ``own`` is set, by
the library's calls.  The cache is paged: k and v are [pages, kv heads, page,
head dim] in f16, bf16, or int8 levels with one f16 scale per 32 values
("q8"); a sequence's table lists its pages.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
DEV = "cuda"


# ---- the cases ---------------------------------------------------------------------

def listed():
    return [
        # one decode token of one sequence: the launch latency is all there is
        dict(name="append 1 row f16", op="append", B=1, R=1, n_q=32, n_kv=8, D=128, page=64, type="f16", keys=1500,
             ragged=False, empty=False, norm=False, paired=False),
        # a full decode batch with per-head norms into the int8 cache
        dict(name="append 64 rows q8 norm", op="append", B=64, R=1, n_q=32, n_kv=8, D=128, page=64, type="q8",
             keys=1024, ragged=True, empty=False, norm=True, paired=False),
        # a piece of one prompt, neighbouring pairs rotated, an odd row count
        dict(name="append 61-row prompt piece bf16", op="append", B=1, R=61, n_q=40, n_kv=8, D=128, page=16,
             type="bf16", keys=4093, ragged=False, empty=False, norm=False, paired=True),
        # one sequence, a short context: latency
        dict(name="attn 1 x 1023 f16", op="attn", B=1, R=1, n_q=32, n_kv=8, D=128, page=64, type="f16", keys=1023,
             ragged=False, empty=False),
        # one sequence, a very long context: the keys split over the whole GPU
        dict(name="attn 1 x 131071 q8", op="attn", B=1, R=1, n_q=32, n_kv=8, D=128, page=64, type="q8", keys=131071,
             ragged=False, empty=False),
        # a serving batch of ragged contexts with padding rows
        dict(name="attn 16 ragged 16384 bf16", op="attn", B=16, R=1, n_q=40, n_kv=8, D=128, page=16, type="bf16",
             keys=16384, ragged=True, empty=True),
        # the largest decode batch
        dict(name="attn 64 x 8192 f16", op="attn", B=64, R=1, n_q=32, n_kv=8, D=128, page=64, type="f16", keys=8192,
             ragged=False, empty=False),
        # a piece of a prompt behind a long context
        dict(name="attn 64-row prompt piece 32768 bf16", op="attn", B=1, R=64, n_q=32, n_kv=8, D=128, page=64,
             type="bf16", keys=32768, ragged=False, empty=False),
        # drafted tokens verified in one pass, smaller heads
        dict(name="attn 7 x 5 drafts 3001 q8 D64", op="attn", B=7, R=5, n_q=16, n_kv=4, D=64, page=32, type="q8",
             keys=3001, ragged=True, empty=False),
        # a few questions about one document
        dict(name="shared 5 on 2000 f16", op="shared", B=5, R=1, n_q=32, n_kv=8, D=128, page=16, type="f16", keys=77,
             prefix=2000, ragged=True, empty=False),
        # a full batch behind one long system prompt
        dict(name="shared 64 on 32768 bf16", op="shared", B=64, R=1, n_q=32, n_kv=8, D=128, page=64, type="bf16",
             keys=300, prefix=32768, ragged=True, empty=False),
        # the same from the int8 cache
        dict(name="shared 24 on 16384 q8", op="shared", B=24, R=1, n_q=32, n_kv=8, D=128, page=64, type="q8",
             keys=515, prefix=16384, ragged=True, empty=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "shared"])
    n_kv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 7, 8])
    c = dict(op=op, n_q=n_kv * g, n_kv=n_kv, D=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             type=rng.choice(["f16", "bf16", "q8"]), ragged=rng.random() < 0.6, empty=False)
    if op == "append":
        c["R"] = rng.choice([1, 1, 1, 2, 5, 16])
        c["B"] = _log(rng, 1, 64 // c["R"])
        c["keys"] = max(c["R"], _log(rng, 16, 8192))
        c.update(norm=rng.random() < 0.5, paired=rng.random() < 0.5)
        return c
    if op == "attn":
        c["R"] = rng.choice([1, 1, 1, 1, 2, 5, 16])
        c["B"] = _log(rng, 1, 64 // c["R"])
        most = min(131072, (1 << 19) // c["B"], (1 << 24) // (c["B"] * c["R"] * g))
        c["keys"] = max(c["R"], _log(rng, 16, max(17, most)))
        c["empty"] = rng.random() < 0.3 and c["B"] > 1
        return c
    c["R"] = rng.choice([1, 1, 1, 4])
    c["B"] = _log(rng, 2, 64 // c["R"])
    c["keys"] = max(c["R"], _log(rng, 4, 1024))
    c["prefix"] = _log(rng, 64, min(65536, (1 << 23) // (c["B"] * c["R"] * g)))
    return c


def _lens(case):
    """The sequences' numbers of keys: all the same, or ragged from a quarter
    up to the longest; `empty` leaves every fifth sequence out."""
    r = random.Random(case["keys"] * 64 + case["B"])
    n = []
    for b in range(case["B"]):
        v = case["keys"] if not case["ragged"] or b == 0 else r.randint(max(case["R"], case["keys"] // 4),
                                                                         case["keys"])
        n.append(0 if case["empty"] and b % 5 == 3 else v)
    return n


def _visible(case):
    """Keys that the rows of each sequence see of their own, row by row."""
    return [[max(0, n - case["R"] + 1 + r) for r in range(case["R"])] for n in _lens(case)]


def work(case):
    R, D, n_q, n_kv = case["R"], case["D"], case["n_q"], case["n_kv"]
    M = case["B"] * R
    e = 2.0 if case["type"] != "q8" else 1.0625
    if case["op"] == "append":
        return {"bytes": M * (4 * D * (2 * n_q + 2 * n_kv) + 4 * D + 2 * n_kv * D * e), "flops": 3 * M * D * (n_q + n_kv)}
    p = case.get("prefix", 0)
    keys = sum(_lens(case)) + p
    pairs = sum(v + p for s in _visible(case) for v in s)
    return {"bytes": 2 * n_kv * D * e * keys + 8.0 * M * n_q * D, "flops": 4.0 * n_q * D * pairs}


# ---- inputs ------------------------------------------------------------------------

def _pages(x, page, type_):
    """Pages of f32 values [pages, heads, page, D] in the cache's type:
    (values or levels, scales or None)."""
    if type_ != "q8":
        return x.to(DT[type_]), None
    b = x.view(*x.shape[:-1], x.shape[-1] // 32, 32)
    s = (b.abs().amax(-1) / 127.0).to(torch.float16)
    q = torch.round(b / s.float().unsqueeze(-1)).clamp_(-127, 127).to(torch.int8)
    return q.view(x.shape), s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    B, R, n_q, n_kv, D, page = (case[k] for k in ("B", "R", "n_q", "n_kv", "D", "page"))
    M, lens = B * R, _lens(case)
    shared = case["op"] == "shared"
    p_pages = -(-case["prefix"] // page) if shared else 0
    width = max(1, -(-max(lens) // page))
    n_pages = p_pages + B * width + 3
    s = dict(case)
    # pages lie in the cache in no order
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    s["prefix_table"] = order[:p_pages].contiguous()
    s["table"] = order[p_pages:p_pages + B * width].view(B, width).contiguous()
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    shape = (n_pages, n_kv, page, D)
    for name, shift in (("k", 0.0), ("v", 0.1)):
        if case["op"] == "append":
            x = torch.zeros(shape, device=DEV)
        else:
            x = torch.randn(shape, generator=g, device=DEV).add_(shift)
        s[name], s[name + "s"] = _pages(x, page, case["type"])
        del x
    if case["op"] == "append":
        # one row of the fused q|k|v projection per new token
        s["qkv"] = torch.randn((M, (n_q + 2 * n_kv) * D), generator=g, device=DEV)
        n_pos = case["keys"] + 1
        ang = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * torch.pow(
            torch.tensor(1e6, dtype=torch.float64, device=DEV),
            -torch.arange(D // 2, dtype=torch.float64, device=DEV) * 2 / D)[None]
        s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
        s["q_gain"] = s["k_gain"] = None
        if case["norm"]:
            s["q_gain"] = 1 + 0.1 * torch.randn((D,), generator=g, device=DEV)
            s["k_gain"] = 1 + 0.1 * torch.randn((D,), generator=g, device=DEV)
        s["out"] = torch.zeros((M, n_q * D), device=DEV)
        s["where"] = _written(s)
    else:
        s["q"] = 2 * torch.randn((M, n_q * D), generator=g, device=DEV)
        s["out"] = torch.zeros((M, n_q * D), device=DEV)
    if own:
        from q8_quantized_gemv_gb300 import lk
        s["cache"] = lk.KvCache(s["k"], s["v"], s["ks"], s["vs"])
        if case["op"] != "append":
            s["ws"] = torch.empty((lk.lk_attn_workspace_bytes(n_q, n_kv, D, B, R, shared),), dtype=torch.uint8,
                                  device=DEV)
    return s


# ---- the calls and their plain forms -----------------------------------------------

def _head_norm(x, gain, eps=1e-6):
    """x [M, heads, D] over the root of its mean square, times the gain: in 64
    bits, rounded once."""
    x = x.double()
    return (x * gain.double() / (x.square().mean(-1, keepdim=True) + eps).sqrt()).float()


def _rotate(x, cos, sin, paired):
    """Rotate x [M, heads, D] by the angles of its row: the pairs (i, i + D/2),
    or the neighbours (2i, 2i + 1) where `paired`."""
    c, s = cos[:, None], sin[:, None]
    a, b = (x[..., 0::2], x[..., 1::2]) if paired else x.chunk(2, -1)
    u, v = a * c - b * s, b * c + a * s
    return torch.stack((u, v), -1).flatten(-2) if paired else torch.cat((u, v), -1)


def _written(s):
    """Page and slot of the new rows, and the rows' positions."""
    pos = (s["lens"][:, None] - s["R"] + torch.arange(s["R"], device=DEV)).long()
    page = s["table"].gather(1, pos // s["page"]).long()
    return pos.flatten(), page.flatten(), (pos % s["page"]).flatten()


def _append_out(s):
    if s["type"] != "q8":
        return {"q": s["out"], "k": s["k"], "v": s["v"]}
    # the values that the new rows' levels stand for
    _, page, slot = s["where"]

    def value(q, sc):
        q, sc = q[page, :, slot], sc[page, :, slot].float()
        return q.view(*sc.shape, 32) * sc.unsqueeze(-1)
    return {"q": s["out"], "k": value(s["k"], s["ks"]), "v": value(s["v"], s["vs"])}


def _run_append(s):
    n_q, n_kv, D = s["n_q"], s["n_kv"], s["D"]
    q, k, v = s["qkv"].split((n_q * D, n_kv * D, n_kv * D), 1)
    if own:
        from q8_quantized_gemv_gb300 import lk
        lk.lk_kv_append(s["cache"], q, k, v, s["table"], s["lens"], s["cos"], s["sin"], s["out"], R=s["R"],
                        paired=s["paired"], q_gain=s["q_gain"], k_gain=s["k_gain"])
        return _append_out(s)
    pos, page, slot = _written(s)
    q, k, v = q.reshape(-1, n_q, D), k.reshape(-1, n_kv, D), v.reshape(-1, n_kv, D)
    if s["norm"]:
        q, k = _head_norm(q, s["q_gain"]), _head_norm(k, s["k_gain"])
    cos, sin = s["cos"][pos], s["sin"][pos]
    s["out"].copy_(_rotate(q, cos, sin, s["paired"]).flatten(1))
    k = _rotate(k, cos, sin, s["paired"])
    if s["type"] != "q8":
        s["k"][page, :, slot] = k.to(s["k"].dtype)
        s["v"][page, :, slot] = v.to(s["v"].dtype)
        return _append_out(s)
    for x, lv, sc in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
        x = x.view(-1, n_kv, D // 32, 32)
        a = x.abs().amax(-1)
        d = (a / torch.full_like(a, 127.0)).clamp(max=65504.0).to(torch.float16)
        f = d.float().unsqueeze(-1)
        z = torch.where(f > 0, torch.round(x / f).clamp(-127, 127), torch.zeros_like(x))
        lv[page, :, slot] = z.to(torch.int8).view(-1, n_kv, D)
        sc[page, :, slot] = d
    return _append_out(s)


def _gather(s, name, table):
    """The values of the listed pages: [sequences, kv heads, keys, D] in f32."""
    t = table.long()
    x = s[name][t].float()
    if s["type"] == "q8":
        sc = s[name + "s"][t].float()
        x = (x.view(*x.shape[:-1], -1, 32) * sc.unsqueeze(-1)).view(x.shape)
    x = x.transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _run_attn(s):
    B, R, n_q, n_kv, D = (s[k] for k in ("B", "R", "n_q", "n_kv", "D"))
    if own:
        from q8_quantized_gemv_gb300 import lk
        if s["op"] == "shared":
            lk.lk_attn_shared(s["cache"], s["q"], s["prefix_table"], s["prefix"], s["table"], s["lens"], s["ws"], R=R,
                              out=s["out"])
        else:
            lk.lk_attn(s["cache"], s["q"], s["table"], s["lens"], s["ws"], R=R, out=s["out"])
        return s["out"]
    G = n_q // n_kv
    # rows of a kv head: [B, kv heads, R * G, D]
    q = (s["q"] * D ** -0.5).view(B, R, n_kv, G, D).permute(0, 2, 1, 3, 4).reshape(B, n_kv, R * G, D)
    k, v = _gather(s, "k", s["table"]), _gather(s, "v", s["table"])
    x = q @ k.transpose(-1, -2)
    see = s["lens"][:, None] - R + 1 + torch.arange(R, device=DEV)
    ok = torch.arange(k.shape[2], device=DEV) < see.repeat_interleave(G, 1)[:, None, :, None]
    x = torch.where(ok, x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    if s["op"] == "shared":
        n = s["prefix"]
        pk, pv = _gather(s, "k", s["prefix_table"])[:, :n], _gather(s, "v", s["prefix_table"])[:, :n]
        # all rows of a kv head on the one prefix
        y = q.transpose(0, 1).reshape(n_kv, B * R * G, D) @ pk.transpose(-1, -2)
        y = y.view(n_kv, B, R * G, n).transpose(0, 1)
        m = torch.maximum(m, y.amax(-1, keepdim=True))
        py = torch.exp(y - m)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    p = torch.exp(x - m)
    total, o = p.sum(-1, keepdim=True), p @ v
    if s["op"] == "shared":
        total = total + py.sum(-1, keepdim=True)
        o = o + (py.transpose(0, 1).reshape(n_kv, B * R * G, n) @ pv).view(n_kv, B, R * G, D).transpose(0, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.view(B, n_kv, R, G, D).permute(0, 2, 1, 3, 4).reshape(B * R, n_q * D)


def run(state):
    return _run_append(state) if state["op"] == "append" else _run_attn(state)


# ---- the definitions in 64 bits ----------------------------------------------------

def _unpaged(s, name, pages, n):
    """The first n keys (or values) of a list of pages in 64 bits: [kv heads, n, D]."""
    x = torch.index_select(s[name], 0, pages.long()).double()
    if s["type"] == "q8":
        x = x * torch.index_select(s[name + "s"], 0, pages.long()).double().repeat_interleave(32, -1)
    return x.permute(1, 0, 2, 3).flatten(1, 2)[:, :n]


def exact(case, seed):
    s = prepare(case, seed)
    B, R, n_q, n_kv, D = (case[k] for k in ("B", "R", "n_q", "n_kv", "D"))
    lens = _lens(case)
    if case["op"] == "append":
        x = s["qkv"].double().view(B * R, n_q + 2 * n_kv, D)
        pos = torch.tensor([n - R + r for n in lens for r in range(R)], device=DEV)
        if case["norm"]:
            gain = torch.cat((s["q_gain"].double().expand(n_q, D), s["k_gain"].double().expand(n_kv, D)))
            h = x[:, :n_q + n_kv]
            x = torch.cat((h * gain * (h.pow(2).sum(-1, keepdim=True) / D + 1e-6).rsqrt(), x[:, n_q + n_kv:]), 1)
        # the rotation as a product of complex numbers
        turn = torch.complex(s["cos"].double(), s["sin"].double())[pos][:, None]
        h = x[:, :n_q + n_kv]
        if case["paired"]:
            z = turn * torch.view_as_complex(h.reshape(B * R, n_q + n_kv, D // 2, 2).contiguous())
            h = torch.view_as_real(z).reshape(B * R, n_q + n_kv, D)
        else:
            z = turn * torch.complex(h[..., :D // 2].contiguous(), h[..., D // 2:].contiguous())
            h = torch.cat((z.real, z.imag), -1)
        out = {"q": h[:, :n_q].reshape(B * R, n_q * D), "k": None, "v": None}
        if case["type"] != "q8":
            for name, new in (("k", h[:, n_q:]), ("v", x[:, n_q + n_kv:])):
                full = s[name].double()
                for i in range(B * R):
                    p = int(pos[i])
                    full[int(s["table"][i // R, p // case["page"]]), :, p % case["page"]] = new[i]
                out[name] = full
        return out
    q = s["q"].double().view(B, R, n_kv, n_q // n_kv, D)
    n_p = case.get("prefix", 0)
    if n_p:
        pk, pv = _unpaged(s, "k", s["prefix_table"], n_p), _unpaged(s, "v", s["prefix_table"], n_p)
    out = torch.zeros((B, R, n_kv, n_q // n_kv, D), dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        if n == 0 and not n_p:
            continue
        k, v = _unpaged(s, "k", s["table"][b], n), _unpaged(s, "v", s["table"][b], n)
        if n_p:
            k, v = torch.cat((pk, k), 1), torch.cat((pv, v), 1)
        z = torch.einsum("rhgd,hkd->hrgk", q[b], k) / math.sqrt(D)
        at = torch.arange(n_p + n, device=DEV)
        last = n_p + n - R + torch.arange(R, device=DEV)
        z = z.masked_fill((at[None] > last[:, None])[None, :, None], -math.inf)
        out[b] = torch.einsum("hrgk,hkd->rhgd", torch.softmax(z, -1), v)
    return out.view(B * R, n_q * D)
