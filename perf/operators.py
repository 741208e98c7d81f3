"""Measured cases of the attention-side operators: head norms with the
rotation (forward, with cache append, and backward), causal attention over
packed sequences (forward, and forward with backward), and attention of new
or drafted tokens over a paged cache.

`run` computes a case with the library where `own` is true, and otherwise in
plain torch operations in binary32.  Head layouts are (query heads, key/value
heads, head size): those of 896-, 1536-, 2048- and 2560-wide blocks
(14/2/64, 12/2/128, 16/2/128, 20/5/128) and one without grouping (8/8/64).
"""
import math

import torch

own = False

LAYOUTS = ((14, 2, 64), (12, 2, 128), (16, 2, 128), (20, 5, 128), (8, 8, 64))
EPS = 1e-6
BASE = 10000.0
SCRATCH = 1 << 30  # device scratch that the program keeps for calls that need one


def _ints(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------ cases

def _rope(kind, tokens, layout, x, norm, fused, max_pos, name=None):
    hq, hkv, d = layout
    case = {"kind": kind, "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "x": x, "norm": norm, "fused": fused,
            "max_pos": max_pos}
    return {"name": name, **case} if name else case


def _attn(kind, q_lens, k_lens, layout, name=None):
    hq, hkv, d = layout
    case = {"kind": kind, "q_lens": ",".join(map(str, q_lens)), "k_lens": ",".join(map(str, k_lens)), "hq": hq,
            "hkv": hkv, "d": d}
    return {"name": name, **case} if name else case


def _cache(lens, draft, layout, page, name=None):
    hq, hkv, d = layout
    case = {"kind": "cache", "lens": ",".join(map(str, lens)), "draft": draft, "hq": hq, "hkv": hkv, "d": d,
            "page": page}
    return {"name": name, **case} if name else case


def listed():
    packed = [2111, 517, 1, 3890, 64, 1025, 584]
    small = [1, 37, 130, 4]
    train = [4096, 1500, 2049, 547]
    train_small = [300, 129, 83]
    many = [1024 + (i * 977) % 7169 for i in range(64)]
    return [
        # one serving step of 64 sequences: head norms, rotation, K and V rows appended to the cache
        _rope("rope_cache", 64, (16, 2, 128), "f32", True, False, 32768, "rope_step"),
        # a prompt of an odd length, from one fused bf16 projection whose rows q, k and v share
        _rope("rope", 6001, (14, 2, 64), "bf16", True, True, 32768, "rope_fused_odd"),
        # the backward of a training step on binary32 projections, gradients of the norms' weights included
        _rope("rope_grad", 8192, (20, 5, 128), "f32", True, False, 8192, "rope_grad"),
        # the smallest prompts, where latency counts
        _attn("attn", small, small, (14, 2, 64), "attn_small"),
        # prompts of very different lengths packed into one batch
        _attn("attn", packed, packed, (20, 5, 128), "attn_packed"),
        # one long prompt, the largest case
        _attn("attn", [16384], [16384], (16, 2, 128), "attn_long"),
        # the next pieces of two prompts, behind what was read before
        _attn("attn", [512, 391], [7680, 4099], (12, 2, 128), "attn_chunk"),
        # a small training batch with small heads, forward and backward
        _attn("attn_train", train_small, train_small, (14, 2, 64), "attn_train_small"),
        # a packed training batch, forward and backward
        _attn("attn_train", train, train, (20, 5, 128), "attn_train"),
        # one sequence, one new token, a long cache
        _cache([32768], 1, (20, 5, 128), 64, "cache_one"),
        # a serving step of 64 sequences of different lengths
        _cache(many, 1, (16, 2, 128), 16, "cache_many"),
        # drafted trees of 24 tokens behind contexts from none to long
        _cache([9001, 4500, 130, 7777, 24, 6007, 2500, 8192], 24, (20, 5, 128), 128, "cache_tree"),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _parts(rng, total, most):
    """`total` tokens as one to `most` sequences of uneven lengths."""
    cuts = sorted({rng.randint(1, total - 1) for _ in range(rng.randint(0, most - 1))}) if total > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def draw(rng):
    layout = rng.choice(LAYOUTS)
    kind = rng.choice(("rope_cache", "rope", "rope_grad", "attn", "attn", "attn_train", "attn_train", "cache", "cache"))
    if kind.startswith("rope"):
        tokens = _log_uniform(rng, 1, 256) if kind == "rope_cache" else _log_uniform(rng, 17, 8192)
        return _rope(kind, tokens, layout, rng.choice(("f32", "bf16")), rng.random() < 0.6, rng.random() < 0.5,
                     rng.choice((8192, 32768, 65536)))
    if kind == "attn":
        q = _parts(rng, _log_uniform(rng, 16, 8192), 8)
        more = rng.random() < 0.3
        return _attn(kind, q, [n + (_log_uniform(rng, 1, 2048) if more else 0) for n in q], layout)
    if kind == "attn_train":
        q = _parts(rng, _log_uniform(rng, 64, 6000), 6)
        return _attn(kind, q, q, layout)
    draft = rng.choice((1, 1, 1, 2, 7, 16, 33, 64))
    batch = _log_uniform(rng, 1, 64 if draft == 1 else 8)
    return _cache([draft + _log_uniform(rng, 1, 8192) for _ in range(batch)], draft, layout,
                  rng.choice((16, 32, 64, 128, 256)))


# ----------------------------------------------------------------- inputs

def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def _prepare_rope(case, gen):
    tokens, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    dtype = torch.float32 if case["x"] == "f32" else torch.bfloat16
    wide = (hq + 2 * hkv) * d
    x = _normal(gen, tokens, wide, dtype=dtype)
    cut = (hq * d, (hq + hkv) * d)
    q, k, v = x[:, :cut[0]], x[:, cut[0]:cut[1]], x[:, cut[1]:]
    if not case["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    p = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)
    f = BASE ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) * 2 / d)
    a = p[:, None] * f
    s = {"kind": case["kind"], "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "q": q, "k": k, "v": v,
         "table": torch.stack((a.cos(), a.sin()), -1).float().contiguous(),
         "pos": torch.randint(0, case["max_pos"], (tokens,), generator=gen, device="cuda", dtype=torch.int32),
         "qw": None, "kw": None}
    if case["norm"]:
        s["qw"] = 1 + 0.2 * _normal(gen, d, dtype=torch.float32)
        s["kw"] = 1 + 0.2 * _normal(gen, d, dtype=torch.float32)
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    if case["kind"] == "rope_grad":
        s["dq"], s["dk"] = _normal(gen, tokens, hq * d), _normal(gen, tokens, hkv * d)
        s["gq"], s["gk"] = torch.empty(tokens, hq * d, **bf), torch.empty(tokens, hkv * d, **bf)
        s["gqw"], s["gkw"] = (torch.empty(d, device="cuda"), torch.empty(d, device="cuda")) if case["norm"] else (None, None)
        s["ws"] = torch.empty(SCRATCH, dtype=torch.uint8, device="cuda")
        return s
    s["qo"] = torch.empty(tokens, hq * d, **bf)
    s["slots"] = None
    rows = tokens
    if case["kind"] == "rope_cache":
        rows = 64 * tokens
        s["slots"] = torch.randperm(rows, generator=gen, device="cuda")[:tokens].contiguous()
    s["ko"], s["vo"] = torch.zeros(rows, hkv * d, **bf), torch.zeros(rows, hkv * d, **bf)
    return s


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _side(lens):
    """Device index tensors of one packed side: starts, padded places, and each row's sequence and place in it."""
    starts, most = _starts(lens), max(lens)
    cu = torch.tensor(starts, dtype=torch.int32, device="cuda")
    first = cu[:-1].long()
    n = (cu[1:] - cu[:-1]).long()
    place = torch.arange(most, device="cuda")
    at = (first[:, None] + place).clamp(max=max(starts[-1] - 1, 0))
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    return {"cu": cu, "len": n, "at": at, "seq": seq, "place": torch.arange(starts[-1], device="cuda") - first[seq],
            "total": starts[-1]}


def _prepare_attn(case, gen):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    a, b = _side(_ints(case["q_lens"])), _side(_ints(case["k_lens"]))
    tq, tk = a["total"], b["total"]
    bf = {"dtype": torch.bfloat16, "device": "cuda"}
    s = {"kind": case["kind"], "hq": hq, "hkv": hkv, "d": d, "scale": d ** -0.5, "batch": len(a["len"]), "qs": a,
         "ks": b, "q": _normal(gen, tq, hq * d, std=1.5), "k": _normal(gen, tk, hkv * d), "v": _normal(gen, tk, hkv * d),
         "o": torch.empty(tq, hq * d, **bf), "lse": torch.empty(hq, tq, device="cuda"),
         "ws": torch.empty(SCRATCH, dtype=torch.uint8, device="cuda")}
    if case["kind"] == "attn_train":
        s["do"] = _normal(gen, tq, hq * d)
        s["dq"], s["dk"], s["dv"] = (torch.empty(tq, hq * d, **bf), torch.empty(tk, hkv * d, **bf),
                                     torch.empty(tk, hkv * d, **bf))
    return s


def _tree(gen, batch, draft):
    """For each sequence a random tree over the drafted tokens: bit j of row i says that token i sees token j."""
    parent = torch.randint(0, 1 << 30, (batch, draft), generator=gen, device="cuda").tolist()
    rows = []
    for b in range(batch):
        seen = []
        for i in range(draft):
            m = (seen[parent[b][i] % i] if i else 0) | (1 << i)
            seen.append(m)
        rows.append([m - (1 << 64) if m >> 63 else m for m in seen])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _prepare_cache(case, gen):
    hq, hkv, d, draft, page = case["hq"], case["hkv"], case["d"], case["draft"], case["page"]
    lens = _ints(case["lens"])
    batch, most = len(lens), max(lens)
    per = -(-most // page)
    used = sum(-(-n // page) for n in lens)
    pool = used + 3
    order = torch.randperm(pool, generator=gen, device="cuda").tolist()
    table, at = [], 0
    for n in lens:
        c = -(-n // page)
        table.append(order[at:at + c] + [0] * (per - c))
        at += c
    return {"kind": "cache", "hq": hq, "hkv": hkv, "d": d, "draft": draft, "page": page, "batch": batch,
            "scale": d ** -0.5, "most": most,
            "q": _normal(gen, batch * draft, hq * d, std=1.5), "k": _normal(gen, pool * page, hkv * d),
            "v": _normal(gen, pool * page, hkv * d),
            "pages": torch.tensor(table, dtype=torch.int32, device="cuda"),
            "lens": torch.tensor(lens, dtype=torch.int32, device="cuda"),
            "tree": _tree(gen, batch, draft) if draft > 1 else None,
            "o": torch.empty(batch * draft, hq * d, dtype=torch.bfloat16, device="cuda"),
            "ws": torch.empty(SCRATCH, dtype=torch.uint8, device="cuda")}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["kind"].startswith("rope"):
        return _prepare_rope(case, gen)
    return _prepare_cache(case, gen) if case["kind"] == "cache" else _prepare_attn(case, gen)


# ------------------------------------------------------------ plain forms

def _angles(s):
    t = s["table"][s["pos"].long()]
    return t[:, None, :, 0], t[:, None, :, 1]


def _rotate(x, c, s):
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _normed(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _plain_rope(s):
    c, n = _angles(s)
    t, d = s["tokens"], s["d"]
    q = _rotate(_normed(s["q"].float().reshape(t, s["hq"], d), s["qw"]), c, n)
    k = _rotate(_normed(s["k"].float().reshape(t, s["hkv"], d), s["kw"]), c, n)
    s["qo"].copy_(q.view(t, -1))
    if s["slots"] is None:
        s["ko"].copy_(k.view(t, -1))
        s["vo"].copy_(s["v"])
    else:
        s["ko"][s["slots"]] = k.view(t, -1).bfloat16()
        s["vo"][s["slots"]] = s["v"].bfloat16()
    return {"q": s["qo"], "k": s["ko"], "v": s["vo"]}


def _plain_rope_grad_of(x, dy, w, c, n, t, h, d):
    g = _rotate(dy.float().reshape(t, h, d), c, -n)
    if w is None:
        return g.reshape(t, -1).bfloat16(), None
    x = x.float().reshape(t, h, d)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    x = x * r
    dw = (g * x).sum((0, 1))
    g = g * w
    return (r * (g - x * (g * x).mean(-1, keepdim=True))).reshape(t, -1).bfloat16(), dw


def _plain_rope_grad(s):
    c, n = _angles(s)
    gq, gqw = _plain_rope_grad_of(s["q"], s["dq"], s["qw"], c, n, s["tokens"], s["hq"], s["d"])
    gk, gkw = _plain_rope_grad_of(s["k"], s["dk"], s["kw"], c, n, s["tokens"], s["hkv"], s["d"])
    return {"q": gq, "k": gk, **({"qw": gqw, "kw": gkw} if gqw is not None else {})}


def _padded(x, side, heads, d):
    """[rows, heads * d] as binary32 [batch, heads, longest, d]."""
    return x[side["at"]].view(*side["at"].shape, heads, d).transpose(1, 2).float()


def _packed(x, side):
    """[batch, heads, longest, d] back to [rows, heads * d]."""
    return x[side["seq"], :, side["place"]].reshape(side["total"], -1)


def _visible(s):
    nq, nk = s["qs"]["len"], s["ks"]["len"]
    i = torch.arange(s["qs"]["at"].shape[1], device="cuda")
    j = torch.arange(s["ks"]["at"].shape[1], device="cuda")
    return ((j <= i[:, None] + (nk - nq)[:, None, None]) & (j < nk[:, None, None]) & (i[:, None] < nq[:, None, None]))[:, None, None]


def _plain_attn(s):
    b, hq, hkv, d = s["batch"], s["hq"], s["hkv"], s["d"]
    q = _padded(s["q"], s["qs"], hq, d)
    k, v = _padded(s["k"], s["ks"], hkv, d), _padded(s["v"], s["ks"], hkv, d)
    mq, mk = q.shape[2], k.shape[2]
    q = q.reshape(b, hkv, -1, d)
    hidden = ~_visible(s)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, hq // hkv, mq, mk).masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    p = p.view(b, hkv, -1, mk)
    o = (torch.matmul(p, v).view(b, hkv, hq // hkv, mq, d) / torch.where(z > 0, z, 1)).view(b, hq, mq, d)
    lse = (m + z.log()).view(b, hq, mq)
    out = {"o": _packed(o, s["qs"]).bfloat16(), "lse": lse[s["qs"]["seq"], :, s["qs"]["place"]].t().contiguous()}
    if s["kind"] == "attn":
        return out
    g = _padded(s["do"], s["qs"], hq, d).masked_fill_(~(s["qs"]["len"][:, None] > torch.arange(mq, device="cuda"))[:, None, :, None], 0)
    p = p.view(b, hq, mq, mk).div_(torch.where(z > 0, z, 1).view(b, hq, mq, 1)).view(b, hkv, -1, mk)
    dot = (g * o).sum(-1).view(b, hkv, -1, 1)
    g = g.reshape(b, hkv, -1, d)
    dv = torch.matmul(p.transpose(2, 3), g)
    ds = torch.matmul(g, v.transpose(2, 3)).sub_(dot).mul_(p)
    dq = torch.matmul(ds, k).mul_(s["scale"]).view(b, hq, mq, d)
    dk = torch.matmul(ds.transpose(2, 3), q).mul_(s["scale"])
    return {**out, "dq": _packed(dq, s["qs"]).bfloat16(), "dk": _packed(dk, s["ks"]).bfloat16(),
            "dv": _packed(dv, s["ks"]).bfloat16()}


def _plain_cache(s):
    b, hq, hkv, d, t, page, n = s["batch"], s["hq"], s["hkv"], s["d"], s["draft"], s["page"], s["most"]
    j = torch.arange(n, device="cuda")
    row = s["pages"].long()[:, j // page] * page + j % page
    k = s["k"][row].view(b, n, hkv, d).transpose(1, 2).float()
    v = s["v"][row].view(b, n, hkv, d).transpose(1, 2).float()
    q = s["q"].float().view(b, t, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)
    i = torch.arange(t, device="cuda")
    at = j - (s["lens"].long()[:, None] - t)  # place among the drafted tokens; below 0 in the context
    bits = s["tree"] if s["tree"] is not None else ((2 << i) - 1).expand(b, t)
    seen = (at[:, None] < 0) | ((bits[:, :, None] >> at.clamp(0, 63)[:, None]) & 1 == 1)
    seen = seen & (at[:, None] < t)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, -1, t, n).masked_fill_(~seen[:, None, None], -math.inf)
    p = (x - x.amax(-1, keepdim=True)).exp()
    p = (p / p.sum(-1, keepdim=True)).view(b, hkv, -1, n)
    o = torch.matmul(p, v).view(b, hkv, hq // hkv, t, d).permute(0, 3, 1, 2, 4)
    return {"o": o.reshape(b * t, hq * d).bfloat16()}


# ------------------------------------------------------------ the library

def _own(s):
    from sparse_linear_layers_group_amd import bitlinear as bl
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    if s["kind"] in ("rope", "rope_cache"):
        bl.bitlinear_qk_rope(s["q"], s["k"], s["v"], s["tokens"], hq, hkv, d, s["qw"], s["kw"], EPS, s["table"],
                             s["pos"], s["qo"], s["ko"], s["vo"], slots=s["slots"])
        return {"q": s["qo"], "k": s["ko"], "v": s["vo"]}
    if s["kind"] == "rope_grad":
        bl.bitlinear_qk_rope_bwd(s["q"], s["k"], s["tokens"], hq, hkv, d, s["qw"], s["kw"], EPS, s["table"], s["pos"],
                                 s["dq"], s["dk"], s["gq"], s["gk"], s["gqw"], s["gkw"], ws=s["ws"])
        return {"q": s["gq"], "k": s["gk"], **({"qw": s["gqw"], "kw": s["gkw"]} if s["gqw"] is not None else {})}
    if s["kind"] == "cache":
        bl.bitlinear_attn_cache(s["q"], s["k"], s["v"], s["pages"], s["page"], s["lens"], s["tree"], s["batch"],
                                s["draft"], hq, hkv, d, s["scale"], s["o"], ws=s["ws"])
        return {"o": s["o"]}
    cq, ck = s["qs"]["cu"], s["ks"]["cu"]
    bl.bitlinear_attn_fwd(s["q"], s["k"], s["v"], cq, ck, s["batch"], hq, hkv, d, s["scale"], s["o"], s["lse"],
                          ws=s["ws"])
    if s["kind"] == "attn":
        return {"o": s["o"], "lse": s["lse"]}
    bl.bitlinear_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], cq, ck, s["batch"], hq, hkv, d, s["scale"],
                          s["dq"], s["dk"], s["dv"], ws=s["ws"])
    return {"o": s["o"], "lse": s["lse"], "dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


def run(state):
    if own:
        return _own(state)
    if state["kind"] == "cache":
        return _plain_cache(state)
    if state["kind"] == "rope_grad":
        return _plain_rope_grad(state)
    return _plain_rope(state) if state["kind"].startswith("rope") else _plain_attn(state)


# ------------------------------------------------------------------- work

def _pairs(nq, nk):
    """Visible (query, key) pairs of one sequence."""
    full = min(nq, nk)
    return sum(range(nk - full + 1, nk + 1)) if full < 2 else (nk - full + 1 + nk) * full // 2


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["kind"].startswith("rope"):
        t = case["tokens"]
        x = 4 if case["x"] == "f32" else 2
        table = min(t, case["max_pos"]) * d * 4 + t * 4
        qk = t * (hq + hkv) * d
        if case["kind"] == "rope_grad":
            return {"bytes": qk * (4 + (x if case["norm"] else 0)) + table, "flops": qk * (14 if case["norm"] else 3)}
        both = t * (hq + 2 * hkv) * d
        return {"bytes": both * (x + 2) + table + (8 * t if case["kind"] == "rope_cache" else 0),
                "flops": qk * (7 if case["norm"] else 3)}
    if case["kind"] == "cache":
        lens, t = _ints(case["lens"]), case["draft"]
        return {"bytes": 4 * (sum(lens) * hkv + len(lens) * t * hq) * d, "flops": 4 * sum(lens) * t * hq * d}
    nq, nk = _ints(case["q_lens"]), _ints(case["k_lens"])
    pairs = sum(_pairs(a, b) for a, b in zip(nq, nk)) * hq
    q, k = 2 * sum(nq) * hq * d, 2 * sum(nk) * hkv * d  # bytes of one tensor of each side
    if case["kind"] == "attn":
        return {"bytes": 2 * q + 2 * k + 4 * sum(nq) * hq, "flops": 4 * pairs * d}
    return {"bytes": 4 * q + 4 * k + 4 * sum(nq) * hq, "flops": 14 * pairs * d}


# ------------------------------------------------------------ 64-bit form

def _exact_heads(x, w, h, d):
    x = x.double().reshape(x.shape[0], h, d)
    if w is None:
        return x, None
    r = 1 / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt()
    return x, r


def _exact_rope(s):
    d, half = s["d"], s["d"] // 2
    z = torch.view_as_complex(s["table"].double())[s["pos"].long()][:, None]

    def turned(x, w, h):
        x, r = _exact_heads(x, w, h, d)
        x = x if w is None else x * r * w.double()
        y = torch.complex(x[..., :half], x[..., half:]) * z
        return torch.cat((y.real, y.imag), -1).reshape(x.shape[0], h * d)

    q, k, v = turned(s["q"], s["qw"], s["hq"]), turned(s["k"], s["kw"], s["hkv"]), s["v"].double()
    if s["slots"] is not None:
        rows = torch.zeros(s["ko"].shape, dtype=torch.float64, device="cuda")
        k, v = rows.index_copy(0, s["slots"], k), rows.index_copy(0, s["slots"], v)
    return {"q": q, "k": k, "v": v}


def _exact_rope_grad(s):
    d, half = s["d"], s["d"] // 2
    z = torch.view_as_complex(s["table"].double())[s["pos"].long()][:, None].conj()
    out = {}
    for name, x, dy, w, h in (("q", s["q"], s["dq"], s["qw"], s["hq"]), ("k", s["k"], s["dk"], s["kw"], s["hkv"])):
        g = dy.double().reshape(-1, h, d)
        g = torch.complex(g[..., :half], g[..., half:]) * z
        g = torch.cat((g.real, g.imag), -1)
        x, r = _exact_heads(x, w, h, d)
        if w is not None:
            out[name + "w"] = torch.einsum("thd,thd,th->d", g, x, r[..., 0])
            a = g * w.double()
            g = a * r - x * r.pow(3) / d * (a * x).sum(-1, keepdim=True)
        out[name] = g.reshape(-1, h * d)
    return out


def _exact_attn(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    group = hq // hkv
    train = s["kind"] == "attn_train"
    like = lambda x: torch.zeros(x.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"o": like(s["o"]), "lse": torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")}
    if train:
        out |= {"dq": like(s["q"]), "dk": like(s["k"]), "dv": like(s["v"])}
    cq, ck = s["qs"]["cu"].tolist(), s["ks"]["cu"].tolist()
    for q0, q1, k0, k1 in zip(cq, cq[1:], ck, ck[1:]):
        n, shown = q1 - q0, torch.ones(q1 - q0, k1 - k0, dtype=torch.bool, device="cuda").tril(k1 - k0 - q1 + q0)
        for h in range(hq):
            a, b = slice(h * d, h * d + d), slice(h // group * d, h // group * d + d)
            q, k, v = s["q"][q0:q1, a].double(), s["k"][k0:k1, b].double(), s["v"][k0:k1, b].double()
            x = torch.where(shown, s["scale"] * (q @ k.T), -math.inf)
            lse = torch.logsumexp(x, 1)
            p = torch.where(shown, torch.exp(x - lse[:, None]), 0.0)
            del x
            o = p @ v
            out["o"][q0:q1, a], out["lse"][h, q0:q1] = o, lse
            if train and n:
                g = s["do"][q0:q1, a].double()
                dp = g @ v.T
                ds = p * dp
                ds = s["scale"] * (ds - p * ds.sum(1, keepdim=True))
                out["dv"][k0:k1, b] += p.T @ g
                out["dq"][q0:q1, a] = ds @ k
                out["dk"][k0:k1, b] += ds.T @ q
    return out


def _exact_cache(s):
    hq, hkv, d, t, page = s["hq"], s["hkv"], s["d"], s["draft"], s["page"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        rows = (s["pages"][b].long()[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:n]
        k, v = s["k"][rows].double().view(n, hkv, d), s["v"][rows].double().view(n, hkv, d)
        for i in range(t):
            m = int(s["tree"][b, i]) if s["tree"] is not None else (2 << i) - 1
            at = list(range(n - t)) + [n - t + j for j in range(t) if m >> j & 1]
            ki, vi = k[at].repeat_interleave(hq // hkv, 1), v[at].repeat_interleave(hq // hkv, 1)
            q = s["q"][b * t + i].double().view(hq, d)
            p = torch.softmax(s["scale"] * (ki * q).sum(-1), 0)
            o[b * t + i] = (p[..., None] * vi).sum(0).reshape(-1)
    return {"o": o}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "cache":
        return _exact_cache(s)
    if case["kind"] == "rope_grad":
        return _exact_rope_grad(s)
    return _exact_rope(s) if case["kind"].startswith("rope") else _exact_attn(s)
