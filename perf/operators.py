"""Cases of the decode-step operators around the MoE block and the head: appending keys and
values to the paged cache (with the heads' RMSNorm and the rotary positions applied on the way),
single-token attention over that cache for a batch that may share a long prefix, and sampling from
the head's logits.  Where `own` is false, `run` computes them in plain torch operations; where it
is true, through int4_expert_routing_b200."""
import math

import numpy as np
import torch

own = False

EPS = 1e-6  # of the heads' RMSNorm
E4M3_MAX = 448.0

# ------------------------------------------------------------------ cases


def listed():
    return [
        # one decode step of a small batch, the model's own heads: latency
        dict(name="append decode", op="append", T=4, q_heads=32, kv_heads=4, dim=128, rope=128,
             interleaved=False, norm=True, kv="bf16", page=16, start=100_000),
        # a long prompt in one call
        dict(name="append prompt", op="append", T=16384, q_heads=32, kv_heads=4, dim=128, rope=128,
             interleaved=False, norm=True, kv="bf16", page=64, start=0),
        # a ragged chunk of a prompt into an 8-bit cache, rotary on half of each head
        dict(name="append chunk 8-bit", op="append", T=1037, q_heads=16, kv_heads=8, dim=64,
             rope=32, interleaved=True, norm=False, kv="e4m3", page=48, start=4093),
        # one user, a short chat: latency
        dict(name="attend short", op="attend", B=1, q_heads=32, kv_heads=4, dim=128, prefix=0,
             lo=701, hi=701, window=0, sinks=True, kv="bf16", page=16),
        # a sliding-window layer of a serving batch
        dict(name="attend window", op="attend", B=48, q_heads=32, kv_heads=4, dim=128, prefix=0,
             lo=37, hi=6000, window=513, sinks=True, kv="bf16", page=64),
        # few users, long documents of very different lengths, a full layer
        dict(name="attend long", op="attend", B=8, q_heads=32, kv_heads=4, dim=128, prefix=0,
             lo=5003, hi=131072, window=0, sinks=True, kv="bf16", page=64),
        # agents on one long system prompt, each with a little of its own
        dict(name="attend shared 32", op="attend", B=32, q_heads=32, kv_heads=4, dim=128,
             prefix=32001, lo=1, hi=700, window=0, sinks=True, kv="bf16", page=64),
        # many samples of one document
        dict(name="attend shared 256", op="attend", B=256, q_heads=32, kv_heads=4, dim=128,
             prefix=16384, lo=1, hi=1024, window=0, sinks=True, kv="bf16", page=64),
        # the 8-bit cache
        dict(name="attend 8-bit", op="attend", B=64, q_heads=32, kv_heads=4, dim=128, prefix=2048,
             lo=100, hi=4096, window=0, sinks=False, kv="e4m3", page=32),
        # one step of a small batch over the whole vocabulary of the head
        dict(name="sample 4", op="sample", B=4, V=150_144, temperature=1.0, top_k=20, top_p=0.95,
             min_p=0.0, tail=1.3),
        # a large batch, nucleus and min-p only: the kept sets are long
        dict(name="sample 128", op="sample", B=128, V=150_144, temperature=1.0, top_k=0,
             top_p=0.9, min_p=1e-5, tail=1.1),
        # a small vocabulary, odd sizes, mixed requests (greedy ones among them)
        dict(name="sample small", op="sample", B=7, V=5003, temperature=0.6, top_k=100, top_p=0.8,
             min_p=0.02, tail=1.0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "sample"])
    if op == "append":
        dim = rng.choice([64, 128])
        q, kv = rng.choice([(32, 4), (16, 2), (8, 8), (12, 4), (16, 1), (20, 4)])
        return dict(op=op, T=_spread(rng, 1, 12000), q_heads=q, kv_heads=kv, dim=dim,
                    rope=rng.choice([0, dim // 2, dim, dim]), interleaved=rng.random() < 0.4,
                    norm=rng.random() < 0.6, kv=rng.choice(["bf16", "bf16", "e4m3"]),
                    page=rng.choice([16, 32, 48, 64, 128]), start=rng.randrange(0, 500_000))
    if op == "sample":
        return dict(op=op, B=_spread(rng, 1, 120), V=_spread(rng, 100, 150_144),
                    temperature=round(rng.uniform(0.3, 1.5), 3),
                    top_k=rng.choice([0, 0, _spread(rng, 1, 2000)]),
                    top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                    min_p=rng.choice([0.0, round(rng.uniform(1e-4, 0.2), 5)]),
                    tail=round(rng.uniform(0.5, 2.0), 3))
    most = _weight(work(next(c for c in listed() if c["name"] == "attend shared 256")))
    while True:
        q, kv = rng.choice([(32, 4), (32, 4), (16, 2), (8, 8), (12, 4), (16, 1), (20, 4)])
        hi = _spread(rng, 1, 60_000)
        c = dict(op=op, B=_spread(rng, 1, 200), q_heads=q, kv_heads=kv,
                 dim=rng.choice([128, 128, 64]),
                 prefix=rng.choice([0, _spread(rng, 1, 30_000)]), lo=rng.randrange(0, hi + 1),
                 hi=hi, window=rng.choice([0, 0, _spread(rng, 1, 5000)]),
                 sinks=rng.random() < 0.6, kv=rng.choice(["bf16", "bf16", "e4m3"]),
                 page=rng.choice([16, 32, 48, 64, 128]))
        if _weight(work(c)) <= most and c["B"] * (hi + c["prefix"]) * c["q_heads"] <= 1 << 27:
            return c


def _weight(w):
    return max(w["bytes"], w["flops"] / 50)


def _lens(case):
    """Each sequence's own keys: from lo to hi, spread unevenly, fixed for a case (the seed only
    says which sequence has which)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    f = [((b * 0.6180339887498949 + 0.5) % 1.0) ** 2 for b in range(B)]
    n = [lo + int(round((hi - lo) * x)) for x in f]
    n[0] = hi
    return n


def work(case):
    if case["op"] == "append":
        T, q, kv, d = case["T"], case["q_heads"], case["kv_heads"], case["dim"]
        e = 2 if case["kv"] == "bf16" else 1
        moved = T * d * (2 * (2 * q + 2 * kv) + e * 2 * kv) + 12 * T
        return {"bytes": moved, "flops": T * d * (q + kv) * 7}
    if case["op"] == "sample":
        return {"bytes": 4 * case["B"] * case["V"], "flops": 4 * case["B"] * case["V"]}
    q, kv, d, P, w = (case[k] for k in ("q_heads", "kv_heads", "dim", "prefix", "window"))
    e = 2 if case["kv"] == "bf16" else 1
    n = _lens(case)
    if w:
        mine = sum(min(x, w) for x in n)
        both = mine + sum(min(P, max(0, w - x)) for x in n)
        shared = min(P, max(max(0, w - x) for x in n))
    else:
        mine, both, shared = sum(n), sum(n) + case["B"] * P, P
    return {"bytes": (mine + shared) * kv * d * 2 * e + case["B"] * q * d * 4,
            "flops": 4 * both * q * d}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _pool(g, case, pages):
    """K or V pages [pages][kv_heads][page][dim], full of what earlier sequences left."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(0, 1, generator=g)
    return x if case["kv"] == "bf16" else (2 * x).to(torch.float8_e4m3fn)


def _scales(g, case):
    """One scale for each KV head of the 8-bit cache (codes are about 2 x N(0, 1))."""
    if case["kv"] == "bf16":
        return None
    return 0.5 + 0.1 * torch.rand(case["kv_heads"], generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "append":
        T, q, kv, d, page = (case[k] for k in ("T", "q_heads", "kv_heads", "dim", "page"))
        # the fused projection's rows: q heads, k heads, v heads
        qkv = _normal(g, T, (q + 2 * kv) * d)
        qkv[:, 3::97] *= 8  # a few large channels
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv[:, :q * d], qkv[:, q * d:(q + kv) * d], qkv[:, (q + kv) * d:]
        pages = -(-T // page) + 3
        s["k_pages"], s["v_pages"] = _pool(g, case, pages), _pool(g, case, pages)
        s["k_scale"], s["v_scale"] = _scales(g, case), _scales(g, case)
        t = torch.arange(T, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda")
        off = int(torch.randint(0, page, (1,), generator=g, device="cuda"))
        s["slots"] = order[(t + off) // page] * page + (t + off) % page
        s["pos"] = (t + case["start"]).to(torch.int32)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"] = (1 + 0.1 * _normal(g, d)).to(torch.bfloat16)
            s["k_norm"] = (1 + 0.1 * _normal(g, d)).to(torch.bfloat16)
        s["q_out"] = torch.empty(T, q * d, device="cuda", dtype=torch.bfloat16)
        return s
    if case["op"] == "sample":
        B, V = case["B"], case["V"]
        e = -torch.log(1 - torch.rand(B, V, generator=g, device="cuda", dtype=torch.float64))
        s["logits"] = (case["tail"] * e).float() + 0.1 * _normal(g, B, V) - 3
        r = torch.rand(B, generator=g, device="cuda")
        s["temperature"] = case["temperature"] * (0.8 + 0.4 * r)
        s["top_k"] = torch.full((B,), case["top_k"], device="cuda", dtype=torch.int32)
        if B > 4:
            s["temperature"][::6] = 0  # greedy requests among the others
            s["top_k"][1::5] = 0
        s["top_p"] = torch.full((B,), case["top_p"], device="cuda")
        s["min_p"] = torch.full((B,), case["min_p"], device="cuda")
        s["u"] = torch.rand(B, generator=g, device="cuda")
        s["token"] = torch.empty(B, device="cuda", dtype=torch.int32)
        s["logprob"] = torch.empty(B, device="cuda")
        return s
    B, q, kv, d, page, P = (case[k] for k in ("B", "q_heads", "kv_heads", "dim", "page", "prefix"))
    n = torch.tensor(_lens(case), device="cuda")
    n = n[torch.randperm(B, generator=g, device="cuda")]
    need = -(-n // page)
    most = max(1, int(need.max()))
    total = int(need.sum()) + -(-P // page) + 3
    s["k_pages"], s["v_pages"] = _pool(g, case, total), _pool(g, case, total)
    s["k_scale"], s["v_scale"] = _scales(g, case), _scales(g, case)
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(most, device="cuda")
    first = torch.cumsum(need, 0) - need
    table = order[(first[:, None] + at).clamp(max=total - 1)]
    s["table"] = torch.where(at < need[:, None], table, -1).to(torch.int32)
    s["lens"] = n.to(torch.int32)
    s["prefix_pages"] = order[total - -(-P // page):].contiguous() if P else None
    s["q"] = (1.5 * _normal(g, B, q * d)).to(torch.bfloat16)
    s["sinks"] = 2 + 3 * _normal(g, q) if case["sinks"] else None
    s["scale"] = 1 / math.sqrt(d)
    s["out"] = torch.empty(B, q * d, device="cuda", dtype=torch.bfloat16)
    s["lse"] = torch.empty(B, q, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms


def _heads(x, case, heads, weight, pos, rope):
    """Rows of heads in 32 bits: RMSNorm with `weight` (if any), then the rotation of the first
    `rope` elements by the position's angles (in 64 bits: positions go far)."""
    d = case["dim"]
    x = x.reshape(x.shape[0], heads, d).float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    if not rope:
        return x
    half = rope // 2
    freq = 10_000.0 ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / rope)
    angle = pos.double()[:, None, None] * freq
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:rope:2], x[..., 1:rope:2]
        y[..., 0:rope:2], y[..., 1:rope:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rope]
        y[..., :half], y[..., half:rope] = a * cos - b * sin, b * cos + a * sin
    return y


def _store(pages, x, slots, scale):
    page = pages.shape[2]
    if scale is None:
        x = x.to(torch.bfloat16)
    else:
        x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    # written byte by byte where the cache holds 8 bits: the same elements either way
    if scale is not None:
        pages, x = pages.view(torch.uint8), x.view(torch.uint8)
    pages[slots // page, :, slots % page] = x


def _append(s):
    c = s["case"]
    q = _heads(s["q"], c, c["q_heads"], s["q_norm"], s["pos"], c["rope"])
    k = _heads(s["k"], c, c["kv_heads"], s["k_norm"], s["pos"], c["rope"])
    v = s["v"].reshape(c["T"], c["kv_heads"], c["dim"]).float()
    _store(s["k_pages"], k, s["slots"], s["k_scale"])
    _store(s["v_pages"], v, s["slots"], s["v_scale"])
    return {"q": q.reshape(c["T"], -1).to(torch.bfloat16), "k_pages": s["k_pages"],
            "v_pages": s["v_pages"]}


def _rows(pages, table, scale):
    """The pages of `table` [..., pages] in 32 bits, as [..., kv_heads, keys, dim]."""
    x = pages.view(torch.uint8)[table.long()].view(pages.dtype) if scale is not None \
        else pages[table.long()]
    x = x.transpose(-4, -3).flatten(-3, -2).float()
    return x if scale is None else x * scale[:, None, None]


def _attend(s):
    c = s["case"]
    B, P, H, d = c["B"], c["prefix"], c["kv_heads"], c["dim"]
    G = c["q_heads"] // H
    q = s["q"].reshape(B, H, G, d).float() * s["scale"]
    n = s["lens"].long()[:, None]
    table = s["table"].clamp(min=0)
    k, v = _rows(s["k_pages"], table, s["k_scale"]), _rows(s["v_pages"], table, s["v_scale"])
    at = P + torch.arange(k.shape[2], device=q.device)
    seen = at < P + n
    if c["window"]:
        seen &= at > P + n - 1 - c["window"]
    scores = torch.matmul(q, k.transpose(-1, -2))
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    top = scores.amax(-1)
    if P:
        kp = _rows(s["k_pages"], s["prefix_pages"], s["k_scale"])[:, :P]
        vp = _rows(s["v_pages"], s["prefix_pages"], s["v_scale"])[:, :P]
        qp = q.permute(1, 0, 2, 3).reshape(H, B * G, d)
        before = torch.matmul(qp, kp.transpose(-1, -2)).view(H, B, G, P)
        if c["window"]:
            old = torch.arange(P, device=q.device) <= P + n - 1 - c["window"]
            before.masked_fill_(old[None, :, None], -math.inf)
        top = torch.maximum(top, before.amax(-1).transpose(0, 1))
    if s["sinks"] is not None:
        top = torch.maximum(top, s["sinks"].view(H, G))
    base = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(scores - base[..., None])
    total = p.sum(-1)
    out = torch.matmul(p, torch.where(seen[:, None, :, None], v, 0.0))
    if P:
        p = torch.exp(before - base.transpose(0, 1)[..., None])
        total = total + p.sum(-1).transpose(0, 1)
        out = out + torch.matmul(p.view(H, B * G, P), vp).view(H, B, G, d).transpose(0, 1)
    if s["sinks"] is not None:
        total = total + torch.exp(s["sinks"].view(H, G) - base)
    out = out / torch.where(total > 0, total, 1.0)[..., None]
    lse = base + torch.log(total)
    return {"out": out.reshape(B, -1).to(torch.bfloat16), "lse": lse.reshape(B, -1)}


def _sample(s):
    z = s["logits"].double()
    z = torch.where(torch.isnan(z), -math.inf, z)
    B, V = z.shape
    z, index = torch.sort(z, dim=1, descending=True, stable=True)
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    far = (z - z[:, :1]) / torch.where(greedy, 1.0, t)
    p = torch.exp(torch.where(z == z[:, :1], 0.0, far))
    rank = torch.arange(V, device=z.device)
    k = s["top_k"].long()[:, None]
    k = torch.where((k <= 0) | (k > V), V, k)
    k = torch.where(greedy, 1, k)
    p = torch.where(rank < k, p, 0.0)
    upto = torch.cumsum(p, 1)
    top_p = s["top_p"].double()[:, None]
    kept = (p > 0) & ((upto - p < top_p * upto[:, -1:]) | (rank == 0) | ~(top_p < 1))
    kept &= (p >= s["min_p"].double()[:, None]) | (rank == 0)
    p = torch.where(kept, p, 0.0)
    p = torch.zeros_like(p).scatter_(1, index, p)  # back in the order of the tokens
    upto = torch.cumsum(p, 1)
    total = upto[:, -1:]
    goal = s["u"].double()[:, None] * total
    token = (upto <= goal).sum(1).clamp(max=V - 1)
    none = z[:, 0] == -math.inf
    logprob = torch.log(p.gather(1, token[:, None]) / total)[:, 0]
    return {"token": torch.where(none, -1, token).to(torch.int32),
            "logprob": torch.where(none, -math.inf, logprob).float()}


# ------------------------------------------------------------------ the framework's calls

_workspaces = {}


def _workspace(F, op, nbytes):
    """A program's workspace for one kind of call: initialized once, as large as it needs."""
    w = _workspaces.get(op)
    if w is None or w.numel() < nbytes:
        w = _workspaces[op] = torch.empty(nbytes, device="cuda", dtype=torch.uint8)
        F.flint_workspace_init(w, nbytes)
    return w


def _call(s):
    import int4_expert_routing_b200 as F
    c = s["case"]
    if c["op"] == "sample":
        F.flint_sample(s["logits"], c["V"], c["B"], c["V"], s["temperature"], s["top_k"],
                       s["top_p"], s["min_p"], s["u"], s["token"], s["logprob"])
        return {"token": s["token"], "logprob": s["logprob"]}
    if "cache" not in s:  # the handle that a program keeps with its pages
        s["cache"] = F.make_kv_cache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    d = c["dim"]
    if c["op"] == "append":
        nb = F.flint_workspace_bytes(F.FLINT_OP_APPEND, c["T"])
        row = (c["q_heads"] + 2 * c["kv_heads"]) * d
        F.flint_kv_append(s["cache"], s["q"], row, s["k"], row, s["v"], row, c["T"], c["q_heads"],
                          s["slots"], s["pos"], c["rope"], c["interleaved"], 10_000.0,
                          s["q_norm"], s["k_norm"], s["q_out"], c["q_heads"] * d,
                          _workspace(F, "append", nb), nb)
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    nb = F.flint_attn_workspace_bytes(c["B"], c["q_heads"], c["kv_heads"], d)
    F.flint_attn_decode(s["cache"], s["q"], c["q_heads"] * d, c["B"], c["q_heads"], s["table"],
                        s["table"].shape[1], s["lens"], s["prefix_pages"], c["prefix"], s["scale"],
                        c["window"], s["sinks"], s["out"], c["q_heads"] * d, s["lse"],
                        _workspace(F, "attend", nb), nb)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _call(state)
    return {"append": _append, "attend": _attend, "sample": _sample}[state["case"]["op"]](state)


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_append(s):
    c = s["case"]
    d, rope = c["dim"], c["rope"]
    pos = s["pos"].cpu().numpy().astype(np.float64)

    def turned(x, weight):
        x = x.float().cpu().numpy().astype(np.float64).reshape(c["T"], -1, d)
        if weight is not None:
            x = x / np.sqrt(np.mean(x * x, axis=2, keepdims=True) + EPS)
            x = x * weight.float().cpu().numpy().astype(np.float64)
        out = x.copy()
        for i in range(rope // 2):
            j, k = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + rope // 2)
            turn = (pos * 10_000.0 ** (-2.0 * i / rope))[:, None]
            out[:, :, j] = x[:, :, j] * np.cos(turn) - x[:, :, k] * np.sin(turn)
            out[:, :, k] = x[:, :, k] * np.cos(turn) + x[:, :, j] * np.sin(turn)
        return out

    q, k = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"])
    v = s["v"].float().cpu().numpy().astype(np.float64).reshape(c["T"], -1, d)
    slots = s["slots"].cpu().numpy()
    got = {"q": torch.from_numpy(q.reshape(c["T"], -1))}
    for name, x in (("k", k), ("v", v)):
        pages = s[name + "_pages"].float().cpu().numpy().astype(np.float64)
        if s[name + "_scale"] is not None:
            x = x / s[name + "_scale"].cpu().numpy().astype(np.float64)[:, None]
            x = np.clip(x, -E4M3_MAX, E4M3_MAX)
        pages[slots // c["page"], :, slots % c["page"]] = x
        got[name + "_pages"] = torch.from_numpy(pages)
    return got


def _exact_attend(s):
    c = s["case"]
    P, H, d, page = c["prefix"], c["kv_heads"], c["dim"], c["page"]
    G = c["q_heads"] // H
    lens = s["lens"].tolist()
    out = torch.zeros(c["B"], H, G, d, dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], H, G), -math.inf, dtype=torch.float64, device="cuda")

    def keys(name, pages, count):
        x = s[name + "_pages"]
        rows = [x[int(i)].double() for i in pages[:-(-count // page)]]
        if not rows:
            return torch.zeros(H, 0, d, dtype=torch.float64, device="cuda")
        x = torch.cat(rows, 1)[:, :count]
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"].double()[:, None, None]
        return x

    first = s["prefix_pages"].tolist() if P else []
    kp, vp = keys("k", first, P), keys("v", first, P)
    table = s["table"].tolist()
    for b in range(c["B"]):
        k = torch.cat([kp, keys("k", table[b], lens[b])], 1)
        v = torch.cat([vp, keys("v", table[b], lens[b])], 1)
        if c["window"]:
            k, v = k[:, -c["window"]:], v[:, -c["window"]:]
        x = s["q"][b].double().view(H, G, d) @ k.transpose(1, 2) * s["scale"]
        if s["sinks"] is not None:
            x = torch.cat([x, s["sinks"].double().view(H, G, 1)], 2)
            v = torch.cat([v, torch.zeros(H, 1, d, dtype=torch.float64, device="cuda")], 1)
        if x.shape[2]:
            lse[b] = torch.logsumexp(x, 2)
            out[b] = torch.exp(x - lse[b][..., None]) @ v
    return {"out": out.reshape(c["B"], -1), "lse": lse.reshape(c["B"], -1)}


def _exact_sample(s):
    B, V = s["case"]["B"], s["case"]["V"]
    logits = s["logits"].double().cpu().numpy()
    t, k, top_p, min_p, u = (s[n].double().cpu().numpy()
                             for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    token, logprob = np.full(B, -1), np.full(B, -np.inf)
    for b in range(B):
        z = np.where(np.isnan(logits[b]), -np.inf, logits[b])
        best = int(np.argmax(z))
        if z[best] == -np.inf:
            continue
        if not t[b] > 0:
            token[b], logprob[b] = best, 0.0
            continue
        order = np.argsort(-z, kind="stable")
        if 0 < k[b] < V:
            order = order[:int(k[b])]
        p = np.exp((z[order] - z[best]) / t[b])
        if top_p[b] < 1:
            before = np.concatenate([[0.0], np.cumsum(p)[:-1]])
            order = order[before < max(top_p[b], 1e-300) * p.sum()]
        order = np.sort(order)
        p = np.exp((z[order] - z[best]) / t[b])
        p = np.where((p >= min_p[b]) | (order == best), p, 0.0)
        upto = np.cumsum(p)
        i = min(int(np.searchsorted(upto, u[b] * upto[-1], side="right")), len(p) - 1)
        token[b], logprob[b] = order[i], math.log(p[i] / upto[-1])
    return {"token": torch.from_numpy(token.astype(np.int32)), "logprob": torch.from_numpy(logprob)}


def exact(case, seed):
    f = {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]]
    return f(prepare(case, seed))
