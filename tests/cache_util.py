"""Plain 64-bit statements of the cache, its attention and the sampling, and the inputs of their
tests (torch on the CPU; nothing of the library)."""
import math

import torch

E4M3_MAX = 448.0
NAN8 = 0x7F  # an E4M3 NaN


def half_step(dtype):
    """Half a step of a type relative to the value: the most one rounding is off."""
    return torch.finfo(dtype).eps / 2


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float32)


# ------------------------------------------------------------------ append
def turned(x, weight, pos, rope, interleaved, theta, eps=1e-6):
    """Heads [T][heads][dim] in 64 bits: RMSNorm with `weight` (None: none), then the rotation of
    the first `rope` elements.  Also the size |a| + |b| of what each output is summed from."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    y, size = x.clone(), x.abs()
    for i in range(rope // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rope // 2)
        t = (pos.double() * theta ** (-2.0 * i / rope))[:, None]
        y[:, :, a] = x[:, :, a] * torch.cos(t) - x[:, :, b] * torch.sin(t)
        y[:, :, b] = x[:, :, b] * torch.cos(t) + x[:, :, a] * torch.sin(t)
        size[:, :, a] = size[:, :, b] = x[:, :, a].abs() + x[:, :, b].abs()
    return y, size


# ------------------------------------------------------------------ attention
def make_pages(g, kv, pages, heads, page, dim, fill=None):
    """K or V pages of N(0, 1) values in the cache's type; `fill` every element instead."""
    x = normal(g, pages, heads, page, dim)
    if fill is not None:
        x = torch.full_like(x, fill)
    return x.to(torch.bfloat16) if kv == "bf16" else x.to(torch.float8_e4m3fn)


def attend(q, keys, values, scale, window, sinks, prefix_only=False):
    """One sequence in 64 bits.  q [heads][dim], keys and values [kv_heads][n][dim] (prefix and own,
    all visible before the window).  Returns out, lse and the size sum p |v| / sum."""
    Hq, d = q.shape
    H, n, _ = keys.shape
    if window > 0:
        keys, values = keys[:, -window:], values[:, -window:]
    k, v = keys.double(), values.double()
    s = q.double().view(H, Hq // H, d) @ k.transpose(1, 2) * scale
    if sinks is not None:
        s = torch.cat([s, sinks.double().view(H, -1, 1)], 2)
        v = torch.cat([v, torch.zeros(H, 1, d, dtype=torch.float64)], 1)
    if s.shape[2] == 0:
        return torch.zeros(Hq, d).double(), torch.full((Hq,), -math.inf).double(), \
            torch.zeros(Hq, d).double()
    lse = torch.logsumexp(s, 2)
    p = torch.exp(s - lse[..., None])
    return (p @ v).reshape(Hq, d), lse.reshape(Hq), (p @ v.abs()).reshape(Hq, d)


# ------------------------------------------------------------------ sampling
def sample(z, temperature, top_k, top_p, min_p, u):
    """One row in 64 bits: (token, logprob, shares).  shares: each token's end of its share of
    the kept mass in index order, relative to the total, and the share of the order's last kept
    token."""
    z = z.double()
    z = torch.where(torch.isnan(z), -math.inf, z)
    V = z.numel()
    top = z.max()
    if top == -math.inf:
        return -1, -math.inf, None
    order = torch.sort(z, descending=True, stable=True).indices
    if not temperature > 0:
        return int(order[0]), 0.0, None
    p = torch.where(z == top, 0.0, (z - top) / temperature).exp()
    k = top_k if 0 < top_k < V else V
    order = order[:k]
    if top_p < 1:
        before = torch.cumsum(p[order], 0) - p[order]
        keep = before < top_p * p[order].sum()
        keep[0] = True
        order = order[keep]
    keep = p[order] >= min_p if min_p > 0 else torch.ones(len(order), dtype=torch.bool)
    keep[0] = True
    order = order[keep & (p[order] > 0)]
    last = float(p[order[-1]])
    order = torch.sort(order).values
    run = torch.cumsum(p[order], 0)
    total = float(run[-1])
    u = min(max(u, 0.0), 1.0) if u == u else 0.0
    at = min(int((run <= u * total).sum()), len(order) - 1)
    ends = torch.cumsum(torch.zeros_like(p).scatter_(0, order, p[order]), 0) / total
    return int(order[at]), math.log(float(p[order[at]]) / total), (ends, last / total)
