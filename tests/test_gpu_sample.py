"""flint_sample on the GPU against the definition in 64 bits.

The kernel's weights p are 2^-d with d in fp32 (three roundings of d, at most 2^-22 relative; for
the d below 40 that carry the mass, 2^-17 of p) and ex2's 2^-22; the masses of bins add 2^-23 an
element.  So a running mass is within 2^-16 of the definition's, and the cut of top-p may fall one
token off where the target is that near a token's end, which moves the total by that token's share:
a token's end, relative to the total, is within 2^-15 plus the last kept token's share.  Where u is
further than that from both ends of the definition's token, the token has to be it; nearer, u has
to be within that of the share of the token that came."""
import math

import pytest

import int4_expert_routing_b200 as F
from cache_util import gen, sample
from gpu_util import torch as _torch

pytestmark = pytest.mark.gpu
torch = _torch()
NEAR = 2.0 ** -15


def call(z, T, k, p, m, u, stride=None, logprob=True):
    B, V = z.shape
    dev = [None if x is None else x.cuda() for x in (T, k, p, m, u)]
    z = z.cuda()
    token = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), 7.0, device="cuda") if logprob else None
    F.flint_sample(z, stride or V, B, V, *dev, token, lp)
    torch.cuda.synchronize()
    return token.cpu(), None if lp is None else lp.cpu()


def check(z, T, k, p, m, u):
    B, V = z.shape
    token, lp = call(z, T, k, p, m, u)
    for b in range(B):
        want, wlp, share = sample(z[b], float(T[b]) if T is not None else 1.0,
                                  int(k[b]) if k is not None else 0,
                                  float(p[b]) if p is not None else 1.0,
                                  float(m[b]) if m is not None else 0.0, float(u[b]))
        got, x = int(token[b]), min(max(float(u[b]), 0.0), 1.0)
        off = 0.0
        if share is not None:
            ends, last = share
            off = NEAR + last
            lo, hi = (float(ends[want - 1]) if want else 0.0), float(ends[want])
            if 0 < x < 1 and min(x - lo, hi - x) < off:
                assert 0 <= got < V
                lo, hi = (float(ends[got - 1]) if got else 0.0), float(ends[got])
                assert lo - off <= x <= hi + off, (b, got, want, lo, hi, x)
                # its weight against the kept mass
                y = (float(z[b, got]) - float(z[b][~z[b].isnan()].max())) / (float(T[b]) if T is not None else 1.0)
                wy = (float(z[b, want]) - float(z[b][~z[b].isnan()].max())) / (float(T[b]) if T is not None else 1.0)
                if math.isfinite(y) and math.isfinite(wy):
                    wlp += y - wy
                want = got
        assert got == want, (b, got, want, share and off, float(u[b]))
        if math.isinf(wlp):
            assert float(lp[b]) == wlp
        else:
            assert abs(float(lp[b]) - wlp) <= 2 * (NEAR + off) + 2.0 ** -22 * abs(wlp), \
                (b, float(lp[b]), wlp)


def full(B, v, dtype=torch.float32):
    return torch.full((B,), v, dtype=dtype)


@pytest.mark.parametrize("V", [1, 2, 3, 31, 127, 1000, 2049, 5003, 32768, 50001, 150144, 262144])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (20, 0.95, 0.0), (0, 0.9, 1e-5), (700, 0.5, 0.02),
                                   (0, 0.999, 0.0)])
def test_sample_sizes(V, k, p, m):
    B = 3
    g = gen(V + k)
    z = 1.2 * torch.empty(B, V).exponential_(generator=g) + 0.3 * torch.randn(B, V, generator=g)
    u = torch.rand(B, generator=g)
    check(z, full(B, 0.9), full(B, k, torch.int32), full(B, p), full(B, m), u)


@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.1, 1.0, 10.0, 1000.0])
def test_sample_spreads(spread):
    """From all logits equal to one far above the rest; top-p cuts among ties by index."""
    B, V = 6, 20011
    g = gen(int(spread * 1000))
    z = spread * torch.randn(B, V, generator=g) - 2
    u = torch.tensor([0.0, 0.2, 0.5, 0.77, 0.93, 0.99999])
    check(z, full(B, 1.0), full(B, 5000, torch.int32), full(B, 0.83), None, u)
    check(z, None, None, full(B, 0.83), None, u)


def test_sample_ties():
    """Logits of a few values each thousands of times (16-bit heads give such rows): the cut falls
    inside a value and goes by index."""
    B, V = 4, 50000
    g = gen(2)
    z = torch.randint(0, 6, (B, V), generator=g).float() * 0.25
    z[1] = z[1].neg().where(z[1] != 0, torch.tensor(-0.0))     # +0 and -0 are one value
    z[1, ::3] = z[1, ::3].abs()
    z[2] = 0.0
    z[2, 1::2] = -0.0
    for k, p in ((3000, 1.0), (12345, 1.0), (0, 0.31), (40000, 0.6)):
        check(z, full(B, 1.0), full(B, k, torch.int32), full(B, p), None,
              torch.rand(B, generator=g))


def test_sample_masked_and_odd_values():
    """-inf, the type's lowest value, NaN and +inf among the logits; rows with nothing left."""
    V = 3001
    g = gen(3)
    z = torch.randn(10, V, generator=g)
    low = torch.finfo(torch.float32).min
    z[0, 100:] = -math.inf
    z[1, 100:] = low
    z[2, ::2] = math.nan
    z[3] = -math.inf
    z[4] = math.nan
    z[5, [7, 9, 2000]] = math.inf
    z[6] = low
    z[7] = -math.inf
    z[7, 2999] = low
    z[8] = math.inf
    z[9, 50:] = math.nan
    z[9, :50] = -math.inf
    for k, p, m in ((0, 1.0, 0.0), (200, 1.0, 0.0), (200, 0.9, 0.01), (0, 0.5, 0.0)):
        check(z, full(10, 0.8), full(10, k, torch.int32), full(10, p), full(10, m),
              torch.linspace(0.05, 0.95, 10))
    token, lp = call(z, None, None, None, None, full(10, 0.5))
    assert token[[3, 4, 9]].tolist() == [-1, -1, -1]
    assert torch.isinf(lp[[3, 4, 9]]).all()
    assert int(token[5]) == 9 and abs(float(lp[5]) + math.log(3)) < 1e-6


def test_sample_parameters():
    """Off and extreme settings: greedy, k = 1, top_p 0 and tiny, min_p 1 and above, temperatures
    from tiny to huge, u outside [0, 1)."""
    V = 4099
    g = gen(4)
    z = torch.randn(20, V, generator=g) * 2
    z[:, 17] = z[:, 4000] = 9.0          # the best twice: greedy takes the lower index
    T = torch.tensor([0.0, -1.0, math.nan, 1e-30, 1e30, math.inf, 0.5, 1, 1, 1,
                      1, 1, 1, 1, 1, 1, 1, 1, 1, 1])
    k = torch.tensor([0, 5, 0, 0, 0, 0, 1, -3, V, V + 5, 2, 1, 0, 0, 0, 0, 3, 0, 0, 0],
                     dtype=torch.int32)
    p = torch.tensor([1.0] * 10 + [0.5, 0.5, 0.0, -1.0, 1e-30, math.nan, 2.0, 1.0, 1.0, 1.0])
    m = torch.tensor([0.0] * 16 + [math.nan, 1.0, 1.5, -2.0])
    u = torch.full((20,), 0.6)
    u[16:] = torch.tensor([0.1, 0.7, 0.7, 0.3])
    # the definition's comparisons with NaN: off
    clean = lambda x, off: torch.where(x.isnan(), off, x)  # noqa: E731
    token, lp = call(z, T, k, p, m, u)
    for b in range(20):
        want, wlp, _ = sample(z[b], float(T[b]) if T[b] == T[b] else 0.0, int(k[b]),
                              float(clean(p[b], 1.0)), float(clean(m[b], 0.0)), float(u[b]))
        assert int(token[b]) == want, b
        assert abs(float(lp[b]) - wlp) <= NEAR + 2.0 ** -23 * abs(wlp)
    for u0, at in ((-0.5, 0), (math.nan, 0), (1.0, -1), (7.0, -1)):
        t2, _ = call(z[7:8], None, torch.tensor([50], dtype=torch.int32), None, None,
                     torch.tensor([u0]))
        kept = torch.sort(torch.sort(z[7], descending=True, stable=True).indices[:50]).values
        assert int(t2[0]) == int(kept[at])


@pytest.mark.parametrize("V,stride", [(1001, 1003), (50001, 50005), (50001, 50001)])
def test_sample_strides_batches_and_repeats(V, stride):
    """Rows at odd strides; a row's result does not depend on the batch, the stream or the run."""
    B = 37
    g = gen(5)
    buf = torch.full((B, stride), 1e9)
    buf[:, :V] = torch.empty(B, V).exponential_(generator=g)
    u = torch.rand(B, generator=g)
    k, p, m = full(B, 900, torch.int32), full(B, 0.9), full(B, 1e-4)
    d = [x.cuda() for x in (buf, k, p, m, u)]
    token = torch.zeros(B, dtype=torch.int32, device="cuda")
    lp = torch.zeros(B, device="cuda")
    F.flint_sample(d[0], stride, B, V, None, *d[1:], token, lp)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    t2, lp2 = torch.zeros_like(token), torch.zeros_like(lp)
    torch.cuda.synchronize()
    for _ in range(5):
        F.flint_sample(d[0], stride, B, V, None, *d[1:], t2, lp2, stream=side)
    side.synchronize()
    assert torch.equal(token, t2) and torch.equal(lp, lp2)
    for b in (0, 11, 36):
        t1, lp1 = call(buf[b:b + 1, :V], None, k[:1], p[:1], m[:1], u[b:b + 1])
        assert int(t1[0]) == int(token[b]) and float(lp1[0]) == float(lp[b])
    check(buf[:, :V], None, k, p, m, u)
    t3, none = call(buf[:, :V], None, k, p, m, u, logprob=False)
    assert none is None and torch.equal(t3, token.cpu())


@pytest.mark.parametrize("V", [9000, 150144])
@pytest.mark.parametrize("k", [1, 20, 100, 256])
def test_sample_few_of_uneven_rows(V, k):
    """Top-k of up to 256 where the parts of a row are far apart: sorted both ways, all but one end
    masked, one end far above, a single finite logit, more equal logits than a list holds."""
    g = gen(V + k)
    z = torch.empty(9, V).exponential_(generator=g)
    z[1] = torch.sort(z[1]).values
    z[2] = torch.sort(z[2], descending=True).values
    z[3, V // 8:] = -math.inf
    z[4, :V - 300] = -math.inf
    z[5, :V // 9] += 100
    z[6] = -math.inf
    z[6, V - 1] = -5.0
    z[7, :] = 1.0
    z[8, 500:4500] = 30.0
    u = torch.rand(9, generator=g)
    B = 9
    check(z, full(B, 0.9), full(B, k, torch.int32), full(B, 0.95), full(B, 0.0), u)
    for b in range(9):
        check(z[b:b + 1], full(1, 0.9), full(1, k, torch.int32), None, None, u[b:b + 1])


@pytest.mark.parametrize("k,p,m", [(0, 0.9, 0.0), (0, 0.999, 1e-4), (400, 1.0, 0.0), (900, 0.8, 0.01),
                                   (30, 0.9, 0.0), (0, 1.0, 0.05)])
@pytest.mark.parametrize("T", [0.2, 1.0])
def test_sample_large_batch_equals_single_rows(k, p, m, T):
    """Rows that a full batch reads again from L2 give the bits that they give alone: heavy and
    flat tails, equal logits, masked ones, infinities, more than a list of a bin's elements."""
    g = gen(k + int(1000 * p))
    B, V, stride = 70, 50001, 50003
    z = torch.empty(B, stride).exponential_(generator=g) * 1.1
    z[1] = 0.25
    z[2] = torch.floor(4 * z[2])
    z[3, ::3] = -math.inf
    z[4, 7:9], z[5, 40000] = math.inf, math.inf
    z[6, ::5] = math.nan
    z[7] *= 1e-3
    z[8] *= 1e3
    z[9, :] = -math.inf
    z[10, :25000] = z[10, 0]
    u = torch.rand(B, generator=g)
    u[11], u[12] = 0.0, 1.0
    par = [full(B, T), full(B, k, torch.int32), full(B, p), full(B, m), u]
    token, lp = call_strided(z, V, par)
    for b in list(range(16)) + [69]:
        one, l1 = call(z[b:b + 1, :V].contiguous(), *[x[b:b + 1] for x in par])
        assert int(one[0]) == int(token[b]), b
        assert torch.equal(l1[0], lp[b]), b
    rows = [0, 1, 2, 3, 7, 13, 69]
    check(z[rows, :V].contiguous(), *[x[rows] for x in par])


def call_strided(z, V, par):
    z, dev = z.cuda(), [x.cuda() for x in par]
    token = torch.full((z.shape[0],), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((z.shape[0],), 7.0, device="cuda")
    F.flint_sample(z, z.shape[1], z.shape[0], V, *dev, token, lp)
    torch.cuda.synchronize()
    return token.cpu(), lp.cpu()


def test_sample_distribution():
    """20,000 rows of one small distribution: each token as often as it should be, within six
    standard deviations."""
    B, V = 20000, 8
    z = torch.tensor([0.0, 1.0, -1.0, 2.0, 0.5, -3.0, 1.5, 0.1]).repeat(B, 1)
    u = torch.rand(B, generator=gen(6))
    token, _ = call(z, None, full(B, 6, torch.int32), None, None, u)
    p = torch.softmax(z[0].double(), 0)
    p[[2, 5]] = 0
    p /= p.sum()
    got = torch.bincount(token.long(), minlength=V).double() / B
    assert ((got - p).abs() <= 6 * (p * (1 - p) / B).sqrt() + 1e-12).all()


def test_sample_captured():
    B, V = 5, 7000
    g = gen(7)
    z = torch.randn(B, V, generator=g).cuda()
    u = torch.rand(B, generator=g).cuda()
    k = full(B, 40, torch.int32).cuda()
    token = torch.zeros(B, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.flint_sample(z, V, B, V, None, k, None, None, u, token, None)
    for seed in (8, 9):
        z.copy_(torch.randn(B, V, generator=gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        want, _ = call(z.cpu(), None, k.cpu(), None, None, u.cpu())
        assert torch.equal(token.cpu(), want)
