"""flint_attn_decode on the GPU against the definition in 64 bits.

Tolerance, relative to the size A = sum p |v| / sum of what an output is summed from: one rounding
of the output to bf16 (2^-8 of the value); before it in fp32 the scores (head_dim products of
|q k| <= 100 in all: below 2^-12 of p after the exponential), the sums of n weights and products
(n 2^-24 <= 2^-10 of A for the tests' lengths) and the weights' rounding in the second product:
two bf16 terms (2^-16) or fp16 (2^-11) for a sequence's own keys; for the shared prefix one bf16
term where the tensor cores take it (2^-8).  Together 2^-9 of A without a prefix, 2^-7 with one."""
import math

import pytest

import int4_expert_routing_b200 as F
from cache_util import NAN8, attend, gen, half_step, make_pages, normal
from gpu_util import torch as _torch

pytestmark = pytest.mark.gpu
torch = _torch()


def build(seed, lens, q_heads, heads, dim, kv, page, prefix, sinks, spare=3, garbage=True):
    """Pages in random order; every row that no sequence owns holds NaN."""
    g = gen(seed)
    need = [max(0, -(-n // page)) for n in lens]
    first = -(-prefix // page)
    total = sum(need) + first + spare
    order = torch.randperm(total, generator=g).tolist()
    k, v = (make_pages(g, kv, total, heads, page, dim) for _ in range(2))
    ks = vs = None
    if kv == "e4m3":
        ks, vs = (0.5 + torch.rand(heads, generator=g) for _ in range(2))
    used = torch.zeros(total, page, dtype=torch.bool)
    pre = [order.pop() for _ in range(first)]
    for i, pg in enumerate(pre):
        used[pg, :max(0, min(page, prefix - i * page))] = True
    most = max(1, max(need) + 1)
    table = torch.full((len(lens), most), -5, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = order.pop()
            used[table[b, i], :max(0, min(page, lens[b] - i * page))] = True
    if garbage:
        for x in (k, v):
            if kv == "bf16":
                x.transpose(1, 2)[~used] = math.nan
            else:
                x.view(torch.uint8).transpose(1, 2)[~used] = NAN8
    q = (1.3 * normal(g, len(lens), q_heads * dim)).to(torch.bfloat16)
    sk = 1.5 * normal(g, q_heads) if sinks else None
    return dict(k=k, v=v, ks=ks, vs=vs, table=table, lens=torch.tensor(lens, dtype=torch.int32),
                pre=torch.tensor(pre, dtype=torch.int32) if prefix else None, prefix=prefix, q=q,
                sinks=sk, heads=heads, dim=dim, q_heads=q_heads, page=page)


def to_dev(s):
    return {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in s.items()}


def call(d, scale, window=0, out=None, lse=None, ws=None, stream=None, q=None, q_stride=None,
         cache=None, lens=None):
    B, width = d["lens"].numel(), d["q_heads"] * d["dim"]
    out = torch.full((B, width), 9.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((B, d["q_heads"]), 9.0, device="cuda") if lse is None else lse
    nb = F.flint_attn_workspace_bytes(B, d["q_heads"], d["heads"], d["dim"])
    if ws is None:
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        F.flint_workspace_init(ws, nb)
    c = cache or F.make_kv_cache(d["k"], d["v"], d["ks"], d["vs"])
    F.flint_attn_decode(c, d["q"] if q is None else q, q_stride or width, B, d["q_heads"],
                        d["table"], d["table"].shape[1], d["lens"], d["pre"], d["prefix"], scale,
                        window, d["sinks"], out, out.stride(0), lse, ws, nb, stream)
    return out, lse, ws


def reference(s, b, scale, window):
    """Sequence b of the host inputs."""
    n, heads, dim = int(s["lens"][b]), s["heads"], s["dim"]

    def rows(x, sc, pages, count):
        if count <= 0:
            return torch.zeros(heads, 0, dim).double()
        y = torch.cat([x[int(p)].double() for p in pages[:-(-count // s["page"])]], 1)[:, :count]
        return y if sc is None else y * sc.double()[:, None, None]

    if n < 0:
        pre = 0
    else:
        pre = s["prefix"]
    keys, values = (torch.cat([rows(x, sc, s["pre"] if pre else [], pre),
                               rows(x, sc, s["table"][b], n)], 1)
                    for x, sc in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    return attend(s["q"][b].view(-1, dim), keys, values, scale, window, s["sinks"])


def check(s, out, lse, scale, window=0, rows=None):
    B, dim = s["lens"].numel(), s["dim"]
    weight = 2.0 ** -7 if s["prefix"] else 2.0 ** -9
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(B) if rows is None else rows:
        want, wl, size = reference(s, b, scale, window)
        got = out[b].view(-1, dim)
        assert torch.isfinite(got).all(), b
        tol = half_step(torch.bfloat16) * want.abs() + weight * size + 1e-30
        worst = ((got - want).abs() / tol).max()
        assert worst <= 1, (b, float(worst))
        inf = torch.isinf(wl)
        assert torch.equal(torch.isinf(lse[b]), inf)
        assert ((lse[b] - wl)[~inf].abs() <= 2.0 ** -11).all(), b


@pytest.mark.parametrize("q_heads,heads,dim,kv,page", [
    (32, 4, 128, "bf16", 16), (8, 8, 64, "bf16", 64), (12, 4, 128, "e4m3", 32),
    (16, 1, 64, "e4m3", 48), (16, 1, 128, "bf16", 128), (10, 2, 128, "e4m3", 112),
    (9, 1, 128, "bf16", 4096), (7, 7, 64, "e4m3", 16)])
@pytest.mark.parametrize("sinks", [False, True])
def test_own_keys(q_heads, heads, dim, kv, page, sinks):
    """Ragged lengths from none to several tiles, the ends inside tiles and pages."""
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 200, 1025, -1, 300]
    s = build(q_heads + dim + page, lens, q_heads, heads, dim, kv, page, 0, sinks)
    out, lse, ws = call(to_dev(s), dim ** -0.5)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_OK
    check(s, out, lse, dim ** -0.5)
    assert (out[[0, 12]] == 0).all()


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 100, 513])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("prefix", [0, 1, 77, 200])
def test_window(window, kv, prefix):
    """The last `window` keys: inside the own keys, reaching into the prefix, or all of both.  The
    values before the window are NaN for the sequence with the least left."""
    lens = [0, 1, 40, 64, 101, 600, -1]
    s = build(window + prefix, lens, 16, 2, 128, kv, 32, prefix, True)
    out, lse, ws = call(to_dev(s), 0.1, window)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_OK
    check(s, out, lse, 0.1, window)


def test_window_hides_nan():
    """Keys and values that no window reaches hold NaN and infinities; each sequence's own window
    stays clean though others' masked rows share its tiles."""
    for kv in ("bf16", "e4m3"):
        s = build(11, [100, 130, 90], 8, 2, 64, kv, 16, 150, False)
        W = 70
        for x in (s["k"], s["v"]):
            for b, n in enumerate(s["lens"].tolist()):
                for j in range(n - W):
                    row = x[int(s["table"][b, j // 16])][:, j % 16]
                    if kv == "bf16":
                        row[:] = math.nan if j % 2 else math.inf
                    else:
                        row.view(torch.uint8)[:] = NAN8
            for j in range(150):   # the windows end inside the own keys
                row = x[int(s["pre"][j // 16])][:, j % 16]
                if kv == "bf16":
                    row[:] = math.nan
                else:
                    row.view(torch.uint8)[:] = NAN8
        out, lse, _ = call(to_dev(s), 0.125, W)
        check(s, out, lse, 0.125, W)


@pytest.mark.parametrize("B,q_heads,heads,dim,kv,page,prefix", [
    (1, 32, 4, 128, "bf16", 16, 1), (1, 8, 8, 64, "bf16", 64, 130), (2, 32, 4, 128, "bf16", 48, 777),
    (3, 16, 1, 128, "e4m3", 32, 500), (5, 32, 4, 128, "bf16", 64, 4097),
    (16, 32, 4, 128, "bf16", 64, 1000), (17, 32, 4, 128, "bf16", 128, 2048),
    (33, 12, 4, 64, "bf16", 16, 300), (40, 32, 4, 128, "e4m3", 64, 1111),
    (70, 16, 2, 128, "bf16", 32, 63), (9, 20, 4, 64, "e4m3", 16, 640),
    (130, 8, 8, 128, "bf16", 64, 129), (64, 16, 1, 64, "bf16", 80, 333)])
@pytest.mark.parametrize("sinks", [False, True])
def test_shared_prefix(B, q_heads, heads, dim, kv, page, prefix, sinks):
    lens = [(37 * b * b + 5 * b) % 150 for b in range(B)]
    lens[0] = 0
    if B > 4:
        lens[3] = -1
    s = build(B + prefix, lens, q_heads, heads, dim, kv, page, prefix, sinks)
    out, lse, ws = call(to_dev(s), dim ** -0.5)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_OK
    check(s, out, lse, dim ** -0.5, rows=range(0, B, max(1, B // 12)))


def test_prefix_equals_own_keys():
    """The same keys as a shared prefix and as each sequence's own: the same function."""
    B, P, page = 20, 256, 64
    s = build(21, [P + 30] * B, 32, 4, 128, "bf16", page, 0, True)
    for b in range(1, B):
        s["table"][b, :P // page] = s["table"][0, :P // page]
    a, la, _ = call(to_dev(s), 0.1)
    t = dict(s, pre=s["table"][0, :P // page].clone(), prefix=P,
             table=s["table"][:, P // page:].contiguous(), lens=s["lens"] - P)
    b_, lb, _ = call(to_dev(t), 0.1)
    check(s, a, la, 0.1, rows=range(0, B, 3))
    check(t, b_, lb, 0.1, rows=range(0, B, 3))


def test_large_and_small_scores():
    """Scores far apart (a softmax of one key), far below the sink, and scale 0."""
    s = build(31, [700, 90, 1], 16, 2, 128, "bf16", 64, 0, True)
    for scale in (0.0, 4.0, -1.0):
        out, lse, _ = call(to_dev(s), scale)
        out, lse = out.cpu().double(), lse.cpu().double()
        for b in range(3):
            want, wl, size = reference(s, b, scale, 0)
            # scores reach 4 * 500: 2^-20 of them is 2^-9 of p
            tol = half_step(torch.bfloat16) * want.abs() + 2.0 ** -7 * size + 1e-6
            assert ((out[b].view(-1, 128) - want).abs() <= tol).all()
            assert ((lse[b] - wl).abs() <= 2.0 ** -20 * (wl.abs() + 500)).all()


@pytest.mark.parametrize("kv,dim,B", [("bf16", 128, 20), ("e4m3", 64, 40), ("bf16", 64, 1)])
def test_shared_prefix_scales(kv, dim, B):
    """Scale 0 (all keys alike), a negative and a tiny one, the prefix ending inside a tile."""
    s = build(33 + dim, [(7 * b) % 40 for b in range(B)], 16, 2, dim, kv, 32, 300, False)
    for scale in (0.0, -0.1, 1e-30):
        out, lse, _ = call(to_dev(s), scale)
        check(s, out, lse, scale, rows=range(0, B, 4))


def test_nan_and_inf_where_they_are_seen():
    """A NaN key or value shows in its own sequence and KV head, and in no other."""
    s = build(41, [100, 100, 100], 8, 2, 64, "bf16", 16, 0, False)
    s["k"][int(s["table"][1, 2]), 1, 3, 5] = math.nan
    s["v"][int(s["table"][2, 0]), 0, 7, 9] = math.nan
    out, lse, _ = call(to_dev(s), 0.125)
    o = out.cpu().view(3, 2, 4, 64)
    assert torch.isfinite(o[0]).all() and torch.isfinite(o[1, 0]).all()
    assert o[1, 1].isnan().all()
    bad = o[2].isnan()
    assert bad[0, :, 9].all() and int(bad.sum()) == 4


@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("e4m3", 64)])
def test_strides_in_place_and_streams(kv, dim):
    """Heads inside rows and K and V in one allocation, q as part of a fused row, out over q,
    another stream: the same bits."""
    s = build(51, [70, 3, 0, 200], 8, 2, dim, kv, 16, 90, True)
    d = to_dev(s)
    want, wl, _ = call(d, 0.1)
    torch.cuda.synchronize()
    pages = d["k"].shape[0]
    both = torch.empty(pages, 2, 16, 2, dim, dtype=d["k"].dtype, device="cuda")
    both[:, 0], both[:, 1] = d["k"].transpose(1, 2), d["v"].transpose(1, 2)
    cache = F.make_kv_cache(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2), d["ks"], d["vs"])
    width = 8 * dim
    wide = torch.full((4, width + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :width] = d["q"]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(d, 0.1, q=wide, q_stride=width + 64, out=wide, stream=side, cache=cache,
         lse=(l2 := torch.zeros_like(wl)))
    side.synchronize()
    assert torch.equal(wide[:, :width], want) and torch.equal(l2, wl)
    assert (wide[:, width:] == 5.0).all()


def test_repeats_and_shared_workspace():
    """Run to run the same bits, the workspace dirty from other calls."""
    a = to_dev(build(61, [500, 3, 1000, 64], 32, 4, 128, "bf16", 64, 700, True))
    b = to_dev(build(62, [20] * 30, 32, 4, 128, "bf16", 16, 100, False))
    nb = max(F.flint_attn_workspace_bytes(4, 32, 4, 128), F.flint_attn_workspace_bytes(30, 32, 4, 128))
    ws = torch.randint(0, 255, (nb,), dtype=torch.uint8, device="cuda")
    F.flint_workspace_init(ws, 256)  # the status word; the rest stays dirty
    first = call(a, 0.1, ws=ws)[0].clone()
    for _ in range(4):
        call(b, 0.1, ws=ws)
        assert torch.equal(call(a, 0.1, ws=ws)[0], first)
    assert F.flint_read_status(ws) == F.FLINT_OK


def test_two_graphs_on_one_workspace():
    """Two captured calls that share a workspace, replayed in turn with changing lengths."""
    s, t = (build(71 + i, [130, 40, 7, 260], 16, 2, 128, "bf16", 32, 90 * i, True) for i in (0, 1))
    ds, dt = to_dev(s), to_dev(t)
    nb = F.flint_attn_workspace_bytes(4, 16, 2, 128)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    call(ds, 0.1, ws=ws)
    torch.cuda.synchronize()
    for d in (ds, dt):
        out = torch.zeros(4, 16 * 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(4, 16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(d, 0.1, ws=ws, out=out, lse=lse)
        outs.append((out, lse)), graphs.append(graph)
    for lens in ([130, 40, 7, 260], [129, 0, 7, 31], [1, -1, 2, 3]):
        for x, dx in ((s, ds), (t, dt)):
            x["lens"] = torch.tensor(lens, dtype=torch.int32)
            dx["lens"].copy_(x["lens"])
        for i in (0, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        check(s, *outs[0], 0.1)
        check(t, *outs[1], 0.1)
    del graphs
    assert F.flint_read_status(ws) == F.FLINT_OK


def test_many_sequences():
    """More sequences than a block scans at once, most of them empty."""
    lens = [0] * 1500
    for b in (0, 3, 159, 160, 161, 799, 1499):
        lens[b] = 50 + b % 97
    lens[700:710] = [-1] * 10
    s = build(81, lens, 4, 2, 64, "bf16", 16, 0, True)
    out, lse, ws = call(to_dev(s), 0.125)
    check(s, out, lse, 0.125, rows=[0, 1, 3, 159, 160, 161, 705, 799, 1498, 1499])
    s = build(82, lens, 4, 2, 64, "bf16", 16, 100, False)
    out, lse, ws = call(to_dev(s), 0.125)
    check(s, out, lse, 0.125, rows=[0, 1, 3, 159, 160, 161, 705, 799, 1498, 1499])


def test_bad_pages_and_lengths_reported():
    """A page number outside the cache counts as zero keys, a length past the table is cut; both
    are reported, and the other sequences are as they should be."""
    s = build(91, [40, 40, 40], 8, 2, 64, "bf16", 16, 0, False)
    s["table"] = s["table"][:, :3].contiguous()
    for page in (-1, s["k"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = dict(s, table=s["table"].clone())
        t["table"][1, 1] = page
        out, lse, ws = call(to_dev(t), 0.125)
        torch.cuda.synchronize()
        assert F.flint_read_status(ws) == F.FLINT_EDEVICE
        check(t, out, lse, 0.125, rows=[0, 2])
        assert torch.isfinite(out[1]).all()
    t = dict(s, lens=torch.tensor([40, 49, 2 ** 31 - 1], dtype=torch.int32))
    out, lse, ws = call(to_dev(t), 0.125)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_EDEVICE
    check(t, out, lse, 0.125, rows=[0])
    t = dict(build(92, [5] * 20, 32, 4, 128, "bf16", 16, 64, False))
    t["pre"][2] = -7
    out, lse, ws = call(to_dev(t), 0.125)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_EDEVICE


def test_long_cache():
    """Pages past 2^32 elements from the base, and a sequence split over every CTA."""
    page, heads, dim = 4096, 4, 128
    per = page * heads * dim
    pages = (1 << 32) // per + 3
    if torch.cuda.mem_get_info()[0] < 3 * per * pages * 2:
        pytest.skip("not enough device memory")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k = torch.zeros(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    far = [pages - 1, 0, pages - 2]
    for p in far:
        k[p].normal_(generator=g), v[p].normal_(generator=g)
    n = 2 * page + 1777
    q = torch.empty(1, 32 * dim, device="cuda").normal_(generator=g).to(torch.bfloat16)
    d = dict(k=k, v=v, ks=None, vs=None, table=torch.tensor([far], dtype=torch.int32, device="cuda"),
             lens=torch.tensor([n], dtype=torch.int32, device="cuda"), pre=None, prefix=0, q=q,
             sinks=None, heads=heads, dim=dim, q_heads=32, page=page)
    out, lse, ws = call(d, 0.09)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_OK
    keys, values = (torch.cat([x[p].cpu() for p in far], 1)[:, :n] for x in (k, v))
    want, wl, size = attend(q[0].cpu().view(32, dim), keys, values, 0.09, 0, None)
    err = (out.cpu().double().view(32, dim) - want).abs()
    assert (err <= half_step(torch.bfloat16) * want.abs() + 2.0 ** -9 * size).all()
    assert ((lse.cpu().double()[0] - wl).abs() <= 2.0 ** -11).all()
