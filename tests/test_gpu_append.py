"""flint_kv_append on the GPU against the definition in 64 bits.

Tolerance of a value y = a cos t - b sin t from bf16 inputs: one rounding to the stored type (half
a step of it, or of its smallest subnormal), and in fp32 before it: the norm (128 squares summed
by 8 lanes of 16 and a tree, a reciprocal root of 2 units, two products: below 32 units of 2^-24),
the angle (a fraction of a turn rounded to fp32: pi 2^-24, sincospi's 2 units) and three roundings,
all relative to |a| + |b|: together below 2^-18 of it."""
import pytest

import int4_expert_routing_b200 as F
from cache_util import E4M3_MAX, gen, half_step, make_pages, normal, turned
from gpu_util import torch as _torch

pytestmark = pytest.mark.gpu
torch = _torch()


def build(seed, T, q_heads, heads, dim, kv, page, start, extra_pages=2, layout="hnd"):
    g = gen(seed)
    rows = normal(g, T, (q_heads + 2 * heads) * dim)
    rows[:, 5::41] *= 10
    qkv = rows.to(torch.bfloat16)
    pages = -(-T // page) + extra_pages
    k, v = (make_pages(g, kv, pages, heads, page, dim) for _ in range(2))
    order = torch.randperm(pages * page, generator=g)[:T]
    pos = torch.arange(T) + start
    return g, qkv, k, v, order, pos.to(torch.int32)


def run(qkv, k, v, slots, pos, q_heads, rope, inter, theta, qn, kn, ks=None, vs=None, cache=None,
        stream=None):
    T, heads, dim = qkv.shape[0], k.shape[1], k.shape[3]
    dev = [x.cuda() if x is not None else None for x in (qkv, k, v, slots, pos, qn, kn, ks, vs)]
    qkv, k, v, slots, pos, qn, kn, ks, vs = dev
    q_out = torch.full((T, max(q_heads, 1) * dim), 7.0, dtype=torch.bfloat16, device="cuda")
    nb = F.flint_workspace_bytes(F.FLINT_OP_APPEND, T)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    F.flint_workspace_init(ws, nb)
    c = F.make_kv_cache(k, v, ks, vs)
    row = qkv.shape[1]
    F.flint_kv_append(c, qkv if q_heads else None, row, qkv[:, q_heads * dim:], row,
                      qkv[:, (q_heads + heads) * dim:], row, T, q_heads, slots, pos, rope, inter,
                      theta, qn, kn, q_out if q_heads else None, q_out.shape[1], ws, nb, stream)
    torch.cuda.synchronize()
    return q_out.cpu(), k.cpu(), v.cpu(), F.flint_read_status(ws)


def near(got, want, size, dtype, scale=1.0):
    """Within one rounding to `dtype` and the fp32 work before it."""
    got, want = got.double(), want / scale
    if dtype == torch.float8_e4m3fn:
        want = want.clamp(-E4M3_MAX, E4M3_MAX)
    least = 2.0 ** -10 if dtype == torch.float8_e4m3fn else 2.0 ** -134
    before = 2.0 ** -18 * size / scale
    tol = half_step(dtype) * (want.abs() + before) + least + before
    assert torch.isfinite(got).all()
    worst = ((got - want).abs() / tol).max()
    assert worst <= 1, float(worst)


@pytest.mark.parametrize("T,q_heads,heads,dim,rope,inter,norm,kv,page,start", [
    (1, 32, 4, 128, 128, False, True, "bf16", 16, 0),
    (5, 32, 4, 128, 128, False, True, "bf16", 16, 1_000_003),
    (33, 32, 4, 128, 0, False, True, "bf16", 64, 17),
    (1037, 16, 8, 64, 32, True, False, "e4m3", 48, 4093),
    (2500, 32, 4, 128, 128, False, True, "bf16", 64, 0),     # blocks of four tokens, ragged end
    (2501, 8, 8, 128, 64, True, True, "e4m3", 32, 99),
    (77, 3, 1, 64, 64, False, True, "bf16", 16, 2_000_000_000),
    (19, 0, 2, 128, 128, True, True, "e4m3", 4096, 5),       # keys and values alone
    (7, 16, 1, 64, 16, False, False, "bf16", 112, 31),
])
def test_append(T, q_heads, heads, dim, rope, inter, norm, kv, page, start):
    g, qkv, k, v, slots, pos = build(T + dim, T, q_heads, heads, dim, kv, page, start)
    qn = kn = ks = vs = None
    if norm:
        qn, kn = ((1 + 0.2 * normal(g, dim)).to(torch.bfloat16) for _ in range(2))
    if kv == "e4m3":
        ks, vs = (0.2 + torch.rand(heads, generator=g) for _ in range(2))
    q1, k1, v1, status = run(qkv, k, v, slots, pos, q_heads, rope, inter, 10_000.0, qn, kn, ks, vs)
    assert status == F.FLINT_OK
    d = dim
    if q_heads:
        want, size = turned(qkv[:, :q_heads * d].view(T, -1, d), qn, pos, rope, inter, 10_000.0)
        near(q1.view(T, -1, d), want, size, torch.bfloat16)
    want, size = turned(qkv[:, q_heads * d:(q_heads + heads) * d].view(T, -1, d), kn, pos, rope,
                        inter, 10_000.0)
    vw = qkv[:, (q_heads + heads) * d:].view(T, -1, d).double()
    pg, row = slots // page, slots % page
    for new, old, w, sz, sc in ((k1, k, want, size, ks), (v1, v, vw, 0 * vw, vs)):
        got = new.double()[pg, :, row]
        near(got, w, sz, new.dtype, 1.0 if sc is None else sc.double()[None, :, None])
        # every other row is as it was
        new, old = new.view(torch.int16 if kv == "bf16" else torch.uint8), \
            old.view(torch.int16 if kv == "bf16" else torch.uint8)
        left = torch.ones(old.shape[0], page, dtype=torch.bool)
        left[pg, row] = False
        assert torch.equal(new.transpose(1, 2)[left], old.transpose(1, 2)[left])


def test_append_values_exact():
    """V in bf16 is a copy, NaN and infinities included; E4M3 saturates and keeps NaN."""
    _, qkv, k, v, slots, pos = build(3, 6, 4, 2, 64, "bf16", 16, 0)
    qkv[1, -64:] = float("inf")
    qkv[2, -64:] = float("nan")
    _, _, v1, _ = run(qkv, k, v, slots, pos, 4, 64, False, 1e4, None, None)
    want = qkv[:, 6 * 64:].view(6, 2, 64)
    got = v1[slots // 16, :, slots % 16]
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[~got.isnan()], want[~want.isnan()])
    k8, v8 = (x.to(torch.float8_e4m3fn) for x in (k, v))
    _, _, v1, _ = run(qkv, k8, v8, slots, pos, 4, 64, False, 1e4, None, None)
    got = v1.float()[slots // 16, :, slots % 16]
    assert (got[1, 1] == E4M3_MAX).all() and got[2, 1].isnan().all()


def test_append_padding_and_bad_slots():
    """A negative slot writes nothing, its q row neither; a slot past the last page is reported
    and skipped; the tokens around them are written."""
    _, qkv, k, v, slots, pos = build(4, 9, 4, 2, 128, "bf16", 16, 0)
    good = run(qkv, k, v, slots, pos, 4, 128, False, 1e4, None, None)
    pad = slots.clone()
    pad[3] = -1
    pad[8] = -(1 << 40)
    q1, k1, v1, status = run(qkv, k, v, pad, pos, 4, 128, False, 1e4, None, None)
    assert status == F.FLINT_OK
    assert (q1[[3, 8]] == 7.0).all()
    rest = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(q1[rest], good[0][rest])
    kw, vw = good[1].clone(), good[2].clone()
    for t in (3, 8):
        kw[slots[t] // 16, :, slots[t] % 16] = k[slots[t] // 16, :, slots[t] % 16]
        vw[slots[t] // 16, :, slots[t] % 16] = v[slots[t] // 16, :, slots[t] % 16]
    assert torch.equal(k1, kw) and torch.equal(v1, vw)
    pad[3] = k.shape[0] * 16      # the first slot behind the cache
    pad[8] = 1 << 62
    q2, k2, v2, status = run(qkv, k, v, pad, pos, 4, 128, False, 1e4, None, None)
    assert status == F.FLINT_EDEVICE
    assert torch.equal(q2, q1) and torch.equal(k2, kw) and torch.equal(v2, vw)


@pytest.mark.parametrize("dim,kv", [(128, "bf16"), (64, "e4m3")])
def test_append_layouts_in_place_and_streams(dim, kv):
    """Pages with heads inside rows, K and V in one allocation, queries turned in place, another
    stream: the same bits as the dense call."""
    _, qkv, k, v, slots, pos = build(5, 40, 8, 2, dim, kv, 16, 7)
    want = run(qkv, k, v, slots, pos, 8, dim, False, 1e4, None, None)
    kc, vc = k.cuda(), v.cuda()
    both = torch.empty(k.shape[0], 2, 16, 2, dim, dtype=k.dtype, device="cuda")  # [pages][k, v][row][head]
    both[:, 0], both[:, 1] = kc.transpose(1, 2), vc.transpose(1, 2)
    cache = F.make_kv_cache(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))
    x, sl, ps = qkv.cuda(), slots.cuda(), pos.cuda()
    nb = F.flint_workspace_bytes(F.FLINT_OP_APPEND, 40)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    row = x.shape[1]
    F.flint_kv_append(cache, x, row, x[:, 8 * dim:], row, x[:, 10 * dim:], row, 40, 8, sl, ps, dim,
                      False, 1e4, None, None, x, row, ws, nb, stream=side)
    side.synchronize()
    assert torch.equal(x[:, :8 * dim].cpu(), want[0])
    assert torch.equal(x[:, 8 * dim:].cpu(), qkv[:, 8 * dim:])
    bits = torch.int16 if kv == "bf16" else torch.uint8
    assert torch.equal(both[:, 0].transpose(1, 2).cpu().contiguous().view(bits), want[1].view(bits))
    assert torch.equal(both[:, 1].transpose(1, 2).cpu().contiguous().view(bits), want[2].view(bits))


def test_append_captured():
    """Captured once, replayed with other slots and positions in the same buffers."""
    _, qkv, k, v, slots, pos = build(6, 12, 4, 2, 128, "bf16", 16, 0)
    kc, vc, x, sl, ps = (t.cuda() for t in (k, v, qkv, slots, pos))
    q_out = torch.zeros(12, 4 * 128, dtype=torch.bfloat16, device="cuda")
    nb = F.flint_workspace_bytes(F.FLINT_OP_APPEND, 12)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    cache = F.make_kv_cache(kc, vc)
    row = x.shape[1]

    def call():
        F.flint_kv_append(cache, x, row, x[:, 512:], row, x[:, 768:], row, 12, 4, sl, ps, 128, True,
                          1e4, None, None, q_out, 512, ws, nb)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for shift in (0, 3):
        sl.copy_((slots + shift) % (k.shape[0] * 16))
        ps.copy_(pos + 50 * shift)
        kc.copy_(k), vc.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = run(qkv, k, v, (slots + shift) % (k.shape[0] * 16), pos + 50 * shift, 4, 128, True,
                   1e4, None, None)
        assert torch.equal(q_out.cpu(), want[0]) and torch.equal(kc.cpu(), want[1])
        assert torch.equal(vc.cpu(), want[2])


def test_append_far_page():
    """A page whose first element is past 2^32 elements from the cache's base."""
    page, heads, dim = 4096, 8, 128
    per = page * heads * dim
    pages = (1 << 32) // per + 2
    if torch.cuda.mem_get_info()[0] < 3 * per * pages * 2:
        pytest.skip("not enough device memory")
    kc = torch.zeros(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = gen(8)
    kv = normal(g, 2, 2 * heads * dim).to(torch.bfloat16).cuda()
    slots = torch.tensor([pages * page - 1, 0], device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    nb = F.flint_workspace_bytes(F.FLINT_OP_APPEND, 2)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    row = kv.shape[1]
    F.flint_kv_append(F.make_kv_cache(kc, vc), None, 0, kv, row, kv[:, heads * dim:], row, 2, 0,
                      slots, pos, 0, False, 1e4, None, None, None, 0, ws, nb)
    torch.cuda.synchronize()
    assert F.flint_read_status(ws) == F.FLINT_OK
    assert torch.equal(kc[-1, :, -1].reshape(-1), kv[0, :heads * dim])
    assert torch.equal(vc[-1, :, -1].reshape(-1), kv[0, heads * dim:])
    assert torch.equal(kc[0, :, 0].reshape(-1), kv[1, :heads * dim])
    assert int((kc[1:-1] != 0).sum()) == 0
