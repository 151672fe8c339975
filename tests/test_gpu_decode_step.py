"""One decode step as a program runs it: for each layer the qkv projection (flint_int4_gemv), the
append, the attention, the output projection and the MoE block (flint_moe_decode_residual), then
the head and the sampling, captured into one graph on one stream and replayed token after token.

Teacher-forced: every call is checked against the definition in 64 bits on the GPU's own inputs
to it.  Layer 0 has a window and rotary positions, layer 1 neither and reads the batch's shared
prefix.  Tolerances as in the calls' own tests."""
import math

import pytest

import int4_expert_routing_b200 as F
import synth
from cache_util import attend, gen, half_step, normal, sample, turned
from gpu_util import torch as _torch
from gpu_util import workspace

pytestmark = pytest.mark.gpu
torch = _torch()

HQ, H, D, HID, V, PAGE, PREFIX, WINDOW = 32, 4, 128, 2048, 5003, 16, 70, 33
SCALE = D ** -0.5


class Int4:
    """Weights of an int4 GEMV and its call's buffers."""

    def __init__(self, seed, N, K, B):
        q = synth.random_bytes(seed, 77, N * K // 2).reshape(N, K // 2)
        s = synth.scale_bits(seed, 78, N * K // 128).reshape(N, K // 128)
        self.q, self.s = torch.from_numpy(q).cuda(), torch.from_numpy(s.view("int16")).cuda()
        self.N, self.K, self.B = N, K, B
        self.y = torch.zeros(B, N, device="cuda")
        self.nb = F.flint_gemv_workspace_bytes(N, B)
        self.ws = torch.zeros(self.nb, dtype=torch.uint8, device="cuda")
        F.flint_workspace_init(self.ws, self.nb)

    def __call__(self, x):
        F.flint_int4_gemv(self.q, self.s, self.N, self.K, x, self.B, self.y, None, self.ws, self.nb)
        return self.y


class Step:
    def __init__(self, B, lens):
        g = gen(B)
        self.B = B
        pages = 40 + -(-PREFIX // PAGE)
        order = torch.randperm(pages, generator=g).tolist()
        self.pre = torch.tensor([order.pop() for _ in range(-(-PREFIX // PAGE))], dtype=torch.int32)
        self.table = torch.tensor([[order.pop() for _ in range(4)] for _ in range(B)],
                                  dtype=torch.int32)
        self.lens0 = lens
        dev = dict(device="cuda")
        self.slots, self.pos = torch.zeros(B, dtype=torch.int64, **dev), torch.zeros(B, dtype=torch.int32, **dev)
        self.lens = torch.zeros(B, dtype=torch.int32, **dev)
        self.h = torch.zeros(B, HID, **dev)
        self.u = torch.zeros(B, **dev)
        self.token = torch.zeros(B, dtype=torch.int32, **dev)
        self.logprob = torch.zeros(B, **dev)
        self.sinks = normal(g, HQ).cuda()
        self.norms = [(1 + 0.1 * normal(g, D)).to(torch.bfloat16).cuda() for _ in range(2)]
        self.d_pre, self.d_table = self.pre.cuda(), self.table.cuda()
        self.layers = []
        for l in range(2):
            kv = "bf16" if l else "e4m3"
            t = torch.bfloat16 if l else torch.float8_e4m3fn
            k, v = (normal(g, pages, H, PAGE, D).to(t).cuda() for _ in range(2))
            ks, vs = (None, None) if l else ((0.02 + 0.02 * torch.rand(2, H, generator=g)).cuda())
            self.layers.append(dict(
                k=k, v=v, ks=ks, vs=vs, cache=F.make_kv_cache(k, v, ks, vs), kv=kv,
                qkv=Int4(10 + l, (HQ + 2 * H) * D, HID, B), o=Int4(20 + l, HID, HQ * D, B),
                moe=F.make_layer(synth.layer_device(l, "cuda")),
                rows=torch.zeros(B, (HQ + 2 * H) * D, dtype=torch.bfloat16, **dev),
                q_out=torch.zeros(B, HQ * D, dtype=torch.bfloat16, **dev),
                att=torch.zeros(B, HQ * D, dtype=torch.bfloat16, **dev),
                lse=torch.zeros(B, HQ, **dev), rope=0 if l else D, window=0 if l else WINDOW))
        self.head = Int4(30, V, HID, B)
        self.ws_a, self.nb_a = workspace(F.FLINT_OP_APPEND, B)
        self.nb_t = F.flint_attn_workspace_bytes(B, HQ, H, D)
        self.ws_t = torch.zeros(self.nb_t, dtype=torch.uint8, device="cuda")
        F.flint_workspace_init(self.ws_t, self.nb_t)
        self.ws_m, self.nb_m = workspace(F.FLINT_OP_DECODE, B)

    def norm(self):
        h = self.h
        return (h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def run(self):
        B, width = self.B, (HQ + 2 * H) * D
        for y in self.layers:
            rows = y["rows"]
            rows.copy_(y["qkv"](self.norm()))
            F.flint_kv_append(y["cache"], rows, width, rows[:, HQ * D:], width,
                              rows[:, (HQ + H) * D:], width, B, HQ, self.slots, self.pos, y["rope"],
                              False, 1e4, *self.norms, y["q_out"], HQ * D, self.ws_a, self.nb_a)
            F.flint_attn_decode(y["cache"], y["q_out"], HQ * D, B, HQ, self.d_table, 4, self.lens,
                                self.d_pre, PREFIX, SCALE, y["window"], self.sinks, y["att"],
                                HQ * D, y["lse"], self.ws_t, self.nb_t)
            self.h += y["o"](y["att"])
            F.flint_moe_decode_residual(y["moe"], self.h, B, None, None, self.ws_m, self.nb_m)
        F.flint_sample(self.head(self.norm()), V, B, V, None, None, None, None, self.u, self.token,
                       self.logprob)

    def place(self, step, g):
        """The step's token of every sequence: where it goes and what enters the layers."""
        n = [x + step + 1 for x in self.lens0]
        self.lens.copy_(torch.tensor(n, dtype=torch.int32))
        self.pos.copy_(torch.tensor([PREFIX + x - 1 for x in n], dtype=torch.int32))
        self.slots.copy_(torch.tensor([int(self.table[b, (x - 1) // PAGE]) * PAGE + (x - 1) % PAGE
                                       for b, x in enumerate(n)]))
        self.h.copy_(normal(g, self.B, HID))
        self.u.copy_(torch.rand(self.B, generator=g))
        return n

    def outputs(self):
        return [self.h, self.token, self.logprob, self.head.y] + \
            [y[n] for y in self.layers for n in ("q_out", "att", "lse")] + \
            [y[n].view(torch.uint8) for y in self.layers for n in ("k", "v")]

    def check(self, n):
        pos = self.pos.cpu()
        for y in self.layers:
            rows = y["rows"].cpu().double()
            q, size = turned(rows[:, :HQ * D].view(-1, HQ, D), self.norms[0].cpu(), pos, y["rope"],
                             False, 1e4)
            got = y["q_out"].cpu().double().view(-1, HQ, D)
            # one rounding to bf16; fp32 norm and rotation before it
            assert ((got - q).abs() <= half_step(torch.bfloat16) * q.abs() + 2.0 ** -18 * size).all()
            k, size = turned(rows[:, HQ * D:(HQ + H) * D].view(-1, H, D), self.norms[1].cpu(), pos,
                             y["rope"], False, 1e4)
            t = torch.bfloat16 if y["kv"] == "bf16" else torch.float8_e4m3fn
            sc = [1.0 if s is None else s.cpu().double()[:, None, None] for s in (y["ks"], y["vs"])]
            ck, cv = (y[x].cpu().double() * s for x, s in zip(("k", "v"), sc))
            for b, x in enumerate(n):
                page, r = int(self.table[b, (x - 1) // PAGE]), (x - 1) % PAGE
                for c, want, s in ((ck, k[b], sc[0]),
                                   (cv, rows[b, (HQ + H) * D:].view(H, D), sc[1])):
                    s = s[:, 0] if torch.is_tensor(s) else s
                    most = 448 * s if y["kv"] == "e4m3" else math.inf
                    top = torch.as_tensor(most, dtype=torch.float64)
                    # below E4M3's normal numbers a step is 2^-9
                    least = 2.0 ** -10 * s if y["kv"] == "e4m3" else 0.0
                    want = torch.minimum(torch.maximum(want, -top), top)
                    tol = half_step(t) * want.abs() * (1 + 2.0 ** -10) + 2.0 ** -18 * size[b] + least
                    assert ((c[page, :, r] - want).abs() <= tol).all()
                keys, values = (torch.cat(
                    [torch.cat([c[int(p)] for p in self.pre], 1)[:, :PREFIX],
                     torch.cat([c[int(p)] for p in self.table[b]], 1)[:, :x]], 1)
                    for c in (ck, cv))
                want, wl, size_o = attend(y["q_out"][b].cpu().view(HQ, D), keys, values, SCALE,
                                          y["window"], self.sinks.cpu())
                err = (y["att"][b].cpu().double().view(HQ, D) - want).abs()
                assert (err <= half_step(torch.bfloat16) * want.abs() + 2.0 ** -7 * size_o).all()
                assert ((y["lse"][b].cpu().double() - wl).abs() <= 2.0 ** -11).all()
        for b in range(self.B):
            u = float(self.u[b])
            token, logprob, (ends, last) = sample(self.head.y[b].cpu(), 1.0, 0, 1.0, 0.0, u)
            i = int(self.token[b])
            # a running mass is within 2^-16 of the definition's (test_gpu_sample.py)
            assert i == token or abs(float(ends[min(i, token)]) - u) <= 2.0 ** -15
            if i == token:
                assert abs(float(self.logprob[b]) - logprob) <= 2.0 ** -14 + 2.0 ** -22 * abs(logprob)
        for ws in (self.ws_a, self.ws_t, self.ws_m):
            assert F.flint_read_status(ws) == F.FLINT_OK


@pytest.mark.parametrize("B", [1, 3, 7])
def test_decode_step(B):
    """Eager and replayed steps give the same bits (cache contents included), each call its
    definition's result."""
    F.build()
    a, b = Step(B, [0, 14, 31, 1, 15, 16, 40][:B]), Step(B, [0, 14, 31, 1, 15, 16, 40][:B])
    a.place(0, gen(5)), b.place(0, gen(5))
    a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    for step in range(4):
        n = a.place(step, gen(step))
        b.place(step, gen(step))
        a.run()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.outputs(), b.outputs()):
            assert torch.equal(x, y)
        b.check(n)
    del graph
