"""Arguments that the cache, attention and sampling calls refuse on the host, before any launch
(no GPU: the pointers are never dereferenced)."""
import ctypes

import pytest

import int4_expert_routing_b200 as F

P = 1 << 20  # aligned, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    F.build()
    return F.lib()


def cache(**kw):
    c = dict(k=P, v=P, type=F.FLINT_KV_BF16, num_pages=10, page_size=16, heads=4, head_dim=128,
             page_stride=4 * 16 * 128, head_stride=16 * 128, token_stride=128, k_scale=None,
             v_scale=None)
    c.update(kw)
    return F.flint_kv_cache(**c)


def append(c=None, **kw):
    a = dict(q=P, q_stride=4096, k=P, k_stride=512, v=P, v_stride=512, T=3, q_heads=32, slots=P,
             pos=P, rope_dim=128, interleaved=False, theta=1e4, q_norm=P, k_norm=P, q_out=P,
             q_out_stride=4096, ws=P, ws_bytes=256, stream=0)
    a.update(kw)
    F.flint_kv_append(c if c is not None else cache(), **a)


def attend(c=None, **kw):
    a = dict(q=P, q_stride=4096, B=3, q_heads=32, page_table=P, max_pages=5, lens=P,
             prefix_pages=P, prefix_len=20, scale=0.1, window=0, sinks=P, out=P + 65536,
             out_stride=4096, lse=P, ws=P, ws_bytes=1 << 40, stream=0)
    a.update(kw)
    F.flint_attn_decode(c if c is not None else cache(), **a)


def refused(f, *args, **kw):
    with pytest.raises(F.FlintError) as e:
        f(*args, **kw)
    assert e.value.code == F.FLINT_EINVAL, kw


BAD_CACHES = [
    dict(k=None), dict(v=P + 8), dict(type=2), dict(type=-1), dict(num_pages=0), dict(page_size=0),
    dict(page_size=8), dict(page_size=24), dict(page_size=4112), dict(heads=0), dict(heads=257),
    dict(head_dim=96), dict(head_dim=256), dict(token_stride=64), dict(token_stride=132),
    dict(head_stride=100), dict(page_stride=0), dict(page_stride=-16), dict(page_stride=1 << 41),
    dict(head_stride=8 * 128), dict(type=F.FLINT_KV_E4M3, token_stride=136),
    dict(type=F.FLINT_KV_E4M3, k_scale=P + 2), dict(type=F.FLINT_KV_E4M3, v_scale=P + 1)]


@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches(kw):
    refused(append, cache(**kw))
    refused(attend, cache(**kw))


@pytest.mark.parametrize("kw", [
    dict(T=0), dict(T=-1), dict(T=F.MAX_APPEND_T + 1), dict(q_heads=0), dict(q_heads=30),
    dict(q_heads=68), dict(q_stride=4095), dict(q_stride=4097), dict(k_stride=511),
    dict(v_stride=516), dict(k=None), dict(v=None), dict(k=P + 2), dict(slots=None),
    dict(slots=P + 4), dict(pos=None), dict(pos=P + 2), dict(rope_dim=-16), dict(rope_dim=8),
    dict(rope_dim=144), dict(theta=0.0), dict(theta=-1.0), dict(theta=float("nan")),
    dict(theta=float("inf")), dict(q_norm=P + 2), dict(k_norm=P + 8), dict(q_out=None),
    dict(q_out=P, q_out_stride=4104), dict(q_out=P + 65536, q_out_stride=4000), dict(ws=None),
    dict(ws=P + 4), dict(ws_bytes=255), dict(q=None)])
def test_bad_appends(kw):
    refused(append, **kw)


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(B=F.MAX_ATTN_B + 1), dict(q_heads=0), dict(q_heads=2), dict(q_heads=31),
    dict(q_heads=68), dict(q=None), dict(q=P + 2), dict(q_stride=4088), dict(q_stride=4100),
    dict(out=None), dict(out_stride=4000), dict(out=P, out_stride=4104), dict(page_table=None),
    dict(page_table=P + 2), dict(max_pages=0), dict(lens=None), dict(lens=P + 1),
    dict(prefix_len=-1), dict(prefix_pages=None), dict(prefix_pages=P + 3), dict(max_pages=1 << 27),
    dict(prefix_len=1 << 30), dict(scale=float("nan")), dict(window=-1), dict(sinks=P + 2),
    dict(lse=P + 2), dict(ws=None), dict(ws=P + 8), dict(ws_bytes=1000)])
def test_bad_attention(kw):
    refused(attend, **kw)


@pytest.mark.parametrize("kw", [
    dict(logits=None), dict(logits=P + 4), dict(B=0), dict(B=65536), dict(V=0),
    dict(V=F.MAX_VOCAB + 1, stride=1 << 20), dict(stride=99), dict(stride=-100),
    dict(temperature=P + 2), dict(top_k=P + 1), dict(top_p=P + 2), dict(min_p=P + 3), dict(u=None),
    dict(u=P + 2), dict(token=None), dict(token=P + 2), dict(logprob=P + 1)])
def test_bad_samples(kw):
    a = dict(logits=P, stride=100, B=2, V=100, temperature=P, top_k=P, top_p=P, min_p=P, u=P,
             token=P, logprob=P, stream=0)
    a.update(kw)
    refused(F.flint_sample, **a)


def test_workspace_sizes():
    W = F.flint_attn_workspace_bytes
    assert W(0, 32, 4, 128) == 0 and W(F.MAX_ATTN_B + 1, 32, 4, 128) == 0
    assert W(1, 32, 5, 128) == 0 and W(1, 68, 4, 128) == 0 and W(1, 32, 4, 96) == 0
    assert 0 < W(1, 32, 4, 64) < W(1, 32, 4, 128) <= W(64, 32, 4, 128) < W(4096, 32, 4, 128)
    assert F.flint_workspace_bytes(F.FLINT_OP_APPEND, 1) == 256
    assert F.flint_workspace_bytes(F.FLINT_OP_APPEND, F.MAX_APPEND_T + 1) == 0


def test_null_cache():
    code = F.lib().flint_kv_append(None, P, 4096, P, 512, P, 512, 1, 32, P, P, 0, 0, 1e4, None,
                                   None, P, 4096, P, 256, None)
    assert code == F.FLINT_EINVAL
    code = F.lib().flint_attn_decode(None, P, 4096, 1, 32, P, 1, P, None, 0, 0.1, 0, None, P, 4096,
                                     None, P, 1 << 40, None)
    assert code == F.FLINT_EINVAL


def test_binding_refuses_host_tensors_and_odd_pages():
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    refused(F.make_kv_cache, k, k)          # not on the device
    for v in (k[:2], k.transpose(1, 2), k.float(), k.to(torch.float8_e4m3fn)):
        with pytest.raises((ValueError, F.FlintError)):
            F.make_kv_cache(k, v)
    with pytest.raises(ValueError):
        F.make_kv_cache(k.float(), k.float())
    with pytest.raises(ValueError):
        F.make_kv_cache(k.transpose(2, 3), k.transpose(2, 3))
    z = torch.zeros(1, 10)
    refused(F.flint_sample, z, 10, 1, 10, None, None, None, None, z, z, None, stream=0)


def test_struct_matches_the_header():
    """The binding's struct has flint.h's fields in its order."""
    import os
    import re
    text = open(os.path.join(os.path.dirname(F.HERE), "include", "flint.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\} flint_kv_cache;", text).group(1)
    names = re.findall(r"(\w+)\s*;", body)
    assert names == [n for n, _ in F.flint_kv_cache._fields_]
    assert ctypes.sizeof(F.flint_kv_cache) == 80


def test_theta_below_one_and_tables_too_large():
    """Angles that grow with the pair's number, and more tiles in all than the plan counts."""
    refused(append, theta=0.5)
    refused(attend, B=F.MAX_ATTN_B, max_pages=1 << 20, prefix_len=20)


def test_binding_refuses_a_cache_of_another_device(monkeypatch):
    """The cache's tensors are on device 1, the call's (raw addresses) wherever the current one is."""
    c = cache()
    c._device = 1
    monkeypatch.setattr(F, "_device", lambda: 0)
    refused(append, c)
    refused(attend, c)
