"""Host-side checks of the paged-cache entry points (no GPU needed): every bad
argument is refused with the documented status before anything is enqueued,
and the binding refuses what it can see."""
import ctypes

import pytest
import torch

import bit_group_quantized_qgemv_gb300 as q
from bit_group_quantized_qgemv_gb300._binding import KVCacheStruct

EINVAL, ENULL, EALIGN = -1, -2, -3
L = q.lib


def ptr(v=0x10000):
    return ctypes.c_void_p(v)


def cache(**kw):
    d = dict(k=0x10000, v=0x20000, page_table=0x30000, kv_len=0x40000, n_pages=10, page_size=16,
             n_kv=2, head_dim=128, n_seqs=3, max_pages=4)
    d.update(kw)
    return KVCacheStruct(*[d[n] for n, _ in KVCacheStruct._fields_])


def rope(c=None, **kw):
    p = ptr()
    d = dict(qkv=p, qkv_stride=8 * 128, n_tokens=5, n_q=4, q_start=p, positions=p, inv_freq=p,
             rotary=128, inter=0, q_norm=None, k_norm=None, eps=1e-6, q_out=p, q_stride=512,
             pos=None, mass=None, err=None, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return L.qgemv_qk_norm_rope_append(None if c == 0 else ctypes.byref(c or cache()), *d.values())


def attention(c=None, **kw):
    p = ptr()
    d = dict(q=p, q_stride=512, n_tokens=5, n_q=4, q_start=p, max_q=2, scale=0.1, out=p,
             out_stride=512, lse=None, ws=None, ws_bytes=0, err=None, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return L.qgemv_paged_attention(None if c == 0 else ctypes.byref(c or cache()), *d.values())


def mass(c=None, **kw):
    p = ptr()
    d = dict(q=p, q_stride=512, n_tokens=5, n_q=4, q_start=p, max_q=2, scale=0.1, lse=p, mass=None,
             mass_out=p, err=None, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return L.qgemv_attention_mass(None if c == 0 else ctypes.byref(c or cache()), *d.values())


def evict(c=None, **kw):
    d = dict(mass=ptr(0x1000), pos=ptr(0x2000), nxt=ptr(0x3000), keep=8, sink=1, recent=2,
             kept=ptr(0x4000), mass_out=ptr(0x5000), pos_out=ptr(0x6000), len_out=ptr(0x7000),
             err=None, stream=None)
    assert set(kw) <= set(d)
    d.update(kw)
    return L.qgemv_cache_evict(None if c == 0 else ctypes.byref(c or cache()), *d.values())


CALLS = [rope, attention, mass, evict]


@pytest.mark.parametrize("call", CALLS)
def test_cache_descriptor(call):
    assert call(0) == ENULL
    for n in ("k", "v", "page_table", "kv_len"):
        assert call(cache(**{n: None})) == ENULL
    for kw in (dict(page_size=8), dict(page_size=512), dict(page_size=48), dict(page_size=0),
               dict(page_size=-16), dict(head_dim=32), dict(head_dim=96), dict(head_dim=256),
               dict(n_pages=0), dict(n_kv=0), dict(n_kv=1025), dict(n_seqs=0), dict(n_seqs=65536),
               dict(max_pages=0), dict(max_pages=-1), dict(max_pages=(1 << 25) + 1),
               dict(n_pages=1 << 26, n_kv=2)):
        assert call(cache(**kw)) == EINVAL, kw
    for kw in (dict(k=0x10008), dict(v=0x10002), dict(page_table=0x10002), dict(kv_len=0x10001)):
        assert call(cache(**kw)) == EALIGN, kw


def test_rope_append_checks():
    p = ptr()
    for n in ("qkv", "q_start", "positions", "inv_freq", "q_out"):
        assert rope(**{n: None}) == ENULL
    assert rope(q_norm=p) == ENULL and rope(k_norm=p) == ENULL
    for kw in (dict(n_tokens=-1), dict(n_q=3), dict(n_q=0), dict(n_q=65536), dict(rotary=130),
               dict(rotary=-8), dict(rotary=12), dict(rotary=136), dict(qkv_stride=8 * 128 - 4),
               dict(qkv_stride=8 * 128 + 2), dict(q_stride=508), dict(q_stride=514),
               dict(q_norm=p, k_norm=p, eps=0.0), dict(q_norm=p, k_norm=p, eps=float("nan")),
               dict(q_norm=p, k_norm=p, eps=float("inf"))):
        assert rope(**kw) == EINVAL, kw
    for n in ("qkv", "q_out"):
        assert rope(**{n: ptr(0x10004)}) == EALIGN
    for n in ("q_start", "positions", "inv_freq", "pos", "mass", "err"):
        assert rope(**{n: ptr(0x10002)}) == EALIGN
    assert rope(q_norm=ptr(0x10004), k_norm=p) == EALIGN
    assert rope(n_tokens=0) == 0                     # nothing to do, nothing enqueued


@pytest.mark.parametrize("call", [attention, mass])
def test_query_checks(call):
    for kw in (dict(n_tokens=-1), dict(n_q=0), dict(n_q=3), dict(n_q=65536), dict(max_q=0),
               dict(max_q=(1 << 24) + 1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(q_stride=504),
               dict(q_stride=516), dict(max_q=1 << 24, n_q=1000, q_stride=128000)):
        assert call(**kw) == EINVAL, kw
    assert call(q=ptr(0x10008)) == EALIGN
    for n in ("q_start", "lse", "err"):
        assert call(**{n: ptr(0x10002)}) == EALIGN


def test_attention_checks():
    for n in ("q", "q_start", "out"):
        assert attention(**{n: None}) == ENULL
    assert attention(ws_bytes=16) == ENULL
    for kw in (dict(out_stride=504), dict(out_stride=516)):
        assert attention(**kw) == EINVAL, kw
    assert attention(out=ptr(0x10008)) == EALIGN
    assert attention(ws=ptr(0x10008), ws_bytes=64) == EALIGN
    assert attention(n_tokens=0) == 0


def test_mass_checks():
    for n in ("q", "q_start", "lse", "mass_out"):
        assert mass(**{n: None}) == ENULL
    for n in ("mass", "mass_out"):
        assert mass(**{n: ptr(0x10002)}) == EALIGN


def test_evict_checks():
    for n in ("mass", "pos", "nxt", "kept", "mass_out", "pos_out", "len_out"):
        assert evict(**{n: None}) == ENULL
    for kw in (dict(keep=0), dict(keep=-1), dict(keep=(1 << 30) + 1), dict(sink=-1), dict(recent=-1), dict(sink=5, recent=4),
               dict(sink=2 ** 31 - 1, recent=2 ** 31 - 1), dict(mass_out=ptr(0x1000)),
               dict(pos_out=ptr(0x2000)), dict(len_out=ptr(0x40000))):
        assert evict(**kw) == EINVAL, kw
    for n in ("mass", "pos", "nxt", "kept", "mass_out", "pos_out", "len_out", "err"):
        assert evict(**{n: ptr(0x1002)}) == EALIGN


def test_workspace_size_of_bad_arguments_is_zero():
    f = L.qgemv_paged_attention_workspace_bytes
    assert f(None, 5, 4, 2) == 0
    assert f(ctypes.byref(cache(head_dim=96)), 5, 4, 2) == 0
    assert f(ctypes.byref(cache()), 5, 3, 2) == 0
    assert f(ctypes.byref(cache()), 5, 4, 0) == 0


def test_binding_refuses_cpu_tensors():
    k = torch.zeros(2, 1, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        q.kv_cache(k, k, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))


def test_attention_out_is_not_q():
    assert attention(q=ptr(0x20000), out=ptr(0x20000)) == EINVAL
