"""Host side of the INT8 cache's operators: refusals, before any CUDA call."""
import ctypes

import numpy as np
import pytest

import split_kv_flashdecoding_gb300 as fd
from tests.test_cache_cpu import _append

P = ctypes.c_void_p


def test_scale_heads():
    assert [fd.scale_heads(n) for n in (1, 2, 3, 4, 5, 8, 9)] == [4, 4, 4, 4, 8, 8, 12]


def _decode(**kw):
    ip, last = np.array([0, 2], dtype=np.int32), np.array([5], dtype=np.int32)
    a = dict(batch=1, hq=8, hkv=8, d=128, page=16, pages=4, ip=ip.ctypes.data_as(P), last=last.ctypes.data_as(P),
             ipd=P(256), lastd=P(256), ids=P(256), q=P(256), k=P(256), v=P(256), ks=P(256), vs=P(256), scale=0.1,
             o=P(256), lse=P(256), ws=P(256), wsb=1 << 30)
    a.update(kw)
    return fd.lib().fd_decode_paged_int8(*a.values(), None)




@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(d=64), -2), (dict(page=8), -2), (dict(page=0), -2), (dict(ip=None), -1),
    (dict(last=None), -1),
], ids=str)
def test_decode_int8_refusals(kw, code):
    assert _decode(**kw) == code


def test_bindings_refuse_wrong_caches():
    import torch
    i32 = torch.int32
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    pool, scale = torch.zeros((4, 16, 8, 128), dtype=torch.int8), torch.zeros((4, 8))
    z = torch.zeros(2, dtype=i32)
    with pytest.raises(fd.FdError):   # tables of another length
        fd.decode_paged_int8(q, pool, pool, scale, scale, [0, 1, 2], [3], z, z, z, 0.1)
    with pytest.raises(fd.FdError):   # not on a GPU
        fd.decode_paged_int8(q, pool, pool, scale, scale, [0, 1], [3], z, z, z, 0.1)


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(n=-1), -1), (dict(hkv=0), -1), (dict(hq=-1), -1), (dict(entries=-1), -1),
    (dict(d=64), -2), (dict(page=8), -2), (dict(pages=0), -1), (dict(pages=1 << 28), -1), (dict(ws=None), -3),
    (dict(wsb=255), -3), (dict(q=None), -1), (dict(vp=None), -1), (dict(k=P(264)), -1), (dict(kp=P(264)), -1),
    (dict(sk=None), -1), (dict(sv=P(258)), -1), (dict(n=1 << 28, hkv=8), -1), (dict(batch=0), 0), (dict(n=0), 0),
], ids=str)
def test_append_int8_refusals(kw, code):
    assert _append("fd_append_paged_int8", **kw) == code


def test_append_int8_refuses_queries_written_over_inputs():
    base, pool = 1 << 20, P(1 << 30)
    inputs = dict(n=5, hq=8, hkv=4, q=P(base), qs=2176, k=P(base + 2 * 1024), ks=2176, v=P(base + 2 * 1536), vs=2176)
    for at in (8, 512, 1600):
        assert _append("fd_append_paged_int8", **inputs, qo=P(base + 2 * at), qos=2176, kp=pool, vp=pool) == -1
