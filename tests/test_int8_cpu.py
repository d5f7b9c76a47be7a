"""Host side of the INT8 cache's operators: refusals, before any CUDA call."""
import ctypes
import os

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


def _plan_prefill(**kw):
    a = dict(batch=2, hq=8, hkv=4, d=128, page=16, qi=[0, 5, 7], ip=[0, 2, 3], last=[3, 16], causal=1, sms=152, chunk=0)
    a.update(kw)
    for x in ("qi", "ip", "last"):
        a[x] = None if a[x] is None else np.array(a[x], dtype=np.int32).ctypes.data_as(P)
    plan = fd.PrefillPlan()
    return fd.lib().fd_plan_prefill_paged(*a.values(), ctypes.byref(plan)), plan


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(hkv=3), -1), (dict(hq=12), -2), (dict(hq=64), -2),
    (dict(d=64), -2), (dict(page=8), -2), (dict(page=0), -2), (dict(qi=None), -1), (dict(ip=None), -1),
    (dict(last=None), -1), (dict(qi=[1, 5, 7]), -1), (dict(qi=[0, 5, 4]), -1), (dict(ip=[0, 3, 2]), -1),
    (dict(last=[0, 16]), -1), (dict(last=[3, 17]), -1), (dict(chunk=64), -1), (dict(chunk=-128), -1),
    (dict(chunk=1 << 19), -1), (dict(sms=-1), -1), (dict(qi=[0, 5, 2 ** 31 - 1]), -1), (dict(), 0),
    (dict(qi=[0, 0, 0]), 0), (dict(ip=[0, 0, 0], last=[0, 0]), 0),
], ids=str)
def test_plan_prefill_refusals(kw, code):
    assert _plan_prefill(**kw)[0] == code


def test_plan_prefill_counts():
    rc, p = _plan_prefill(hq=32, hkv=8, qi=[0, 100, 101], ip=[0, 63, 64], last=[16, 1], chunk=256)
    # 400 rows a KV head: 2 blocks, 1008 keys: 4 splits; 4 rows: 1 block, 1 split
    assert rc == 0 and p.num_items == 2 * 4 * 8 + 8 and p.num_merged_rows == 100 * 32 and p.num_partial_rows == 100 * 32 * 4
    assert p.workspace_bytes >= 256 + p.num_partial_rows * 129 * 4
    assert _plan_prefill(qi=[0, 0, 0])[1].num_items == 0
    # few rows behind many keys are split over the SMs, many rows are not
    assert _plan_prefill(batch=1, hq=32, hkv=8, qi=[0, 4], ip=[0, 4096], last=[16])[1].num_items >= 140
    assert _plan_prefill(batch=1, hq=32, hkv=8, qi=[0, 40000], ip=[0, 2500], last=[16])[1].num_merged_rows == 0


def _prefill(plan=None, **kw):
    plan = plan or _plan_prefill()[1]
    a = dict(pages=4, qi=P(256), ip=P(256), last=P(256), ids=P(256), q=P(256), qs=1024,
             k=P(256), v=P(256), ks=P(256), vs=P(256), scale=0.1, o=P(256), lse=P(256), ws=P(256), wsb=1 << 30)
    a.update(kw)
    return fd.lib().fd_prefill_paged_int8(ctypes.byref(plan), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(pages=0), -1), (dict(pages=1 << 28), -1), (dict(qi=None), -1), (dict(ip=None), -1),
    (dict(last=None), -1), (dict(ids=None), -1), (dict(q=None), -1), (dict(q=P(264)), -1), (dict(qs=1016), -1),
    (dict(qs=1028), -1), (dict(k=None), -1), (dict(v=P(264)), -1), (dict(ks=None), -1), (dict(vs=P(258)), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(o=None), -1), (dict(o=P(264)), -1),
    (dict(lse=P(258)), -1), (dict(ws=None), -3), (dict(wsb=1000), -3), (dict(ws=P(264)), -1),
], ids=str)
def test_prefill_refusals(kw, code):
    assert _prefill(**kw) == code


@pytest.mark.parametrize("field,value,code", [
    ("num_items", -1, -1), ("num_partial_rows", 1 << 20, -1), ("num_merged_rows", 1 << 20, -1), ("chunk", 100, -1),
    ("head_dim", 64, -2), ("page_size", 8, -2), ("num_kv_heads", 3, -1), ("num_qo_heads", 12, -2), ("workspace_bytes", 0, -1),
    ("num_tokens", -1, -1), ("num_page_entries", -1, -1),
])
def test_prefill_refuses_plans_that_do_not_hold_together(field, value, code):
    plan = _plan_prefill()[1]
    setattr(plan, field, value)
    assert _prefill(plan) == code


def test_prefill_of_nothing_is_nothing():
    assert fd.lib().fd_prefill_paged_int8(None, *[0] * 1, *[None] * 5, 0, *[None] * 4, 0.1, *[None] * 3, 0, None) == -1
    assert _prefill(_plan_prefill(qi=[0, 0, 0])[1], q=None, o=None) == 0


@pytest.mark.parametrize("name", ["prefill_kernel.cu", "tc_stream.cuh"])
def test_no_load_past_the_coherent_path(name):
    """The kernels start while the grid before them may still write their inputs."""
    source = open(os.path.join(os.path.dirname(fd.__file__), "csrc", name)).read()
    code = "\n".join(line.split("//")[0] for line in source.splitlines())
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in code, word


@pytest.mark.parametrize("keys", [262144, 262145, 400000])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8)])
def test_plan_prefill_of_long_prompts(keys, hq, hkv):
    """From 262145 keys on a request is cut, and has its partial rows, whatever its tokens."""
    pages = -(-keys // 16)
    rc, p = _plan_prefill(batch=1, hq=hq, hkv=hkv, qi=[0, keys], ip=[0, pages], last=[keys - 16 * (pages - 1)])
    splits = -(-keys // 262144)
    assert rc == 0 and p.num_partial_rows == (0 if splits == 1 else splits * keys * hq)
    assert p.workspace_bytes >= p.num_partial_rows * 516


def test_plan_prefill_beyond_32_bits_of_rows():
    kw = dict(batch=1, hq=32, hkv=8, ip=[0, 18750], last=[16])   # 300000 keys, two splits
    rc, p = _plan_prefill(qi=[0, (1 << 25) - 1], **kw)
    assert rc == 0 and p.num_partial_rows == ((1 << 25) - 1) * 64
    assert _plan_prefill(qi=[0, 1 << 25], **kw)[0] == -2
    plan = _plan_prefill()[1]
    plan.num_merged_rows = plan.num_partial_rows = 2 ** 31 - 1
    plan.workspace_bytes = 1 << 62
    assert _prefill(plan, wsb=(1 << 63) - 1) == -1


def test_prefill_refuses_outputs_over_other_queries():
    """o over q itself is one thing, over other rows of it another (-3: without a workspace
    it goes no further)."""
    q, row = 1 << 20, 2 * 8 * 128   # bytes of a token's heads, 7 tokens
    for o in (q, q + 7 * row, q - 7 * row):
        assert _prefill(o=P(o), q=P(q), qs=1024, ws=None) == -3
    for o in (q + 16, q + row, q - row, q + 7 * row - 16, q - 7 * row + 16):
        assert _prefill(o=P(o), q=P(q), qs=1024, ws=None) == -1
    assert _prefill(o=P(q), q=P(q), qs=1032, ws=None) == -1
