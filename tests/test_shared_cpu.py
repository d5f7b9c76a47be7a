"""Host side of shared-prefix decode: the plan's counts against the layout
written out, and the refusals, all without a GPU."""
import ctypes

import numpy as np
import pytest

import split_kv_flashdecoding_gb300 as fd

P = ctypes.c_void_p
PREFIXES = [([4], [2048]), ([32], [65536]), ([1], [1]), ([3, 0, 70], [300, 1000, 129]),
            ([5, 9], [0, 4097]), ([200, 1, 31], [7777, 128, 20001]), ([256], [32768])]


def indptr(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


def counts(reqs, lens, Hq, Hkv, chunk):
    """CTAs and partial rows of a plan, prefix by prefix."""
    items = rows = 0
    for r, n in zip(reqs, lens):
        if r and n:
            splits = -(-n // chunk)
            length = -(-(-(-n // splits)) // 128) * 128
            assert (splits - 1) * length < n <= splits * length and length <= chunk
            items += splits * -(-r * Hq // Hkv // 256) * Hkv
            rows += splits * r * Hq
    return items, rows


@pytest.mark.parametrize("reqs,lens", PREFIXES)
@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (32, 8), (64, 8), (2, 1)])
@pytest.mark.parametrize("chunk", [0, 128, 4096])
def test_plan_counts(reqs, lens, Hq, Hkv, chunk):
    B = sum(reqs)
    p = fd.plan_shared(B, Hq, Hkv, 128, indptr(reqs), indptr(lens), 100, num_sms=152, chunk=chunk)
    assert p.chunk % 128 == 0 and (not chunk or p.chunk == chunk)
    assert (p.num_items, p.num_partial_rows) == counts(reqs, lens, Hq, Hkv, p.chunk)
    assert p.workspace_bytes >= p.suffix.workspace_bytes + p.num_partial_rows * 129 * 4
    assert p.suffix.total_tokens == 100 and p.prefix_rows == sum(lens) and p.page_size == 0
    assert p.timeout_ns == fd.DEFAULT_TIMEOUT_NS


@pytest.mark.parametrize("page", [16, 48, 128])
def test_paged_plan_is_the_plan_of_its_keys(page):
    reqs, lens = [3, 40, 1], [1000, 48 * 16, 5]
    cnt = -(-np.array(lens) // page)
    a = fd.plan_shared(44, 32, 8, 128, indptr(reqs), indptr(lens), 64, num_sms=152)
    b = fd.plan_shared_paged(44, 32, 8, 128, page, indptr(reqs), indptr(cnt),
                             np.array(lens) - (cnt - 1) * page, 64, num_sms=152)
    assert (a.chunk, a.num_items, a.num_partial_rows, a.workspace_bytes) == \
        (b.chunk, b.num_items, b.num_partial_rows, b.workspace_bytes)
    assert b.page_size == page and b.prefix_rows == cnt.sum()


def test_one_long_prefix_fills_the_sms_in_one_wave():
    p = fd.plan_shared(32, 32, 8, 128, [0, 32], [0, 65536], 0, num_sms=152)
    assert 144 <= p.num_items <= 152


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), -1), (dict(batch=3), -1), (dict(Hq=7), -1), (dict(Hq=24), -2), (dict(D=64), -2),
    (dict(req=[1, 4]), -1), (dict(ip=[1, 4]), -1), (dict(req=[0, 5, 4], ip=[0, 1, 2]), -1),
    (dict(req=[0, 4], ip=[0, -1]), -1), (dict(room=-1), -1), (dict(room=1 << 31), -1), (dict(chunk=64), -1),
    (dict(chunk=-128), -1), (dict(req=[0, 4], ip=[0, 1, 2]), -1),
], ids=str)
def test_plan_refusals(kw, code):
    a = dict(batch=4, Hq=8, Hkv=8, D=128, req=[0, 4], ip=[0, 100], room=10, chunk=0) | kw
    with pytest.raises(fd.FdError) as e:
        fd.plan_shared(a["batch"], a["Hq"], a["Hkv"], a["D"], a["req"], a["ip"], a["room"], num_sms=152,
                       chunk=a["chunk"])
    assert e.value.code == code


@pytest.mark.parametrize("page,last,code", [(8, [4], -2), (0, [4], -2), (16, [0], -1), (16, [17], -1),
                                            (16, [4, 4], -1)])
def test_paged_plan_refusals(page, last, code):
    with pytest.raises(fd.FdError) as e:
        fd.plan_shared_paged(4, 8, 8, 128, page, [0, 4], [0, 3], last, 10, num_sms=152)
    assert e.value.code == code


def _plan(room=10, paged=False):
    if paged:
        return fd.plan_shared_paged(4, 8, 8, 128, 16, [0, 4], [0, 7], [4], room, num_sms=152)
    return fd.plan_shared(4, 8, 8, 128, [0, 4], [0, 100], room, num_sms=152)


def _call(plan, **kw):
    a = dict(req=P(256), ip=P(256), kv=P(256), q=P(256), kp=P(256), vp=P(256), k=P(256), v=P(256), scale=0.1,
             o=P(256), lse=P(256), ws=P(256), wsb=1 << 40)
    a.update(kw)
    return fd.lib().fd_decode_shared(None if plan is None else ctypes.byref(plan), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(req=None), -1), (dict(ip=None), -1), (dict(kv=None), -1), (dict(q=None), -1), (dict(kp=None), -1),
    (dict(v=None), -1), (dict(o=None), -1), (dict(lse=None), -1), (dict(q=P(8)), -1), (dict(kp=P(8)), -1),
    (dict(k=P(8)), -1), (dict(o=P(8)), -1), (dict(lse=P(2)), -1), (dict(req=P(2)), -1), (dict(ws=None), -3),
    (dict(wsb=1000), -3), (dict(ws=P(8)), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
], ids=str)
def test_decode_refusals(kw, code):
    assert _call(_plan(), **kw) == code


def test_decode_refuses_a_bad_plan():
    assert _call(None) == -1
    for field, value in (("chunk", 100), ("chunk", 0), ("num_items", -1), ("num_prefixes", 0), ("page_size", 16),
                         ("prefix_rows", -1)):
        p = _plan()
        setattr(p, field, value)
        assert _call(p) == -1, field
    p = _plan()
    p.suffix.num_work += 1
    assert _call(p) == -1
    assert _call(_plan(paged=True)) == -1


def test_decode_refuses_a_plan_that_its_workspace_does_not_hold():
    """A plan changed by hand: what the kernels would write lies behind the
    workspace that the plan asks for."""
    changes = [dict(chunk=128 * 40), dict(num_partial_rows=1 << 20), dict(workspace_bytes=0), dict(prefix_rows=1 << 31),
               dict(chunk=128 * 40, num_items=1 << 20)]
    for change in changes:
        p = _plan()
        for field, value in change.items():
            setattr(p, field, value)
        assert _call(p) == -1, change
    p = _plan()
    p.suffix.workspace_bytes -= 1024
    assert _call(p) == -1


def _paged(plan, **kw):
    a = dict(pages=9, req=P(256), ip=P(256), last=P(256), ids=P(256), kv=P(256), kvl=P(256), kvi=P(256), e=3,
             q=P(256), k=P(256), v=P(256), scale=0.1, o=P(256), lse=P(256), ws=P(256), wsb=1 << 40)
    a.update(kw)
    return fd.lib().fd_decode_shared_paged(ctypes.byref(plan), *a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(pages=0), dict(pages=1 << 28), dict(last=None), dict(ids=None), dict(kv=None), dict(kvl=None),
    dict(kvi=None), dict(e=-1), dict(k=None), dict(ids=P(2)), dict(kvi=P(3)), dict(v=P(24)),
], ids=str)
def test_paged_decode_refusals(kw):
    assert _paged(_plan(paged=True), **kw) == -1


def test_paged_decode_refuses_a_ragged_plan():
    assert _paged(_plan()) == -1
