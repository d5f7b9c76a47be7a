"""Host side of the cache operators: rotary plans and the refusals of
fd_append_paged, fd_fork_pages, fd_compact_pages and fd_copy_pages, all before
any CUDA call."""
import ctypes
import math
import os

import numpy as np
import pytest

import split_kv_flashdecoding_gb300 as fd

P = ctypes.c_void_p


def frequencies(rotary, base, scaling):
    """f_i in radians per position, written out pair by pair."""
    out = []
    for i in range(rotary // 2):
        f = 1.0 / base ** (2.0 * i / rotary)
        kind = scaling[0] if scaling else None
        if kind == "linear":
            f /= scaling[1]
        elif kind == "bands":
            _, factor, trained, low, high = scaling
            wave = 2 * math.pi / f
            if wave > trained / low:
                f /= factor
            elif wave >= trained / high:
                s = (trained / wave - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        elif kind == "yarn":
            _, factor, trained, low, high = scaling
            pair = lambda n: rotary * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rotary - 1)
            ramp = min(1.0, max(0.0, (i - a) / max(b - a, 1e-3)))
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("rotary", [16, 32, 96, 128])
@pytest.mark.parametrize("scaling", [None, ("linear", 4.0), ("bands", 8.0, 8192, 1.0, 4.0),
                                     ("yarn", 16.0, 4096, 1.0, 32.0)], ids=lambda s: s[0] if s else "plain")
def test_rope_steps_are_the_frequencies(rotary, scaling):
    for base in (10000.0, 500000.0, 1234.5):
        info = fd.plan_rope(128, rotary, base=base, scaling=scaling)
        got = np.array([s / 2.0 ** 64 for s in info.step[: rotary // 2]])
        want = frequencies(rotary, base, scaling) / (2 * math.pi)
        # some ten roundings of 2^-53 each on both sides, and the cut at 2^-64
        # of the fixed-point step (which is over 2^-53 of a step below 2^-11)
        assert np.all(np.abs(got - want) <= 64 * 2.0 ** -53 * want + 2.0 ** -64)
        assert all(s == 0 for s in info.step[rotary // 2:])
        gain = 0.1 * math.log(16.0) + 1 if scaling and scaling[0] == "yarn" else 1.0
        assert abs(info.gain - gain) <= 2.0 ** -23
    # position 1 turns the first pair by one radian
    assert abs(fd.plan_rope(128, 128).step[0] / 2.0 ** 64 - 1 / (2 * math.pi)) < 1e-15


@pytest.mark.parametrize("args,kw,code", [
    ((64, 64), {}, -2), ((128, 8), {}, -2), ((128, 0), {}, -1), ((128, 144), {}, -1),
    ((128, 128), dict(base=0.0), -1), ((128, 128), dict(base=float("nan")), -1),
    ((128, 128), dict(base=0.5), -1), ((128, 128), dict(scaling=("linear", 0.0)), -1),
    ((128, 128), dict(scaling=("linear", float("inf"))), -1),
    ((128, 128), dict(scaling=("bands", 2.0, 0.0, 1.0, 4.0)), -1),
    ((128, 128), dict(scaling=("bands", 2.0, 8192, 4.0, 4.0)), -1),
    ((128, 128), dict(scaling=("yarn", 2.0, 8192, 1.0, 32.0), base=1.0), -1),
    ((128, 128), dict(scaling=("none", 2.0)), -1), ((128, 128), dict(scaling=("bands", 2.0)), -1),
])
def test_rope_refusals(args, kw, code):
    with pytest.raises(fd.FdError) as e:
        fd.plan_rope(*args, **kw)
    assert e.value.code == code


def _append(name="fd_append_paged", **kw):
    a = dict(batch=1, n=1, hq=8, hkv=8, d=128, page=16, pages=4, rope=None, q=P(256), qs=1024, k=P(256),
             ks=1024, v=P(256), vs=1024, ip=P(256), pip=P(256), last=P(256), ids=P(256), entries=1,
             pos=None, qo=P(256), qos=1024, kp=P(256), vp=P(256), ws=P(256), wsb=256)
    a.update(kw)
    scales = [kw.get("sk", P(256)), kw.get("sv", P(256))] if name != "fd_append_paged" else []
    order = ["batch", "n", "hq", "hkv", "d", "page", "pages", "rope", "q", "qs", "k", "ks", "v", "vs", "ip",
             "pip", "last", "ids", "entries", "pos", "qo", "qos", "kp", "vp"]
    return getattr(fd.lib(), name)(*[a[x] for x in order], *scales, a["ws"], a["wsb"], None)


@pytest.mark.parametrize("name", ["fd_append_paged", "fd_append_paged_fp8", "fd_append_paged_int4"])
@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), -1), (dict(n=-1), -1), (dict(hkv=0), -1), (dict(hq=-1), -1), (dict(entries=-1), -1),
    (dict(d=64), -2), (dict(page=8), -2), (dict(page=0), -2), (dict(pages=0), -1),
    (dict(pages=1 << 28), -1), (dict(ws=None), -3), (dict(wsb=255), -3), (dict(q=None), -1),
    (dict(qo=None), -1), (dict(k=None), -1), (dict(vp=None), -1), (dict(ip=None), -1), (dict(ids=None), -1),
    (dict(k=P(264)), -1), (dict(kp=P(264)), -1), (dict(pos=P(258)), -1), (dict(qs=1023), -1),
    (dict(ks=1016), -1), (dict(vs=1028), -1), (dict(qos=512), -1), (dict(ws=P(264)), -1),
    (dict(batch=0), 0), (dict(n=0), 0),
], ids=str)
def test_append_refusals(name, kw, code):
    assert _append(name, **kw) == code


@pytest.mark.parametrize("name", ["fd_append_paged", "fd_append_paged_fp8", "fd_append_paged_int4"])
@pytest.mark.parametrize("n,at,stride", [
    # q, k, v of 8, 4 and 4 heads at values 0, 1024 and 1536 of rows of 2176
    (5, 0, 1024), (5, 8, 2176), (5, 512, 2176), (5, 1024, 2176), (5, 1600, 2176), (5, 2040, 2176), (5, 2176, 2176),
    (5, 4 * 2176 + 2040, 2176), (1, -1016, 2176), (5, -1024, 1024),
], ids=str)
def test_append_refuses_queries_written_over_inputs(name, n, at, stride):
    base, pool = 1 << 20, P(1 << 30)
    inputs = dict(n=n, hq=8, hkv=4, q=P(base), qs=2176, k=P(base + 2 * 1024), ks=2176, v=P(base + 2 * 1536), vs=2176)
    assert _append(name, **inputs, qo=P(base + 2 * at), qos=stride, kp=pool, vp=pool) == -1


def test_append_refuses_missing_scales():
    for name in ("fd_append_paged_fp8", "fd_append_paged_int4"):
        assert _append(name, sk=None) == -1
        assert _append(name, sv=P(258)) == -1


def test_append_refuses_a_bad_rope():
    info = fd.plan_rope(128, 64)
    info.rotary_dim = 136
    assert _append(rope=ctypes.addressof(info)) == -1


def _fork(**kw):
    a = dict(old=1, new=1, page=16, pages=4, parent=P(256), ip=P(256), last=P(256), ids=P(512), e=1,
             nip=P(256), ne=1, refs=P(256), nids=P(1024), nrefs=P(256), src=P(256), dst=P(256), ws=P(256),
             wsb=1 << 20)
    a.update(kw)
    return fd.lib().fd_fork_pages(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(old=-1), -1), (dict(new=-1), -1), (dict(page=0), -1), (dict(pages=0), -1), (dict(e=-1), -1),
    (dict(ne=-1), -1), (dict(old=32769), -2), (dict(new=32769, wsb=1 << 30), -2), (dict(ws=None), -3),
    (dict(wsb=512), -3), (dict(refs=None), -1), (dict(nrefs=None), -1), (dict(parent=None), -1),
    (dict(ip=None), -1), (dict(src=None), -1), (dict(nids=P(512)), -1), (dict(last=P(257)), -1),
    (dict(e=4, nids=P(524)), -1), (dict(ne=4, nids=P(500)), -1), (dict(nrefs=P(260)), -1),
], ids=str)
def test_fork_refusals(kw, code):
    assert _fork(**kw) == code


def _compact(**kw):
    a = dict(pages=4, refs=P(256), ids=P(256), e=1, limit=0, moves=2, nids=P(256), nrefs=P(256), src=P(256),
             dst=P(256), ws=P(256), wsb=1 << 20)
    a.update(kw)
    return fd.lib().fd_compact_pages(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(pages=0), -1), (dict(e=-1), -1), (dict(limit=-1), -1), (dict(moves=-1), -1), (dict(ws=None), -3),
    (dict(wsb=1000), -3), (dict(refs=None), -1), (dict(ids=None), -1), (dict(src=None), -1),
    (dict(dst=P(255)), -1), (dict(e=4, nids=P(264)), -1), (dict(nrefs=P(268)), -1),
], ids=str)
def test_compact_refusals(kw, code):
    assert _compact(**kw) == code


def _copy(**kw):
    a = dict(n=1, pools=(P * 1)(256), size=(ctypes.c_int64 * 1)(64), pages=4, copies=1, src=P(256),
             dst=P(256), ws=None, wsb=0)
    a.update(kw)
    return fd.lib().fd_copy_pages(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), -1), (dict(pages=-1), -1), (dict(copies=-1), -1), (dict(pools=None), -1),
    (dict(pools=(P * 1)(264)), -1), (dict(size=(ctypes.c_int64 * 1)(24)), -1),
    (dict(size=(ctypes.c_int64 * 1)(0)), -1), (dict(src=None), -1), (dict(ws=P(256), wsb=8), -3),
    (dict(copies=0), 0), (dict(n=0), 0),
], ids=lambda k: ",".join(k) if isinstance(k, dict) else str(k))
def test_copy_refusals(kw, code):
    assert _copy(**kw) == code


@pytest.mark.parametrize("size,copies", [(1 << 40, 64), ((1 << 63) - 16, 1), (1 << 62, 1 << 20)])
@pytest.mark.parametrize("at", [0, 127, 128, 299])
def test_copies_too_many_for_a_launch_are_refused_before_the_first(size, copies, at):
    """More segments than a grid has, in any of the pools: no pool is copied (which
    would fail here, without a GPU, in another way)."""
    sizes = [64] * 300
    sizes[at] = size
    assert _copy(n=300, pools=(P * 300)(*[256] * 300), size=(ctypes.c_int64 * 300)(*sizes), copies=copies) == -1


def test_pages_workspace_grows_with_pages_and_children():
    a, b, c = fd.pages_workspace_bytes(1000), fd.pages_workspace_bytes(100000), fd.pages_workspace_bytes(1000, 500)
    assert 256 + 4000 < a < c < b
    with pytest.raises(fd.FdError):
        fd.pages_workspace_bytes(-1)


@pytest.mark.parametrize("pages", [2 ** 27, 2 ** 31 - 1024, 2 ** 31 - 1])
def test_more_pages_than_a_cache_has_are_refused(pages):
    with pytest.raises(fd.FdError) as e:
        fd.pages_workspace_bytes(pages)
    assert e.value.code == -1
    assert _fork(pages=pages, wsb=1 << 40) == -1
    assert _compact(pages=pages, wsb=1 << 40) == -1
    assert fd.pages_workspace_bytes(2 ** 27 - 1) > 4 * (2 ** 27 - 1)


def test_new_status_has_a_name():
    assert fd.status_string(-7) == "FD_ERR_NO_PAGES" == fd.STATUS_NAMES[-7]


def test_bindings_refuse_cpu_tensors():
    import torch
    z = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    pool = torch.zeros((1, 16, 8, 128), dtype=torch.bfloat16)
    with pytest.raises((fd.FdError, RuntimeError, AssertionError)):
        fd.append_paged(x, x, x, pool, pool, z[:2], z[:2], z[:1], z[:1], workspace=z)
    with pytest.raises(fd.FdError):
        fd.copy_pages([pool], z[:1], z[:1])


@pytest.mark.parametrize("name", ["append_kernel.cu", "pages_kernel.cu", "shared_kernel.cuh", "split_kernel.cuh"])
def test_no_load_past_the_coherent_path(name):
    """Every kernel of these files starts while the grid before it may still write
    its inputs, so none may read them by loads for constant memory."""
    source = open(os.path.join(os.path.dirname(fd.__file__), "csrc", name)).read()
    code = "\n".join(line.split("//")[0] for line in source.splitlines())
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in code, word
