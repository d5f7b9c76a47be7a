"""fd_append_paged_int8 on the GPU against the rotation and the page scales
written out in 64 bits.

Tolerances: fp32 arithmetic on a rotated value leaves 2^-20 of |a| + |b| of its
pair (as for the other appends); a scale is the largest of such values over 127,
two roundings of 2^-24 more; a code is off by half a step of its scale, plus the
rounding of the quotient (2^-22 of the value); a code that is carried over is off
by half a step of the new scale, plus as much of its value."""
import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd
from tests.int8_util import D
from tests.test_append_gpu import FP32, ROPES, check_bf16, make, rotated, to_dev

pytestmark = pytest.mark.gpu
SMALLEST = 2.0 ** -126

SHAPES = [
    ("step", [5, 0, 31, 16, 100], [1, 1, 1, 1, 1], 32, 8, 16),
    ("prompt", [0, 7, 0], [33, 0, 130], 8, 2, 48),
    ("long", [0, 100], [1500, 700], 4, 1, 64),
    ("long_mha", [0, 30], [700, 100], 8, 8, 64),
    ("one", [0], [1], 1, 1, 16),
    ("three_heads", [3, 15, 17], [13, 1, 5], 12, 3, 32),
    ("many_heads", [9, 40], [100, 7], 20, 20, 128),
    ("large_pages", [0, 1000, 5], [2500, 300, 1], 8, 4, 1024),
    ("large_pages_one_head", [600], [700], 1, 1, 1024),
    ("mixed", [5, 0, 31, 100, 62, 7], [1, 300, 3, 70, 4, 5], 32, 8, 64),
    ("few_rows_one_head", [14, 0, 3], [4, 3, 2], 2, 1, 16),
    ("one_head_pages_of_128", [0, 30], [300, 90], 4, 1, 128),
]


def pools(i, rng, dev):
    n, p, hkv = i["num_pages"], i["page"], i["hkv"]
    out = {}
    for x in ("k", "v"):
        out[x] = torch.from_numpy(rng.randint(-127, 128, (n, p, hkv, D)).astype(np.int8)).to(dev)
        s = np.full((n, fd.scale_heads(hkv)), -5.0, dtype=np.float32)
        s[:, :hkv] = rng.random_sample((n, hkv)) * 0.04
        out[x + "s"] = torch.from_numpy(s).to(dev)
    return out


def expected(i, cached, new, codes, scale, y, mag):
    """Values and their tolerance [pages, page, Hkv, D], scales and theirs, after an
    append of y [n, Hkv, D] (fp64)."""
    p, hkv = i["page"], i["hkv"]
    val = codes.astype(np.float64) * scale[:, None, :hkv, None]
    tol = np.zeros_like(val)
    s_out, s_tol = scale.astype(np.float64).copy(), np.zeros(scale.shape)
    for b in range(len(new)):
        done, a = 0, i["append_indptr"][b]
        while done < new[b]:
            key = int(cached[b]) + done
            page, at = i["ids"][i["page_indptr"][b] + key // p], key % p
            take = min(p - at, int(new[b]) - done)
            rows, m = y[a + done: a + done + take], mag[a + done: a + done + take]
            old = scale[page, :hkv].astype(np.float64) if at else np.zeros(hkv)
            now = np.maximum(np.maximum(old, np.abs(rows).max(axis=(0, 2)) / 127), SMALLEST)
            st = FP32 * m.max(axis=(0, 2)) / 127 + 2.0 ** -22 * now
            s_out[page, :hkv], s_tol[page, :hkv] = now, st
            grown = now > old - st
            step = (now + st)[:, None] / 2
            v = val[page, :at]
            tol[page, :at] = np.where(grown[:, None], step + 2.0 ** -21 * np.abs(v), 0.0)
            val[page, at: at + take] = rows
            tol[page, at: at + take] = step + FP32 * m + 2.0 ** -22 * np.abs(rows)
            rest = codes[page, at + take:].astype(np.float64)   # rows behind keep their codes
            val[page, at + take:] = rest * now[:, None]
            tol[page, at + take:] = np.abs(rest) * (st + 2.0 ** -40 * now)[:, None]
            done += take
    return val, tol, s_out, s_tol


def call(t, c, tables, **kw):
    return fd.append_paged_int8(t["q"], t["k"], t["v"], c["k"], c["v"], c["ks"], c["vs"], *tables, **kw)


@pytest.mark.parametrize("rope", ROPES, ids=lambda r: f"{r[0]}{'i' if r[1] else 'h'}{r[3][0] if r[3] else ''}")
@pytest.mark.parametrize("name,cached,new,hq,hkv,page", SHAPES, ids=[s[0] for s in SHAPES])
def test_append_int8_matches_64_bits(cuda_device, name, cached, new, hq, hkv, page, rope):
    rotary, inter, base, scaling = rope
    pad = 2
    i = make(cached, new, hq, hkv, page, seed=len(name) + rotary, pad=pad)
    t, tables = to_dev(i, cuda_device)
    rng = np.random.RandomState(5)
    pos = rng.randint(0, 1 << 17, i["n"]).astype(np.int32)
    c = pools(i, rng, cuda_device)
    before = {x: c[x].cpu().numpy() for x in c}
    info = fd.plan_rope(D, rotary, interleaved=inter, base=base, scaling=scaling)
    ws = torch.zeros(fd.WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=cuda_device)
    q_out = torch.full((i["n"] + pad, hq, D), 9.0, dtype=torch.bfloat16, device=cuda_device)
    positions = torch.from_numpy(np.append(pos, [0] * pad).astype(np.int32)).to(cuda_device)
    call(t, c, tables, rope=info, positions=positions, q_out=q_out, workspace=ws)
    assert fd.get_device_status(ws) == 0
    gain = float(info.gain)
    n = i["n"]
    x = {k: v[:n].double().cpu().numpy() for k, v in t.items()}
    want, mag = rotated(x["q"], pos, rotary, inter, base, scaling, gain)
    check_bf16(q_out[:n], want, mag)
    assert torch.all(q_out[n:] == 9.0)
    for part in ("k", "v"):
        y, mag = rotated(x["k"], pos, rotary, inter, base, scaling, gain) if part == "k" else (x["v"], np.abs(x["v"]))
        val, tol, s, st = expected(i, cached, new, before[part], before[part + "s"], y, mag)
        got_s = c[part + "s"].double().cpu().numpy()
        worst = float(np.max(np.abs(got_s - s) - st))
        assert worst <= 0
        codes = c[part].cpu().numpy().astype(np.float64)
        got = codes * got_s[:, None, :hkv, None]
        worst = float(np.max(np.abs(got - val) - tol))
        assert worst <= 0
        untouched = np.ones(i["num_pages"], bool)
        untouched[np.unique(i["rows"] // page)] = False
        assert np.array_equal(codes[untouched], before[part][untouched])


@pytest.mark.parametrize("log2", [100, 30, -30, -100])
def test_append_int8_values_of_any_size(cuda_device, log2):
    cached, new, hkv, page = [5, 0, 40], [20, 70, 1], 4, 32
    i = make(cached, new, 4, hkv, page, seed=3)
    i["qkv"] *= np.float32(2.0 ** log2)
    t, tables = to_dev(i, cuda_device)
    rng = np.random.RandomState(7)
    c = pools(i, rng, cuda_device)
    before = {x: c[x].cpu().numpy() for x in c}
    info = fd.plan_rope(D, 128)
    call(t, c, tables, rope=info)
    x = {k: v.double().cpu().numpy() for k, v in t.items()}
    for part in ("k", "v"):
        y, mag = rotated(x["k"], i["key"], 128, False, 10000.0, None) if part == "k" else (x["v"], np.abs(x["v"]))
        val, tol, s, st = expected(i, cached, new, before[part], before[part + "s"], y, mag)
        got_s = c[part + "s"].double().cpu().numpy()
        assert np.all(np.abs(got_s - s) <= st)
        got = c[part].cpu().numpy().astype(np.float64) * got_s[:, None, :hkv, None]
        assert np.all(np.abs(got - val) <= tol)


def test_append_int8_without_queries_or_rotation_uses_key_positions(cuda_device):
    i = make([5, 40], [20, 3], 8, 4, 16, seed=2)
    t, tables = to_dev(i, cuda_device)
    rng = np.random.RandomState(1)
    c = pools(i, rng, cuda_device)
    d = {x: c[x].clone() for x in c}
    info = fd.plan_rope(D, 128)
    key = torch.from_numpy(i["key"].astype(np.int32)).to(cuda_device)
    call(t, c, tables, rope=info)
    fd.append_paged_int8(None, t["k"], t["v"], d["k"], d["v"], d["ks"], d["vs"], *tables, rope=info, positions=key)
    assert all(torch.equal(c[x], d[x]) for x in c)


def test_append_int8_token_by_token_is_within_a_step_a_growth(cuda_device):
    """128 keys one at a time, in pages of 64 whose scales grow: each value off by at
    most half a final step for each time that its page's scale grew behind it."""
    rng = np.random.RandomState(4)
    hkv, page, n = 4, 64, 128
    x = torch.from_numpy((rng.standard_normal((n, 3 * hkv, D)) * np.linspace(0.2, 3, n)[:, None, None])
                         .astype(np.float32)).to(cuda_device).to(torch.bfloat16)
    c = dict(k=torch.zeros((2, page, hkv, D), dtype=torch.int8, device=cuda_device), ks=torch.full((2, 4), 77.0, device=cuda_device))
    c.update(v=c["k"].clone(), vs=c["ks"].clone())
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    ids = i32(1, 0)
    growths = torch.zeros((2, n, hkv), device=cuda_device)   # behind each key
    for j in range(n):
        row = x[j: j + 1]
        old = torch.stack([c["ks"], c["vs"]]).clone()
        fd.append_paged_int8(row[:, :hkv], row[:, hkv: 2 * hkv], row[:, 2 * hkv:], c["k"], c["v"], c["ks"], c["vs"],
                             i32(0, 1), i32(0, j // page + 1), i32(j % page + 1), ids)
        if j % page:
            g = torch.stack([c["ks"], c["vs"]])[:, int(ids[j // page])] > old[:, int(ids[j // page])]
            growths[:, j // page * page: j] += g[:, None].float()
    for which, (codes, scale) in enumerate(((c["k"], c["ks"]), (c["v"], c["vs"]))):
        s = scale[ids.long()][:, None].expand(2, page, 4).reshape(n, hkv)
        got = codes[ids.long()].reshape(n, hkv, D).double() * s[..., None].double()
        want = x[:, (1 + which) * hkv: (2 + which) * hkv].double()
        # a rounding to codes is off by half a step, and rounds a quotient that fp32 has to
        # two roundings of 2^-24 (so a half-way point may go either way): 2^-22 of the value
        times = (growths[which] + 1)[..., None].double()
        tol = times * (s[..., None].double() / 2 + 2.0 ** -22 * (want.abs() + got.abs()))
        worst = float(((got - want).abs() - tol).max())
        assert worst <= 0
        top = want.view(2, page, hkv, D).abs().amax(dim=(1, 3)) / 127
        assert torch.allclose(scale[ids.long()].double(), top, rtol=2.0 ** -22, atol=0)
    assert growths.max() > 5


def test_append_int8_zeros_infinities_and_nan(cuda_device):
    i = make([0, 0, 0, 8], [16, 16, 16, 1], 4, 2, 16, seed=3)
    t, tables = to_dev(i, cuda_device)
    c = pools(i, np.random.RandomState(0), cuda_device)
    v = t["v"]
    v[:16, 0] = 0
    v[20, 0, 7] = float("nan")
    v[40, 0, 9] = float("inf")
    v[48, 0, 1] = float("-inf")
    call(t, c, tables)
    page = [int(i["ids"][i["page_indptr"][b]]) for b in range(4)]
    s = c["vs"][page, 0]
    assert float(s[0]) == SMALLEST and torch.isnan(s[1]) and torch.isinf(s[2]) and torch.isinf(s[3])
    assert torch.all(c["v"][page[0], :, 0] == 0) and torch.all(c["v"][page[1], :, 0] == 0)
    assert torch.all(c["v"][page[2], :, 0] == 0) and torch.all(c["v"][page[3], :9, 0] == 0)
    assert torch.isfinite(c["vs"][page, 1]).all() and torch.isfinite(c["ks"][page, :2]).all()
    # keys behind zeros take a scale of their own, and the zeros stay zeros
    j = make([3], [2], 4, 2, 16, seed=9)
    u, tab = to_dev(j, cuda_device)
    d = pools(j, np.random.RandomState(0), cuda_device)
    pg = int(j["ids"][0])
    d["v"][pg] = 0
    d["vs"][pg] = SMALLEST
    call(u, d, tab)
    assert torch.all(d["v"][pg, :3] == 0)
    want = u["v"].double()
    got = d["v"][pg, 3:5].double() * d["vs"][pg, :2].double()[None, :, None]
    assert bool(((got - want).abs() <= d["vs"][pg, :2].double()[None, :, None] * (0.5 + 2.0 ** -15)).all())


@pytest.mark.parametrize("what", ["page", "page_low", "last", "keys", "entries"])
def test_append_int8_outside_the_tables_is_flagged(cuda_device, what):
    i = make([5, 0, 20], [10, 20, 3], 4, 2, 16, seed=6)
    t, tables = to_dev(i, cuda_device)
    c = pools(i, np.random.RandomState(0), cuda_device)
    ws = torch.zeros(fd.WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=cuda_device)
    good = {x: c[x].clone() for x in c}
    call(t, good, tables)
    _, page_indptr, last, ids = tables
    e = int(i["page_indptr"][1])
    if what == "page":
        ids[e] = i["num_pages"]
    elif what == "page_low":
        ids[e] = -1
    elif what == "last":
        last[1] = 17
    elif what == "entries":
        tables[3] = ids[: len(ids) - 4]   # the third request's table ends behind the list
    else:
        last[1] = 3                        # 19 keys for 20 tokens
    call(t, c, tables, workspace=ws)
    assert fd.get_device_status(ws) == -6 and fd.get_device_status(ws) == 0
    # the other requests' pages are as without the fault
    others = [0] if what == "entries" else [0, 2]
    for b in others:
        for j in range(i["page_indptr"][b], i["page_indptr"][b + 1]):
            pg = int(i["ids"][j])
            assert torch.equal(c["k"][pg], good["k"][pg]) and torch.equal(c["vs"][pg], good["vs"][pg])


def test_append_int8_many_requests_and_graph(cuda_device):
    """700 requests (more than a CTA's threads), captured and replayed: the second
    replay finds the scales grown and changes nothing."""
    rng = np.random.RandomState(11)
    cached, new = rng.randint(0, 40, 700), rng.randint(0, 4, 700)
    i = make(cached, new, 8, 2, 16, seed=1)
    t, tables = to_dev(i, cuda_device)
    c = pools(i, rng, cuda_device)
    d = {x: c[x].clone() for x in c}
    e = {x: c[x].clone() for x in c}
    call(t, c, tables)
    ws = torch.zeros(fd.WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=cuda_device)
    q_out = torch.empty_like(t["q"].contiguous())
    call(t, e, tables, q_out=q_out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(t, d, tables, q_out=q_out, workspace=ws)
    for _ in range(2):
        g.replay()
        assert all(torch.equal(c[x], d[x]) for x in c)
    rows = i["rows"]
    got = (c["v"].double() * c["vs"][:, None, :2, None].double()).view(-1, 2, D)[rows].cpu().numpy()
    step = c["vs"].double().cpu().numpy()[rows // 16, :2]
    assert np.all(np.abs(got - t["v"].double().cpu().numpy()) <= step[..., None] * (0.5 + 2.0 ** -15))
