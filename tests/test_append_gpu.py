"""fd_append_paged, _fp8 and _int4 on the GPU against the rotation and the
quantisation written out in 64 bits.

Tolerances, per value: half a step of the stored type (bf16 2^-8 of the value,
E4M3 2^-4 of it or 2^-10 below its smallest normal, INT4 half a code), plus the
fp32 arithmetic: the angle is rounded to 2^-25 half turns and cos, sin to 2 units
in the last place, under 4e-7 of |a| + |b| in all, and the two sides' 64-bit
frequencies differ by under 64 roundings of 2^-53, which 2^24 positions make an
angle of 1.2e-7; taken as 2^-20 in all."""
import numpy as np
import pytest
import torch

import oracle
import split_kv_flashdecoding_gb300 as fd
from tests.test_cache_cpu import frequencies

pytestmark = pytest.mark.gpu
D = 128
FP32 = 2.0 ** -20


def make(cached, new, hq, hkv, page, seed=0, pad=0, entries_pad=2):
    """Inputs of one call: fused projections, tables that count the new keys in."""
    rng = np.random.RandomState(seed)
    cached, new = np.array(cached), np.array(new)
    have = cached + new
    pages_of = -(-have // page)
    n, num_pages = int(new.sum()), int(pages_of.sum()) + 3
    ids = rng.permutation(num_pages)[: num_pages - 3]
    indptr = lambda c: np.concatenate([[0], np.cumsum(c)]).astype(np.int32)  # noqa: E731
    i = dict(n=n, page=page, hq=hq, hkv=hkv, num_pages=num_pages, append_indptr=indptr(new),
             page_indptr=indptr(pages_of), last=np.where(have > 0, have - (pages_of - 1) * page, 0).astype(np.int32),
             ids=np.concatenate([ids, np.full(entries_pad, -7)]).astype(np.int32))
    i["qkv"] = rng.standard_normal((n + pad, (hq + 2 * hkv) * D)).astype(np.float32)
    rows, key = [], []
    for b in range(len(new)):
        k = cached[b] + np.arange(new[b])
        key.append(k)
        rows.append(ids[i["page_indptr"][b] + k // page] * page + k % page)
    i["rows"] = np.concatenate(rows + [np.zeros(0, int)]).astype(np.int64)
    i["key"] = np.concatenate(key + [np.zeros(0, int)]).astype(np.int64)
    return i


def to_dev(i, dev):
    x = torch.from_numpy(i["qkv"]).to(dev).to(torch.bfloat16).view(-1, i["hq"] + 2 * i["hkv"], D)
    hq, hkv = i["hq"], i["hkv"]
    t = dict(q=x[:, :hq], k=x[:, hq: hq + hkv], v=x[:, hq + hkv:])
    tables = [torch.from_numpy(i[k]).to(dev) for k in ("append_indptr", "page_indptr", "last", "ids")]
    return t, tables


def rotated(x, pos, rotary, inter, base, scaling, gain=1.0):
    """x [n, H, D] fp64 turned as complex pairs; also |a| + |b| of each value's pair."""
    y, mag = x.copy(), np.abs(x)
    turn = gain * np.exp(1j * pos[:, None].astype(np.float64) * frequencies(rotary, base, scaling))[:, None]
    ia, ib = (np.arange(0, rotary, 2), np.arange(1, rotary, 2)) if inter else \
        (np.arange(rotary // 2), np.arange(rotary // 2, rotary))
    z = (x[..., ia] + 1j * x[..., ib]) * turn
    y[..., ia], y[..., ib] = z.real, z.imag
    m = gain * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    mag[..., ia], mag[..., ib] = m, m
    return y, mag


def check_bf16(got, want, mag):
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + FP32 * mag)


def check_fp8(got, want, mag, scale):
    y, m = want / scale[:, None], mag / scale[:, None]
    y = np.clip(y, -448, 448)
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + FP32 * m
    assert np.all(np.abs(got.cpu().view(torch.float8_e4m3fn).double().numpy() - y) <= tol)


def check_int4(codes, scales, want, mag):
    amax = np.abs(want).max(-1)
    ref = np.where(amax > 0, amax / 7, 1.0)
    s = scales.double().cpu().numpy()
    top = mag.max(-1)
    assert np.all(np.abs(s - ref) <= FP32 * top + 2.0 ** -23 * ref)
    vals = oracle.int4_codes(codes.cpu().numpy()) * s[..., None]
    assert np.all(np.abs(vals - want) <= s[..., None] / 2 + FP32 * mag + 2.0 ** -22 * np.abs(want))


ROPES = [(128, False, 10000.0, None), (128, True, 500000.0, ("bands", 8.0, 8192, 1.0, 4.0)),
         (64, False, 10000.0, ("linear", 4.0)), (96, True, 500000.0, ("yarn", 4.0, 32768, 1.0, 32.0)),
         (16, True, 10000.0, None)]
SHAPES = [
    ("step", [5, 0, 31, 16, 100], [1, 1, 1, 1, 1], 32, 8, 16),
    ("prompt", [0, 7, 0], [33, 0, 130], 8, 2, 48),
    ("long", [0, 100], [1500, 700], 4, 1, 64),
    ("one", [0], [1], 1, 1, 16),
    ("mha", [3, 15, 17], [13, 1, 5], 8, 8, 32),
]


@pytest.mark.parametrize("rope", ROPES, ids=lambda r: f"{r[0]}{'i' if r[1] else 'h'}{r[3][0] if r[3] else ''}")
@pytest.mark.parametrize("name,cached,new,hq,hkv,page", SHAPES, ids=[s[0] for s in SHAPES])
@pytest.mark.parametrize("kv", ["bf16", "fp8", "int4"])
def test_append_matches_64_bits(cuda_device, kv, name, cached, new, hq, hkv, page, rope):
    rotary, inter, base, scaling = rope
    pad = 2
    i = make(cached, new, hq, hkv, page, seed=len(name) + rotary, pad=pad)
    t, tables = to_dev(i, cuda_device)
    rng = np.random.RandomState(3)
    # far positions for some: the angle keeps its fraction
    pos = rng.randint(0, 1 << 17, i["n"]).astype(np.int32)
    pos[::7] = 2 ** 24 - 1 - np.arange(len(pos[::7]))
    use_pos = rotary != 128 or inter
    info = fd.plan_rope(D, rotary, interleaved=inter, base=base, scaling=scaling)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    q_out = torch.full((i["n"] + pad, hq, D), 3.0, dtype=torch.bfloat16, device=cuda_device)
    kw = dict(rope=info, q_out=q_out, workspace=ws,
              positions=torch.from_numpy(np.concatenate([pos, [0] * pad]).astype(np.int32)).to(cuda_device)
              if use_pos else None)
    rows, N = i["rows"], i["num_pages"] * page
    scale = torch.rand(2, hkv, device=cuda_device) * 0.02 + 0.004
    if kv == "bf16":
        pools = [torch.full((i["num_pages"], page, hkv, D), 9.0, dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]
        fd.append_paged(t["q"], t["k"], t["v"], *pools, *tables, **kw)
    elif kv == "fp8":
        pools = [torch.full((i["num_pages"], page, hkv, D), 77, dtype=torch.uint8, device=cuda_device) for _ in "kv"]
        fd.append_paged_fp8(t["q"], t["k"], t["v"], *pools, scale[0], scale[1], *tables, **kw)
    else:
        pools = [torch.full((i["num_pages"], page, hkv, D // 2), 77, dtype=torch.uint8, device=cuda_device) for _ in "kv"]
        sc = [torch.full((hkv, N), -5.0, device=cuda_device) for _ in "kv"]
        fd.append_paged_int4(t["q"], t["k"], t["v"], *pools, *sc, *tables, **kw)
    torch.cuda.synchronize()
    assert fd.get_device_status(ws) == 0
    p = pos if use_pos else i["key"]
    x = {n: t[n][: i["n"]].double().cpu().numpy() for n in "qkv"}
    want_q, mag_q = rotated(x["q"], p, rotary, inter, base, scaling, info.gain)
    check_bf16(q_out[: i["n"]], want_q, mag_q)
    assert torch.all(q_out[i["n"]:] == 3.0)   # rows behind the last request
    want_k, mag_k = rotated(x["k"], p, rotary, inter, base, scaling, info.gain)
    for pool, j, want, mag in ((pools[0], 0, want_k, mag_k), (pools[1], 1, x["v"], np.abs(x["v"]))):
        flat = pool.view(N, hkv, -1)
        if kv == "bf16":
            check_bf16(flat[rows], want, mag)
        elif kv == "fp8":
            check_fp8(flat[rows], want, mag, scale[j].double().cpu().numpy())
        else:
            check_int4(flat[rows], sc[j][:, rows].T, want, mag)
        rest = np.setdiff1d(np.arange(N), rows)   # every other row is as it was
        assert torch.all(flat[rest] == (9.0 if kv == "bf16" else 77))
        if kv == "int4":
            assert torch.all(sc[j][:, rest] == -5.0)


def test_v_is_copied_and_no_rope_copies_all(cuda_device):
    i = make([3], [40], 2, 2, 16)
    t, tables = to_dev(i, cuda_device)
    pools = [torch.zeros((i["num_pages"], 16, 2, D), dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]
    q = fd.append_paged(t["q"], t["k"], t["v"], *pools, *tables)
    torch.cuda.synchronize()
    assert torch.equal(q, t["q"])
    for pool, x in zip(pools, (t["k"], t["v"])):
        assert torch.equal(pool.view(-1, 2, D)[i["rows"]], x)


def test_in_place_queries_no_queries_and_strides(cuda_device):
    i = make([0, 9], [20, 3], 4, 2, 16)
    t, tables = to_dev(i, cuda_device)
    info = fd.plan_rope(D, 128)
    new_pools = lambda: [torch.zeros((i["num_pages"], 16, 2, D), dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]  # noqa: E731
    a, b, c = new_pools(), new_pools(), new_pools()
    want = fd.append_paged(t["q"], t["k"], t["v"], *a, *tables, rope=info)
    qc, kc, vc = (t[n].contiguous() for n in "qkv")
    got = fd.append_paged(qc, kc, vc, *b, *tables, rope=info)
    assert torch.equal(want, got) and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert fd.append_paged(None, kc, vc, *c, *tables, rope=info) is None
    assert torch.equal(a[0], c[0]) and torch.equal(a[1], c[1])
    fd.append_paged(t["q"], t["k"], t["v"], *c, *tables, rope=info, q_out=t["q"])   # inside the fused buffer
    torch.cuda.synchronize()
    assert torch.equal(t["q"], want)


@pytest.mark.parametrize("at", [0, 1, 2])
def test_queries_between_the_rows_of_the_inputs(cuda_device, at):
    """q_out as further heads of the fused buffer that q, k and v lie in: in front
    of them, behind them, and over the queries of one token."""
    i = make([0, 9], [20, 3], 4, 2, 16)
    t, tables = to_dev(i, cuda_device)
    info = fd.plan_rope(D, 128)
    pools = [torch.zeros((i["num_pages"], 16, 2, D), dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]
    want = fd.append_paged(t["q"], t["k"], t["v"], *pools, *tables, rope=info)
    if at < 2:
        buf = torch.zeros((i["n"], 12, D), dtype=torch.bfloat16, device=cuda_device)
        x = buf[:, 4:] if at == 0 else buf[:, :8]
        x[:, :4], x[:, 4:6], x[:, 6:] = t["q"], t["k"], t["v"]
        q_out = buf[:, :4] if at == 0 else buf[:, 8:]
        got = fd.append_paged(x[:, :4], x[:, 4:6], x[:, 6:], *pools, *tables, rope=info, q_out=q_out)
    else:
        tables[0] = torch.tensor([0, 0, 1], dtype=torch.int32, device=cuda_device)   # the last key of request 1
        q, k, v = (t[n][-1:].contiguous() for n in "qkv")
        got = fd.append_paged(q, k, v, *pools, *tables, rope=info, q_out=q)
        want = want[-1:]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_tokens_outside_the_tables_are_skipped_and_flagged(cuda_device):
    i = make([0, 5], [4, 4], 2, 2, 16)
    t, tables = to_dev(i, cuda_device)
    for j, bad in ((1, [0, 2, 2]), (2, [4, 17]), (2, [3, 9]), (3, [i["num_pages"], 1]), (3, [-1, 1])):
        tabs = [x.clone() for x in tables]
        tabs[j][: len(bad)] = torch.tensor(bad, dtype=torch.int32)
        pools = [torch.zeros((i["num_pages"], 16, 2, D), dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]
        ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
        fd.append_paged(t["q"], t["k"], t["v"], *pools, *tabs, workspace=ws)
        assert fd.get_device_status(ws) == -6, (j, bad)
        assert fd.get_device_status(ws) == 0   # cleared


@pytest.mark.parametrize("torn", [[0, 9, 1, 2], [0, 9, 1, 9], [5, 4, 8, 9], [-3, -2, -1, 0], [0, 4, 2 ** 31 - 1, 9]])
def test_torn_append_lists_write_no_row_twice(cuda_device, torn):
    """Lists that do not rise: a token whose request does not hold it is skipped
    or flagged; every row written is one of a new key."""
    i = make([0, 5, 2], [4, 4, 1], 2, 2, 16)
    t, tables = to_dev(i, cuda_device)
    tables[0] = torch.tensor(torn, dtype=torch.int32, device=cuda_device)
    pools = [torch.zeros((i["num_pages"], 16, 2, D), dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    fd.append_paged(t["q"], t["k"], t["v"], *pools, *tables, workspace=ws)
    assert fd.get_device_status(ws) == (0 if torn[-1] == 0 else -6)
    pages = {int(x) for x in i["ids"] if x >= 0}
    written = pools[0].view(i["num_pages"], -1).ne(0).any(1).nonzero().flatten().tolist()
    assert set(written) <= pages


def test_quantised_rows_of_zeros_infinities_and_nan(cuda_device):
    i = make([0], [4], 1, 1, 16)
    t, tables = to_dev(i, cuda_device)
    k, v = t["k"].contiguous(), t["v"].contiguous()
    v[0] = 0
    v[1, 0, 5] = float("nan")
    v[2, 0, 7] = float("inf")
    one = torch.ones(1, device=cuda_device)
    p8 = [torch.zeros((i["num_pages"], 16, 1, D), dtype=torch.uint8, device=cuda_device) for _ in "kv"]
    fd.append_paged_fp8(None, k, v, *p8, one, one, *tables)
    f = p8[1].view(torch.float8_e4m3fn).float().view(-1, D)[i["rows"]]
    assert torch.all(f[0] == 0) and torch.isnan(f[1, 5]) and f[2, 7] == 448 and torch.isfinite(f[2]).all()
    p4 = [torch.zeros((i["num_pages"], 16, 1, D // 2), dtype=torch.uint8, device=cuda_device) for _ in "kv"]
    sc = [torch.zeros((1, i["num_pages"] * 16), device=cuda_device) for _ in "kv"]
    fd.append_paged_int4(None, k, v, *p4, *sc, *tables)
    s = sc[1][0, i["rows"]]
    assert s[0] == 1 and torch.isnan(s[1]) and torch.isinf(s[2])
    assert torch.all(p4[1].view(-1, D // 2)[i["rows"][0]] == 0)


@pytest.mark.parametrize("scales", [(0.03, 0.3, 0.02, 1 / 3, 0.7, 7.0, 0.0123, 3 / 448),
                                    (1e-39, 1e-40, 2e-38, 1.0, 3e38, 2.0 ** -126, -0.03, 448.0)], ids=["usual", "far"])
def test_fp8_codes_of_every_value_are_the_rounded_quotients(cuda_device, scales):
    """Every finite bf16 value over each scale: E4M3 of the quotient, ties to even.
    Both roundings are IEEE's, so the codes are equal."""
    x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x)].view(-1, 1, D).expand(-1, 8, D).contiguous()
    n, page = len(x), 16
    scale = torch.tensor(scales)
    pages = -(-n // page)
    pools = [torch.zeros((pages, page, 8, D), dtype=torch.uint8, device=cuda_device) for _ in "kv"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    v = x.to(cuda_device)
    fd.append_paged_fp8(None, v, v, *pools, scale.to(cuda_device), scale.to(cuda_device), i32([0, n]), i32([0, pages]),
                        i32([n - (pages - 1) * page]), torch.arange(pages, dtype=torch.int32, device=cuda_device))
    want = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for pool in pools:   # K without a rotation is stored as V is
        assert torch.equal(pool.view(-1, 8, D)[:n].cpu(), want)


def test_captured_append_follows_its_tables(cuda_device):
    """One captured step, replayed with new positions, tables and inputs."""
    i, j = make([5, 40], [1, 1], 4, 2, 16, seed=1), make([21, 2], [1, 1], 4, 2, 16, seed=2)
    t, tables = to_dev(i, cuda_device)
    u, tables2 = to_dev(j, cuda_device)
    n = max(i["num_pages"], j["num_pages"])
    info, ws = fd.plan_rope(D, 128), torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    pools = [torch.zeros((n, 16, 2, D), dtype=torch.bfloat16, device=cuda_device) for _ in "kv"]
    q_out = torch.empty((2, 4, D), dtype=torch.bfloat16, device=cuda_device)
    ids = torch.full((16,), -1, dtype=torch.int32, device=cuda_device)
    tables[3] = ids
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            fd.append_paged(t["q"], t["k"], t["v"], *pools, *tables, rope=info, q_out=q_out, workspace=ws)
    for case, src, tabs in ((i, None, None), (j, u, tables2)):
        if src is not None:
            for a in "qkv":
                t[a].copy_(src[a])
            for a, b in zip(tables[:3], tabs[:3]):
                a.copy_(b)
        ids[: len(case["ids"])].copy_(torch.from_numpy(case["ids"]).to(cuda_device))
        g.replay()
        torch.cuda.synchronize()
        x = t["k"].double().cpu().numpy()
        want, mag = rotated(x, case["key"], 128, False, 10000.0, None)
        check_bf16(pools[0].view(-1, 2, D)[case["rows"]], want, mag)
        assert fd.get_device_status(ws) == 0
