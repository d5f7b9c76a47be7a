"""fd_decode_paged_int8 on the GPU against attention in 64 bits over the values
that codes and page scales stand for.

Tolerances: O and LSE are fp32.  A weight enters the product with V in two f16
parts (2^-22 of it), a logit of up to some 30 is rounded a few times in fp32
(2^-24 each, so its weight by 30 * 4 * 2^-24 = 7e-6 at most and as much either
way), and sums of up to 16000 terms are rounded in fp32 in runs of 32: 1e-5 of O
in the 2-norm, 1e-4 of the largest value at a single element, 2e-5 in LSE."""
import zlib

import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd
from tests.int8_util import D, attention, cache, dev_tables, tables
from tests.parity_util import assert_within, errors

pytestmark = pytest.mark.gpu
TIGHT = dict(max_abs=1e-4, rel_l2=1e-5, lse_abs=2e-5)

CASES = [
    ("single_key", 4, 4, [1], 16),
    ("one_short_of_a_tile", 8, 2, [31], 16),
    ("ragged_with_empty", 16, 8, [0, 77, 0, 300, 1], 48),
    ("last_page_16_keys", 32, 8, [16, 32, 48, 4112], 16),
    ("several_tiles_g8", 64, 8, [1000, 1537], 32),
    ("mha_long", 8, 8, [4099], 64),
    ("odd_heads", 12, 3, [700, 65], 16),
    ("one_head_g8", 8, 1, [5, 33, 2049], 48),
    ("multi_wave_g8", 64, 8, [16000, 16000, 3000], 16),
    ("multi_wave_g4", 32, 8, [16000, 16000, 3000], 32),
    ("multi_wave_g2", 16, 8, [16000, 16001, 2999], 48),
    ("multi_wave_g1", 8, 8, [16001, 15999, 3000], 128),
]


def make(name, hq, hkv, lengths, page, kind, dev):
    rng = np.random.RandomState(zlib.crc32(name.encode()) % 1000)
    t = tables(lengths, page, rng)
    c = cache(t, hkv, rng, dev, kind)
    q = torch.from_numpy(rng.standard_normal((len(lengths), hq, D)).astype(np.float32)).to(dev).to(torch.bfloat16)
    return t, c, q


def run(t, c, q, scale=D ** -0.5, **kw):
    return fd.decode_paged_int8(q, c["k"], c["v"], c["ks"], c["vs"], t["ip"], t["last"], *dev_tables(t, q.device),
                                scale, **kw)


def compare(got, want, what):
    o, lse = got
    err = errors(o.cpu().numpy(), lse.cpu().numpy(), want[0].cpu().numpy(), want[1].cpu().numpy())
    assert_within(err, **TIGHT, what=what)


@pytest.mark.parametrize("kind", ["quantised", "random"])
@pytest.mark.parametrize("name,hq,hkv,lengths,page", CASES, ids=[c[0] for c in CASES])
def test_int8_decode_matches_64_bits(cuda_device, name, hq, hkv, lengths, page, kind):
    t, c, q = make(name, hq, hkv, lengths, page, kind, cuda_device)
    need = fd.plan_paged(len(lengths), hq, hkv, D, page, t["ip"], t["last"]).workspace_bytes
    ws = torch.zeros(need, dtype=torch.uint8, device=cuda_device)
    for _ in range(2):   # the second call finds the tickets and counters as the first left them
        got = run(t, c, q, workspace=ws)
        assert fd.get_device_status(ws) == 0
    compare(got, attention(q, t, c, D ** -0.5), f"{name} {kind}")


@pytest.mark.parametrize("hq", [4, 32])
def test_int8_scales_of_far_apart_pages(cuda_device, hq):
    """V scales that grow and fall by 2^30 from page to page, pages of zeros under
    the smallest scale, K scales of zero: weights and O keep their accuracy."""
    t, c, q = make("far", hq, 4, [500, 90], 16, "quantised", cuda_device)
    e = torch.from_numpy(np.random.RandomState(3).randint(-60, 60, (t["num_pages"], 4))).to(cuda_device)
    c["vs"] *= torch.exp2(e.float())
    c["ks"][::5] = 0
    c["v"][::3] = 0
    c["vs"][::3] = 2.0 ** -126
    o, lse = run(t, c, q)
    o_ref, lse_ref = attention(q, t, c, D ** -0.5)
    err = (o.double() - o_ref).norm(dim=-1) / o_ref.norm(dim=-1)
    assert float(err.max()) <= 1e-5   # of each row: its largest scale rules it
    assert float((lse.double() - lse_ref).abs().max()) <= 2e-5


def test_int8_rows_behind_the_last_key_and_foreign_pages_do_not_matter(cuda_device):
    t, c, q = make("leak", 16, 4, [45, 70, 16], 48, "random", cuda_device)
    want = run(t, c, q)
    mine = torch.zeros(t["num_pages"], 48, dtype=torch.bool, device=cuda_device)
    for b in range(3):
        for j in range(t["ip"][b], t["ip"][b + 1]):
            mine[t["ids"][j], : t["last"][b] if j == t["ip"][b + 1] - 1 else 48] = True
    for x in ("k", "v"):
        c[x][~mine] = -128
        c[x + "s"][~mine.any(1)] = float("nan")
    c["ks"][:, 4:] = c["vs"][:, 4:] = float("nan")
    got = run(t, c, q)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("hq", [4, 32])
def test_int8_scales_that_are_no_numbers_reach_their_request_alone(cuda_device, which, value, hq):
    t, c, q = make("nan", hq, 4, [300, 200], 16, "random", cuda_device)
    want = run(t, c, q)
    page = int(t["ids"][t["ip"][1] + 2])
    c[which][page, 1] = value
    o, lse = run(t, c, q)
    g = hq // 4
    assert torch.equal(o[0], want[0][0]) and torch.equal(lse[0], want[1][0])
    assert torch.equal(o[1, :g], want[0][1, :g]) and torch.equal(o[1, 2 * g:], want[0][1, 2 * g:])
    assert not torch.isfinite(o[1, g: 2 * g]).any()


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("hq", [1, 8])
def test_int8_no_number_is_nan_whatever_the_codes(cuda_device, which, value, sign, hq):
    # scores of one sign, an infinite scale of either: not a weight of 0, nor an infinity
    t, c, _ = make("all", hq, 1, [300, 1], 16, "quantised", cuda_device)
    c["k"].fill_(3 * sign)
    c["v"].fill_(5)
    q = torch.ones((2, hq, D), dtype=torch.bfloat16, device=cuda_device)
    for b, page in ((0, 7), (1, 0)):
        c[which][int(t["ids"][t["ip"][b] + page]), 0] = value
    o, lse = run(t, c, q)
    assert bool(o.isnan().all()) and (which == "vs" or bool(lse.isnan().all()))


@pytest.mark.parametrize("log2", [118, 60, -60, -105])
@pytest.mark.parametrize("hq", [4, 32])
def test_int8_queries_of_any_size(cuda_device, hq, log2):
    # bf16 reaches beyond f16 on both sides; the factor of the scores brings these back
    t, c, q = make("sizes", hq, 4, [300, 20], 32, "quantised", cuda_device)
    big = (q.double() * 2.0 ** log2).to(torch.bfloat16)
    assert torch.equal(big.double(), q.double() * 2.0 ** log2)
    got = run(t, c, big, scale=D ** -0.5 * 2.0 ** -log2)
    compare(got, attention(q, t, c, D ** -0.5), str(log2))


def test_int8_pages_outside_the_pool_are_flagged(cuda_device):
    t, c, q = make("bad", 8, 8, [100], 16, "random", cuda_device)
    need = fd.plan_paged(1, 8, 8, D, 16, t["ip"], t["last"]).workspace_bytes
    for bad in (-1, t["num_pages"], 1 << 30):
        ws = torch.zeros(need, dtype=torch.uint8, device=cuda_device)
        u = dict(t, ids=t["ids"].copy())
        u["ids"][3] = bad
        run(u, c, q, workspace=ws)
        assert fd.get_device_status(ws) == -6
        assert fd.get_device_status(ws) == 0


def test_int8_far_rows_of_a_large_pool(cuda_device):
    """Rows past 2^32 bytes of the pool and page rows past 2^24."""
    page, hkv, pages = 16, 8, 300000   # 4.9e9 bytes a pool, 4.8e6 rows
    dev = cuda_device
    rng = np.random.RandomState(8)
    t = tables([700, 33], page, rng)
    small = cache(t, hkv, rng, dev)
    at = torch.from_numpy(np.sort(rng.choice(pages - 1000, t["num_pages"], replace=False)) + 1000).to(dev)
    c = {}
    for x in ("k", "v"):
        c[x] = torch.full((pages, page, hkv, D), 77, dtype=torch.int8, device=dev)
        c[x][at] = small[x]
        c[x + "s"] = torch.full((pages, hkv), 3.0, device=dev)
        c[x + "s"][at] = small[x + "s"]
    u = dict(t, ids=at.cpu().numpy()[t["ids"]].astype(np.int32), num_pages=pages)
    q = torch.randn((2, 32, D), device=dev).to(torch.bfloat16)
    compare(run(u, c, q), attention(q, t, small, D ** -0.5), "far rows")


def test_int8_streams_and_graphs(cuda_device):
    """A call on another stream, and one captured and replayed with other queries."""
    t, c, q = make("graph", 32, 8, [3000, 100], 32, "quantised", cuda_device)
    want = run(t, c, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(t, c, q, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0])
    need = fd.plan_paged(2, 32, 8, D, 32, t["ip"], t["last"]).workspace_bytes
    ws = torch.zeros(need, dtype=torch.uint8, device=cuda_device)
    o, lse, tab = torch.empty_like(want[0]), torch.empty_like(want[1]), dev_tables(t, cuda_device)
    qs = q.clone()

    def call():
        fd.decode_paged_int8(qs, c["k"], c["v"], c["ks"], c["vs"], t["ip"], t["last"], *tab, D ** -0.5, o=o, lse=lse,
                             workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(3):
        qs.copy_(q * (k + 1) / 2)
        g.replay()
        compare((o, lse), attention(qs, t, c, D ** -0.5), f"replay {k}")
