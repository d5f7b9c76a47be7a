"""fd_prefill_paged_int8 on the GPU against attention in 64 bits over the values
that codes and page scales stand for.

Tolerances, per value of O: half a step of bf16 (2^-8 of it), and for the softmax
weights w_j, each rounded to f16 once (2^-11 of it at most; one below 2^-15 of the
row's reference by 2^-26 of that at most, where the row's sum is at least the
reference: 2^-19 covers 128 such keys' errors of one sign) and off by up to 2e-5 through the rounding of their fp32 logits (30 * 4 * 2^-24, twice):
(2^-11 + 2^-15) A + 2^-19 max|v| with A = sum_j w_j |v_j|.  LSE is fp32: 2e-5, as for
single tokens, where a row's logits are below 30 or so."""
import math
import zlib

import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd
from tests.int8_util import D, attention, cache, dev_tables, indptr, tables

pytestmark = pytest.mark.gpu
LSE = 2e-5

CASES = [
    # name, Hq, Hkv, tokens, keys (of a causal call: with the tokens' own), page
    ("one_token", 4, 4, [1], [1], 16),
    ("steps", 32, 8, [1, 1, 1, 1], [77, 1, 300, 16], 16),
    ("drafts", 32, 8, [5, 5, 5], [1000, 5, 4000], 16),
    ("prompt", 8, 2, [300], [300], 48),
    ("prompt_g8", 16, 2, [1000], [1000], 64),
    ("prompt_g1", 4, 4, [513], [513], 32),
    ("chunk_behind", 16, 4, [257], [2000], 64),
    ("ragged", 8, 4, [130, 0, 1, 64, 700, 129], [130, 50, 900, 64, 705, 640], 16),
    ("odd_pages", 12, 3, [33, 100], [1111, 100], 80),
    ("large_pages", 8, 8, [200, 3], [1500, 700], 1024),
    ("long", 8, 1, [40], [9001], 128),
]


def make(name, hq, hkv, tokens, keys, page, dev, kind="quantised"):
    rng = np.random.RandomState(zlib.crc32(name.encode()) % 1000)
    t = tables(keys, page, rng)
    c = cache(t, hkv, rng, dev, kind)
    for x in ("ks", "vs"):
        c[x] = c[x].abs()
    q = torch.from_numpy(rng.standard_normal((sum(tokens), hq, D)).astype(np.float32)).to(dev).to(torch.bfloat16)
    return t, c, q, indptr(tokens)


def plan_of(t, q, hkv, qi, causal, **kw):
    return fd.plan_prefill_paged(len(t["keys"]), q.shape[1], hkv, D, t["page"], qi, t["ip"], t["last"], causal=causal, **kw)


def run(t, c, q, qi, causal, scale=D ** -0.5, plan=None, check=True, **kw):
    plan = plan or plan_of(t, q, c["k"].shape[2], qi, causal)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=q.device)
    out = fd.prefill_paged_int8(plan, q, c["k"], c["v"], c["ks"], c["vs"], torch.from_numpy(qi).to(q.device),
                                *dev_tables(t, q.device), scale, workspace=ws, **kw)
    if check:
        assert fd.get_device_status(ws) == 0
    return out


def compare(got, t, c, q, qi, causal, scale=D ** -0.5, what="", lse_abs=LSE):
    o, lse = got
    n = int(qi[-1])
    want, lse_want = attention(q[:n], t, c, scale, qi, causal)
    mags = dict(c, v=c["v"].clamp(min=-127).abs())   # (abs of -128 is not an int8)
    a, _ = attention(q[:n], t, mags, scale, qi, causal)
    a = a.abs()
    big = (mags["v"].amax(dim=(1, 3)).double() * c["vs"][:, : c["v"].shape[2]].double()).amax()
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -15) * a + 2.0 ** -19 * big
    over = float(((o[:n].double() - want).abs() - tol).max()) if n else 0.0
    assert over <= 0, f"{what}: O beyond its tolerance by {over}"
    none = lse_want == -math.inf
    assert torch.equal(lse[:n] == -math.inf, none), what
    assert bool((o[:n][none] == 0).all()), what
    worst = float((lse[:n].double() - lse_want)[~none].abs().max()) if bool((~none).any()) else 0.0
    assert worst <= lse_abs, f"{what}: LSE off by {worst}"


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", ["quantised", "random"])
@pytest.mark.parametrize("name,hq,hkv,tokens,keys,page", CASES, ids=[c[0] for c in CASES])
def test_prefill_matches_64_bits(cuda_device, name, hq, hkv, tokens, keys, page, kind, causal):
    t, c, q, qi = make(name, hq, hkv, tokens, keys, page, cuda_device, kind)
    if kind == "random":   # codes of 74 rms and scales of up to 0.03: smaller logits
        q = q * 0.5
    compare(run(t, c, q, qi, causal), t, c, q, qi, causal, what=f"{name} {kind} {causal}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("chunk", [128, 256, 640])
@pytest.mark.parametrize("name", ["drafts", "chunk_behind", "ragged", "prompt_g8"])
def test_prefill_in_splits(cuda_device, name, chunk, causal):
    """Splits of the keys, with some that a block's rows do not reach."""
    _, hq, hkv, tokens, keys, page = next(c for c in CASES if c[0] == name)
    t, c, q, qi = make(name, hq, hkv, tokens, keys, page, cuda_device)
    plan = plan_of(t, q, hkv, qi, causal, chunk=chunk)
    assert plan.num_merged_rows > 0
    compare(run(t, c, q, qi, causal, plan=plan), t, c, q, qi, causal, what=f"{name} {chunk}")


@pytest.mark.parametrize("chunk", [0, 128])
def test_prefill_rows_without_keys(cuda_device, chunk):
    """Requests without keys, and causal ones of more tokens than keys."""
    t, c, q, qi = make("none", 8, 4, [5, 200, 70, 3], [0, 130, 64, 300], 16, cuda_device)
    for causal in (True, False):
        plan = plan_of(t, q, 4, qi, causal, chunk=chunk)
        got = run(t, c, q, qi, causal, plan=plan)
        compare(got, t, c, q, qi, causal)
        assert torch.all(got[0][:5] == 0) and torch.all(got[1][:5] == -math.inf)
        if causal:
            assert torch.all(got[1][5:75] == -math.inf) and torch.isfinite(got[1][75:205]).all()
    e = tables([0, 0], 16, np.random.RandomState(0))
    z, lse = run(e, c, q[:7], indptr([4, 3]), True)
    assert torch.all(z == 0) and torch.all(lse == -math.inf)


def test_prefill_of_one_token_is_decode(cuda_device):
    t, c, q, qi = make("steps", 32, 8, [1, 1, 1], [4000, 100, 33], 16, cuda_device)
    o, lse = run(t, c, q, qi, True)
    od, lsed = fd.decode_paged_int8(q, c["k"], c["v"], c["ks"], c["vs"], t["ip"], t["last"], *dev_tables(t, cuda_device), D ** -0.5)
    compare((o, lse), t, c, q, qi, True)
    assert float((lse - lsed).abs().max()) <= 2 * LSE
    assert float((o.float() - od).abs().max()) <= 2.0 ** -8 * float(od.abs().max()) + 2.0 ** -10


@pytest.mark.parametrize("at", [0, 100, 900, 1500])
@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("nats", [6, 20, 90])
def test_prefill_scores_that_jump(cuda_device, at, two, nats):
    """One key far above all others, anywhere: its weight leaves f16's range in the
    first pass, or E has to follow; rows in front of it (causal) do not see it."""
    tokens = 300 if two else 20
    t, c, q, qi = make("jump", 4, 4, [tokens], [1600], 16, cuda_device)
    # the key's codes are those of the mean query's direction, its page's scale grows
    q = (q * 0.2 + torch.sign(torch.randn(4, D, device=cuda_device, generator=torch.Generator(cuda_device).manual_seed(1))))
    q = q.to(torch.bfloat16)
    page, r = int(t["ids"][at // 16]), at % 16
    c["k"][page] = 0
    c["k"][page, r] = (127 * torch.sign(q.float().mean(0))).to(torch.int8)
    c["ks"][page] = nats / (127 * D ** 0.5)
    for causal in (True, False):
        compare(run(t, c, q, qi, causal), t, c, q, qi, causal, what=f"{at} {nats} {causal}", lse_abs=2e-5 + nats * 2.0 ** -20)


def test_prefill_v_scales_far_apart(cuda_device):
    """Pages of zeros with the smallest scale (the first ones among them), scales that
    grow and fall by 2^20: each row as exact as its own keys allow."""
    rng = np.random.RandomState(2)
    for tokens in ([20], [300]):
        t, c, q, qi = make("vfar", 4, 4, tokens, [700], 16, cuda_device)
        e = torch.from_numpy(rng.randint(-10, 10, (t["num_pages"], 4))).to(cuda_device)
        c["vs"] *= torch.exp2(e.float())
        for j in (0, 1, 2, 3, 4, 5, 6, 7, 8, 20, 40):
            c["v"][int(t["ids"][j])] = 0
            c["vs"][int(t["ids"][j])] = 2.0 ** -126
        compare(run(t, c, q, qi, True), t, c, q, qi, True, what=str(tokens))
        compare(run(t, c, q, qi, False), t, c, q, qi, False, what=str(tokens))


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens", [20, 200])
def test_prefill_scales_that_are_no_numbers_reach_what_sees_them(cuda_device, which, value, tokens):
    t, c, q, qi = make("nan", 8, 4, [tokens, 30], [300, 200], 16, cuda_device)
    want = run(t, c, q, qi, True)
    at = 300 - 16 - 12   # page of keys 272 .. 287: seen from token tokens - 28 on
    c[which][int(t["ids"][at // 16]), 1] = value
    o, lse = run(t, c, q, qi, True)
    first = max(0, tokens - 300 + 272)
    bad = torch.zeros(o.shape[:2], dtype=torch.bool, device=cuda_device)
    bad[first:tokens, 2:4] = True
    got = ~torch.isfinite(o.float()).all(-1)
    # a row that sees an infinite K scale gets NaN unless all its scores there are -inf
    assert torch.equal(got & ~bad, torch.zeros_like(bad))
    assert float((got & bad).sum()) >= 0.9 * float(bad.sum())
    close = (o.float() - want[0].float()).abs() <= 2.0 ** -7 * want[0].float().abs() + 2.0 ** -9
    assert bool(close.all(-1)[~bad].all())


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), -0.01])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("tokens", [20, 200])
def test_prefill_no_number_is_nan_whatever_the_codes(cuda_device, which, value, sign, tokens):
    # scores of one sign and a scale that append never leaves: not a weight of 0, nor an infinity
    t, c, q, qi = make("all", 4, 1, [tokens, 1], [300, 1], 16, cuda_device)
    c["k"].fill_(3 * sign)
    c["v"].fill_(5)
    q.fill_(1.0)
    for page in (0, int(t["ip"][1])):   # the first page of either request
        c[which][int(t["ids"][page]), 0] = value
    o, _ = run(t, c, q, qi, True)
    assert bool(o.isnan().all())


def test_prefill_rows_behind_the_last_key_and_foreign_pages_do_not_matter(cuda_device):
    t, c, q, qi = make("leak", 16, 4, [30, 70, 16], [45, 70, 16], 48, cuda_device)
    want = run(t, c, q, qi, True)
    mine = torch.zeros(t["num_pages"], 48, dtype=torch.bool, device=cuda_device)
    for b in range(3):
        for j in range(t["ip"][b], t["ip"][b + 1]):
            mine[t["ids"][j], : t["last"][b] if j == t["ip"][b + 1] - 1 else 48] = True
    for x in ("k", "v"):
        c[x][~mine] = -128
        c[x + "s"][~mine.any(1)] = float("nan")
    got = run(t, c, q, qi, True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prefill_strides_padding_and_negative_scale(cuda_device):
    """Queries inside a fused projection, a padded batch, a negative softmax scale."""
    t, c, q, qi = make("stride", 8, 4, [37, 200], [100, 200], 16, cuda_device)
    wide = torch.full((240, 20, D), float("nan"), dtype=torch.bfloat16, device=cuda_device)
    wide[:237, 4:12] = q
    o = torch.full((240, 8, D), 5.0, dtype=torch.bfloat16, device=cuda_device)
    lse = torch.full((240, 8), 5.0, device=cuda_device)
    for scale in (D ** -0.5, -0.07, 0.0):
        run(t, c, wide[:, 4:12], qi, True, scale=scale, o=o, lse=lse)
        compare((o, lse), t, c, q, qi, True, scale=scale, what=str(scale))
        assert torch.all(o[237:] == 5.0) and torch.all(lse[237:] == 5.0)


def test_prefill_is_the_same_each_time_and_replayed(cuda_device):
    t, c, q, qi = make("again", 32, 8, [64, 5], [3000, 2000], 16, cuda_device)
    plan = plan_of(t, q, 8, qi, True)
    assert plan.num_merged_rows > 0
    want = run(t, c, q, qi, True, plan=plan)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=cuda_device)
    o, lse, qs = torch.empty_like(want[0]), torch.empty_like(want[1]), q.clone()
    tab, qid = dev_tables(t, cuda_device), torch.from_numpy(qi).to(cuda_device)

    def call():
        fd.prefill_paged_int8(plan, qs, c["k"], c["v"], c["ks"], c["vs"], qid, *tab, D ** -0.5, o=o, lse=lse, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
        call()
    for k in range(3):
        qs.copy_(q * (k + 1) / 2)
        g.replay()
        compare((o, lse), t, c, qs, qi, True, what=f"replay {k}")
    assert fd.get_device_status(ws) == 0


@pytest.mark.parametrize("log2", [118, 60, -60, -105])
def test_prefill_queries_of_any_size(cuda_device, log2):
    # bf16 reaches beyond f16 on both sides; the factor of the scores brings these back
    t, c, q, qi = make("sizes", 8, 2, [70, 3], [300, 200], 16, cuda_device)
    big = (q.double() * 2.0 ** log2).to(torch.bfloat16)
    assert torch.equal(big.double(), q.double() * 2.0 ** log2)
    got = run(t, c, big, qi, True, scale=D ** -0.5 * 2.0 ** -log2)
    compare(got, t, c, q, qi, True, what=str(log2))


def test_prefill_of_many_requests(cuda_device):
    # more requests than a warp looks at at once, some without tokens, keys or both; in
    # splits of 128 keys those of 129 on have partial rows
    rng = np.random.RandomState(5)
    tokens, keys = rng.randint(0, 4, 700), rng.randint(0, 300, 700)
    keys[rng.rand(700) < 0.1] = 0
    t, c, q, qi = make("many", 4, 2, list(tokens), list(keys), 16, cuda_device)
    for causal in (True, False):
        for chunk in (0, 128):
            plan = plan_of(t, q, 2, qi, causal, chunk=chunk)
            compare(run(t, c, q, qi, causal, plan=plan), t, c, q, qi, causal, what=f"{causal} {chunk}")


def test_prefill_calls_at_once(cuda_device):
    """Calls of other plans, and single tokens, on three streams, a workspace each."""
    sets = [make("one", 32, 8, [300, 70], [3000, 2000], 32, cuda_device),
            make("other", 16, 16, [40, 1, 7], [700, 5000, 90], 48, cuda_device)]
    tab = [dev_tables(x[0], cuda_device) + [torch.from_numpy(x[3]).to(cuda_device)] for x in sets]
    plans = [plan_of(x[0], x[2], x[1]["k"].shape[2], x[3], True) for x in sets]
    want = [run(*x, True, plan=p) for x, p in zip(sets, plans)]
    t, c = sets[0][:2]
    q1 = sets[0][2][:2].contiguous()
    single = fd.decode_paged_int8(q1, c["k"], c["v"], c["ks"], c["vs"], t["ip"], t["last"], *tab[0][:3], D ** -0.5)
    ws = [torch.zeros(p.workspace_bytes, dtype=torch.uint8, device=cuda_device) for p in plans]
    ws.append(torch.zeros(fd.plan_paged(2, 32, 8, D, 32, t["ip"], t["last"]).workspace_bytes, dtype=torch.uint8,
                          device=cuda_device))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (t, c, q, _), p, w, s, tb in zip(sets, plans, ws, streams, tab):
            got.append(fd.prefill_paged_int8(p, q, c["k"], c["v"], c["ks"], c["vs"], tb[3], *tb[:3], D ** -0.5, workspace=w,
                                             stream=s))
        t, c = sets[0][:2]
        got.append(fd.decode_paged_int8(q1, c["k"], c["v"], c["ks"], c["vs"], t["ip"], t["last"], *tab[0][:3], D ** -0.5,
                                        workspace=ws[2], stream=streams[2]))
    torch.cuda.synchronize()
    for n, (o, lse) in enumerate(got):
        w = (want + [single])[n % 3]
        assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
    assert all(fd.get_device_status(w) == 0 for w in ws)


def test_prefill_far_rows_of_a_large_pool(cuda_device):
    page, hkv, pages, dev = 16, 8, 300000, cuda_device   # 4.9e9 bytes a pool
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
    q = torch.randn((103, 16, D), device=dev).to(torch.bfloat16)
    qi = indptr([70, 33])
    compare(run(u, c, q, qi, True), t, small, q, qi, True)


def test_prefill_outside_the_plan_is_flagged(cuda_device):
    t, c, q, qi = make("bad", 8, 4, [40, 40], [100, 60], 16, cuda_device)
    plan = plan_of(t, q, 4, qi, True)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=cuda_device)
    tab, qid = dev_tables(t, cuda_device), torch.from_numpy(qi).to(cuda_device)

    def call(qid, ip, last, ids, plan=plan, ws=ws):
        fd.prefill_paged_int8(plan, q, c["k"], c["v"], c["ks"], c["vs"], qid, ip, last, ids, D ** -0.5, workspace=ws)
        return fd.get_device_status(ws)
    assert call(qid, *tab) == 0
    for bad in (-1, t["num_pages"], 1 << 30):
        ids = tab[2].clone()
        ids[2] = bad
        assert call(qid, tab[0], tab[1], ids) == -6
    ends = qid.clone()
    ends[2] = 81
    assert call(ends, *tab) == -6
    more = tab[0].clone()
    more[2] += 1
    assert call(qid, more, *tab[1:]) == -6
    last = tab[1].clone()
    last[0] = 17
    assert call(qid, tab[0], last, tab[2]) == -6
    many = plan_of(t, q, 4, indptr([40, 40]), True, chunk=128)   # (100 keys: no splits)
    assert call(qid, *tab, plan=many) == 0
    # a plan for fewer items than the tables need
    few = plan_of(dict(t, keys=t["keys"]), q, 4, indptr([79, 1]), True)
    few.num_items = 4
    assert call(qid, *tab, plan=few) == -6
    assert call(qid, *tab) == 0


def test_prefill_waits_are_bounded(cuda_device):
    t, c, q, qi = make("late", 8, 4, [40, 300], [100, 1000], 16, cuda_device)
    plan = plan_of(t, q, 4, qi, True, timeout_ns=0)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device=cuda_device)
    fd.prefill_paged_int8(plan, q, c["k"], c["v"], c["ks"], c["vs"], torch.from_numpy(qi).to(cuda_device),
                          *dev_tables(t, cuda_device), D ** -0.5, workspace=ws)
    assert fd.get_device_status(ws) == -5
    compare(run(t, c, q, qi, True), t, c, q, qi, True)


@pytest.mark.parametrize("chunk", [0, 128])
def test_prefill_over_its_own_queries(cuda_device, chunk):
    t, c, q, qi = make("over", 8, 4, [300, 1, 40], [300, 700, 640], 16, cuda_device)
    for causal in (True, False):
        plan = plan_of(t, q, 4, qi, causal, chunk=chunk)
        want = run(t, c, q, qi, causal, plan=plan)
        x = q.clone()
        o, lse = run(t, c, x, qi, causal, plan=plan, o=x)
        assert o.data_ptr() == x.data_ptr() and torch.equal(x, want[0]) and torch.equal(lse, want[1])
