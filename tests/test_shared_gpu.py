"""Shared-prefix decode on the GPU against the fp64 oracle's unsplit attention
over each request's whole list of keys (its prefix, then its own).

Tolerances as for fd_decode at small sizes: O within 1e-4 and 1e-5 in the 2-norm,
LSE within 2e-5.  The weights enter the second product as hi + lo 16-bit parts
(each within 2^-17 of itself), scores and sums are fp32."""
import numpy as np
import pytest
import torch

import oracle
import split_kv_flashdecoding_gb300 as fd
from tests.parity_util import assert_within, errors

pytestmark = pytest.mark.gpu
D = 128
TIGHT = dict(max_abs=1e-4, rel_l2=1e-5, lse_abs=2e-5)
SCALE = float(np.float32(1 / np.sqrt(128)))


def indptr(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def make(Hq, Hkv, reqs, lens, own, seed=0, kmul=1.0, room=None, spare=5):
    """Ragged inputs; rows past the last key hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B, T, S = sum(reqs), sum(lens), int(sum(own))
    room = S if room is None else room
    rand = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    i = dict(Hq=Hq, Hkv=Hkv, B=B, reqs=reqs, lens=lens, own=np.array(own, dtype=np.int64), room=room, scale=SCALE)
    i["q"] = rand(B, Hq, D)
    for n in "kv":
        for part, rows, extra in (("p", T, spare), ("", S, room - S)):
            x = rand(rows, Hkv, D) * (kmul if n == "k" else 1.0)
            i[n + part] = torch.cat([x, torch.full((extra, Hkv, D), float("nan"), dtype=torch.bfloat16)])
    return i


def reference(i, kv=None):
    kp, vp, k, v = kv or (i["kp"], i["vp"], i["k"], i["v"])
    pi, oi = indptr(i["lens"]), indptr(i["own"])
    K, V, n, b = [], [], [], 0
    for g, r in enumerate(i["reqs"]):
        for _ in range(r):
            K += [kp[pi[g]: pi[g + 1]], k[oi[b]: oi[b + 1]]]
            V += [vp[pi[g]: pi[g + 1]], v[oi[b]: oi[b + 1]]]
            n.append(i["lens"][g] + i["own"][b])
            b += 1
    return oracle.decode(i["q"], torch.cat(K), torch.cat(V), indptr(n), i["scale"])


def ragged(i, chunk=0, ws=None, stream=None, timeout_ns=None):
    req, pi = indptr(i["reqs"]), indptr(i["lens"])
    p = fd.plan_shared(i["B"], i["Hq"], i["Hkv"], D, req, pi, i["room"], chunk=chunk, timeout_ns=timeout_ns)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda") if ws is None else ws
    d = {n: i[n].cuda() for n in ("q", "kp", "vp", "k", "v")}
    tables = i32(req), i32(pi), i32(indptr(i["own"])) if i["room"] else None
    if stream is not None:   # the inputs are made on the current stream
        stream.wait_stream(torch.cuda.current_stream())
    o, lse = fd.decode_shared(p, d["q"], d["kp"], d["vp"], d["k"] if i["room"] else None,
                              d["v"] if i["room"] else None, *tables, i["scale"], workspace=ws, stream=stream)
    return o, lse, fd.get_device_status(ws, stream)


def to_pages(i, page, seed=0):
    """The same keys in pools; rows past a last key and spare pages hold NaN."""
    rng = np.random.RandomState(seed)
    pc, oc = -(-np.array(i["lens"]) // page), -(-i["own"] // page)
    total = int(pc.sum() + oc.sum())
    ids = rng.permutation(total + 3)[:total]
    pools = {}
    for n in "kv":
        pool = torch.full((total + 3, page, i["Hkv"], D), float("nan"), dtype=torch.bfloat16)
        at = 0
        for x, ip, cnt in ((i[n + "p"], indptr(i["lens"]), pc), (i[n], indptr(i["own"]), oc)):
            for r in range(len(cnt)):
                rows = x[ip[r]: ip[r + 1]]
                for j in range(int(cnt[r])):
                    part = rows[j * page: (j + 1) * page]
                    pool[ids[at], : len(part)] = part
                    at += 1
        pools[n] = pool
    last = lambda n, c: np.where(c > 0, n - (c - 1) * page, 0)  # noqa: E731
    np_ = int(pc.sum())
    return dict(pools=pools, pc=pc, oc=oc, pl=last(np.array(i["lens"]), pc), ol=last(i["own"], oc),
                pids=ids[:np_], oids=ids[np_:])


def paged(i, page, chunk=0, seed=0, pg=None):
    pg = to_pages(i, page, seed) if pg is None else pg
    req = indptr(i["reqs"])
    p = fd.plan_shared_paged(i["B"], i["Hq"], i["Hkv"], D, page, req, indptr(pg["pc"]), pg["pl"], i["room"], chunk=chunk)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    own = (i32(indptr(pg["oc"])), i32(pg["ol"]), i32(np.append(pg["oids"], 0))) if i["room"] else (None,) * 3
    o, lse = fd.decode_shared_paged(p, i["q"].cuda(), pg["pools"]["k"].cuda(), pg["pools"]["v"].cuda(), i32(req),
                                    i32(indptr(pg["pc"])), i32(pg["pl"]), i32(np.append(pg["pids"], 0)), *own,
                                    i["scale"], workspace=ws)
    return o, lse, fd.get_device_status(ws)


def check(i, out, ref=None, what=""):
    o, lse, status = out
    assert status == 0
    o_ref, lse_ref = reference(i) if ref is None else ref
    assert_within(errors(o.cpu().numpy(), lse.cpu().numpy(), o_ref.reshape(o.shape), lse_ref.reshape(lse.shape)),
                  **TIGHT, what=what)


def own_lengths(B, most, seed=1):
    n = np.random.RandomState(seed).randint(0, most + 1, B)
    n[::3] = 0
    return n


SMALL = [
    ("one_key", 8, 8, [2], [1]), ("tile_less_1", 8, 8, [2], [127]), ("tile", 32, 8, [3], [128]),
    ("tile_1", 32, 8, [3], [129]), ("two_tiles_1", 8, 2, [4], [257]), ("odd", 64, 8, [5], [1001]),
    ("rows_128", 32, 8, [32], [300]), ("rows_129", 3 * 1, 3, [129], [300]), ("rows_256", 8, 2, [64], [515]),
    ("rows_257", 1, 1, [257], [400]), ("rows_600", 16, 2, [75], [260]),
    ("three", 32, 8, [3, 40, 7], [300, 129, 1000]), ("gaps", 16, 8, [2, 0, 5, 3], [200, 77, 0, 1]),
    ("many", 4, 2, [1] * 37, list(range(1, 371, 10))),
]


@pytest.mark.parametrize("chunk", [0, 128, 256])
@pytest.mark.parametrize("name,Hq,Hkv,reqs,lens", SMALL, ids=[c[0] for c in SMALL])
def test_ragged_matches_oracle(cuda_device, name, Hq, Hkv, reqs, lens, chunk):
    i = make(Hq, Hkv, reqs, lens, own_lengths(sum(reqs), 70), seed=len(name))
    check(i, ragged(i, chunk), what=name)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 256])
@pytest.mark.parametrize("name,Hq,Hkv,reqs,lens", SMALL, ids=[c[0] for c in SMALL])
def test_paged_matches_oracle(cuda_device, name, Hq, Hkv, reqs, lens, page):
    i = make(Hq, Hkv, reqs, lens, own_lengths(sum(reqs), 70), seed=len(name) + page)
    check(i, paged(i, page, chunk=128 if page == 48 else 0, seed=page), what=f"{name} P={page}")


@pytest.mark.parametrize("Hq,Hkv,B,L", [(32, 8, 32, 20000), (32, 8, 61, 9999), (64, 8, 100, 5000)])
def test_long_prefixes(cuda_device, Hq, Hkv, B, L):
    i = make(Hq, Hkv, [B], [L], own_lengths(B, 500), seed=B)
    ref = reference(i)
    check(i, ragged(i), ref, f"{B} x {L}")
    check(i, paged(i, 16), ref, f"{B} x {L} paged")


@pytest.mark.parametrize("Hq,Hkv,B,L", [(1, 1, 1, 9000), (8, 8, 3, 1100), (32, 8, 8, 4100), (64, 8, 5, 3000)])
def test_few_rows_of_many_splits(cuda_device, Hq, Hkv, B, L):
    """More partials a row than a warp of the merge loads at once."""
    i = make(Hq, Hkv, [B], [L], own_lengths(B, 40), seed=L)
    check(i, ragged(i, 128), what="own keys")
    j = make(Hq, Hkv, [B, 1], [L, 130], np.zeros(B + 1, int), seed=L, room=0)
    check(j, ragged(j, 128), what="prefixes alone")
    j["kp"][L // 2, 0, 3] = float("nan")
    o, lse, status = ragged(j, 128)
    bad = torch.isnan(o).any(-1).cpu()
    want = torch.zeros(B + 1, Hq, dtype=torch.bool)
    want[:B, : Hq // Hkv] = True
    assert status == 0 and torch.equal(bad, want) and torch.equal(torch.isnan(lse).cpu(), want)


@pytest.mark.parametrize("L", [1024, 1025, 2176, 2177, 4100, 20000])
@pytest.mark.parametrize("B", [5, 33, 64])
def test_long_splits(cuda_device, B, L):
    """One split for all keys: O goes over to fp32 sums every few tiles, in one
    row tile (two streams of keys) and in two."""
    i = make(8, 2, [B], [L], np.zeros(B, int), seed=L, room=0)
    check(i, ragged(i, -(-L // 128) * 128), what=f"{B} x {L}")


def levels(L):
    """A key's first value when the queries' first value is the same for all: the
    last third counts most, the others are 8.5 below it by SCALE with queries of
    16 (in nats), the first three tiles 45, 40 and 30.  The weights of the first
    pass, which refer to the first tile, leave their range."""
    x = torch.zeros(L)
    x[: L * 2 // 3] = -6.0
    x[:128], x[128:256], x[256:384] = -32.0, -28.0, -21.0
    return x


@pytest.mark.parametrize("L", [1500, 6000, 12001])
@pytest.mark.parametrize("B", [5, 64])
def test_long_splits_out_of_range(cuda_device, B, L):
    """One split whose first pass leaves the weights' range: the second raises
    the maximum and goes over to fp32 sums as well."""
    i = make(8, 2, [B], [L], np.zeros(B, int), seed=L, room=0)
    i["q"][..., 0] = 16.0
    i["kp"][:L, :, 0] = levels(L)[:, None].to(torch.bfloat16)
    ref = reference(i)
    check(i, ragged(i, -(-L // 128) * 128), ref, f"{B} x {L}")
    check(i, paged(i, 16, -(-L // 128) * 128), ref, f"{B} x {L} paged")


@pytest.mark.parametrize("B", [5, 64])
def test_fp8_long_splits_out_of_range(cuda_device, B):
    L = 6000
    f = to_fp8(make(8, 2, [B], [L], np.full(B, 3), seed=7), seed=7)
    sk = f["sk"].cpu()
    f["q"][..., 0] = 1024.0   # the scales are up to 1 / 64
    f["kp8"][:L, :, 0] = (levels(L)[:, None] * sk.sign()).to(torch.float8_e4m3fn).view(torch.uint8)
    f["kpd"][:L, :, 0] = (levels(L)[:, None] * sk.abs()).double().numpy()
    o, lse, status = ragged_fp8(f, -(-L // 128) * 128)
    ref = fp8_reference(f)
    assert status == 0
    assert_within(errors(o.cpu().numpy(), lse.cpu().numpy(), *ref), max_abs=1e-4, rel_l2=1e-5,
                  lse_abs=2e-5 * max(1.0, np.abs(ref[1]).max() / 16))


@pytest.mark.parametrize("rows", [3, 40])
def test_no_suffix_and_no_keys(cuda_device, rows):
    i = make(32, 8, [rows, 2], [700, 0], np.zeros(rows + 2, int), room=0)
    check(i, ragged(i))
    check(i, paged(i, 16))
    j = make(32, 8, [rows], [0], np.zeros(rows, int), room=64)   # room for keys, none yet
    o, lse, status = ragged(j)
    assert status == 0 and torch.all(o == 0) and torch.all(lse == -float("inf"))


def test_a_call_without_keys_waits_for_its_tables(cuda_device):
    """The tables come from page copies, whose grid lets the next one start early;
    the only grid of a call without any key reads them."""
    B, pages = 6, 600
    p = fd.plan_shared(B, 8, 8, D, [0, B], [0, 0], 0)
    q = torch.zeros((B, 8, D), dtype=torch.bfloat16, device="cuda")
    big = torch.zeros((pages, 65536), dtype=torch.uint8, device="cuda")
    small = torch.zeros((pages, 4), dtype=torch.int32, device="cuda")   # page 0: [0, B, 0, 0], the last: torn
    small[0, 1] = B
    src, dst = i32(np.arange(pages // 2)), i32(np.arange(pages - 1, pages // 2 - 1, -1))
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        small[-1] = -7
        fd.copy_pages([big, small], src, dst)   # page 0 to the last
        o, lse = fd.decode_shared(p, q, None, None, None, None, small[-1, :2], small[-1, 2:], None, SCALE, workspace=ws)
        assert fd.get_device_status(ws) == 0
        assert torch.all(o == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.5])
def test_scales(cuda_device, scale):
    i = make(32, 8, [5, 60], [513, 300], own_lengths(65, 40))
    i["scale"] = float(np.float32(scale))
    o, lse, status = ragged(i)
    assert status == 0
    o_ref, lse_ref = reference(i)
    # LSE grows with the scores (up to 1.5 * 60): fp32's steps with it
    err = errors(o.cpu().numpy(), lse.cpu().numpy(), o_ref.reshape(o.shape), lse_ref.reshape(lse.shape))
    assert_within(err, max_abs=1e-4, rel_l2=1e-5, lse_abs=2e-5 * max(1.0, abs(lse_ref).max() / 16))


@pytest.mark.parametrize("order", ["rising", "falling", "outliers"])
def test_scores_that_move_the_maximum(cuda_device, order):
    """Keys whose scores rise tile by tile raise the running maximum every
    time; falling ones never do; a few large ones do it once."""
    for B in (6, 50):
        i = make(32, 8, [B], [1500], own_lengths(B, 30), seed=3)
        f = torch.linspace(0.1, 6.0, 1500) if order == "rising" else torch.linspace(6.0, 0.1, 1500)
        if order == "outliers":
            f = torch.where(torch.rand(1500, generator=torch.Generator().manual_seed(1)) < 0.01, 16.0, 1.0)
        i["kp"][:1500] = (i["kp"][:1500].float() * f[:, None, None]).to(torch.bfloat16)
        ref = reference(i)
        for out in (ragged(i), ragged(i, 128), paged(i, 32)):
            o, lse, status = out
            assert status == 0
            assert_within(errors(o.cpu().numpy(), lse.cpu().numpy(), ref[0].reshape(o.shape),
                                 ref[1].reshape(lse.shape)), max_abs=1e-4, rel_l2=1e-5,
                          lse_abs=2e-5 * max(1.0, abs(ref[1]).max() / 16), what=order)


def test_identical_keys_give_the_mean(cuda_device):
    i = make(32, 8, [40], [900], np.zeros(40, int), room=0)
    i["kp"][:900] = i["kp"][0]
    o, lse, status = ragged(i)
    mean = i["vp"][:900].double().mean(0).repeat_interleave(4, 0)
    assert status == 0 and torch.all((o.cpu().double() - mean).abs() < 1e-5)


def test_nan_spreads_to_its_own_rows_only(cuda_device):
    i = make(16, 8, [3, 4], [300, 200], own_lengths(7, 20), spare=0)
    i["kp"][310, 2] = float("nan")   # a key of the second prefix
    o, lse, status = ragged(i)
    assert status == 0
    bad = torch.isnan(o).any(-1).cpu()
    want = torch.zeros(7, 16, dtype=torch.bool)
    want[3:, 4:6] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(lse).cpu(), want)
    j = dict(i, kp=i["kp"].nan_to_num(0.0))
    ref_o, _ = reference(j)
    ok = ~want
    assert np.abs(o.cpu().double().numpy() - ref_o.reshape(o.shape))[ok.numpy()].max() < 1e-4


def test_matches_decode_over_whole_lists(cuda_device):
    """The same requests through decode_paged, each with the prefix's pages at
    the head of its own table."""
    i = make(32, 8, [9], [640], own_lengths(9, 90), seed=8)
    pg = to_pages(i, 64)
    o, lse, status = paged(i, 64, pg=pg)
    assert status == 0
    at, tables = indptr(pg["oc"]), []
    for b in range(9):
        tables.append(np.concatenate([pg["pids"], pg["oids"][at[b]: at[b + 1]]]))
    ip = indptr([len(t) for t in tables])
    ll = np.where(pg["oc"] > 0, pg["ol"], 64).astype(np.int32)
    o2, lse2 = fd.decode_paged(i["q"].cuda(), pg["pools"]["k"].cuda(), pg["pools"]["v"].cuda(), ip, ll, i32(ip),
                               i32(ll), i32(np.concatenate(tables)), i["scale"])
    assert (o - o2).abs().max() < 2e-5 and (lse - lse2).abs().max() < 2e-5


def test_repeats_are_identical_and_other_streams_work(cuda_device):
    """Prefixes alone: the split kernel of the suffixes claims its items as CTAs
    come free when they are more than a wave, and which warp sums which tile
    (the last bit) goes with the claim."""
    i = make(32, 8, [50], [3000], np.zeros(50, int), room=0)
    first = ragged(i)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = ragged(i)
    third = ragged(i, stream=s)
    s.synchronize()
    for what, other in (("current stream", second), ("given stream", third)):
        assert torch.equal(first[0], other[0]) and torch.equal(first[1], other[1]), what


def test_what_a_call_allocates_belongs_to_its_stream(cuda_device):
    """No workspace or outputs given, and the current stream busy: nothing of
    the call waits for it, and its memory is not handed on meanwhile."""
    i = make(32, 8, [50], [3000], own_lengths(50, 40))
    req, pi, oi = indptr(i["reqs"]), indptr(i["lens"]), indptr(i["own"])
    p = fd.plan_shared(50, 32, 8, D, req, pi, i["room"])
    d = {n: i[n].cuda() for n in ("q", "kp", "vp", "k", "v")}
    args = (p, d["q"], d["kp"], d["vp"], d["k"], d["v"], i32(req), i32(pi), i32(oi), SCALE)
    s, x = torch.cuda.Stream(), torch.ones(4096, 4096, device="cuda")
    torch.full((p.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")   # freed: what torch hands out next
    torch.cuda.synchronize()
    for _ in range(8):
        x = x @ x * 1e-4
    o, lse = fd.decode_shared(*args, stream=s)
    torch.full((p.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    s.synchronize()
    check(i, (o, lse, 0))


def test_a_stream_of_another_device_is_refused(cuda_device):
    refs = torch.zeros(4, dtype=torch.int32, device="cuda")

    class Other:
        device, cuda_stream = torch.device("cuda", 1), 0
    with pytest.raises(fd.FdError):
        fd.compact_pages(refs, refs, 0, stream=Other())


def test_workspace_serves_call_after_call(cuda_device):
    """Calls queued on one workspace without waiting, of two inputs in turn."""
    a, b = (make(32, 8, [20, 9], [1000, 333], own_lengths(29, 60, s), seed=s, room=2000) for s in (1, 2))
    req, pi = indptr(a["reqs"]), indptr(a["lens"])
    p = fd.plan_shared(29, 32, 8, D, req, pi, 2000)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    dev = [{n: x[n].cuda() for n in ("q", "kp", "vp", "k", "v")} | dict(ip=i32(indptr(x["own"]))) for x in (a, b)]
    outs = []
    for r in range(6):
        d = dev[r % 2]
        outs.append(fd.decode_shared(p, d["q"], d["kp"], d["vp"], d["k"], d["v"], i32(req), i32(pi), d["ip"], SCALE,
                                     workspace=ws))
    assert fd.get_device_status(ws) == 0
    for x, got in ((a, outs[0::2]), (b, outs[1::2])):
        check(x, (*got[0], 0))
        for o, lse in got[1:]:   # up to the split kernel's last bits (see above)
            assert (o - got[0][0]).abs().max() < 2e-6 and (lse - got[0][1]).abs().max() < 2e-6


@pytest.mark.parametrize("is_paged", [False, True])
def test_captured_steps_follow_the_suffixes(cuda_device, is_paged):
    """One capture, replayed while the requests grow (from no keys at all)."""
    B, page, room = 21, 16, 21 * 48
    i = make(32, 8, [13, 8], [777, 130], np.full(B, 48), seed=5)
    pg = to_pages(i, page)
    req = indptr(i["reqs"])
    o = torch.empty((B, 32, D), device="cuda")
    lse = torch.empty((B, 32), device="cuda")
    q = i["q"].cuda()
    if is_paged:
        p = fd.plan_shared_paged(B, 32, 8, D, page, req, indptr(pg["pc"]), pg["pl"], room)
        k, v = pg["pools"]["k"].cuda(), pg["pools"]["v"].cuda()
        t = [i32(req), i32(indptr(pg["pc"])), i32(pg["pl"]), i32(pg["pids"])]
        live = [i32(np.zeros(B + 1)), i32(np.zeros(B)), i32(np.zeros(B * 3))]
    else:
        p = fd.plan_shared(B, 32, 8, D, req, indptr(i["lens"]), room)
        kp, vp = i["kp"].cuda(), i["vp"].cuda()
        k, v = (torch.zeros((room, 8, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        t = [i32(req), i32(indptr(i["lens"]))]
        live = [i32(np.zeros(B + 1))]
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        if is_paged:
            fd.decode_shared_paged(p, q, k, v, *t, *live, SCALE, o=o, lse=lse, workspace=ws)
        else:
            fd.decode_shared(p, q, kp, vp, k, v, *t, *live, SCALE, o=o, lse=lse, workspace=ws)
    at = indptr(i["own"])
    for step in (0, 1, 17, 48):
        own = np.minimum(np.arange(B) % 5 * step, 48)
        rows = np.concatenate([np.arange(at[b], at[b] + own[b]) for b in range(B)]).astype(np.int64)
        j = dict(i, own=own, k=i["k"][rows], v=i["v"][rows])
        if is_paged:
            cnt = -(-own // page)
            ids = np.concatenate([pg["oids"][3 * b: 3 * b + cnt[b]] for b in range(B)] + [np.zeros(0, int)])
            live[0].copy_(i32(indptr(cnt)))
            live[1].copy_(i32(np.where(cnt > 0, own - (cnt - 1) * page, 0)))
            live[2][: len(ids)].copy_(i32(ids))
        else:
            live[0].copy_(i32(indptr(own)))
            k[: len(rows)] = j["k"].cuda()
            v[: len(rows)] = j["v"].cuda()
        g.replay()
        check(j, (o, lse, fd.get_device_status(ws)), what=f"step {step}")


def test_tables_beyond_the_plan_are_flagged(cuda_device):
    i = make(8, 8, [4], [300], [5, 6, 7, 8], room=26)
    req, pi = indptr(i["reqs"]), indptr(i["lens"])
    d = {n: i[n].cuda() for n in ("q", "kp", "vp", "k", "v")}
    for own_ip, pre, code in (([0, 5, 11, 18, 26], [0, 300], 0), ([0, 5, 11, 18, 27], [0, 300], -6),
                              ([0, 5, 11, 18, 26], [0, 301], -6), ([0, 5, 11, 18, 26], [-1, 299], -6)):
        p = fd.plan_shared(4, 8, 8, D, req, pi, 26)
        ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
        fd.decode_shared(p, d["q"], d["kp"], d["vp"], d["k"], d["v"], i32(req), i32(pre), i32(own_ip), SCALE,
                         workspace=ws)
        assert fd.get_device_status(ws) == code


@pytest.mark.parametrize("own,code", [([0, 0, 0, 0], 0), ([0, 0, 1, 0], -6), ([5, 6, 7, 8], -6)])
def test_own_keys_without_room_are_flagged(cuda_device, own, code):
    """A plan without room for own keys, called with their tables all the same."""
    i = make(8, 8, [4], [300], own)
    req, pg = indptr(i["reqs"]), to_pages(i, 16)
    p = fd.plan_shared(4, 8, 8, D, req, indptr(i["lens"]), 0)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    d = {n: i[n].cuda() for n in ("q", "kp", "vp", "k", "v")}
    for k, v in ((d["k"], d["v"]), (None, None)):
        fd.decode_shared(p, d["q"], d["kp"], d["vp"], k, v, i32(req), i32(indptr(i["lens"])), i32(indptr(own)), SCALE,
                         workspace=ws)
        assert fd.get_device_status(ws) == code
    p = fd.plan_shared_paged(4, 8, 8, D, 16, req, indptr(pg["pc"]), pg["pl"], 0)
    tables = i32(req), i32(indptr(pg["pc"])), i32(pg["pl"]), i32(pg["pids"])
    for last, ids in ((i32(pg["ol"]), i32(np.append(pg["oids"], 0))), (None, None)):
        fd.decode_shared_paged(p, d["q"], pg["pools"]["k"].cuda(), pg["pools"]["v"].cuda(), *tables, i32(indptr(pg["oc"])),
                               last, ids, SCALE, workspace=ws)
        assert fd.get_device_status(ws) == code
    with pytest.raises(fd.FdError):   # a table of another length than the batch's
        fd.decode_shared(p, d["q"], d["kp"], d["vp"], None, None, i32(req), i32(indptr(i["lens"])), i32([0, 0]), SCALE)


BIG = 2 ** 31 - 1


@pytest.mark.parametrize("req,pre", [
    ([0, 4, 9], [0, 300, BIG]), ([0, 4, 9], [0, -1, 430]), ([0, 4, 9], [0, 500, 430]), ([0, 4, BIG], [0, 300, 430]),
    ([0, -5, 9], [0, 300, 430]), ([5, 4, 9], [0, 300, 430]), ([0, 10, -BIG], [0, 300, 430]),
    ([0, 4, 9], [-BIG, 300, 430]), ([-BIG, BIG, 9], [-BIG, BIG, 430]), ([0, 0, 9], [0, 0, 430]),
])
def test_torn_tables_are_flagged(cuda_device, req, pre):
    """Tables that are no lists of lengths, or longer ones than the plan's."""
    i = make(32, 8, [4, 5], [300, 130], np.zeros(9, int), room=0)
    d = {n: i[n].cuda() for n in ("q", "kp", "vp")}
    p = fd.plan_shared(9, 32, 8, D, [0, 4, 9], [0, 300, 430], 0, chunk=128)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    fd.decode_shared(p, d["q"], d["kp"], d["vp"], None, None, i32(req), i32(pre), None, SCALE, workspace=ws)
    assert fd.get_device_status(ws) == -6


@pytest.mark.parametrize("req", [[0, 63, 128], [0, 65, 128], [0, 64, 128]])
def test_prefixes_that_need_more_items_than_the_plan_are_flagged(cuda_device, req):
    """Requests that change prefixes: as many keys and partial rows as planned, but
    260 query rows of a KV head are two blocks where 256 were one."""
    i = make(32, 8, [64, 64], [1000, 1000], np.zeros(128, int), room=0)
    d = {n: i[n].cuda() for n in ("q", "kp", "vp")}
    p = fd.plan_shared(128, 32, 8, D, [0, 64, 128], [0, 1000, 2000], 0, chunk=128)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    fd.decode_shared(p, d["q"], d["kp"], d["vp"], None, None, i32(req), i32([0, 1000, 2000]), None, SCALE, workspace=ws)
    assert fd.get_device_status(ws) == (0 if req[1] == 64 else -6)


def test_page_outside_the_pool_is_flagged(cuda_device):
    i = make(8, 8, [4], [300], np.zeros(4, int), room=0)
    for bad in (-1, 10 ** 6):
        pg = to_pages(i, 16)
        pg["pids"][7] = bad
        assert paged(i, 16, pg=pg)[2] == -6


def test_a_wait_that_runs_out_is_reported(cuda_device):
    """timeout_ns = 0: every wait gives up at once, the call reports it, and the
    next call with a zeroed workspace is right."""
    for B in (4, 60):
        i = make(32, 8, [B], [2000], np.zeros(B, int), room=0)
        assert ragged(i, timeout_ns=0)[2] == -5
        check(i, ragged(i))


def test_binding_refusals(cuda_device):
    i = make(8, 8, [4], [300], [5, 6, 7, 8])
    req, pi, oi = i32(indptr(i["reqs"])), i32(indptr(i["lens"])), i32(indptr(i["own"]))
    p = fd.plan_shared(4, 8, 8, D, indptr(i["reqs"]), indptr(i["lens"]), 26)
    d = {n: i[n].cuda() for n in ("q", "kp", "vp", "k", "v")}
    good = [p, d["q"], d["kp"], d["vp"], d["k"], d["v"], req, pi, oi, SCALE]
    fd.decode_shared(*good)
    for at, x in ((1, d["q"][:3]), (1, d["q"].float()), (1, i["q"]), (2, d["kp"][:299]), (3, d["vp"].half()),
                  (4, d["k"][:25]), (4, None), (2, d["kp"].transpose(0, 1)), (6, req.long()), (7, pi[:1]), (8, None),
                  (8, oi[:4]), (8, oi.cpu())):
        bad = list(good)
        bad[at] = x
        with pytest.raises(fd.FdError):
            fd.decode_shared(*bad)


def test_missing_tensors_are_refused(cuda_device):
    i = make(8, 8, [4], [300], [5, 6, 7, 8])
    pg = to_pages(i, 16)
    d = {n: i[n].cuda() for n in ("q", "kp", "vp", "k", "v")}
    p = fd.plan_shared(4, 8, 8, D, indptr(i["reqs"]), indptr(i["lens"]), 26)
    good = [p, d["q"], d["kp"], d["vp"], d["k"], d["v"], i32(indptr(i["reqs"])), i32(indptr(i["lens"])),
            i32(indptr(i["own"])), SCALE]
    pp = fd.plan_shared_paged(4, 8, 8, D, 16, indptr(i["reqs"]), indptr(pg["pc"]), pg["pl"], 26)
    paged_good = [pp, d["q"], pg["pools"]["k"].cuda(), pg["pools"]["v"].cuda(), i32(indptr(i["reqs"])),
                  i32(indptr(pg["pc"])), i32(pg["pl"]), i32(pg["pids"]), i32(indptr(pg["oc"])), i32(pg["ol"]),
                  i32(pg["oids"]), SCALE]
    for call, args, missing in ((fd.decode_shared, good, (2, 3, 4, 5, 8)), (fd.decode_shared_paged, paged_good, (8, 9))):
        call(*args)
        for at in missing:
            bad = list(args)
            bad[at] = None
            with pytest.raises(fd.FdError):
                call(*bad)


# ------------------------------------------------------------------------ FP8

def to_fp8(i, seed=0):
    """Random E4M3 codes for the keys and values (NaN codes only past the last
    key), with scales per head, one of them negative; and what they stand for."""
    rng = np.random.RandomState(seed)
    f = dict(i)
    sc = {n: (rng.uniform(0.3, 1.0, i["Hkv"]) / 64).astype(np.float32) for n in "kv"}
    sc["k"][0] *= -1
    for n in "kv":
        for part in ("p", ""):
            x = i[n + part]
            nan = torch.isnan(x.float()).numpy()
            codes = rng.randint(0, 256, x.shape).astype(np.uint8)
            codes[(codes & 0x7F) == 0x7F] = 0x3A
            codes[(codes & 0x78) == 0x78] &= 0xB7   # magnitudes up to 30: scores of a softmax
            f[n + part + "8"] = torch.from_numpy(np.where(nan, 0x7F, codes).astype(np.uint8))
            f[n + part + "d"] = oracle.dequant_fp8(np.where(nan, 0, codes).astype(np.uint8), sc[n])
    f["sk"], f["sv"] = (torch.from_numpy(sc[n]).cuda() for n in "kv")
    return f


def fp8_reference(f):
    """fp64 attention over the dequantised values, request by request."""
    pi, oi, g = indptr(f["lens"]), indptr(f["own"]), f["Hq"] // f["Hkv"]
    q = f["q"].double().numpy()
    o, lse, b = np.zeros((f["B"], f["Hq"], D)), np.full((f["B"], f["Hq"]), -np.inf), 0
    for p, r in enumerate(f["reqs"]):
        for _ in range(r):
            K = np.concatenate([f["kpd"][pi[p]: pi[p + 1]], f["kd"][oi[b]: oi[b + 1]]])
            V = np.concatenate([f["vpd"][pi[p]: pi[p + 1]], f["vd"][oi[b]: oi[b + 1]]])
            if len(K):
                s = np.einsum("hd,lhd->hl", q[b], np.repeat(K, g, 1)) * f["scale"]
                m = s.max(1, keepdims=True)
                w = np.exp(s - m)
                lse[b] = m[:, 0] + np.log(w.sum(1))
                o[b] = np.einsum("hl,lhd->hd", w / w.sum(1, keepdims=True), np.repeat(V, g, 1))
            b += 1
    return o, lse


def ragged_fp8(f, chunk=0):
    req, pi = indptr(f["reqs"]), indptr(f["lens"])
    p = fd.plan_shared(f["B"], f["Hq"], f["Hkv"], D, req, pi, f["room"], chunk=chunk)
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    d = {n: f[n].cuda() for n in ("q", "kp8", "vp8", "k8", "v8")}
    o, lse = fd.decode_shared_fp8(p, d["q"], d["kp8"], d["vp8"], d["k8"], d["v8"], f["sk"], f["sv"], i32(req), i32(pi),
                                  i32(indptr(f["own"])), f["scale"], workspace=ws)
    return o, lse, fd.get_device_status(ws)


def paged_fp8(f, page, seed=0):
    j = dict(f, **{n + part: f[n + part + "8"] for n in "kv" for part in ("p", "")})
    pg = to_pages(dict(j, **{n: j[n].float() for n in ("kp", "vp", "k", "v")}), page, seed)
    pools = {n: torch.where(torch.isnan(x.float()), torch.tensor(127.0), x.float()).to(torch.uint8).cuda()
             for n, x in pg["pools"].items()}
    req = indptr(f["reqs"])
    p = fd.plan_shared_paged(f["B"], f["Hq"], f["Hkv"], D, page, req, indptr(pg["pc"]), pg["pl"], f["room"])
    ws = torch.zeros(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    o, lse = fd.decode_shared_paged_fp8(p, f["q"].cuda(), pools["k"], pools["v"], f["sk"], f["sv"], i32(req),
                                        i32(indptr(pg["pc"])), i32(pg["pl"]), i32(np.append(pg["pids"], 0)),
                                        i32(indptr(pg["oc"])), i32(pg["ol"]), i32(np.append(pg["oids"], 0)),
                                        f["scale"], workspace=ws)
    return o, lse, fd.get_device_status(ws)


@pytest.mark.parametrize("name,Hq,Hkv,reqs,lens", SMALL, ids=[c[0] for c in SMALL])
def test_fp8_matches_64_bits(cuda_device, name, Hq, Hkv, reqs, lens):
    f = to_fp8(make(Hq, Hkv, reqs, lens, own_lengths(sum(reqs), 40), seed=len(name)), seed=len(name))
    ref = fp8_reference(f)
    # scores reach tens: fp32 steps of the LSE grow with it
    lse_abs = 2e-5 * max(1.0, np.abs(ref[1][np.isfinite(ref[1])]).max(initial=0) / 16)
    for what, out in (("ragged", ragged_fp8(f)), ("chunks", ragged_fp8(f, 128)), ("paged 16", paged_fp8(f, 16, 1)),
                      ("paged 48", paged_fp8(f, 48, 2)), ("paged 256", paged_fp8(f, 256, 3))):
        o, lse, status = out
        assert status == 0
        assert_within(errors(o.cpu().numpy(), lse.cpu().numpy(), *ref), max_abs=1e-4, rel_l2=1e-5, lse_abs=lse_abs,
                      what=f"{name} {what}")


def test_fp8_nan_codes_spread(cuda_device):
    f = to_fp8(make(8, 8, [3, 2], [300, 200], np.full(5, 4), spare=0))
    f["vp8"][350, 5, 7] = 0xFF
    o, lse, status = ragged_fp8(f)
    bad = torch.isnan(o).cpu()
    want = torch.zeros(5, 8, 128, dtype=torch.bool)
    want[3:, 5, 7] = True
    assert status == 0 and torch.equal(bad, want) and torch.isfinite(lse).all()


def test_fp8_binding_refusals(cuda_device):
    f = to_fp8(make(8, 8, [4], [300], [5, 6, 7, 8]))
    req, pi, oi = i32(indptr(f["reqs"])), i32(indptr(f["lens"])), i32(indptr(f["own"]))
    p = fd.plan_shared(4, 8, 8, D, indptr(f["reqs"]), indptr(f["lens"]), 26)
    d = {n: f[n].cuda() for n in ("q", "kp8", "vp8", "k8", "v8", "kp")}
    good = [p, d["q"], d["kp8"], d["vp8"], d["k8"], d["v8"], f["sk"], f["sv"], req, pi, oi, SCALE]
    fd.decode_shared_fp8(*good)
    for at, x in ((2, d["kp"]), (6, f["sk"][:7]), (7, f["sv"].double()), (7, f["sv"].cpu())):
        bad = list(good)
        bad[at] = x
        with pytest.raises(fd.FdError):
            fd.decode_shared_fp8(*bad)
