"""fd_fork_pages, fd_compact_pages and fd_copy_pages on the GPU against their
definitions written out entry by entry.  Whole numbers: everything is equal."""
import threading

import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd

pytestmark = pytest.mark.gpu


def indptr(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def fork_reference(parent, ip, last, ids, nip, refs, page):
    refs_in, refs = refs, refs.copy()
    free = [p for p in range(len(refs)) if refs_in[p] == 0]
    first, at, out, src, dst = {}, 0, [], [], []
    for i, par in enumerate(parent):
        if par >= 0:
            first.setdefault(int(par), i)
    for i, par in enumerate(parent):
        table = [] if par < 0 else list(ids[ip[par]: ip[par + 1]])
        s = d = -1
        if table and last[par] < page and not (first[int(par)] == i and refs_in[table[-1]] == 1):
            s, d = table[-1], free[at]
            table[-1] = d
            at += 1
        while len(table) < nip[i + 1] - nip[i]:
            table.append(free[at])
            at += 1
        out += table
        src.append(s)
        dst.append(d)
    for p in ids[: ip[-1]]:
        refs[p] -= 1
    for p in out:
        refs[p] += 1
    as32 = lambda x: np.array(x, dtype=np.int32)  # noqa: E731
    return as32(out), refs, as32(src), as32(dst)


def random_tables(rng, batch, page, num_pages, most, share=True):
    keys = rng.randint(0, most * page + 1, batch)
    keys[rng.rand(batch) < 0.2] //= page
    keys[rng.rand(batch) < 0.2] *= page
    keys = np.minimum(keys, most * page)
    cnt = -(-keys // page)
    ids, tables, at = rng.permutation(num_pages), [], 0
    for b in range(batch):
        t = ids[at: at + cnt[b]].copy()
        at += int(cnt[b])
        if share and b and rng.rand() < 0.5:
            h = min(len(t), len(tables[-1])) // 2
            t[:h] = tables[-1][:h]
        tables.append(t)
    flat = np.concatenate(tables + [np.zeros(0, int)]).astype(np.int32)
    refs = np.bincount(flat, minlength=num_pages).astype(np.int32)
    return indptr(cnt), (keys - (cnt - 1) * page * (cnt > 0)).astype(np.int32) * (cnt > 0), flat, refs


def dev(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda() for a in arrays]


def fork(parent, ip, last, ids, nip, refs, page, inplace=False, ws=None):
    t = dev(parent, ip, last, ids, nip, refs)
    ws = torch.zeros(fd.pages_workspace_bytes(len(refs), len(parent)), dtype=torch.uint8, device="cuda") if ws is None else ws
    out = fd.fork_pages(*t[:5], int(nip[-1]), page, t[5], new_page_refs=t[5] if inplace else None, workspace=ws)
    status = fd.get_device_status(ws)
    return [x.cpu().numpy() for x in out], status


CASES = [(1, 1, 5, 1), (3, 7, 40, 4), (8, 32, 1024, 20), (5, 1, 1023, 30), (17, 40, 1025, 12),
         (64, 251, 5000, 40), (2, 0, 33, 3), (1500, 2100, 9000, 2),
         (30, 90, 65537, 25), (9, 20, 300000, 300)]


@pytest.mark.parametrize("batch,children,num_pages,most", CASES)
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("seed", [0, 1])
def test_fork_matches_the_definition(cuda_device, batch, children, num_pages, most, page, seed):
    rng = np.random.RandomState(seed + 7 * children)
    ip, last, ids, refs = random_tables(rng, batch, page, num_pages, most)
    held = rng.permutation(np.flatnonzero(refs == 0))[: np.count_nonzero(refs == 0) // 8]
    refs[held] += 2   # pages that other tables hold
    parent = rng.randint(-1, batch, children)
    have = np.where(parent < 0, 0, (ip[1:] - ip[:-1])[np.maximum(parent, 0)]) if children else np.zeros(0, int)
    spare = np.count_nonzero(refs == 0)
    grow = rng.randint(0, 3, children)
    grow[np.cumsum(grow + 1) > spare] = 0
    want = None
    nip = indptr(have + grow)
    if children <= spare or children == 0:
        want = fork_reference(parent, ip, last, ids, nip, refs, page)
    if want is None:
        pytest.skip("too few pages for this draw")
    for inplace in (False, True):
        got, status = fork(parent, ip, last, ids, nip, refs, page, inplace)
        assert status == 0
        for g, w in zip(got, want):
            assert np.array_equal(g, w)


def test_fork_without_children_frees_everything(cuda_device):
    ip, last, ids, refs = random_tables(np.random.RandomState(4), 6, 16, 100, 10)
    got, status = fork(np.zeros(0), ip, last, ids, indptr([]), refs, 16)
    assert status == 0 and not got[1].any()


def test_fork_from_nothing_takes_the_lowest_pages(cuda_device):
    refs = np.zeros(20, np.int32)
    refs[[0, 2, 3]] = 1
    got, status = fork([-1, -1], [0], [], [0], indptr([2, 3]), refs, 16)
    assert status == 0 and got[0].tolist() == [1, 4, 5, 6, 7] and got[2].tolist() == [-1, -1]


@pytest.mark.parametrize("what", ["pages", "parent", "shrink", "entries", "tail", "last"])
def test_a_refused_fork_changes_nothing(cuda_device, what):
    ip, last, ids, refs = np.array([0, 2, 3]), np.array([3, 16]), np.array([4, 1, 2]), np.array([0, 1, 1, 0, 1, 0])
    parent, nip, code = np.array([0, 0, 1]), np.array([0, 2, 4, 5]), -6
    good, status = fork(parent, ip, last, ids, nip, refs, 16)
    assert status == 0 and good[0].tolist() == [4, 1, 4, 0, 2] and good[3].tolist() == [-1, 0, -1]
    if what == "pages":
        nip, code = np.array([0, 2, 5, 8]), -7
    elif what == "parent":
        parent = np.array([0, 2, 1])
    elif what == "shrink":
        nip = np.array([0, 1, 3, 4])
    elif what == "entries":
        ip = np.array([0, 2, 9])
    elif what == "tail":
        ids = np.array([4, 6, 2])
    else:
        last = np.array([17, 16])
    got, status = fork(parent, ip, last, ids, nip, refs, 16)
    assert status == code
    assert np.all(got[0] == -1) and np.array_equal(got[1], refs) and np.all(got[2] == -1) and np.all(got[3] == -1)


LOWEST = -2 ** 31


@pytest.mark.parametrize("ip,nip", [
    ([0, 2, 3], [0, LOWEST, 4, 5]), ([0, 2, 3], [1, LOWEST, 4, 5]), ([0, 2, 3], [3, 1, 4, 5]), ([0, 2, 3], [0, 6, 4, 5]),
    ([1, LOWEST, 3], [0, 2, 4, 5]), ([3, 1, 3], [0, 2, 4, 5]), ([-1, 2, 3], [0, 2, 4, 5]),
])
def test_torn_tables_change_nothing(cuda_device, ip, nip):
    last, ids, refs = np.array([3, 16]), np.array([4, 1, 2]), np.array([0, 1, 1, 0, 1, 0])
    got, status = fork(np.array([0, 0, 1]), np.array(ip), last, ids, np.array(nip), refs, 16)
    assert status == -6
    assert np.all(got[0] == -1) and np.array_equal(got[1], refs) and np.all(got[2] == -1) and np.all(got[3] == -1)


@pytest.mark.parametrize("batch", [3, 1500])
@pytest.mark.parametrize("at,bad", [(1, LOWEST), (1, 3), (1, -1), (0, 2), (0, -2), (2, 0), (2, 4), (2, 2 ** 31 - 1)])
def test_a_torn_table_of_a_request_that_ends_changes_nothing(cuda_device, batch, at, bad):
    """Nobody's parent has the torn range: it lies outside the entries, or falls."""
    n = batch - 3   # requests of no pages before the three that the ranges are of
    ip, last = np.concatenate([np.zeros(n), [0, 1, 2, 3]]), np.concatenate([np.zeros(n), [3, 16, 7]])
    ids, refs = np.array([4, 1, 2]), np.array([0, 1, 1, 0, 1, 0])
    going_on = {0: 2, 1: 2, 2: 0}[at]   # its range does not touch the torn entry
    parent, nip = np.array([n + going_on]), np.array([0, 1])
    good, status = fork(parent, ip, last, ids, nip, refs, 16)
    assert status == 0 and good[1].sum() == 1
    ip = ip.copy()
    ip[n + at] = bad
    got, status = fork(parent, ip, last, ids, nip, refs, 16)
    assert status == -6
    assert np.all(got[0] == -1) and np.array_equal(got[1], refs) and np.all(got[2] == -1) and np.all(got[3] == -1)


def compact_reference(refs, ids, limit):
    live = np.flatnonzero(refs > 0)
    limit = limit or len(live)
    move, slot = live[live >= limit], np.flatnonzero(refs[:limit] <= 0)[: np.count_nonzero(live >= limit)]
    to = np.arange(len(refs))
    to[move] = slot
    out = refs.copy()
    out[slot] = refs[move]
    out[move] = 0
    return to[ids], out, move, slot


@pytest.mark.parametrize("num_pages", [1, 2, 33, 1023, 1024, 1025, 5000, 200000])
@pytest.mark.parametrize("density", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact_matches_the_definition(cuda_device, num_pages, density):
    rng = np.random.RandomState(num_pages + int(100 * density))
    refs = (rng.rand(num_pages) < density).astype(np.int32) * rng.randint(1, 4, num_pages).astype(np.int32)
    live = np.flatnonzero(refs)
    ids = rng.permutation(np.repeat(live, refs[live])) if len(live) else np.zeros(0, int)
    for limit in {0, len(live), min(num_pages, len(live) + num_pages // 5), num_pages}:
        want_ids, want_refs, move, slot = compact_reference(refs, ids, limit)
        most = min(len(live), num_pages - len(live))
        for inplace in (False, True):
            r, i = dev(refs, ids)
            ws = torch.zeros(fd.pages_workspace_bytes(num_pages), dtype=torch.uint8, device="cuda")
            kw = dict(new_page_indices=i, new_page_refs=r) if inplace else {}
            got = [x.cpu().numpy() for x in fd.compact_pages(r, i, most, limit=limit, workspace=ws, **kw)]
            assert fd.get_device_status(ws) == 0
            assert np.array_equal(got[0], want_ids) and np.array_equal(got[1], want_refs)
            pad = np.full(most - len(move), -1)
            assert np.array_equal(got[2], np.concatenate([move, pad])) and np.array_equal(got[3], np.concatenate([slot, pad]))


def test_a_refused_compaction_changes_nothing(cuda_device):
    refs, ids = np.array([0, 1, 2, 0, 1, 1]), np.array([5, 2, 1, 2, 4])
    for limit, most in ((2, 4), (0, 1)):   # too few free pages before the limit; too few moves allowed
        r, i = dev(refs, ids)
        ws = torch.zeros(fd.pages_workspace_bytes(6), dtype=torch.uint8, device="cuda")
        got = [x.cpu().numpy() for x in fd.compact_pages(r, i, most, limit=limit, workspace=ws)]
        assert fd.get_device_status(ws) == -7
        assert np.array_equal(got[0], ids) and np.array_equal(got[1], refs) and np.all(got[2] == -1) and np.all(got[3] == -1)


@pytest.mark.parametrize("page_bytes", [16, 64, 8192, 16384, 16400, 50000 // 16 * 16])
@pytest.mark.parametrize("num_pools", [1, 5, 131])
def test_copies_move_whole_pages_only(cuda_device, page_bytes, num_pools):
    rng, pages = np.random.RandomState(page_bytes + num_pools), 37
    pools = [torch.randint(0, 256, (pages, page_bytes >> (j % 2 if page_bytes % 32 == 0 else 0)), dtype=torch.uint8, device="cuda")
             for j in range(num_pools)]
    perm = rng.permutation(pages)
    src, dst = perm[:18].copy(), perm[18:36].copy()
    src[1] = src[0]          # one page to two places
    src[5] = -1
    before = [x.clone() for x in pools]
    s, d = dev(src, dst)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fd.copy_pages(pools, s, d, workspace=ws)
    assert fd.get_device_status(ws) == 0
    keep = src >= 0
    for x, b in zip(pools, before):
        b[d[torch.from_numpy(keep)].long()] = b[s[torch.from_numpy(keep)].long()]
        assert torch.equal(x, b)


def test_copies_outside_the_pool_are_skipped(cuda_device):
    x = torch.arange(6 * 16, dtype=torch.uint8, device="cuda").view(6, 16)
    before = x.clone()
    for bad in ((6, 0), (0, 6), (0, -1)):
        s, d = dev([bad[0], 1], [bad[1], 2])
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        fd.copy_pages([x], s, d, workspace=ws)
        assert fd.get_device_status(ws) == -6
        fd.copy_pages([x], s, d)   # without a workspace: skipped all the same
    before[2] = before[1]
    assert torch.equal(x, before)


def test_captured_fork_and_copy_follow_their_tables(cuda_device):
    rng, page, pages = np.random.RandomState(9), 16, 200
    draws = []
    for _ in range(3):
        ip, last, ids, refs = random_tables(rng, 6, page, pages, 8)
        parent = rng.randint(-1, 6, 11)
        nip = indptr(np.where(parent < 0, 1, (ip[1:] - ip[:-1])[np.maximum(parent, 0)] + 1))
        draws.append((parent, ip, last, ids, nip, refs))
    pad = lambda x, n: np.concatenate([x, np.zeros(n - len(x), int)])  # noqa: E731
    t = dev(*draws[0][:3], pad(draws[0][3], 100), draws[0][4], draws[0][5])
    ws = torch.zeros(fd.pages_workspace_bytes(pages, 11), dtype=torch.uint8, device="cuda")
    pool = torch.randint(0, 256, (pages, 512), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fd.fork_pages(*t[:5], 200, page, t[5], workspace=ws)
        fd.copy_pages([pool], out[2], out[3], workspace=ws)
    for d in draws:
        for x, y in zip(t, dev(*d[:3], pad(d[3], 100), *d[4:])):
            x.copy_(y)
        b = pool.clone()
        g.replay()
        want = fork_reference(*d[:6], page)
        n = len(want[0])
        assert fd.get_device_status(ws) == 0
        assert np.array_equal(out[0][:n].cpu().numpy(), want[0]) and np.array_equal(out[1].cpu().numpy(), want[1])
        ok = want[2] >= 0
        b[want[3][ok]] = b[want[2][ok]]
        assert torch.equal(pool, b)


@pytest.mark.parametrize("batch,children", [(0, 0), (4, 0), (0, 3), (5, 12)])
@pytest.mark.parametrize("head,tail", [(0, 1), (0, 700), (3, 2000), (300, 0)])
def test_entries_that_no_table_has_become_none(cuda_device, batch, children, head, tail):
    """A list with room in front of its tables and behind them; the compaction of
    the whole list renames the tables' pages and reports nothing."""
    rng, pages, page = np.random.RandomState(batch + tail), 400, 16
    ip, last, ids, refs = random_tables(rng, batch, page, pages, 8)
    parent = rng.randint(-1, batch, children) if batch else np.full(children, -1)
    grow = np.where(parent < 0, 0, (ip[1:] - ip[:-1])[np.maximum(parent, 0)] if batch else 0) + 1
    nip = indptr(grow)
    want = fork_reference(parent, ip, last, ids, nip, refs, page)
    t = dev(parent, ip, last, ids, nip + head, refs)
    n = head + int(nip[-1]) + tail
    out = dev(np.full(n, 12345))[0]
    ws = torch.zeros(fd.pages_workspace_bytes(pages, children), dtype=torch.uint8, device="cuda")
    got = fd.fork_pages(*t[:5], n, page, t[5], new_page_indices=out, workspace=ws)
    assert fd.get_device_status(ws) == 0
    whole = np.concatenate([np.full(head, -1), want[0], np.full(tail, -1)])
    for g, w in zip(got, (whole, *want[1:])):
        assert np.array_equal(g.cpu().numpy(), w)
    live = np.flatnonzero(want[1] > 0)
    to, refs2, move, slot = compact_reference(want[1], np.arange(pages), 0)
    most = min(len(live), pages - len(live))
    for inplace in (False, True):
        kw = dict(new_page_indices=got[0].clone()) if not inplace else dict(new_page_indices=got[0])
        moved = fd.compact_pages(got[1], got[0], most, workspace=ws, **kw)
        assert fd.get_device_status(ws) == 0
        assert np.array_equal(moved[0].cpu().numpy(), np.where(whole < 0, -1, to[whole]))
        assert np.array_equal(moved[1].cpu().numpy(), refs2)


def test_compaction_reports_other_ids_outside_the_pool(cuda_device):
    refs = np.array([0, 1, 1])
    for bad in (-2, 3, LOWEST):
        r, i = dev(refs, [2, -1, bad, 1])
        ws = torch.zeros(fd.pages_workspace_bytes(3), dtype=torch.uint8, device="cuda")
        got = fd.compact_pages(r, i, 1, workspace=ws)
        assert fd.get_device_status(ws) == -6
        assert got[0].tolist() == [0, -1, bad, 1]


def test_forks_of_many_requests_from_several_threads(cuda_device):
    """Tables too large for the shared memory that a launch has by default, of
    different sizes at once: no call takes the room of another."""
    rounds, errors = 5000, []
    start = threading.Barrier(4)

    def run(batch):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                t = dev([batch - 1], np.zeros(batch + 1), np.zeros(batch), np.zeros(1), [0, 1], np.zeros(64))
                ws = torch.zeros(fd.pages_workspace_bytes(64, 1), dtype=torch.uint8, device="cuda")
                out = fd.fork_pages(*t[:5], 1, 16, t[5], workspace=ws)
                kw = dict(zip(("new_page_indices", "new_page_refs", "copy_src", "copy_dst"), out))
                start.wait()
                for _ in range(rounds):
                    fd.fork_pages(*t[:5], 1, 16, t[5], workspace=ws, **kw)
                assert fd.get_device_status(ws, s) == 0 and out[0].tolist() == [0]
        except Exception as e:   # to the test's thread
            errors.append((batch, e))
            start.abort()

    threads = [threading.Thread(target=run, args=(b,)) for b in (10300, 32768, 12000, 30000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
