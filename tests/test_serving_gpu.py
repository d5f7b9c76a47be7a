"""A serving loop's cache operators together: a prompt is appended, forks into
several samples, each step appends a token and attends over the shared prompt and
the sample's own keys, samples end, and the cache is compacted."""
import numpy as np
import pytest
import torch

import oracle
import split_kv_flashdecoding_gb300 as fd
from tests.parity_util import assert_within, errors

pytestmark = pytest.mark.gpu
D, HQ, HKV, P, PAGES = 128, 8, 2, 16, 96
SCALE = float(np.float32(1 / np.sqrt(128)))
TIGHT = dict(max_abs=1e-4, rel_l2=1e-5, lse_abs=2e-5)


def indptr(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Cache:
    """What a program keeps: pools, the device's page ids and counts, and the
    host's lengths; `values` holds every sample's V rows as they were put in."""

    def __init__(self, fp8):
        self.fp8 = fp8
        dt = torch.uint8 if fp8 else torch.bfloat16
        self.pools = [torch.zeros((PAGES, P, HKV, D), dtype=dt, device="cuda") for _ in "kv"]
        self.scale = torch.tensor([0.02, 0.03], device="cuda") if fp8 else None
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.rope = fd.plan_rope(D, 64, interleaved=True, base=500000.0, scaling=("yarn", 4.0, 4096, 1.0, 32.0))
        self.ws = torch.zeros(fd.pages_workspace_bytes(PAGES, 16), dtype=torch.uint8, device="cuda")

    def append(self, q, k, v, new, ip, last, ids, positions):
        args = (i32(indptr(new)), i32(ip), i32(last), ids)
        kw = dict(rope=self.rope, positions=i32(positions), workspace=self.ws)
        if self.fp8:
            return fd.append_paged_fp8(q, k, v, *self.pools, self.scale, self.scale, *args, **kw)
        return fd.append_paged(q, k, v, *self.pools, *args, **kw)

    def fork(self, parent, ip, last, ids, nip):
        ids, self.refs, src, dst = fd.fork_pages(i32(parent), i32(ip), i32(last), ids, i32(nip), int(nip[-1]), P,
                                                 self.refs, workspace=self.ws)
        fd.copy_pages(self.pools, src, dst, workspace=self.ws)
        return ids

    def rows(self, ids, n):
        """K and V rows of a list of n keys, as fp64 numpy."""
        ids = ids.cpu().numpy()
        at = torch.from_numpy(np.concatenate([np.arange(P) + i * P for i in ids] + [np.zeros(0, int)])[:n].astype(np.int64)).cuda()
        out = []
        for pool in self.pools:
            x = pool.view(-1, HKV, D)[at]
            out.append(x.view(torch.float8_e4m3fn).double().cpu().numpy() * self.scale.double().cpu().numpy()[:, None]
                       if self.fp8 else x.double().cpu().numpy())
        return out


def attend(q, K, V):
    g = HQ // HKV
    s = np.einsum("hd,lhd->hl", q, np.repeat(K, g, 1)) * SCALE
    m = s.max(1, keepdims=True)
    w = np.exp(s - m)
    return np.einsum("hl,lhd->hd", w / w.sum(1, keepdims=True), np.repeat(V, g, 1)), m[:, 0] + np.log(w.sum(1))


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_fork_steps_and_compaction(cuda_device, fp8):
    rng = torch.Generator().manual_seed(5)
    rand = lambda n, h: torch.randn((n, h, D), generator=rng).to(torch.bfloat16).cuda()  # noqa: E731
    c, L = Cache(fp8), 150
    # the prompt: 9 full pages, which all samples share, and a partly filled one
    ids = c.fork([-1], [0], [], torch.zeros(1, dtype=torch.int32, device="cuda"), indptr([-(-L // P)]))
    k, v = rand(L, HKV), rand(L, HKV)
    c.append(rand(L, HQ), k, v, [L], [0, 10], [L - 9 * P], ids, np.arange(L))
    pre_ids, ids = ids[:9].clone(), ids[9:].clone()
    prefix, values = 9 * P, [v.cpu()]
    # five samples: the first keeps the last page, the others get copies of it
    own = np.full(5, L - prefix)
    ids = c.fork(np.zeros(5), [0, 1], [own[0]], ids, indptr([1] * 5))
    values = [v.cpu() for _ in range(5)]
    n = 5
    for step in range(24):
        if step == 12:   # two samples end, one forks once more; then the cache is compacted
            cnt, parent = -(-own // P), np.array([0, 2, 2, 4])
            last = own - (cnt - 1) * P
            ids = c.fork(parent, indptr(cnt), last, ids, indptr(cnt[parent]))
            own, values, n = own[parent], [values[p].clone() for p in parent], 4
            tables = torch.cat([pre_ids, ids])
            moved, c.refs, src, dst = fd.compact_pages(c.refs, tables, PAGES // 2, workspace=c.ws)
            fd.copy_pages(c.pools, src, dst, workspace=c.ws)
            pre_ids, ids = moved[:9].clone(), moved[9:].clone()
            live = int((c.refs > 0).sum())
            assert int(c.refs.nonzero().max()) == live - 1
        # a page for those whose last one is full, then the step's tokens
        cnt = -(-own // P)
        nxt = -(-(own + 1) // P)
        if (nxt > cnt).any():
            ids = c.fork(np.arange(n), indptr(cnt), own - (cnt - 1) * P, ids, indptr(nxt))
        own = own + 1
        ip, last = indptr(nxt), own - (nxt - 1) * P
        k, v, q = rand(n, HKV), rand(n, HKV), rand(n, HQ)
        q = c.append(q, k, v, np.ones(n, int), ip, last, ids, prefix + own - 1)
        values = [torch.cat([values[b], v[b: b + 1].cpu()]) for b in range(n)]
        plan = fd.plan_shared_paged(n, HQ, HKV, D, P, [0, n], [0, 9], [P], 256)
        ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        args = (i32([0, n]), i32([0, 9]), i32([P]), pre_ids, i32(ip), i32(last), ids, SCALE)
        if fp8:
            o, lse = fd.decode_shared_paged_fp8(plan, q, *c.pools, c.scale, c.scale, *args, workspace=ws)
        else:
            o, lse = fd.decode_shared_paged(plan, q, *c.pools, *args, workspace=ws)
        assert fd.get_device_status(ws) == 0 and fd.get_device_status(c.ws) == 0
        for b in range(n):
            K, V = c.rows(torch.cat([pre_ids, ids[ip[b]: ip[b + 1]]]), prefix + int(own[b]))
            # every sample's list holds the values that were put in, in order
            want = values[b].double().numpy()
            tol = np.maximum(2.0 ** -4 * np.abs(want), 0.03 * 2.0 ** -10) * 1.001 if fp8 else 0
            assert np.all(np.abs(V - want) <= tol)
            ref = attend(q[b].double().cpu().numpy(), K, V)
            assert_within(errors(o[b].cpu().numpy(), lse[b].cpu().numpy(), *ref), **TIGHT, what=f"step {step} sample {b}")
        # the same through decode_paged, each sample with its whole list
        if not fp8:
            tables = [torch.cat([pre_ids, ids[ip[b]: ip[b + 1]]]) for b in range(n)]
            whole = indptr([len(t) for t in tables])
            o2, lse2 = fd.decode_paged(q, *c.pools, whole, last.astype(np.int32), i32(whole), i32(last), torch.cat(tables), SCALE)
            assert (o - o2).abs().max() < 2e-5 and (lse - lse2).abs().max() < 2e-5


def test_int4_cache_through_append_forks_copies_and_compaction(cuda_device):
    """The same loop over an INT4 cache, whose scales are pools of their own: prompt,
    forks with copies of codes and scales, steps through decode_paged_int4 over each
    sample's whole list, ends and a compaction."""
    gen = torch.Generator().manual_seed(11)
    rand = lambda n, h: torch.randn((n, h, D), generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    L, pages = 150, 64
    codes = [torch.zeros((pages, P, HKV, D // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.full((HKV, pages * P), float("nan"), device="cuda") for _ in "kv"]
    pools = [*codes, *(x for sc in scales for x in sc.view(HKV, pages, P))]
    rope = fd.plan_rope(D, D, base=500000.0)
    ws = torch.zeros(fd.pages_workspace_bytes(pages, 16), dtype=torch.uint8, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")

    def fork(refs, parent, own, ids, nxt):
        cnt = -(-own // P)
        ids, refs, src, dst = fd.fork_pages(i32(parent), i32(indptr(cnt)), i32(own - (cnt - 1) * P), ids, i32(indptr(nxt)),
                                            int(np.sum(nxt)), P, refs, workspace=ws)
        fd.copy_pages(pools, src, dst, workspace=ws)
        return ids, refs

    def append(new, own, ids, k, v, q):
        cnt = -(-own // P)
        return fd.append_paged_int4(q, k, v, *codes, *scales, i32(indptr(new)), i32(indptr(cnt)), i32(own - (cnt - 1) * P),
                                    ids, rope=rope, workspace=ws)

    def rows(ids, n):
        at = np.concatenate([np.arange(P) + i * P for i in ids.cpu().numpy()])[:n]
        return [oracle.int4_codes(c.view(-1, HKV, D // 2)[at]) * sc[:, at].T.double().cpu().numpy()[..., None]
                for c, sc in zip(codes, scales)], scales[1][:, at].T.double().cpu().numpy()

    ids, refs = fork(refs, np.array([-1]), np.zeros(0, int), i32([]), np.array([-(-L // P)]))
    k, v = rand(L, HKV), rand(L, HKV)
    append([L], np.array([L]), ids, k, v, rand(L, HQ))
    own, values = np.full(5, L), [v.cpu()] * 5
    cnt = -(-own // P)
    ids, refs = fork(refs, np.zeros(5, int), np.array([L]), ids, cnt)
    for step in range(24):
        n = len(own)
        if step == 12:   # two samples end, one forks once more; then the cache is compacted
            parent = np.array([0, 2, 2, 4])
            ids, refs = fork(refs, parent, own, ids, (-(-own // P))[parent])
            own, values, n = own[parent], [values[p] for p in parent], 4
            ids, refs, src, dst = fd.compact_pages(refs, ids, pages // 2, workspace=ws)
            fd.copy_pages(pools, src, dst, workspace=ws)
            assert int(refs.nonzero().max()) == int((refs > 0).sum()) - 1
        nxt = -(-(own + 1) // P)
        if (nxt > -(-own // P)).any():
            ids, refs = fork(refs, np.arange(n), own, ids, nxt)
        own = own + 1
        k, v = rand(n, HKV), rand(n, HKV)
        q = append(np.ones(n, int), own, ids, k, v, rand(n, HQ))
        values = [torch.cat([values[b], v[b: b + 1].cpu()]) for b in range(n)]
        ip, last = indptr(nxt), (own - (nxt - 1) * P).astype(np.int32)
        o, lse = fd.decode_paged_int4(q, *codes, *scales, ip, last, i32(ip), i32(last), ids, SCALE)
        assert fd.get_device_status(ws) == 0
        for b in range(n):
            (K, V), sv = rows(ids[ip[b]: ip[b + 1]], int(own[b]))
            # half a code, and the scale's and the quotient's roundings (7 codes of 2^-24 each)
            want = values[b].double().numpy()
            assert np.all(np.abs(V - want) <= sv[..., None] * (0.5 + 2.0 ** -20))
            ref = attend(q[b].double().cpu().numpy(), K, V)
            assert_within(errors(o[b].cpu().numpy(), lse[b].cpu().numpy(), *ref), **TIGHT, what=f"step {step} sample {b}")


@pytest.mark.parametrize("big", [(64, 32, 8), (4200, 4, 4)], ids=str)
def test_one_workspace_for_plans_and_page_operators(cuda_device, big):
    """Zeroed once: a small plan, a fork and a compaction leave their partials and
    lists where they may; a larger plan's requests of several splits, before and
    behind them, are merged all the same."""
    def inputs(B, Hq, Hkv, own, seed):
        g = torch.Generator().manual_seed(seed)
        rand = lambda n, h: torch.randn((n, h, D), generator=g).to(torch.bfloat16)  # noqa: E731
        return dict(B=B, Hq=Hq, Hkv=Hkv, own=own, q=rand(B, Hq), kp=rand(130, Hkv), vp=rand(130, Hkv),
                    k=rand(int(own.sum()), Hkv), v=rand(int(own.sum()), Hkv))

    own = np.random.RandomState(1).randint(0, 4, big[0])
    own[::50] = 700
    own[big[0] // 2] = 3000
    cases = [inputs(2, 8, 8, np.array([300, 900]), 1), inputs(*big, own, 2)]
    pages = 5000
    plans = [fd.plan_shared(c["B"], c["Hq"], c["Hkv"], D, [0, c["B"]], [0, 130], int(c["own"].sum())) for c in cases]
    assert all((c["own"] > p.suffix.chunk).any() for c, p in zip(cases, plans))
    ws = torch.zeros(max(fd.pages_workspace_bytes(pages, 40), *(p.workspace_bytes for p in plans)), dtype=torch.uint8,
                     device="cuda")
    dev = [{n: c[n].cuda() for n in ("q", "kp", "vp", "k", "v")} for c in cases]

    def decode(j):
        d = dev[j]
        return fd.decode_shared(plans[j], d["q"], d["kp"], d["vp"], d["k"], d["v"], i32([0, cases[j]["B"]]),
                                i32([0, 130]), i32(indptr(cases[j]["own"])), SCALE, workspace=ws)

    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[::3] = 0
    outs = []
    for j in (0, 1, 0, "fork", 1, "compact", 0, 1, 1):
        if j == "fork":
            fd.fork_pages(i32(np.full(40, -1)), i32([0]), i32([]), i32([]), i32(np.arange(41)), 40, P, refs, workspace=ws)
        elif j == "compact":
            fd.compact_pages(refs, i32(np.flatnonzero(refs.cpu().numpy())), pages, workspace=ws)
        else:
            outs.append((j, decode(j)))
    assert fd.get_device_status(ws) == 0
    for j, c in enumerate(cases):
        K, V, at = [], [], indptr(c["own"])
        for b in range(c["B"]):
            K += [c["kp"], c["k"][at[b]: at[b + 1]]]
            V += [c["vp"], c["v"][at[b]: at[b + 1]]]
        o_ref, lse_ref = oracle.decode(c["q"], torch.cat(K), torch.cat(V), indptr(130 + c["own"]), SCALE)
        for _, (o, lse) in (x for x in outs if x[0] == j):
            assert_within(errors(o.cpu().numpy(), lse.cpu().numpy(), o_ref.reshape(o.shape), lse_ref.reshape(lse.shape)),
                          **TIGHT, what=f"case {j}")
