"""An INT8 cache as a server uses it: a prompt is appended in two chunks that attend
causally, forks into samples with copies of partly filled pages and their scales,
each step appends one token (decode) or three drafted ones (a check of them in one
pass), samples end, the cache is compacted, and a second sequence's queries attend
an encoder's states in the same pool.  One workspace for the page operators and the
attention's plans; decode keeps its own, laid out by its batch."""
import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd
from tests.int8_util import D, attention, indptr
from tests.parity_util import assert_within, errors
from tests.test_int8_gpu import TIGHT
from tests.test_prefill_gpu import compare

pytestmark = pytest.mark.gpu
HQ, HKV, P, PAGES, SCALE = 8, 2, 16, 80, D ** -0.5


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("hkv", [2, 5])
def test_int8_cache_through_prompts_forks_steps_and_compaction(cuda_device, hkv):
    hq = 4 * hkv
    gen = torch.Generator().manual_seed(hkv)
    # values that grow along the sequence, so that pages' scales do, too
    count = [0]

    def rand(n, h):
        count[0] += n
        return (torch.randn((n, h, D), generator=gen) * (0.5 + count[0] / 300)).to(torch.bfloat16).cuda()
    c = {x: torch.randint(-128, 128, (PAGES, P, hkv, D), dtype=torch.int8, device="cuda") for x in "kv"}
    for x in "kv":
        c[x + "s"] = torch.full((PAGES, fd.scale_heads(hkv)), float("nan"), device="cuda")
    pools = [c["k"], c["v"], c["ks"], c["vs"]]
    rope = fd.plan_rope(D, 64, interleaved=True, base=500000.0)
    ws = torch.zeros(max(fd.pages_workspace_bytes(PAGES, 16), 1 << 21), dtype=torch.uint8, device="cuda")
    refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")

    def fork(refs, parent, own, ids, nxt):
        cnt = -(-own // P)
        ids, refs, src, dst = fd.fork_pages(i32(parent), i32(indptr(cnt)), i32(own - (cnt - 1) * P), ids, i32(indptr(nxt)),
                                            int(np.sum(nxt)), P, refs, workspace=ws)
        fd.copy_pages(pools, src, dst, workspace=ws)
        return ids, refs

    def tables(own, ids):
        cnt = -(-own // P)
        return dict(keys=own, page=P, num_pages=PAGES, ip=indptr(cnt), last=(own - (cnt - 1) * P).astype(np.int32),
                    ids=ids.cpu().numpy())

    def append(new, own, ids, k, v, q):
        t = tables(own, ids)
        return fd.append_paged_int8(q, k, v, *pools, i32(indptr(new)), i32(t["ip"]), i32(t["last"]), ids, rope=rope,
                                    workspace=ws)

    def attend(q, new, own, ids, causal=True):
        t, qi = tables(own, ids), indptr(new)
        plan = fd.plan_prefill_paged(len(own), q.shape[1], hkv, D, P, qi, t["ip"], t["last"], causal=causal)
        got = fd.prefill_paged_int8(plan, q, *pools, i32(qi), i32(t["ip"]), i32(t["last"]), ids, SCALE, workspace=ws)
        assert fd.get_device_status(ws) == 0
        used = dict(c, ks=c["ks"].nan_to_num(0.0), vs=c["vs"].nan_to_num(0.0))   # (pages of nobody: NaN)
        compare(got, t, used, q, qi, causal)
        return got

    # the prompt, in two chunks
    own, ids, values = np.zeros(1, int), i32([]), [torch.zeros((0, hkv, D))]
    for n in (70, 61):
        nxt = -(-(own + n) // P)
        if own[0] == 0:
            ids, refs = fork(refs, np.array([-1]), np.zeros(0, int), i32([]), nxt)
        else:
            ids, refs = fork(refs, np.zeros(1, int), own, ids, nxt)
        own = own + n
        k, v = rand(n, hkv), rand(n, hkv)
        q = append([n], own, ids, k, v, rand(n, hq))
        attend(q, [n], own, ids)
        values = [torch.cat([values[0], v.cpu().float()])]
    # an encoder's states: one more request's pages, attended as a whole
    encoder = fork(refs, np.array([0, -1]), own, ids, np.array([-(-own[0] // P), 3]))
    ids, refs = encoder
    both = np.array([own[0], 40])
    append([0, 40], both, ids, rand(40, hkv), rand(40, hkv), rand(40, hq))
    attend(rand(9, hq), [2, 7], both, ids, causal=False)
    ids, refs = fork(refs, np.array([0]), both, ids, -(-own // P))   # the encoder's pages go back
    # samples
    samples = 4
    ids, refs = fork(refs, np.zeros(samples, int), own, ids, np.repeat(-(-own // P), samples))
    own, values = np.repeat(own, samples), values * samples
    for step in range(14):
        n = len(own)
        if step == 7:   # a sample ends, one forks once more; then the cache is compacted
            parent = np.array([0, 2, 2, 3])
            ids, refs = fork(refs, parent, own, ids, (-(-own // P))[parent])
            own, values = own[parent], [values[p] for p in parent]
            ids, refs, src, dst = fd.compact_pages(refs, ids, PAGES // 2, workspace=ws)
            fd.copy_pages(pools, src, dst, workspace=ws)
            assert int(refs.nonzero().max()) == int((refs > 0).sum()) - 1
        new = 3 if step % 4 == 2 else 1
        ids, refs = fork(refs, np.arange(n), own, ids, -(-(own + new) // P))
        own = own + new
        k, v = rand(n * new, hkv), rand(n * new, hkv)
        q = append([new] * n, own, ids, k, v, rand(n * new, hq))
        values = [torch.cat([values[b], v[b * new: (b + 1) * new].cpu().float()]) for b in range(n)]
        t = tables(own, ids)
        if new > 1:
            attend(q, [new] * n, own, ids)
        else:
            o, lse = fd.decode_paged_int8(q, *pools, t["ip"], t["last"], i32(t["ip"]), i32(t["last"]), ids, SCALE)
            want = attention(q, t, c, SCALE)
            assert_within(errors(o.cpu().numpy(), lse.cpu().numpy(), want[0].cpu().numpy(), want[1].cpu().numpy()),
                          **TIGHT, what=f"step {step}")
        assert fd.get_device_status(ws) == 0
    # the values are those that were put in, to half a step for each time they were rounded
    for b in range(len(own)):
        at = torch.from_numpy(t["ids"][t["ip"][b]: t["ip"][b + 1]].astype(np.int64)).cuda()
        s = c["vs"][at][:, :hkv].double()
        got = (c["v"][at].double() * s[:, None, :, None]).reshape(-1, hkv, D)[: own[b]].cpu()
        s = s[:, None].expand(-1, P, -1).reshape(-1, hkv)[: own[b], :, None].cpu()
        off = (got - values[b].double()).abs() / s
        assert float(off.max()) <= 0.5 * P
        assert float(off.mean()) <= 1.0
