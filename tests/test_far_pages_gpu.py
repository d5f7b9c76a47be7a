"""The serving operators over page pools of more than 2^32 bytes: what they do
to pages at the far end is, bit for bit, what they do to the same pages of a
small pool; and over many prefixes and two streams at once."""
import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd

pytestmark = pytest.mark.gpu
D, HQ, HKV, PAGE, B = 128, 32, 8, 16, 6
FAR = (2 ** 32 + 2 ** 27) // (PAGE * HKV * D * 2)   # pages of bf16 that 32-bit byte offsets do not reach


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def indptr(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_far_pages(cuda_device, kv):
    """A prefix and the requests' own pages, appended, attended and copied."""
    own, pre = np.array([3, 20, 16, 1, 40, 33]), 300
    oc, pc = -(-own // PAGE), -(-pre // PAGE)
    n = int(oc.sum()) + pc
    pages = FAR * (1 if kv == "bf16" else 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(pre + int(own.sum()), HQ + 2 * HKV, D, device="cuda", generator=g).to(torch.bfloat16)
    rope = fd.plan_rope(D, D)
    one = torch.full((HKV,), 0.02, device="cuda")
    scales = () if kv == "bf16" else (one, one)
    append = fd.append_paged if kv == "bf16" else fd.append_paged_fp8
    decode = fd.decode_shared_paged if kv == "bf16" else fd.decode_shared_paged_fp8
    order = np.random.RandomState(1).permutation(n)
    plan = fd.plan_shared_paged(B, HQ, HKV, D, PAGE, [0, B], [0, pc], [pre - (pc - 1) * PAGE], int(own.sum()))
    got = []
    for total in (n, pages):
        pools = [torch.empty((total, PAGE, HKV, D), dtype=torch.bfloat16 if kv == "bf16" else torch.uint8, device="cuda")
                 for _ in "kv"]
        ids = total - n + order
        pre_ids, own_ids = i32(ids[:pc]), i32(ids[pc:])
        pre_last, own_last = i32([pre - (pc - 1) * PAGE]), i32(own - (oc - 1) * PAGE)
        k, v = x[:, HQ: HQ + HKV], x[:, HQ + HKV:]
        ws = torch.zeros(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
        append(None, k[:pre], v[:pre], *pools, *scales, i32([0, pre]), i32([0, pc]), pre_last, pre_ids, rope=rope,
               workspace=ws)
        positions = i32(pre + np.concatenate([np.arange(m) for m in own]))
        q = append(x[pre:, :HQ], k[pre:], v[pre:], *pools, *scales, i32(indptr(own)), i32(indptr(oc)), own_last,
                   own_ids, rope=rope, positions=positions, workspace=ws)
        q = q[torch.from_numpy(np.cumsum(own) - 1).cuda()].contiguous()
        o, lse = decode(plan, q, *pools, *scales, i32([0, B]), i32([0, pc]), pre_last, pre_ids, i32(indptr(oc)),
                        own_last, own_ids, 0.088, workspace=ws)
        assert fd.get_device_status(ws) == 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()
        if total == pages:   # to the near end
            fd.copy_pages(pools, i32(ids), i32(np.arange(n)), workspace=ws)
            assert fd.get_device_status(ws) == 0
            far = torch.from_numpy(ids).cuda()
            for pool in pools:
                assert torch.equal(pool[:n].view(torch.uint8), pool[far].view(torch.uint8))
        rows = torch.from_numpy(ids[: pc - 1]).cuda()   # full pages
        got.append((q, o, lse, *[p[rows].view(torch.uint8) for p in pools]))
        del pools
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_many_prefixes(cuda_device):
    """Several hundred prefixes of a few requests each, some of no keys."""
    rng = np.random.RandomState(2)
    P = 333
    reqs, lens = rng.randint(0, 5, P), rng.randint(0, 200, P)
    reqs[-1] = 2
    n, T = int(reqs.sum()), int(lens.sum())
    q = torch.randn(n, 4, D, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn(T, 2, D, device="cuda").to(torch.bfloat16) for _ in "kv")
    plan = fd.plan_shared(n, 4, 2, D, indptr(reqs), indptr(lens), 0)
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    o, lse = fd.decode_shared(plan, q, k, v, None, None, i32(indptr(reqs)), i32(indptr(lens)), None, 0.088, workspace=ws)
    assert fd.get_device_status(ws) == 0
    at, ip = indptr(reqs), indptr(lens)
    for p in range(P):
        r = slice(at[p], at[p + 1])
        if reqs[p] == 0:
            continue
        if lens[p] == 0:
            assert torch.all(o[r] == 0) and torch.all(lse[r] == -float("inf"))
            continue
        K, V = (y[ip[p]: ip[p + 1]].double().repeat_interleave(2, 1) for y in (k, v))
        s = torch.einsum("bhd,lhd->bhl", q[r].double(), K) * 0.088
        ref = torch.einsum("bhl,lhd->bhd", s.softmax(-1), V)
        assert (o[r] - ref).abs().max() < 1e-4 and (lse[r] - s.logsumexp(-1)).abs().max() < 2e-5
        assert (o[r] - ref).norm() < 1e-5 * ref.norm()


def test_two_calls_at_once(cuda_device):
    """Two streams with a workspace each, forks and prefixes at once, many times."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    plan = fd.plan_shared(40, 32, 8, D, [0, 30, 40], [0, 3000, 5000], 0)
    jobs = []
    for j in range(2):
        g = torch.Generator(device="cuda").manual_seed(j)
        q = torch.randn(40, 32, D, device="cuda", generator=g).to(torch.bfloat16)
        k, v = (torch.randn(5000, 8, D, device="cuda", generator=g).to(torch.bfloat16) for _ in "kv")
        refs = i32([1] * 600 + [0] * 3000)
        tables = (i32([0, 0, 1]), i32([0, 400, 600]), i32([5, 16]), i32(np.random.RandomState(j).permutation(600)),
                  i32([0, 400, 900, 1200]), 1200, PAGE, refs)
        jobs.append(((q, k, v, None, None, i32([0, 30, 40]), i32([0, 3000, 5000]), None, 0.088), tables,
                     torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda"),
                     torch.zeros(fd.pages_workspace_bytes(3600, 3), dtype=torch.uint8, device="cuda")))

    def run(j, stream=None):
        a, tables, ws, pw = jobs[j]
        return (*fd.decode_shared(plan, *a, workspace=ws, stream=stream),
                *fd.fork_pages(*tables, workspace=pw, stream=stream))
    alone = [run(0), run(1)]
    torch.cuda.synchronize()
    both = [[run(j, streams[j]) for j in range(2)] for _ in range(20)]
    torch.cuda.synchronize()
    for j in range(2):
        assert fd.get_device_status(jobs[j][2]) == 0 and fd.get_device_status(jobs[j][3]) == 0
        for outs in both:
            assert all(torch.equal(x, y) for x, y in zip(outs[j], alone[j]))
