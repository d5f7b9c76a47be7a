"""A NaN among one split's keys reaches the whole request's O and LSE, whichever
warp merges that split, and no other request."""
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq", [4, 16, 32])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("key", [0, 131, 1999])
def test_nan_of_one_split_reaches_the_output(cuda_device, kv, hq, key):
    lengths, hkv = [2000, 300], 4
    ip = torch.tensor([0, 2000, 2300], dtype=torch.int32)
    torch.manual_seed(key + hq)
    q = torch.randn((2, hq, 128), device=cuda_device).to(torch.bfloat16)
    k, v = (torch.randn((sum(lengths), hkv, 128), device=cuda_device).to(torch.bfloat16) for _ in range(2))
    if kv == "fp8":
        k, v = (x.to(torch.float8_e4m3fn) for x in (k, v))
        one = torch.ones(hkv, device=cuda_device)

    def run():
        if kv == "fp8":
            return fd.decode_fp8(q, k, v, one, one, ip, ip.to(cuda_device), 0.09)
        return fd.decode(q, k, v, ip, ip.to(cuda_device), 0.09)
    want = run()
    if kv == "fp8":
        k.view(torch.uint8)[key, 1, 5] = 0x7F
    else:
        k[key, 1, 5] = float("nan")
    o, lse = run()
    g = hq // hkv
    bad = torch.zeros((2, hq), dtype=torch.bool, device=cuda_device)
    bad[0, g: 2 * g] = True
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.isnan(o[bad]).all() and torch.equal(o[~bad], want[0][~bad]) and torch.equal(lse[~bad], want[1][~bad])


@pytest.mark.parametrize("others", [[], [float("-inf")], [0.25], [float("-inf"), 0.25, -3.0]])
@pytest.mark.parametrize("at", [0, -1])
def test_nan_state_reaches_the_merged_row(cuda_device, others, at):
    """A row with a NaN among its states' LSEs is NaN in O and LSE, whatever the others;
    the rows beside it are not, empty ones O = 0, LSE = -inf."""
    lse = torch.tensor(others, device=cuda_device).repeat(3, 1).T.contiguous().reshape(len(others), 3)
    nan = torch.tensor([[float("-inf"), float("nan"), 1.5]], device=cuda_device)
    lse = torch.cat([nan, lse] if at == 0 else [lse, nan])
    torch.manual_seed(1)
    o = torch.randn((*lse.shape, 128), device=cuda_device)
    o[lse == float("-inf")] = 0.0
    got, got_lse = fd.merge_states(o, lse)
    assert got[1].isnan().all() and bool(got_lse[1].isnan())
    w = torch.exp(lse.double()).nan_to_num(0.0)
    for r in (0, 2):
        d = w[:, r].sum()
        want = (w[:, r, None] * o[:, r].double()).sum(0) / d if float(d) else torch.zeros(128, device=cuda_device).double()
        assert float((got[r].double() - want).abs().max()) <= 1e-6 * float(o.abs().max())
        if float(d) == 0:
            assert float(got_lse[r]) == float("-inf")
        else:
            assert abs(float(got_lse[r]) - float(d.log())) <= 1e-5
    # a further merge does not lose it
    again, again_lse = fd.merge_states(torch.stack([got, torch.zeros_like(got)]),
                                       torch.stack([got_lse, torch.full_like(got_lse, float("-inf"))]))
    assert again[1].isnan().all() and bool(again_lse[1].isnan())


def test_nan_key_of_a_shard_reaches_the_merged_output(cuda_device):
    """Decode of two shards, a NaN in the only one that has the second request's keys."""
    torch.manual_seed(3)
    q = torch.randn((2, 8, 128), device=cuda_device).to(torch.bfloat16)
    states = []
    for lengths in ([700, 300], [500, 0]):
        ip = torch.tensor([0, lengths[0], sum(lengths)], dtype=torch.int32)
        k, v = (torch.randn((sum(lengths), 2, 128), device=cuda_device).to(torch.bfloat16) for _ in range(2))
        if lengths[1]:
            k[lengths[0] + 5, 1, 7] = float("nan")
        states.append(fd.decode(q, k, v, ip, ip.to(cuda_device), 0.09))
    o, lse = fd.merge_states(torch.stack([s[0] for s in states]), torch.stack([s[1] for s in states]))
    bad = torch.zeros((2, 8), dtype=torch.bool, device=cuda_device)
    bad[1, 4:] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
