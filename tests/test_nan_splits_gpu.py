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
