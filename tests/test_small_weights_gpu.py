"""Decode beside a key with nearly all of a row's weight and V = 0 (an attention sink): O is
the sum of the other keys' small weights, judged by its own norm, for every K/V type.

Weights are two parts of the MMA's type, 2^-16 (bf16) or 2^-22 (f16) of each or better, and
an f16 one's 2^-40 of the row's largest: 2^-17 of a weight of 2^-23.  The fp32 logits of up to
30 in log2 are off by 2^-19 or so, the large key's for all others at once.  5e-5 of the norm."""
import math

import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd
from tests.int8_util import D

pytestmark = pytest.mark.gpu
SCALE = D ** -0.5


def quantise(x, dims, top):
    s = x.abs().amax(dims, keepdim=True) / top
    s = torch.where(s == 0, 1.0, s)
    return (x / s).round().clamp(-8 if top == 7 else -127, top), s


def decode(kind, q, k, v, lens):
    """(O, LSE, K, V): what the kernel gives, and the keys and values it was given, fp64."""
    dev, hkv = q.device, k.shape[1]
    ip = torch.tensor([0, *np.cumsum(lens)], dtype=torch.int32)
    if kind == "bf16":
        k, v = k.bfloat16(), v.bfloat16()
        return *fd.decode(q, k, v, ip, ip.to(dev), SCALE), k.double(), v.double()
    if kind == "fp8":
        k, v, one = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.ones(hkv, device=dev)
        return *fd.decode_fp8(q, k, v, one, one, ip, ip.to(dev), SCALE), k.double(), v.double()
    if kind == "int4":
        (kc, ks), (vc, vs) = quantise(k, -1, 7), quantise(v, -1, 7)
        pack = lambda c: ((c.int()[..., 0::2] & 15) | ((c.int()[..., 1::2] & 15) << 4)).to(torch.uint8)  # noqa: E731
        o = fd.decode_int4(q, pack(kc), pack(vc), *(s[..., 0].T.contiguous() for s in (ks, vs)), ip, ip.to(dev), SCALE)
        return *o, kc.double() * ks.double(), vc.double() * vs.double()
    page = 64   # INT8: whole pages
    n = sum(lens) // page
    pages = [quantise(x.view(n, page, hkv, D), (1, 3), 127) for x in (k, v)]
    scales = []
    for _, s in pages:
        scales.append(torch.zeros((n, fd.scale_heads(hkv)), device=dev))
        scales[-1][:, :hkv] = s[:, 0, :, 0]
    pip = (ip // page).numpy().astype(np.int32)
    last = np.full(len(lens), page, dtype=np.int32)
    o = fd.decode_paged_int8(q, *(c.to(torch.int8) for c, _ in pages), *scales, pip, last, torch.from_numpy(pip).to(dev),
                             torch.from_numpy(last).to(dev), torch.arange(n, device=dev, dtype=torch.int32), SCALE)
    return *o, *((c.double() * s.double()).view(-1, hkv, D) for c, s in pages)


@pytest.mark.parametrize("share", [0.9, 0.99])
@pytest.mark.parametrize("lens", [[65536], [16384] * 6], ids=["one wave", "several"])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 4), (16, 4), (32, 4)])
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4", "int8"])
def test_decode_of_keys_beside_one_that_takes_nearly_all(cuda_device, kind, hq, hkv, lens, share):
    gen = torch.Generator(cuda_device).manual_seed(hq)
    starts = np.concatenate([[0], np.cumsum(lens)])
    k, v = (torch.randn((int(starts[-1]), hkv, D), generator=gen, device=cuda_device) for _ in range(2))
    # dimension 0 is the large key's alone; the others' logits have a deviation of about 1
    k[..., 0] = 0
    for s in starts[:-1]:
        k[s], v[s] = 0, 0
        k[s, :, 0] = 3
    q = torch.randn((len(lens), hq, D), generator=gen, device=cuda_device).bfloat16()
    q[..., 0] = (math.log(share / (1 - share)) + math.log(lens[0]) + 0.5) / (3 * SCALE)
    o, lse, kd, vd = decode(kind, q, k, v, lens)
    for b in range(len(lens)):
        at = slice(int(starts[b]), int(starts[b + 1]))
        s = torch.einsum("hgd,nhd->hgn", q[b].double().view(hkv, -1, D), kd[at]) * SCALE
        want = torch.einsum("hgn,nhd->hgd", torch.softmax(s, -1), vd[at]).reshape(hq, D)
        off = float(((o[b].double() - want).norm(dim=-1) / want.norm(dim=-1)).max())
        assert off <= 5e-5, off
        assert float((lse[b].double() - torch.logsumexp(s, -1).reshape(hq)).abs().max()) <= 2e-5
