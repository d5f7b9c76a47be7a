"""fd_prefill_paged_int8 where f16's range of softmax weights ends, against attention in 64
bits."""
import math

import numpy as np
import pytest
import torch

from tests.int8_util import D, attention, cache, indptr, tables
from tests.test_prefill_gpu import plan_of, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", ["first", "behind"])
@pytest.mark.parametrize("tokens", [4, 150])
@pytest.mark.parametrize("share,keys", [(0.9, 65536), (0.97, 65536), (0.99, 30720), (0.99, 2000)])
def test_prefill_of_keys_beside_one_that_takes_nearly_all(cuda_device, share, keys, tokens, at):
    """A key with `share` of every row's weight and V = 0 (an attention sink): O is the sum of
    the other keys' small weights, and judged by its own norm.

    Half a step of bf16 a value, 2^-8 of the norm at most.  The others' weights are
    independent normal logits, their errors independent of the codes, so those errors add
    up as the weights' squares do: 2^-11 where f16's numbers are normal, and in the tiles
    beside the large key, before E follows (5 tiles of 128 keys and two streams at the
    most), weights of 2^-21.5 of it and 2 times that as stored, off by up to 2^-25 each:
    2^-4.5 over sqrt(3) of them, on a share of sqrt(1280 / 30720) of the norm: 0.5 %.  2^-8 +
    2^-7 covers all of it."""
    rng = np.random.RandomState(7)
    gen = torch.Generator(cuda_device).manual_seed(7)
    t = tables([keys], 64, rng)
    c = cache(t, 1, rng, cuda_device)
    where = 0 if at == "first" else keys // 2 - 5
    page, r = int(t["ids"][where // 64]), where % 64
    # dimension 0 is the large key's alone; the others' logits have a deviation of about 1
    scale, step = D ** -0.5, 1.0 / 38
    c["ks"][:, 0] = step
    c["k"].copy_((torch.randn(c["k"].shape, device=cuda_device, generator=gen) / step).round().clamp(-127, 127))
    c["k"][..., 0] = 0
    c["k"][page, r] = 0
    c["k"][page, r, 0, 0] = 127
    c["v"][page, r] = 0
    q = torch.randn((tokens, 4, D), device=cuda_device, generator=gen).to(torch.bfloat16)
    q[..., 0] = (math.log(share / (1 - share)) + math.log(keys) + 0.5) / (127 * step * scale)
    qi = indptr([tokens])
    want, lse_want = attention(q, t, c, scale, qi, False)
    for chunk in (0, 128 * math.ceil(keys / 128)):   # as planned, in one split
        o, lse = run(t, c, q, qi, False, plan=plan_of(t, q, 1, qi, False, chunk=chunk))
        off = float(((o.double() - want).norm(dim=-1) / want.norm(dim=-1)).max())
        assert off <= 2.0 ** -8 + 2.0 ** -7, f"{chunk}: {off}"
        assert float((lse.double() - lse_want).abs().max()) <= 2e-5
