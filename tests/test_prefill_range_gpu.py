"""fd_prefill_paged_int8 where f16's range of softmax weights and fp32's of V scales end,
against attention in 64 bits."""
import math

import numpy as np
import pytest
import torch

import split_kv_flashdecoding_gb300 as fd
from tests.int8_util import D, attention, cache, dev_tables, indptr, tables
from tests.test_prefill_gpu import make, plan_of, run

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


def compare_by_row(got, t, c, q, qi, causal, what, lse_abs=2e-5):
    """O against 64 bits, each row by its own keys' V scales.  Half a step of bf16; the
    weights' f16 (2^-11); exponents of up to 2^8, rounded a few times by 2^-17, in the
    weights' and in the sum's (2^-13); of weights that f16 does not have, 2^-36 of the
    largest each, 2^-24 of the row's values as if all of its codes were 127."""
    o, lse = got
    want, lse_want = attention(q, t, c, D ** -0.5, qi, causal)
    a, _ = attention(q, t, dict(c, v=c["v"].clamp(min=-127).abs()), D ** -0.5, qi, causal)
    most, _ = attention(q, t, dict(c, v=torch.full_like(c["v"], 127)), D ** -0.5, qi, causal)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -13) * a.abs() + 2.0 ** -24 * most.abs() + 2.0 ** -133
    over = (o.double() - want).abs() / tol
    assert float(over.max()) <= 1, f"{what}: {float(over.max())} of the tolerance"
    assert float((lse.double() - lse_want).abs().max()) <= lse_abs, what


@pytest.mark.parametrize("tokens", [20, 300])
@pytest.mark.parametrize("log2", [-110, -63, -41, 41, 100])
def test_prefill_v_values_of_any_size(cuda_device, tokens, log2):
    t, c, q, qi = make("vsize", 4, 2, [tokens], [700], 16, cuda_device)
    c["vs"] *= 2.0 ** log2
    for causal in (True, False):
        compare_by_row(run(t, c, q, qi, causal), t, c, q, qi, causal, f"{causal}")


@pytest.mark.parametrize("tokens", [20, 300])
@pytest.mark.parametrize("first", ["zeros", "ordinary", "large", "no scale"])
@pytest.mark.parametrize("log2", [-110, -63, -45, 30, 90])
def test_prefill_v_values_far_from_the_first_ones(cuda_device, tokens, first, log2):
    """A tile of zeros, or of values of another size, before values of one size."""
    t, c, q, qi = make("vfirst", 4, 2, [tokens], [700], 16, cuda_device)
    plain = c["vs"].clone()
    c["vs"] *= 2.0 ** log2
    for j in range(8 if first != "large" else 3):
        page = int(t["ids"][j])
        if first == "zeros":
            c["v"][page] = 0
            c["vs"][page] = 2.0 ** -126
        elif first == "no scale":
            c["vs"][page] = 0
        else:
            c["vs"][page] = plain[page] * 2.0 ** (20 if first == "large" else 0)
    for causal in (True, False):
        compare_by_row(run(t, c, q, qi, causal), t, c, q, qi, causal, f"{causal}")
    o, _ = run(t, c, q[-1:], indptr([1]), True)
    od, _ = fd.decode_paged_int8(q[-1:], c["k"], c["v"], c["ks"], c["vs"], t["ip"], t["last"], *dev_tables(t, cuda_device), D ** -0.5)
    assert float((o.double() - od.double()).abs().max()) <= 2.0 ** -7 * float(od.abs().max())


@pytest.mark.parametrize("tokens", [20, 300])
@pytest.mark.parametrize("chunk", [0, 256])
def test_prefill_v_scales_over_all_of_fp32(cuda_device, tokens, chunk):
    """A page's scale anywhere between 2^-110 and 2^110, some 0: each row as exact as its
    own keys allow, whichever pages it sees first."""
    t, c, q, qi = make("vall", 4, 2, [tokens, 3], [900, 40], 16, cuda_device)
    rng = np.random.RandomState(tokens)
    e = torch.from_numpy(rng.randint(-110, 110, (t["num_pages"], 4))).to(cuda_device)
    c["vs"] *= torch.exp2(e[:, : c["vs"].shape[1]].float())
    c["vs"][torch.from_numpy(t["ids"][::7].astype(np.int64)).to(cuda_device)] = 0
    for causal in (True, False):
        got = run(t, c, q, qi, causal, plan=plan_of(t, q, 2, qi, causal, chunk=chunk))
        compare_by_row(got, t, c, q, qi, causal, f"{causal}")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -1.0])
@pytest.mark.parametrize("tokens", [20, 200])
def test_prefill_v_scales_far_apart_and_no_numbers(cuda_device, tokens, value):
    t, c, q, qi = make("vbad", 8, 4, [tokens], [300], 16, cuda_device)
    c["vs"][int(t["ids"][3])] *= 2.0 ** 60
    c["vs"][int(t["ids"][17]), 1] = value   # keys 272 .. 287, head 1
    o, lse = run(t, c, q, qi, True)
    first = max(0, tokens - 300 + 272)
    bad = torch.zeros(o.shape[:2], dtype=torch.bool, device=cuda_device)
    bad[first:tokens, 2:4] = True
    assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad)


def test_prefill_of_many_partial_rows(cuda_device):
    """More than 2^24 partial rows of 512 bytes: offsets in values beyond 32 bits.  O within
    half a step of bf16, and 2^-10 of sum w |v| for the weights' f16 and the logits."""
    tokens, keys = 70000, 1024
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    t, c, _, _ = make("rows", 32, 8, [1], [keys], 16, cuda_device)
    gen = torch.Generator(cuda_device).manual_seed(1)
    q = torch.randn((tokens, 32, D), device=cuda_device, generator=gen, dtype=torch.bfloat16)
    qi = indptr([tokens])
    plan = plan_of(t, q, 8, qi, False, chunk=128)
    assert plan.num_partial_rows * D > 2 ** 31
    o, lse = run(t, c, q, qi, False, plan=plan)
    at = torch.tensor([0, 1, 64, 32767, 32768, 65535, 65536, 69998, 69999], device=cuda_device)
    want, lse_want = attention(q[at], t, c, D ** -0.5, indptr([len(at)]), False)
    a, _ = attention(q[at], t, dict(c, v=c["v"].clamp(min=-127).abs()), D ** -0.5, indptr([len(at)]), False)
    assert float(((o[at].double() - want).abs() / (2.0 ** -8 * want.abs() + 2.0 ** -10 * a)).max()) <= 1
    assert float((lse[at].double() - lse_want).abs().max()) <= 2e-5


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), -0.5])
@pytest.mark.parametrize("tokens", [20, 200])
def test_prefill_scales_that_are_no_numbers_reach_all_that_see_them(cuda_device, which, value, tokens):
    """O and LSE of each row that attends the page are NaN, all others as without it (two
    roundings of bf16, since a second pass may have other references)."""
    t, c, q, qi = make("nan", 8, 4, [tokens, 30], [300, 200], 16, cuda_device)
    want, lse_want = run(t, c, q, qi, True)
    c[which][int(t["ids"][17]), 1] = value   # keys 272 .. 287 of the first request, head 1
    o, lse = run(t, c, q, qi, True)
    bad = torch.zeros(o.shape[:2], dtype=torch.bool, device=cuda_device)
    bad[max(0, tokens - 300 + 272): tokens, 2:4] = True
    assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad)
    close = (o.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -9
    assert bool(close.all(-1)[~bad].all()) and float((lse - lse_want)[~bad].abs().max()) <= 4e-5


@pytest.mark.parametrize("tokens", [4, 20, 300])
@pytest.mark.parametrize("deviation", [4, 10])
@pytest.mark.parametrize("chunk", [0, 2560])
def test_prefill_scores_that_jump_in_many_tiles(cuda_device, tokens, deviation, chunk):
    """Independent logits of a large deviation, in nats: most rows meet scores beyond f16's
    range of the reference before them, in several tiles, and the items are done twice.
    Logits of up to 64 in log2 are rounded by 2^-18 a few times: 4e-5 in the LSE."""
    t, c, q, qi = make("wide", 8, 2, [tokens, 30], [2400, 1000], 16, cuda_device)
    gen = torch.Generator(cuda_device).manual_seed(tokens)
    c["ks"][:, :2] = deviation / 38
    c["k"].copy_((torch.randn(c["k"].shape, device=cuda_device, generator=gen) * 38).round().clamp(-127, 127))
    for causal in (True, False):
        got = run(t, c, q, qi, causal, plan=plan_of(t, q, 2, qi, causal, chunk=chunk))
        compare_by_row(got, t, c, q, qi, causal, f"{causal}", lse_abs=4e-5)
