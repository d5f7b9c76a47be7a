"""Workloads of the INT8 paged KV cache: one scale per page (block of tokens)
and KV head.

Three operators, as a server with such a cache uses them:
  append   rotary positions on new queries and keys, and the write of the new
           keys and values as INT8 codes; a page's scale grows with its keys
  decode   split-KV decode attention, one query token a request
  prefill  attention of one to many query tokens a request over the cache:
           causal (a prompt, a chunk of one behind cached keys, the check of
           drafted tokens) or over all keys (cross attention to an encoder's
           states of another length)

`run` computes them in elementary torch operations, or, where `own` is true,
through split_kv_flashdecoding_gb300.  `exact` restates each in 64 bits.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"
BASE = 500000.0
SMALLEST = 2.0 ** -126   # the scale of a page of zeros


# --------------------------------------------------------------- the cases

def listed():
    """Shapes: 8/8, 32/8 and 64/8 heads of dimension 128, 2k to 64k keys and the
    ragged batch are this repository's decode workloads; the rest are odd or
    generic sizes."""
    return [
        # a short conversation's next token: latency
        dict(name="decode_b1_l2048", op="decode", hq=8, hkv=8, batch=1, keys=2048, even=True, page=16),
        # one long document, 16-key pages
        dict(name="decode_b1_l65536_p16", op="decode", hq=32, hkv=8, batch=1, keys=65536, even=True, page=16),
        # a server's mixed batch
        dict(name="decode_b64_ragged_p64", op="decode", hq=32, hkv=8, batch=64, keys=16384, even=False, page=64),
        # long contexts of a model with 64 heads
        dict(name="decode_b16_h64_l32768_p32", op="decode", hq=64, hkv=8, batch=16, keys=32768, even=True, page=32),
        # one decode step of a batch: latency
        dict(name="append_b64_step", op="append", hq=32, hkv=8, batch=64, new=64, cached=8192, page=16,
             rotary=128, inter=False, scaling="bands"),
        # a decode step of a large batch, 64-key pages, half of each head rotated
        dict(name="append_b256_step", op="append", hq=64, hkv=8, batch=256, new=256, cached=4096, page=64,
             rotary=64, inter=True, scaling="none"),
        # an odd chunk of prompts behind cached keys, far positions
        dict(name="append_prompt_12345", op="append", hq=32, hkv=8, batch=7, new=12345, cached=65536, page=32,
             rotary=96, inter=True, scaling="yarn"),
        # prompts of a new batch
        dict(name="append_prompt_32768", op="append", hq=32, hkv=8, batch=4, new=32768, cached=0, page=64,
             rotary=128, inter=False, scaling="linear"),
        # five drafted tokens of each of 16 requests checked in one pass
        dict(name="prefill_draft_b16_t5", op="prefill", hq=32, hkv=8, batch=16, tokens=5, keys=8192, causal=True,
             page=16),
        # text that attends images or audio of other lengths, some requests without any
        dict(name="cross_b9_t500_l1500", op="prefill", hq=16, hkv=16, batch=9, tokens=500, keys=1500, causal=False,
             page=48),
        # a prompt from its start
        dict(name="prefill_prompt_8192", op="prefill", hq=32, hkv=8, batch=1, tokens=8192, keys=0, causal=True,
             page=64),
        # a chunk of a long prompt behind what is cached of it
        dict(name="prefill_chunk_h64_l30001", op="prefill", hq=64, hkv=8, batch=1, tokens=2047, keys=30001,
             causal=True, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "append", "prefill"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "decode":
        batch, keys = _log(rng, 1, 64), _log(rng, 100, 131072)
        while batch * keys * hkv > 16 * 32768 * 8:
            batch, keys = max(1, batch * 3 // 4), keys * 4 // 5
        return dict(op=op, hq=hq, hkv=hkv, batch=batch, keys=keys, even=rng.random() < 0.4, page=page)
    if op == "append":
        batch = _log(rng, 1, 256)
        new = batch if rng.random() < 0.5 else _log(rng, max(batch, 16), 32768)
        return dict(op=op, hq=hq, hkv=hkv, batch=batch, new=new, cached=rng.choice([0, _log(rng, 1, 16384)]),
                    page=page, rotary=rng.choice([128, 128, 96, 64, 32]), inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "bands", "yarn"]))
    causal = rng.random() < 0.7
    batch, tokens = _log(rng, 1, 32), _log(rng, 1, 4096)
    keys = rng.choice([0, _log(rng, 1, 32768)]) if causal else _log(rng, 1, 4096)
    while batch * hq * tokens * (keys + (tokens if causal else 0)) > 64 * 2047 * 32048:
        if batch > 1:
            batch = batch * 2 // 3
        else:
            tokens, keys = max(1, tokens * 3 // 4), keys * 3 // 4
    return dict(op=op, hq=hq, hkv=hkv, batch=batch, tokens=tokens, keys=keys, causal=causal, page=page)


# ------------------------------------------------ lengths, from the case alone

def _mix(n, salt):
    """n fixed numbers that look random, int64 in [0, 2^20)."""
    x = (np.arange(1, n + 1, dtype=np.uint64) * np.uint64(2654435761) + np.uint64(salt * 40503)) & np.uint64(0xFFFFFFFF)
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(2246822519)) & np.uint64(0xFFFFFFFF)
    return ((x >> np.uint64(9)) & np.uint64(0xFFFFF)).astype(np.int64)


def _indptr(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _decode_lengths(c):
    b, n = c["batch"], c["keys"]
    if c["even"]:
        return np.full(b, n, dtype=np.int64)
    lo = max(1, n // 32)
    return lo + _mix(b, 1) % max(1, n - lo + 1)


def _append_lengths(c):
    """Tokens in the cache before, and new ones, of each request."""
    b, n = c["batch"], c["new"]
    if n == b:
        new = np.ones(b, dtype=np.int64)
    else:
        w = 1 + _mix(b, 2) % 1000
        if b > 4:
            w[2] = 0
        new = n * w // w.sum()
        new[0] += n - new.sum()
    cached = _mix(b, 3) % c["cached"] if c["cached"] else np.zeros(b, dtype=np.int64)
    return cached, new


def _prefill_lengths(c):
    """Query tokens and keys of each request (the keys count the tokens' own
    where the attention is causal)."""
    b = c["batch"]
    small = c["tokens"] <= 8   # drafted tokens: as many for each
    tokens = np.full(b, c["tokens"], dtype=np.int64)
    if not small:
        tokens -= _mix(b, 4) % (c["tokens"] // 2)
        tokens[0] = c["tokens"]
        if b > 5:
            tokens[5] = 0
    if c["causal"]:
        keys = tokens + (c["keys"] - (_mix(b, 5) % (c["keys"] // 2 + 1)) * (b > 1) if c["keys"] else 0)
    else:
        keys = 1 + _mix(b, 6) % c["keys"]
        keys[0] = c["keys"]
        keys[3::7] = 0
    return tokens, keys


def _scaling(c):
    return {"none": None, "linear": ("linear", 4.0), "bands": ("bands", 8.0, 8192, 1.0, 4.0),
            "yarn": ("yarn", 4.0, 32768, 1.0, 32.0)}[c["scaling"]]


# ------------------------------------------------------------ the inputs

def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def _cache(pages, page, hkv, gen):
    """Codes int8 [pages, page, Hkv, D] of normal values and their pages' scales
    fp32 [pages, Hkv rounded up to 4]; heads and pages of different magnitude."""
    x = torch.randn((pages, page, hkv, D), generator=gen, device=DEV)
    x *= (0.25 + 2 * torch.rand((1, 1, hkv, 1), generator=gen, device=DEV)) * \
        (0.5 + torch.rand((pages, 1, hkv, 1), generator=gen, device=DEV))
    amax = x.abs().amax(dim=(1, 3))
    scale = torch.zeros((pages, -(-hkv // 4) * 4), device=DEV)
    scale[:, :hkv] = amax / 127
    return (x / scale[:, None, :hkv, None]).round_().to(torch.int8), scale


def _tables(s, keys, p, rng, spare=3):
    """Page tables of requests with these many keys, pages anywhere in the pool."""
    cnt = -(-keys // p)
    pages = int(cnt.sum()) + spare
    s["ip_host"], s["last_host"] = _indptr(cnt), np.where(cnt > 0, keys - (cnt - 1) * p, 0).astype(np.int32)
    s["kv_indptr"], s["kv_last"] = _dev(s["ip_host"]), _dev(s["last_host"])
    s["kv_ids"] = _dev(np.append(rng.permutation(pages)[: pages - spare], 0))
    s["len"], s["len_max"] = _dev(keys, torch.int64), max(1, int(keys.max()))
    return pages


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    c = dict(case)
    return {"decode": _prepare_decode, "append": _prepare_append, "prefill": _prepare_prefill}[c["op"]](c, gen, rng)


def _prepare_decode(c, gen, rng):
    b, hq, hkv, p = c["batch"], c["hq"], c["hkv"], c["page"]
    s = dict(case=c, scale=1.0 / math.sqrt(D))
    pages = _tables(s, _decode_lengths(c), p, rng)
    s["k_pages"], s["k_scale"] = _cache(pages, p, hkv, gen)
    s["v_pages"], s["v_scale"] = _cache(pages, p, hkv, gen)
    s["q"] = torch.randn((b, hq, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    if own:
        import split_kv_flashdecoding_gb300 as fd
        need = fd.plan_paged(b, hq, hkv, D, p, s["ip_host"], s["last_host"]).workspace_bytes
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
        s["o"] = torch.empty((b, hq, D), dtype=torch.float32, device=DEV)
        s["lse"] = torch.empty((b, hq), dtype=torch.float32, device=DEV)
    return s


def _prepare_append(c, gen, rng):
    cached, new = _append_lengths(c)
    b, hq, hkv, p = c["batch"], c["hq"], c["hkv"], c["page"]
    n = int(new.sum())
    rows = n + 3   # a padded batch: the rows behind the last request stay as they were
    have = cached + new
    np_ = -(-have // p)
    # the pool holds every page that gets keys; a long cached part before them is
    # kept in one page that the tables repeat, as no call here reads it
    first = cached // p
    uniq = np.where(np_ > 0, np_ - first, 0)
    pages = int(uniq.sum()) + 5
    ids = rng.permutation(pages)
    tables, at = [], 0
    for i in range(b):
        tables += [np.full(first[i], ids[-1]), ids[at: at + uniq[i]]]
        at += int(uniq[i])
    s = dict(case=c, n=n)
    s["qkv"] = torch.randn((rows, (hq + 2 * hkv) * D), generator=gen, device=DEV, dtype=torch.bfloat16)
    s["q_out"] = torch.full((rows, hq, D), 7.0, device=DEV, dtype=torch.bfloat16)
    s["k_pages"], s["k_scale"] = _cache(pages, p, hkv, gen)
    s["v_pages"], s["v_scale"] = _cache(pages, p, hkv, gen)
    s["k_val"], s["v_val"] = (torch.empty((pages, p, hkv, D), device=DEV, dtype=torch.float16) for _ in range(2))
    s["indptr"] = _dev(_indptr(new))
    s["kv_indptr"], s["kv_last"] = _dev(_indptr(np_)), _dev(np.where(np_ > 0, have - (np_ - 1) * p, 0))
    s["kv_ids"] = _dev(np.concatenate(tables + [[0]]))
    # every third request sits behind a shared prefix: its positions start later
    base = np.where(np.arange(b) % 3 == 2, 1000, 0) + cached
    pos = np.concatenate([base[i] + np.arange(new[i]) for i in range(b)] + [np.zeros(rows - n, dtype=np.int64)])
    s["pos"] = _dev(pos)
    if own:
        import split_kv_flashdecoding_gb300 as fd
        s["rope"] = fd.plan_rope(D, c["rotary"], interleaved=c["inter"], base=BASE, scaling=_scaling(c))
        s["ws"] = torch.zeros(fd.WORKSPACE_HEADER_BYTES, dtype=torch.uint8, device=DEV)
    return s


def _prepare_prefill(c, gen, rng):
    tokens, keys = _prefill_lengths(c)
    b, hq, hkv, p = c["batch"], c["hq"], c["hkv"], c["page"]
    s = dict(case=c, scale=1.0 / math.sqrt(D), n=int(tokens.sum()))
    pages = _tables(s, keys, p, rng)
    s["k_pages"], s["k_scale"] = _cache(pages, p, hkv, gen)
    s["v_pages"], s["v_scale"] = _cache(pages, p, hkv, gen)
    s["q"] = torch.randn((s["n"], hq, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    s["q_indptr"] = _dev(_indptr(tokens))
    s["t_max"] = max(1, int(tokens.max()))
    if own:
        import split_kv_flashdecoding_gb300 as fd
        s["plan"] = fd.plan_prefill_paged(b, hq, hkv, D, p, _indptr(tokens), s["ip_host"], s["last_host"],
                                          causal=c["causal"])
        s["ws"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device=DEV)
        s["o"] = torch.empty((s["n"], hq, D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((s["n"], hq), dtype=torch.float32, device=DEV)
    return s


# ------------------------------------------------------------- one pass

def run(state):
    return {"decode": _run_decode, "append": _run_append, "prefill": _run_prefill}[state["case"]["op"]](state)


def _gathered(s):
    """K and V [B, L, Hkv, D] in fp32 and which of the L places hold a key [B, L]."""
    p, hkv = s["case"]["page"], s["case"]["hkv"]
    at = torch.arange(s["len_max"], device=DEV)
    has = at[None] < s["len"][:, None]
    page = s["kv_ids"][torch.where(has, s["kv_indptr"][:-1, None] + at[None] // p, 0)].long()
    row = page * p + at[None] % p
    return [codes.view(-1, hkv, D)[row].float() * scale[page][..., :hkv, None]
            for codes, scale in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"]))] + [has]


def _run_decode(s):
    c = s["case"]
    b, hq, hkv = c["batch"], c["hq"], c["hkv"]
    if own:
        import split_kv_flashdecoding_gb300 as fd
        return fd.decode_paged_int8(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["ip_host"],
                                    s["last_host"], s["kv_indptr"], s["kv_last"], s["kv_ids"], s["scale"],
                                    o=s["o"], lse=s["lse"], workspace=s["ws"])
    k, v, has = _gathered(s)
    sc = torch.matmul(s["q"].float().view(b, hkv, hq // hkv, D) * s["scale"], k.permute(0, 2, 3, 1))
    sc.masked_fill_(~has[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    sc.sub_(m).exp_()
    den = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc, v.permute(0, 2, 1, 3)) / den
    return o.reshape(b, hq, D), (m + den.log()).reshape(b, hq)


def _run_prefill(s):
    c = s["case"]
    b, hq, hkv = c["batch"], c["hq"], c["hkv"]
    if own:
        import split_kv_flashdecoding_gb300 as fd
        return fd.prefill_paged_int8(s["plan"], s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                     s["q_indptr"], s["kv_indptr"], s["kv_last"], s["kv_ids"], s["scale"],
                                     o=s["o"], lse=s["lse"], workspace=s["ws"])
    # the requests' tokens padded to [B, T], their rows of a KV head side by side
    g, t_max = hq // hkv, s["t_max"]
    k, v, has = _gathered(s)
    t = torch.arange(t_max, device=DEV)
    row = s["q_indptr"][:-1, None] + t[None]
    real = row < s["q_indptr"][1:, None]
    q = s["q"].float()[torch.where(real, row, 0)] * s["scale"]
    q = q.view(b, t_max, hkv, g, D).permute(0, 2, 1, 3, 4).reshape(b, hkv, t_max * g, D)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)).view(b, hkv, t_max, g, -1)
    hide = ~has[:, None]
    if c["causal"]:   # token t of T is the key T - t places before the end
        last = s["len"][:, None] - (s["q_indptr"][1:] - s["q_indptr"][:-1])[:, None] + t[None]
        hide = hide | (torch.arange(sc.shape[-1], device=DEV) > last[..., None])
    sc.masked_fill_(hide[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    sc.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    den = sc.sum(-1, keepdim=True)
    o = torch.matmul(sc.view(b, hkv, t_max * g, -1), v.permute(0, 2, 1, 3)).view(b, hkv, t_max, g, D)
    o = torch.where(den > 0, o / den, 0.0)
    lse = (m + den.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(b, t_max, hq, D)[real]
    return o.to(torch.bfloat16), lse.permute(0, 2, 1, 3).reshape(b, t_max, hq)[real]


def _frequencies(c):
    """Radians per position of each pair, in 64 bits."""
    r, sc = c["rotary"], _scaling(c)
    i = torch.arange(r // 2, device=DEV, dtype=torch.float64)
    f = BASE ** (-2.0 * i / r)
    if sc is None:
        return f, 1.0
    if sc[0] == "linear":
        return f / sc[1], 1.0
    if sc[0] == "bands":   # short wavelengths stay, long ones are stretched, a ramp between
        _, factor, trained, low, high = sc
        turns = trained * f / (2 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    _, factor, trained, slow, fast = sc
    dim = lambda turns: r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
    low, high = max(math.floor(dim(fast)), 0), min(math.ceil(dim(slow)), r - 1)
    keep = 1 - ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
    return f * keep + f / factor * (1 - keep), 0.1 * math.log(factor) + 1


def _rotate(x, cos, sin, r, inter):
    a, b = (x[..., :r:2], x[..., 1:r:2]) if inter else (x[..., : r // 2], x[..., r // 2: r])
    y, z = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((y, x[..., r:]), -1)


def _values(s):
    """The caches as the values they stand for, one product each."""
    hkv = s["case"]["hkv"]
    torch.mul(s["k_pages"], s["k_scale"][:, None, :hkv, None], out=s["k_val"])
    torch.mul(s["v_pages"], s["v_scale"][:, None, :hkv, None], out=s["v_val"])
    return s["q_out"], s["k_scale"], s["v_scale"], s["k_val"], s["v_val"]


def _run_append(s):
    c, n = s["case"], s["n"]
    hq, hkv, p = c["hq"], c["hkv"], c["page"]
    x = s["qkv"].view(-1, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
    if own:
        import split_kv_flashdecoding_gb300 as fd
        fd.append_paged_int8(q, k, v, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["indptr"],
                             s["kv_indptr"], s["kv_last"], s["kv_ids"], rope=s["rope"], positions=s["pos"],
                             q_out=s["q_out"], workspace=s["ws"])
        return _values(s)
    freq, gain = _frequencies(c)
    ang = s["pos"][:n, None].double() * freq
    cos, sin = (gain * ang.cos()).float()[:, None], (gain * ang.sin()).float()[:, None]
    s["q_out"][:n] = _rotate(q[:n].float(), cos, sin, c["rotary"], c["inter"]).to(torch.bfloat16)
    kr = _rotate(k[:n].float(), cos, sin, c["rotary"], c["inter"])
    # page and place of each new token: the last keys of its request's table
    t = torch.arange(n, device=DEV)
    b = torch.searchsorted(s["indptr"][1:], t, right=True)
    cnt = s["kv_indptr"][b + 1] - s["kv_indptr"][b]
    key = (cnt - 1) * p + s["kv_last"][b] - (s["indptr"][b + 1] - t)
    page, at = s["kv_ids"][s["kv_indptr"][b] + key // p].long(), key % p
    # keys that each page has from before: its first new token's place
    pages = s["k_pages"].shape[0]
    before = torch.full((pages,), p, device=DEV, dtype=torch.int64).scatter_reduce_(0, page, at.long(), "amin")
    touched = before < p
    for codes, scale, y in ((s["k_pages"], s["k_scale"], kr), (s["v_pages"], s["v_scale"], v[:n].float())):
        old = torch.where((touched & (before == 0))[:, None], 0.0, scale[:, :hkv])
        most = torch.zeros_like(old).scatter_reduce_(0, page[:, None].expand(-1, hkv), y.abs().amax(-1), "amax")
        new = torch.where(touched[:, None], torch.maximum(old, most / 127).clamp(min=SMALLEST), scale[:, :hkv])
        ratio = torch.where(new > old, old / new, 1.0)[:, None, :, None]
        mine = (touched & (before > 0))[:, None] & (torch.arange(p, device=DEV)[None] < before[:, None])
        codes.copy_(torch.where(mine[..., None, None], (codes * ratio).round_(), codes.float()))
        codes[page, at] = (y / new[page][..., None]).round_().to(torch.int8)
        scale[:, :hkv] = new
    return _values(s)


# ----------------------------------------------------------------- the work

def work(case):
    c = case
    hq, hkv, p = c["hq"], c["hkv"], c["page"]
    if c["op"] == "decode":
        keys = _decode_lengths(c)
        pages = int((-(-keys // p)).sum())
        return {"bytes": 2 * hkv * (int(keys.sum()) * D + 4 * pages) + c["batch"] * hq * (2 * D + 4 * D + 4),
                "flops": 4.0 * hq * D * float(keys.sum())}
    if c["op"] == "append":
        cached, new = _append_lengths(c)
        touched = int(np.where(new > 0, (cached + new - 1) // p - cached // p + 1, 0).sum())
        return {"bytes": c["new"] * (D * (4 * hq + 6 * hkv) + 4) + 12 * c["batch"] + 16 * hkv * touched,
                "flops": c["new"] * (3.0 * c["rotary"] * (hq + hkv) + 4.0 * D * hkv)}
    tokens, keys = _prefill_lengths(c)
    pages = int((-(-keys // p)).sum())
    # a causal request's first token sees keys - tokens + 1, the last all of them
    pairs = tokens * keys - (tokens * (tokens - 1) // 2 if c["causal"] else 0)
    return {"bytes": 2 * hkv * (int(keys.sum()) * D + 4 * pages) + int(tokens.sum()) * hq * (4 * D + 4),
            "flops": 4.0 * hq * D * float(pairs.sum())}


# ------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_attention, "append": _exact_append, "prefill": _exact_attention}[s["case"]["op"]](s)


def _exact_attention(s):
    """Request by request, KV head by KV head, softmax over the request's keys."""
    c = s["case"]
    hq, hkv, p = c["hq"], c["hkv"], c["page"]
    g = hq // hkv
    if c["op"] == "decode":
        keys = _decode_lengths(c)
        ends, causal = np.arange(c["batch"] + 1), False
    else:
        tokens, keys = _prefill_lengths(c)
        ends, causal = np.concatenate([[0], np.cumsum(tokens)]), c["causal"]
    ids = s["kv_ids"].cpu().numpy().astype(np.int64)
    o = torch.zeros((int(ends[-1]), hq, D), dtype=torch.float64, device=DEV)
    lse = torch.full((int(ends[-1]), hq), -math.inf, dtype=torch.float64, device=DEV)
    for i, n in enumerate(keys):
        t0, t1, n = int(ends[i]), int(ends[i + 1]), int(n)
        if t0 == t1 or n == 0:
            continue
        pg = _dev(ids[s["ip_host"][i]: s["ip_host"][i + 1]], torch.int64)
        for h in range(hkv):
            kh, vh = ((x[pg, :, h].double() * y[pg, h].double()[:, None, None]).view(-1, D)[:n]
                      for x, y in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            scores = (s["q"][t0:t1, h * g: (h + 1) * g].double() @ kh.T) * s["scale"]   # [T, G, n]
            if causal:
                behind = torch.arange(n, device=DEV)[None] > (n - (t1 - t0) + torch.arange(t1 - t0, device=DEV))[:, None]
                scores.masked_fill_(behind[:, None], -math.inf)
            z = torch.logsumexp(scores, -1)
            o[t0:t1, h * g: (h + 1) * g] = scores.sub_(z[..., None]).exp_() @ vh
            lse[t0:t1, h * g: (h + 1) * g] = z
    return o, lse


def _exact_append(s):
    """Each pair of a head as a complex number, turned by its angle; then page
    by page of each request's new keys."""
    c, n = s["case"], s["n"]
    hq, hkv, p, r = c["hq"], c["hkv"], c["page"], c["rotary"]
    sc, freq, gain = _scaling(c), [], 1.0
    for i in range(r // 2):
        f = 1.0 / BASE ** (2.0 * i / r)
        if sc and sc[0] == "linear":
            f /= sc[1]
        elif sc and sc[0] == "bands":
            wave = 2 * math.pi / f
            if wave > sc[2] / sc[3]:
                f /= sc[1]
            elif wave >= sc[2] / sc[4]:
                smooth = (sc[2] / wave - sc[3]) / (sc[4] - sc[3])
                f = (1 - smooth) * f / sc[1] + smooth * f
        elif sc:
            lo = r * math.log(sc[2] / (2 * math.pi * sc[4])) / (2 * math.log(BASE))
            hi = r * math.log(sc[2] / (2 * math.pi * sc[3])) / (2 * math.log(BASE))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 1e-3)))
            f = f / sc[1] * ramp + f * (1 - ramp)
            gain = 0.1 * math.log(sc[1]) + 1
        freq.append(f)
    pos = s["pos"][:n].cpu().numpy().astype(np.float64)
    turn = gain * np.exp(1j * (pos[:, None] * np.array(freq)[None]))[:, None]
    x = s["qkv"].view(-1, hq + 2 * hkv, D)[:n].double().cpu().numpy()

    def rotated(y):
        y = y.copy()
        ia, ib = (slice(0, r, 2), slice(1, r, 2)) if c["inter"] else (slice(0, r // 2), slice(r // 2, r))
        z = (y[..., ia] + 1j * y[..., ib]) * turn
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    q_out = s["q_out"].double().cpu().numpy()
    q_out[:n] = rotated(x[:, :hq])
    cached, new = _append_lengths(c)
    ids, ip = s["kv_ids"].cpu().numpy(), s["kv_indptr"].cpu().numpy()
    start = _indptr(new)
    scales, values = [], []
    for name, y in (("k", rotated(x[:, hq: hq + hkv])), ("v", x[:, hq + hkv:])):
        codes = s[name + "_pages"].cpu().numpy().astype(np.float64)
        scale = s[name + "_scale"].double().cpu().numpy()
        for i in range(c["batch"]):
            done = 0
            while done < new[i]:
                key = int(cached[i]) + done
                page, at = ids[ip[i] + key // p], key % p
                take = min(p - at, int(new[i]) - done)
                rows = y[start[i] + done: start[i] + done + take]          # [take, Hkv, D]
                old = scale[page, :hkv].copy() if at else np.zeros(hkv)
                now = np.maximum(np.maximum(old, np.abs(rows).max(axis=(0, 2)) / 127), SMALLEST)
                codes[page, :at] = np.rint(codes[page, :at] * (old / now)[:, None])
                codes[page, at: at + take] = np.rint(rows / now[:, None])
                scale[page, :hkv] = now
                done += take
        scales.append(scale)
        values.append(codes * scale[:, None, :hkv, None])
    return tuple(torch.from_numpy(a) for a in (q_out, *scales, *values))
