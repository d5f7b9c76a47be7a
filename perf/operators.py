"""Workloads of the serving operators around paged split-KV decode attention.

Four operators, as one serving step uses them:
  shared   decode attention for a batch whose requests share long prefixes:
           each prefix is attended once for all of its requests, each
           request's own keys (its suffix) by the split-KV kernel, and the two
           states are merged
  append   rotary positions on new queries and keys, and the write of the new
           keys and values into a paged cache (bf16 or FP8)
  fork     the page tables of the next step: requests that fork, go on, start
           or end, with reference counts, fresh pages and the copies of
           partly filled last pages
  compact  moving the live pages of a cache to its front

`run` computes them in elementary torch operations, or, where `own` is true,
through split_kv_flashdecoding_gb300.  `exact` restates each in 64 bits.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"


# --------------------------------------------------------------- the cases

def listed():
    """Shapes: 32/8 and 64/8 heads of dimension 128 and 64k contexts are this
    repository's decode workloads; the rest are odd or generic sizes."""
    return [
        # four samples of one short prompt, right after it: latency
        dict(name="shared_b4_l2048", op="shared", paged=False, page=16, kv="bf16", hq=32, hkv=8,
             groups=1, batch=4, prefix=2048, suffix=64),
        # a long document that 32 users ask about, 16-key pages: the prefix's bytes
        dict(name="shared_b32_l65536_p16", op="shared", paged=True, page=16, kv="bf16", hq=32,
             hkv=8, groups=1, batch=32, prefix=65536, suffix=512),
        # a large batch behind one long system prompt: the products
        dict(name="shared_b256_h64_l32768", op="shared", paged=False, page=16, kv="bf16", hq=64,
             hkv=8, groups=1, batch=256, prefix=32768, suffix=128),
        # three prompts of odd lengths in one batch, FP8 cache in 64-key pages
        dict(name="shared_fp8_b45_3x20001", op="shared", paged=True, page=64, kv="fp8", hq=32,
             hkv=8, groups=3, batch=45, prefix=20001, suffix=333),
        # one decode step of a batch: latency
        dict(name="append_b64_step", op="append", kv="bf16", hq=32, hkv=8, batch=64, new=64,
             cached=8192, page=16, rotary=128, inter=False, scaling="bands"),
        # a decode step of a large batch into an FP8 cache, half of each head rotated
        dict(name="append_fp8_b256_step", op="append", kv="fp8", hq=64, hkv=8, batch=256, new=256,
             cached=4096, page=16, rotary=64, inter=True, scaling="none"),
        # prompts of a new batch
        dict(name="append_prompt_32768", op="append", kv="bf16", hq=32, hkv=8, batch=4, new=32768,
             cached=0, page=64, rotary=128, inter=False, scaling="linear"),
        # an odd chunk of prompts behind cached ones, far positions
        dict(name="append_fp8_prompt_12345", op="append", kv="fp8", hq=32, hkv=8, batch=7,
             new=12345, cached=65536, page=32, rotary=96, inter=True, scaling="yarn"),
        # four samples of each of 8 prompts, one layer's cache
        dict(name="fork_b8_to_32", op="fork", batch=8, children=32, length=1500, page=16, pages=2000,
             pools=2, hkv=8),
        # a beam step of 64 requests over four layers' caches
        dict(name="fork_b64_to_251", op="fork", batch=64, children=251, length=900, page=16,
             pages=4096, pools=8, hkv=8),
        # a half-empty small cache
        dict(name="compact_1000", op="compact", batch=9, length=900, page=16, pages=1000, pools=2,
             hkv=8, room=0),
        # shrinking four layers' caches after most requests have ended
        dict(name="compact_4096x8", op="compact", batch=37, length=700, page=16, pages=4096, pools=8,
             hkv=8, room=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared", "append", "fork", "compact"])
    if op == "shared":
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 8])
        batch, prefix = _log(rng, 2, 256), _log(rng, 200, 131072)
        while batch * hq * prefix > 256 * 64 * 32768:
            batch = max(2, batch // 2)
            prefix = prefix * 3 // 4
        suffix = _log(rng, 1, 1024)
        return dict(op=op, paged=rng.random() < 0.6, page=rng.choice([16, 32, 48, 64]),
                    kv=rng.choice(["bf16", "fp8"]), hq=hq, hkv=hkv,
                    groups=min(batch, rng.choice([1, 1, 2, 3, 5])), batch=batch, prefix=prefix,
                    suffix=suffix)
    if op == "append":
        hkv = rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 256)
        new = batch if rng.random() < 0.5 else _log(rng, max(batch, 16), 32768)
        return dict(op=op, kv=rng.choice(["bf16", "fp8"]), hq=hkv * rng.choice([1, 2, 4, 8]) if hkv < 8 else 32,
                    hkv=hkv, batch=batch, new=new, cached=rng.choice([0, _log(rng, 1, 16384)]),
                    page=rng.choice([16, 32, 48, 64]), rotary=rng.choice([128, 128, 96, 64, 32]),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "bands", "yarn"]))
    batch, length = _log(rng, 2, 64), _log(rng, 20, 1000)
    page = rng.choice([16, 16, 32])
    need = batch * (-(-length // page) + 1)
    if op == "fork":
        children = _log(rng, 2, 256)
        return dict(op=op, batch=batch, children=children, length=length, page=page,
                    pages=min(4096, need + 2 * children * 4 + rng.randrange(500)) if need < 2000 else 4096 + need,
                    pools=2 * rng.randint(1, 2), hkv=rng.choice([1, 2, 4]))
    pages = need + rng.randrange(10, need + 11)
    return dict(op=op, batch=batch, length=length, page=page, pages=pages, pools=2 * rng.randint(1, 2),
                hkv=rng.choice([1, 2, 4]), room=rng.choice([0, 0, need + 1]))


# ------------------------------------------------ lengths, from the case alone

def _mix(n, salt):
    """n fixed numbers that look random, int64 in [0, 2^20)."""
    x = (np.arange(1, n + 1, dtype=np.uint64) * np.uint64(2654435761) + np.uint64(salt * 40503)) & np.uint64(0xFFFFFFFF)
    x ^= x >> np.uint64(15)
    x = (x * np.uint64(2246822519)) & np.uint64(0xFFFFFFFF)
    return ((x >> np.uint64(9)) & np.uint64(0xFFFFF)).astype(np.int64)


def _indptr(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def _shared_lengths(c):
    """Requests of each prefix, keys of each prefix, keys of each request's own (some have none)."""
    g, b = c["groups"], c["batch"]
    req = np.full(g, b // g, dtype=np.int64)
    req[: b % g] += 1
    prefix = np.array([max(1, c["prefix"] * (g - i) // g - 7 * i) for i in range(g)], dtype=np.int64)
    own_keys = 1 + _mix(b, 1) % c["suffix"]
    own_keys[3::7] = 0
    return req, prefix, own_keys


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


def _table_lengths(c):
    """Keys of each request of a table; every fifth ends on a page's end."""
    n = 1 + c["length"] // 2 + _mix(c["batch"], 4) % (1 + c["length"] // 2)
    n[::5] = -(-n[::5] // c["page"]) * c["page"]
    return n


def _parents(c):
    """Which request each next one comes from; -1: a new one.  Some requests end."""
    p = np.sort(_mix(c["children"], 5) % c["batch"])
    p[5::11] = -1
    return p


def _scaling(c):
    return {"none": None, "linear": ("linear", 4.0), "bands": ("bands", 8.0, 8192, 1.0, 4.0),
            "yarn": ("yarn", 4.0, 32768, 1.0, 32.0)}[c["scaling"]]


BASE = 500000.0


# ------------------------------------------------------------ the inputs

def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dtype)


def _quantise(x, scale):
    return (x / scale).to(torch.float8_e4m3fn)


def _kv(shape, gen, fp8):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32 if fp8 else torch.bfloat16)
    return x.mul_(80.0).clamp_(-448, 448).to(torch.float8_e4m3fn) if fp8 else x


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 31))
    c = dict(case)
    if c["op"] == "shared":
        return _prepare_shared(c, gen, rng)
    if c["op"] == "append":
        return _prepare_append(c, gen, rng)
    return _prepare_table(c, gen, rng)


def _prepare_shared(c, gen, rng):
    req, prefix, own_keys = _shared_lengths(c)
    b, hq, hkv, p, fp8 = c["batch"], c["hq"], c["hkv"], c["page"], c["kv"] == "fp8"
    room = b * c["suffix"]   # keys the requests may grow to: what the plan is made for
    s = dict(case=c, scale=1.0 / math.sqrt(D), req=_dev(_indptr(req)), total=int(own_keys.sum()))
    s["q"] = torch.randn((b, hq, D), generator=gen, device=DEV, dtype=torch.bfloat16)
    s["k_scale"] = s["v_scale"] = None
    if fp8:
        s["k_scale"] = (0.5 + torch.rand(hkv, generator=gen, device=DEV)) / 80.0
        s["v_scale"] = (0.5 + torch.rand(hkv, generator=gen, device=DEV)) / 80.0
    if c["paged"]:
        pp, op = -(-prefix // p), -(-own_keys // p)
        pages = int(pp.sum() + op.sum()) + 3
        ids = rng.permutation(pages)[: pages - 3]
        s["k_pages"], s["v_pages"] = (_kv((pages, p, hkv, D), gen, fp8) for _ in range(2))
        s["pre_indptr"], s["pre_last"] = _dev(_indptr(pp)), _dev(prefix - (pp - 1) * p)
        s["pre_ids"] = _dev(ids[: pp.sum()])
        s["kv_indptr"], s["kv_last"] = _dev(_indptr(op)), _dev(np.where(op > 0, own_keys - (op - 1) * p, 0))
        s["kv_ids"] = _dev(np.append(ids[pp.sum():], 0))
    else:
        s["k_pre"], s["v_pre"] = (_kv((int(prefix.sum()), hkv, D), gen, fp8) for _ in range(2))
        s["k"], s["v"] = (_kv((max(room, 1), hkv, D), gen, fp8) for _ in range(2))
        s["pre_indptr"], s["kv_indptr"] = _dev(_indptr(prefix)), _dev(_indptr(own_keys))
    # where each prefix's keys and each request's own keys are, for the plain form
    s["pre_len"], s["own_len"] = _dev(prefix, torch.int64), _dev(own_keys, torch.int64)
    s["pre_max"], s["own_max"], s["req_max"] = int(prefix.max()), max(1, int(own_keys.max())), int(req.max())
    if own:
        import split_kv_flashdecoding_gb300 as fd
        if c["paged"]:
            s["plan"] = fd.plan_shared_paged(b, hq, hkv, D, p, _indptr(req), _indptr(-(-prefix // p)),
                                             (prefix - (-(-prefix // p) - 1) * p).astype(np.int32), room)
        else:
            s["plan"] = fd.plan_shared(b, hq, hkv, D, _indptr(req), _indptr(prefix), room)
        s["ws"] = torch.zeros(s["plan"].workspace_bytes, dtype=torch.uint8, device=DEV)
        s["o"] = torch.empty((b, hq, D), dtype=torch.float32, device=DEV)
        s["lse"] = torch.empty((b, hq), dtype=torch.float32, device=DEV)
    return s


def _prepare_append(c, gen, rng):
    cached, new = _append_lengths(c)
    b, hq, hkv, p, fp8 = c["batch"], c["hq"], c["hkv"], c["page"], c["kv"] == "fp8"
    n = int(new.sum())
    rows = n + 3   # a padded batch: the rows behind the last request stay as they were
    have = cached + new
    np_ = -(-have // p)
    # the cache holds every page of the requests' tables; a long cached part is
    # kept in a few pages that the tables repeat, as no call here reads it
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
    s["k_pages"], s["v_pages"] = (_kv((pages, p, hkv, D), gen, fp8) for _ in range(2))
    s["k_scale"] = s["v_scale"] = None
    if fp8:
        s["k_scale"], s["v_scale"] = ((0.5 + torch.rand(hkv, generator=gen, device=DEV)) / 80.0 for _ in range(2))
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


def _prepare_table(c, gen, rng):
    keys, p, pages = _table_lengths(c), c["page"], c["pages"]
    cnt = -(-keys // p)
    ids, tables, at = rng.permutation(pages), [], 0
    for i in range(c["batch"]):
        t = ids[at: at + cnt[i]].copy()
        at += int(cnt[i])
        if i % 2:   # half of its pages are those of the request before: a common prompt
            h = int(min(cnt[i], cnt[i - 1])) // 2
            t[:h] = tables[-1][:h]
        tables.append(t)
    flat = np.concatenate(tables)
    s = dict(case=c, indptr=_dev(_indptr(cnt)), last=_dev(keys - (cnt - 1) * p), ids=_dev(flat),
             refs=_dev(np.bincount(flat, minlength=pages)))
    s["pools"] = [torch.randn((pages, p, c["hkv"], D), generator=gen, device=DEV, dtype=torch.bfloat16)
                  for _ in range(c["pools"])]
    if c["op"] == "fork":
        par = _parents(c)
        last = keys - (cnt - 1) * p
        # a page more where the last one is full: the next token's; a new request gets two
        nxt = np.where(par < 0, 2, cnt[par] + (last[par] == p))
        s["parent"], s["new_indptr"], s["entries"] = _dev(par), _dev(_indptr(nxt)), int(nxt.sum())
    else:
        live = int((np.bincount(flat, minlength=pages) > 0).sum())
        s["limit"] = c["room"] if c["room"] >= live else 0
        # what the host knows of the number of moves: no more than there are live or free pages
        s["most"] = max(1, min(live, pages - live))
    if own:
        import split_kv_flashdecoding_gb300 as fd
        s["ws"] = torch.zeros(fd.pages_workspace_bytes(pages, c.get("children", 0)), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------- one pass

def run(state):
    return {"shared": _run_shared, "append": _run_append, "fork": _run_fork,
            "compact": _run_compact}[state["case"]["op"]](state)


def _run_shared(s):
    c = s["case"]
    if own:
        import split_kv_flashdecoding_gb300 as fd
        fp8 = c["kv"] == "fp8"
        out = dict(o=s["o"], lse=s["lse"], workspace=s["ws"])
        if c["paged"]:
            call = fd.decode_shared_paged_fp8 if fp8 else fd.decode_shared_paged
            scales = (s["k_scale"], s["v_scale"]) if fp8 else ()
            return call(s["plan"], s["q"], s["k_pages"], s["v_pages"], *scales, s["req"], s["pre_indptr"],
                        s["pre_last"], s["pre_ids"], s["kv_indptr"], s["kv_last"], s["kv_ids"],
                        s["scale"], **out)
        call = fd.decode_shared_fp8 if fp8 else fd.decode_shared
        scales = (s["k_scale"], s["v_scale"]) if fp8 else ()
        return call(s["plan"], s["q"], s["k_pre"], s["v_pre"], s["k"], s["v"], *scales, s["req"],
                    s["pre_indptr"], s["kv_indptr"], s["scale"], **out)
    # Plain: the prefixes gathered to [prefixes, keys], the requests of each to
    # [prefixes, requests], one product of all of a prefix's queries with its keys.
    b, hq, hkv, p = c["batch"], c["hq"], c["hkv"], c["page"]
    g = hq // hkv
    at = torch.arange(s["pre_max"], device=DEV)
    has = at[None] < s["pre_len"][:, None]                                      # [P, L]
    at_own = torch.arange(s["own_max"], device=DEV)
    has_own = at_own[None] < s["own_len"][:, None]                              # [B, S]
    if c["paged"]:
        rows = _paged_rows(s["pre_indptr"], s["pre_ids"], at, has, p)
        own_rows = _paged_rows(s["kv_indptr"], s["kv_ids"], at_own, has_own, p)
        kp, vp = s["k_pages"].view(-1, hkv, D), s["v_pages"].view(-1, hkv, D)
        ko, vo = kp, vp
    else:
        rows = torch.where(has, s["pre_indptr"][:-1, None] + at[None], 0)
        own_rows = torch.where(has_own, s["kv_indptr"][:-1, None] + at_own[None], 0)
        kp, vp, ko, vo = s["k_pre"], s["v_pre"], s["k"], s["v"]
    r_at = torch.arange(s["req_max"], device=DEV)
    r_idx = s["req"][:-1, None] + r_at[None]                                    # [P, R]
    r_has = r_idx < s["req"][1:, None]
    r_idx = torch.where(r_has, r_idx, 0)
    qf = s["q"].float() * s["scale"]
    qp = qf[r_idx].view(-1, s["req_max"], hkv, g, D).permute(0, 2, 1, 3, 4).reshape(-1, hkv, s["req_max"] * g, D)
    kx, vx = _values(kp, rows, s["k_scale"]), _values(vp, rows, s["v_scale"])  # [P, L, Hkv, D]
    sc = torch.matmul(qp, kx.permute(0, 2, 3, 1))                              # [P, Hkv, R G, L]
    sc.masked_fill_(~has[:, None, None, :], -math.inf)
    mp = sc.amax(-1, keepdim=True)
    sc = sc.sub_(mp).exp_()
    lp = sc.sum(-1, keepdim=True)
    ap = torch.matmul(sc, vx.permute(0, 2, 1, 3))                              # [P, Hkv, R G, D]
    del sc

    def by_request(x):   # [P, Hkv, R G, n] -> [B, Hkv, G, n], the prefixes' requests in order
        x = x.view(x.shape[0], hkv, s["req_max"], g, -1).permute(0, 2, 1, 3, 4)
        row = torch.arange(b, device=DEV)
        pre = torch.searchsorted(s["req"][1:], row, right=True)
        return x[pre, row - s["req"][pre]]

    mp, lp, ap = by_request(mp), by_request(lp), by_request(ap)
    ks, vs = _values(ko, own_rows, s["k_scale"]), _values(vo, own_rows, s["v_scale"])   # [B, S, Hkv, D]
    so = torch.matmul(qf.view(b, hkv, g, D), ks.permute(0, 2, 3, 1))           # [B, Hkv, G, S]
    so.masked_fill_(~has_own[:, None, None, :], -math.inf)
    m = torch.maximum(mp, so.amax(-1, keepdim=True))
    po = (so - m).exp()
    f = (mp - m).exp()
    den = lp * f + po.sum(-1, keepdim=True)
    o = (ap * f + torch.matmul(po, vs.permute(0, 2, 1, 3))) / den
    return o.reshape(b, hq, D), (m + den.log()).reshape(b, hq)


def _paged_rows(indptr, ids, at, has, p):
    entry = torch.where(has, indptr[:-1, None] + at[None] // p, 0)
    return torch.where(has, ids[entry] * p + at[None] % p, 0)


def _values(x, rows, scale):
    x = x.view(torch.uint8)[rows].view(x.dtype).float() if x.dtype == torch.float8_e4m3fn else x[rows].float()
    return x if scale is None else x * scale[:, None]


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


def _run_append(s):
    c, n = s["case"], s["n"]
    hq, hkv, p = c["hq"], c["hkv"], c["page"]
    x = s["qkv"].view(-1, hq + 2 * hkv, D)
    q, k, v = x[:, :hq], x[:, hq: hq + hkv], x[:, hq + hkv:]
    if own:
        import split_kv_flashdecoding_gb300 as fd
        args = (s["indptr"], s["kv_indptr"], s["kv_last"], s["kv_ids"])
        kw = dict(rope=s["rope"], positions=s["pos"], q_out=s["q_out"], workspace=s["ws"])
        if c["kv"] == "fp8":
            fd.append_paged_fp8(q, k, v, s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], *args, **kw)
        else:
            fd.append_paged(q, k, v, s["k_pages"], s["v_pages"], *args, **kw)
        return s["q_out"], s["k_pages"], s["v_pages"]
    freq, gain = _frequencies(c)
    ang = s["pos"][:n, None].double() * freq
    cos, sin = (gain * ang.cos()).float()[:, None], (gain * ang.sin()).float()[:, None]
    s["q_out"][:n] = _rotate(q[:n].float(), cos, sin, c["rotary"], c["inter"]).to(torch.bfloat16)
    kr = _rotate(k[:n].float(), cos, sin, c["rotary"], c["inter"])
    # the row of each new token: the last keys of its request's table
    t = torch.arange(n, device=DEV)
    b = torch.searchsorted(s["indptr"][1:], t, right=True)
    cnt = s["kv_indptr"][b + 1] - s["kv_indptr"][b]
    key = (cnt - 1) * p + s["kv_last"][b] - (s["indptr"][b + 1] - t)
    row = s["kv_ids"][s["kv_indptr"][b] + key // p].long() * p + key % p
    if c["kv"] == "fp8":
        for pool, y, sc in ((s["k_pages"], kr, s["k_scale"]), (s["v_pages"], v[:n].float(), s["v_scale"])):
            y = (y / sc[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            pool.view(torch.uint8).view(-1, hkv, D)[row] = y.view(torch.uint8)
    else:
        s["k_pages"].view(-1, hkv, D)[row] = kr.to(torch.bfloat16)
        s["v_pages"].view(-1, hkv, D)[row] = v[:n]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _copy(pools, src, dst):
    """Pages src[i] to dst[i] of every pool; none where src[i] < 0."""
    if own:
        import split_kv_flashdecoding_gb300 as fd
        fd.copy_pages(pools, src, dst)
        return
    none = src < 0
    # a place that no copy writes stands in for the entries that copy nothing
    spare = torch.where(none.all(), 0, torch.where(none, -1, src).amax())
    src, dst = torch.where(none, spare, src), torch.where(none, spare, dst)
    for pool in pools:
        pool[dst] = pool[src]


def _run_fork(s):
    c = s["case"]
    if own:
        import split_kv_flashdecoding_gb300 as fd
        ids, refs, src, dst = fd.fork_pages(s["parent"], s["indptr"], s["last"], s["ids"], s["new_indptr"],
                                            s["entries"], c["page"], s["refs"], workspace=s["ws"])
    else:
        par, refs = s["parent"].long(), s["refs"]
        child = torch.arange(par.numel(), device=DEV)
        old = par.clamp(min=0)
        have = torch.where(par < 0, 0, s["indptr"][old + 1] - s["indptr"][old])
        tail = s["ids"][(s["indptr"][old + 1] - 1).long()]
        # a partly filled last page goes on in its request's first child, where
        # no other request has it, and is copied for every other
        first = torch.full_like(s["last"], par.numel(), dtype=torch.int64).scatter_reduce(
            0, old, torch.where(par < 0, par.numel(), child), "amin")
        part = (have > 0) & (s["last"][old] < c["page"])
        copies = part & ~((first[old] == child) & (refs[tail.long()] == 1))
        e = torch.arange(s["entries"], device=DEV)
        i = torch.searchsorted(s["new_indptr"][1:], e, right=True)
        j = e - s["new_indptr"][i]
        is_tail = j == have[i] - 1
        fresh = (j >= have[i]) | (is_tail & copies[i])
        free = torch.argsort((refs != 0).to(torch.int8), stable=True)
        kept = s["ids"][torch.where(fresh, 0, s["indptr"][old[i]] + j)]
        rank = (torch.cumsum(fresh, 0) - 1).clamp(min=0)
        ids = torch.where(fresh, free[rank].to(torch.int32), kept)
        one = torch.ones_like(ids)
        new_refs = refs.clone().index_add_(0, s["ids"], -torch.ones_like(s["ids"])).index_add_(0, ids, one)
        at = (s["new_indptr"][:-1] + have - 1).clamp(min=0).long()
        src = torch.where(copies, tail, -1)
        dst = torch.where(copies, ids[at], -1)
        refs = new_refs
    _copy(s["pools"], src, dst)
    return [ids, refs, src, dst, *s["pools"]]


def _run_compact(s):
    if own:
        import split_kv_flashdecoding_gb300 as fd
        ids, refs, src, dst = fd.compact_pages(s["refs"], s["ids"], s["most"], limit=s["limit"], workspace=s["ws"])
    else:
        live = s["refs"] > 0
        page = torch.arange(live.numel(), device=DEV)
        limit = s["limit"] if s["limit"] else live.sum()
        mover, slot = live & (page >= limit), ~live & (page < limit)
        slots = torch.argsort((~slot).to(torch.int8), stable=True)
        movers = torch.argsort((~mover).to(torch.int8), stable=True)
        rank = (torch.cumsum(mover, 0) - 1).clamp(min=0)
        to = torch.where(mover, slots[rank], page)
        ids = to[s["ids"]].to(torch.int32)
        refs = torch.zeros_like(s["refs"]).index_add_(0, to, s["refs"])
        k = torch.arange(s["most"], device=DEV) < mover.sum()
        src = torch.where(k, movers[: s["most"]], -1).to(torch.int32)
        dst = torch.where(k, slots[: s["most"]], -1).to(torch.int32)
    _copy(s["pools"], src, dst)
    return [ids, refs, src, dst, *s["pools"]]


# ----------------------------------------------------------------- the work

def work(case):
    c = case
    if c["op"] == "shared":
        req, prefix, own_keys = _shared_lengths(c)
        b, hq, hkv = c["batch"], c["hq"], c["hkv"]
        row = 2 * hkv * D * (1 if c["kv"] == "fp8" else 2)
        keys = int(prefix.sum() + own_keys.sum())
        return {"bytes": keys * row + b * hq * (2 * D + 4 * D + 4),
                "flops": 4.0 * hq * D * float((req * prefix).sum() + own_keys.sum())}
    if c["op"] == "append":
        size = 1 if c["kv"] == "fp8" else 2
        per = D * (4 * c["hq"] + 2 * c["hkv"] * (2 + size))
        return {"bytes": c["new"] * (per + 4) + 12 * c["batch"],
                "flops": 3.0 * c["new"] * c["rotary"] * (c["hq"] + c["hkv"])}
    keys, p = _table_lengths(c), c["page"]
    cnt = -(-keys // p)
    shared_ = np.minimum(cnt[1::2], cnt[: 2 * len(cnt[1::2]): 2]) // 2
    live, page = int(cnt.sum() - shared_.sum()), c["pools"] * p * c["hkv"] * D * 2
    if c["op"] == "fork":
        par, last = _parents(c), keys - (cnt - 1) * p
        ok = par >= 0
        part = ok & (last[par] < p)
        copies = int(part.sum()) - len(set(par[part]))
        out = int(np.where(ok, cnt[par] + (last[par] == p), 2).sum())
        # every reference count in and out, every table entry in and out
        return {"bytes": 2 * copies * page + 8 * c["pages"] + 4 * (int(cnt.sum()) + out + 3 * c["children"]),
                "flops": 1.0 * (c["pages"] + out)}
    limit = c["room"] if c["room"] >= live else live
    # live pages lie anywhere: those behind the limit have to move
    moves = max(1, int(live * (c["pages"] - limit) / c["pages"]))
    return {"bytes": 2 * moves * page + 8 * c["pages"] + 8 * int(cnt.sum()), "flops": 1.0 * c["pages"]}


# ------------------------------------------------- the definitions, 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "shared":
        return _exact_shared(s)
    if c["op"] == "append":
        return _exact_append(s)
    return _exact_table(s)


def _exact_shared(s):
    """Request by request softmax over the request's whole list of keys, the
    prefix's product taken head by head for all of its requests."""
    c = s["case"]
    b, hq, hkv, p = c["batch"], c["hq"], c["hkv"], c["page"]
    g = hq // hkv
    req, prefix, own_keys = _shared_lengths(c)

    def keys(which, i, n):
        if c["paged"]:
            ip, ids = (s["pre_indptr"], s["pre_ids"]) if which == "pre" else (s["kv_indptr"], s["kv_ids"])
            a = int(ip[i])
            rows = (ids[a: a + -(-n // p)].long()[:, None] * p + torch.arange(p, device=DEV)).reshape(-1)[:n]
            return s["k_pages"].view(-1, hkv, D), s["v_pages"].view(-1, hkv, D), rows
        ip = s["pre_indptr"] if which == "pre" else s["kv_indptr"]
        a = int(ip[i])
        rows = torch.arange(a, a + n, device=DEV)
        return (s["k_pre"], s["v_pre"], rows) if which == "pre" else (s["k"], s["v"], rows)

    def head(x, rows, h, scale):
        if x.dtype == torch.float8_e4m3fn:
            x = x.view(torch.uint8)[rows, h].view(torch.float8_e4m3fn)
        else:
            x = x[rows, h]
        return x.double() * (1.0 if scale is None else float(scale[h]))

    o = torch.zeros((b, hq, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((b, hq), dtype=torch.float64, device=DEV)
    r0 = 0
    for i in range(len(req)):
        r1 = r0 + int(req[i])
        kp, vp, rows = keys("pre", i, int(prefix[i]))
        own_lists = [keys("own", r, int(own_keys[r]))[2] for r in range(r0, r1)]
        ko, vo, _ = keys("own", r0, 0)
        flat = torch.cat(own_lists)
        of = torch.repeat_interleave(torch.arange(r1 - r0, device=DEV), _dev(own_keys[r0:r1], torch.int64))
        for h in range(hkv):
            q = s["q"][r0:r1, h * g: (h + 1) * g].double().reshape(-1, D) * s["scale"]
            vals = [head(vp, rows, h, s["v_scale"]), head(vo, flat, h, s["v_scale"])]
            scores = torch.cat([q @ head(kp, rows, h, s["k_scale"]).T, q @ head(ko, flat, h, s["k_scale"]).T], 1)
            mine = (of[None] == torch.arange(r1 - r0, device=DEV).repeat_interleave(g)[:, None])
            scores[:, int(prefix[i]):].masked_fill_(~mine, -math.inf)
            z = torch.logsumexp(scores, 1)
            w = (scores - z[:, None]).exp_()
            o[r0:r1, h * g: (h + 1) * g] = (w @ torch.cat(vals)).view(r1 - r0, g, D)
            lse[r0:r1, h * g: (h + 1) * g] = z.view(r1 - r0, g)
        r0 = r1
    return o, lse


def _exact_append(s):
    """Each pair of a head as a complex number, turned by its angle."""
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
    turn = torch.from_numpy(gain * np.exp(1j * (pos[:, None] * np.array(freq)[None]))).to(DEV)[:, None]
    x = s["qkv"].view(-1, hq + 2 * hkv, D)[:n].double()

    def rotated(y):
        y = y.clone()
        if c["inter"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
        else:
            a, b = y[..., : r // 2], y[..., r // 2: r]
        z = torch.complex(a.contiguous(), b.contiguous()) * turn
        a.copy_(z.real)
        b.copy_(z.imag)
        return y

    q_out = s["q_out"].double()
    q_out[:n] = rotated(x[:, :hq])
    cached, new = _append_lengths(c)
    ids, ip = s["kv_ids"].cpu().numpy(), s["kv_indptr"].cpu().numpy()
    rows = []
    for i in range(c["batch"]):
        key = cached[i] + np.arange(new[i])
        rows.append(ids[ip[i] + key // p].astype(np.int64) * p + key % p)
    rows = _dev(np.concatenate(rows), torch.int64)
    out = []
    for name, y in (("k", rotated(x[:, hq: hq + hkv])), ("v", x[:, hq + hkv:])):
        pool = s[name + "_pages"].float().double().view(-1, hkv, D)
        if c["kv"] == "fp8":
            y = (y / s[name + "_scale"].double()[:, None]).clamp(-448, 448)
        pool[rows] = y
        out.append(pool.view(s[name + "_pages"].shape))
    return q_out, out[0], out[1]


def _exact_table(s):
    """Whole numbers are held equal to the plain form's; the pools are only moved."""
    return None
