"""An INT8 paged cache with a scale per page and KV head, and attention over it
in 64 bits, written out for the tests."""
import math

import numpy as np
import torch

import split_kv_flashdecoding_gb300 as fd

D = 128


def indptr(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


def tables(keys, page, rng, spare=3):
    """Page tables (host int32) of requests with these many keys; pages anywhere."""
    keys = np.asarray(keys, dtype=np.int64)
    cnt = -(-keys // page)
    pages = int(cnt.sum()) + spare
    ids = rng.permutation(pages)[: int(cnt.sum())]
    return dict(keys=keys, page=page, num_pages=pages, ip=indptr(cnt),
                last=np.where(cnt > 0, keys - (cnt - 1) * page, 0).astype(np.int32),
                ids=np.append(ids, 0).astype(np.int32))


def cache(t, hkv, rng, dev, kind="quantised"):
    """Pools and scales: normal values quantised as an append does, or every code
    with scales of either sign."""
    n, p = t["num_pages"], t["page"]
    out = {}
    for x in ("k", "v"):
        if kind == "quantised":
            val = rng.standard_normal((n, p, hkv, D)) * (0.3 + 2 * rng.random_sample((n, 1, hkv, 1)))
            sc = (np.abs(val).max(axis=(1, 3)) / 127).astype(np.float32)
            codes = np.rint(val / sc[:, None, :, None])
        else:
            codes = rng.randint(-128, 128, (n, p, hkv, D))
            sc = (rng.random_sample((n, hkv)) * 0.03 * rng.choice([-1, 1], (n, hkv))).astype(np.float32)
        scale = np.zeros((n, fd.scale_heads(hkv)), dtype=np.float32)
        scale[:, :hkv] = sc
        out[x] = torch.from_numpy(codes.astype(np.int8)).to(dev)
        out[x + "s"] = torch.from_numpy(scale).to(dev)
    return out


def dev_tables(t, dev):
    return [torch.from_numpy(t[x]).to(dev) for x in ("ip", "last", "ids")]


def values(t, c, b, h):
    """K and V of request b and head h, fp64 [keys, D]."""
    ids = torch.from_numpy(t["ids"][t["ip"][b]: t["ip"][b + 1]].astype(np.int64)).to(c["k"].device)
    n = int(t["keys"][b])
    return [(c[x][ids, :, h].double() * c[x + "s"][ids, h].double()[:, None, None]).reshape(-1, D)[:n]
            for x in ("k", "v")]


def attention(q, t, c, scale, ends=None, causal=False):
    """fp64 O and LSE of query rows ends[b] .. ends[b + 1] (None: one a request);
    a causal request's rows are its last keys'.  No keys: O = 0, LSE = -inf."""
    batch = len(t["keys"])
    ends = np.arange(batch + 1) if ends is None else ends
    hq, hkv = q.shape[1], c["k"].shape[2]
    g = hq // hkv
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for b in range(batch):
        a, e, n = int(ends[b]), int(ends[b + 1]), int(t["keys"][b])
        if a == e or n == 0:
            continue
        for h in range(hkv):
            k, v = values(t, c, b, h)
            s = torch.einsum("tgd,nd->tgn", q[a:e, h * g: (h + 1) * g].double(), k) * scale
            if causal:
                pos = n - (e - a) + torch.arange(e - a, device=q.device)
                s.masked_fill_(torch.arange(n, device=q.device)[None, None] > pos[:, None, None], -math.inf)
            z = torch.logsumexp(s, -1)
            w = torch.where(z[..., None] == -math.inf, 0.0, (s - z[..., None]).exp())
            o[a:e, h * g: (h + 1) * g] = w @ v
            lse[a:e, h * g: (h + 1) * g] = z
    return o, lse
