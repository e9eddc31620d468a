"""The operators of the paged key-value cache: what is measured, their plain forms, and their values in 64 bits.

Three operators on one paged cache (pages of `page` slots; K and V pools [pages, kv heads, page, head_dim]; one row of page
numbers a request):
  append  new tokens' keys and values into the pages, with per-head RMSNorm and rotary embedding of queries and keys
  attn    attention of one new token a request over its pages, and the attention weight that each slot has received so far
  evict   the slots with the least accumulated weight leave the cache; the others move together

`own = False` runs the plain forms in torch, `own = True` the library's entry points.
"""
import math
import weakref

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "e4m3": 1}
E4M3_MAX = 448.0
ROPE_BASE = 500000.0
EPS = 1e-5


# ------------------------------------------------------------------- cases --
def _append(name, B, lo, hi, start, nq=32, nkv=8, hd=128, page=16, dtype="bf16", cache="bf16", norm=True):
    return dict(name=name, op="append", B=B, lo=lo, hi=hi, start=start, nq=nq, nkv=nkv, hd=hd, page=page, dtype=dtype,
                cache=cache, norm=norm)


def _attn(name, B, lo, hi, nq=32, nkv=8, hd=128, page=16, dtype="bf16", cache="bf16", track=False):
    return dict(name=name, op="attn", B=B, lo=lo, hi=hi, nq=nq, nkv=nkv, hd=hd, page=page, dtype=dtype, cache=cache,
                track=track)


def _evict(name, B, lo, hi, budget, recent, sink, nq=32, nkv=8, hd=128, page=16, dtype="bf16", cache="bf16"):
    return dict(name=name, op="evict", B=B, lo=lo, hi=hi, budget=budget, recent=recent, sink=sink, nq=nq, nkv=nkv, hd=hd,
                page=page, dtype=dtype, cache=cache)


def listed():
    return [
        # one decode step of a full batch: one token a request
        _append("append: one token each, 64", 64, 1, 1, 2304),
        # a step that takes in eight ragged prompts at once
        _append("append: 8 ragged prompts", 8, 511, 1537, 0),
        # a chunk of two long documents far behind their starts, 8-bit cache, no per-head norm
        _append("append: long chunk, e4m3", 2, 8001, 8193, 100000, nq=64, cache="e4m3", page=64, norm=False),
        # one request in a short conversation: latency
        _attn("attn: 1 x 517", 1, 517, 517),
        # a small batch at the decode layer's context range
        _attn("attn: 16 x 512..4096", 16, 512, 4096),
        # a full batch that records the weight each slot receives
        _attn("attn: 64 x 512..4096, weights", 64, 512, 4096, track=True),
        # many short requests of a model without grouped heads; a page that no tile divides
        _attn("attn: 128 x 1..900, fp16 mha", 128, 1, 900, nq=16, nkv=16, hd=64, page=24, dtype="fp16", cache="fp16"),
        # a few very long contexts with an 8-bit cache and eight query heads a key head
        _attn("attn: 8 x 20000..65000, e4m3", 8, 20000, 65000, nq=64, cache="e4m3", page=64),
        # one long request alone
        _attn("attn: 1 x 131071", 1, 131071, 131071, page=32),
        # one request brought back to its budget
        _evict("evict: 1 x 4096 to 1024", 1, 4096, 4096, 1024, 256, 4),
        # a batch of which some requests are still below the budget
        _evict("evict: 32 x 1500..4096 to 2048", 32, 1500, 4096, 2048, 512, 4),
        # long contexts cut to an eighth, 8-bit cache
        _evict("evict: 4 x 65537 to 8192, e4m3", 4, 65537, 65537, 8192, 1000, 0, nq=64, cache="e4m3", page=64),
    ]


def draw(rng):
    most = max(_cost(c) for c in listed())

    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    while True:
        op = rng.choice(["append", "attn", "attn", "evict"])
        hd = rng.choice([64, 128, 128, 128, 256])
        nkv = rng.choice([1, 2, 4, 8, 8, 16])
        group = rng.choice([1, 2, 4, 4, 5, 8, 16])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        dims = dict(nq=nkv * group, nkv=nkv, hd=hd, page=rng.choice([8, 16, 16, 32, 64, 24, 128]), dtype=dtype,
                    cache="e4m3" if rng.random() < 0.3 else dtype)
        B = logint(1, 160)
        if op == "append":
            hi = logint(1, 8000)
            c = _append("", B, rng.randint(1, hi), hi, rng.choice([0, logint(1, 200000)]), norm=rng.random() < 0.5, **dims)
        else:
            hi = logint(8, 140000)
            lo = rng.randint(1, hi)
            if op == "attn":
                c = _attn("", B, lo, hi, track=rng.random() < 0.3, **dims)
            else:
                budget = rng.randint(max(1, hi // 8), hi)
                recent = rng.randint(0, budget)
                c = _evict("", B, lo, hi, budget, recent, rng.randint(0, min(4, budget - recent)), **dims)
        del c["name"]
        if _cost(c) <= most:
            return c


def _lens(c):
    """Lengths evenly spread over lo..hi: every seed gives the same ones, in another order."""
    B = c["B"]
    return [c["hi"]] if B == 1 else [c["lo"] + (c["hi"] - c["lo"]) * i // (B - 1) for i in range(B)]


def _cost(c):
    """Bytes and padded slots of a case, for the bound on drawn ones."""
    w = work(c)
    padded = c["B"] * max(_lens(c)) * c["nkv"] * c["hd"] * 8  # what the plain form holds at once
    return max(w["bytes"], w["flops"] / 50, padded / 8)


def work(c):
    es, ces = BYTES[c["dtype"]], BYTES[c["cache"]]
    nq, nkv, hd, lens = c["nq"], c["nkv"], c["hd"], _lens(c)
    row = nkv * hd
    if c["op"] == "append":
        n = sum(lens)
        return {"bytes": n * (2 * nq * hd * es + 2 * row * es + 2 * row * ces), "flops": 10 * n * (nq + nkv) * hd}
    if c["op"] == "attn":
        n = sum(lens)
        b = n * row * 2 * ces + 2 * c["B"] * nq * hd * es + (8 * n * nkv if c["track"] else 0)
        return {"bytes": b, "flops": 4 * n * nq * hd}
    kept = [min(n, c["budget"]) for n in lens]
    picked = sum(n for n in lens if n > c["budget"])
    return {"bytes": 4 * nkv * picked + sum(kept) * (2 * 2 * row * ces + nkv * (8 + 4)), "flops": 0}


# ------------------------------------------------------------------ inputs --
def _pool(c, gen, n_pages, std=1.0):
    shape = (n_pages, c["nkv"], c["page"], c["hd"])
    x = torch.empty(shape, dtype=DTYPES[c["dtype"]], device="cuda").normal_(0.0, std, generator=gen)
    return x.to(DTYPES[c["cache"]])


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, B, nq, nkv, hd, page = DTYPES[c["dtype"]], c["B"], c["nq"], c["nkv"], c["hd"], c["page"]
    lens = rng.permutation(np.array(_lens(c)))
    cols = -(-int(lens.max()) // page)
    used = -(-lens // page)
    n_dst = -(-np.minimum(lens, c["budget"]) // page) if c["op"] == "evict" else np.zeros(B, np.int64)
    n_pages = int(used.sum() + n_dst.sum()) + 3
    free = rng.permutation(n_pages).astype(np.int32)
    table, dst = np.full((B, cols), -1, np.int32), np.full((B, cols), -1, np.int32)
    at = np.arange(cols)
    table[at < used[:, None]] = free[:int(used.sum())]
    dst[at < n_dst[:, None]] = free[int(used.sum()):int(used.sum() + n_dst.sum())]
    quant = c["cache"] == "e4m3"
    s = dict(c=c, K=_pool(c, gen, n_pages, 32.0 if quant else 1.0), V=_pool(c, gen, n_pages, 32.0 if quant else 1.0),
             table=torch.from_numpy(table).cuda(), lens=torch.from_numpy(lens.astype(np.int32)).cuda(), k_scale=None,
             v_scale=None, acc=None, max_len=int(lens.max()))
    if quant:  # one scale a key-value head, as a calibration leaves them
        s["k_scale"] = (0.9 + 0.2 * torch.rand(nkv, generator=gen, device="cuda")) / 32.0
        s["v_scale"] = (0.9 + 0.2 * torch.rand(nkv, generator=gen, device="cuda")) / 32.0
    if c["op"] == "append":
        n = int(lens.sum())
        req = np.repeat(np.arange(B), lens)
        slot = np.arange(n) - np.repeat(np.cumsum(lens) - lens, lens)
        qkv = torch.empty(n, (nq + 2 * nkv) * hd, dtype=dt, device="cuda").normal_(0.0, 1.0, generator=gen)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, hd)) for x in qkv.split([nq * hd, nkv * hd, nkv * hd], 1))
        s["q_out"] = torch.zeros(n, nq, hd, dtype=dt, device="cuda")
        s["req"] = torch.from_numpy(req.astype(np.int32)).cuda()
        s["slots"] = torch.from_numpy(slot.astype(np.int32)).cuda()
        s["pos"] = torch.from_numpy((slot + c["start"]).astype(np.int32)).cuda()
        gains = torch.empty(2, hd, dtype=dt, device="cuda").normal_(1.0, 0.1, generator=gen)
        s["gq"], s["gk"] = (gains[0], gains[1]) if c["norm"] else (None, None)
    if c["op"] == "attn":
        s["q"] = torch.empty(B, nq, hd, dtype=dt, device="cuda").normal_(0.0, 1.0, generator=gen)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, nq, device="cuda")
    if c["op"] == "evict" or c.get("track"):
        # weights gathered over a few hundred steps: most slots got little, some much
        s["acc"] = torch.empty(n_pages, nkv, page, device="cuda").exponential_(generator=gen) ** 3 / max(1, s["max_len"])
    if c["op"] == "evict":
        s["dst"] = torch.from_numpy(dst).cuda()
        s["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros(B, nkv, c["budget"], dtype=torch.int32, device="cuda")
    if own:
        s["kv"], s["pool"] = _handle(s, n_pages)
    return s


class _Kv:
    """A handle of the library that goes with its last user."""

    def __init__(self, et, *a, **k):
        self.et, self.h = et, et.et_build_kv(*a, **k)
        weakref.finalize(self, et.et_destroy_kv, self.h)  # at the interpreter's end too, while the library is still there


def _handle(s, n_pages):
    import event_driven_persistent_b200 as et
    c = s["c"]
    kv = _Kv(et, c["B"], s["max_len"], n_pages, page_size=c["page"], n_heads=c["nq"], n_kv_heads=c["nkv"], head_dim=c["hd"],
             dtype=c["dtype"], cache_dtype=c["cache"], track_weights=int(bool(c.get("track"))), rope_base=ROPE_BASE, rms_eps=EPS)
    return kv, et.et_kv_pool(kv.h, s["K"], s["V"], k_scale=s["k_scale"], v_scale=s["v_scale"], acc=s["acc"])


# --------------------------------------------------------------- operators --
def run(s):
    op = s["c"]["op"]
    if own:
        et, h = s["kv"].et, s["kv"].h
        if op == "append":
            et.et_run_kv_append(h, s["pool"], s["table"], s["slots"], s["k"], s["v"], q=s["q"], q_out=s["q_out"],
                                pos=s["pos"], req=s["req"], gq=s["gq"], gk=s["gk"])
        elif op == "attn":
            et.et_run_kv_attn(h, s["pool"], s["table"], s["lens"], s["q"], s["out"], lse=s["lse"], accumulate=s["c"]["track"])
        else:
            et.et_run_kv_evict(h, s["pool"], s["table"], s["lens"], s["c"]["budget"], s["dst"], s["new_lens"],
                               kept=s["kept"], n_recent=s["c"]["recent"], n_sink=s["c"]["sink"])
    else:
        {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}[op](s)
    if op == "append":
        return s["q_out"], s["K"], s["V"]
    if op == "attn":
        return (s["out"], s["lse"], s["acc"]) if s["c"]["track"] else (s["out"], s["lse"])
    return s["kept"], s["new_lens"], s["K"], s["V"], s["acc"]


def _rms(x, gain):
    return x if gain is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.float()


def _rotate(x, pos):
    half = x.shape[-1] // 2
    freq = ROPE_BASE ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    angle = pos.double()[:, None, None] * freq  # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _store(x, scale, dtype):
    if dtype != torch.float8_e4m3fn:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(dtype)


def _put(pool, page, slot, rows):
    """pool[page, :, slot] = rows, by bytes where the type has no indexing of its own."""
    if pool.dtype == torch.float8_e4m3fn:
        pool, rows = pool.view(torch.uint8), rows.view(torch.uint8)
    pool[page, :, slot] = rows


def _plain_append(s):
    page = s["c"]["page"]
    q, k = (_rotate(_rms(x.float(), g), s["pos"]) for x, g in ((s["q"], s["gq"]), (s["k"], s["gk"])))
    s["q_out"].copy_(q)
    slot = s["slots"].long()
    at = s["table"][s["req"].long(), slot // page].long()
    _put(s["K"], at, slot % page, _store(k, s["k_scale"], s["K"].dtype))
    _put(s["V"], at, slot % page, _store(s["v"].float(), s["v_scale"], s["V"].dtype))


def _rows(s, pool, scale):
    """A pool's rows by request: fp32 [B, kv heads, slots, hd]."""
    x = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
    x = x[s["table"].clamp(min=0).long()].view(pool.dtype).float()
    x = x.transpose(1, 2).flatten(2, 3)
    return x if scale is None else x * scale[:, None, None]


def _plain_attn(s):
    c = s["c"]
    B, nq, nkv, hd, page = c["B"], c["nq"], c["nkv"], c["hd"], c["page"]
    K = _rows(s, s["K"], s["k_scale"])
    there = (torch.arange(K.shape[2], device="cuda") < s["lens"][:, None])[:, None]  # [B, 1, slots]
    x = s["q"].float().view(B, nkv, nq // nkv, hd) @ K.transpose(2, 3) / math.sqrt(hd)
    del K
    x = x.masked_fill(~there[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    p = p / total
    s["lse"].copy_((top + total.log()).view(B, nq))
    if c["track"]:
        slots = torch.arange(p.shape[-1], device="cuda")
        at = s["table"].long()[:, None, slots // page].expand(B, nkv, -1)
        head = torch.arange(nkv, device="cuda")[None, :, None].expand_as(at)
        inside = there.expand_as(at)
        s["acc"].index_put_((at[inside], head[inside], (slots % page).expand_as(at)[inside]), p.sum(2)[inside], accumulate=True)
    V = _rows(s, s["V"], s["v_scale"]).masked_fill(~there[..., None], 0.0)
    s["out"].copy_((p @ V).view(B, nq, hd))


def _plain_evict(s):
    c = s["c"]
    page, budget = c["page"], c["budget"]
    acc = s["acc"][s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2)  # [B, kv heads, slots]
    slots = torch.arange(acc.shape[2], device="cuda")
    lens = s["lens"][:, None, None]
    held = (slots < c["sink"]) | (slots >= lens - c["recent"])
    rank = acc.masked_fill(held, math.inf).masked_fill(slots >= lens, -math.inf)
    kept = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    place = torch.arange(budget, device="cuda")
    new = lens.clamp(max=budget)
    if kept.shape[-1] < budget:
        kept = torch.cat([kept, kept.new_zeros(*kept.shape[:2], budget - kept.shape[-1])], -1)
    kept = kept.masked_fill(place >= new, 1 << 40).sort(dim=-1).values
    inside = place < new
    s["kept"].copy_(kept.masked_fill(~inside.expand_as(kept), -1))
    s["new_lens"].copy_(new.view(-1))
    b, h, j = inside.expand_as(kept).nonzero(as_tuple=True)
    src = kept[b, h, j]
    at, to = s["table"][b, src // page].long(), s["dst"][b, j // page].long()
    for name in ("K", "V", "acc"):
        x = s[name].view(torch.uint8) if s[name].dtype == torch.float8_e4m3fn else s[name]
        x[to, h, j % page] = x[at, h, src % page]


# ---------------------------------------------------------- values in 64 bits --
def exact(case, seed):
    global own
    before, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = before
    return {"append": _exact_append, "attn": _exact_attn, "evict": _exact_evict}[case["op"]](s)


def _f64(pool):
    return pool.float().double()


def _exact_append(s):
    page, half = s["c"]["page"], s["c"]["hd"] // 2
    pos = s["pos"].cpu().numpy().astype(np.float64)
    turn = np.exp(1j * pos[:, None] * np.power(ROPE_BASE, -np.arange(half) / half))  # e^(i angle)
    turn = torch.from_numpy(turn).cuda()[:, None]

    def turned(x, g):
        x = x.double()
        if g is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * g.double()
        z = torch.complex(x[..., :half], x[..., half:]) * turn
        return torch.cat([z.real, z.imag], -1)

    out = [turned(s["q"], s["gq"])]
    slot = s["slots"].long()
    at = s["table"][s["req"].long(), slot // page].long()
    for name, x, scale in (("K", turned(s["k"], s["gk"]), s["k_scale"]), ("V", s["v"].double(), s["v_scale"])):
        pool = _f64(s[name])
        pool[at, :, slot % page] = x if scale is None else (x / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        out.append(pool)
    return tuple(out)


def _exact_attn(s):
    c = s["c"]
    if work(c)["bytes"] > 4e9:
        return None
    nkv, hd, page = c["nkv"], c["hd"], c["page"]
    acc = s["acc"].double() if c["track"] else None
    outs, lses = [], []
    for b, n in enumerate(s["lens"].tolist()):
        pages = s["table"][b, : -(-n // page)].long()

        def rows(pool, scale):
            x = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool
            x = _f64(x[pages].view(pool.dtype)).permute(1, 0, 2, 3).reshape(nkv, -1, hd)[:, :n]
            return x if scale is None else x * scale.double()[:, None, None]

        q = s["q"][b].double().view(nkv, -1, hd)
        x = torch.einsum("hgd,hnd->hgn", q, rows(s["K"], s["k_scale"])) / math.sqrt(hd)
        lse = torch.logsumexp(x, -1)
        p = torch.exp(x - lse[..., None])
        outs.append(torch.einsum("hgn,hnd->hgd", p, rows(s["V"], s["v_scale"])).reshape(-1, hd))
        lses.append(lse.reshape(-1))
        if acc is not None:
            w = torch.zeros(nkv, len(pages) * page, dtype=torch.float64, device="cuda")
            w[:, :n] = p.sum(1)
            acc[pages] += w.view(nkv, -1, page).transpose(0, 1)
    out = (torch.stack(outs), torch.stack(lses))
    return out + (acc,) if acc is not None else out


def _exact_evict(s):
    c = s["c"]
    page, budget, nkv = c["page"], c["budget"], c["nkv"]
    table, dst, lens = (s[k].cpu().numpy() for k in ("table", "dst", "lens"))
    acc = s["acc"].cpu().numpy()
    kept = np.full((c["B"], nkv, budget), -1, np.int64)
    src, to = [], []
    for b, n in enumerate(lens):
        for h in range(nkv):
            keep = np.arange(n)
            if n > budget:
                weights = acc[table[b, : -(-n // page)], h].reshape(-1)[:n]
                mid = np.arange(c["sink"], n - c["recent"])
                best = mid[np.lexsort((mid, -weights[mid]))][: budget - c["sink"] - c["recent"]]
                keep = np.sort(np.concatenate([keep[: c["sink"]], best, keep[n - c["recent"]:]]))
            kept[b, h, : len(keep)] = keep
            j = np.arange(len(keep))
            src.append(np.stack([table[b, keep // page], np.full_like(keep, h), keep % page]))
            to.append(np.stack([dst[b, j // page], np.full_like(j, h), j % page]))
    src, to = (torch.from_numpy(np.concatenate(x, 1)).long().cuda() for x in (src, to))
    out = [torch.from_numpy(kept).cuda(), torch.from_numpy(np.minimum(lens, budget)).cuda()]
    for name in ("K", "V", "acc"):
        x = _f64(s[name])
        x[to[0], to[1], to[2]] = x[src[0], src[1], src[2]]
        out.append(x)
    return tuple(out)
