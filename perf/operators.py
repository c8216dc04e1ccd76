"""What the operators of the cached-history path are measured on: per-head norm and rotation (forward and
backward), writing K|V rows to a paged cache and reading them back, and attention over that cache.

`listed()` names the measured cases and `draw(rng)` gives more of the same ranges; `prepare` makes a case's
inputs from a seed, `run` is one pass (the library's calls where `own` is true, elementary torch operations in
32 bits otherwise), `exact` the same result in 64 bits, and `work` what one pass cannot do without.

Conventions. Sequence b of a chunk has `new[b]` rows, packed one sequence after another, and `length[b]` positions in the
cache, of which its rows are the last new[b] (append, read, causal attention). A cache page holds, for each
plane (K, V) and K|V head, `page` rows of d_head numbers; an e4m3 row stands for its numbers times a power
of two of its own.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6
E_LO, E_HI = -100, 119  # exponents a row's scale may have


# ----------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------
def listed():
    return [
        # one request's 16 tokens meet one new event: latency alone counts
        dict(name="norm_rotate request", op="norm_rotate", dtype="bf16", heads=8, kv_heads=8, dh=32, rows_q=16, rows_k=1,
             rot=32, layout="halves", pos=15000),
        # a training batch of the 15k-history workload (d 512, 8 heads): 64 x 32 queries, the keys of 403481
        # history rows, read where the K|V projection left them (row stride 1024)
        dict(name="norm_rotate hist15k", op="norm_rotate", dtype="bf16", heads=8, kv_heads=8, dh=64, rows_q=2048,
             rows_k=403481, rot=64, layout="halves", pos=15000),
        # fp32 mode, half of each head rotated, neighbouring columns paired, far positions, row counts of no tile
        dict(name="norm_rotate_backward fp32", op="norm_rotate_backward", dtype="fp32", grad="fp32", heads=8, kv_heads=8,
             dh=32, rows_q=1021, rows_k=60013, rot=16, layout="adjacent", pos=1 << 20),
        # the gradients of a quarter of that batch's queries and keys, bf16
        dict(name="norm_rotate_backward hist15k", op="norm_rotate_backward", dtype="bf16", grad="bf16", heads=8,
             kv_heads=8, dh=64, rows_q=512, rows_k=109605, rot=64, layout="halves", pos=15000),
        # serving: every user of a batch of 64 has one new event
        dict(name="append event", op="append", fmt="e4m3", heads=8, kv_heads=8, dh=64, shared=False, page=64, B=64,
             lens="hist15k", seed=4, new_lo=1, new_hi=1),
        # filling the cache with the histories of 24 users (d 512)
        dict(name="append histories", op="append", fmt="e4m3", heads=8, kv_heads=8, dh=64, shared=False, page=64, B=24,
             lens="hist15k", seed=5, new_lo=-1, new_hi=-1),
        # the last rows of a few users back as bf16 from a bf16 cache of small pages (a recompute of their tail)
        dict(name="read tails", op="read", fmt="bf16", heads=4, kv_heads=4, dh=32, shared=False, page=16, B=5,
             lens="stack", seed=6, new_lo=1, new_hi=301),
        # whole histories back (d 256, histories of 3000 to 6000 rows)
        dict(name="read histories", op="read", fmt="e4m3", heads=8, kv_heads=8, dh=32, shared=False, page=128, B=48,
             lens="stack", seed=7, new_lo=-1, new_hi=-1),
        # one request, one token, four query heads to a K|V head: the smallest attention
        dict(name="attend request", op="attend", fmt="bf16", heads=8, kv_heads=2, dh=64, shared=False, page=64, B=1,
             lens="stack", seed=8, new_lo=1, new_hi=1, causal=True),
        # one new event of each of 64 users against histories of up to 15000 rows
        dict(name="attend event hist15k", op="attend", fmt="bf16", heads=8, kv_heads=8, dh=64, shared=False, page=64,
             B=64, lens="hist15k", seed=4, new_lo=1, new_hi=1, causal=True),
        # the 15k-history workload's own queries (32 tokens per user, no mask) over the e4m3 cache
        dict(name="attend tokens hist15k", op="attend", fmt="e4m3", heads=8, kv_heads=8, dh=64, shared=False, page=64,
             B=64, lens="hist15k", seed=4, new_lo=32, new_hi=32, causal=False),
        # chunks of new events of four users, each event seeing what came before it (d 256)
        dict(name="attend chunks", op="attend", fmt="bf16", heads=8, kv_heads=8, dh=32, shared=False, page=128, B=4,
             lens="hist15k", seed=9, new_lo=700, new_hi=4096, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        w = work(c)
        if not c["op"].startswith("norm_rotate") and not _lengths(c)[1].any():
            continue  # nothing new in any sequence: no output
        if w["bytes"] <= 8.2e8 and w["flops"] <= 5e10 and _dense(c) <= 8e8:
            return c


def _draw(rng):
    op = rng.choice(["norm_rotate", "norm_rotate_backward", "append", "read", "attend", "attend"])
    heads, dh = rng.choice([4, 8, 8, 16]), rng.choice([32, 64])
    if op.startswith("norm_rotate"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        c = dict(op=op, dtype=dtype, heads=heads, kv_heads=rng.choice([heads, heads, heads // 4]), dh=dh,
                 rows_q=_log(rng, 1, 20000), rows_k=_log(rng, 1, 200000), rot=rng.choice([dh, dh, dh // 2, 16]),
                 layout=rng.choice(["halves", "adjacent"]), pos=_log(rng, 2, 1 << 20))
        if op == "norm_rotate_backward":
            c["grad"] = "fp32" if dtype == "fp32" else rng.choice(["bf16", "fp32"])
        return c
    c = dict(op=op, fmt=rng.choice(["bf16", "e4m3"]), heads=heads, kv_heads=rng.choice([heads, heads, heads // 4]), dh=dh,
             shared=rng.random() < 0.2, page=rng.choice([16, 32, 64, 128, 256]), B=_log(rng, 1, 96),
             lens=rng.choice(["hist15k", "stack", "any"]), seed=rng.randrange(1 << 20))
    if op == "attend":
        hi = _log(rng, 1, 3000)
        c |= dict(new_lo=rng.choice([hi, max(1, hi // 4), 0]), new_hi=hi, causal=rng.random() < 0.6)
    elif rng.random() < 0.5:
        c |= dict(new_lo=-1, new_hi=-1)
    else:
        c |= dict(new_lo=0, new_hi=_log(rng, 1, 2000))
    return c


def _lengths(c):
    """(cached positions, new rows) of each sequence, from the case alone."""
    g = np.random.default_rng(c["seed"])
    if c["lens"] == "hist15k":
        n = np.clip(np.round(g.lognormal(math.log(6000.0), 0.5, c["B"])), 64, 15000).astype(np.int64)
    elif c["lens"] == "stack":
        n = g.integers(3000, 6001, c["B"])
    else:
        n = np.round(np.exp(g.uniform(0, math.log(9000.0), c["B"]))).astype(np.int64)
    new = n.copy() if c["new_lo"] < 0 else g.integers(c["new_lo"], c["new_hi"] + 1, c["B"])
    if c["op"] != "attend" or c["causal"]:
        new = np.minimum(new, n)
    return n, new


def _dense(c):
    """Scores of the padded plain form."""
    if c["op"] != "attend":
        return 0
    n, new = _lengths(c)
    return c["B"] * c["heads"] * int(n.max()) * max(1, int(new.max()))


def work(c):
    if c["op"].startswith("norm_rotate"):
        es, rows = (4 if c["dtype"] == "fp32" else 2), c["rows_q"] + c["rows_k"]
        n = (c["rows_q"] * c["heads"] + c["rows_k"] * c["kv_heads"]) * c["dh"]
        if c["op"] == "norm_rotate":
            return {"bytes": 2 * n * es + 4 * rows + 8 * c["dh"], "flops": 8 * n}
        gs = 4 if c["grad"] == "fp32" else 2
        return {"bytes": n * (es + 2 * gs) + 4 * rows + 16 * c["dh"], "flops": 16 * n}
    n, new = _lengths(c)
    planes = 1 if c["shared"] else 2
    row = planes * c["kv_heads"] * (2 * c["dh"] if c["fmt"] == "bf16" else c["dh"] + 1)  # one cached position
    tables = 4 * int(np.sum(-(-n // c["page"])))
    t = int(new.sum())
    if c["op"] != "attend":
        vals = t * planes * c["kv_heads"] * c["dh"]
        return {"bytes": t * row + 2 * vals + tables, "flops": 2 * vals}
    pairs = int(np.sum(new * n - (new * (new - 1) // 2 if c["causal"] else 0)))
    return {"bytes": int(n[new > 0].sum()) * row + 4 * t * c["heads"] * c["dh"] + tables,
            "flops": 4 * pairs * c["heads"] * c["dh"]}


# ----------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------
def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 11)
    rand = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device=DEV, dtype=torch.float32).to(dtype)  # noqa: E731
    if c["op"].startswith("norm_rotate"):
        dt = _dt(c["dtype"])
        s = {"case": c}
        for part, rows, h in (("q", c["rows_q"], c["heads"]), ("k", c["rows_k"], c["kv_heads"])):
            width = h * c["dh"]
            # keys are the first half of K|V rows, as the projection leaves them
            x = rand(rows, width if part == "q" else 2 * width, dtype=dt)[:, :width]
            s["x" + part] = x
            s["g" + part] = 0.5 + torch.rand(c["dh"], generator=g, device=DEV)
            s["p" + part] = torch.randint(0, c["pos"], (rows,), generator=g, device=DEV, dtype=torch.int32)
            if c["op"] == "norm_rotate_backward":
                s["d" + part] = rand(rows, width, dtype=_dt(c["grad"]))
        return s
    n, new = _lengths(c)
    planes = 1 if c["shared"] else 2
    P, hk, dh = c["page"], c["kv_heads"], c["dh"]
    need = -(-n // P)
    n_pages = int(need.sum()) + 3
    order = np.random.default_rng(seed).permutation(n_pages)
    stride = int(need.max()) + 1
    table = np.zeros((c["B"], stride), np.int32)
    at = 0
    for b in range(c["B"]):
        table[b, : need[b]] = order[at : at + need[b]]
        at += need[b]
    off = np.concatenate([[0], np.cumsum(new)])
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)  # noqa: E731
    s = {"case": c, "table": dev(table), "offsets": dev(off), "lengths": dev(n), "total": int(off[-1]),
         "max_new": int(new.max()), "max_len": int(n.max()), "pages": None, "scales": None, "n_pages": n_pages}
    shape = (n_pages, planes, hk, P, dh)
    if c["op"] == "append":
        s["pages"] = torch.zeros(shape, device=DEV, dtype=torch.bfloat16 if c["fmt"] == "bf16" else torch.uint8)
        s["scales"] = torch.full(shape[:4], 127, device=DEV, dtype=torch.uint8) if c["fmt"] == "e4m3" else None
        # rows of different sizes, as projected states are: the scales differ from row to row
        kv = rand(s["total"], planes * hk * dh)
        s["kv"] = kv * torch.exp(0.5 * rand(s["total"], 1))
        return s
    if c["fmt"] == "bf16":
        s["pages"] = rand(*shape)
    else:
        s["pages"] = torch.empty(shape, device=DEV, dtype=torch.uint8)
        s["scales"] = torch.empty(shape[:4], device=DEV, dtype=torch.uint8)
        for lo in range(0, n_pages, 1024):
            v = torch.randn(min(1024, n_pages - lo), *shape[1:], generator=g, device=DEV)
            s["pages"][lo : lo + 1024], s["scales"][lo : lo + 1024] = _quantise(v)
    if c["op"] == "attend":
        s["q"] = rand(s["total"], c["heads"] * dh)
    return s


# ----------------------------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------------------------
def _quantise(x):
    """Rows of fp32 numbers -> (e4m3 bytes, scale codes): the smallest power of two that brings the row into +-448."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m * 2 <= 1.75, e - 9, e - 8).clamp(E_LO, E_HI)
    e = torch.where(m == 0, torch.zeros_like(e), e)
    v = (x * torch.exp2(-e.float())[..., None]).clamp(-448.0, 448.0)
    return v.to(torch.float8_e4m3fn).view(torch.uint8), (e + 127).to(torch.uint8)


def _rotate(n, pos, c, sign):
    """Heads n [rows, h, dh] (fp32) turned by sign * position * 10000^(-2 i / rot)."""
    rot = c["rot"]
    i = torch.arange(rot // 2, device=n.device, dtype=torch.float64)
    a = pos.double()[:, None] * torch.exp2(i * (-2.0 / rot * math.log2(10000.0)))
    cos, sin = torch.cos(a).float()[:, None, :], (sign * torch.sin(a)).float()[:, None, :]
    if c["layout"] == "halves":
        u, v = n[..., : rot // 2], n[..., rot // 2 : rot]
        return torch.cat([u * cos - v * sin, u * sin + v * cos, n[..., rot:]], -1)
    u, v = n[..., 0:rot:2], n[..., 1:rot:2]
    return torch.cat([torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2), n[..., rot:]], -1)


def _heads(x, c):
    return x.float().reshape(x.shape[0], -1, c["dh"])


def _norm_rotate(x, gain, pos, c):
    x32 = _heads(x, c)
    n = x32 * torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS) * gain
    return _rotate(n, pos, c, 1.0).flatten(1).to(x.dtype)


def _norm_rotate_backward(x, gain, pos, dy, c):
    x32 = _heads(x, c)
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    dn = _rotate(_heads(dy, c), pos, c, -1.0)
    dg = (dn * x32 * r).sum((0, 1), dtype=torch.float64).float()
    dn = dn * gain
    dx = r * dn - x32 * (r * r * r) * (dn * x32).mean(-1, keepdim=True)
    return dx.flatten(1).to(dy.dtype), dg


def _slots(s):
    """Page and row within the page of every row of the chunk."""
    r = torch.arange(s["total"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(s["offsets"], r, right=True) - 1
    pos = (s["lengths"][b] - s["offsets"][b + 1] + r).long()
    P = s["case"]["page"]
    return s["table"][b, pos // P].long(), pos % P


def _append(s):
    c = s["case"]
    page, slot = _slots(s)
    v = s["kv"].reshape(s["total"], -1, c["kv_heads"], c["dh"])
    if c["fmt"] == "bf16":
        s["pages"][page, :, :, slot] = v
    else:
        s["pages"][page, :, :, slot], s["scales"][page, :, :, slot] = _quantise(v.float())
    return _stored(s)


def _stored(s):
    if s["scales"] is None:
        return {"pages": s["pages"]}
    return {"pages": s["pages"].view(torch.float8_e4m3fn), "scales": s["scales"].view(torch.float8_e8m0fnu)}


def _values(s, page, slot):
    """Cached rows as fp32, [..., planes, kv_heads, dh]."""
    v = s["pages"][page, :, :, slot]
    if s["scales"] is None:
        return v.float()
    return v.view(torch.float8_e4m3fn).float() * torch.exp2(s["scales"][page, :, :, slot].float() - 127.0)[..., None]


def _attend(s):
    c = s["case"]
    B, T, L, dh, hk = c["B"], s["max_new"], s["max_len"], c["dh"], c["kv_heads"]
    G = c["heads"] // hk
    i, j = torch.arange(T, device=DEV), torch.arange(L, device=DEV)
    n, new = s["lengths"].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    real = i[None] < new[:, None]
    at = torch.where(real, s["offsets"][:-1, None].long() + i[None], s["total"])
    q = torch.cat([s["q"].float(), torch.zeros(1, c["heads"] * dh, device=DEV)])[at].reshape(B, T, hk, G, dh)
    page = s["table"][:, : -(-L // c["page"])].long()[:, j // c["page"]]
    kv = _values(s, page, (j % c["page"])[None].expand(B, L))  # [B, L, planes, hk, dh]
    k, v = kv[:, :, 0], kv[:, :, -1]
    seen = j[None, None] < n[:, None, None]
    if c["causal"]:
        seen = seen & (j[None, None] <= (n - new)[:, None, None] + i[None, :, None])
    seen = seen[:, None]  # [B, 1, T or 1, L]
    sc = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, hk, G * T, dh), k.permute(0, 2, 3, 1)).reshape(B, hk * G, T, L)
    sc = (sc * (dh ** -0.5)).masked_fill_(~seen, -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-1e30))
    a = torch.matmul(p.reshape(B, hk, G * T, L), v.permute(0, 2, 1, 3)).reshape(B, hk * G, T, dh)
    a = a / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return a.permute(0, 2, 1, 3).reshape(B, T, -1)[real].to(torch.bfloat16)


# ----------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------
def run(s):
    c = s["case"]
    if own:
        return _own(s)
    if c["op"] == "norm_rotate":
        return {p: _norm_rotate(s["x" + p], s["g" + p], s["p" + p], c) for p in "qk"}
    if c["op"] == "norm_rotate_backward":
        return {p: _norm_rotate_backward(s["x" + p], s["g" + p], s["p" + p], s["d" + p], c) for p in "qk"}
    if c["op"] == "append":
        return _append(s)
    if c["op"] == "read":
        page, slot = _slots(s)
        return _values(s, page, slot).flatten(1).to(torch.bfloat16)
    return _attend(s)


def _plan(s):
    """What a program keeps from call to call: the descriptors, the workspace and the output buffers."""
    from wukong_hstu_cross_b200 import whale as W

    c = s["case"]
    buf = lambda nbytes: torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=DEV)  # noqa: E731
    if c["op"].startswith("norm_rotate"):
        cfg = W.make_config(1, c["heads"] * c["dh"], c["heads"], 1, 64, 64, W.WHALE_FP32 if c["dtype"] == "fp32" else W.WHALE_BF16, eps=EPS)
        rotary = W.make_rotary(c["rot"], layout=W.WHALE_ROTATE_HALVES if c["layout"] == "halves" else W.WHALE_ROTATE_ADJACENT)
        if c["op"] == "norm_rotate":
            out = {p: torch.empty_like(s["x" + p], memory_format=torch.contiguous_format) for p in "qk"}
            parts = [W.head_rows(s["x" + p], s["g" + p], s["p" + p], y=out[p]) for p in "qk"]
            return lambda: W.whale_norm_rotate(cfg, rotary, *parts), out
        out = {p: (torch.empty_like(s["d" + p]), torch.empty(c["dh"], device=DEV)) for p in "qk"}
        parts = [W.head_rows(s["x" + p], s["g" + p], s["p" + p]) for p in "qk"]
        grads = [W.head_grads(s["d" + p], out[p][0], out[p][1]) for p in "qk"]
        gt = W.WHALE_FP32 if c["grad"] == "fp32" else W.WHALE_BF16
        ws = buf(W.whale_norm_rotate_workspace_size(cfg, *parts))
        return lambda: W.whale_norm_rotate_backward(cfg, rotary, *parts, *grads, gt, ws), out
    cfg = W.make_config(1, c["heads"] * c["dh"], c["heads"], 1, 64, 64, W.WHALE_BF16, flags=W.WHALE_SHARED_KV if c["shared"] else 0)
    cache = W.make_cache(s["pages"], s["scales"])
    chunk = W.make_chunk(s["offsets"], s["lengths"], s["table"], max_new=s["max_new"], max_length=s["max_len"], total_new=s["total"])
    if c["op"] == "append":
        return lambda: W.whale_cache_append(cfg, cache, chunk, s["kv"]), _stored(s)
    if c["op"] == "read":
        planes = 1 if c["shared"] else 2
        out = torch.empty(s["total"], planes * c["kv_heads"] * c["dh"], dtype=torch.bfloat16, device=DEV)
        return lambda: W.whale_cache_read(cfg, cache, chunk, out), out
    out = torch.empty_like(s["q"])
    ws = buf(W.whale_cache_attention_workspace_size(cfg, cache, chunk))
    flags = W.WHALE_ATTEND_CAUSAL if c["causal"] else 0
    return lambda: W.whale_cache_attention(cfg, cache, chunk, s["q"], out, ws, flags=flags), out


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    call, out = s["plan"]
    call()
    return out


# ----------------------------------------------------------------------------------------------
# the same in 64 bits
# ----------------------------------------------------------------------------------------------
def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    if c["op"].startswith("norm_rotate"):
        return {p: _exact_rows(s, p, c) for p in "qk"}
    n, new = _lengths(c)
    off = np.concatenate([[0], np.cumsum(new)])
    P, out = c["page"], []
    table = s["table"].cpu().numpy()
    if c["op"] == "append":
        pages = s["pages"].double()
        scales = None if s["scales"] is None else torch.ones(s["scales"].shape, device=DEV, dtype=torch.float64)
    for b in range(c["B"]):
        t = int(new[b])
        first = int(n[b]) - t if c["op"] != "attend" else 0
        where = torch.arange(first, int(n[b]), device=DEV)
        page, slot = torch.from_numpy(table[b].astype(np.int64)).to(DEV)[where // P], where % P
        if c["op"] == "append":
            x = s["kv"][off[b] : off[b + 1]].double().reshape(t, -1, c["kv_heads"], c["dh"])
            if c["fmt"] == "bf16":
                pages[page, :, :, slot] = x
                continue
            big = x.abs().amax(-1).clamp(min=1e-300)
            e = torch.ceil(torch.log2(big / 448.0))
            e = torch.where(big > 448.0 * torch.exp2(e), e + 1, torch.where(big <= 224.0 * torch.exp2(e), e - 1, e))
            e = torch.where(x.abs().amax(-1) == 0, torch.zeros_like(e), e.clamp(E_LO, E_HI))
            y = x / torch.exp2(e)[..., None]
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0**-6))) - 3)  # spacing of e4m3 numbers there
            pages[page, :, :, slot] = torch.round(y / step) * step
            scales[page, :, :, slot] = torch.exp2(e)
            continue
        kv = s["pages"][page, :, :, slot]
        if c["fmt"] == "bf16":
            kv = kv.double()
        else:
            kv = kv.view(torch.float8_e4m3fn).double() * torch.exp2(s["scales"][page, :, :, slot].double() - 127)[..., None]
        if c["op"] == "read":
            out.append(kv.flatten(1))
            continue
        q = s["q"][off[b] : off[b + 1]].double().reshape(t, c["heads"], c["dh"])
        a = torch.zeros_like(q)
        for h in range(c["heads"]):
            g = h * c["kv_heads"] // c["heads"]
            z = q[:, h] @ kv[:, 0, g].T / math.sqrt(c["dh"])
            if c["causal"]:
                z = z.masked_fill(where[None] > int(n[b]) - t + torch.arange(t, device=DEV)[:, None], -math.inf)
            a[:, h] = torch.softmax(z, -1) @ kv[:, -1, g]
        out.append(a.flatten(1))
    if c["op"] == "append":
        return {"pages": pages} if scales is None else {"pages": pages, "scales": scales}
    return torch.cat(out)


def _exact_rows(s, p, c):
    x = s["x" + p].double().reshape(-1, c["heads"] if p == "q" else c["kv_heads"], c["dh"])
    rot = c["rot"]
    w = 10000.0 ** (-2.0 * torch.arange(rot // 2, device=DEV, dtype=torch.float64) / rot)
    turn = torch.polar(torch.ones((), device=DEV, dtype=torch.float64), s["p" + p].double()[:, None] * w)[:, None]
    r = 1.0 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
    gain = s["g" + p].double()
    pair = (lambda v: v.reshape(*v.shape[:2], 2, -1).transpose(2, 3)) if c["layout"] == "halves" else (lambda v: v.reshape(*v.shape[:2], -1, 2))
    back = (lambda v: v.transpose(2, 3).flatten(2)) if c["layout"] == "halves" else (lambda v: v.flatten(2))

    def turned(v, z):
        y = torch.view_as_real(torch.view_as_complex(pair(v[..., :rot]).contiguous()) * z)
        return torch.cat([back(y), v[..., rot:]], -1)

    if c["op"] == "norm_rotate":
        return turned(x * r * gain, turn).flatten(1)
    dn = turned(s["d" + p].double().reshape(x.shape), turn.conj())
    dg = (dn * x * r).sum((0, 1))
    u = dn * gain
    return (r * (u - x * r * r * (u * x).mean(-1, keepdim=True))).flatten(1), dg
