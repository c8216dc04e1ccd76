"""Cached-history operators on the GPU against the fp64 oracle: per-head norm and rotation with its backward
pass, rows into and out of the paged cache, attention over it, and the chain a serving program runs.

Tolerances count roundings. u = eps / 2 is one rounding (bf16 2^-8, fp32 2^-24).
 norm_rotate          u |y| + 40 * 2^-24 (|n_u| + |n_v|) + the angle's |p| 2^-51 (fp64 product, in kernel and oracle)
                      (at most 16 + 5 adds of the mean, one rsqrt of 2 ulp, three products, sine and cosine 2 ulp)
 its backward         u |dx| + 64 * 2^-24 (|r dn g| + |x| r^3 mean |dn g x|); d_gain 1.2e-5 sum |dn x r|: chains of
                      at most 160 serial fp32 adds per lane at these sizes, 40 for the factors
 append, read         equal
 attention            u |a| + (2^-8 + 6e-4) sum_j p_j |v_j|: the weights are rounded to bf16 once, 2^x has 7.5e-5, the
                      fp32 sums 64 * 2^-24 * (|q| . |k|) / sqrt(d_head) * 2 <= 1e-4 at |q| . |k| <= 100, both in p and in its sum
"""
import numpy as np
import pytest
import torch

from oracle import history_oracle as H
from tests.gpu_util import bf16_randn
from wukong_hstu_cross_b200 import inputs as I

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from wukong_hstu_cross_b200 import build
    build.build()
    from wukong_hstu_cross_b200 import whale as W

DEV = "cuda"
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _dt(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _gpu(a, name="fp32"):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV).to(_dt(name))


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _close(got, ref, tol, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - ref)
    if err.size and (err > tol).any():
        i = np.unravel_index(np.argmax(err - tol), err.shape)
        raise AssertionError(f"{what}: {err[i]:.3e} > {np.broadcast_to(tol, err.shape)[i]:.3e} at {i} ({got[i]} for {ref[i]}), "
                             f"{int((err > tol).sum())} of {err.size}")


def _cfg(h, dh, dtype="bf16", shared=False, eps=1e-6):
    return W.make_config(1, h * dh, h, 1, 64, 64, W.WHALE_FP32 if dtype == "fp32" else W.WHALE_BF16,
                         W.WHALE_SHARED_KV if shared else 0, eps)


def _ws(n):
    return torch.full((max(int(n), 256),), 0xFF, dtype=torch.uint8, device=DEV)  # its contents must not matter


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert W.whale_get_device_error() == 0


# ----------------------------------------------------------------------------------------------
# norm and rotation
# ----------------------------------------------------------------------------------------------
class Part:
    """Rows of one part in a wider tensor (row stride `pad` larger), on the CPU in fp64 and on the GPU."""

    def __init__(self, rng, rows, heads, dh, dtype, pos, pad=0, scale=1.0):
        self.rows, self.heads, self.dh = rows, heads, dh
        wide = bf16_randn(rng, rows, heads * dh + pad, scale=scale)
        if dtype == "fp32":
            wide = (rng.standard_normal(wide.shape) * scale).astype(np.float32)
        self.wide = _gpu(wide, dtype)
        self.x = self.wide[:, : heads * dh]
        self.h = wide[:, : heads * dh].astype(np.float64).reshape(rows, heads, dh)
        self.gain = rng.uniform(0.5, 1.5, dh).astype(np.float32)
        self.pos = rng.integers(-pos if pos < 1 << 20 else 0, pos, rows).astype(np.int32)
        self.g, self.p = _gpu(self.gain), _int(self.pos)

    def angle(self):
        return np.abs(self.pos.astype(np.float64))[:, None, None] * 2.0 ** -51


def _pair_mag(n, rot, layout):
    m = np.abs(n).copy()
    if rot:
        u, v = H.pair_columns(rot, layout)
        s = m[..., u] + m[..., v]
        m[..., u] = s
        m[..., v] = s
    return m


NR = [  # dtype, dh, q heads, k heads, q rows, k rows, rot, layout, positions, pad
    ("bf16", 64, 8, 8, 1, 0, 64, H.HALVES, 100, 0), ("bf16", 64, 8, 2, 33, 1000, 32, H.HALVES, 15000, 512),
    ("bf16", 32, 4, 4, 257, 63, 32, H.ADJACENT, 1 << 20, 8), ("bf16", 32, 16, 4, 5, 77, 16, H.HALVES, 15000, 0),
    ("bf16", 64, 2, 2, 3, 9, 0, H.HALVES, 5, 0), ("bf16", 32, 2, 2, 3, 9, 16, H.ADJACENT, 1 << 31, 16),
    ("fp32", 8, 2, 1, 17, 300, 8, H.HALVES, 500, 4), ("fp32", 16, 3, 3, 64, 5, 8, H.ADJACENT, 500, 0),
    ("fp32", 32, 8, 8, 0, 129, 16, H.HALVES, 1 << 20, 0), ("fp32", 64, 5, 1, 31, 31, 64, H.ADJACENT, 15000, 64),
    ("fp32", 128, 2, 2, 10, 1, 128, H.HALVES, 15000, 0), ("fp32", 128, 1, 1, 10, 1, 64, H.HALVES, 15000, 0),
]


@pytest.mark.parametrize("case", NR, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rotate(case, in_place):
    dtype, dh, hq, hk, rq, rk, rot, layout, pos, pad = case
    rng = np.random.default_rng(dh + rq + rot)
    parts = [Part(rng, r, h, dh, dtype, pos, pad) for r, h in ((rq, hq), (rk, hk))]
    rotary = W.make_rotary(rot, 10000.0, layout)
    rows, out = [], []
    for p in parts:
        before = p.wide.clone()
        y = p.x if in_place else torch.full((p.rows, p.heads * dh + 16), 7.0, device=DEV, dtype=_dt(dtype))[:, : p.heads * dh]
        out.append((y, before))
        rows.append(W.head_rows(p.x, p.g, p.p, y=y))
    W.whale_norm_rotate(_cfg(hq, dh, dtype), rotary, *rows)
    torch.cuda.synchronize()
    for p, (y, before), name in zip(parts, out, "qk"):
        ref = H.norm_rotate(p.h, p.gain, p.pos, rot, 10000.0, layout, 1e-6)
        n = H.norm_rotate(p.h, p.gain, p.pos, 0, 10000.0, layout, 1e-6)
        mag = _pair_mag(n, rot, layout)
        _close(_np(y).reshape(ref.shape), ref, U[dtype] * np.abs(ref) + (40 * 2.0 ** -24 + p.angle()) * mag, name)
        if in_place:  # the other columns of the rows stay
            assert torch.equal(p.wide[:, p.heads * dh:], before[:, p.heads * dh:])
        else:
            assert torch.equal(p.wide, before)
            if p.rows:
                assert (y._base[:, p.heads * dh:] == 7.0).all()


def test_norm_rotate_one_part_alone_and_zero_rows_of_numbers():
    rng = np.random.default_rng(3)
    p = Part(rng, 40, 8, 32, "bf16", 50)
    p.x.zero_()
    y = torch.empty_like(p.x)
    cfg, rotary = _cfg(8, 32), W.make_rotary(32)
    W.whale_norm_rotate(cfg, rotary, None, W.head_rows(p.x, p.g, p.p, y=y))
    assert not y.any()
    W.whale_norm_rotate(cfg, rotary, None, None)
    with pytest.raises(ValueError):
        W.whale_norm_rotate(_cfg(4, 64), rotary, W.head_rows(p.x, p.g, p.p, y=y), None)
    with pytest.raises(ValueError):
        W.head_rows(p.x, p.g, p.p[:5], y=y)
    with pytest.raises(ValueError):
        W.head_rows(p.x, p.g, p.p, y=y.float())


NRB = [  # dtype, grad, dh, q heads, k heads, q rows, k rows, rot, layout, positions, pad
    ("bf16", "bf16", 64, 8, 8, 33, 700, 64, H.HALVES, 15000, 512), ("bf16", "fp32", 64, 8, 2, 1, 300, 32, H.HALVES, 15000, 0),
    ("bf16", "bf16", 32, 4, 4, 257, 63, 32, H.ADJACENT, 1 << 20, 8), ("bf16", "fp32", 32, 16, 4, 5, 0, 16, H.ADJACENT, 99, 0),
    ("bf16", "bf16", 32, 2, 2, 20000, 3, 32, H.HALVES, 99, 0),
    ("fp32", "fp32", 8, 2, 1, 17, 300, 8, H.HALVES, 500, 4), ("fp32", "fp32", 16, 3, 3, 64, 5, 8, H.ADJACENT, 500, 0),
    ("fp32", "fp32", 32, 8, 8, 129, 1000, 16, H.HALVES, 1 << 20, 0), ("fp32", "fp32", 64, 5, 1, 31, 31, 0, H.HALVES, 9, 64),
    ("fp32", "fp32", 128, 2, 2, 10, 1, 128, H.ADJACENT, 15000, 0),
]


@pytest.mark.parametrize("case", NRB, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rotate_backward(case, in_place):
    dtype, grad, dh, hq, hk, rq, rk, rot, layout, pos, pad = case
    rng = np.random.default_rng(dh + rq + rot)
    cfg, rotary = _cfg(hq, dh, dtype), W.make_rotary(rot, 10000.0, layout)
    parts = [Part(rng, r, h, dh, dtype, pos, pad) for r, h in ((rq, hq), (rk, hk))]
    dys = [bf16_randn(rng, p.rows, p.heads * dh) for p in parts]
    results = []
    for _ in range(2):
        rows, grads, out = [], [], []
        for p, dy in zip(parts, dys):
            t = torch.zeros(p.rows, p.heads * dh + 16, device=DEV, dtype=_dt(grad))[:, : p.heads * dh]
            t.copy_(_gpu(dy, grad))
            dx = t if in_place else torch.full_like(t, 7.0)
            out.append((dx, torch.full((dh,), 7.0, device=DEV)))
            rows.append(W.head_rows(p.x, p.g, p.p))
            grads.append(W.head_grads(t, *out[-1]))
        n = W.whale_norm_rotate_workspace_size(cfg, *rows)
        W.whale_norm_rotate_backward(cfg, rotary, *rows, *grads, W.WHALE_FP32 if grad == "fp32" else W.WHALE_BF16, _ws(n))
        torch.cuda.synchronize()
        results.append(out)
    for p, dy, (dx, dg), (dx2, dg2), name in zip(parts, dys, *results, "qk"):
        assert torch.equal(dx, dx2) and torch.equal(dg, dg2)  # the sums have a fixed order
        up = dy.astype(np.float64).reshape(p.h.shape)
        rdx, rdg = H.norm_rotate_backward(p.h, p.gain, p.pos, rot, 10000.0, layout, 1e-6, up)
        r = 1.0 / np.sqrt(np.mean(p.h ** 2, -1, keepdims=True) + 1e-6)
        dn = _pair_mag(up, rot, layout)
        mag = r * dn * p.gain + np.abs(p.h) * r ** 3 * np.mean(dn * p.gain * np.abs(p.h), -1, keepdims=True)
        tol = U[grad] * np.abs(rdx) + (64 * 2.0 ** -24 + 2 * p.angle()) * mag
        _close(_np(dx).reshape(rdx.shape), rdx, tol, f"dx {name}")
        _close(_np(dg), rdg, np.sum((1.2e-5 + 2 * p.angle()) * dn * np.abs(p.h) * r, (0, 1)), f"d_gain {name}")


def test_norm_rotate_backward_against_differences():
    """fp32, directional: (f(x + t v) - f(x - t v)) / 2 t for f = sum(dy y), t = 2^-7. Central differences are off
    by t^2 / 6 times the third derivative (below 1e-2 of the gradient's scale at unit rows: 1e-5) and by 40 *
    2^-24 * sum |dy| |y| / t (sum of 4096 terms of about 1: 1.3 in the worst case, 40 sqrt(4096) 2^-24 / t = 0.02 typical)."""
    rng = np.random.default_rng(7)
    p = Part(rng, 64, 2, 32, "fp32", 900)
    cfg, rotary = _cfg(2, 32, "fp32"), W.make_rotary(32)
    dy, v = rng.standard_normal((64, 64)), rng.standard_normal((64, 64))
    dx, dg = torch.empty_like(p.x), torch.empty(32, device=DEV)
    r = W.head_rows(p.x, p.g, p.p)
    W.whale_norm_rotate_backward(cfg, rotary, r, None, W.head_grads(_gpu(dy), dx, dg), None, W.WHALE_FP32,
                                 _ws(W.whale_norm_rotate_workspace_size(cfg, r, None)))

    def f(x, gain):
        y = torch.empty_like(p.x)
        W.whale_norm_rotate(cfg, rotary, W.head_rows(_gpu(x), _gpu(gain), p.p, y=y), None)
        return float(np.sum(dy.astype(np.float32).astype(np.float64) * _np(y)))

    x0, t = p.h.reshape(64, 64), 2.0 ** -7
    got = (f(x0 + t * v, p.gain) - f(x0 - t * v, p.gain)) / (2 * t)
    want = float(np.sum(_np(dx) * v))
    assert abs(got - want) <= 0.02 * 4 + 1e-3 * abs(want), (got, want)
    vg = rng.standard_normal(32)
    got = (f(x0, p.gain + t * vg) - f(x0, p.gain - t * vg)) / (2 * t)
    assert abs(got - float(np.sum(_np(dg) * vg))) <= 0.02 * 4 + 1e-3 * abs(got)


# ----------------------------------------------------------------------------------------------
# cache
# ----------------------------------------------------------------------------------------------
class Cache:
    """A cache, its sequences and their true contents. `values[b]` [length, planes, kv_heads, dh] fp64."""

    def __init__(self, rng, lengths, new, h, hk, dh, page, fmt, shared=False, spare=2, scale=1.0, fill=True, stride=1):
        self.h, self.hk, self.dh, self.page, self.fmt = h, hk, dh, page, fmt
        self.planes = 1 if shared else 2
        self.lengths, self.new = np.asarray(lengths), np.asarray(new)
        self.B = len(lengths)
        need = -(-self.lengths // page)
        self.n_pages = int(need.sum()) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.B, max(int(need.max()), 0) + stride), -1, np.int32)  # unused entries are no page
        at = 0
        for b in range(self.B):
            self.table[b, : need[b]] = order[at : at + need[b]]
            at += need[b]
        self.off = np.concatenate([[0], np.cumsum(self.new)])
        self.total = int(self.off[-1])
        shape = (self.n_pages, self.planes, hk, page, dh)
        # unwritten rows are NaN: nothing may use them
        if fmt == "bf16":
            self.pages, self.scales = torch.full(shape, float("nan"), device=DEV, dtype=torch.bfloat16), None
        else:
            self.pages = torch.full(shape, 0x7F, device=DEV, dtype=torch.uint8)
            self.scales = torch.full(shape[:4], 0xFF, device=DEV, dtype=torch.uint8)
        self.values = []
        for b in range(self.B):
            x = bf16_randn(rng, int(self.lengths[b]), self.planes, hk, dh, scale=scale).astype(np.float64)
            x *= 2.0 ** rng.integers(-2, 3, x.shape[:3])[..., None]
            self.values.append(x)
        self.cfg = _cfg(h, dh, "bf16", shared)
        if fill:
            self.store([(b, 0, int(self.lengths[b])) for b in range(self.B)])

    def store(self, spans):
        pages = self.pages.cpu()
        scales = None if self.scales is None else self.scales.cpu()
        for b, lo, hi in spans:
            pos = np.arange(lo, hi)
            pg, sl = torch.from_numpy(self.table[b, pos // self.page].astype(np.int64)), torch.from_numpy(pos % self.page)
            if self.fmt == "bf16":
                pages[pg, :, :, sl] = torch.from_numpy(self.values[b][lo:hi].astype(np.float32)).bfloat16()
            else:
                v, e = H.quantise(self.values[b][lo:hi])
                pages[pg, :, :, sl] = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
                scales[pg, :, :, sl] = torch.from_numpy((e + 127).astype(np.uint8))
                self.values[b][lo:hi] = v * 2.0 ** e[..., None].astype(np.float64)
        self.pages.copy_(pages)
        if scales is not None:
            self.scales.copy_(scales)

    def handle(self):
        return W.make_cache(self.pages, self.scales)

    def chunk(self, **kw):
        f = dict(offsets=_int(self.off), lengths=_int(self.lengths), page_table=_int(self.table),
                 max_new=int(self.new.max()), max_length=int(self.lengths.max()), total_new=self.total)
        f.update(kw)
        return W.make_chunk(**f)

    def width(self):
        return self.planes * self.hk * self.dh

    def rows(self):
        """The chunk's rows, [total, width]: the last new[b] positions of each sequence."""
        return np.concatenate([self.values[b][int(self.lengths[b]) - int(self.new[b]):].reshape(-1, self.width())
                               for b in range(self.B)])

    def bytes(self):
        return self.pages.view(torch.uint8).clone(), None if self.scales is None else self.scales.clone()


def _rows_tensor(c, pad, extra):
    return torch.full((c.total + extra, c.width() + pad), 7.0, device=DEV, dtype=torch.bfloat16)[:, : c.width()]


ROWS = [  # lengths, new, h, hk, dh, page, shared
    ([1], [1], 4, 4, 64, 16, False), ([5, 0, 130, 64], [2, 0, 130, 0], 8, 8, 32, 16, False),
    ([300, 17, 1], [300, 0, 1], 8, 2, 64, 128, False), ([63, 64, 65], [63, 64, 65], 2, 1, 32, 64, True),
    ([1000] * 3, [1, 999, 500], 16, 4, 32, 256, False), ([40] * 70, list(range(35)) * 2, 8, 8, 64, 32, True),
    ([2000, 3], [1025, 0], 8, 8, 64, 1024, False),
]


@pytest.mark.parametrize("case", ROWS, ids=lambda c: f"{len(c[0])}x{c[0][0]} h{c[2]}/{c[3]} d{c[4]} page{c[5]}")
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_append_and_read(case, fmt):
    lengths, new, h, hk, dh, page, shared = case
    rng = np.random.default_rng(page + dh)
    c = Cache(rng, lengths, new, h, hk, dh, page, fmt, shared, fill=False)
    before = c.bytes()
    kv = _rows_tensor(c, 8, 3)
    if c.total:
        kv[: c.total].copy_(_gpu(c.rows(), "bf16"))
    got = (c.pages, c.scales)
    W.whale_cache_append(c.cfg, c.handle(), c.chunk(total_new=c.total + 3), kv)
    torch.cuda.synchronize()
    # the same rows stored by the oracle into an untouched copy: written rows agree and no other byte changed
    c.pages, c.scales = before[0].view(got[0].dtype).reshape(got[0].shape).clone(), before[1]
    c.store([(b, lengths[b] - new[b], lengths[b]) for b in range(len(lengths))])
    assert torch.equal(got[0].view(torch.uint8), c.pages.view(torch.uint8))
    if fmt == "e4m3":
        assert torch.equal(got[1], c.scales)
    out = _rows_tensor(c, 24, 3)
    W.whale_cache_read(c.cfg, c.handle(), c.chunk(total_new=c.total + 3), out)
    torch.cuda.synchronize()
    if c.total:
        assert np.array_equal(_np(out[: c.total]), c.rows())
    assert (out[c.total:] == 7.0).all() and (out._base[:, c.width():] == 7.0).all()


def test_append_special_rows():
    """Zeros, the scale's borders and ends, infinities and NaNs."""
    dh, page = 32, 16
    rows = np.zeros((11, dh), np.float32)
    rows[1, 4], rows[2, 5], rows[3, 6] = 448.0, 450.0, 1.75
    rows[4, :] = 1e-38
    rows[5, 0], rows[5, 1] = 3.0e38, -1.0
    rows[6, 0], rows[6, 1] = np.inf, 2.0
    rows[7, 0], rows[7, 1] = -np.inf, 1e30
    rows[8, 0], rows[8, 1] = np.nan, 3.0
    rows[9, :] = np.nan
    rows[10, :] = -0.0
    rows = I.bf16_round(rows)
    c = Cache(np.random.default_rng(0), [11], [11], 2, 2, dh, page, "e4m3", shared=True, fill=False)
    kv = _gpu(np.concatenate([rows, rows], 1), "bf16")
    W.whale_cache_append(c.cfg, c.handle(), c.chunk(), kv)
    out = torch.empty_like(kv)
    W.whale_cache_read(c.cfg, c.handle(), c.chunk(), out)
    torch.cuda.synchronize()
    codes = c.scales[int(c.table[0, 0]), 0, 0, :11].cpu().numpy().astype(int) - 127
    assert list(codes) == [0, 0, 1, -8, -100, 119, 119, 119, -7, 0, 0]
    got = _np(out)[:, :dh]
    v, e = H.quantise(rows[:6])
    assert np.array_equal(got[:6], v * 2.0 ** e[:, None])
    top = 448.0 * 2.0 ** 119
    assert got[6, 0] == top and got[7, 0] == -top and np.isnan(got[8, 0]) and got[8, 1] == 3.0 and np.isnan(got[9]).all()
    assert not got[10].any()


def test_rows_in_no_page():
    """Positions below 0 and past the bounds, and entries of the table outside the cache: rows are not written, come
    back as zeros, and are reported; attention sees zero keys and values there."""
    rng = np.random.default_rng(5)
    for fmt in ("bf16", "e4m3"):
        c = Cache(rng, [100, 100, 100], [100, 20, 100], 4, 4, 32, 16, fmt)
        good = c.chunk()
        kv = _gpu(c.rows(), "bf16")
        c.table[0, 2] = c.n_pages
        c.table[2, 1] = -5
        lengths = c.lengths.copy()
        lengths[1] = 7  # 13 of the 20 rows are at positions below 0
        before = c.bytes()[0]
        bad = c.chunk(page_table=_int(c.table), lengths=_int(lengths), max_length=90)
        out = torch.full_like(kv, 7.0)
        W.whale_cache_read(c.cfg, c.handle(), bad, out)
        torch.cuda.synchronize()
        assert W.whale_get_device_error() == W.WHALE_DEVERR_PAGES
        ref = c.rows()
        ref[32:48] = 0
        ref[90:100] = 0
        ref[100:113] = 0
        ref[113:120] = c.values[1][:7].reshape(7, -1)
        ref[120 + 16 : 120 + 32] = 0
        ref[120 + 90 :] = 0
        assert np.array_equal(_np(out), ref), fmt
        # the same rows again: no value changes. (Of an e4m3 row the bytes may: a largest number that was rounded
        # down to 1.75 * 2^k fits the next smaller scale, where every number of the row is exact too.)
        W.whale_cache_append(c.cfg, c.handle(), bad, out)
        torch.cuda.synchronize()
        assert W.whale_get_device_error() == W.WHALE_DEVERR_PAGES
        if fmt == "bf16":
            assert torch.equal(before, c.bytes()[0])
        W.whale_cache_read(c.cfg, c.handle(), good, out)
        assert torch.equal(out, kv), fmt
        q = bf16_randn(rng, c.total, 4 * 32)
        for causal in (False, True):
            a = torch.empty(c.total, 128, device=DEV, dtype=torch.bfloat16)
            W.whale_cache_attention(c.cfg, c.handle(), bad, _gpu(q, "bf16"), a,
                                    _ws(W.whale_cache_attention_workspace_size(c.cfg, c.handle(), bad)),
                                    flags=W.WHALE_ATTEND_CAUSAL if causal else 0)
            torch.cuda.synchronize()
            assert W.whale_get_device_error() == W.WHALE_DEVERR_PAGES
            vals = [v.copy() for v in c.values]
            vals[0][32:48] = 0
            vals[2][16:32] = 0
            for b, n in ((0, 90), (1, 7), (2, 90)):
                lo, hi = c.off[b], c.off[b + 1]
                first = int(lengths[b]) - int(hi - lo)
                ref, mag = H.attention(q[lo:hi].reshape(-1, 4, 32), vals[b][:n, 0], vals[b][:n, 1], causal, first)
                _close(_np(a[lo:hi]).reshape(ref.shape), ref, _attend_tol(ref, mag), f"{fmt} {causal} {b}")


def _attend_tol(ref, mag):
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 6e-4) * mag


def _attend(c, q, causal, pad=0, extra=0, ws=None):
    wide = torch.full((c.total + extra, c.h * c.dh + pad), 7.0, device=DEV, dtype=torch.bfloat16)
    wide[: c.total, : c.h * c.dh].copy_(_gpu(q, "bf16"))
    out = torch.full((c.total + extra, c.h * c.dh + 2 * pad), 7.0, device=DEV, dtype=torch.bfloat16)
    a, chunk = out[:, : c.h * c.dh], c.chunk(total_new=c.total + extra)
    n = W.whale_cache_attention_workspace_size(c.cfg, c.handle(), chunk)
    W.whale_cache_attention(c.cfg, c.handle(), chunk, wide[:, : c.h * c.dh], a, _ws(n) if ws is None else ws,
                            flags=W.WHALE_ATTEND_CAUSAL if causal else 0)
    torch.cuda.synchronize()
    assert (out[c.total:] == 7.0).all() and (out[:, c.h * c.dh:] == 7.0).all()
    return a[: c.total]


def _check_attend(c, q, a, causal, rows=None):
    for b in range(c.B):
        lo, hi = int(c.off[b]), int(c.off[b + 1])
        first = int(c.lengths[b]) - (hi - lo)
        idx = np.arange(hi - lo) if rows is None else np.unique(np.clip(rows, 0, hi - lo - 1)) if hi > lo else []
        for i in ([None] if rows is None else idx):
            sl = slice(lo, hi) if i is None else slice(lo + int(i), lo + int(i) + 1)
            f = first if i is None else first + int(i)
            ref, mag = H.attention(q[sl].reshape(-1, c.h, c.dh), c.values[b][:, 0], c.values[b][:, -1], causal, f)
            _close(_np(a[sl]).reshape(ref.shape), ref, _attend_tol(ref, mag), f"sequence {b} row {i}")


ATTEND = [  # lengths, new, h, hk, dh, page, shared
    ([1], [1], 4, 4, 64, 16, False), ([5000], [1], 8, 2, 64, 64, False),
    ([3, 0, 130, 64, 700], [1, 1, 1, 0, 1], 8, 8, 32, 16, False),
    ([0, 0], [3, 1], 8, 8, 64, 32, False),
    ([300, 17, 1, 257], [2, 3, 1, 5], 16, 4, 32, 128, False),
    ([900, 1, 64, 2047], [32, 32, 32, 32], 8, 8, 64, 64, False),
    ([900, 33, 640], [31, 33, 17], 8, 8, 32, 128, False),
    ([63, 64, 65, 127, 128, 129], [5] * 6, 2, 1, 32, 64, True),
    ([2500, 128], [16, 16], 8, 2, 64, 1024, True),
    ([129, 700, 260], [129, 100, 257], 4, 4, 64, 16, False),
    ([400, 513], [200, 300], 8, 2, 32, 32, False),
    ([700, 300, 0, 9], [300, 129, 0, 9], 4, 1, 64, 128, True),
    ([600, 256], [255, 128], 4, 4, 32, 256, False),
    ([640, 0, 3, 129, 5000], [17, 4, 20, 0, 32], 8, 8, 32, 16, False),
    ([2000, 128, 127], [8, 7, 1], 8, 2, 64, 32, True),
    ([1537] * 4, [29, 1, 32, 2], 2, 2, 32, 512, True),
]


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: f"{len(c[0])}x{c[0][0]}+{c[1][0]} h{c[2]}/{c[3]} d{c[4]} page{c[5]}")
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [False, True])
def test_attention(case, fmt, causal):
    lengths, new, h, hk, dh, page, shared = case
    rng = np.random.default_rng(page + dh + h)
    c = Cache(rng, lengths, new, h, hk, dh, page, fmt, shared)
    q = bf16_randn(rng, c.total, h * dh)
    a = _attend(c, q, causal, pad=8, extra=2)
    if c.total <= 200:
        _check_attend(c, q, a, causal)
    else:
        _check_attend(c, q, a, causal, rows=np.concatenate([np.arange(4), rng.integers(0, 300, 20), [31, 32, 63, 64, 127, 128, 299]]))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 32, 200])
def test_attention_rows_before_the_history(fmt, n):
    """More rows than positions: causal rows at negative positions see nothing and give 0."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [n // 2, 70], [n, min(n, 90)], 8, 2, 64, 16, fmt)
    q = bf16_randn(rng, c.total, 8 * 64)
    a = _attend(c, q, True)
    assert not a[: n - n // 2].any()
    _check_attend(c, q, a, True, rows=np.arange(0, n, max(1, n // 9)))


@pytest.mark.parametrize("n", [1, 32, 200])
@pytest.mark.parametrize("dh", [32, 64])
def test_attention_large_scores(n, dh):
    """Scores in the hundreds with the largest late in the history, so that the running maximum rises often; each
    row's weight is then on one key. fp32 sums of |q| . |k| <= 64 * 30 * 30 / 8: 64 * 2^-24 * 2 * 7200 / 2 is below 3e-2 of a weight."""
    rng = np.random.default_rng(n + dh)
    c = Cache(rng, [1500], [n], 4, 4, dh, 64, "bf16", fill=False)
    c.values[0][:, 0] *= (1.0 + np.arange(1500) / 300.0)[:, None, None]
    c.values[0] = I.bf16_round(c.values[0].astype(np.float32)).astype(np.float64)
    c.store([(0, 0, 1500)])
    q = bf16_randn(rng, n, 4 * dh, scale=4.0)
    a = _attend(c, q, False)
    rows = [0] if n == 1 else np.arange(0, n, 11)
    for i in rows:
        ref, mag = H.attention(q[i : i + 1].reshape(1, 4, dh), c.values[0][:, 0], c.values[0][:, 1], False, 0)
        _close(_np(a[i : i + 1]).reshape(ref.shape), ref, 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 3e-2) * mag, f"row {i}")


def test_attention_equal_keys_average_the_values():
    rng = np.random.default_rng(2)
    c = Cache(rng, [4097], [1], 8, 8, 32, 128, "bf16", fill=False)
    c.values[0][:, 0] = 1.0
    c.store([(0, 0, 4097)])
    q = bf16_randn(rng, 1, 256)
    a = _attend(c, q, True)
    ref = c.values[0][:, 1].mean(0)[None]
    _close(_np(a).reshape(ref.shape), ref, _attend_tol(ref, np.abs(c.values[0][:, 1]).mean(0)[None]), "mean")


def test_attention_long_sequence_and_shared_pages():
    """15000 positions in pages of 16; two sequences whose tables share their first pages."""
    rng = np.random.default_rng(4)
    c = Cache(rng, [15000, 15000], [1, 3], 4, 4, 64, 16, "e4m3")
    c.table[1, :900] = c.table[0, :900]
    c.values[1][: 900 * 16] = c.values[0][: 900 * 16]
    q = bf16_randn(rng, 4, 256)
    _check_attend(c, q, _attend(c, q, True), True)


def test_repeated_calls_agree_bit_for_bit():
    rng = np.random.default_rng(6)
    for n in (1, 40, 150):
        c = Cache(rng, [3000, 100, 2000], [n, n // 2, n], 8, 8, 64, 64, "e4m3")
        q = bf16_randn(rng, c.total, 512)
        first = _attend(c, q, True)
        for _ in range(3):
            assert torch.equal(first, _attend(c, q, True))


def test_graphs_that_share_a_workspace_and_another_stream():
    rng = np.random.default_rng(8)
    cs = [Cache(rng, [2000, 77], [n, n], 8, 8, 64, 64, "bf16") for n in (1, 48)]
    qs = [bf16_randn(rng, c.total, 512) for c in cs]
    want = [_attend(c, q, False) for c, q in zip(cs, qs)]
    n = max(W.whale_cache_attention_workspace_size(c.cfg, c.handle(), c.chunk()) for c in cs)
    ws, st, graphs, outs, keep = _ws(n), torch.cuda.Stream(), [], [], []
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for c, q in zip(cs, qs):
            args = (c.cfg, c.handle(), c.chunk(), _gpu(q, "bf16"), torch.zeros(c.total, 512, device=DEV, dtype=torch.bfloat16), ws)
            W.whale_cache_attention(*args)
            st.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                W.whale_cache_attention(*args)
            graphs.append(g)
            outs.append(args[4])
            keep.append(args)
        for order in ((0, 1), (1, 0), (0, 0, 1)):
            for o in outs:
                o.fill_(7.0)
            for i in order:
                graphs[i].replay()
            st.synchronize()
            assert all(torch.equal(o, w) for o, w in zip(outs, want)), order


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [3, 20, 150])
def test_rows_beyond_the_hosts_bound_stay(fmt, n):
    """max_new below a sequence's rows: the rows beyond it are left as they are, and reported."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [300, 40], [n, 2], 4, 4, 32, 16, fmt)
    q = bf16_randn(rng, c.total, 128)
    want = _attend(c, q, True)
    a = torch.full_like(want, 7.0)
    chunk = c.chunk(max_new=2)
    W.whale_cache_attention(c.cfg, c.handle(), chunk, _gpu(q, "bf16"), a,
                            _ws(W.whale_cache_attention_workspace_size(c.cfg, c.handle(), chunk)), flags=W.WHALE_ATTEND_CAUSAL)
    torch.cuda.synchronize()
    assert W.whale_get_device_error() == W.WHALE_DEVERR_OFFSETS
    assert (a[2:n] == 7.0).all()
    for rows in (slice(0, 2), slice(n, n + 2)):
        ref, mag = _np(want[rows]), np.abs(c.values[0 if rows.start == 0 else 1][:, -1]).max()
        _close(_np(a[rows]), ref, 2 * _attend_tol(ref, mag), "rows within the bound")


def test_two_streams_at_once():
    """Two calls in flight at once, each with its own workspace and output, over one cache."""
    rng = np.random.default_rng(13)
    for n in (1, 24, 140):
        c = Cache(rng, [4000, 900], [n, n], 8, 8, 64, 64, "e4m3")
        qs = [bf16_randn(rng, c.total, 512) for _ in range(2)]
        want = [_attend(c, q, False) for q in qs]
        qt = [_gpu(q, "bf16") for q in qs]
        size = W.whale_cache_attention_workspace_size(c.cfg, c.handle(), c.chunk())
        ws, out = [_ws(size) for _ in qs], [torch.zeros_like(w) for w in want]
        chunk, streams = c.chunk(), [torch.cuda.Stream() for _ in qs]
        torch.cuda.synchronize()
        for _ in range(5):
            for s, q, o, w in zip(streams, qt, out, ws):
                W.whale_cache_attention(c.cfg, c.handle(), chunk, q, o, w, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(out, want))


def test_no_rows_at_all():
    """Sequences without rows, a batch of none, and a cache of no pages."""
    rng = np.random.default_rng(14)
    c = Cache(rng, [50, 0, 7], [0, 0, 0], 4, 4, 32, 16, "bf16")
    q = torch.full((5, 128), 3.0, device=DEV, dtype=torch.bfloat16)
    kv, a = torch.full((5, 256), 3.0, device=DEV, dtype=torch.bfloat16), torch.full_like(q, 7.0)
    before = c.bytes()[0]
    for max_new in (0, 4, 200):
        chunk = c.chunk(total_new=5, max_new=max_new)
        W.whale_cache_attention(c.cfg, c.handle(), chunk, q, a, _ws(W.whale_cache_attention_workspace_size(c.cfg, c.handle(), chunk)))
        W.whale_cache_append(c.cfg, c.handle(), chunk, kv)
        W.whale_cache_read(c.cfg, c.handle(), chunk, kv)
        torch.cuda.synchronize()
        assert (a == 7.0).all() and (kv == 3.0).all() and torch.equal(before, c.bytes()[0])
    # rows of an empty history, which has no page: attention gives zeros, and nothing is reported
    none = W.make_cache(torch.empty(0, 2, 4, 16, 32, device=DEV, dtype=torch.bfloat16))
    for n in (1, 200):
        chunk = W.make_chunk(_int([0, n]), _int([0]), torch.empty(1, 0, device=DEV, dtype=torch.int32), n, 0, n)
        q, a = torch.ones(n, 128, device=DEV, dtype=torch.bfloat16), torch.full((n, 128), 7.0, device=DEV, dtype=torch.bfloat16)
        W.whale_cache_attention(c.cfg, none, chunk, q, a, _ws(W.whale_cache_attention_workspace_size(c.cfg, none, chunk)))
        torch.cuda.synchronize()
        assert not a.any()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("h,hk", [(8, 8), (8, 2)])
def test_mixed_batch(fmt, h, hk):
    """Many sequences with a few rows beside one with many: each kind is taken by its own kernel."""
    rng = np.random.default_rng(h + hk)
    for long, short in ((140, 1), (300, 5), (90, 4)):
        B = 40
        lengths, new = rng.integers(1, 400, B), np.minimum(rng.integers(0, short + 1, B), 8)
        lengths[17], new[17] = 700, long
        lengths[3], new[3] = 0, 1
        c = Cache(rng, lengths, new, h, hk, 32, 32, fmt)
        q = bf16_randn(rng, c.total, h * 32)
        for causal in (False, True):
            a = _attend(c, q, causal)
            _check_attend(c, q, a, causal, rows=np.arange(0, 300, 13))
            assert torch.equal(a, _attend(c, q, causal))


def test_many_sequences():
    """More sequences than a block has threads, most of them without rows or history."""
    rng = np.random.default_rng(15)
    B = 1500
    lengths = np.where(rng.random(B) < 0.3, rng.integers(1, 60, B), 0)
    new = np.where(rng.random(B) < 0.4, rng.integers(0, 4, B), 0)
    for fmt, scale in (("bf16", 1), ("e4m3", 20)):
        c = Cache(rng, lengths, np.minimum(new * scale, 70), 2, 2, 32, 16, fmt)
        q = bf16_randn(rng, c.total, 64)
        _check_attend(c, q, _attend(c, q, False), False, rows=None if scale == 1 else np.array([0, 19, 59]))


def test_tensors_must_fit_the_call():
    rng = np.random.default_rng(9)
    c = Cache(rng, [40], [3], 8, 8, 32, 16, "bf16")
    q = torch.zeros(3, 256, device=DEV, dtype=torch.bfloat16)
    for bad in (q[:2], q[:, :128], q.float(), q.t()):
        with pytest.raises(ValueError):
            W.whale_cache_attention(c.cfg, c.handle(), c.chunk(), bad, q.clone(), _ws(1 << 20))
        with pytest.raises(ValueError):
            W.whale_cache_append(c.cfg, c.handle(), c.chunk(), bad)
    with pytest.raises(ValueError):
        W.whale_cache_attention(_cfg(4, 64), c.handle(), c.chunk(), q, q.clone(), _ws(1 << 20))
    with pytest.raises(ValueError):
        W.make_cache(c.pages, torch.zeros(3, device=DEV, dtype=torch.uint8))
    with pytest.raises(ValueError):
        W.make_chunk(_int([0, 3]), _int([40, 1]), _int(c.table), 3, 40, 3)


# ----------------------------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_serving_chain_matches_the_packed_path(fmt):
    """Histories grow by two appends: project new rows, norm and rotate the keys in place, append, attend; against
    the whole history projected at once and packed cross-attention of the same rotated queries (bf16 cache),
    or the oracle over what the e4m3 cache reads back."""
    rng = np.random.default_rng(11)
    d, h, dh, N, lens = 256, 8, 32, 16, np.array([170, 33, 0, 401])
    B, page = len(lens), 32
    cfg = W.make_config(1, d, h, N, 256, 512, W.WHALE_BF16, 0, 1e-6)
    g = _gpu(rng.uniform(0.5, 1.5, d))
    gain = _gpu(rng.uniform(0.5, 1.5, dh))
    wkv = _gpu(np.concatenate([I.xavier_uniform(rng, d, d), I.xavier_uniform(rng, d, d)]), "bf16")
    states = [_gpu(bf16_randn(rng, int(n), d), "bf16") for n in lens]
    ws, rotary = _ws(64 << 20), W.make_rotary(dh)

    def project(rows, positions):
        kv = torch.empty(rows.shape[0], 2 * d, device=DEV, dtype=torch.bfloat16)
        if rows.shape[0]:
            W.whale_project_kv(cfg, rows.shape[0], rows.contiguous(), g, wkv, kv, ws)
            W.whale_norm_rotate(cfg, rotary, None, W.head_rows(kv[:, :d], gain, _int(positions), y=kv[:, :d]))
        return kv

    c = Cache(rng, lens, lens, h, h, dh, page, fmt, fill=False)
    first = lens // 2
    for lo, hi in ((np.zeros(B, int), first), (first, lens)):
        new = hi - lo
        rows = torch.cat([s[a:b] for s, a, b in zip(states, lo, hi)])
        kv = project(rows, np.concatenate([np.arange(a, b) for a, b in zip(lo, hi)]))
        chunk = c.chunk(offsets=_int(np.concatenate([[0], np.cumsum(new)])), lengths=_int(hi), max_new=int(new.max()),
                        total_new=int(new.sum()))
        W.whale_cache_append(c.cfg, c.handle(), chunk, kv)
    q = _gpu(bf16_randn(rng, B * N, d), "bf16")
    qpos = np.repeat(lens, N)
    W.whale_norm_rotate(cfg, rotary, W.head_rows(q, gain, _int(qpos), y=q), None)
    off = np.arange(B + 1) * N
    chunk = c.chunk(offsets=_int(off), max_new=N, total_new=B * N)
    a = torch.empty_like(q)
    W.whale_cache_attention(c.cfg, c.handle(), chunk, q, a, ws)
    whole = c.chunk()
    back = torch.empty(int(lens.sum()), 2 * d, device=DEV, dtype=torch.bfloat16)
    W.whale_cache_read(c.cfg, c.handle(), whole, back)
    all_kv = project(torch.cat(states), np.concatenate([np.arange(n) for n in lens]))
    torch.cuda.synchronize()
    hoff = np.concatenate([[0], np.cumsum(lens)])
    if fmt == "bf16":
        # the same numbers up to the projection's tiling: equal or one bf16 step apart
        assert (back.float() - all_kv.float()).abs().max() <= 2.0 ** -7 * all_kv.float().abs().max()
        packed = torch.empty_like(q)
        W.whale_cross_attention(cfg, q, back, _int(hoff), packed, W.make_hint(B, int(lens.max()), int(lens.sum())), ws)
        torch.cuda.synchronize()
    kvn, qn = _np(back).reshape(-1, 2, h, dh), _np(q).reshape(-1, h, dh)
    for b in range(B):
        k = kvn[hoff[b]:hoff[b + 1]]
        ref, mag = H.attention(qn[off[b]:off[b + 1]], k[:, 0], k[:, 1], False, 0)
        _close(_np(a[off[b]:off[b + 1]]).reshape(ref.shape), ref, _attend_tol(ref, mag), f"sequence {b}")
        if fmt == "bf16":
            got, other = _np(a[off[b]:off[b + 1]]).reshape(ref.shape), _np(packed[off[b]:off[b + 1]]).reshape(ref.shape)
            _close(got, other, 2 * _attend_tol(ref, mag), f"packed {b}")


# ----------------------------------------------------------------------------------------------
# values of very different sizes
# ----------------------------------------------------------------------------------------------
def _spread_values(rng, kind, length):
    """Powers of two by which a history's V rows are multiplied."""
    e = np.zeros(length)
    if kind == "zero rows":        # whose scale stands for 1, beside rows of about 2^-30
        e[:] = -30
    elif kind == "tiny":           # the least scales
        e[:] = -96
    elif kind == "any":
        e = rng.integers(-60, 61, length).astype(np.float64)
    elif kind == "late":           # the last event, which only the last row may see, and one early one that all see
        e[-1] = 40
        e[length // 3] = 12
    elif kind == "largest":        # the last event's numbers past the largest scale's
        e[-1] = 127
    return e


@pytest.mark.parametrize("kind", ["zero rows", "tiny", "any", "late", "largest"])
@pytest.mark.parametrize("n", [1, 5, 24, 40])
@pytest.mark.parametrize("dh", [32, 64])
def test_attention_over_e4m3_values_of_any_size(kind, n, dh):
    """V rows of one history whose scales differ by up to 2^226: positions that a row does not see, and rows of
    zeros, cost the others nothing. Up to 32 rows the weights are f16 of 2^(s - m) beside values of its own scale's
    neighbourhood: off by half a step of 2^-24 / 2^-8 / 2^7 at most, 2^-24 of the largest weight, for each position."""
    rng = np.random.default_rng(n + dh)
    lengths = [40, 2000]
    c = Cache(rng, lengths, [n, n], 4, 4, dh, 32, "e4m3", fill=False)
    for b, length in enumerate(lengths):
        v = c.values[b][:, 1] * (2.0 ** _spread_values(rng, kind, length))[:, None, None]
        v = np.clip(v, -3.3e38, 3.3e38)
        if kind == "zero rows":
            v[rng.random(length) < 0.1] = 0.0
        c.values[b][:, 1] = I.bf16_round(v.astype(np.float32)).astype(np.float64)
    c.store([(b, 0, n_b) for b, n_b in enumerate(lengths)])
    q = bf16_randn(rng, c.total, 4 * dh)
    a = _attend(c, q, True)
    for b, length in enumerate(lengths):
        lo = int(c.off[b])
        for i in range(n):
            end = length - n + i + 1
            ref, mag = H.attention(q[lo + i : lo + i + 1].reshape(1, 4, dh), c.values[b][:, 0], c.values[b][:, 1], True, end - 1)
            small = 2.0 ** -24 * np.abs(c.values[b][:end, 1]).sum(0)[None]
            _close(_np(a[lo + i : lo + i + 1]).reshape(ref.shape), ref, _attend_tol(ref, mag) + small, f"sequence {b} row {i}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 24, 40])
def test_attention_of_a_value_near_the_largest(fmt, n):
    """V of 3e38 at one position, whose score exceeds all those before it by 2^5 (less than makes the running
    reference rise): its weight times V stays finite."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [2048], [n], 4, 4, 64, 64, fmt, fill=False)
    k, v = np.zeros_like(c.values[0][:, 0]), np.zeros_like(c.values[0][:, 1])
    k[:, :, 0] = -2.0
    k[::8, :, 0] = 0.0
    k[165, :, 0] = 3.5  # q 8: 28 / 8 / ln 2 = 5.05 in powers of two
    v[165] = 3e38
    v[165, :, ::3] = -2e38
    c.values[0][:, 0], c.values[0][:, 1] = k, I.bf16_round(v.astype(np.float32)).astype(np.float64)
    c.store([(0, 0, 2048)])
    q = np.zeros((n, 256), np.float32)
    q[:, ::64] = 8.0
    a = _attend(c, q, False)
    ref, mag = H.attention(q[:1].reshape(1, 4, 64), c.values[0][:, 0], c.values[0][:, 1], False, 0)
    for i in range(n):
        _close(_np(a[i : i + 1]).reshape(ref.shape), ref, _attend_tol(ref, mag), f"row {i}")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 20, 150])
def test_a_bound_of_no_rows_is_reported(fmt, n):
    """max_new 0 and sequences with rows: none is taken, all stay, and the call says so; lengths past max_length too."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [300, 40], [n, 2], 4, 4, 32, 16, fmt)
    q = _gpu(bf16_randn(rng, c.total, 128), "bf16")
    for kw, code in ((dict(max_new=0), W.WHALE_DEVERR_OFFSETS), (dict(max_length=299), W.WHALE_DEVERR_PAGES),
                     (dict(max_new=0, max_length=299), W.WHALE_DEVERR_OFFSETS | W.WHALE_DEVERR_PAGES)):
        a, chunk = torch.full((c.total, 128), 7.0, device=DEV, dtype=torch.bfloat16), c.chunk(**kw)
        W.whale_cache_attention(c.cfg, c.handle(), chunk, q, a, _ws(W.whale_cache_attention_workspace_size(c.cfg, c.handle(), chunk)))
        torch.cuda.synchronize()
        assert W.whale_get_device_error() == code
        assert (a == 7.0).all() == ("max_new" in kw)


@pytest.mark.parametrize("shared", [False, True])
def test_a_layer_whose_histories_are_cached(shared):
    """A whole fusion layer with its history cached in two appends: project, append, query projection, attention over the cache,
    fusion MLP and FFN, against the oracle of the layer and the layer's own entry point, both at the bound of whole layers."""
    from tests.gpu_util import BF16_TOL, assert_parity
    from oracle import whale_oracle as O
    from wukong_hstu_cross_b200 import harness as Hn
    w = I.WORKLOADS["stack_d256"].replace(batch=3, n_layers=1, lengths=("uniform", 1, 900))
    p = Hn.build_problem(w, gains="random", shared_kv=shared)
    lw, N, d, h, B = p.weights[0], w.n_tokens, w.d, w.n_heads, w.batch
    c = Cache(np.random.default_rng(0), p.lengths, p.lengths, h, h, d // h, 64, "bf16", shared, fill=False)
    ws = _ws(64 << 20)
    lo = np.zeros(B, np.int64)
    for hi in (p.lengths // 2, p.lengths):
        rows = torch.cat([p.states[0, p.offsets[b] + lo[b] : p.offsets[b] + hi[b]] for b in range(B)])
        kv = torch.empty(rows.shape[0], c.width(), device=DEV, dtype=torch.bfloat16)
        W.whale_project_kv(p.cfg, rows.shape[0], rows, lw["g_kv"], lw["w_kv"], kv, ws)
        new = hi - lo
        W.whale_cache_append(p.cfg, c.handle(), c.chunk(offsets=_int(np.concatenate([[0], np.cumsum(new)])), lengths=_int(hi),
                                                        max_new=int(new.max()), total_new=int(new.sum())), kv)
        lo = hi
    x = p.tokens.reshape(B * N, d)
    q, a, f, y = (torch.empty_like(x) for _ in range(4))
    W.whale_project_queries(p.cfg, B * N, x, lw["g_q"], lw["w_q"], q, ws)
    chunk = c.chunk(offsets=_int(np.arange(B + 1) * N), max_new=N, total_new=B * N)
    W.whale_cache_attention(p.cfg, c.handle(), chunk, q, a, ws)
    W.whale_fusion_mlp(p.cfg, B * N, a, x, lw["w_f1"], lw["w_f2"], f, ws)
    W.whale_swiglu_ffn(p.cfg, B * N, f, lw["g_ffn"], lw["w_upgate"], lw["w_down"], y, ws)
    layer = Hn.run_forward(p)
    torch.cuda.synchronize()
    for b in range(B):
        ref = O.fusion_stack_example(I.tokens_of_example(w, b), Hn.states_of_example_host(p, b), p.host_weights, h, w.eps, **p.flags)
        got = y.reshape(B, N, d)[b]
        assert_parity(got, ref, "bf16", rms_rel=2e-2, what=f"example {b}")
        assert np.all(np.abs(_np(got) - _np(layer[b])) <= 2 * BF16_TOL * (1.0 + np.abs(ref)))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 24, 40])
def test_attention_of_queries_near_the_largest(fmt, n):
    """Queries with one number of 2^122 and more where the keys are zero, the others 2^-19 of it and exact in f16 beside it:
    finite scores of about 1."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [300], [n], 4, 4, 64, 64, fmt, fill=False)
    c.values[0][:, 0] *= 2.0 ** -103
    c.values[0][:, 0, :, 0] = 0.0
    c.store([(0, 0, 300)])
    q = bf16_randn(rng, n, 256, scale=2.0 ** 103)
    q[:, ::64] = 2.0 ** rng.integers(121, 124, (n, 4))
    a = _attend(c, q, False)
    _check_attend(c, q, a, False)


@pytest.mark.parametrize("fmt,dh", [("bf16", 64), ("e4m3", 32)])
def test_a_pool_past_32_bits(fmt, dh):
    """The same pages in a small pool and at the end of one of 4.5 GB: equal results of every operator."""
    rng = np.random.default_rng(dh)
    for n in (1, 20, 150):
        c = Cache(rng, [700, 200], [n, n], 8, 8, dh, 64, fmt)
        q, kv = _gpu(bf16_randn(rng, c.total, 8 * dh), "bf16"), _gpu(bf16_randn(rng, c.total, c.width()), "bf16")
        pool = (9 << 29) // c.pages[0].nbytes
        big = torch.empty(pool, *c.pages.shape[1:], device=DEV, dtype=c.pages.dtype)
        scales = None if c.scales is None else torch.empty(pool, *c.scales.shape[1:], device=DEV, dtype=torch.uint8)
        big[-c.n_pages:].copy_(c.pages)
        if scales is not None:
            scales[-c.n_pages:].copy_(c.scales)
        out = []
        for cache, table in ((c.handle(), c.table), (W.make_cache(big, scales), np.where(c.table < 0, -1, c.table + pool - c.n_pages))):
            chunk = c.chunk(page_table=_int(table))
            a, back = torch.empty_like(q), torch.empty_like(kv)
            W.whale_cache_attention(c.cfg, cache, chunk, q, a, _ws(W.whale_cache_attention_workspace_size(c.cfg, cache, chunk)))
            W.whale_cache_append(c.cfg, cache, chunk, kv)
            W.whale_cache_read(c.cfg, cache, chunk, back)
            out.append((a, back))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(*out))
        assert torch.equal(big[-c.n_pages:].view(torch.uint8), c.pages.view(torch.uint8))
        if scales is not None:
            assert torch.equal(scales[-c.n_pages:], c.scales)
