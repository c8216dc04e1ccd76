"""Host side of the cached-history operators (CPU): argument checks of every entry point before any CUDA call,
buffer sizes, struct layouts against the header, and the index and scale arithmetic of csrc/chunk_index.h
(compiled for the host) over good and bad page tables: no index leaves the cache, whatever the tables hold."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import history_oracle as H
from wukong_hstu_cross_b200 import build

build.build()
from wukong_hstu_cross_b200 import whale as W  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # aligned and never dereferenced: every call below fails its checks first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4


def _cfg(d=256, h=8, dtype=W.WHALE_BF16, flags=0, eps=1e-6):
    return W.make_config(1, d, h, 1, 64, 64, dtype, flags, eps)


def _rows(**kw):
    f = dict(x=FAKE, y=FAKE, gain=FAKE, positions=FAKE, rows=4, ld_x=256, ld_y=256, n_heads=8)
    f.update(kw)
    return W.whale_head_rows(*f.values())


def _grads(**kw):
    f = dict(dy=FAKE, dx=FAKE, d_gain=FAKE, ld_dy=256, ld_dx=256)
    f.update(kw)
    return W.whale_head_grads(*f.values())


def _cache(**kw):
    f = dict(pages=FAKE, scales=None, n_pages=10, page_size=64, n_kv_heads=8, format=W.WHALE_CACHE_BF16)
    f.update(kw)
    return W.whale_cache(*f.values())


def _chunk(**kw):
    f = dict(offsets=FAKE, lengths=FAKE, page_table=FAKE, table_stride=4, B=2, max_new=5, max_length=200, total_new=7)
    f.update(kw)
    return W.whale_chunk(*f.values())


def test_norm_rotate_refusals():
    call = lambda cfg=_cfg(), rot=W.make_rotary(32), q=_rows(), k=None: W.whale_norm_rotate(  # noqa: E731
        cfg, rot, q, k, stream=0, raw=True)
    bad = [dict(x=None), dict(y=None), dict(gain=None), dict(positions=None), dict(x=FAKE + 2), dict(y=FAKE + 8),
           dict(ld_x=248), dict(ld_y=248), dict(ld_x=257), dict(ld_y=260), dict(rows=-1), dict(rows=1 << 31),
           dict(n_heads=0), dict(n_heads=(1 << 20) + 1)]
    for b in bad:
        assert call(q=_rows(**b)) == INVALID, b
        assert call(q=None, k=_rows(**b)) == INVALID, b
    for r in (W.make_rotary(-16), W.make_rotary(48), W.make_rotary(32, base=0.0), W.make_rotary(32, base=float("nan")),
              W.make_rotary(32, base=float("inf")), W.make_rotary(32, layout=2)):
        assert call(rot=r) == INVALID
    assert call(rot=W.make_rotary(8)) == UNSUPPORTED                       # bf16: steps of 16
    assert call(cfg=_cfg(d=128, h=1)) == UNSUPPORTED                       # d_head 128 only in fp32 mode
    assert call(cfg=_cfg(d=255)) == INVALID
    assert call(q=None, k=None) == OK and call(q=_rows(rows=0, x=None, y=None, gain=None, positions=None)) == OK


def test_norm_rotate_backward_refusals():
    cfg = _cfg()
    need = W.whale_norm_rotate_workspace_size(cfg, _rows(), None)
    assert need > 0 and W.whale_norm_rotate_workspace_size(cfg, _rows(rows=-1), None) == 0

    def call(cfg=cfg, rot=W.make_rotary(32), q=_rows(y=None), dq=_grads(), gt=W.WHALE_BF16, ws=FAKE, n=need, k=None,
             dk=None):
        return W.whale_norm_rotate_backward(cfg, rot, q, k, dq, dk, gt, ws, n, stream=0, raw=True)

    for b in (dict(dy=None), dict(dx=None), dict(d_gain=None), dict(dy=FAKE + 2), dict(dx=FAKE + 2), dict(ld_dy=240),
              dict(ld_dx=240), dict(ld_dy=257), dict(ld_dx=257)):
        assert call(dq=_grads(**b)) == INVALID, b
    assert call(dq=None) == INVALID and call(q=None, k=_rows(), dk=None) == INVALID
    assert call(gt=7) == INVALID
    assert call(cfg=_cfg(dtype=W.WHALE_FP32), gt=W.WHALE_BF16) == UNSUPPORTED
    assert call(n=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(ws=FAKE + 16) == WORKSPACE
    assert call(q=None, dq=None) == OK


def test_cache_refusals_and_sizes():
    cfg, shared = _cfg(), _cfg(flags=W.WHALE_SHARED_KV)
    e4m3 = dict(format=W.WHALE_CACHE_E4M3, scales=FAKE)
    assert W.whale_cache_pages_size(cfg, _cache()) == 10 * 2 * 8 * 64 * 32 * 2
    assert W.whale_cache_pages_size(shared, _cache()) == 10 * 8 * 64 * 32 * 2
    assert W.whale_cache_pages_size(cfg, _cache(**e4m3)) == 10 * 2 * 8 * 64 * 32
    assert W.whale_cache_scales_size(cfg, _cache(**e4m3)) == 10 * 2 * 8 * 64
    assert W.whale_cache_scales_size(cfg, _cache()) == 0
    ws = 1 << 30
    calls = {
        "append": lambda cfg=cfg, k=_cache(), c=_chunk(), x=FAKE, ld=512: W._lib.whale_cache_append(
            cfg, k, c, x, ld, 0),
        "read": lambda cfg=cfg, k=_cache(), c=_chunk(), x=FAKE, ld=512: W._lib.whale_cache_read(cfg, k, c, x, ld, 0),
        "attend": lambda cfg=cfg, k=_cache(), c=_chunk(), x=FAKE, ld=512: W._lib.whale_cache_attention(
            cfg, k, c, x, ld, FAKE, 256, 0, FAKE, ws, 0),
    }
    for name, call in calls.items():
        for b in (dict(n_pages=-1), dict(page_size=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(format=2),
                  dict(pages=None), dict(pages=FAKE + 8), dict(format=W.WHALE_CACHE_E4M3),
                  dict(format=W.WHALE_CACHE_E4M3, scales=FAKE + 1)):
            assert call(k=_cache(**b)) == INVALID, (name, b)
        for b in (dict(page_size=48), dict(page_size=8), dict(page_size=2048), dict(n_pages=1 << 22)):
            assert call(k=_cache(**b)) == UNSUPPORTED, (name, b)
            assert W.whale_cache_pages_size(cfg, _cache(**b)) == 0
        for b in (dict(B=-1), dict(max_new=-1), dict(max_length=-1), dict(total_new=-1), dict(total_new=1 << 31),
                  dict(table_stride=-1), dict(offsets=None), dict(lengths=None), dict(page_table=None)):
            assert call(c=_chunk(**b)) == INVALID, (name, b)
        assert call(x=None) == INVALID and call(x=FAKE + 8) == INVALID, name
        assert call(ld=248) == INVALID and call(ld=516) == INVALID, name
        assert call(cfg=_cfg(dtype=W.WHALE_FP32)) == UNSUPPORTED, name
        assert call(cfg=None) == INVALID and call(k=None) == INVALID and call(c=None) == INVALID, name
        empty = dict(offsets=None, lengths=None, page_table=None)
        assert call(c=_chunk(B=0, **empty)) == OK and call(c=_chunk(total_new=0, **empty)) == OK, name
    need = W.whale_cache_attention_workspace_size(cfg, _cache(), _chunk())
    assert need > 0 and W.whale_cache_attention_workspace_size(cfg, _cache(page_size=8), _chunk()) == 0

    def attend(a=FAKE, ld_a=256, flags=0, w=FAKE, n=need):
        return W._lib.whale_cache_attention(cfg, _cache(), _chunk(), FAKE, 256, a, ld_a, flags, w, n, 0)

    big = lambda **kw: W.whale_cache_attention_workspace_size(cfg, _cache(), _chunk(**kw))  # noqa: E731
    assert big(max_length=1 << 30, table_stride=1 << 20) > 0 and big(max_length=(1 << 30) + 1) == 0
    assert big(total_new=(1 << 28) - 1, max_new=1) > 0 and big(total_new=1 << 28, max_new=1) == 0  # 8 heads
    for kw in (dict(max_length=(1 << 30) + 1), dict(total_new=1 << 28)):
        assert W._lib.whale_cache_attention(cfg, _cache(), _chunk(**kw), FAKE, 256, FAKE, 256, 0, FAKE, ws, 0) == UNSUPPORTED
    assert attend(a=None) == INVALID and attend(a=FAKE + 8) == INVALID and attend(ld_a=248) == INVALID
    assert attend(ld_a=257) == INVALID and attend(flags=2) == INVALID
    assert attend(w=None) == WORKSPACE and attend(n=need - 1) == WORKSPACE and attend(w=FAKE + 128) == WORKSPACE


STRUCTS = {"whale_rotary": W.whale_rotary, "whale_head_rows": W.whale_head_rows, "whale_head_grads": W.whale_head_grads,
           "whale_cache": W.whale_cache, "whale_chunk": W.whale_chunk}


def _run(tmp_path, name, compiler, args, source):
    cc = shutil.which(compiler)
    if cc is None:
        pytest.skip(f"no {compiler}")
    src, exe = tmp_path / name, tmp_path / "program"
    src.write_text(source)
    subprocess.run([cc, *args, str(src), "-o", str(exe)], check=True, capture_output=True, text=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=120).stdout


def test_struct_layouts_match_the_header(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    out = _run(tmp_path, "p.c", "gcc", ["-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include")],
               '#include <stddef.h>\n#include <stdio.h>\n#include "whale_fusion.h"\nint main(void) {\n'
               + "\n".join(lines) + "\nreturn 0; }\n")
    got = dict(line.rsplit(" ", 1) for line in out.splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(got[f"{name}.{f[0]}"]) == getattr(cls, f[0]).offset, (name, f[0])


INDEX = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "chunk_index.h"
using namespace whale;

int main() {
  unsigned seed = 1;
  auto rnd = [&](int n) { seed = seed * 1664525u + 1013904223u; return (int)((seed >> 8) % (unsigned)n); };
  long long good = 0, bad = 0;
  for (int t = 0; t < 4000; ++t) {
    ChunkView c{};
    c.B = 1 + rnd(6);
    c.page_shift = 4 + rnd(4);
    c.n_pages = rnd(9);
    c.planes = 1 + rnd(2);
    c.kv_heads = 1 + rnd(8);
    c.table_stride = rnd(5);
    const long long page = 1ll << c.page_shift;
    const long long max_length = rnd(400);
    c.capacity = std::min<long long>(max_length, c.table_stride * page);
    std::vector<int> off(c.B + 1, 0), len(c.B), table((size_t)c.B * c.table_stride);
    for (int b = 0; b < c.B; ++b) {
      off[b + 1] = off[b] + (rnd(3) ? rnd(90) : 0);
      const int k = rnd(8);
      len[b] = k == 0 ? -2147483647 - 1 : (k == 1 ? 2147483647 : rnd(500) - 50);
    }
    for (auto& p : table) p = rnd(6) ? rnd(10) - 1 : (rnd(2) ? 2147483647 : -2147483647 - 1);
    c.offsets = off.data();
    c.lengths = len.data();
    c.table = table.data();
    c.total = off[c.B] + rnd(3);
    for (long long row = 0; row < off[c.B]; ++row) {
      const int b = chunk_seq(c, row);
      if (b < 0 || b >= c.B || off[b] > row || off[b + 1] <= row) return printf("sequence of row %lld\n", row), 1;
      const long long pos = (long long)c.lengths[b] - (c.offsets[b + 1] - row);
      const long long at = cache_row(c, b, pos);
      const bool in = pos >= 0 && pos < max_length && pos < c.table_stride * page &&
                      (unsigned)table[(size_t)b * c.table_stride + pos / page] < (unsigned)c.n_pages;
      if (in != (at >= 0)) return printf("membership of position %lld\n", pos), 1;
      if (!in) { ++bad; continue; }
      ++good;
      const long long want =
          (long long)table[(size_t)b * c.table_stride + pos / page] * c.planes * c.kv_heads * page + pos % page;
      if (at != want) return printf("row of position %lld\n", pos), 1;
      const long long last = at + (long long)(c.planes * c.kv_heads - 1) * page;  // the last plane and head
      if (last >= (long long)c.n_pages * c.planes * c.kv_heads * page) return printf("past the cache\n"), 1;
    }
  }
  if (good < 1000 || bad < 1000) return printf("coverage %lld %lld\n", good, bad), 1;
  const float amax[] = {448.f, 448.0625f, 224.f, 224.03125f, 1.75f, 1.7500001f, 0.f, 1e-38f, 1e-45f, 3e38f, 1.f, 5e-31f, 1e30f};
  for (float a : amax) printf("%.9g %d\n", a, scale_exponent(a));
  printf("inf %d\n", scale_exponent(1.0f / 0.0f));
  return 0;
}
"""


def test_index_and_scale_arithmetic(tmp_path):
    out = _run(tmp_path, "index.cpp", "g++",
               ["-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-D_GLIBCXX_ASSERTIONS",
                "-include", "algorithm", "-I", os.path.join(ROOT, "wukong_hstu_cross_b200", "csrc")], INDEX)
    for line in out.splitlines():
        a, e = line.split()
        if a == "inf":
            assert int(e) == H.E_HI
        else:
            assert int(e) == int(H.quantise(np.array([[np.float32(a)]]))[1][0]), line


CUTS = r"""
#include <cstdio>
#include "chunk_index.h"
using namespace whale;

int main() {
  unsigned seed = 7;
  auto rnd = [&](int n) { seed = seed * 1664525u + 1013904223u; return (int)((seed >> 8) % (unsigned)n); };
  const int far[] = {-2147483647 - 1, -1, 0, 1, 2147483647};
  auto any = [&](int n) { return rnd(4) ? rnd(n) : far[rnd(5)]; };  // what memory may hold
  long long good = 0, bad = 0;
  for (int t = 0; t < 3000000; ++t) {
    ChunkView c{};
    const int group = 1 + rnd(4), bm = rnd(2) ? 16 : 256, slices = 1 + rnd(40), slice = rnd(slices);
    c.kv_heads = 1 + rnd(3);
    c.total = rnd(60);
    const int first_row = any(60), row0 = any(80), n_rows = any(20), head0 = any(12), parts = any(40);
    const int slot = rnd(2) ? 2 * slice + rnd(2) : any(80);
    if (!cut_valid(c, group, bm, slices, slice, first_row, row0, n_rows, head0, parts, slot)) { ++bad; continue; }
    ++good;
    for (int k = 0; k < parts; ++k) {
      const int s = k == 0 ? slot : 2 * (slice + k);
      if (s < 0 || s >= 2 * slices) return printf("slot %d of %d slices\n", s, slices), 1;
    }
    if (n_rows < 1 || n_rows > bm) return printf("rows\n"), 1;
    for (int r = row0; r < row0 + n_rows; ++r) {
      const long long row = (long long)first_row + r / group;
      const int head = head0 + r % group;
      if (r < 0 || row < 0 || row >= c.total || head < 0 || head >= c.kv_heads * group) return printf("row %lld head %d\n", row, head), 1;
    }
  }
  // one that a slice leaves: 3 slices, rows 4 .. 6 of a sequence at row 10
  ChunkView c{};
  c.kv_heads = 2;
  c.total = 14;
  if (!cut_valid(c, 2, 16, 5, 1, 10, 4, 3, 2, 3, 3) || cut_valid(c, 2, 16, 5, 1, 0, 0, 0, 0, 0, 0)) return printf("cut\n"), 1;
  if (good < 1000 || bad < 1000) return printf("coverage %lld %lld\n", good, bad), 1;
  return 0;
}
"""


def test_a_join_takes_only_cuts_in_range(tmp_path):
    """A slice whose wait ran out leaves no word of its item; whatever the workspace then holds, the join of the partials
    forms no index outside them or the rows."""
    _run(tmp_path, "cuts.cpp", "g++", ["-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                                       "-I", os.path.join(ROOT, "wukong_hstu_cross_b200", "csrc")], CUTS)


@pytest.mark.parametrize("h,hk,dh", [(8, 8, 64), (8, 2, 64), (4, 1, 32), (16, 4, 32)])
@pytest.mark.parametrize("fmt", [W.WHALE_CACHE_BF16, W.WHALE_CACHE_E4M3])
def test_the_attention_workspace_of_larger_bounds_serves_smaller_ones(h, hk, dh, fmt):
    """A program that allocates once, for its largest chunk: no smaller or sparser one may need more."""
    cfg = _cfg(d=h * dh, h=h)
    k = _cache(n_kv_heads=hk, format=fmt, scales=FAKE)
    size = lambda n, total, B, length: W.whale_cache_attention_workspace_size(  # noqa: E731
        cfg, k, _chunk(max_new=n, total_new=total, B=B, max_length=length, table_stride=1024))
    news, totals, batches = (0, 1, 2, 4, 8, 9, 16, 17, 32, 33, 100, 4096), (1, 2, 16, 17, 33, 640, 2048, 1 << 18), (1, 2, 20, 64, 1500)
    for lengths in (0, 100, 1 << 16):
        for i, n in enumerate(news):
            for j, total in enumerate(totals):
                for b, B in enumerate(batches):
                    got = size(n, total, B, lengths)
                    assert got > 0
                    for less in ((news[max(i - 1, 0)], total, B), (n, totals[max(j - 1, 0)], B), (n, total, batches[max(b - 1, 0)])):
                        assert size(*less, lengths) <= got, ((n, total, B), less)


def test_descriptors_of_another_device_are_refused(monkeypatch):
    """Descriptors are checked when they are made and once more at the call, when another device may be current. Empty
    calls, so that nothing is launched either way; CPU tensors stand for those of another device."""
    import torch

    zeros = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    bf16 = torch.bfloat16
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    rows = W.head_rows(zeros(0, 256, dtype=bf16), zeros(32, dtype=torch.float32), zeros(0), y=zeros(0, 256, dtype=bf16))
    grads = W.head_grads(zeros(0, 256, dtype=bf16), zeros(0, 256, dtype=bf16), zeros(32, dtype=torch.float32))
    cache = W.make_cache(zeros(2, 2, 8, 16, 32, dtype=bf16))
    chunk = W.make_chunk(zeros(1), zeros(0), zeros(0, 1), 0, 0, 0)
    ws, cfg, rotary = zeros(1 << 16, dtype=torch.uint8), _cfg(), W.make_rotary(32)
    calls = [
        lambda: W.whale_norm_rotate(cfg, rotary, rows, None, stream=0),
        lambda: W.whale_norm_rotate(cfg, rotary, None, rows, stream=0),
        lambda: W.whale_norm_rotate_backward(cfg, rotary, None, None, grads, None, W.WHALE_BF16, FAKE, 0, stream=0),
        lambda: W.whale_norm_rotate_backward(cfg, rotary, None, None, None, None, W.WHALE_BF16, ws, stream=0),
        lambda: W.whale_cache_append(cfg, cache, _chunk(B=0), FAKE, stream=0),
        lambda: W.whale_cache_read(cfg, _cache(), chunk, FAKE, stream=0),
        lambda: W.whale_cache_attention(cfg, cache, _chunk(B=0), FAKE, FAKE, FAKE, 0, stream=0),
        lambda: W.whale_cache_attention(cfg, _cache(), chunk, FAKE, FAKE, FAKE, 0, stream=0),
        lambda: W.whale_cache_attention(cfg, _cache(), _chunk(B=0), FAKE, FAKE, ws, stream=0),
    ]
    for call in calls:
        call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for call in calls:
        with pytest.raises(ValueError):
            call()
