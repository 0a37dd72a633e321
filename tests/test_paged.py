"""The paged cache without a GPU: the book of pages, the scalings of rotary
frequencies, and what the C entry points refuse."""
from __future__ import annotations

import ctypes
import math
import os
import random
import subprocess
import sys

import numpy as np
import pytest
import torch

import entropy_coded_kv_b200 as ecco
from entropy_coded_kv_b200 import _lib
from entropy_coded_kv_b200.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


# ------------------------------------------------------------------ the book of pages
def consistent(a, seqs):
    users = [0] * a.n_pages
    for s in seqs:
        assert len(a.pages(s)) == -(-a.length(s) // a.page_size)
        assert len(set(a.pages(s))) == len(a.pages(s))
        for p in a.pages(s):
            users[p] += 1
    assert users == a._users
    assert sorted(a._free) == [p for p in range(a.n_pages) if users[p] == 0]


@pytest.mark.parametrize("page_size", [1, 3, 16])
def test_book_against_a_model_of_the_tokens(page_size):
    """Random requests; a model holds what each sequence's tokens are, pages are
    written only by the sequence that extends, and no sequence's tokens change
    through another's."""
    rng = random.Random(page_size)
    a = ecco.PageAllocator(40, page_size)
    want, memory = {}, {}
    stamp = 0
    for _ in range(800):
        op = rng.choice(["add", "extend", "extend", "extend", "fork", "free", "shrink", "compact"])
        if op == "add" and len(want) < 6:
            want[a.add()] = []
        elif op == "fork" and want and len(want) < 8:
            s = rng.choice(list(want))
            want[a.fork(s)] = list(want[s])
        elif op == "free" and want:
            s = rng.choice(list(want))
            a.free(s)
            del want[s]
        elif op == "shrink" and want:
            s = rng.choice(list(want))
            n = rng.randint(0, len(want[s]))
            a.shrink(s, n)
            want[s] = want[s][:n]
        elif op == "compact" and want:
            seqs = rng.sample(list(want), rng.randint(1, min(2, len(want))))
            before = {s: a.pages(s) for s in want}, a.free_pages
            try:
                fresh = a.replace(seqs)
            except ecco.OutOfPages:
                assert ({s: a.pages(s) for s in want}, a.free_pages) == before
                continue
            kept = [[t for t in want[s] if rng.random() < 0.5] for s in seqs]
            for pages, tokens in zip(fresh, kept):
                for i, t in enumerate(tokens):
                    memory[pages[i // page_size], i % page_size] = t
            a.settle(seqs, fresh, [len(k) for k in kept])
            want.update(zip(seqs, kept))
        elif op == "extend" and want:
            seqs = rng.sample(list(want), rng.randint(1, min(3, len(want))))
            new = [rng.randint(0, 2 * page_size + 1) for _ in seqs]
            before = {s: (a.pages(s), a.length(s)) for s in want}, a.free_pages
            try:
                copies = a.extend(seqs, new)
            except ecco.OutOfPages:
                assert ({s: (a.pages(s), a.length(s)) for s in want}, a.free_pages) == before
                continue
            src, dst = [c[0] for c in copies], [c[1] for c in copies]
            assert len(set(dst)) == len(dst) and not set(dst) & set(src)
            snapshot = dict(memory)
            for f, t in copies:
                for i in range(page_size):
                    if (f, i) in snapshot:
                        memory[t, i] = snapshot[f, i]
            for s, n in zip(seqs, new):
                for _ in range(n):
                    i = len(want[s])
                    stamp += 1
                    memory[a.pages(s)[i // page_size], i % page_size] = stamp
                    want[s].append(stamp)
        consistent(a, want)
        for s, tokens in want.items():
            assert a.length(s) == len(tokens)
            assert [memory[a.pages(s)[i // page_size], i % page_size] for i in range(len(tokens))] == tokens


def test_book_refusals():
    a = ecco.PageAllocator(2, 4)
    s = a.add()
    for seqs, new in (([s, s], [1, 1]), ([s], [1, 2]), ([s], [-1])):
        with pytest.raises(ValueError):
            a.extend(seqs, new)
    with pytest.raises(ecco.OutOfPages):
        a.extend([s], [9])
    assert a.free_pages == 2 and a.length(s) == 0
    a.extend([s], [5])
    with pytest.raises(ValueError):
        a.shrink(s, 6)
    with pytest.raises(ValueError):
        a.replace([s, s])
    with pytest.raises(KeyError):
        a.free(99)


# ------------------------------------------------------------------ rotary frequencies
def test_frequencies():
    f, m = ecco.rope_frequencies(64, 500000.0)
    assert m == 1.0 and f == [500000.0 ** (-i / 32) for i in range(32)]
    assert ecco.rope_frequencies(64, scaling={"kind": "linear", "factor": 4})[0] == [x / 4 for x in ecco.rope_frequencies(64)[0]]
    g, _ = ecco.rope_frequencies(64, scaling={"kind": "ntk", "factor": 4})
    base = ecco.rope_frequencies(64)[0]
    assert g[0] == base[0] and math.isclose(g[-1], base[-1] / 4, rel_tol=1e-12)
    for kind in ("bands", "yarn"):
        g, m = ecco.rope_frequencies(128, 10000.0, {"kind": kind, "factor": 8, "original": 4096})
        base = ecco.rope_frequencies(128)[0]
        turns = [4096 * x / (2 * math.pi) for x in base]
        ratio = [x / y for x, y in zip(g, base)]
        assert all(a >= b - 1e-12 for a, b in zip(ratio, ratio[1:]))  # slower pairs are stretched more
        high = 4 if kind == "bands" else 32
        assert all(math.isclose(r, 1.0) for r, t in zip(ratio, turns) if t > high * 1.3)
        assert all(math.isclose(r, 0.125) for r, t in zip(ratio, turns) if t < 1 / 1.3)
        assert any(0.13 < r < 0.99 for r in ratio)
        assert math.isclose(m, 1.0 if kind == "bands" else 0.1 * math.log(8) + 1)
    # halfway between the bands' bounds, in turns
    x = 2.5 * 2 * math.pi / 4096
    i = min(range(64), key=lambda i: abs(base[i] - x))
    keep = (4096 * base[i] / (2 * math.pi) - 1) / 3
    g, _ = ecco.rope_frequencies(128, 10000.0, {"kind": "bands", "factor": 8, "original": 4096})
    assert math.isclose(g[i], base[i] * keep + base[i] / 8 * (1 - keep))
    for bad in ({"kind": "other", "factor": 2}, {"kind": "linear", "factor": 0.5}, {"kind": "yarn", "factor": 2, "original": 0},
                {"kind": "bands", "factor": 2, "original": 100, "low": 5, "high": 4}, {"kind": "linear", "factor": float("inf")}):
        with pytest.raises(ValueError):
            ecco.rope_frequencies(64, 10000.0, bad)
    with pytest.raises(ValueError):
        ecco.rope_frequencies(63)
    with pytest.raises(ValueError):
        ecco.rope_frequencies(64, 1.0)


def test_yarn_on_its_ramp():
    """Pinned by hand: 128 values, base 10000, a context of 4096 stretched 8 times.  The pair that turns t times has the
    index 128 ln(4096 / (2 pi t)) / (2 ln 10000): 20.94 for 32 turns, 45.03 for one.  So the ramp goes from 20 to 46:
    pair 33 is halfway, kept by 1/2 and stretched by 1/2: 1/2 + 1/16 of its frequency."""
    base = ecco.rope_frequencies(128)[0]
    f, m = ecco.rope_frequencies(128, 10000.0, {"kind": "yarn", "factor": 8, "original": 4096})
    ratio = [x / y for x, y in zip(f, base)]
    for i, want in ((0, 1.0), (20, 1.0), (21, 25 / 26 + 1 / 208), (33, 0.5625), (45, 1 / 26 + 25 / 208), (46, 0.125), (63, 0.125)):
        assert math.isclose(ratio[i], want, rel_tol=1e-12), i
    assert math.isclose(m, 1.2079441541679836, rel_tol=1e-14)  # 0.1 ln 8 + 1
    # other bounds of the ramp: 16 turns 25.76, 2 turns 40.21: from 25 to 41, pair 33 halfway again
    f, _ = ecco.rope_frequencies(128, 10000.0, {"kind": "yarn", "factor": 2, "original": 4096, "low": 2, "high": 16})
    assert math.isclose(f[33] / base[33], 0.75, rel_tol=1e-12) and math.isclose(f[29] / base[29], 0.875, rel_tol=1e-12)


# ------------------------------------------------------------------ refusals, no device
def paged(**kw):
    f = dict(n_pages=8, page_size=16, kv_heads=2, batch=1, max_pages=4, table_stride=4, page_table=4096, kv_lens=4096,
             cu_q=4096)
    f.update(kw)
    return _lib.Paged(*f.values())


def compact(lib, p, keep=4096, keep_stride=64, dst=4096, dst_stride=4, dst_max=4, lens=4096, pages=4096):
    return lib.ecco_compact_pages(p, pages, pages, keep, keep_stride, dst, dst_stride, dst_max, lens, None)


BAD_PAGED = [dict(n_pages=-1), dict(page_size=0), dict(page_size=65537), dict(kv_heads=0), dict(kv_heads=1025),
             dict(batch=-1), dict(batch=1025), dict(max_pages=-1), dict(max_pages=1 << 27), dict(table_stride=-1),
             dict(batch=2, table_stride=3), dict(page_table=None), dict(kv_lens=None), dict(n_pages=1 << 31),
             dict(n_pages=0x7fffffff, kv_heads=1024, page_size=65536, max_pages=1)]


@pytest.mark.parametrize("bad", BAD_PAGED, ids=lambda d: ",".join(f"{k}={v}" for k, v in d.items()))
def test_bad_caches_are_refused(lib, bad):
    assert compact(lib, paged(**bad)) == _lib.ECCO_ERR_ARG


def test_compact_refusals(lib):
    p = paged()
    assert compact(lib, p, keep=None) == _lib.ECCO_ERR_ARG
    assert compact(lib, p, keep_stride=-1) == _lib.ECCO_ERR_ARG
    assert compact(lib, p, dst=None) == _lib.ECCO_ERR_ARG
    assert compact(lib, p, dst_max=-1) == _lib.ECCO_ERR_ARG
    assert compact(lib, p, lens=None) == _lib.ECCO_ERR_ARG
    assert compact(lib, p, pages=None) == _lib.ECCO_ERR_ARG
    assert compact(lib, paged(batch=2), dst_stride=3) == _lib.ECCO_ERR_ARG
    assert compact(lib, p, pages=4104) == _lib.ECCO_ERR_ALIGN
    assert compact(lib, p, lens=4098) == _lib.ECCO_ERR_ALIGN
    assert compact(lib, paged(page_table=4097)) == _lib.ECCO_ERR_ALIGN
    # lengths written where others are read
    assert compact(lib, p) == _lib.ECCO_ERR_ARG
    assert compact(lib, paged(batch=3, kv_lens=8192), lens=8200) == _lib.ECCO_ERR_ARG
    assert compact(lib, paged(batch=3, kv_lens=8200), lens=8192) == _lib.ECCO_ERR_ARG
    assert compact(lib, paged(batch=0)) == _lib.ECCO_OK  # nothing to do


def test_copy_refusals(lib):
    def copy(src, dst, n_pages=8, page_bytes=128, k=4096, v=4096, n=None):
        a, b = ((ctypes.c_int32 * len(x))(*x) for x in (src, dst))
        return lib.ecco_copy_pages(k, v, n_pages, page_bytes, a, b, len(src) if n is None else n, None)

    assert copy([], []) == _lib.ECCO_OK
    for src, dst in (([0], [8]), ([8], [0]), ([-1], [0]), ([0], [-1]), ([0, 1], [2, 2]), ([0, 2], [2, 3]), ([1], [1])):
        assert copy(src, dst) == _lib.ECCO_ERR_ARG, (src, dst)
    assert copy([0], [1], n=-1) == _lib.ECCO_ERR_ARG
    assert copy([0], [1], n=9) == _lib.ECCO_ERR_ARG
    assert copy([0], [1], n_pages=-1) == _lib.ECCO_ERR_ARG
    assert copy([0], [1], page_bytes=100) == _lib.ECCO_ERR_ARG
    assert copy([0], [1], page_bytes=0) == _lib.ECCO_ERR_ARG
    assert copy([0], [1], k=None) == _lib.ECCO_ERR_ARG
    assert copy([0], [1], v=4100) == _lib.ECCO_ERR_ALIGN


def test_rope_refusals(lib):
    base = dict(x=4096, xt=256, xh=128, y=8192, yt=256, yh=128, dtype=0, tokens=3, heads=2, dim=128, table=4096, n=16,
                rotary=64, positions=4096, flags=0)

    def rope(**kw):
        return lib.ecco_rope(*{**base, **kw}.values(), None)

    for bad in (dict(dtype=3), dict(tokens=-1), dict(heads=0), dict(heads=65536), dict(dim=4), dict(dim=1032), dict(dim=132),
                dict(rotary=0), dict(rotary=8), dict(rotary=144), dict(rotary=40), dict(n=0), dict(flags=4), dict(x=None),
                dict(y=None), dict(table=None), dict(positions=None), dict(xt=-8), dict(yh=120), dict(yt=128),
                dict(yt=0), dict(yh=0), dict(y=4096, yt=512)):
        assert rope(**bad) == _lib.ECCO_ERR_ARG, bad
    for bad in (dict(xt=260), dict(yh=132), dict(x=4104), dict(y=8200), dict(table=4104), dict(positions=4098)):
        assert rope(**bad) == _lib.ECCO_ERR_ALIGN, bad
    assert rope(tokens=0) == _lib.ECCO_OK
    f = (ctypes.c_double * 2)(1.0, 0.5)
    table = lambda freq=f, n=2, mag=1.0, pos=4, out=4096: lib.ecco_rope_table(freq, n, mag, pos, out, None)  # noqa: E731
    for bad in (dict(freq=None), dict(n=0), dict(n=513), dict(mag=math.inf), dict(pos=0), dict(out=None),
                dict(freq=(ctypes.c_double * 2)(math.nan, 1.0))):
        assert table(**bad) == _lib.ECCO_ERR_ARG, bad
    assert table(out=4100) == _lib.ECCO_ERR_ALIGN


def test_calls_without_tables_are_refused(lib):
    p = paged()
    assert lib.ecco_paged_append(None, None, p, 4096, 256, 128, 4096, 256, 128, 1, 4096, 4096, None, 0, 0, None, 0, None,
                                 None) == _lib.ECCO_ERR_ARG
    assert lib.ecco_paged_attention(None, None, p, 4096, 4096, 4096, 256, 128, 1, 1, 1, 64, 0, 1.0, 4096, 256, 128, None,
                                    4096, 1 << 30, None) == _lib.ECCO_ERR_ARG


def test_workspace_sizes(lib):
    size = lib.ecco_paged_attention_workspace_bytes
    for bad in ((-1, 1, 1, 1, 1), (1025, 1, 1, 1, 1), (1, 0, 1, 1, 1), (1, 1025, 1, 1, 1), (1, 1, 0, 1, 1), (1, 1, 17, 1, 1),
                (1, 1, 1, -1, 1), (1, 1, 1, 1, -1), (1, 1, 1, 1, (1 << 30) + 1), (1024, 1, 1, 1, 1 << 30)):
        assert size(*bad) == 0, bad
    # K and V tiles of 128 tokens x 256 bytes, the KV heads in rounds of at most 1 GiB
    tiles = lambda batch, heads, kv: 2 * batch * heads * -(-kv // 128) * 128 * 256  # noqa: E731
    assert size(8, 8, 4, 1, 4096) >= tiles(8, 8, 4096)
    assert size(4, 8, 4, 1, 131072) < tiles(4, 8, 131072) + (1 << 30) // 16
    assert size(1, 8, 4, 1, 0) > 0


def test_workspace_sizes_never_shrink():
    """One workspace, sized for the largest bounds, serves every smaller call."""
    size = ecco.paged_attention_workspace_bytes
    base = dict(batch=1, kv_heads=8, group=4, max_q=500, max_kv=262144)
    steps = {"batch": range(1, 70), "kv_heads": range(1, 70), "group": range(1, 17), "max_q": range(0, 300),
             "max_kv": [n for m in range(1, 4000, 7) for n in (128 * m, 128 * m + 1)]}
    for at in (base, dict(base, batch=3, max_kv=50000), dict(base, batch=16, max_q=1, max_kv=16384), dict(base, kv_heads=3, max_q=1)):
        for name, values in steps.items():
            got = [size(**{**at, name: v}) for v in values]
            assert all(0 < a <= b for a, b in zip(got, got[1:])), (at, name)
    assert size(1, 8, 4, 500, 262144) <= size(1, 8, 4, 500, 300000)
    assert size(16, 8, 4, 1, 16384) <= size(17, 8, 4, 1, 16384)


def test_workspace_bounds_are_the_ones_the_header_states():
    """batch to 1024, group to 16, max_q to 2^26, max_kv to 2^30, batch * ceil(max_kv / 128) to 2^24, whatever the KV heads."""
    size = ecco.paged_attention_workspace_bytes
    for good, bad in (((1024, 1024, 1, 1, 1 << 21), (1024, 1, 1, 1, (1 << 21) + 1)), ((1, 1, 16, 1 << 26, 1), (1, 1, 16, (1 << 26) + 1, 1)),
                      ((2, 1024, 16, 1, 1 << 30), (2, 1, 1, 1, (1 << 30) + 1)), ((1024, 1024, 16, 1, 1), (1025, 1, 1, 1, 1))):
        assert size(*good) > 0 and size(*bad) == 0
    src = open(os.path.join(ROOT, "include", "ecco.h")).read()
    assert "max_q up to 2^26, max_kv up to 2^30, batch * ceil(max_kv / 128)\n *               up to 2^24" in src


@pytest.mark.parametrize("at", range(5))
@pytest.mark.parametrize("value", [1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 31) - 1, -(1 << 32) + 4])
def test_workspace_sizes_of_numbers_past_32_bits_are_refused(at, value):
    """ctypes would pass their low 32 bits: 2^32 + 1 as one."""
    args = [1, 1, 1, 1, 1]
    args[at] = value
    with pytest.raises(ValueError):
        ecco.paged_attention_workspace_bytes(*args)


def test_page_numbers_are_taken_whole():
    """Lists and arrays of ints; a fraction or a number past 32 bits is no page number."""
    from entropy_coded_kv_b200.paged import _host_ids

    for good in ([3, 0, 7], (3, 0, 7), np.array([3, 0, 7]), torch.tensor([3, 0, 7], dtype=torch.int32),
                 torch.tensor([3, 9, 0, 9, 7, 9], dtype=torch.int32)[::2]):
        t = _host_ids(good, "src")
        assert t.dtype == torch.int32 and t.is_contiguous() and t.tolist() == [3, 0, 7]
    assert _host_ids([], "src").tolist() == []
    whole = np.arange(5, dtype=np.int32)
    assert _host_ids(whole, "src").data_ptr() == whole.ctypes.data and _host_ids(whole[::2], "src").tolist() == [0, 2, 4]
    with pytest.raises(TypeError):
        _host_ids(whole[:4].reshape(2, 2), "src")
    for bad in ([1.5], [1.0], np.array([1.0]), "1", ["1"], [[1]], torch.tensor([1]), torch.tensor([[1]], dtype=torch.int32), torch.tensor([1.0])):
        with pytest.raises(TypeError):
            _host_ids(bad, "src")
    for bad in ([1 << 31], [0, (1 << 32) + 1], np.array([(1 << 32) + 1]), [-(1 << 31) - 1]):
        with pytest.raises(ValueError):
            _host_ids(bad, "src")


@pytest.mark.parametrize("call", [
    lambda x: ecco.rope(x, x, x),
    lambda x: ecco.copy_pages(x, x, [0], [1]),
    lambda x: ecco.compact_pages(x, x, x, x, x, x),
])
def test_host_tensors_are_refused(call):
    with pytest.raises((TypeError, ValueError)):
        call(torch.zeros(2, 2, 2, 64, dtype=torch.uint8))
    with pytest.raises((TypeError, ValueError)):
        call(torch.zeros(2, 2, 64))


def test_the_package_imports_on_a_torch_without_cuda(lib):
    """Such a torch has none of _C's CUDA calls; the formats, the book of pages and the frequencies need no device."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_get")]:
    delattr(torch._C, name)
import entropy_coded_kv_b200 as ecco
assert ecco.PageAllocator(2, 4).free_pages == 2 and len(ecco.rope_frequencies(64)[0]) == 32
try:
    ecco.copy_pages(torch.zeros(2, 1, 1, 64, dtype=torch.uint8), torch.zeros(2, 1, 1, 64, dtype=torch.uint8), [0], [1])
except ValueError:
    print("refused")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "refused", r.stderr
