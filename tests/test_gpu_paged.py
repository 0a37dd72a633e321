"""The paged cache's operators on the GPU against plain 64-bit forms over the
oracle's codec (tests/paged_reference.py, which derives the tolerances)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import workloads as W
import entropy_coded_kv_b200 as ecco
from entropy_coded_kv_b200 import _lib
from paged_reference import attend, bits, f64, pool_decode, rotate, rotate_f32
from test_gpu_parity import inputs, table_set, to_dev_bf16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ rotary positions
def test_rope_table_values():
    for rotary, scaling in ((128, None), (64, {"kind": "yarn", "factor": 16, "original": 8192}), (16, {"kind": "linear", "factor": 3})):
        t = ecco.rope_table(131073, rotary, scaling=scaling).cpu().numpy()
        f, m = ecco.rope_frequencies(rotary, scaling=scaling)
        for p in (0, 1, 777, 65535, 131072):
            a = p * np.asarray(f)
            # one fp32 rounding of an fp64 value: half a step, and 2^-40 for fp64's own roundings of a far angle
            for got, want in ((t[p, :, 0], m * np.cos(a)), (t[p, :, 1], m * np.sin(a))):
                assert (np.abs(got - want) <= 2.0**-24 * np.abs(want) + 2.0**-36).all()


ROPE = [
    # tokens, heads, dim, rotary, interleaved, inverse, dtype
    (1, 1, 128, 128, False, False, torch.bfloat16),
    (7, 3, 128, 64, True, False, torch.bfloat16),
    (33, 5, 256, 192, False, True, torch.float16),
    (5, 2, 64, 16, True, True, torch.float32),
    (3, 1, 1024, 1024, False, False, torch.float32),
    (257, 8, 128, 96, False, False, torch.float16),
    (2000, 32, 128, 128, True, False, torch.bfloat16),
    (9, 4, 24, 16, False, False, torch.bfloat16),
]


@pytest.mark.parametrize("tokens,heads,dim,rotary,inter,inv,dtype", ROPE)
def test_rope(tokens, heads, dim, rotary, inter, inv, dtype):
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, heads, dim, generator=g).to(dtype)
    pos = torch.randint(0, 5000, (tokens,), generator=g, dtype=torch.int32)
    pos[0] = 4999
    table = ecco.rope_table(5000, rotary)
    y = ecco.rope(x.to(DEV), table, pos.to(DEV), interleaved=inter, inverse=inv).cpu()
    tn = table.cpu().numpy()
    want, size = rotate(x.double().numpy(), tn, pos.numpy(), rotary, inter, inv)
    # two products and a sum, half a step of fp32 each, then half a step of the type
    half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    assert (np.abs(y.double().numpy() - want) <= 2.0**-24 * 2.01 * size + half * 1.01 * np.abs(want) + 1e-7 * (dtype == torch.float16)).all()
    exact = torch.from_numpy(rotate_f32(x.float().numpy(), tn, pos.numpy(), rotary, inter, inv)).to(dtype)
    assert torch.equal(y, exact)


def test_rope_strides_in_place_and_far_positions():
    g = torch.Generator(device=DEV).manual_seed(1)
    table = ecco.rope_table(100, 64)
    big = torch.randn(19, 6, 4, 160, generator=g, device=DEV).to(torch.bfloat16)
    x = big[:, 1, :, 16:144]                     # a head's 128 values inside a wider row
    pos = i32([-5, 1000] + list(range(17)))      # outside the table: its first and last row
    clear = i32([0, 99] + list(range(17)))
    want = ecco.rope(x.contiguous(), table, clear)
    before = big.clone()
    assert torch.equal(ecco.rope(x, table, pos), want)
    out = torch.zeros(4, 19, 128, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    assert ecco.rope(x, table, pos, out=out) is out and torch.equal(out, want)
    assert torch.equal(big, before)
    ecco.rope(x, table, pos, out=x)              # in place: only these values change
    assert torch.equal(x, want)
    before[:, 1, :, 16:144] = want
    assert torch.equal(big, before)
    assert ecco.rope(x[:0], table, pos[:0]).shape == (0, 4, 128)
    # one token, one head: strides that say nothing
    one = torch.randn(128, 3, device=DEV)[:, :1].t().unsqueeze(0).contiguous().to(torch.bfloat16)
    assert ecco.rope(one, table, pos[:1]).shape == one.shape


@pytest.mark.parametrize("inter", [False, True])
def test_rope_gradient(inter):
    """The turn is linear: its gradient is the turn back, by the formula and by differences."""
    g = torch.Generator().manual_seed(3)
    x, dy = torch.randn(11, 2, 64, generator=g), torch.randn(11, 2, 64, generator=g)
    pos = torch.randint(0, 300, (11,), generator=g, dtype=torch.int32)
    table = ecco.rope_table(300, 48)
    tn = table.cpu().numpy()
    got = ecco.rope(dy.to(DEV), table, pos.to(DEV), interleaved=inter, inverse=True).cpu().double().numpy()
    i = np.arange(24)
    ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + 24)
    cs, sn = (tn[pos.numpy(), :, k][:, None].astype(np.float64) for k in (0, 1))
    d = dy.double().numpy()
    want = d.copy()  # d/da of (a cos - b sin) da + (b cos + a sin) db, and d/db
    want[..., ia], want[..., ib] = d[..., ia] * cs + d[..., ib] * sn, d[..., ib] * cs - d[..., ia] * sn
    assert (np.abs(got - want) <= 2.0**-24 * 2.01 * (np.abs(want) + 2 * np.abs(d).max())).all()
    f = lambda v: float((ecco.rope(v.to(DEV), table, pos.to(DEV), interleaved=inter).cpu().double() * dy.double()).sum())  # noqa: E731
    for at in ((0, 0, 0), (3, 1, 30), (10, 0, 47), (5, 1, 60)):
        h = torch.zeros_like(x)
        h[at] = 8.0  # linear: a large step loses nothing but roundings (1408 values of size 10 at 2^-23)
        assert abs((f(h) - f(-h)) / 16 - got[at]) <= 1408 * 10 * 2.0**-23


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("inv", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_records_its_gradient(inter, inv, dtype):
    """Through autograd: the same bits as the call for the gradient, by the formula and by differences."""
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(11, 3, 80, generator=g).to(dtype).to(DEV).requires_grad_()
    dy = torch.randn(11, 2, 64, generator=g).to(dtype).to(DEV)
    pos = torch.randint(0, 300, (11,), generator=g, dtype=torch.int32).to(DEV)
    table = ecco.rope_table(300, 48, scaling={"kind": "yarn", "factor": 4, "original": 100})
    x = wide[:, 1:, 8:72]
    with torch.no_grad():
        assert not ecco.rope(x, table, pos).requires_grad
    y = ecco.rope(x, table, pos, interleaved=inter, inverse=inv)
    assert torch.equal(y, ecco.rope(x.detach(), table, pos, interleaved=inter, inverse=inv))
    (got,) = torch.autograd.grad(y, wide, dy, retain_graph=True)
    want = torch.zeros_like(got)
    want[:, 1:, 8:72] = ecco.rope(dy, table, pos, interleaved=inter, inverse=not inv)
    assert torch.equal(got, want)
    formula, size = rotate(dy.cpu().double().numpy(), table.cpu().numpy(), pos.cpu().numpy(), 48, inter, not inv)
    half = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    assert (np.abs(got[:, 1:, 8:72].cpu().double().numpy() - formula) <= 2.0**-24 * 2.01 * size + half * 1.01 * np.abs(formula)).all()
    if dtype == torch.float32:
        f = lambda v: float((ecco.rope(v, table, pos, interleaved=inter, inverse=inv).double() * dy.double()).sum())  # noqa: E731
        for at in ((0, 0, 0), (3, 1, 30), (10, 0, 47), (5, 1, 60)):
            h = torch.zeros(11, 2, 64, device=DEV)
            h[at] = 8.0  # linear: a large step loses nothing but roundings (at most 4 values of size 10 at 2^-23)
            assert abs((f(h) - f(-h)) / 16 - float(got[:, 1:, 8:72][at])) <= 1408 * 10 * 2.0**-23
    # gradients that are one value everywhere, or begin between two 16-byte pieces; and the gradient's gradient
    ones = torch.ones_like(dy)
    (got,) = torch.autograd.grad(y.sum(), wide, retain_graph=True)
    assert torch.equal(got[:, 1:, 8:72], ecco.rope(ones, table, pos, interleaved=inter, inverse=not inv))
    odd = torch.zeros(dy.numel() + 1, dtype=dtype, device=DEV)[1:].view(dy.shape)
    odd.copy_(dy)
    (got,) = torch.autograd.grad(y, wide, odd, retain_graph=True)
    assert torch.equal(got, want)
    w = dy.clone().requires_grad_()
    (first,) = torch.autograd.grad(y, wide, w, create_graph=True)
    (second,) = torch.autograd.grad(first[:, 1:, 8:72], w, ones)
    assert torch.equal(second, ecco.rope(ones, table, pos, interleaved=inter, inverse=inv))
    for out in (x, torch.empty_like(dy)):
        with pytest.raises(ValueError):
            ecco.rope(x, table, pos, out=out)
    with torch.no_grad():
        out = torch.empty_like(dy)
        assert ecco.rope(x, table, pos, out=out) is out


def test_rope_and_its_gradient_captured():
    table, pos = ecco.rope_table(64, 64), torch.arange(9, dtype=torch.int32, device=DEV)
    x = torch.randn(9, 2, 64, device=DEV, requires_grad=True)
    dy = torch.randn(9, 2, 64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        (dx,) = torch.autograd.grad(ecco.rope(x, table, pos), x, dy)
    for seed in range(2):
        dy.copy_(torch.randn(9, 2, 64, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        assert torch.equal(dx, ecco.rope(dy, table, pos, inverse=True))


# ------------------------------------------------------------------ append
def meta(lens, new, page_size, n_pages, seed, width=None):
    """(page_table, kv_lens, cu_q) with pages drawn at random, -1 past a sequence's pages."""
    rng = np.random.default_rng(seed)
    width = width or max(1, max(-(-n // page_size) for n in lens))
    ids = list(rng.permutation(n_pages))
    table = np.full((len(lens), width), -1, np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // page_size)):
            table[b, i] = ids.pop()
    return table, np.asarray(lens, np.int32), np.cumsum([0] + list(new)).astype(np.int32)


def encode_ref(blob, x):
    return oracle.encode(blob, np.ascontiguousarray(x).reshape(-1, 128).reshape(-1), nthreads=8)


APPEND = [
    # new, lens, H, page, rotary, interleaved, k kind, v kind
    ([1], [1], 1, 16, 128, False, "kv", "kv"),
    ([1, 1, 1], [5, 64, 65], 8, 64, 128, False, "kv", "special"),
    ([70, 0, 3, 200], [70, 9, 131, 450], 2, 48, 64, True, "special", "t5"),
    ([33, 5], [40, 5], 3, 1, 32, False, "kv", "gauss"),
    ([400], [1000], 4, 100, 0, False, "c1", "kv"),
    ([17], [300], 5, 128, 96, True, "kv", "kv"),
]


@pytest.mark.parametrize("new,lens,H,page,rotary,inter,kk,vk", APPEND)
def test_append_matches_the_oracle(new, lens, H, page, rotary, inter, kk, vk):
    kt, vt = table_set("learned_kv"), table_set("random1")
    T, n_pages = sum(new), sum(-(-n // page) for n in lens) + 2
    table, kvl, cu = meta(lens, new, page, n_pages, seed=T)
    pad = 3  # rows before the first sequence and behind the last: not read into any page
    k = to_dev_bf16(inputs(kk, (T + 2 * pad) * H, seed=1).reshape(T + 2 * pad, H, 128))
    v = to_dev_bf16(inputs(vk, (T + 2 * pad) * H, seed=2).reshape(T + 2 * pad, H, 128))
    kp = torch.randint(0, 256, (n_pages, H, page, 64), dtype=torch.uint8, device=DEV)
    vp = torch.randint(0, 256, (n_pages, H, page, 64), dtype=torch.uint8, device=DEV)
    wk, wv = kp.cpu().numpy(), vp.cpu().numpy()
    rt = ecco.rope_table(max(lens), rotary) if rotary else None
    stats = ecco.new_stats(DEV)
    ecco.paged_append(k, v, kp, vp, ecco.Tables(kt), ecco.Tables(vt), i32(table), i32(kvl), i32(cu + pad), rope=rt,
                      interleaved=inter, stats=stats)
    b = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)]).astype(np.int64)
    kb, vb = bits(k)[pad:pad + T], bits(v)[pad:pad + T]
    if rotary:
        turned = rotate_f32(f64(kb).astype(np.float32), rt.cpu().numpy(), pos, rotary, inter)
        kb = bits(torch.from_numpy(turned).to(torch.bfloat16))
    (ek, sk), (ev, sv) = encode_ref(kt, kb), encode_ref(vt, vb)
    wk[table[b, pos // page], :, pos % page] = ek.reshape(T, H, 64)
    wv[table[b, pos // page], :, pos % page] = ev.reshape(T, H, 64)
    np.testing.assert_array_equal(kp.cpu().numpy(), wk)
    np.testing.assert_array_equal(vp.cpu().numpy(), wv)
    got = ecco.read_stats(stats)
    for name in ("n_groups", "n_zero", "n_clipped", "n_padded", "n_records", "n_nonfinite", "payload_bits"):
        assert got[name] == getattr(sk, name) + getattr(sv, name), name


def test_append_strides_positions_and_bad_entries():
    """k and v inside a fused projection's output, other angles than the
    positions, and tokens that have no place: they leave the pools alone."""
    kt = vt = table_set("learned_kv")
    H, page, n_pages = 4, 16, 6
    lens, new = [40, 3, 20], [8, 5, 4]          # the second: two of its tokens lie before position 0
    table = np.array([[0, 1, 2], [3, -1, -1], [99, 4, -1]], np.int32)
    cu = np.cumsum([0] + new).astype(np.int32)
    qkv = to_dev_bf16(inputs("kv", 17 * 12, seed=5).reshape(17, 12, 128))
    k, v = qkv[:, 4:8], qkv[:, 8:12]
    pos = np.arange(100, 117).astype(np.int32)
    rt = ecco.rope_table(110, 128)
    kp = torch.randint(0, 256, (n_pages, H, page, 64), dtype=torch.uint8, device=DEV)
    vp = kp.clone()
    wk, wv = kp.cpu().numpy(), vp.cpu().numpy()
    ecco.paged_append(k, v, kp, vp, ecco.Tables(kt), ecco.Tables(vt), i32(table), i32(lens), i32(cu), rope=rt, positions=i32(pos))
    turned = rotate_f32(f64(bits(k)).astype(np.float32), rt.cpu().numpy(), pos, 128, False)
    ek = encode_ref(kt, bits(torch.from_numpy(turned).to(torch.bfloat16)))[0].reshape(17, H, 64)
    ev = encode_ref(vt, bits(v))[0].reshape(17, H, 64)
    for b in range(3):
        for i in range(new[b]):
            p = lens[b] - new[b] + i
            if p < 0 or not 0 <= table[b, p // page] < n_pages:
                continue
            wk[table[b, p // page], :, p % page] = ek[cu[b] + i]
            wv[table[b, p // page], :, p % page] = ev[cu[b] + i]
    np.testing.assert_array_equal(kp.cpu().numpy(), wk)
    np.testing.assert_array_equal(vp.cpu().numpy(), wv)
    # lengths past the row's pages, and below zero
    for bad in (1000, -3, 2**31 - 1, -2**31):
        ecco.paged_append(k[:1], v[:1], kp, vp, ecco.Tables(kt), ecco.Tables(vt), i32(table[:1]), i32([bad]), i32([0, 1]))
    np.testing.assert_array_equal(kp.cpu().numpy(), wk)


# ------------------------------------------------------------------ attention
def fill_pool(blob, n_pages, H, page, kind, seed):
    b, _ = oracle.encode(blob, inputs(kind, n_pages * H * page, seed=seed), nthreads=8)
    return b.reshape(n_pages, H, page, 64)


ATTEND = [
    # new, lens, H, G, page, window, scale, K tables, V tables, K kind, V kind
    ([1], [1], 1, 1, 16, 0, 0.0884, "learned_kv", "learned_kv", "kv", "kv"),
    ([1], [650], 2, 4, 16, 0, 0.0884, "learned_kv", "learned_kv", "kv", "kv"),
    ([1, 1, 1, 1], [127, 128, 129, 1000], 2, 4, 64, 0, 0.0884, "learned_kv", "random1", "kv", "kv"),
    ([64], [64], 1, 4, 64, 0, 0.0884, "learned_kv", "learned_kv", "kv", "kv"),
    ([65, 1, 0, 33], [65, 300, 17, 200], 2, 5, 48, 0, 0.0884, "random0", "learned_kv", "gauss", "kv"),
    ([129], [700], 1, 8, 100, 0, 0.0884, "learned_kv", "learned_kv", "kv", "t5"),
    ([40, 7], [350, 129], 1, 3, 1, 100, 0.0884, "learned_kv", "learned_kv", "kv", "kv"),
    ([200, 1], [600, 513], 2, 2, 128, 130, -0.05, "learned_kv", "learned_kv", "kv", "kv"),
    ([5, 3], [2, 0], 2, 4, 16, 0, 0.0884, "learned_kv", "learned_kv", "kv", "kv"),     # rows that see nothing
    ([3], [260], 1, 16, 33, 1, 0.0884, "learned_kv", "learned_kv", "kv", "kv"),        # a window of one: the values themselves
    ([10], [150], 3, 7, 16, 0, 0.0, "learned_kv", "learned_kv", "kv", "kv"),           # scale 0: the mean
    ([30], [257], 1, 4, 24, 0, 0.0884, "random3", "random2", "special", "special"),
    ([300], [300], 1, 1, 64, 0, 1.0, "learned_kv", "learned_kv", "kv", "kv"),          # scores of hundreds
]


def run_attention(kb, vb, kt, vt, q, table, lens, cu, scale, **kw):
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    got = ecco.paged_attention(q, torch.from_numpy(kb).to(DEV), torch.from_numpy(vb).to(DEV), ecco.Tables(kt), ecco.Tables(vt),
                               i32(table), i32(lens), i32(cu), scale, out=out, lse=lse, **kw)
    assert got is out
    return f64(bits(out)), lse.cpu().double().numpy()


def check_attention(out, lse, ref):
    want, wlse, tol, tol_lse, written = ref
    assert (out[~written] == 7.0).all() and (lse[~written] == 7.0).all()
    out, lse, want, wlse, tol, tol_lse = (a[written] for a in (out, lse, want, wlse, tol, tol_lse))
    assert np.isfinite(out).all()
    err = np.abs(out - want)
    assert (err <= tol).all(), f"worst excess {(err / np.maximum(tol, 1e-38)).max():.3f} of the tolerance"
    none = np.isneginf(wlse)
    assert np.isneginf(lse[none]).all() and (out[none] == 0).all()
    assert (np.abs(lse[~none] - wlse[~none]) <= tol_lse[~none]).all()


@pytest.mark.parametrize("new,lens,H,G,page,window,scale,ktn,vtn,kk,vk", ATTEND)
def test_attention(new, lens, H, G, page, window, scale, ktn, vtn, kk, vk):
    one_attention(new, lens, H, G, page, window, scale, ktn, vtn, kk, vk)


def one_attention(new, lens, H, G, page, window, scale, ktn, vtn, kk, vk, **bounds):
    kt, vt = table_set(ktn), table_set(vtn)
    n_pages = sum(-(-n // page) for n in lens) + 1
    table, kvl, cu = meta(lens, new, page, n_pages, seed=len(lens) + page)
    kb, vb = fill_pool(kt, n_pages, H, page, kk, 3), fill_pool(vt, n_pages, H, page, vk, 4)
    pad = 2
    T = sum(new) + 2 * pad
    q = torch.randn(T, H * G, 128, generator=torch.Generator().manual_seed(T)).to(torch.bfloat16).to(DEV)
    out, lse = run_attention(kb, vb, kt, vt, q, table, kvl, cu + pad, scale, window=window, **bounds)
    ref = attend(f64(bits(q)), pool_decode(kt, kb), pool_decode(vt, vb), table, kvl, cu + pad, scale, window)
    check_attention(out, lse, ref)


@pytest.mark.parametrize("new,lens,H,G,page,window,scale,ktn,vtn,kk,vk", ATTEND)
def test_attention_with_a_wide_bound(new, lens, H, G, page, window, scale, ktn, vtn, kk, vk):
    """max_kv far above every length chooses the kernels, not the result."""
    one_attention(new, lens, H, G, page, window, scale, ktn, vtn, kk, vk, max_kv=1 << 14)


FEW = [
    # new, lens, H, G, page, window, scale: at most 32 rows an item over few tiles
    ([1], [128], 8, 4, 16, 0, 0.0884),
    ([1], [129], 8, 4, 16, 0, 0.0884),
    ([1], [650], 8, 4, 16, 0, 0.0884),
    ([1, 1], [1000, 90], 8, 4, 64, 0, 0.0884),
    ([1], [1100], 3, 5, 24, 0, 0.0884),
    ([1, 2], [2500, 300], 2, 4, 48, 0, 0.0884),
    ([1] * 37, list(range(1, 112, 3)), 4, 1, 8, 0, 0.0884),
    ([1, 2, 0, 3], [900, 513, 300, 2], 3, 4, 100, 0, -0.05),
    ([8], [1100], 2, 4, 24, 200, 0.0884),
    ([32], [33], 1, 1, 7, 0, 0.0884),
    ([16, 5], [256, 5], 2, 2, 32, 3, 0.0884),
    ([4, 2, 1], [1, 0, 300], 2, 4, 16, 0, 0.0884),     # rows that see nothing
    ([4, 2], [1, 0], 2, 4, 16, 0, 0.0884),             # in a call of one tile
    ([2], [700], 1, 16, 33, 1, 0.0884),
    ([3], [300], 2, 7, 16, 0, 0.0),
    ([6], [400], 1, 4, 128, 0, 1.0),
    ([2, 1, 0, 2, 2], [0, 300, 500, 1, 129], 2, 3, 16, 0, 0.0884),
    ([2, 1], [1000, 500], 3, 4, 48, 300, -0.05),
    ([8, 8], [1024, 8], 1, 1, 32, 2, 0.0884),
]


@pytest.mark.parametrize("new,lens,H,G,page,window,scale", FEW)
@pytest.mark.parametrize("kk,vk,max_kv", [("kv", "kv", None), ("special", "special", None), ("kv", "kv", 1 << 14)])
def test_attention_few_rows(new, lens, H, G, page, window, scale, kk, vk, max_kv):
    one_attention(new, lens, H, G, page, window, scale, "learned_kv", "random1", kk, vk, max_q=max(new), max_kv=max_kv)


@pytest.mark.parametrize("most_new,most_kv,H,G,window", [(1, 128, 8, 4, 0), (1, 700, 5, 3, 0), (30, 300, 4, 4, 0), (2, 1500, 3, 2, 140)])
def test_attention_many_short_sequences(most_new, most_kv, H, G, window):
    """More items than CTAs, of one to a few tiles: runs of equal, shorter and longer ones, some with no row or no key."""
    rng = np.random.default_rng(most_kv)
    new = rng.integers(0, most_new + 1, 110)
    new[new == 0] = rng.integers(0, 2, (new == 0).sum())
    lens = rng.integers(0, most_kv + 1, 110)
    lens[:40] = np.repeat(lens[:10], 4)  # neighbours of the same length
    one_attention(new.tolist(), lens.tolist(), H, G, 64, window, 0.0884, "learned_kv", "random1", "kv", "kv", max_q=most_new)


@pytest.mark.parametrize("new,lens,H,G,window", [([530], [700], 2, 16, 0), ([1100, 3], [1300, 90], 1, 16, 300), ([5, 600], [400, 600], 1, 16, 0)])
def test_attention_many_items_of_a_sequence(new, lens, H, G, window):
    """More than 32 items of 256 rows in a sequence, more than 64 too: a share's first item is searched 32 at a time, and
    so are a sequence's units summed."""
    assert max(new) * G > 32 * 256
    one_attention(new, lens, H, G, 64, window, 0.0884, "learned_kv", "random1", "kv", "kv")


@pytest.mark.parametrize("new,lens,H,G,window", [([1], [131072], 1, 4, 0), ([1, 2], [100_001, 50_000], 1, 2, 0), ([3], [131_000], 1, 4, 100_000),
                                                 ([40], [70_000], 1, 4, 0)])
def test_attention_over_a_long_context(new, lens, H, G, window):
    """An item cut into tens of parts, all of them joined."""
    one_attention(new, lens, H, G, 64, window, 0.0884, "learned_kv", "random1", "kv", "kv", max_q=max(new))


def test_attention_few_rows_bounds_garbage_and_bad_pages():
    kt, vt = table_set("learned_kv"), table_set("random1")
    rng = np.random.default_rng(9)
    H, G, page, n_pages = 2, 4, 24, 40
    kb, vb = (rng.integers(0, 256, (n_pages, H, page, 64), dtype=np.uint8) for _ in range(2))
    table = rng.permutation(n_pages)[:39].reshape(3, 13).astype(np.int32)
    table[0, 2], table[1, 5], table[2, 0] = -1, n_pages, 2**31 - 1
    lens, new = np.array([300, 1000, 130], np.int32), [8, 5, 1]
    cu = np.cumsum([0] + new).astype(np.int32)
    q = torch.randn(14, H * G, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    kd, vd = pool_decode(kt, kb), pool_decode(vt, vb)
    for max_q, max_kv, window in ((8, 312, 0), (8, 131, 0), (7, 312, 140), (1, 1, 0), (8, 0, 0), (8, 2000, 130), (3, 128, 0), (2, 312, 0), (2, 2000, 140)):
        out, lse = run_attention(kb, vb, kt, vt, q, table, lens, cu, 1e-3, max_q=max_q, max_kv=max_kv, window=window)
        check_attention(out, lse, attend(f64(bits(q)), kd, vd, table, lens, cu, 1e-3, window, max_q, max_kv))
    for bad_lens, bad_cu in (([-5, 2**31 - 1, -2**31], cu), (lens, [0, 40, 60, 90]), (lens, [-7, 3, 2, 30])):
        for window in (0, 100):
            run_attention(kb, vb, kt, vt, q, table, bad_lens, bad_cu, 1e-3, max_q=8, window=window)
            torch.cuda.synchronize()


@pytest.mark.parametrize("kv,G", [(100, 4), (900, 4), (1300, 4), (900, 1)])
def test_attention_few_rows_nan_query_and_strides(kv, G):
    """A NaN or infinite query spoils its own row only; q and out inside wider arrays, and one array."""
    kt = vt = table_set("learned_kv")
    H, page, new = 2, 16, [7]
    table, kvl, cu = meta([kv], new, page, -(-kv // page) + 1, seed=1)
    kb, vb = (torch.from_numpy(fill_pool(kt, -(-kv // page) + 1, H, page, "kv", n)).to(DEV) for n in (3, 4))
    wide = torch.randn(7, 3, H * G, 136, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    q = wide[:, 1, :, 8:]
    rest = (kb, vb, ecco.Tables(kt), ecco.Tables(vt), i32(table), i32(kvl), i32(cu), 0.0884)
    clean = ecco.paged_attention(q.contiguous(), *rest)
    q[5, 1, 5], q[2, 0, 0] = float("nan"), float("inf")
    home = torch.zeros(H * G, 7, 144, dtype=torch.bfloat16, device=DEV)
    out = home.transpose(0, 1)[..., :128]
    ecco.paged_attention(q, *rest, out=out)
    assert out[5, 1].isnan().all()
    same = torch.ones(7, H * G, dtype=torch.bool, device=DEV)
    same[5, 1] = same[2, 0] = False
    assert torch.equal(out[same], clean[same]) and (home[..., 128:] == 0).all()
    assert ecco.paged_attention(q, *rest, out=q) is q and torch.equal(q[same], clean[same])


def test_attention_bounds_garbage_and_bad_pages():
    """Random bytes as blocks, entries that name no page, lengths past the row's
    pages, and bounds below what the arrays say."""
    kt, vt = table_set("learned_kv"), table_set("random1")
    rng = np.random.default_rng(8)
    H, G, page, n_pages = 2, 4, 24, 20
    kb, vb = (rng.integers(0, 256, (n_pages, H, page, 64), dtype=np.uint8) for _ in range(2))
    table = rng.permutation(n_pages)[:18].reshape(3, 6).astype(np.int32)
    table[0, 2], table[1, 5], table[2, 0] = -1, n_pages, 2**31 - 1
    lens, new = np.array([140, 1000, 130], np.int32), [20, 9, 1]
    cu = np.cumsum([0] + new).astype(np.int32)
    q = torch.randn(30, H * G, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    kd, vd = pool_decode(kt, kb), pool_decode(vt, vb)
    for max_q, max_kv in ((20, 144), (20, 131), (7, 144), (1, 1), (20, 0)):
        out, lse = run_attention(kb, vb, kt, vt, q, table, lens, cu, 1e-3, max_q=max_q, max_kv=max_kv)
        check_attention(out, lse, attend(f64(bits(q)), kd, vd, table, lens, cu, 1e-3, 0, max_q, max_kv))
    # arrays that make no sense stay inside the buffers and write no row twice
    for bad_lens, bad_cu in (([-5, 2**31 - 1, -2**31], cu), (lens, [0, 40, 60, 90]), (lens, [-7, 3, 2, 30])):
        run_attention(kb, vb, kt, vt, q, table, bad_lens, bad_cu, 1e-3)
        torch.cuda.synchronize()


def test_attention_nan_query_and_strides():
    """A NaN or infinite query spoils its own row only; q and out inside wider arrays."""
    kt = vt = table_set("learned_kv")
    H, G, page, lens, new = 2, 4, 16, [200], [40]
    table, kvl, cu = meta(lens, new, page, 14, seed=1)
    kb, vb = fill_pool(kt, 14, H, page, "kv", 3), fill_pool(vt, 14, H, page, "kv", 4)
    wide = torch.randn(40, 3, H * G, 136, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    q = wide[:, 1, :, 8:]
    clean = ecco.paged_attention(q.contiguous(), torch.from_numpy(kb).to(DEV), torch.from_numpy(vb).to(DEV), ecco.Tables(kt),
                                 ecco.Tables(vt), i32(table), i32(kvl), i32(cu), 0.0884)
    q[7, 3, 5], q[11, 0, 0] = float("nan"), float("inf")
    home = torch.zeros(H * G, 40, 144, dtype=torch.bfloat16, device=DEV)
    out = home.transpose(0, 1)[..., :128]
    ecco.paged_attention(q, torch.from_numpy(kb).to(DEV), torch.from_numpy(vb).to(DEV), ecco.Tables(kt), ecco.Tables(vt),
                         i32(table), i32(kvl), i32(cu), 0.0884, out=out)
    assert out[7, 3].isnan().all()
    same = torch.ones(40, H * G, dtype=torch.bool, device=DEV)
    same[7, 3] = same[11, 0] = False
    assert torch.equal(out[same], clean[same]) and (home[..., 128:] == 0).all()


def test_attention_masked_slots_never_count():
    """Blocks past a sequence's length, in its last page and in pages behind it, change nothing."""
    kt = vt = table_set("learned_kv")
    H, G, page, lens, new = 1, 4, 64, [130, 70], [3, 70]
    table, kvl, cu = meta(lens, new, page, 9, seed=2, width=4)
    table[table < 0] = 9  # a tenth page, no sequence's own
    kb, vb = fill_pool(kt, 10, H, page, "kv", 3), fill_pool(vt, 10, H, page, "kv", 4)
    q = torch.randn(73, G, 128, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    a = run_attention(kb, vb, kt, vt, q, table, kvl, cu, 0.0884)
    rng = np.random.default_rng(0)
    for b in range(2):
        for i in range(lens[b], table.shape[1] * page):
            kb[table[b, i // page], :, i % page] = rng.integers(0, 256, (H, 64))
            vb[table[b, i // page], :, i % page] = rng.integers(0, 256, (H, 64))
    b = run_attention(kb, vb, kt, vt, q, table, kvl, cu, 0.0884)
    np.testing.assert_array_equal(a[0], b[0])
    np.testing.assert_array_equal(a[1], b[1])


def test_single_token_matches_decode_attention():
    """One token a sequence over equal lengths is the framework's decode-phase
    attention: both within their tolerances of one 64-bit reference, so of each
    other within the sum."""
    kt = vt = table_set("learned_kv")
    B, H, G, S, page = 3, 2, 4, 1000, 40
    kb, vb = fill_pool(kt, B, H, S, "kv", 3), fill_pool(vt, B, H, S, "kv", 4)
    kp, vp = (x.reshape(B, H, S // page, page, 64).transpose(0, 2, 1, 3, 4).reshape(-1, H, page, 64).copy() for x in (kb, vb))
    table = np.arange(B * (S // page), dtype=np.int32).reshape(B, -1)
    q = torch.randn(B, H * G, 128, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(DEV)
    out, _ = run_attention(kp, vp, kt, vt, q, table, [S] * B, np.arange(B + 1), 0.0884)
    t = ecco.Tables(kt)
    other = ecco.decode_attention(torch.from_numpy(kb).to(DEV), torch.from_numpy(vb).to(DEV), t, t, q, S, 0.0884).cpu().double().numpy()
    ref = attend(f64(bits(q)), pool_decode(kt, kp), pool_decode(vt, vp), table, [S] * B, np.arange(B + 1), 0.0884, 0)
    assert (np.abs(out - other) <= ref[2] + 1e-3 * ref[2] * 2.0**8).all()


def test_attention_many_sequences_share_pages():
    """More sequences than a warp plans at once, most of them on the same pages
    (a shared prefix), lengths from zero on, in another order than the pages."""
    kt, vt = table_set("learned_kv"), table_set("random1")
    H, G, page, n_pages, B = 1, 2, 16, 30, 700
    rng = np.random.default_rng(11)
    kb, vb = fill_pool(kt, n_pages, H, page, "kv", 3), fill_pool(vt, n_pages, H, page, "kv", 4)
    lens = rng.integers(0, 160, B).astype(np.int32)
    new = np.minimum(rng.choice([0, 1, 1, 1, 2, 70], B), np.maximum(lens, 1)).astype(np.int32)
    table = rng.integers(0, n_pages, (B, 10)).astype(np.int32)
    table[:, 0] = 7
    cu = np.cumsum(np.r_[0, new]).astype(np.int32)
    q = torch.randn(int(cu[-1]), H * G, 128, generator=torch.Generator().manual_seed(12)).to(torch.bfloat16).to(DEV)
    ref = attend(f64(bits(q)), pool_decode(kt, kb), pool_decode(vt, vb), table, lens, cu, 0.0884, 0)
    out, lse = run_attention(kb, vb, kt, vt, q, table, lens, cu, 0.0884)
    check_attention(out, lse, ref)
    for _ in range(3):  # the same call gives the same bits
        again = run_attention(kb, vb, kt, vt, q, table, lens, cu, 0.0884)
        np.testing.assert_array_equal(again[0], out)
        np.testing.assert_array_equal(again[1], lse)
    # one token each, no more than 32 rows an item
    one, cu1 = np.minimum(lens, 1), np.cumsum(np.r_[0, np.minimum(lens, 1)]).astype(np.int32)
    q1 = q[: int(cu1[-1])].contiguous()
    out, lse = run_attention(kb, vb, kt, vt, q1, table, lens, cu1, 0.0884, max_q=1)
    check_attention(out, lse, attend(f64(bits(q1)), pool_decode(kt, kb), pool_decode(vt, vb), table, lens, cu1, 0.0884, 0))


def test_attention_in_rounds_of_heads():
    """Bounds that allow so many keys that the KV heads are taken one by one."""
    kt = vt = table_set("learned_kv")
    H, G, page, lens, new = 3, 4, 64, [300, 1], [70, 1]
    table, kvl, cu = meta(lens, new, page, 8, seed=3, width=1 << 13)
    kb, vb = fill_pool(kt, 8, H, page, "kv", 3), fill_pool(vt, 8, H, page, "kv", 4)
    q = torch.randn(71, H * G, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    assert 1 << 30 < ecco.paged_attention_workspace_bytes(2, H, G, 71, page << 13) < (1 << 30) + (1 << 26)
    out, lse = run_attention(kb, vb, kt, vt, q, table, kvl, cu, 0.0884)
    check_attention(out, lse, attend(f64(bits(q)), pool_decode(kt, kb), pool_decode(vt, vb), table, kvl, cu, 0.0884, 0))


def test_attention_in_rounds_of_one_head():
    """Bounds at which one head's tiles take more than a round: the heads one by one, 2 GiB each."""
    kt = vt = table_set("learned_kv")
    H, G, page, lens, new = 3, 4, 64, [300, 1], [70, 1]
    table, kvl, cu = meta(lens, new, page, 8, seed=3, width=1 << 14)
    kb, vb = fill_pool(kt, 8, H, page, "kv", 3), fill_pool(vt, 8, H, page, "kv", 4)
    q = torch.randn(71, H * G, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    size = ecco.paged_attention_workspace_bytes(2, H, G, 71, 2 * page << 14)
    assert 2 << 30 < size < (2 << 30) + (1 << 26) and size == ecco.paged_attention_workspace_bytes(2, 1, G, 71, 2 * page << 14)
    out, lse = run_attention(kb, vb, kt, vt, q, table, kvl, cu, 0.0884, max_kv=2 * page << 14)
    check_attention(out, lse, attend(f64(bits(q)), pool_decode(kt, kb), pool_decode(vt, vb), table, kvl, cu, 0.0884, 0))


def test_attention_with_a_workspace_of_larger_bounds():
    """A workspace sized once for the largest batch and length, at bounds below them."""
    kt = vt = table_set("learned_kv")
    H, G, page, lens, new = 8, 4, 64, [300, 1, 130], [70, 1, 2]
    ws = torch.empty(ecco.paged_attention_workspace_bytes(3, H, G, 100, 100_000), dtype=torch.uint8, device=DEV)
    table, kvl, cu = meta(lens, new, page, 12, seed=3)
    kb, vb = fill_pool(kt, 12, H, page, "kv", 3), fill_pool(vt, 12, H, page, "kv", 4)
    q = torch.randn(73, H * G, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    ref = attend(f64(bits(q)), pool_decode(kt, kb), pool_decode(vt, vb), table, kvl, cu, 0.0884, 0)
    for max_kv in (1 << 16, 87_381, 90_000, 100_000, 1000, 300):  # 8 heads a round, then 7, then 6
        out, lse = run_attention(kb, vb, kt, vt, q, table, kvl, cu, 0.0884, max_q=70, max_kv=max_kv, workspace=ws)
        check_attention(out, lse, ref)


def test_attention_empty_tables_and_pools():
    t = ecco.Tables(table_set("learned_kv"))
    q = torch.randn(3, 4, 128, device=DEV).to(torch.bfloat16)
    for kp in (torch.zeros(0, 2, 16, 64, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)):
        for width in (0, 3):
            lse = torch.zeros(3, 4, device=DEV)
            table = torch.full((2, width), 9, dtype=torch.int32, device=DEV)
            out = ecco.paged_attention(q, kp, kp, t, t, table, i32([0, 0]), i32([0, 1, 3]), 1.0, lse=lse)
            assert (out == 0).all() and torch.isneginf(lse).all()
            ecco.paged_append(q[:, :2].contiguous(), q[:, :2].contiguous(), kp, kp.clone(), t, t, table, i32([0, 0]), i32([0, 1, 3]))
            assert ecco.compact_pages(kp, kp.clone(), table, i32([5, 5]), torch.ones(2, 64, dtype=torch.bool, device=DEV), table).tolist() == (
                [0, 0] if width == 0 else [5, 5])  # counted, but no page to move to
    none = torch.zeros(0, 4, 128, dtype=torch.bfloat16, device=DEV)
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    assert ecco.paged_attention(none, kp, kp, t, t, i32(np.zeros((0, 3))), i32([]), i32([0]), 1.0).shape == (0, 4, 128)
    with pytest.raises(ecco.EccoError):  # keys and values into one pool
        ecco.paged_append(q[:, :2].contiguous(), q[:, :2].contiguous(), kp, kp, t, t, i32([[0], [1]]), i32([1, 2]), i32([0, 1, 3]))


def test_pools_past_32_bits():
    """Pages whose byte offsets need more than 32 bits: append, attention, copy, compaction."""
    kt = vt = table_set("learned_kv")
    H, G, page, n_pages = 8, 4, 64, 150_000  # 4.9 GB a pool
    kT = ecco.Tables(kt)
    kp, vp = (torch.zeros(n_pages, H, page, 64, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = np.array([[149_999, 3, 140_000], [131_073, 149_998, 7]], np.int32)
    lens, new = [150, 130], [150, 130]
    cu = [0, 150, 280]
    k, v = (to_dev_bf16(inputs("kv", 280 * H, seed=s).reshape(280, H, 128)) for s in (1, 2))
    ecco.paged_append(k, v, kp, vp, kT, kT, i32(table), i32(lens), i32(cu))
    used = table.reshape(-1)
    rows = torch.from_numpy(used.astype(np.int64)).to(DEV)
    small = lambda pool: pool[rows].cpu().numpy()  # noqa: E731
    want = encode_ref(kt, bits(k))[0].reshape(280, H, 64)
    got = small(kp).reshape(2, 3, H, page, 64)
    for b in range(2):
        for t in range(new[b]):
            np.testing.assert_array_equal(got[b, t // page, :, t % page], want[cu[b] + t])
    q = torch.randn(280, H * G, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).to(DEV)
    sub = np.arange(6, dtype=np.int32).reshape(2, 3)

    def compare(tab):
        out = ecco.paged_attention(q, kp, vp, kT, kT, i32(tab), i32(lens), i32(cu), 0.0884)
        alone = ecco.paged_attention(q, kp[rows].contiguous(), vp[rows].contiguous(), kT, kT, i32(sub), i32(lens), i32(cu), 0.0884)
        assert torch.equal(out, alone)

    compare(table)
    other = np.array([[139_000, 149_000, 148_000], [5, 147_000, 146_000]], np.int32)
    ecco.copy_pages(kp, vp, used.tolist(), other.reshape(-1).tolist())
    assert torch.equal(kp[rows], kp[torch.from_numpy(other.reshape(-1).astype(np.int64)).to(DEV)])
    compare(other)
    third = np.array([[120_000, 149_997], [149_996, 8]], np.int32)
    keep = torch.zeros(2, 192, dtype=torch.bool, device=DEV)
    keep[:, 1::2] = True
    assert ecco.compact_pages(kp, vp, i32(other), i32(lens), keep, i32(third)).tolist() == [75, 65]
    for b in range(2):
        for t in range(65):
            assert torch.equal(vp[third[b, t // page], :, t % page], vp[other[b, (2 * t + 1) // page], :, (2 * t + 1) % page])


@pytest.mark.parametrize("lens,new", [([700, 90], [100, 1]), ([700, 90], [1, 1]), ([1500, 90], [3, 1])])
def test_attention_in_place_and_on_two_streams(lens, new):
    """out = q, and two calls at once on two streams with a workspace each."""
    kt = vt = table_set("learned_kv")
    H, G, page = 2, 4, 16
    table, kvl, cu = meta(lens, new, page, 110, seed=1)
    kp, vp = (torch.from_numpy(fill_pool(kt, 110, H, page, "kv", s)).to(DEV) for s in (3, 4))
    kT, tb, kv, cq = ecco.Tables(kt), i32(table), i32(kvl), i32(cu)
    qs = [torch.randn(sum(new), H * G, 128, device=DEV).to(torch.bfloat16) for _ in range(2)]
    want = [ecco.paged_attention(q, kp, vp, kT, kT, tb, kv, cq, 0.0884) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for s, q, o in zip(streams, qs, outs):
            with torch.cuda.stream(s):
                o.append(ecco.paged_attention(q, kp, vp, kT, kT, tb, kv, cq, 0.0884))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
    for w, q in zip(want, qs):
        assert ecco.paged_attention(q, kp, vp, kT, kT, tb, kv, cq, 0.0884, out=q) is q and torch.equal(q, w)


def test_attention_refuses_after_a_wait_gave_up():
    """The diagnostic kernel's wait runs out: the next attention call says so, until the flag is cleared."""
    import ctypes

    lib = _lib.load()
    n = ctypes.c_uint()
    assert lib.ecco_device_timeouts(ctypes.byref(n)) == _lib.ECCO_OK
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device=DEV)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    call = lambda: ecco.paged_attention(q, kp, kp, t, t, i32([[0]]), i32([1]), i32([0, 1]), 1.0)  # noqa: E731
    call()
    assert lib.ecco_selftest_wait_timeout(None) == _lib.ECCO_OK
    torch.cuda.synchronize()
    with pytest.raises(ecco.EccoError) as e:
        call()
    assert e.value.code == _lib.ECCO_ERR_TIMEOUT
    m = ctypes.c_uint()
    assert lib.ecco_device_timeouts(ctypes.byref(m)) == _lib.ECCO_OK and m.value == n.value + 1
    call()


# ------------------------------------------------------------------ pages
@pytest.mark.parametrize("pairs,H,page", [(1, 1, 1), (5, 8, 16), (4000, 1, 3), (7, 3, 100)])
def test_copy_pages(pairs, H, page):
    rng = np.random.default_rng(pairs)
    n = 2 * pairs + 1
    kp, vp = (torch.from_numpy(rng.integers(0, 256, (n, H, page, 64), dtype=np.uint8)).to(DEV) for _ in range(2))
    order = rng.permutation(n).astype(np.int32)
    src, dst = order[:pairs].copy(), order[pairs:2 * pairs]
    src[pairs // 2:] = src[0]  # one source for many
    wk, wv = kp.clone(), vp.clone()
    for w, p in ((wk, kp), (wv, vp)):
        w[torch.from_numpy(dst).long()] = p[torch.from_numpy(src).long()]
    ecco.copy_pages(kp, vp, torch.from_numpy(src), dst.tolist())
    assert torch.equal(kp, wk) and torch.equal(vp, wv)


@pytest.mark.parametrize("lens,H,page,kept", [([1], 1, 16, 1.0), ([0, 5], 2, 16, 0.5), ([3000, 1, 1024, 1025], 3, 48, 0.5),
                                              ([2500], 2, 7, 0.02), ([700, 650], 8, 64, 0.0), ([1024], 1, 128, 1.0)])
def test_compact_pages(lens, H, page, kept):
    rng = np.random.default_rng(sum(lens))
    width = max(1, max(-(-n // page) for n in lens))
    n_pages = 2 * len(lens) * width + 1
    kp, vp = (torch.from_numpy(rng.integers(0, 256, (n_pages, H, page, 64), dtype=np.uint8)).to(DEV) for _ in range(2))
    ids = rng.permutation(n_pages)[:2 * len(lens) * width].reshape(2, len(lens), width).astype(np.int32)
    keep = rng.random((len(lens), width * page)) < kept
    wk, wv = kp.cpu().numpy(), vp.cpu().numpy()
    want = []
    for b, n in enumerate(lens):
        t = np.flatnonzero(keep[b, :n])
        k = np.arange(len(t))
        for w in (wk, wv):
            w[ids[1, b, k // page], :, k % page] = w[ids[0, b, t // page], :, t % page]
        want.append(len(t))
    got = ecco.compact_pages(kp, vp, i32(ids[0]), i32(lens), torch.from_numpy(keep).to(DEV), i32(ids[1]))
    assert got.tolist() == want
    np.testing.assert_array_equal(kp.cpu().numpy(), wk)
    np.testing.assert_array_equal(vp.cpu().numpy(), wv)


def test_compact_bounds():
    """Too few destination pages, entries that name no page, lengths past the row, a short mask."""
    rng = np.random.default_rng(4)
    kp, vp = (torch.from_numpy(rng.integers(0, 256, (10, 2, 8, 64), dtype=np.uint8)).to(DEV) for _ in range(2))
    table, dst = np.array([[0, -1, 2, 10]], np.int32), np.array([[5, 77, 6]], np.int32)
    keep = np.ones((1, 30), np.uint8)
    wk = kp.cpu().numpy()
    for t in range(24):  # 30 tokens counted (the mask's end), room for 24; page 1 of the source and of the destination are missing
        if t // 8 != 1:
            wk[dst[0, t // 8], :, t % 8] = wk[table[0, t // 8], :, t % 8]
    got = ecco.compact_pages(kp, vp, i32(table), i32([1000]), torch.from_numpy(keep).to(DEV), i32(dst))
    assert got.tolist() == [24]
    np.testing.assert_array_equal(kp.cpu().numpy(), wk)


# ------------------------------------------------------------------ together
def test_cache_from_prompt_to_fork_to_compaction():
    """A run as a server makes it: prompts in chunks, single tokens, a fork whose
    copies diverge, dropped tokens, a freed sequence.  Every attention is
    checked against the 64-bit form over a plain list of (turned, encoded)
    tokens of each sequence."""
    H, G, page, layers, rotary = 2, 4, 16, 2, 64
    blobs = [(table_set("learned_kv"), table_set("random1")), (table_set("random0"), table_set("learned_kv"))]
    cache = ecco.PagedCache(40, page, H, [ecco.Tables(a) for a, _ in blobs], [ecco.Tables(b) for _, b in blobs])
    cache.k_pages.random_(0, 256)
    cache.v_pages.random_(0, 256)
    table = ecco.rope_table(1000, rotary, scaling={"kind": "yarn", "factor": 4, "original": 200})
    tn = table.cpu().numpy()
    g = torch.Generator().manual_seed(9)
    tokens = {}  # sequence -> per layer (k, v) fp64 [n, H, 128]
    position = {}

    def step(seqs, new):
        st = cache.extend(seqs, new)
        T = sum(new)
        pos = np.concatenate([np.arange(position[s], position[s] + n) for s, n in zip(seqs, new)])
        assert st.positions.tolist() == pos.tolist() and st.tokens == T
        for s, n in zip(seqs, new):
            position[s] += n
        for layer in range(layers):
            qkv = (torch.randn(T, (G + 2) * H, 128, generator=g) * 2).to(torch.bfloat16).to(DEV)
            q, k, v = qkv.split([G * H, H, H], 1)
            cache.append(st, layer, k, v, rope=table)
            qr = ecco.rope(q, table, st.positions)
            lse = torch.empty(T, G * H, device=DEV)
            out = cache.attend(st, layer, qr, 0.0884, lse=lse)
            turned = rotate_f32(f64(bits(k)).astype(np.float32), tn, pos, rotary, False)
            kb, vb = bits(torch.from_numpy(turned).to(torch.bfloat16)), bits(v)
            new_k, new_v = (f64(np.asarray(oracle.decode(t, encode_ref(t, x)[0]))).reshape(T, H, 128)
                            for t, x in zip(blobs[layer], (kb, vb)))
            at = 0
            for s, n in zip(seqs, new):
                old = tokens[s][layer]
                tokens[s][layer] = tuple(np.concatenate([a, b[at:at + n]]) for a, b in zip(old, (new_k, new_v)))
                kk, vv = tokens[s][layer]
                ref = attend(f64(bits(qr))[at:at + n], kk[None].transpose(0, 2, 1, 3), vv[None].transpose(0, 2, 1, 3),
                             np.zeros((1, 1), int), [len(kk)], [0, n], 0.0884, 0) if len(kk) else None
                if ref is not None and n:
                    check_attention(f64(bits(out))[at:at + n], lse.cpu().double().numpy()[at:at + n], ref)
                at += n

    def fresh():
        s = cache.add()
        tokens[s], position[s] = [(np.zeros((0, H, 128)),) * 2 for _ in range(layers)], 0
        return s

    a, b = fresh(), fresh()
    step([a, b], [37, 5])
    step([b, a], [20, 1])
    step([a, b], [0, 1])
    c = cache.fork(a)
    tokens[c], position[c] = [tuple(t) for t in tokens[a]], position[a]
    assert cache.book.pages(c) == cache.book.pages(a)
    step([a, c, b], [3, 2, 1])                       # the shared last page parts
    assert cache.book.pages(c)[:-1] == cache.book.pages(a)[:-1] and cache.book.pages(c)[-1] != cache.book.pages(a)[-1]
    step([c], [40])
    keep = torch.rand(2, 128, generator=g) < 0.4
    lens = cache.compact([c, b], keep.to(DEV))
    for s, row, n in zip((c, b), keep.numpy(), lens):
        tokens[s] = [tuple(x[row[:len(x)]] for x in layer) for layer in tokens[s]]
        assert cache.length(s) == n == len(tokens[s][0][0])
    step([a, b, c], [1, 1, 30])
    free = cache.book.free_pages
    cache.free(a)
    assert cache.book.free_pages > free
    d = fresh()
    step([d, c, b], [50, 1, 1])
    with pytest.raises(ecco.OutOfPages):
        cache.extend([d], [10000])
    step([d], [1])


@pytest.mark.parametrize("through_the_book", [False, True])
def test_cache_shrink_gives_positions_again(through_the_book):
    """A draft's rejected tokens: the ones that follow take their places, positions and all, as if the draft had never been."""
    H, G, page = 2, 4, 16
    t = ecco.Tables(table_set("learned_kv"))
    table = ecco.rope_table(64, 128)
    qkv = torch.randn(50, (G + 2) * H, 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)

    def step(cache, s, rows):
        st = cache.extend([s], [len(rows)])
        q, k, v = qkv[rows].split([G * H, H, H], 1)
        cache.append(st, 0, k, v, rope=table)
        return st.positions.tolist(), cache.attend(st, 0, ecco.rope(q, table, st.positions), 0.0884)

    drafted, plain = ecco.PagedCache(8, page, H, t, t), ecco.PagedCache(8, page, H, t, t)
    shrink = (lambda s, n: drafted.book.shrink(s, n)) if through_the_book else drafted.shrink
    a, b = drafted.add(), plain.add()
    step(drafted, a, list(range(30)))
    step(plain, b, list(range(30)))
    draft, _ = step(drafted, a, [30, 31, 32, 33, 34])
    assert draft == [30, 31, 32, 33, 34]
    fork = drafted.fork(a)                           # shares the draft; its own positions go on behind it
    shrink(a, 32)
    assert drafted.length(a) == 32 and drafted.length(fork) == 35
    got, out = step(drafted, a, [40, 41])
    step(plain, b, [30, 31])
    want, ref = step(plain, b, [40, 41])
    assert got == want == [32, 33] and torch.equal(out, ref)
    assert step(drafted, fork, [42])[0] == [35]
    # behind a compaction the positions go on from the last one given, and a draft's are given again
    keep = torch.arange(64, device=DEV)[None] % 2 == 0
    assert drafted.compact([a], keep) == [17]
    assert step(drafted, a, [43, 44])[0] == [34, 35]
    shrink(a, 18)
    assert step(drafted, a, [45])[0] == [35]
    shrink(a, 10)                                    # into the compacted tokens: none of their positions again
    assert step(drafted, a, [46, 47])[0] == [34, 35]
    shrink(a, 0)
    assert step(drafted, a, [48])[0] == [34] and drafted.length(a) == 1
    with pytest.raises(ValueError):
        drafted.shrink(a, 2)


@pytest.mark.parametrize("page", [1, 7, 16])
def test_cache_against_a_model_of_the_tokens(page):
    """Random requests, drafts taken back among them; each sequence's pages hold
    the blocks of its own tokens, turned by the positions that a model gives."""
    rng = np.random.default_rng(page)
    H, layers = 2, 2
    t, u = ecco.Tables(table_set("learned_kv")), ecco.Tables(table_set("random1"))
    cache = ecco.PagedCache(600 // page, page, H, [t, u], [u, t])
    table = ecco.rope_table(2000, 64)
    want, position, floor = {}, {}, {}               # blocks [layer][pool][tokens, H, 64]; next position; length and position after a compaction
    grown = 0

    def check(seq):
        n, pages = cache.length(seq), i32(cache.book.pages(seq)).long()
        assert n == want[seq][0][0].shape[0]
        at = torch.arange(n, device=DEV)
        for layer in range(layers):
            for pool, blocks in zip((cache.k_pages, cache.v_pages), want[seq][layer]):
                assert torch.equal(pool[layer][pages[at // page], :, at % page], blocks)

    for _ in range(150):
        op = rng.choice(["add", "extend", "extend", "extend", "fork", "free", "shrink", "compact"])
        seqs = list(want)
        if op == "add" and len(seqs) < 6:
            s = cache.add()
            want[s], position[s], floor[s] = [[torch.empty(0, H, 64, dtype=torch.uint8, device=DEV)] * 2] * layers, 0, (0, 0)
        elif op == "extend" and seqs:
            some = rng.permutation(seqs)[:rng.integers(1, 4)].tolist()
            new = rng.integers(0, 2 * page + 3, len(some)).tolist()
            try:
                st = cache.extend(some, new)
            except ecco.OutOfPages:
                continue
            assert st.positions.tolist() == [position[s] + i for s, n in zip(some, new) for i in range(n)]
            for layer in range(layers):
                k, v = (torch.randn(sum(new), H, 128, device=DEV).to(torch.bfloat16) for _ in range(2))
                cache.append(st, layer, k, v, rope=table)
                turned = ecco.rope(k, table, st.positions) if sum(new) else k
                blocks = [ecco.encode(x.reshape(-1), tb).view(-1, H, 64) if sum(new) else torch.empty(0, H, 64, dtype=torch.uint8, device=DEV)
                          for x, tb in ((turned, cache.k_tables[layer]), (v, cache.v_tables[layer]))]
                at = 0
                for s, n in zip(some, new):
                    want[s] = [[torch.cat([w, b[at:at + n]]) for w, b in zip(old, blocks)] if i == layer else old for i, old in enumerate(want[s])]
                    at += n
            for s, n in zip(some, new):
                position[s] += n
            grown += 1
        elif op == "fork" and seqs and len(seqs) < 6:
            s = rng.choice(seqs).item()
            f = cache.fork(s)
            want[f], position[f], floor[f] = want[s], position[s], floor[s]
        elif op == "free" and len(seqs) > 2:
            s = rng.choice(seqs).item()
            cache.free(s)
            del want[s], position[s], floor[s]
        elif op == "shrink" and seqs:
            s = rng.choice(seqs).item()
            n = int(rng.integers(0, cache.length(s) + 1))
            (cache if rng.random() < 0.5 else cache.book).shrink(s, n)
            kept, first = floor[s]
            position[s] = first + max(0, n - kept)
            floor[s] = min(n, kept), first
            want[s] = [[x[:n] for x in layer] for layer in want[s]]
        elif op == "compact" and seqs:
            some = rng.permutation(seqs)[:rng.integers(1, 3)].tolist()
            keep = torch.from_numpy(rng.random((len(some), 700)) < 0.6).to(DEV)
            try:
                lens = cache.compact(some, keep)
            except ecco.OutOfPages:
                continue
            for s, row, n in zip(some, keep, lens):
                want[s] = [[x[row[:x.shape[0]]] for x in layer] for layer in want[s]]
                floor[s] = n, position[s]
        for s in want:
            check(s)
    assert grown > 20


def test_cache_refuses_positions_past_the_rope_table():
    """The cache knows the positions: a key past the table would be turned by its last row, like the one before it."""
    t = ecco.Tables(table_set("learned_kv"))
    cache = ecco.PagedCache(8, 16, 2, t, t)
    table = ecco.rope_table(20, 128)
    s, other = cache.add(), cache.add()
    x = torch.randn(24, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    st = cache.extend([s, other], [20, 4])           # 0 .. 19: the table's last row
    assert st.max_position == 19
    cache.append(st, 0, x, x, rope=table)
    before = cache.k_pages.clone()
    st = cache.extend([s, other], [1, 1])            # 20
    with pytest.raises(ValueError, match="position 20"):
        cache.append(st, 0, x[:2], x[:2], rope=table)
    assert torch.equal(cache.k_pages, before)
    cache.append(st, 0, x[:2], x[:2], rope=ecco.rope_table(21, 128))
    cache.append(st, 0, x[:2], x[:2])
    assert cache.extend([other], [1]).max_position == 5
    none = cache.extend([s], [0])
    assert none.max_position == -1
    cache.append(none, 0, x[:0], x[:0], rope=table)


def test_cache_extend_waits_for_nothing():
    """A step is prepared while the device is still busy, the copies of forked pages included."""
    t = ecco.Tables(table_set("learned_kv"))
    cache = ecco.PagedCache(64, 16, 2, [t, t], [t, t])
    a, b = cache.add(), cache.add()
    cache.extend([a, b], [40, 3])
    cache.k_pages.random_(0, 256)
    cache.v_pages.random_(0, 256)
    forks = [cache.fork(a) for _ in range(2)]
    for fork, new in zip(forks, (1, 2)):             # the first one sets up whatever a first call sets up
        pages = cache.book.pages(fork)
        torch.cuda.synchronize()
        torch.cuda._sleep(400_000_000)               # about 0.2 s
        busy = torch.cuda.Event()
        busy.record()
        st = cache.extend([b, fork], [5, new])
        waited = busy.query()
        torch.cuda.synchronize()
    assert not waited
    assert st.page_table.tolist() == [cache.book.pages(b) + [-1] * 2, cache.book.pages(fork)] and len(cache.book.pages(b)) == 1
    assert st.kv_lens.tolist() == [13, 42] and st.cu_q.tolist() == [0, 5, 7] and st.positions.tolist() == [8, 9, 10, 11, 12, 40, 41]
    assert cache.book.pages(fork)[:2] == pages[:2] and cache.book.pages(fork)[2] != pages[2]
    for pool in (cache.k_pages, cache.v_pages):
        assert torch.equal(pool[:, pages[2]], pool[:, cache.book.pages(fork)[2]])
    before = cache.length(a), cache.book.free_pages
    side = torch.cuda.Stream()
    with pytest.raises(RuntimeError, match="captured"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):
            cache.extend([a], [100])
    assert (cache.length(a), cache.book.free_pages) == before
    none = cache.extend([], [])
    assert none.page_table.shape == (0, 0) and none.cu_q.tolist() == [0] and none.positions.numel() == 0


@pytest.mark.parametrize("max_kv", [240, 1 << 14])
def test_captured_step_replays_on_new_lengths_and_streams(max_kv):
    """Append and attention captured into a graph on a side stream; replays
    follow the page table and lengths written between them.  Two graphs share
    one workspace, replayed in order."""
    kt = vt = table_set("learned_kv")
    H, G, page, n_pages, B = 2, 4, 16, 40, 2
    kT, vT = ecco.Tables(kt), ecco.Tables(vt)
    kp, vp = (torch.from_numpy(fill_pool(kt, n_pages, H, page, "kv", s)).to(DEV) for s in (3, 4))
    table = np.random.default_rng(1).permutation(n_pages)[:30].reshape(2, 15).astype(np.int32)
    tb, lens, cu = i32(table), i32([10, 20]), i32([0, 1, 2])
    k, v, q = (torch.randn(B, n, 128, device=DEV).to(torch.bfloat16) for n in (H, H, H * G))
    ws = torch.empty(ecco.paged_attention_workspace_bytes(B, H, G, 1, max_kv), dtype=torch.uint8, device=DEV)
    rt = ecco.rope_table(240, 128)
    outs = [torch.empty_like(q) for _ in range(2)]
    side, graphs = torch.cuda.Stream(), []

    def once(o):
        ecco.paged_append(k, v, kp, vp, kT, vT, tb, lens, cu, rope=rt)
        ecco.paged_attention(q, kp, vp, kT, vT, tb, lens, cu, 0.0884, max_q=1, max_kv=max_kv, out=o, workspace=ws)

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        once(outs[0])
        for o in outs:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                once(o)
            graphs.append(gr)
        for n in ([10, 20], [11, 21], [240, 1], [128, 129]):
            lens.copy_(i32(n))
            k.copy_(torch.randn_like(k, dtype=torch.float32))
            for gr in graphs:
                gr.replay()
            side.synchronize()
            assert torch.equal(outs[0], outs[1])
            ref = attend(f64(bits(q)), pool_decode(kt, kp.cpu().numpy()), pool_decode(vt, vp.cpu().numpy()), table, n, [0, 1, 2], 0.0884, 0)
            assert (np.abs(f64(bits(outs[0])) - ref[0]) <= ref[2]).all()
    torch.cuda.current_stream().wait_stream(side)


def test_refusals_of_the_binding():
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    tb, lens, cu = i32([[0, 1]]), i32([5]), i32([0, 5])
    x = torch.zeros(5, 2, 128, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device=DEV)
    ok = dict(k_pages=kp, v_pages=kp.clone(), k_tables=t, v_tables=t, page_table=tb, kv_lens=lens, cu_q=cu)
    bad = [dict(k_pages=kp.float()), dict(v_pages=kp[:, :, :8]), dict(k_pages=kp[:2]), dict(page_table=tb.long()), dict(page_table=tb[0]),
           dict(kv_lens=i32([1, 2])), dict(cu_q=i32([0])), dict(kv_lens=lens.cpu()), dict(page_table=i32([[0], [1]]).t())]
    for b in bad:
        with pytest.raises((TypeError, ValueError)):
            if "page_table" in b and b["page_table"].dim() == 2 and b["page_table"].dtype == torch.int32:
                b = {**b, "page_table": i32([[0, 9], [1, 9]]).t()[:1]}
            ecco.paged_append(x, x, **{**ok, **b})
    for b in (dict(k=x.float()), dict(v=x[:3]), dict(k=x[..., :64]), dict(rope=torch.zeros(4, 8, device=DEV)),
              dict(positions=i32([1])), dict(stats=torch.zeros(2, dtype=torch.int64, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            ecco.paged_append(**{**dict(k=x, v=x), **ok, **b})
    with pytest.raises(ecco.EccoError):   # a table of more than 128 values
        ecco.paged_append(x, x, **ok, rope=ecco.rope_table(4, 256))
    for b in (dict(q=q[:, :7]), dict(q=q.half()), dict(out=q.float()), dict(lse=torch.zeros(5, 7, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            ecco.paged_attention(**{**dict(q=q, scale=1.0), **ok, **b})
    for b in (dict(scale=float("nan")), dict(window=-1), dict(max_q=-1), dict(max_kv=-1), dict(workspace=torch.zeros(64, dtype=torch.uint8, device=DEV)),
              dict(out=q[:, :1].expand(5, 8, 128)), dict(q=torch.zeros(5, 2 * 17, 128, dtype=torch.bfloat16, device=DEV))):
        with pytest.raises(ecco.EccoError):
            ecco.paged_attention(**{**dict(q=q, scale=1.0), **ok, **b})
    with pytest.raises(ecco.EccoError):
        ecco.copy_pages(kp, kp.clone(), [0, 1], [2, 2])
    with pytest.raises(TypeError):
        ecco.copy_pages(kp, kp.clone(), i32([0]), [1])
    with pytest.raises(ValueError):
        ecco.compact_pages(kp, kp.clone(), tb, lens, torch.ones(2, 9, dtype=torch.bool, device=DEV), tb)


def test_refusals_of_one_array_twice_and_of_wide_steps():
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    tb, lens, cu = i32([[0, 1]]), i32([5]), i32([0, 8])
    q = torch.zeros(8, 8, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ecco.EccoError):  # q's rows, head by head
        ecco.paged_attention(q, kp, kp, t, t, tb, lens, cu, 1.0, out=q.transpose(0, 1))
    with pytest.raises(ecco.EccoError):
        ecco.compact_pages(kp, kp.clone(), tb, lens, torch.ones(1, 32, dtype=torch.bool, device=DEV), i32([[2, 3]]), out_lens=lens)
    cache = ecco.PagedCache(8, 16, 2, t, t)
    seqs = [cache.add() for _ in range(_lib.MAX_BATCH + 1)]
    with pytest.raises(ValueError):
        cache.extend(seqs, [0] * len(seqs))
    with pytest.raises(ValueError):
        cache.compact(seqs, torch.ones(len(seqs), 1, dtype=torch.bool, device=DEV))
    assert cache.extend(seqs[1:], [0] * _lib.MAX_BATCH).tokens == 0


@pytest.mark.parametrize("name", ["max_q", "max_kv", "window"])
def test_bounds_past_32_bits_are_refused(name):
    """Not cut to their low 32 bits: a window of 2^32 + 5 is none of 5."""
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    q = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    for value in (1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32) + 5):
        for w in (None, ws):
            with pytest.raises(ValueError):
                ecco.paged_attention(q, kp, kp, t, t, i32([[0, 1]]), i32([20]), i32([0, 5]), 1.0, workspace=w, **{name: value})
    for value in (20, 64, 1 << 20):
        ecco.paged_attention(q, kp, kp, t, t, i32([[0, 1]]), i32([20]), i32([0, 5]), 1.0, **{name: value})


def test_refused_bounds_are_named():
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(4, 2, 16, 64, dtype=torch.uint8, device=DEV)
    q = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device=DEV)
    rest = (kp, kp, t, t, i32([[0, 1]]), i32([20]), i32([0, 5]), 1.0)
    for w in (None, ws):
        for bad in (dict(max_q=(1 << 26) + 1), dict(max_kv=(1 << 30) + 1)):
            with pytest.raises(ecco.EccoError, match="max_q up to 2.26") as e:
                ecco.paged_attention(q, *rest, workspace=w, **bad)
            assert e.value.code == _lib.ECCO_ERR_ARG
    with pytest.raises(ecco.EccoError, match="workspace of 65536 bytes"):
        ecco.paged_attention(q, *rest, workspace=ws)
    with pytest.raises(ecco.EccoError, match="argument"):
        ecco.paged_attention(q, *rest, window=-1)


def test_a_paged_wait_that_gives_up_is_counted_and_reported():
    """The paged kernels' own wait, on a barrier at which nothing arrives: it
    ends, the paged count goes up by one, and the attention refuses until the
    count is read."""
    import ctypes

    lib = _lib.load()
    n, m = ctypes.c_uint(), ctypes.c_uint()
    assert lib.ecco_device_timeouts(ctypes.byref(n)) == _lib.ECCO_OK
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(1, 1, 16, 64, dtype=torch.uint8, device=DEV)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((1, 1), 7.0, device=DEV)
    call = lambda: ecco.paged_attention(q, kp, kp, t, t, i32([[0]]), i32([1]), i32([0, 1]), 1.0, lse=lse)  # noqa: E731
    assert lib.ecco_selftest_paged_wait_timeout(None) == _lib.ECCO_OK
    torch.cuda.synchronize()
    with pytest.raises(ecco.EccoError) as e:
        call()
    assert e.value.code == _lib.ECCO_ERR_TIMEOUT
    torch.cuda.synchronize()
    assert lse.item() == 7.0  # nothing was enqueued
    assert lib.ecco_device_timeouts(ctypes.byref(m)) == _lib.ECCO_OK and m.value == n.value + 1
    call()
    assert lse.item() == 0.0  # one key of zeros


def test_pools_without_heads_are_refused():
    t = ecco.Tables(table_set("learned_kv"))
    kp = torch.zeros(4, 0, 16, 64, dtype=torch.uint8, device=DEV)
    tb, lens, cu = i32([[0, 1]]), i32([20]), i32([0, 5])
    with pytest.raises(ValueError):
        ecco.paged_attention(torch.zeros(5, 8, 128, dtype=torch.bfloat16, device=DEV), kp, kp, t, t, tb, lens, cu, 1.0)
    none = torch.zeros(5, 0, 128, dtype=torch.bfloat16, device=DEV)
    with pytest.raises((ValueError, ecco.EccoError)):
        ecco.paged_attention(none, kp, kp, t, t, tb, lens, cu, 1.0)
    with pytest.raises((ValueError, ecco.EccoError)):
        ecco.paged_append(none, none, kp, kp.clone(), t, t, tb, lens, cu)
    with pytest.raises((ValueError, ecco.EccoError)):
        ecco.compact_pages(kp, kp.clone(), tb, lens, torch.ones(1, 32, dtype=torch.bool, device=DEV), tb)
    with pytest.raises((ValueError, ecco.EccoError)):
        ecco.rope(none, ecco.rope_table(4, 128), i32([0] * 5))
