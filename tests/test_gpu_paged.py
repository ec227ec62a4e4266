"""Paged 8-bit cache on the GPU against the float64 oracle.

Tolerances.  A code comes from an f32 value x' of the exact x with |x' - x| <=
E: the rotation rounds three times and a sum of 128 products at most 129 times,
E = 132 * 2^-24 * sum |k_i P_ij| (values are not computed, E = 0).  Rounding to
e4m3 is monotone, so the code must lie between the roundings of x - E and x + E;
the page's scale likewise between those of amax - E and amax + E.

Attention: the stored numbers are exact, q~ is exact to f32, and the operands of
the products are sums of e4m3 parts with a remainder of at most 2^-4 each:
2^-24 (six parts, f32 outputs), 2^-16 for q~ and 2^-12 for p (bf16 outputs).
f32 outputs: 1e-5 per row (2-norm), as everywhere in this suite.  bf16 outputs
against the rounded oracle: p is off by at most 2^-12 of itself, which moves an
output by at most 2^-12 sum p|v| / l; for rows of independent values that is
below 2^-12 of a typical element and crosses a rounding border (2^-8 apart) for
1 in 16 elements at most, sqrt(1/16) * 2^-8 * 0.6 < 6e-4 in the 2-norm; the
suite's 2e-3 stands.  lse: off by at most the largest score error, 2^-16 (2^-23)
of sum |q~ k~| scale, plus the f32 of the result.
"""
import numpy as np
import pytest
import torch

import sparse_dimension_attention_b200 as aq
from oracle import aqua_oracle as O
from oracle import paged_oracle as PO
from aqua_testlib import calib_P, check_selection, rel_err_rows, tdev
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make_cache(B, Hkv, page, m, max_pages, seed=0, extra=3, guard=None):
    """A cache with shuffled pages for every table entry, filled with random codes (no NaN)."""
    g = torch.Generator().manual_seed(seed)
    n_pages = B * max_pages + extra
    alloc = guard or (lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda"))
    rnd = lambda *s: (torch.randint(0, 127, s, generator=g) + 128 * torch.randint(0, 2, s, generator=g)).to(torch.uint8)
    bufs = [alloc((n_pages, Hkv, m, page), torch.uint8), alloc((n_pages, Hkv, page, 128), torch.uint8),
            alloc((n_pages, Hkv), torch.float32), alloc((n_pages, Hkv), torch.float32),
            alloc((B, max_pages), torch.int32)]
    bufs[0].copy_(rnd(n_pages, Hkv, m, page))
    bufs[1].copy_(rnd(n_pages, Hkv, page, 128))
    for t in bufs[2:4]:
        t.copy_(2.0 ** torch.randint(-9, -4, (n_pages, Hkv), generator=g).float())
    bufs[4].copy_(torch.randperm(n_pages, generator=g)[:B * max_pages].view(B, max_pages).int())
    return aq.AquaPagedCache.from_buffers(*bufs)


def snap(cache):
    return {n: getattr(cache, n).cpu().numpy().copy() for n in ("k_pages", "v_pages", "k_scale", "v_scale",
                                                                  "block_table")}


def rope_of(kind, n_pos=4096):
    """(AquaRope or None, table or None, interleaved)"""
    if kind is None:
        return None, None, False
    rot, inter = kind
    r = aq.AquaRope.from_theta(n_pos, 10000.0, rot, inter)
    return r, r.cos_sin.cpu().numpy(), inter


def rows_of(rng, n, H, dtype, spread=1.0):
    x = rng.normal(size=(n, H, 128)) * np.exp(spread * rng.normal(size=(n, 1, 1)))
    return torch.from_numpy(x).to(DT[dtype]).double().numpy()


def check_append(cache, before, k, v, P32, start, cu, rope_np, inter, skip=()):
    """Every byte and scale of the cache after an append of k, v (float64 rows) against the oracle."""
    after = snap(cache)
    P = P32.astype(np.float64)
    B, m, page, H = cache.B, cache.d_store, cache.page_size, cache.Hkv
    table = before["block_table"]
    exp = {n: before[n].copy() for n in before}
    touched_k = np.zeros(before["k_pages"].shape, dtype=bool)
    touched_v = np.zeros(before["v_pages"].shape, dtype=bool)
    touched_s = np.zeros(before["k_scale"].shape, dtype=bool)
    for b in range(B):
        lo, hi = (b, b + 1) if cu is None else (cu[b], cu[b + 1])
        if b in skip or hi == lo:
            continue
        pos = np.arange(start[b], start[b] + hi - lo)
        kr = PO.rotate(k[lo:hi], pos, rope_np, inter)
        kt = np.einsum("nhi,hij->hnj", kr, P)[..., :m]
        err = 132 * 2.0 ** -24 * np.einsum("nhi,hij->hnj", np.abs(kr), np.abs(P))[..., :m]
        for p0 in range(int(pos[0]) // page, int(pos[-1]) // page + 1):
            idx = np.nonzero(pos // page == p0)[0]
            pid, fill = int(table[b, p0]), int(pos[idx[0]]) % page
            n = len(idx)
            for h in range(H):
                touched_s[pid, h] = True
                for name, x, e in (("k", kt[h, idx], err[h, idx]), ("v", v[lo:hi][idx, h], 0.0)):
                    s = float(after[name + "_scale"][pid, h])
                    old = float(before[name + "_scale"][pid, h])
                    low, high = PO.page_scale(PO.finite_max(np.abs(x) - e)), PO.page_scale(PO.finite_max(np.abs(x) + e))
                    if fill:
                        low, high = max(low, old), max(high, old)
                    assert low <= s <= high, (name, b, p0, h, low, s, high)
                    codes_b = before[name + "_pages"][pid, h]
                    codes_a = after[name + "_pages"][pid, h]
                    if name == "k":
                        codes_b, codes_a = codes_b.T, codes_a.T
                        touched_k[pid, h, :, :fill + n] = True
                    else:
                        touched_v[pid, h, :fill + n] = True
                    ob = PO.e4m3_decode(codes_b)
                    lo_v = PO.append_to_block(ob, old, fill, x - e, s)
                    hi_v = PO.append_to_block(ob, old, fill, x + e, s)
                    got = PO.e4m3_decode(codes_a)
                    ok = ((lo_v <= got) & (got <= hi_v)) | (np.isnan(got) & np.isnan(lo_v))
                    assert ok[:fill + n].all(), (name, b, p0, h, np.argwhere(~ok)[:4])
    # everything else is as it was
    for name, touched in (("k_pages", touched_k), ("v_pages", touched_v), ("k_scale", touched_s),
                          ("v_scale", touched_s)):
        np.testing.assert_array_equal(after[name][~touched], before[name][~touched], err_msg=name)
    np.testing.assert_array_equal(after["block_table"], table)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("B,Hkv,page,m,dtype,rope,start", [
    (1, 1, 16, 128, "f32", None, [0]),
    (1, 8, 64, 128, "bf16", (128, False), [1000]),
    (5, 2, 64, 96, "bf16", (128, True), [0, 1, 63, 64, 127]),
    (4, 3, 32, 100, "f32", (64, True), [31, 32, 33, 95]),
    (7, 2, 128, 1, "bf16", (2, False), [0, 5, 127, 128, 129, 255, 300]),
    (3, 16, 16, 48, "f32", (32, False), [15, 16, 40]),
    (40, 8, 16, 128, "bf16", (128, False), [(7 * i) % 45 for i in range(40)]),    # several blocks of sequences
])
def test_append_one_token_each(B, Hkv, page, m, dtype, rope, start):
    rng = np.random.default_rng(B * 100 + m)
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, max(start) // page + 2)
    r, rn, inter = rope_of(rope)
    k, v = rows_of(rng, B, Hkv, dtype), rows_of(rng, B, Hkv, dtype)
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k, DT[dtype]), tdev(v, DT[dtype]),
                         torch.tensor(start, dtype=torch.int32, device="cuda"), tdev(P32), rope=r)
    check_append(cache, before, k, v, P32, start, None, rn, inter)
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


@pytest.mark.parametrize("Hkv,page,m,dtype,rope,start,new", [
    (1, 16, 128, "bf16", (128, False), [0], [1]),
    (2, 16, 96, "bf16", (128, False), [0], [129]),
    (2, 64, 128, "f32", (64, True), [10, 0, 64], [54, 0, 65]),             # fills a page exactly, none, page start
    (4, 32, 100, "f32", (128, True), [31, 5, 0, 300], [1, 2, 33, 200]),
    (8, 128, 128, "bf16", (128, False), [1, 127, 128], [127, 130, 128]),
    (3, 128, 17, "bf16", None, [100], [500]),
    (1, 16, 128, "f32", (32, False), [3] * 300, [(i * 5) % 4 for i in range(300)]),   # more runs than a scan's pass
])
def test_append_runs(Hkv, page, m, dtype, rope, start, new):
    rng = np.random.default_rng(sum(new) + m)
    _, P32 = calib_P(Hkv)
    B, n = len(new), sum(new)
    cache = make_cache(B, Hkv, page, m, max(s + x for s, x in zip(start, new)) // page + 1, seed=1)
    r, rn, inter = rope_of(rope)
    k, v = rows_of(rng, n, Hkv, dtype), rows_of(rng, n, Hkv, dtype)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k, DT[dtype]), tdev(v, DT[dtype]),
                         torch.tensor(start, dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=torch.from_numpy(cu).cuda(), rope=r)
    check_append(cache, before, k, v, P32, start, cu, rn, inter)
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


@pytest.mark.parametrize("Hkv,page,m,dtype,rope,start,new", [
    (16, 16, 128, "bf16", (128, False), [3, 0, 127], [260, 100, 129]),      # 128-slot tiles of eight pages, ends inside
    (16, 16, 100, "f32", (128, True), [16, 5], [255, 250]),
    (16, 32, 33, "bf16", (36, False), [0, 31, 40], [300, 1, 180]),          # rotations that are no multiple of 16
    (8, 64, 96, "f32", (6, True), [60, 0], [500, 64]),
    (4, 128, 128, "bf16", None, [0, 130], [256, 400]),                      # whole pages only, then partial ones
    (2, 64, 128, "f32", (48, False), [0, 1, 0], [2000, 0, 63]),             # many tiles a block
    (150, 32, 16, "bf16", (32, True), [7], [90]),                           # more heads than SMs
])
def test_append_long_runs(Hkv, page, m, dtype, rope, start, new):
    """Runs that go to the tensor-core tiles."""
    test_append_runs(Hkv, page, m, dtype, rope, start, new)


def test_append_long_runs_of_many_sequences():
    """More sequences than one pass of the tile kernel's scan, runs of 0 to 60 tokens, rows of very different size,
    the page's scale growing where a run continues one."""
    rng = np.random.default_rng(30)
    Hkv, page, m, B = 16, 32, 20, 700
    _, P32 = calib_P(Hkv)
    start = [int(x) for x in rng.integers(0, 70, B)]
    new = [int(x) for x in rng.integers(0, 61, B)]
    cache = make_cache(B, Hkv, page, m, 5, seed=31)
    n = sum(new)
    k, v = rows_of(rng, n, Hkv, "bf16", 4.0), rows_of(rng, n, Hkv, "bf16", 4.0)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k, torch.bfloat16), tdev(v, torch.bfloat16),
                         torch.tensor(start, dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=torch.from_numpy(cu).cuda())
    check_append(cache, before, k, v, P32, start, cu, None, False)
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


def test_append_long_runs_bad_device_data():
    """Long runs with a page that does not exist, one that does not fit, one before the first slot: those tokens are
    skipped and reported, the others are right."""
    rng = np.random.default_rng(34)
    Hkv, page, m, new, start = 8, 64, 128, [200, 200, 200, 300], [0, 10, 100, -1]
    _, P32 = calib_P(Hkv)
    cache = make_cache(4, Hkv, page, m, 4, seed=35)
    cache.block_table[1, 1] = cache.n_pages
    n = sum(new)
    k, v = rows_of(rng, n, Hkv, "bf16"), rows_of(rng, n, Hkv, "bf16")
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k, torch.bfloat16), tdev(v, torch.bfloat16),
                         torch.tensor(start, dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=torch.from_numpy(cu).cuda())
    after = snap(cache)
    for p0 in (0, 2, 3):                     # the pages of sequence 1 that exist were written
        p = int(before["block_table"][1, p0])
        assert not np.array_equal(before["v_pages"][p], after["v_pages"][p])
        for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
            before[name][p] = after[name][p]
    check_append(cache, before, k, v, P32, start, cu, None, False, skip=(1, 2, 3))      # 2: 100 + 200 > 256
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG


def test_append_long_run_with_infinities():
    """Values: infinities saturate and NaN stays, the finite numbers set the scales.  A key row with an infinity
    spoils no other row."""
    Hkv, page, m, n = 8, 64, 128, 300
    rng = np.random.default_rng(32)
    _, P32 = calib_P(Hkv)
    cache = make_cache(1, Hkv, page, m, 5, seed=33)
    k, v = rows_of(rng, n, Hkv, "f32"), rows_of(rng, n, Hkv, "f32")
    v[10, 2, 5], v[10, 2, 6], v[200, 0, 127], k[100, 3, 7] = np.inf, -np.inf, np.nan, np.inf
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k), tdev(v), torch.zeros(1, dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    after = snap(cache)
    table = after["block_table"][0]
    vals = lambda name, t, h: PO.e4m3_decode(after[name + "_pages"][table[t // page], h][..., t % page] if name == "k"
                                             else after[name + "_pages"][table[t // page], h][t % page])
    for t in range(n):
        for h in range(Hkv):
            s = float(after["v_scale"][table[t // page], h])
            np.testing.assert_array_equal(vals("v", t, h), PO.e4m3_round(v[t, h] / s))
    for p0 in range(5):
        for h in range(Hkv):
            rows = slice(p0 * page, min(n, p0 * page + page))
            assert float(after["v_scale"][table[p0], h]) == PO.page_scale(PO.finite_max(v[rows, h]))
    kt = np.einsum("nhi,hij->nhj", np.where(np.isfinite(k), k, 0), P32.astype(np.float64))
    for t in (99, 101, 64, 127):
        s = float(after["k_scale"][table[t // page], 3])
        assert np.all(np.abs(vals("k", t, 3) * s - kt[t, 3]) <= np.maximum(2.0 ** -4 * np.abs(kt[t, 3]), 2.0 ** -10 * s) * 1.0001)


@pytest.mark.parametrize("runs", [False, True])
def test_append_growing_scale_recodes_the_page(runs):
    """Tokens that get larger and larger: the open page's scale grows each time and its codes follow."""
    rng = np.random.default_rng(3)
    Hkv, page, m = 2, 32, 80
    _, P32 = calib_P(Hkv)
    cache = make_cache(2, Hkv, page, m, 3)
    Pt = tdev(P32)
    at = [0, 7]
    for step, size in enumerate([1e-3, 1.0, 40.0, 40.0, 3e4]):
        n = [2, 3] if runs else [1, 1]
        k = torch.from_numpy(size * rng.normal(size=(sum(n), Hkv, 128))).bfloat16().double().numpy()
        v = torch.from_numpy(size * rng.normal(size=(sum(n), Hkv, 128))).bfloat16().double().numpy()
        cu = np.array([0, n[0], sum(n)], dtype=np.int32) if runs else None
        before = snap(cache)
        aq.aqua_paged_append(cache.desc, tdev(k, torch.bfloat16), tdev(v, torch.bfloat16),
                             torch.tensor(at, dtype=torch.int32, device="cuda"), Pt,
                             cu_new=torch.from_numpy(cu).cuda() if runs else None)
        check_append(cache, before, k, v, P32, at, cu, None, False)
        at = [a + x for a, x in zip(at, n)]


@pytest.mark.parametrize("runs", [False, True])
def test_append_special_values(runs):
    """Zeros, infinities, NaN, the largest and tiny numbers: the finite ones set the scale, inf saturates,
    NaN stays NaN.  P = 1, so a key row's entries stay apart."""
    Hkv, page = 1, 16
    P32 = np.eye(128, dtype=np.float32)[None]
    rows = np.zeros((4, 1, 128))
    rows[1, 0, :4] = [np.inf, -np.inf, 2.0, -3.0]
    rows[2, 0, :3] = [3e38, -1e-30, 1.0]
    rows[3, 0, :3] = [1e-25, -1e-26, 0.0]
    rows = rows.astype(np.float32).astype(np.float64)
    vrows = rows.copy()
    vrows[1, 0, 7] = np.nan
    cache = make_cache(4, Hkv, page, 128, 1)
    cu = torch.arange(5, dtype=torch.int32, device="cuda") if runs else None
    # k rows with inf times the zeros of P would be NaN: only v takes the special values whole
    krows = rows.copy()
    krows[1] = 0
    aq.aqua_paged_append(cache.desc, tdev(krows), tdev(vrows), torch.zeros(4, dtype=torch.int32, device="cuda"),
                         tdev(P32), cu_new=cu)
    a = snap(cache)
    for b in range(4):
        p = int(a["block_table"][b, 0])
        for name, x in (("k", krows[b, 0]), ("v", vrows[b, 0])):
            s = float(a[name + "_scale"][p, 0])
            assert s == PO.page_scale(PO.finite_max(x))
            blk = a[name + "_pages"][p, 0]
            got = PO.e4m3_decode(blk[:, 0] if name == "k" else blk[0])
            np.testing.assert_array_equal(got, PO.e4m3_round(x / s))
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


def test_append_strided_inputs():
    """Keys and values as slices of one fused projection, and head-major keys: same pages as dense copies."""
    Hkv, page, n = 4, 64, 150
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    qkv = torch.randn(n, 8 + 2 * Hkv, 128, device="cuda").bfloat16()
    k, v = qkv[:, 8:8 + Hkv], qkv[:, 8 + Hkv:]
    start = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 60, n], dtype=torch.int32, device="cuda")
    caches = [make_cache(2, Hkv, page, 128, 3) for _ in range(3)]
    aq.aqua_paged_append(caches[0].desc, k.contiguous(), v.contiguous(), start, Pt, cu_new=cu)
    aq.aqua_paged_append(caches[1].desc, k, v, start, Pt, cu_new=cu)
    aq.aqua_paged_append(caches[2].desc, k.transpose(0, 1).contiguous().transpose(0, 1), v, start, Pt, cu_new=cu)
    for c in caches[1:]:
        for name in ("k_pages", "v_pages", "k_scale", "v_scale"):
            assert torch.equal(getattr(c, name), getattr(caches[0], name)), name
    with pytest.raises(aq.AquaError):
        aq.aqua_paged_append(caches[0].desc, k[..., ::1].expand(n, Hkv, 128)[:, :, :64], v[:, :, :64], start, Pt, cu_new=cu)
    with pytest.raises(aq.AquaError):                                        # one row for every token: rows overlap
        aq.aqua_paged_append(caches[0].desc, k[:1].expand(n, Hkv, 128), v, start, Pt, cu_new=cu)


def test_append_bad_device_data_is_reported_and_skipped():
    """Starts, runs and page ids that only the device sees: those sequences are left alone, the rest is right."""
    rng = np.random.default_rng(5)
    Hkv, page, m, B = 2, 16, 64, 6
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    for runs in (False, True):
        cache = make_cache(B, Hkv, page, m, 3)
        cache.block_table[3, 1] = cache.n_pages                              # no such page
        cache.block_table[4, 0] = -1
        start = [-1, 48, 3, 20, 4, 30]                                       # 0: negative, 1: at the capacity
        n = [2] * B if runs else [1] * B
        cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32) if runs else None
        k, v = rows_of(rng, sum(n), Hkv, "bf16"), rows_of(rng, sum(n), Hkv, "bf16")
        before = snap(cache)
        aq.aqua_paged_append(cache.desc, tdev(k, torch.bfloat16), tdev(v, torch.bfloat16),
                             torch.tensor(start, dtype=torch.int32, device="cuda"), Pt,
                             cu_new=torch.from_numpy(cu).cuda() if runs else None)
        check_append(cache, before, k, v, P32, start, cu, None, False, skip=(0, 1, 3, 4))
        assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG
        assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK                # read and cleared
    # runs that overlap, go back or leave the rows
    cache = make_cache(3, Hkv, page, m, 3)
    before = snap(cache)
    k = rows_of(rng, 4, Hkv, "bf16")
    for bad in ([0, 5, 5, 5], [2, 1, 1, 1], [-1, -1, -1, -1]):
        aq.aqua_paged_append(cache.desc, tdev(k, torch.bfloat16), tdev(k, torch.bfloat16),
                             torch.zeros(3, dtype=torch.int32, device="cuda"), Pt,
                             cu_new=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG
    after = snap(cache)
    for name in before:
        np.testing.assert_array_equal(after[name], before[name])
    # positions past the rotation table
    rope, _, _ = rope_of((64, False), n_pos=10)
    aq.aqua_paged_append(cache.desc, tdev(k[:3], torch.bfloat16), tdev(k[:3], torch.bfloat16),
                         torch.tensor([10, 30, 47], dtype=torch.int32, device="cuda"), Pt, rope=rope)
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG
    after = snap(cache)
    for name in before:
        np.testing.assert_array_equal(after[name], before[name])


# ------------------------------------------------------------------ decode

def oracle_decode(state, lens, q, P32, k, rope_np, inter, out_dtype, scale=None):
    """aqua_oracle.decode over what the pages hold, the query rotated to position len - 1."""
    P = P32.astype(np.float64)
    B = len(lens)
    pos = [max(n - 1, 0) for n in lens]
    qr = PO.rotate(q, pos, rope_np, inter)
    H, m = state["k_pages"].shape[1], state["k_pages"].shape[2]
    T = max(1, max(lens))
    Kt, V = np.zeros((B, H, T, m)), np.zeros((B, H, T, 128))
    for b, n in enumerate(lens):
        kk, vv = PO.read_sequence(state["k_pages"], state["v_pages"], state["k_scale"], state["v_scale"],
                                  state["block_table"][b], n)
        Kt[b, :, :n], V[b, :, :n] = kk, vv
    ref = O.decode(qr, P, Kt, V, lens, k, scale=scale, m=m, out_dtype=out_dtype)
    ref["Kt"] = Kt
    return ref


def run_paged_decode(cache, q, lens, Pt, k, rope, out_dtype, io, ws=None, scale=0.0):
    B, Hq, _ = q.shape
    out = torch.full((B, Hq, 128), 7.0, dtype=out_dtype, device="cuda")
    sel = torch.full((B, Hq, k), -1, dtype=torch.int32, device="cuda")
    qp = torch.empty((B, Hq, 128), dtype=torch.float32, device="cuda")
    lse = torch.full((B, Hq), 7.0, dtype=torch.float32, device="cuda")
    if ws is None:
        ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    aq.aqua_paged_decode_attn(cache.desc, tdev(q, io), torch.tensor(lens, dtype=torch.int32, device="cuda"), Pt, Hq, k,
                              out, ws, rope=rope, scale=scale, sel_out=sel, qproj_out=qp, lse_out=lse)
    torch.cuda.synchronize()
    return {"out": out.double().cpu().numpy(), "sel": sel.cpu().numpy(), "qt": qp.cpu().numpy(),
            "lse": lse.cpu().numpy()}


def check_decode(got, ref, lens, k, m, bf16_out):
    check_selection(got["sel"], got["qt"], ref["sel"], ref["qt"], k, m)
    # q~ is the f64 one rounded to f32, which keeps the order: sets can differ only where the two magnitudes at
    # the cut round to one f32 number, a gap of at most 2^-23 of them (2^-22 with the f64 sums' own error)
    mag = -np.sort(-np.abs(ref["qt"][..., :m]), axis=-1)
    clear = np.ones(mag.shape[:2], dtype=bool) if k == m else mag[..., k - 1] - mag[..., k] > 2.0 ** -22 * mag[..., k - 1]
    np.testing.assert_array_equal(got["sel"][clear], ref["sel"][clear])
    np.testing.assert_allclose(got["qt"], ref["qt"], rtol=1e-6, atol=1e-6 * np.abs(ref["qt"]).max())
    tol = 2e-3 if bf16_out else 1e-5
    live = np.array(lens) > 0
    if live.any():
        assert np.max(rel_err_rows(got["out"][live], ref["out"][live])) <= tol
    assert np.all(got["out"][~live] == 0) and np.all(got["lse"][~live] == -np.inf)
    G = ref["qt"].shape[1] // ref["Kt"].shape[1]
    for b in np.nonzero(live)[0]:
        for h in range(ref["qt"].shape[1]):
            qs = np.zeros(128)
            qs[ref["sel"][b, h]] = np.abs(ref["qt"][b, h, ref["sel"][b, h]])
            mag = (np.abs(ref["Kt"][b, h // G, :lens[b]]) @ qs[:m]).max() / np.sqrt(128)
            bound = (2.0 ** -16 if bf16_out else 2.0 ** -23) * mag + 4e-7 * (abs(ref["lse"][b, h]) + mag + 10)
            assert abs(got["lse"][b, h] - ref["lse"][b, h]) <= bound, (b, h)


CASES = [
    # B, Hq, Hkv, page, m, k, lens, rope, io, out
    (1, 4, 1, 64, 128, 96, [255], (128, False), "bf16", "bf16"),
    (1, 1, 1, 16, 128, 128, [1], None, "f32", "f32"),
    (2, 8, 8, 128, 128, 32, [130, 128], (64, True), "bf16", "f32"),
    (3, 4, 2, 32, 96, 64, [0, 33, 500], (128, False), "bf16", "bf16"),
    (4, 12, 4, 16, 100, 1, [15, 16, 17, 129], (128, True), "f32", "f32"),
    (2, 14, 2, 64, 48, 48, [127, 257], (32, False), "f32", "bf16"),
    (2, 16, 2, 128, 128, 64, [1000, 3], (128, False), "bf16", "bf16"),
    (2, 16, 2, 64, 128, 17, [300, 513], (128, False), "f32", "f32"),
    (1, 10, 2, 32, 16, 16, [700], (2, False), "bf16", "f32"),
    (3, 6, 1, 16, 1, 1, [40, 0, 1], None, "bf16", "bf16"),
    (2, 4, 1, 16, 128, 96, [5000, 2049], (128, False), "bf16", "f32"),        # a unit over many blocks
]


@pytest.mark.parametrize("B,Hq,Hkv,page,m,k,lens,rope,io,od", CASES)
def test_decode_matches_the_oracle(B, Hq, Hkv, page, m, k, lens, rope, io, od):
    rng = np.random.default_rng(B * 1000 + Hq * 10 + k)
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, max(lens) // page + 1, seed=2)
    r, rn, inter = rope_of(rope, 8192)
    q = rows_of(rng, B, Hq, io, spread=0.3)
    got = run_paged_decode(cache, q, lens, tdev(P32), k, r, DT[od], DT[io])
    ref = oracle_decode(snap(cache), lens, q, P32, k, rn, inter, od)
    check_decode(got, ref, lens, k, m, od == "bf16")
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


def test_decode_many_sequences():
    """More sequences than a scan's pass and more units than blocks, most of them shorter than a tile."""
    B, Hq, Hkv, page, m, k = 331, 4, 2, 16, 32, 20
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 40, B)]
    lens[17] = 300
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, 19, seed=3)
    q = rows_of(rng, B, Hq, "bf16", spread=0.3)
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, torch.float32, torch.bfloat16)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, "f32")
    check_decode(got, ref, lens, k, m, False)


def torch_decode(cache, q, lens, P, k):
    """The step in f64 on the device, for lengths the loops of the oracle are too slow for (no rotation)."""
    B, Hq, _ = q.shape
    H, m, G = cache.Hkv, cache.d_store, Hq // cache.Hkv
    out = torch.zeros(B, Hq, 128, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        t = cache.block_table[b, :-(-n // cache.page_size)].long()
        kk = cache.k_pages[t].view(torch.float8_e4m3fn).double() * cache.k_scale[t].double()[:, :, None, None]
        vv = cache.v_pages[t].view(torch.float8_e4m3fn).double() * cache.v_scale[t].double()[:, :, None, None]
        kk, vv = kk.permute(1, 2, 0, 3).reshape(H, m, -1)[..., :n], vv.permute(1, 0, 2, 3).reshape(H, -1, 128)[:, :n]
        for h in range(H):
            qt = q[b, h * G:(h + 1) * G].double() @ P[h].double()
            keep = qt[:, :m].abs().topk(k, dim=1).indices
            qm = torch.zeros(G, m, dtype=torch.float64, device="cuda").scatter_(1, keep, qt.gather(1, keep))
            out[b, h * G:(h + 1) * G] = torch.softmax(qm @ kk[h] / 128 ** 0.5, -1) @ vv[h]
    return out


@pytest.mark.parametrize("tiles", [7.99, 8, 8.01, 16, 37.3, 5, 4.99])
def test_decode_long_sequence_in_many_pieces(tiles):
    """One sequence split over all blocks: equal shares, the most later pieces there can be, fewer of them."""
    blocks = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    n = int(blocks * tiles) * 128 - 5
    rng = np.random.default_rng(40)
    _, P32 = calib_P(1)
    cache = make_cache(1, 1, 128, 32, -(-n // 128), seed=41)
    q = tdev(rows_of(rng, 1, 4, "f32", 0.3))
    for od, tol in ((torch.float32, 1e-5), (torch.bfloat16, 4e-3)):         # bf16: against the unrounded result
        out = torch.empty(1, 4, 128, dtype=od, device="cuda")
        ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, 4),), 0xFF, dtype=torch.uint8, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, q, torch.tensor([n], dtype=torch.int32, device="cuda"), tdev(P32), 4, 20, out, ws)
        ref = torch_decode(cache, q, [n], tdev(P32), 20)
        assert float(((out.double() - ref).norm(dim=-1) / ref.norm(dim=-1)).max()) <= tol


def test_decode_ragged_long_batch():
    """Units that end inside pieces of every kind, the same bits on every run."""
    rng = np.random.default_rng(42)
    B, Hq, Hkv, m, k = 24, 16, 8, 96, 64
    lens = [int(x) for x in np.exp(rng.uniform(0, np.log(12000), B))]
    lens[3], lens[11] = 0, 12000
    _, P32 = calib_P(Hkv)
    P = tdev(P32)
    cache = make_cache(B, Hkv, 64, m, 12000 // 64 + 1, seed=43)
    q = tdev(rows_of(rng, B, Hq, "f32", 0.3))
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(6):
        out = torch.empty(B, Hq, 128, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, q, lt, P, Hq, k, out, ws)
        outs.append(out)
    ref = torch_decode(cache, q, lens, P, k)
    live = lt > 0
    assert float(((outs[0].double() - ref).norm(dim=-1)[live] / ref.norm(dim=-1)[live]).max()) <= 1e-5
    assert bool((outs[0][3] == 0).all())
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_decode_ties_and_zero_queries():
    """Equal magnitudes go to the lower dimension; a zero query keeps the first k and attends evenly."""
    B, Hq, Hkv, page, m, k, lens = 2, 4, 1, 16, 90, 33, [70, 20]
    P32 = np.eye(128, dtype=np.float32)[None]
    q = np.ones((B, Hq, 128))
    q[0, 1, ::2] = -1.0
    q[0, 2] = 0.0
    q[0, 3, 40:] = 2.0
    q[1, 0, :] = np.arange(128) % 3
    cache = make_cache(B, Hkv, page, m, 5, seed=4)
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, torch.float32, torch.float32)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, "f32")
    np.testing.assert_array_equal(got["sel"], ref["sel"])
    assert np.max(rel_err_rows(got["out"], ref["out"])) <= 1e-5
    np.testing.assert_array_equal(got["sel"][0, 2], np.arange(k))


def test_decode_ignores_what_lies_behind_a_sequence():
    """NaN codes and NaN or infinite scales behind the length, unset and impossible table entries past it."""
    B, Hq, Hkv, page, m, k, lens = 3, 4, 2, 32, 128, 70, [50, 1, 128]
    rng = np.random.default_rng(11)
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, 8, seed=5)
    q = rows_of(rng, B, Hq, "bf16", spread=0.3)
    clean = run_paged_decode(cache, q, lens, tdev(P32), k, None, torch.float32, torch.bfloat16)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, "f32")
    check_decode(clean, ref, lens, k, m, False)
    for b, n in enumerate(lens):
        full, rest = n // page, n % page
        if rest:
            p = int(cache.block_table[b, full])
            cache.k_pages[p, :, :, rest:] = 0x7F
            cache.v_pages[p, :, rest:] = 0xFF
        first_free = full + (1 if rest else 0)
        if first_free < 8:
            p = int(cache.block_table[b, first_free])
            cache.k_scale[p] = float("nan")
            cache.v_scale[p] = float("inf")
        cache.block_table[b, first_free:] = torch.tensor([-1, 1 << 30, -(1 << 31)] * 3, dtype=torch.int32)[:8 - first_free]
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, torch.float32, torch.bfloat16)
    for name in ("out", "lse", "sel"):
        np.testing.assert_array_equal(got[name], clean[name])
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


def test_decode_nan_stays_where_it_belongs():
    """A NaN value makes its dimension NaN for its KV head; a NaN key in a kept dimension makes the head NaN."""
    B, Hq, Hkv, page, m, lens = 2, 4, 2, 16, 128, [40, 40]
    rng = np.random.default_rng(12)
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, 3, seed=6)
    cache.v_pages[int(cache.block_table[0, 1]), 0, 3, 77] = 0x7F             # sequence 0, KV head 0
    cache.k_pages[int(cache.block_table[1, 2]), 1, 5, 2] = 0xFF              # sequence 1, KV head 1
    q = rows_of(rng, B, Hq, "bf16", spread=0.3)
    got = run_paged_decode(cache, q, lens, tdev(P32), 128, None, torch.float32, torch.bfloat16)
    bad = np.isnan(got["out"])
    want = np.zeros_like(bad)
    want[0, :2, 77] = True
    want[1, 2:] = True
    np.testing.assert_array_equal(bad, want)
    np.testing.assert_array_equal(np.isnan(got["lse"]), np.array([[False] * 4, [False, False, True, True]]))


@pytest.mark.parametrize("od", ["bf16", "f32"])
def test_decode_page_scales_far_apart(od):
    """Pages whose key and value scales differ by up to 2^40, large scores among them."""
    B, Hq, Hkv, page, m, k, lens = 1, 4, 1, 16, 128, 128, [16 * 40]
    rng = np.random.default_rng(13)
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, 40, seed=7)
    n = cache.n_pages
    cache.v_scale.copy_(torch.from_numpy(2.0 ** rng.integers(-30, 11, (n, 1))).float())
    cache.k_scale.copy_(torch.from_numpy(2.0 ** rng.integers(-30, -4, (n, 1))).float())
    q = rows_of(rng, B, Hq, "f32", spread=0.3)
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, DT[od], torch.float32)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, od)
    check_decode(got, ref, lens, k, m, od == "bf16")


def test_decode_bad_device_data_is_reported():
    """Lengths beyond the table or the rotation count as empty; tokens on impossible pages are left out."""
    B, Hq, Hkv, page, m, k = 5, 2, 1, 16, 64, 30
    rng = np.random.default_rng(14)
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, 4, seed=8)
    rope, rn, inter = rope_of((64, False), n_pos=60)
    q = rows_of(rng, B, Hq, "bf16", spread=0.3)
    got = run_paged_decode(cache, q, [65, -3, 61, 60, 20], tdev(P32), k, rope, torch.float32, torch.bfloat16)
    ref = oracle_decode(snap(cache), [0, 0, 0, 60, 20], q, P32, k, rn, inter, "f32")
    assert np.max(rel_err_rows(got["out"][3:], ref["out"][3:])) <= 1e-5
    assert np.all(got["out"][:3] == 0) and np.all(np.isneginf(got["lse"][:3]))
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG
    # a page that does not exist: its 16 tokens drop out
    lens = [64] * B
    state = snap(cache)
    cache.block_table[2, 1] = cache.n_pages + 5
    cache.block_table[4, :] = -7
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, torch.float32, torch.bfloat16)
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG
    ref = oracle_decode(state, lens, q, P32, k, None, False, "f32")
    assert np.max(rel_err_rows(got["out"][[0, 1, 3]], ref["out"][[0, 1, 3]])) <= 1e-5
    for h in range(Hq):
        kk, vv = PO.read_sequence(state["k_pages"], state["v_pages"], state["k_scale"], state["v_scale"],
                                  state["block_table"][2], 64)
        keep = np.r_[0:16, 32:64]
        o, _, _, _ = O.attend_one(O.project(q[2, h], P32[0]), k, kk[0, keep], vv[0, keep], 1 / np.sqrt(128), m)
        assert np.linalg.norm(got["out"][2, h] - o) <= 1e-5 * np.linalg.norm(o)
    assert np.all(got["out"][4] == 0) and np.all(np.isneginf(got["lse"][4]))


def test_decode_scale_argument_and_strided_queries():
    B, Hq, Hkv, page, m, k, lens = 3, 4, 2, 64, 128, 50, [90, 10, 64]
    rng = np.random.default_rng(15)
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    cache = make_cache(B, Hkv, page, m, 2, seed=9)
    q = rows_of(rng, B, Hq, "bf16", spread=0.3)
    got = run_paged_decode(cache, q, lens, Pt, k, None, torch.float32, torch.bfloat16, scale=0.3)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, "f32", scale=0.3)
    assert np.max(rel_err_rows(got["out"], ref["out"])) <= 1e-5
    wide = torch.zeros(B, Hq + 5, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:2 + Hq] = tdev(q, torch.bfloat16)
    outs = []
    for t in (wide[:, 2:2 + Hq], wide[:, 2:2 + Hq].transpose(0, 1).contiguous().transpose(0, 1)):
        out = torch.empty(B, Hq, 128, device="cuda")
        ws = torch.empty(aq.aqua_paged_decode_workspace_size(cache.desc, Hq), dtype=torch.uint8, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, t, torch.tensor(lens, dtype=torch.int32, device="cuda"), Pt, Hq, k, out,
                                  ws, scale=0.3)
        outs.append(out.double().cpu().numpy())
    for o in outs:
        np.testing.assert_array_equal(o, got["out"])


def test_workspace_reuse_graphs_and_streams():
    """One workspace for calls of different shapes in a row; a captured step replayed with new lengths and
    queries; two streams with a workspace each.  Every result bit-identical to a call of its own."""
    rng = np.random.default_rng(16)
    Hkv, page, m = 2, 32, 128
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    big, small = make_cache(40, Hkv, page, m, 20, seed=10), make_cache(2, Hkv, page, m, 4, seed=11)
    ws = torch.zeros(aq.aqua_paged_decode_workspace_size(big.desc, 16), dtype=torch.uint8, device="cuda")
    jobs = [(big, 16, 70, [int(x) for x in rng.integers(0, 600, 40)], torch.bfloat16),
            (small, 2, 128, [100, 3], torch.float32), (big, 8, 20, [600] * 40, torch.float32),
            (small, 16, 1, [0, 128], torch.bfloat16)]
    for cache, Hq, k, lens, od in jobs:
        q = rows_of(rng, cache.B, Hq, "bf16", spread=0.3)
        one = run_paged_decode(cache, q, lens, Pt, k, None, od, torch.bfloat16)
        two = run_paged_decode(cache, q, lens, Pt, k, None, od, torch.bfloat16, ws=ws)
        for n in one:
            np.testing.assert_array_equal(one[n], two[n], err_msg=n)
    # graph
    cache, Hq, k = small, 8, 64
    q = torch.zeros(2, Hq, 128, dtype=torch.bfloat16, device="cuda")
    ln = torch.zeros(2, dtype=torch.int32, device="cuda")
    out = torch.empty(2, Hq, 128, device="cuda")
    kv = torch.zeros(2, Hkv, 128, dtype=torch.bfloat16, device="cuda")
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    wsg = torch.empty(aq.aqua_paged_decode_workspace_size(cache.desc, Hq), dtype=torch.uint8, device="cuda")
    def step():
        aq.aqua_paged_append(cache.desc, kv, kv, start, Pt)
        aq.aqua_paged_decode_attn(cache.desc, q, ln, Pt, Hq, k, out, wsg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for lens in ([5, 77], [128, 1], [64, 64]):
        q.copy_(torch.randn(2, Hq, 128))
        kv.copy_(torch.randn(2, Hkv, 128))
        ln.copy_(torch.tensor(lens, dtype=torch.int32))
        start.copy_(ln - 1)
        g.replay()
        torch.cuda.synchronize()
        ref = run_paged_decode(cache, q.double().cpu().numpy(), lens, Pt, k, None, torch.float32, torch.bfloat16)
        np.testing.assert_array_equal(out.double().cpu().numpy(), ref["out"])
    # two streams, a workspace each
    q2 = rows_of(rng, 40, 8, "bf16", spread=0.3)
    lens2 = [int(x) for x in rng.integers(1, 600, 40)]
    ref = run_paged_decode(big, q2, lens2, Pt, 50, None, torch.float32, torch.bfloat16)
    qt, lt = tdev(q2, torch.bfloat16), torch.tensor(lens2, dtype=torch.int32, device="cuda")
    outs, wss = [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        outs.append(torch.empty(40, 8, 128, device="cuda"))
        wss.append(torch.empty(aq.aqua_paged_decode_workspace_size(big.desc, 8), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(streams, outs, wss):
            aq.aqua_paged_decode_attn(big.desc, qt, lt, Pt, 8, 50, o, w, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        np.testing.assert_array_equal(o.double().cpu().numpy(), ref["out"])


def test_offsets_past_32_bits():
    """A pool of over 4 GB of keys whose used pages lie at its end."""
    Hkv, page, m, n_pages, lens = 8, 128, 128, 33000, [200, 129]
    rng = np.random.default_rng(17)
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    table = torch.tensor([[n_pages - 1, n_pages - 3], [n_pages - 2, 5]], dtype=torch.int32, device="cuda")
    cache = aq.AquaPagedCache.from_buffers(
        torch.empty((n_pages, Hkv, m, page), dtype=torch.uint8, device="cuda"),
        torch.empty((n_pages, Hkv, page, 128), dtype=torch.uint8, device="cuda"),
        torch.ones((n_pages, Hkv), device="cuda"), torch.ones((n_pages, Hkv), device="cuda"), table)
    assert cache.k_pages.numel() > 1 << 32
    k, v = rows_of(rng, sum(lens), Hkv, "bf16"), rows_of(rng, sum(lens), Hkv, "bf16")
    aq.aqua_paged_append(cache.desc, tdev(k, torch.bfloat16), tdev(v, torch.bfloat16),
                         torch.zeros(2, dtype=torch.int32, device="cuda"), Pt,
                         cu_new=torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda"))
    q = rows_of(rng, 2, 16, "bf16", spread=0.3)
    got = run_paged_decode(cache, q, lens, Pt, 100, None, torch.float32, torch.bfloat16)
    ids = table.cpu().numpy().reshape(-1)
    state = {n: getattr(cache, n)[torch.from_numpy(ids).long().cuda()].cpu().numpy()
             for n in ("k_pages", "v_pages", "k_scale", "v_scale")}
    state["block_table"] = np.arange(4).reshape(2, 2)
    ref = oracle_decode(state, lens, q, P32, 100, None, False, "f32")
    check_decode(got, ref, lens, 100, m, False)
    # what was appended is what was given, to half a step of e4m3 (the smaller values: of the subnormals)
    kt = np.einsum("nhi,hij->nhj", k, P32.astype(np.float64))
    for b, (lo, n) in enumerate(((0, lens[0]), (lens[0], lens[1]))):
        kk = ref["Kt"][b, :, :n].transpose(1, 0, 2)
        s = np.repeat(state["k_scale"].reshape(2, 2, Hkv)[b], page, 0)[:n, :, None]
        assert np.all(np.abs(kk - kt[lo:lo + n]) <= np.maximum(2.0 ** -4 * np.abs(kt[lo:lo + n]), 2.0 ** -10 * s) * 1.0001)


def test_guard_words_intact():
    """Canaries around every buffer that the paged calls write or read."""
    B, Hq, Hkv, page, m, k, lens = 3, 14, 2, 16, 100, 60, [33, 0, 129]
    gb = Guarded()
    cache = make_cache(B, Hkv, page, m, 9, seed=12, guard=gb)
    rng = np.random.default_rng(18)
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    rope = aq.AquaRope.from_theta(200, rot_dim=128)
    n = [32, 1, 127]
    cu = torch.tensor([0, 32, 33, 160], dtype=torch.int32, device="cuda")
    x = gb((160, Hkv, 128), torch.float32)
    x.copy_(torch.randn(160, Hkv, 128))
    aq.aqua_paged_append(cache.desc, x, x, torch.tensor([0, 0, 0], dtype=torch.int32, device="cuda"), Pt, cu_new=cu, rope=rope)
    aq.aqua_paged_append(cache.desc, x[:3], x[:3], torch.tensor(n, dtype=torch.int32, device="cuda"), Pt, rope=rope)
    for od in (torch.bfloat16, torch.float32):
        out, sel = gb((B, Hq, 128), od), gb((B, Hq, k), torch.int32)
        qp, lse = gb((B, Hq, 128), torch.float32), gb((B, Hq), torch.float32)
        ws = gb((aq.aqua_paged_decode_workspace_size(cache.desc, Hq),), torch.uint8)
        q = gb((B, Hq, 128), torch.float32)
        q.copy_(torch.randn(B, Hq, 128))
        aq.aqua_paged_decode_attn(cache.desc, q, torch.tensor(lens, dtype=torch.int32, device="cuda"), Pt, Hq, k, out, ws,
                                  rope=rope, sel_out=sel, qproj_out=qp, lse_out=lse)
    kp, vv, ln = gb((B, Hkv, m, 144), torch.bfloat16), gb((B, Hkv, 144, 128), torch.bfloat16), gb((B,), torch.int32)
    dst = aq.aqua_cache(kp.data_ptr(), vv.data_ptr(), ln.data_ptr(), None, None, None, cache.ctrl.data_ptr(), B, Hkv, 128,
                        m, 144, 0, aq.AQUA_BF16, 0)
    aq.aqua_paged_gather(cache.desc, torch.tensor(lens, dtype=torch.int32, device="cuda"), dst, 129)
    gb.check()
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK
    assert bool(torch.isfinite(out).all()) and ln.tolist() == lens


# ------------------------------------------------------------------ gather, and a whole run

@pytest.mark.parametrize("page,m,dtype", [(16, 128, "bf16"), (32, 96, "f32"), (64, 1, "bf16"), (128, 100, "f32")])
def test_gather_is_exact(page, m, dtype):
    B, Hkv, lens = 5, 3, [0, 1, 17, 128, 300]
    cache = make_cache(B, Hkv, page, m, 300 // page + 1, seed=13)
    cache.k_pages[int(cache.block_table[2, 0]), 1, 0, 5] = 0x7F               # a NaN code stays NaN
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    state = snap(cache)
    for idx in (None, [4, 2, 2]):
        n = B if idx is None else len(idx)
        dst = aq.AquaCache(n, Hkv, 304, d_store=m, dtype=DT[dtype])
        dst.k_proj.fill_(5.0)
        dst.v.fill_(5.0)
        aq.aqua_paged_gather(cache.desc, ln, dst.desc, 304,
                             seq_idx=None if idx is None else torch.tensor(idx, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert dst.max_len == 304
        for i in range(n):
            s = i if idx is None else idx[i]
            kk, vv = PO.read_sequence(state["k_pages"], state["v_pages"], state["k_scale"], state["v_scale"],
                                      state["block_table"][s], lens[s])
            np.testing.assert_array_equal(dst.k_proj[i, :, :, :lens[s]].double().cpu().numpy(), kk.transpose(0, 2, 1))
            np.testing.assert_array_equal(dst.v[i, :, :lens[s]].double().cpu().numpy(), vv)
            assert bool((dst.k_proj[i, :, :, lens[s]:] == 5).all()) and bool((dst.v[i, :, lens[s]:] == 5).all())
            assert int(dst.len[i]) == lens[s] == int(dst.n_abs[i])
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


def test_gather_bad_device_data_is_reported():
    B, Hkv, page = 4, 2, 16
    cache = make_cache(B, Hkv, page, 128, 4, seed=14)
    cache.block_table[3, 1] = 10 ** 6
    dst = aq.AquaCache(4, Hkv, 64)
    ln = torch.tensor([40, 65, -1, 33], dtype=torch.int32, device="cuda")
    aq.aqua_paged_gather(cache.desc, ln, dst.desc, 48, seq_idx=torch.tensor([0, 9, -2, 3], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert dst.len.tolist() == [40, 0, 0, 33]
    assert bool((dst.k_proj[3, :, :, 16:32] == 0).all()) and bool((dst.v[3, :, 16:32] == 0).all())
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG
    aq.aqua_paged_gather(cache.desc, ln, dst.desc, 32)                        # 40 and 33 are over the bound, 65 too long
    assert dst.len.tolist() == [0, 0, 0, 0]
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG


def test_prompt_then_decode_steps():
    """As a server runs it: two prompts appended in one call, their pages gathered for the prompt's attention,
    then decode steps of append and attention; each against the oracle over what the pages hold."""
    B, Hq, Hkv, page, m, k = 2, 8, 2, 64, 96, 64
    n = [150, 70]
    rng = np.random.default_rng(20)
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    cache = aq.AquaPagedCache(B, Hkv, 12, 4, page_size=page, d_store=m)
    cache.block_table.copy_(torch.tensor([[7, 2, 9, 1], [0, 11, 4, 3]], dtype=torch.int32))
    rope, rn, inter = rope_of((128, False), 256)
    kp, vp = rows_of(rng, sum(n), Hkv, "bf16", 0.3), rows_of(rng, sum(n), Hkv, "bf16", 0.3)
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    aq.aqua_paged_append(cache.desc, tdev(kp, torch.bfloat16), tdev(vp, torch.bfloat16), zero, Pt,
                         cu_new=torch.tensor([0, n[0], sum(n)], dtype=torch.int32, device="cuda"), rope=rope)
    # the last 40 tokens of the first prompt as a chunk over its gathered history
    dst = aq.AquaCache(1, Hkv, 160, d_store=m)
    ln = torch.tensor(n, dtype=torch.int32, device="cuda")
    aq.aqua_paged_gather(cache.desc, ln, dst.desc, 150, seq_idx=zero[:1])
    L, pos0 = 40, 110
    q = torch.from_numpy(PO.rotate(rows_of(rng, L, Hq, "bf16", 0.3), np.arange(pos0, pos0 + L), rn, inter)).bfloat16()
    out = torch.empty(1, L, Hq, 128, device="cuda")
    ws = torch.empty(aq.aqua_prefill_workspace_size(dst.desc, Hq, L), dtype=torch.uint8, device="cuda")
    aq.aqua_prefill_attn(dst.desc, q[None].cuda(), pos0, L, Pt, Hq, k, out, ws)
    torch.cuda.synchronize()
    st = snap(cache)
    kk, vv = PO.read_sequence(st["k_pages"], st["v_pages"], st["k_scale"], st["v_scale"], st["block_table"][0], 150)
    ref, _ = O.prefill(q.double().numpy(), pos0, P32.astype(np.float64), kk, vv, k, m=m)
    assert np.max(rel_err_rows(out[0].double().cpu().numpy(), ref)) <= 2e-3
    # decode
    lens = list(n)
    for step in range(3):
        kn, vn, qn = (rows_of(rng, B, h, "bf16", 0.3) for h in (Hkv, Hkv, Hq))
        start = torch.tensor(lens, dtype=torch.int32, device="cuda")
        aq.aqua_paged_append(cache.desc, tdev(kn, torch.bfloat16), tdev(vn, torch.bfloat16), start, Pt, rope=rope)
        lens = [x + 1 for x in lens]
        got = run_paged_decode(cache, qn, lens, Pt, k, rope, torch.bfloat16, torch.bfloat16)
        check_decode(got, oracle_decode(snap(cache), lens, qn, P32, k, rn, inter, "bf16"), lens, k, m, True)
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


@pytest.mark.parametrize("B,Hq,Hkv,m,k,longest", [(1100, 4, 1, 32, 20, 400), (90, 64, 8, 128, 70, 1500)])
def test_decode_large_batches_with_shared_prefixes(B, Hq, Hkv, m, k, longest):
    """Several sequences a selection block, a search for a piece's sequence of several rounds, later pieces; the
    first pages of half of the sequences are the same ones, some sequences are empty."""
    rng = np.random.default_rng(50)
    page = 16
    lens = [int(x) for x in rng.integers(0, longest, B)]
    lens[7], lens[B - 1] = 0, 0
    _, P32 = calib_P(Hkv)
    cache = make_cache(B, Hkv, page, m, longest // page + 1, seed=51)
    cache.block_table[::2, :3] = cache.block_table[0, :3].clone()
    q = tdev(rows_of(rng, B, Hq, "f32", 0.3))
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):
        out = torch.empty(B, Hq, 128, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, q, lt, tdev(P32), Hq, k, out, ws)
        outs.append(out)
    ref = torch_decode(cache, q, lens, tdev(P32), k)
    live = lt > 0
    assert float(((outs[0].double() - ref).norm(dim=-1)[live] / ref.norm(dim=-1)[live]).max()) <= 1e-5
    assert bool((outs[0][~live] == 0).all()) and torch.equal(outs[0], outs[1])
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


def test_captured_appends_and_gathers_on_other_streams():
    """Runs long enough for the tensor cores, captured on a stream of their own with the gather after them and
    replayed with other lengths; then appends to two caches at once on two streams.  The same bytes as calls of
    their own."""
    rng = np.random.default_rng(60)
    Hkv, page, m, B, cap = 8, 64, 96, 3, 1024
    _, P32 = calib_P(Hkv)
    Pt = tdev(P32)
    rope, _, _ = rope_of((128, False), cap)
    N = 1500
    k = tdev(rows_of(rng, N, Hkv, "bf16"), torch.bfloat16)
    v = tdev(rows_of(rng, N, Hkv, "bf16"), torch.bfloat16)
    one, two = make_cache(B, Hkv, page, m, cap // page, seed=61), make_cache(B, Hkv, page, m, cap // page, seed=61)
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    ln = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 0, 0, N], dtype=torch.int32, device="cuda")
    dst, ref_dst = aq.AquaCache(2, Hkv, cap, d_store=m), aq.AquaCache(2, Hkv, cap, d_store=m)
    idx = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    def step(cache, d, stream=None):
        aq.aqua_paged_append(cache.desc, k, v, start, Pt, cu_new=cu, rope=rope, stream=stream)
        aq.aqua_paged_gather(cache.desc, ln, d.desc, cap, seq_idx=idx, stream=stream)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step(one, dst)
    for starts, cuts in (([5, 300, 0], [0, 600, 700, 1500]), ([605, 400, 0], [0, 0, 601, 1500]), ([0, 0, 100], [0, 500, 700, 1500])):
        start.copy_(torch.tensor(starts, dtype=torch.int32))
        cu.copy_(torch.tensor(cuts, dtype=torch.int32))
        ln.copy_(start + cu[1:] - cu[:-1])
        g.replay()
        step(two, ref_dst)
        torch.cuda.synchronize()
        a, b = snap(one), snap(two)
        for n in a:
            np.testing.assert_array_equal(a[n], b[n], err_msg=n)
        n = int(ln[2])
        for x, y in ((dst.k_proj[..., :n], ref_dst.k_proj[..., :n]), (dst.v[:, :, :n], ref_dst.v[:, :, :n])):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(dst.v[0, :, :n].view(torch.int16), dst.v[1, :, :n].view(torch.int16))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, c in zip(streams, (one, two)):
        aq.aqua_paged_append(c.desc, k, v, start, Pt, cu_new=cu, rope=rope, stream=s)
        aq.aqua_paged_append(c.desc, k[:B], v[:B], ln, Pt, rope=rope, stream=s)
    torch.cuda.synchronize()
    a, b = snap(one), snap(two)
    for n in a:
        np.testing.assert_array_equal(a[n], b[n], err_msg=n)
    assert aq.aqua_paged_status(one.desc) == aq.AQUA_OK and aq.aqua_paged_status(two.desc) == aq.AQUA_OK


def test_append_short_runs_of_many_sequences():
    """More page segments than blocks: a block takes several, one of them on a page that does not exist."""
    rng = np.random.default_rng(70)
    B, Hkv, page, m = 350, 2, 16, 48
    n = [int(x) for x in rng.integers(0, 5, B)]
    start = [int(x) for x in rng.integers(0, 40, B)]
    n[9], start[9], n[B - 1], start[B - 1] = 4, 14, 3, 30
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    _, P32 = calib_P(Hkv)
    rope, rn, inter = rope_of((128, False))
    for bad in (False, True):
        cache = make_cache(B, Hkv, page, m, 3, seed=71)
        if bad:
            n200 = 200 + next(i for i in range(100) if n[200 + i] > 0 and start[200 + i] // page == (start[200 + i] + n[200 + i] - 1) // page)
            cache.block_table[n200, start[n200] // page] = -1
        k, v = rows_of(rng, sum(n), Hkv, "f32"), rows_of(rng, sum(n), Hkv, "f32")
        before = snap(cache)
        aq.aqua_paged_append(cache.desc, tdev(k), tdev(v), torch.tensor(start, dtype=torch.int32, device="cuda"),
                             tdev(P32), cu_new=torch.from_numpy(cu).cuda(), rope=rope)
        torch.cuda.synchronize()
        check_append(cache, before, k, v, P32, start, cu, rn, inter, skip=(n200,) if bad else ())
        assert aq.aqua_paged_status(cache.desc) == (aq.abi.AQUA_ERR_ARG if bad else aq.AQUA_OK)
