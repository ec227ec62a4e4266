"""Paged 8-bit cache on the GPU at its edges: batches without tokens, numbers at the ends of their range, weights
far apart, long sums of one sign, NaN beside what a head reads.  Against definitions in 64 bits."""
import numpy as np
import pytest
import torch

import sparse_dimension_attention_b200 as aq
from oracle import paged_oracle as PO
from aqua_testlib import calib_P, rel_err_rows, tdev
from test_gpu_paged import DT, check_append, make_cache, oracle_decode, rope_of, rows_of, run_paged_decode, snap, torch_decode

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ batches without tokens

@pytest.mark.parametrize("B,Hq,Hkv,od,rejected", [
    (1, 4, 1, "bf16", False), (400, 8, 2, "f32", False), (400, 16, 2, "bf16", True), (33, 64, 8, "f32", True),
])
def test_decode_of_a_batch_without_tokens(B, Hq, Hkv, od, rejected):
    """Every length 0, or every length one that is refused: the output is 0 and lse -inf for the next kernel on the
    stream, whatever the workspace holds (fresh bytes, or the list of an earlier call with units in many parts)."""
    rng = np.random.default_rng(B)
    page, m, k = 16, 32, 20
    _, P32 = calib_P(Hkv)
    P = tdev(P32)
    cache = make_cache(B, Hkv, page, m, 6, seed=80)
    q = tdev(rows_of(rng, B, Hq, "bf16", 0.3), torch.bfloat16)
    none = torch.tensor([(-1 if i % 2 else 97) if rejected else 0 for i in range(B)], dtype=torch.int32, device="cuda")
    some = torch.tensor(rng.integers(1, 97, B), dtype=torch.int32, device="cuda")
    ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    seen = []
    for turn in range(12):
        if turn % 4 == 3:                     # parts and a list are left behind
            aq.aqua_paged_decode_attn(cache.desc, q, some, P, Hq, k, torch.empty(B, Hq, 128, dtype=DT[od], device="cuda"), ws)
        out = torch.full((B, Hq, 128), 7.0, dtype=DT[od], device="cuda")
        lse = torch.full((B, Hq), 7.0, device="cuda")
        sel = torch.full((B, Hq, k), -1, dtype=torch.int32, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, q, none, P, Hq, k, out, ws, lse_out=lse, sel_out=sel)
        seen.append((out.clone(), lse.clone(), sel.clone()))
    for out, lse, sel in seen:
        assert bool((out == 0).all()) and bool((lse == -np.inf).all()) and torch.equal(sel, seen[0][2])
    assert int(seen[0][2].min()) >= 0 and int(seen[0][2].max()) < m
    assert aq.aqua_paged_status(cache.desc) == (aq.abi.AQUA_ERR_ARG if rejected else aq.AQUA_OK)


# ------------------------------------------------------------------ append at the ends of the range

F32_MAX = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("n,io", [(300, "f32"), (300, "bf16"), (20, "f32"), (10, "f32")])     # tensor-core tiles, CUDA cores
def test_append_projections_past_f32(n, io):
    """Finite rows whose projection leaves f32 in one dimension: the finite ones set the page's scale, the
    others saturate or keep their own code, rows beside them (of the same warp too) are what they would be."""
    Hkv, page, m = 8, 64, 96
    rng = np.random.default_rng(81)
    _, P32 = calib_P(Hkv)
    P = P32.astype(np.float64)
    cache = make_cache(1, Hkv, page, m, -(-n // page), seed=82)
    k, v = rows_of(rng, n, Hkv, io), rows_of(rng, n, Hkv, io)
    big = torch.tensor(3e38).to(DT[io]).double().item()
    huge = [(3, 1, 5, 1.0), (9, 6, 90, -1.0)] + ([(100, 3, 0, 1.0), (107, 3, 64, -1.0), (299, 0, 17, 1.0)] if n > 299 else [])
    for t, h, j, sign in huge:
        k[t, h] = big * sign * np.sign(P[h, :, j])
    kt = np.einsum("nhi,hij->nhj", k, P)[..., :m]
    err = 132 * 2.0 ** -24 * np.einsum("nhi,hij->nhj", np.abs(k), np.abs(P))[..., :m]
    # f32 sums within err of the largest number may go either way
    over, finite = np.abs(kt) - err > F32_MAX, np.abs(kt) + err <= F32_MAX
    assert over.sum() >= len(huge)
    aq.aqua_paged_append(cache.desc, tdev(k, DT[io]), tdev(v, DT[io]), torch.zeros(1, dtype=torch.int32, device="cuda"),
                         tdev(P32), cu_new=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    a = snap(cache)
    for p0 in range(-(-n // page)):
        rows, pid = slice(p0 * page, min(n, p0 * page + page)), int(a["block_table"][0, p0])
        for h in range(Hkv):
            s = float(a["k_scale"][pid, h])
            x, e = kt[rows, h], err[rows, h]
            least = np.where(finite[rows, h], np.abs(x) - e, 0.0).max()
            most = np.where(over[rows, h], 0.0, np.minimum(np.abs(x) + e, F32_MAX)).max()
            assert PO.page_scale(max(least, 0.0)) <= s <= PO.page_scale(most)
            got = PO.e4m3_decode(a["k_pages"][pid, h])[:, :x.shape[0]].T
            ok = (PO.e4m3_round((x - e) / s) <= got) & (got <= PO.e4m3_round((x + e) / s))
            # a sum that left f32 was an infinity (448), or never took the form of an f32 number (its own code)
            ok |= ~finite[rows, h] & (got == np.sign(x) * 448)
            assert np.all(ok), (p0, h)
            np.testing.assert_array_equal(PO.e4m3_decode(a["v_pages"][pid, h][:x.shape[0]]),
                                          PO.e4m3_round(v[rows, h] / float(a["v_scale"][pid, h])))
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


@pytest.mark.parametrize("rope", [(128, False), (64, True), (36, False), (6, True)])
@pytest.mark.parametrize("n", [300, 10, 1])                                         # tensor-core tiles, CUDA cores, one token
def test_append_large_rows_rotated(n, rope):
    """Finite rows near the largest f32 number whose rotated entries may leave f32 while what they project to does not."""
    Hkv, page, m = 8, 64, 128
    rng = np.random.default_rng(86)
    _, P32 = calib_P(Hkv)
    P = P32.astype(np.float64)
    cache = make_cache(1, Hkv, page, m, -(-n // page) + 1, seed=87)
    r, rn, inter = rope_of(rope)
    k, v = rows_of(rng, n, Hkv, "f32"), rows_of(rng, n, Hkv, "f32")
    rot, start = rope[0], 7
    k[::3] = 0
    for i in range(0, n, 3):                  # one rotated pair of each such row: only its rotated entries may leave f32
        j = int(rng.integers(0, rot // 2))
        k[i, :, [2 * j, 2 * j + 1] if inter else [j, j + rot // 2]] = np.float64(np.float32(3.2e38)) * rng.choice([-1, 1], (2, 1))
    kr = PO.rotate(k, np.arange(start, start + n), rn, inter)
    kt, err = np.einsum("nhi,hij->nhj", kr, P), 132 * 2.0 ** -24 * np.einsum("nhi,hij->nhj", np.abs(kr), np.abs(P))
    assert np.all(np.abs(kt) + err < F32_MAX) and (n == 1 or np.abs(kr).max() > F32_MAX)
    cu = None if n == 1 else torch.tensor([0, n], dtype=torch.int32, device="cuda")
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k), tdev(v), torch.tensor([start], dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=cu, rope=r)
    check_append(cache, before, k, v, P32, [start], None if n == 1 else [0, n], rn, inter)


@pytest.mark.parametrize("n", [300, 20, 10])                            # tensor-core tiles, CUDA cores
def test_append_products_of_low_bits(n):
    """x0 = P0 = 1 + l, x1 = -1, P1 = 1 + 2 l with l just below half a step of f16 at 1: all that is left of the sum is
    l^2 = 2^-22, the product of what f16 leaves of both factors.  f32 sums may cut 2^-24 off twice on the way."""
    Hkv, page, m = 8, 64, 128
    l = 2.0 ** -11 - 2.0 ** -22
    k = np.zeros((n, Hkv, 128))
    k[:, :, 0], k[:, :, 1] = 1 + l, -1
    P32 = np.zeros((Hkv, 128, 128), dtype=np.float32)
    P32[:, 0], P32[:, 1] = 1 + l, 1 + 2 * l
    assert (k == k.astype(np.float32)).all() and P32[0, 1, 0] == 1 + 2 * l
    cache = make_cache(1, Hkv, page, m, -(-n // page), seed=85)
    aq.aqua_paged_append(cache.desc, tdev(k), tdev(k), torch.zeros(1, dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=torch.tensor([0, n], dtype=torch.int32, device="cuda"))
    a = snap(cache)
    kk, _ = PO.read_sequence(a["k_pages"], a["v_pages"], a["k_scale"], a["v_scale"], a["block_table"][0], n)
    assert np.abs(kk - l * l).max() <= 2.0 ** -23 + 2.0 ** -4 * l * l


def test_append_runs_that_share_rows():
    """cu_new that steps back between runs: those entries are reported and left alone, every run that is ascending is
    appended whole, although together they have more tokens than there are rows."""
    Hkv, page, m, pairs, n = 2, 16, 32, 13, 64
    rng = np.random.default_rng(83)
    _, P32 = calib_P(Hkv)
    cache = make_cache(2 * pairs - 1, Hkv, page, m, 5, seed=84)
    k, v = rows_of(rng, n, Hkv, "f32"), rows_of(rng, n, Hkv, "f32")
    cu = np.array([0, n] * pairs, dtype=np.int32)
    start = [3] * cache.B
    before = snap(cache)
    aq.aqua_paged_append(cache.desc, tdev(k), tdev(v), torch.tensor(start, dtype=torch.int32, device="cuda"), tdev(P32),
                         cu_new=torch.from_numpy(cu).cuda())
    check_append(cache, before, k, v, P32, start, cu, None, False, skip=tuple(range(1, cache.B, 2)))
    assert aq.aqua_paged_status(cache.desc) == aq.abi.AQUA_ERR_ARG


# ------------------------------------------------------------------ weights far apart, long sums

def pooled(Hkv, B, table, codes_k, codes_v):
    """A cache of B alike sequences whose table names pages of a small pool many times."""
    pool, page = codes_k.shape[0], codes_k.shape[3]
    one = torch.ones(pool, Hkv, device="cuda")
    return aq.AquaPagedCache.from_buffers(codes_k.cuda(), codes_v.cuda(), one, one.clone(),
                                          torch.tensor(np.repeat(table[None], B, 0), dtype=torch.int32, device="cuda"))


def pooled_ref(cache, q, n, k):
    """Output and lse in f64 (P = 1, scale 1 / sqrt(128)); the pages before the last are whole.  Also every token's
    weight relative to the largest of its head, and how often each occurs."""
    pool, H, m, page = cache.k_pages.shape
    G = q.shape[1] // H
    table = cache.block_table[0].long().cpu().numpy()[:-(-n // page)]
    count = np.repeat(np.bincount(table, minlength=pool)[:, None], page, 1).astype(np.float64)
    if n % page:
        count[table[-1], n % page:] -= 1
    c = torch.from_numpy(count).cuda().reshape(-1)
    out, lse, rel = [], [], []
    for h in range(H):
        kk = cache.k_pages[:, h].view(torch.float8_e4m3fn).double().permute(1, 0, 2).reshape(m, -1)
        vv = cache.v_pages[:, h].view(torch.float8_e4m3fn).double().reshape(-1, 128)
        qt = q[0, h * G:(h + 1) * G].double()
        keep = qt[:, :m].abs().topk(k, dim=1).indices
        qm = torch.zeros(G, m, dtype=torch.float64, device="cuda").scatter_(1, keep, qt.gather(1, keep))
        s = (qm @ kk / 128 ** 0.5).masked_fill(c == 0, -np.inf)
        top = s.amax(1, keepdim=True)
        w = torch.exp(s - top)
        total = (w * c).sum(1, keepdim=True)
        out.append((w * c) @ vv / total)
        lse.append((top + total.log())[:, 0])
        rel.append(w)
    return torch.cat(out), torch.cat(lse), torch.cat(rel), c


def decode_pooled(cache, q, n, k, od):
    B, Hq = cache.B, q.shape[1]
    P = torch.eye(128, device="cuda").expand(cache.Hkv, 128, 128).contiguous()
    out = torch.empty(B, Hq, 128, dtype=DT[od], device="cuda")
    lse = torch.empty(B, Hq, device="cuda")
    ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, Hq),), 0xFF, dtype=torch.uint8, device="cuda")
    aq.aqua_paged_decode_attn(cache.desc, q.repeat(B, 1, 1), torch.tensor([n] * B, dtype=torch.int32, device="cuda"), P, Hq,
                              k, out, ws, lse_out=lse)
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK
    return out.double(), lse.double()


@pytest.mark.parametrize("B,G,n,at,od", [
    (1, 8, 131072, 0, "bf16"), (1, 4, 131072, 700, "bf16"), (1, 8, 131072, 1023, "bf16"), (1, 8, 100, 0, "bf16"),
    (1, 1, 1280, 3, "bf16"), (300, 8, 32768, 0, "bf16"), (300, 4, 32768, 5, "bf16"), (300, 8, 32768, 250, "bf16"),
    (1, 8, 131072, 0, "f32"), (1, 4, 131072, 700, "f32"), (1, 8, 131072, 1023, "f32"), (1, 8, 100, 0, "f32"),
    (1, 1, 1280, 3, "f32"),
    (300, 8, 32768, 0, "f32"), (300, 4, 32768, 5, "f32"), (300, 8, 32768, 250, "f32"),
])
def test_decode_one_dominant_key_over_a_long_tail(B, G, n, at, od):
    """One key 12 to 20 nats above all others with a value of nearly nothing: the output is what the others add up to.

    What the weights lose: rounded to f16 they are off by half a step at most, 2^-11 of themselves or 2^-25 where the
    largest is 2^12 or more, so 2^-37 of that; for an f32 output the rest is rounded to f16 again, 2^-22 and 2^-49.
    Over a sum of weights the second is n steps against their sum.  Then q~ (off by 2^-16 and 2^-24, which moves scores
    of up to 20 by 20 times that), the output's own rounding (eps / 2 of bf16, 2^-8) and 1e-5 for all sums in f32."""
    page, m, k, pool = 128, 32, 16, 33
    g = torch.Generator().manual_seed(90)
    ck = torch.randint(0x10, 0x28, (pool, 1, m, page), generator=g) + 128 * torch.randint(0, 2, (pool, 1, m, page), generator=g)
    cv = torch.randint(0x30, 0x38, (pool, 1, page, 128), generator=g)
    ck[:, 0, 0] = 0
    ck[0, 0, :, 37] = 0
    ck[0, 0, 0, 37] = 0x58                     # 16
    cv[0, 0, 37, :64], cv[0, 0, 37, 64:] = 0, 1
    table = np.random.default_rng(91).integers(1, pool, -(-n // page))
    table[at] = 0
    cache = pooled(1, B, table, ck.to(torch.uint8), cv.to(torch.uint8))
    gaps = [17.0] if G == 1 else list(np.linspace(12, 20, G))
    q = torch.zeros(1, G, 128)
    q[0, :, 1:k] = 0.5 + torch.rand(G, k - 1, generator=g)
    q[0, :, 0] = torch.tensor(gaps) / 16 * 128 ** 0.5
    q = q.cuda()
    got, lse = decode_pooled(cache, q, n, k, od)
    ref, lref, w, c = pooled_ref(cache, q, n, k)
    tail = (c.sum() - 1) / ((w * c).sum(1) - 1)          # tokens over the sum of their weights (the dominant one's is 1)
    half_step, grid, query, own = (2.0 ** -11, 2.0 ** -37, 2.0 ** -16, 2.0 ** -8) if od == "bf16" else (2.0 ** -22, 2.0 ** -49, 2.0 ** -24, 0)
    tol = half_step + tail * grid + 20 * query + own + 1e-5
    for half in (slice(0, 64), slice(64, 128)):
        err = ((got - ref)[..., half].norm(dim=-1) / ref[:, half].norm(dim=-1)).amax(0)
        assert bool((err <= tol).all()), (err.tolist(), tol.tolist())
    assert float((lse - lref).abs().max()) <= (20 * 2.0 ** -16 if od == "bf16" else 20 * 2.0 ** -22)


@pytest.mark.parametrize("G,tokens,od,spread", [(4, 30_000_000, "f32", 0), (8, 100_000_000, "f32", 0), (8, 30_000_000, "f32", 1),
                                                (1, 3_000_000, "f32", 1), (4, 100_000_000, "bf16", 1)])
def test_decode_long_sums_of_one_sign(G, tokens, od, spread):
    """Values of one sign over hundreds of tiles a block: sums that are cut off would all lose.
    f32 outputs 1e-5 as everywhere; bf16: its own rounding (eps / 2, 2^-8) and what the header allows the sums, 2^-10."""
    page, m, k, pool = 128, 16, 8, 64
    g = torch.Generator().manual_seed(92)
    ck = torch.randint(0x28, 0x40, (pool, 1, m, page), generator=g) if spread else torch.randint(0x10, 0x28, (pool, 1, m, page), generator=g)
    ck = ck + 128 * torch.randint(0, 2, (pool, 1, m, page), generator=g)
    cv = torch.randint(0x30, 0x38, (pool, 1, page, 128), generator=g)
    n = tokens // page * page
    cache = pooled(1, 1, np.random.default_rng(93).integers(0, pool, n // page), ck.to(torch.uint8), cv.to(torch.uint8))
    q = (torch.randn(1, G, 128, generator=g) * (4 if spread else 1)).cuda()
    got, lse = decode_pooled(cache, q, n, k, od)
    ref, lref, _, _ = pooled_ref(cache, q, n, k)
    err = ((got - ref).norm(dim=-1) / ref.norm(dim=-1)).amax(0)
    assert float(err.max()) <= (1e-5 if od == "f32" else 2.0 ** -8 + 2.0 ** -10), err.tolist()
    assert float((lse - lref).abs().max()) <= (1e-5 if od == "f32" else 2e-4)


# ------------------------------------------------------------------ NaN, and queries at the ends of their range

@pytest.mark.parametrize("od", ["bf16", "f32"])
def test_decode_nan_keys_in_dimensions_that_a_head_left_out(od):
    """A head sums over its own dimensions alone: a NaN code in one it did not keep does nothing, wherever the token
    lies and whether or not another head of the group kept that dimension; in a kept one it makes the head NaN, a
    query entry of 0 too."""
    B, Hq, Hkv, page, m, k = 2, 8, 2, 64, 100, 6
    lens = [1400, 1397]
    rng = np.random.default_rng(94)
    cache = make_cache(B, Hkv, page, m, 22, seed=95)
    for b, h, t, dims in ((0, 0, 3, (7, 50)), (0, 0, 130, (7,)), (0, 0, 300, (50, 20)), (0, 0, 1399, (7, 99)),
                          (1, 1, 700, (7,)), (1, 1, 1301, (20,)), (0, 1, 901, (3,))):
        for j in dims:
            cache.k_pages[int(cache.block_table[b, t // page]), h, j, t % page] = 0x7F if t % 2 else 0xFF
    q = np.zeros((B, Hq, 128))
    q[:, :, 30:36] = rng.normal(size=(B, Hq, 6)) + 4.0          # heads 0, 4: dims 30 .. 35
    for h, j in ((1, 7), (2, 20), (5, 7), (6, 20)):             # and one NaN dimension of sequence 0 or 1
        q[:, h, j] = 9.0
    q[:, 3, 30:] = 0.0                                          # heads 3, 7 keep dims 0 .. 5 at 0
    q[:, 7, 30:] = 0.0
    P32 = np.broadcast_to(np.eye(128, dtype=np.float32), (Hkv, 128, 128)).copy()
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, DT[od], torch.float32)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, od)
    np.testing.assert_array_equal(got["sel"], ref["sel"])
    want = np.zeros((B, Hq), dtype=bool)
    want[0, 1] = want[0, 2] = want[1, 5] = want[1, 6] = want[0, 7] = True
    np.testing.assert_array_equal(np.isnan(ref["out"]).any(-1), want)
    np.testing.assert_array_equal(np.isnan(got["out"]), np.broadcast_to(want[..., None], got["out"].shape))
    np.testing.assert_array_equal(np.isnan(got["lse"]), want)
    assert np.max(rel_err_rows(got["out"][~want], ref["out"][~want])) <= (2e-3 if od == "bf16" else 1e-5)
    assert aq.aqua_paged_status(cache.desc) == aq.AQUA_OK


@pytest.mark.parametrize("n", [900, 20000, 131072])
def test_decode_nan_keys_left_out_in_a_unit_of_many_parts(n):
    """The same where a unit is shared by few and by many blocks: one head left the NaN out, one kept it, one more has a
    whole row of NaN only behind the length."""
    page, m, k, G = 64, 96, 40, 3
    rng = np.random.default_rng(101)
    cache = make_cache(1, 1, page, m, -(-(n + 1) // page), seed=102)
    table = cache.block_table[0].tolist()
    for t in rng.integers(0, n, 5):
        cache.k_pages[table[t // page], 0, 90, int(t) % page] = 0x7F
    cache.k_pages[table[n // page], 0, :, n % page] = 0xFF
    q = rng.normal(size=(1, G, 128)) * 0.1 + 1.0
    q[0, :, 90] = [0.01, 3.0, -0.01]
    qt = tdev(q)
    P = torch.eye(128, device="cuda")[None].contiguous()
    for od, tol in (("f32", 1e-5), ("bf16", 4e-3)):
        out = torch.empty(1, G, 128, dtype=DT[od], device="cuda")
        lse = torch.empty(1, G, device="cuda")
        ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, G),), 0xFF, dtype=torch.uint8, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, qt, torch.tensor([n], dtype=torch.int32, device="cuda"), P, G, k, out, ws, lse_out=lse)
        clean = cache.k_pages.clone()
        codes = clean.view(torch.float8_e4m3fn).float()
        cache.k_pages.masked_fill_(codes.isnan(), 0)
        ref = torch_decode(cache, qt, [n], P, k)
        cache.k_pages.copy_(clean)
        assert bool(out[0, 1].isnan().all()) and bool(lse[0, 1].isnan())
        for h in (0, 2):
            assert float((out[0, h].double() - ref[0, h]).norm() / ref[0, h].norm()) <= tol
            assert bool(lse[0, h].isfinite())


@pytest.mark.parametrize("exponent", [100, 118, 126, -100, -118])
def test_decode_queries_at_the_ends_of_the_range(exponent):
    """Queries of 2^exponent against keys whose page scales bring the scores back to the usual size."""
    B, Hq, Hkv, page, m, k, lens = 1, 4, 1, 16, 64, 40, [300]
    rng = np.random.default_rng(96)
    cache = make_cache(B, Hkv, page, m, 19, seed=97)
    cache.k_scale.fill_(2.0 ** (-6 - exponent))
    q = rng.uniform(0.25, 1.9, size=(B, Hq, 128)) * np.where(rng.random((B, Hq, 128)) < 0.5, -1, 1)
    q = (q * 2.0 ** exponent).astype(np.float32).astype(np.float64)
    P32 = np.eye(128, dtype=np.float32)[None]
    got = run_paged_decode(cache, q, lens, tdev(P32), k, None, torch.float32, torch.float32)
    ref = oracle_decode(snap(cache), lens, q, P32, k, None, False, "f32")
    np.testing.assert_array_equal(got["sel"], ref["sel"])
    assert np.max(rel_err_rows(got["out"], ref["out"])) <= 1e-5


# ------------------------------------------------------------------ P written by the kernel just before

@pytest.mark.parametrize("what", ["step", "tiles", "decode"])
def test_a_projection_that_the_kernel_before_writes(what):
    """P computed on the same stream right before the call, another one each time, with the append or step before still
    on the GPU: each call reads its own P."""
    Hkv, Hq, page, m, k = 2, 8, 64, 128, 128
    rng = np.random.default_rng(98)
    _, P32 = calib_P(Hkv)
    base = tdev(P32)
    n = 600 if what == "tiles" else 2
    x, v = tdev(rows_of(rng, n, Hkv, "f32", 0.3)), tdev(rows_of(rng, n, Hkv, "f32", 0.3))
    q = tdev(rows_of(rng, 2, Hq, "f32", 0.3))
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n // 2, n], dtype=torch.int32, device="cuda") if what == "tiles" else None
    ln = torch.tensor([500, 77], dtype=torch.int32, device="cuda")
    turns = [(1.0, 0), (-2.0, 5), (0.5, 40), (4.0, 99)] * 3
    Ps = [(f * base.roll(r, 2)).contiguous() for f, r in turns]

    def call(cache, P, ws, out):
        if what == "decode":
            aq.aqua_paged_decode_attn(cache.desc, q, ln, P, Hq, k, out, ws)
        else:
            aq.aqua_paged_append(cache.desc, x, v, start, P, cu_new=cu)

    def fresh():
        cache = make_cache(2, Hkv, page, m, 8, seed=99)
        return cache, torch.empty(aq.aqua_paged_decode_workspace_size(cache.desc, Hq), dtype=torch.uint8, device="cuda"), \
            torch.zeros(2, Hq, 128, device="cuda")

    caches, want, got = [fresh() for _ in turns], [], []
    for P, (c, ws, out) in zip(Ps, caches):
        torch.cuda.synchronize()
        call(c, P, ws, out)
        torch.cuda.synchronize()
        want.append((c.k_pages.clone(), c.k_scale.clone(), out.clone()))
    caches = [fresh() for _ in turns]
    P = torch.empty_like(base)
    torch.cuda.synchronize()
    for (f, r), (c, ws, out) in zip(turns, caches):
        torch.mul(base.roll(r, 2), f, out=P)
        call(c, P, ws, out)
    torch.cuda.synchronize()
    for w, (c, ws, out) in zip(want, caches):
        for a, b in zip(w, (c.k_pages, c.k_scale, out)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("size,rise", [(s, r) for s in (24.3, 25.3, 26.3, 30.0) for r in (2.0, 4.0, 8.0, 12.0)])
def test_decode_scores_so_large_that_f32_steps_show(size, rise, od):
    """Scores around 2^size (in powers of two) that rise by about one step of f32 from tile to tile: whatever the
    weights are, all values are 1, and so is the output."""
    page, m, k, G, tiles = 128, 16, 2, 1, 40
    codes = [0x38 + i for i in range(tiles)]                                   # 1, 1.125, ... in dimension 1, one a tile
    ck = torch.zeros(tiles, 1, m, page, dtype=torch.uint8)
    ck[:, 0, 0] = 0x78                                                        # 256 in dimension 0
    for i, c in enumerate(codes):
        ck[i, 0, 1] = c
    cv = torch.full((tiles, 1, page, 128), 0x38, dtype=torch.uint8)
    cache = pooled(1, 64, np.arange(tiles), ck, cv)
    step = 2.0 ** (int(size) - 23)
    q = torch.zeros(1, G, 128)
    q[0, :, 0] = 2.0 ** size / 256 * 0.6931471805599453 * 128 ** 0.5
    q[0, :, 1] = rise * step * 128 ** 0.5
    got, lse = decode_pooled(cache, q.cuda(), tiles * page, k, od)
    assert bool(((got - 1).abs() <= (2.0 ** -8 if od == "bf16" else 1e-5)).all()) and bool(lse.isfinite().all())


@pytest.mark.parametrize("od", ["bf16", "f32"])
def test_decode_parts_of_very_large_scores_keep_their_distance(od):
    """One unit in many parts, the scores of its first half 1.25 * 2^26 and those of its second half 8 more (in powers of
    two, one step of f32; the scale argument makes them exact): the first half weighs 2^-8 of the second."""
    page, m, k, n_pages = 128, 16, 2, 4000
    ck = torch.zeros(2, 1, m, page, dtype=torch.uint8)
    ck[:, 0, 0] = 0x78                                                        # 256
    ck[1, 0, 1] = 0x38                                                        # 1
    cv = torch.full((2, 1, page, 128), 0x38, dtype=torch.uint8)
    cv[1] = 0x30                                                              # 0.5
    scale = float(np.float32(np.log(2)))
    assert np.float32(scale) * np.float32(1.4426950408889634) == 1
    cache = pooled(1, 1, np.repeat([0, 1], n_pages // 2), ck, cv)
    q = torch.zeros(1, 1, 128)
    q[0, 0, 0], q[0, 0, 1] = 1.25 * 2 ** 18, 8
    out, lse = torch.empty(1, 1, 128, dtype=DT[od], device="cuda"), torch.empty(1, 1, device="cuda")
    ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    aq.aqua_paged_decode_attn(cache.desc, q.cuda(), torch.tensor([n_pages * page], dtype=torch.int32, device="cuda"),
                              torch.eye(128, device="cuda")[None].contiguous(), 1, k, out, ws, scale=scale, lse_out=lse)
    want = (2.0 ** -8 + 0.5) / (1 + 2.0 ** -8)
    assert float((out.double() - want).abs().max()) <= (want * 2.0 ** -8 if od == "bf16" else 1e-5)
    # a sum and a product, each half a step (2^-24) off, and ln 2 in f32 (0.5 * 2^-24)
    assert abs(float(lse) / (np.log(2) * (1.25 * 2 ** 26 + 8 + np.log2(n_pages / 2 * page * (1 + 2.0 ** -8)))) - 1) <= 2.5 * 2.0 ** -24


def test_decode_weights_of_bf16_outputs():
    """One token of weight 2 / (1 + e) and value 1, two of weight 1 and value -1: the output is what two nearly equal sums
    leave, -e / 2, for 512 values of e.  The weights of a bf16 output are held to 2^-12 of themselves (an f16 number:
    2^-11, which is most off just above a power of two, where the smaller one lies), its queries to 2^-16."""
    B, G, page, m, k = 64, 8, 16, 16, 1
    ck, cv = torch.zeros(1, 1, m, page, dtype=torch.uint8), torch.full((1, 1, page, 128), 0xB8, dtype=torch.uint8)
    ck[0, 0, 0, 0], cv[0, 0, 0] = 0x38, 0x38
    cache = pooled(1, B, np.zeros(1, dtype=np.int64), ck, cv)
    e = np.exp2(np.random.default_rng(103).uniform(-8, -4, (B, G)))
    q = np.zeros((B, G, 128))
    q[..., 0] = np.log(2 / (1 + e))
    q = torch.from_numpy(q).float().cuda()
    P = torch.eye(128, device="cuda")[None].contiguous()
    for od in ("bf16", "f32"):
        out = torch.empty(B, G, 128, dtype=DT[od], device="cuda")
        ws = torch.full((aq.aqua_paged_decode_workspace_size(cache.desc, G),), 0xFF, dtype=torch.uint8, device="cuda")
        aq.aqua_paged_decode_attn(cache.desc, q, torch.full((B,), 3, dtype=torch.int32, device="cuda"), P, G, k, out, ws, scale=1.0)
        w = torch.exp(q[..., :1].double())
        ref = (w - 2) / (w + 2)
        tol = 0.5 * (2.0 ** -12 + 2.0 ** -16) + 2.0 ** -8 * ref.abs() if od == "bf16" else 1e-6
        assert bool(((out.double() - ref).abs() <= tol).all())
