"""Paged 8-bit cache on the GPU at its edges: batches without tokens, numbers at the ends of their range, weights
far apart, long sums of one sign, NaN beside what a head reads.  Against definitions in 64 bits."""
import numpy as np
import pytest
import torch

import sparse_dimension_attention_b200 as aq
from oracle import paged_oracle as PO
from aqua_testlib import calib_P, rel_err_rows, tdev
from test_gpu_paged import DT, check_append, make_cache, rows_of, run_paged_decode, snap

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


@pytest.mark.parametrize("n,io", [(300, "f32"), (300, "bf16"), (20, "f32")])       # tensor-core tiles, CUDA cores
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
