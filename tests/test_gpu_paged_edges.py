"""Paged 8-bit cache on the GPU at its edges: batches without tokens, numbers at the ends of their range, weights
far apart, long sums of one sign, NaN beside what a head reads.  Against definitions in 64 bits."""
import numpy as np
import pytest
import torch

import sparse_dimension_attention_b200 as aq
from oracle import paged_oracle as PO
from aqua_testlib import calib_P, rel_err_rows, tdev
from test_gpu_paged import DT, make_cache, rows_of, run_paged_decode, snap

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
