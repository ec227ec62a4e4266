"""CPU checks of the paged 8-bit cache: the oracle's pieces against closed forms
and torch's own e4m3 type, the descriptors' layout, and the refusals of the C
entry points and of the Python layer (nothing touches a GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
import sparse_dimension_attention_b200 as aq
from sparse_dimension_attention_b200 import abi


@pytest.fixture(scope="module")
def lib():
    from sparse_dimension_attention_b200 import build
    build.build()
    return aq.load_library()


# ------------------------------------------------------------------ oracle pins

def test_e4m3_table_is_torch_e4m3():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    ref = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(PO.e4m3_decode(codes.numpy()), ref)


def test_e4m3_round_is_nearest_even():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000), PO._POS, -PO._POS,
                        (PO._POS[1:] + PO._POS[:-1]) / 2])                       # numbers and exact ties
    got = PO.e4m3_round(x)
    ref = torch.from_numpy(x).clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).double().numpy()
    exact32 = x.astype(np.float32).astype(np.float64) == x                      # torch goes through f32
    np.testing.assert_array_equal(got[exact32], ref[exact32])
    # brute force: no e4m3 number is nearer
    d = np.abs(np.clip(x, -448, 448)[:, None] - np.concatenate([PO._POS, -PO._POS])[None])
    np.testing.assert_allclose(np.abs(got - np.clip(x, -448, 448)), d.min(1), rtol=0, atol=0)
    assert np.isnan(PO.e4m3_round(np.nan)) and PO.e4m3_round(np.inf) == 448 and PO.e4m3_round(-1e9) == -448


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (1.75, 2.0 ** -8), (1.0, 2.0 ** -8),
                                        (0.0, 2.0 ** -60), (1e-30, 2.0 ** -60), (3e38, 2.0 ** 120)])
def test_page_scale(amax, scale):
    assert PO.page_scale(amax) == scale


def test_rotation_keeps_norms_and_relative_positions():
    rng = np.random.default_rng(1)
    ang = np.arange(50)[:, None] * 10.0 ** -np.linspace(0, 3, 32)[None]
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    for inter in (False, True):
        q, k = rng.normal(size=(2, 1, 1, 128))
        dots = []
        for shift in (0, 7, 30):
            qr, kr = PO.rotate(q, [12 + shift], table, inter), PO.rotate(k, [5 + shift], table, inter)
            assert abs(np.linalg.norm(qr) - np.linalg.norm(q)) < 1e-12
            np.testing.assert_array_equal(qr[..., 64:], q[..., 64:])            # dimensions past rot_dim stay
            dots.append(float((qr * kr).sum()))
        assert max(dots) - min(dots) < 1e-11


def test_append_to_block_recodes_exactly_but_for_subnormals():
    vals = PO._POS.reshape(1, -1)
    out = PO.append_to_block(vals, 1.0, 1, np.zeros((0, 127)), 4.0)
    exact = PO._POS / 4
    normal = exact >= 2.0 ** -6
    np.testing.assert_array_equal(out[0, normal], exact[normal])
    assert np.all(np.abs(out[0] - exact) <= 2.0 ** -10)                          # half a subnormal step


# ------------------------------------------------------------------ layout and refusals

def test_struct_layout():
    assert ctypes.sizeof(abi.aqua_paged_cache) == 6 * 8 + 8 * 4
    assert abi.aqua_paged_cache.B.offset == 48 and abi.aqua_paged_cache.dtype.offset == 48 + 7 * 4
    assert ctypes.sizeof(abi.aqua_rope) == 24 and abi.aqua_rope.interleaved.offset == 16


def _desc(**kw):
    base = dict(k_pages=0x10000, v_pages=0x20000, k_scale=0x3000, v_scale=0x3100, block_table=0x3200, ctrl=0x3300,
                B=2, Hkv=2, d=128, d_store=96, page_size=64, n_pages=8, max_pages=4, dtype=abi.AQUA_E4M3)
    base.update(kw)
    return abi.aqua_paged_cache(**base)


BAD_CACHES = [
    ("k_pages", None, abi.AQUA_ERR_ARG), ("v_pages", None, abi.AQUA_ERR_ARG), ("k_scale", None, abi.AQUA_ERR_ARG),
    ("v_scale", None, abi.AQUA_ERR_ARG), ("block_table", None, abi.AQUA_ERR_ARG), ("ctrl", None, abi.AQUA_ERR_ARG),
    ("k_pages", 0x10008, abi.AQUA_ERR_ARG), ("v_pages", 0x20004, abi.AQUA_ERR_ARG),
    ("k_scale", 0x3002, abi.AQUA_ERR_ARG), ("block_table", 0x3201, abi.AQUA_ERR_ARG),
    ("dtype", abi.AQUA_BF16, abi.AQUA_ERR_UNSUPPORTED), ("d", 64, abi.AQUA_ERR_UNSUPPORTED),
    ("d_store", 0, abi.AQUA_ERR_ARG), ("d_store", 129, abi.AQUA_ERR_ARG),
    ("page_size", 8, abi.AQUA_ERR_UNSUPPORTED), ("page_size", 48, abi.AQUA_ERR_UNSUPPORTED),
    ("page_size", 256, abi.AQUA_ERR_UNSUPPORTED),
    ("B", 0, abi.AQUA_ERR_ARG), ("Hkv", 0, abi.AQUA_ERR_ARG), ("n_pages", 0, abi.AQUA_ERR_ARG),
    ("max_pages", 0, abi.AQUA_ERR_ARG), ("max_pages", 1 << 25, abi.AQUA_ERR_UNSUPPORTED),
    ("B", 1 << 24, abi.AQUA_ERR_UNSUPPORTED),
]


def _append(lib, c, **kw):
    a = dict(k=0x40000, v=0x50000, io=abi.AQUA_BF16, ks=0, kh=0, vs=0, vh=0, n=2, start=0x6000, cu=None, P=0x7000,
             rope=None)
    a.update(kw)
    rope = ctypes.byref(a["rope"]) if a["rope"] is not None else None
    return lib.aqua_paged_append(ctypes.byref(c) if c is not None else None, a["k"], a["v"], a["io"], a["ks"],
                                 a["kh"], a["vs"], a["vh"], a["n"], a["start"], a["cu"], a["P"], rope, None)


def _decode(lib, c, **kw):
    a = dict(len=0x6000, q=0x40000, io=abi.AQUA_BF16, qs=0, qh=0, P=0x7000, rope=None, Hq=8, k=64, out=0x80000,
             od=abi.AQUA_BF16, sel=None, qp=None, lse=None, ws=0x100000, wsb=1 << 40)
    a.update(kw)
    rope = ctypes.byref(a["rope"]) if a["rope"] is not None else None
    return lib.aqua_paged_decode_attn(ctypes.byref(c), a["len"], a["q"], a["io"], a["qs"], a["qh"], a["P"], rope,
                                      a["Hq"], a["k"], 0.0, a["out"], a["od"], a["sel"], a["qp"], a["lse"], a["ws"],
                                      a["wsb"], None)


@pytest.mark.parametrize("field,value,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, field, value, code):
    c = _desc(**{field: value})
    assert _append(lib, c) == code
    assert lib.aqua_last_error().decode() != ""
    assert _decode(lib, c) == code
    assert lib.aqua_paged_decode_workspace_size(ctypes.byref(c), 8) == 0
    dst = abi.aqua_cache(k_proj=0x1000, v=0x2000, len=0x3000, ctrl=0x3100, B=2, Hkv=2, d=128, d_store=96, Tcap=64,
                         dtype=abi.AQUA_BF16)
    assert lib.aqua_paged_gather(ctypes.byref(c), 0x6000, None, ctypes.byref(dst), 64, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), abi.AQUA_ERR_ARG), (dict(v=None), abi.AQUA_ERR_ARG), (dict(start=None), abi.AQUA_ERR_ARG),
    (dict(P=None), abi.AQUA_ERR_ARG), (dict(k=0x40008), abi.AQUA_ERR_ARG), (dict(P=0x7004), abi.AQUA_ERR_ARG),
    (dict(start=0x6001), abi.AQUA_ERR_ARG), (dict(cu=0x6102), abi.AQUA_ERR_ARG),
    (dict(io=abi.AQUA_E4M3), abi.AQUA_ERR_UNSUPPORTED), (dict(io=9), abi.AQUA_ERR_UNSUPPORTED),
    (dict(n=0), abi.AQUA_ERR_ARG), (dict(n=-1), abi.AQUA_ERR_ARG), (dict(n=3), abi.AQUA_ERR_ARG),   # n != B without cu
    (dict(ks=64), abi.AQUA_ERR_ARG), (dict(ks=260), abi.AQUA_ERR_ARG), (dict(vh=132), abi.AQUA_ERR_ARG),
    (dict(kh=-128), abi.AQUA_ERR_ARG), (dict(vs=1 << 40), abi.AQUA_ERR_ARG),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, _desc(), **kw) == code
    assert lib.aqua_last_error().decode() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(cos_sin=None), abi.AQUA_ERR_ARG), (dict(cos_sin=0x9004), abi.AQUA_ERR_ARG), (dict(rot_dim=0), abi.AQUA_ERR_ARG),
    (dict(rot_dim=63), abi.AQUA_ERR_ARG), (dict(rot_dim=130), abi.AQUA_ERR_ARG), (dict(n_pos=0), abi.AQUA_ERR_ARG),
    (dict(interleaved=2), abi.AQUA_ERR_ARG),
])
def test_rope_refusals(lib, kw, code):
    r = dict(cos_sin=0x9000, n_pos=16, rot_dim=64, interleaved=0)
    r.update(kw)
    rope = abi.aqua_rope(**r)
    assert _append(lib, _desc(), rope=rope) == code
    assert _decode(lib, _desc(), rope=rope) == code


@pytest.mark.parametrize("kw,code", [
    (dict(len=None), abi.AQUA_ERR_ARG), (dict(q=None), abi.AQUA_ERR_ARG), (dict(P=None), abi.AQUA_ERR_ARG),
    (dict(out=None), abi.AQUA_ERR_ARG), (dict(ws=None), abi.AQUA_ERR_ARG), (dict(q=0x40008), abi.AQUA_ERR_ARG),
    (dict(out=0x80004), abi.AQUA_ERR_ARG), (dict(ws=0x100010), abi.AQUA_ERR_ARG), (dict(lse=0x9001), abi.AQUA_ERR_ARG),
    (dict(Hq=7), abi.AQUA_ERR_ARG), (dict(Hq=0), abi.AQUA_ERR_ARG), (dict(Hq=18), abi.AQUA_ERR_UNSUPPORTED),
    (dict(k=0), abi.AQUA_ERR_ARG), (dict(k=97), abi.AQUA_ERR_ARG), (dict(io=2), abi.AQUA_ERR_UNSUPPORTED),
    (dict(od=2), abi.AQUA_ERR_UNSUPPORTED), (dict(qs=100), abi.AQUA_ERR_ARG), (dict(qh=129), abi.AQUA_ERR_ARG),
    (dict(wsb=1024), abi.AQUA_ERR_WORKSPACE),
])
def test_decode_refusals(lib, kw, code):
    assert _decode(lib, _desc(), **kw) == code
    assert lib.aqua_last_error().decode() != ""


def test_decode_workspace_size(lib):
    size = lambda Hq, **kw: lib.aqua_paged_decode_workspace_size(ctypes.byref(_desc(**kw)), Hq)
    need = size(8)
    assert 0 < need < size(8, B=64)
    assert _decode(lib, _desc(), wsb=need - 1) == abi.AQUA_ERR_WORKSPACE
    assert size(7) == 0 and size(0) == 0 and size(18) == 0


def test_gather_refusals(lib):
    def gather(c=None, len=0x6000, idx=None, max_len=64, **kw):
        d = dict(k_proj=0x1000, v=0x2000, len=0x3000, ctrl=0x3100, B=2, Hkv=2, d=128, d_store=96, Tcap=64,
                 dtype=abi.AQUA_BF16)
        d.update(kw)
        dst = abi.aqua_cache(**d)
        rc = lib.aqua_paged_gather(ctypes.byref(c or _desc()), len, idx, ctypes.byref(dst), max_len, None)
        assert dst.max_len == 0                                  # unchanged on failure
        return rc
    assert gather(len=None) == abi.AQUA_ERR_ARG
    assert gather(len=0x6002) == abi.AQUA_ERR_ARG
    assert gather(k_proj=None) == abi.AQUA_ERR_ARG
    assert gather(k_proj=0x1008) == abi.AQUA_ERR_ARG
    assert gather(dtype=abi.AQUA_E4M3) == abi.AQUA_ERR_UNSUPPORTED
    assert gather(d_store=128) == abi.AQUA_ERR_ARG
    assert gather(Hkv=4) == abi.AQUA_ERR_ARG
    assert gather(B=3) == abi.AQUA_ERR_ARG                       # another batch without an index
    assert gather(max_len=65) == abi.AQUA_ERR_ARG
    assert gather(max_len=-1) == abi.AQUA_ERR_ARG
    assert gather(Tcap=40, max_len=8) == abi.AQUA_ERR_ARG
    assert gather(dv_store=16) == abi.AQUA_ERR_UNSUPPORTED
    assert gather(pos=0x4000, score=0x4100, n_abs=0x4200) == abi.AQUA_ERR_UNSUPPORTED


def test_python_layer_refuses_what_c_cannot_see():
    """Host tensors, wrong types and shapes: the C side sees addresses only."""
    cache = aq.AquaPagedCache(2, 2, 8, 4, device="cpu")
    assert cache.desc.page_size == 64 and cache.desc.n_pages == 8 and cache.desc.dtype == abi.AQUA_E4M3
    k = torch.zeros(2, 2, 128)
    start = torch.zeros(2, dtype=torch.int32)
    P = torch.zeros(2, 128, 128)
    with pytest.raises(aq.AquaError):
        aq.aqua_paged_append(cache.desc, k, k, start, P)                        # not on a device
    with pytest.raises(aq.AquaError):
        aq.aqua_paged_append(cache.desc, k.half(), k.half(), start, P)
    with pytest.raises(aq.AquaError):
        aq.aqua_paged_decode_attn(cache.desc, k, start, P, 2, 8, k, k)
    with pytest.raises(aq.AquaError):
        aq.aqua_paged_gather(cache.desc, start, abi.aqua_cache(), 0)
    good = [cache.k_pages, cache.v_pages, cache.k_scale, cache.v_scale, cache.block_table]
    for i, bad in enumerate([cache.k_pages.float(), cache.v_pages[:, :, :32], cache.k_scale[:4], cache.v_scale.double(),
                             cache.block_table.long()]):
        with pytest.raises(aq.AquaError):
            aq.AquaPagedCache.from_buffers(*good[:i], bad, *good[i + 1:])
    with pytest.raises(aq.AquaError):
        aq.AquaRope(torch.zeros(4, 64, dtype=torch.float64))
    rope = aq.AquaRope.from_theta(16, rot_dim=32, device="cpu")
    assert rope.desc.n_pos == 16 and rope.desc.rot_dim == 32
    np.testing.assert_allclose(rope.cos_sin[3, 0].item(), np.cos(3.0), rtol=1e-7)


@pytest.mark.parametrize("kw", [
    dict(n_pages=1 << 24, Hkv=2),                                      # 2^31 value rows with pages of 64
    dict(n_pages=(1 << 31) - 1, Hkv=8),
    dict(Hkv=65536, B=1), dict(B=1 << 23, Hkv=4),
    dict(max_pages=(1 << 24) + 1),                                     # over 2^30 slots a sequence
    dict(B=1 << 20, max_pages=(1 << 11) + 1),                          # over 2^37 slots of all sequences
    dict(B=(1 << 24) - 1, Hkv=1, max_pages=(1 << 24)),
])
def test_sizes_past_the_counters_are_refused(lib, kw):
    """Rows, slots and tiles are counted in 32 bits on the device: nothing is launched past that."""
    c = _desc(**kw)
    assert _append(lib, c, n=c.B) == abi.AQUA_ERR_UNSUPPORTED
    assert _decode(lib, c, Hq=c.Hkv) == abi.AQUA_ERR_UNSUPPORTED
    assert lib.aqua_paged_decode_workspace_size(ctypes.byref(c), c.Hkv) == 0


@pytest.mark.parametrize("kw", [
    dict(n_pages=(1 << 24) - 1, Hkv=2), dict(max_pages=1 << 24), dict(B=1 << 20, max_pages=1 << 11),
])
def test_the_largest_sizes_are_accepted(lib, kw):
    c = _desc(**kw)
    assert lib.aqua_paged_decode_workspace_size(ctypes.byref(c), 8) > 0
    assert _append(lib, c, n=0) == abi.AQUA_ERR_ARG                    # the cache passed; the count did not
