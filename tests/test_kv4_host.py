"""The 4-bit cache without a GPU: the reference's own pins, and the refusals of every entry point."""
import ctypes
import math

import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import kv4 as ref
from tests._lib import ensure_library


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


# ---------------------------------------------------------------- the reference
def test_reference_levels_and_scales():
    x = np.zeros((1, 16))
    x[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]  # scale 1; the borders go to the even level
    x[0, 8:] = -x[0, :8] * 0.999
    codes, bits = ref.encode(x)
    assert bits[0, 0] == 15 * 8 and ref.SCALES[bits[0, 0]] == 1
    assert list(ref.LEVELS[codes[0, :8]]) == [6, 0, 1, 1, 2, 2, 4, 4]
    assert list(ref.decode(codes, bits)[0, 8:]) == [-6, 0, -0.5, -1, -1.5, -2, -3, -4]
    assert np.array_equal(np.sort(ref.SCALES), ref.SCALES) and ref.SCALES[224] == 2 ** 13 and ref.SCALES[1] == 2.0 ** -17


def test_reference_scale_is_the_nearest_and_error_is_bounded():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp(rng.uniform(-5, 5, (200, 1)))
    codes, bits = ref.encode(x)
    want = np.abs(x).reshape(200, 4, 16).max(-1) / 6
    assert (np.abs(ref.SCALES[bits] - want) <= want / 16 + 1e-18).all()  # half of a step of 1/8
    off = np.abs(ref.decode(codes, bits) - x).reshape(200, 4, 16)
    # half a step of 2 at the top, and what the scale's rounding cuts off of the largest
    assert (off <= (want * 17 / 16 + want * 6 / 16)[..., None] + 1e-12).all()
    # a value that the format has comes back as itself
    again = ref.encode(ref.decode(codes, bits))
    back = ref.decode(*again)
    full = np.isclose(np.abs(ref.decode(codes, bits)).reshape(200, 4, 16).max(-1), 6 * ref.SCALES[bits])
    assert np.allclose(back.reshape(200, 4, 16)[full], ref.decode(codes, bits).reshape(200, 4, 16)[full])


def test_reference_not_a_number_infinity_and_zero():
    x = np.zeros((4, 16))
    x[0] = np.nan
    x[1, 0], x[1, 1] = np.inf, 1.0
    x[2, 3], x[2, 4] = np.nan, 6.0
    codes, bits = ref.encode(x)
    y = ref.decode(codes, bits)
    assert (y[0] == 0).all() and y[1, 0] == 6 * 2 ** 13 and y[1, 1] == 0 and y[2, 3] == 0 and y[2, 4] == 6 and (y[3] == 0).all()


def test_reference_rows_find_their_place():
    rng = np.random.default_rng(1)
    data = np.zeros((5, 2, 2, 18 * 64), np.uint8)
    pages = np.array([[3, 1], [4, -1]])
    k, v = rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64))
    ref.write(data, pages, [37, 3], [0, 37, 40], k, v)
    for b, n, at in ((0, 37, 0), (1, 3, 37)):
        for h in range(2):
            kk, vv = ref.sequence(data, pages, b, h, n)
            assert np.array_equal(kk, ref.decode(*ref.encode(k[at:at + n, h]))) and np.array_equal(vv, ref.decode(*ref.encode(v[at:at + n, h])))
    assert not data[0].any() and not data[2].any() and not data[1, :, 1].any()


def test_reference_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((7, 8)), rng.standard_normal((7, 8))
    p, o, lse = ref.attend_head(np.zeros((2, 8)), k, v, 0.5)  # equal scores: means over what is seen
    assert np.allclose(o, [v[:6].mean(0), v.mean(0)]) and np.allclose(lse, np.log([6, 7]))
    assert np.allclose(p.sum(1), 1) and p[0, 6] == 0
    k[2] = np.nan
    v[2] = np.nan  # a slot that is not there
    rest = [0, 1, 3, 4, 5, 6]
    q = rng.standard_normal((1, 8))
    p, o, lse = ref.attend_head(q, k, v, 0.5)
    want = ref.attend_head(q, k[rest], v[rest], 0.5)
    assert np.allclose(o, want[1]) and np.allclose(lse, want[2]) and p[0, 2] == 0
    p, o, lse = ref.attend_head(rng.standard_normal((3, 8)), k[:1], v[:1], 0.5)  # more queries than slots
    assert (o[:2] == 0).all() and (lse[:2] == -np.inf).all() and np.allclose(o[2], v[0])


def test_reference_eviction_by_hand():
    w, pos = [5.0, 1.0, 3.0, 3.0, 0.0, 2.0], [0, 9, 1, 2, 8, 3]
    assert ref.keep_order(w, pos, 2) == [1, 4, 0, 2, 3, 5]  # positions 9 and 8 first
    assert ref.evict_moves(w, pos, 3, 2) == [(4, 2)]
    assert ref.keep_order([1.0, math.nan, -math.inf, 1.0], [0, 1, 2, 3], 0) == [0, 3, 2, 1]
    assert ref.evict_moves(w, pos, 6, 2) == [] and ref.evict_moves(w, pos, 9, 2) == []
    assert ref.evict_moves([0, 0, 0, 0], [0, 1, 2, 3], 2, 3) == [(2, 0)]  # more recent ones than slots: the lower of them


# ---------------------------------------------------------------- refusals
def cache(**change):
    """A descriptor that passes every check (its pointers are never followed on the host)."""
    c = zl.zl_kv4_cache(2, 2, 64, 16, 4, 9, 0x1000, 0x2000, 0x3000, 0x4000)
    for k, v in change.items():
        setattr(c, k, v)
    return c


BAD_CACHES = [(dict(head_dim=96), zl.ZL_ERR_UNSUPPORTED), (dict(page=48), zl.ZL_ERR_UNSUPPORTED), (dict(page=0), zl.ZL_ERR_UNSUPPORTED),
              (dict(n_seqs=-1), zl.ZL_ERR_INVALID_ARG), (dict(n_kv_heads=0), zl.ZL_ERR_INVALID_ARG),
              (dict(n_kv_heads=1025), zl.ZL_ERR_INVALID_ARG), (dict(max_pages=-1), zl.ZL_ERR_INVALID_ARG),
              (dict(max_pages=1 << 27), zl.ZL_ERR_INVALID_ARG), (dict(max_pages=1 << 25, n_kv_heads=64), zl.ZL_ERR_INVALID_ARG), (dict(n_pages=-1), zl.ZL_ERR_INVALID_ARG),
              (dict(n_pages=1 << 31), zl.ZL_ERR_INVALID_ARG), (dict(data=0), zl.ZL_ERR_INVALID_ARG),
              (dict(pages=0), zl.ZL_ERR_INVALID_ARG), (dict(lens=0), zl.ZL_ERR_INVALID_ARG), (dict(data=0x1008), zl.ZL_ERR_ALIGN),
              (dict(pages=0x2002), zl.ZL_ERR_ALIGN), (dict(lens=0x3001), zl.ZL_ERR_ALIGN), (dict(status=0x4002), zl.ZL_ERR_ALIGN)]


def write(lib, c, k=0x10000, ks=128, v=0x20000, vs=128, n=2, starts=0x30000, pos=None, slots=None):
    return lib.zl_kv4_write(c, k, ks, v, vs, n, starts, pos, slots, None)


def read(lib, c, k=0x10000, ks=128, v=0x20000, vs=128, n=2, rows=0x30000):
    return lib.zl_kv4_read(c, k, ks, v, vs, n, rows, None)


def attend(lib, c, q=0x10000, qs=256, n=2, hq=4, starts=0x30000, most=1, o=0x40000, lse=0x50000, w=None, wo=None, decay=1.0,
           ws=0x60000, scale=0.5):
    return lib.zl_kv4_attn_fwd(c, q, qs, n, hq, starts, most, o, lse, w, wo, decay, ws, scale, None)


def evict(lib, c, w=0x10000, pos=0x20000, keep=4, recent=1, wo=0x10000, po=0x20000, ws=0x30000):
    return lib.zl_kv4_evict(c, w, pos, keep, recent, wo, po, ws, None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, status):
    c, b = cache(**change), ctypes.c_int64()
    for got in (write(lib, c), read(lib, c), attend(lib, c), evict(lib, c), lib.zl_kv4_attn_workspace(c, 4, 1, 0, ctypes.byref(b)),
                lib.zl_kv4_evict_workspace(c, ctypes.byref(b))):
        assert got == status


def test_every_call_refuses_no_cache(lib):
    assert write(lib, None) == read(lib, None) == attend(lib, None) == evict(lib, None) == zl.ZL_ERR_INVALID_ARG


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), zl.ZL_ERR_INVALID_ARG), (dict(n=1 << 31), zl.ZL_ERR_INVALID_ARG), (dict(k=None), zl.ZL_ERR_INVALID_ARG),
    (dict(v=None), zl.ZL_ERR_INVALID_ARG), (dict(ks=120), zl.ZL_ERR_INVALID_ARG), (dict(vs=132), zl.ZL_ERR_ALIGN),
    (dict(k=0x10008), zl.ZL_ERR_ALIGN), (dict(starts=0x30002), zl.ZL_ERR_ALIGN), (dict(starts=None, n=3), zl.ZL_ERR_INVALID_ARG),
    (dict(pos=0x50000), zl.ZL_ERR_INVALID_ARG), (dict(slots=0x50000), zl.ZL_ERR_INVALID_ARG),
    (dict(pos=0x50002, slots=0x60000), zl.ZL_ERR_ALIGN)])
def test_write_refusals(lib, change, status):
    assert write(lib, cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), zl.ZL_ERR_INVALID_ARG), (dict(k=None), zl.ZL_ERR_INVALID_ARG), (dict(vs=64), zl.ZL_ERR_INVALID_ARG),
    (dict(ks=129), zl.ZL_ERR_ALIGN), (dict(v=0x20004), zl.ZL_ERR_ALIGN), (dict(rows=None), zl.ZL_ERR_INVALID_ARG),
    (dict(rows=0x30004), zl.ZL_ERR_ALIGN)])
def test_read_refusals(lib, change, status):
    assert read(lib, cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(hq=3), zl.ZL_ERR_INVALID_ARG), (dict(hq=0), zl.ZL_ERR_INVALID_ARG), (dict(hq=258), zl.ZL_ERR_UNSUPPORTED),
    (dict(most=0), zl.ZL_ERR_INVALID_ARG), (dict(most=4097), zl.ZL_ERR_UNSUPPORTED), (dict(n=-1), zl.ZL_ERR_INVALID_ARG),
    (dict(starts=None, n=1), zl.ZL_ERR_INVALID_ARG), (dict(scale=0.0), zl.ZL_ERR_INVALID_ARG), (dict(scale=-1.0), zl.ZL_ERR_INVALID_ARG),
    (dict(scale=math.nan), zl.ZL_ERR_INVALID_ARG), (dict(scale=math.inf), zl.ZL_ERR_INVALID_ARG), (dict(decay=math.inf), zl.ZL_ERR_INVALID_ARG),
    (dict(w=0x70000), zl.ZL_ERR_INVALID_ARG), (dict(q=None), zl.ZL_ERR_INVALID_ARG), (dict(qs=248), zl.ZL_ERR_INVALID_ARG),
    (dict(qs=260), zl.ZL_ERR_ALIGN), (dict(o=None), zl.ZL_ERR_INVALID_ARG), (dict(lse=None), zl.ZL_ERR_INVALID_ARG),
    (dict(o=0x40008), zl.ZL_ERR_ALIGN), (dict(lse=0x50002), zl.ZL_ERR_ALIGN), (dict(ws=None), zl.ZL_ERR_INVALID_ARG),
    (dict(ws=0x60008), zl.ZL_ERR_ALIGN), (dict(wo=0x70002), zl.ZL_ERR_ALIGN)])
def test_attention_refusals(lib, change, status):
    assert attend(lib, cache(), **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(keep=0), zl.ZL_ERR_INVALID_ARG), (dict(recent=-1), zl.ZL_ERR_INVALID_ARG), (dict(w=None), zl.ZL_ERR_INVALID_ARG),
    (dict(pos=None), zl.ZL_ERR_INVALID_ARG), (dict(wo=None), zl.ZL_ERR_INVALID_ARG), (dict(po=None), zl.ZL_ERR_INVALID_ARG),
    (dict(ws=None), zl.ZL_ERR_INVALID_ARG), (dict(w=0x10002), zl.ZL_ERR_ALIGN), (dict(ws=0x30008), zl.ZL_ERR_ALIGN)])
def test_evict_refusals(lib, change, status):
    assert evict(lib, cache(), **change) == status


def test_calls_without_work_return_at_once(lib):
    none = cache(n_seqs=0, pages=0, lens=0, data=0)
    assert write(lib, none, n=0, starts=None) == read(lib, none) == attend(lib, none, n=0, starts=None) == evict(lib, none) == zl.ZL_OK
    assert write(lib, cache(), n=0, k=None, v=None) == read(lib, cache(), n=0, k=None, v=None) == zl.ZL_OK
    assert attend(lib, cache(), n=0, q=None, o=None, lse=None, ws=None) == zl.ZL_OK


def test_workspace_sizes(lib):
    b = ctypes.c_int64()
    assert lib.zl_kv4_attn_workspace(cache(), 4, 1, 0, None) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_kv4_attn_workspace(cache(), 4, 1, 2, ctypes.byref(b)) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_kv4_attn_workspace(cache(), 4, 1, 0, ctypes.byref(b)) == zl.ZL_OK
    base = b.value
    assert base > 0 and base % 16 == 0
    assert lib.zl_kv4_attn_workspace(cache(), 4, 1, 1, ctypes.byref(b)) == zl.ZL_OK
    assert b.value == base + 2 * 2 * 64 * 2 * 4  # two rows a key head, every slot of the table
    assert lib.zl_kv4_evict_workspace(cache(), ctypes.byref(b)) == zl.ZL_OK and b.value >= 2 * 2 * 64 * 4
    assert lib.zl_kv4_evict_workspace(cache(), None) == zl.ZL_ERR_INVALID_ARG


def test_binding_takes_cuda_tensors_alone():
    import torch
    with pytest.raises(TypeError):
        zl.Kv4Cache(torch.zeros(1, 1, 1, 18 * 64, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        zl.allocate_kv4(1, 1, 1, 64, page=48, device="cpu")
    with pytest.raises(ValueError):
        zl.allocate_kv4(1, 1, 1, 96, device="cpu")
