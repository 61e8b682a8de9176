"""Causal sequences without a GPU: the reference's own pins (closed forms, finite differences, the limit
cases), the planner's schedule, the frequencies, and the refusals of every entry point."""
import ctypes
import math
import random

import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import causal as ref
from tests._lib import ensure_library


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


# ---------------------------------------------------------------- the reference
def test_reference_attention_closed_forms():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    o, lse = ref.attend(q, k, v, [(0, 5, 0, 5)], 0.3)
    assert np.allclose(o[0], v[0], atol=1e-15)  # the first query sees the first key alone
    assert np.allclose(lse[0], 0.3 * q[0] @ k[0, 0], atol=1e-15)
    o0, lse0 = ref.attend(0 * q, k, v, [(0, 5, 0, 5)], 0.3)  # equal scores: means over the prefix
    for i in range(5):
        assert np.allclose(o0[i], v[:i + 1, 0].mean(0), atol=1e-14) and np.allclose(lse0[i], math.log(i + 1), atol=1e-14)
    # a later key changes nothing before it
    k2, v2 = k.copy(), v.copy()
    k2[4], v2[4] = 9.0, -9.0
    assert np.array_equal(ref.attend(q, k2, v2, [(0, 5, 0, 5)], 0.3)[0][:4], o[:4])
    # the last rows of a longer sequence are its chunk behind the keys already there
    oc, lc = ref.attend(q[3:], k, v, [(0, 2, 0, 5)], 0.3)
    assert np.allclose(oc, o[3:], atol=1e-15) and np.allclose(lc, lse[3:], atol=1e-15)
    oe, le = ref.attend(q, k[:2], v[:2], [(0, 5, 0, 2)], 0.3)  # more queries than keys
    assert (oe[:3] == 0).all() and (le[:3] == -np.inf).all() and np.isfinite(le[3:]).all()


@pytest.mark.parametrize("seqs", [[(0, 4, 0, 4), (4, 1, 4, 3)], [(0, 5, 0, 3), (5, 2, 3, 6)]])
def test_reference_gradient_against_differences(seqs):
    rng = np.random.default_rng(1)
    tq, tk = max(s[0] + s[1] for s in seqs), max(s[2] + s[3] for s in seqs)
    x = [rng.standard_normal((tq, 4, 6)), rng.standard_normal((tk, 2, 6)), rng.standard_normal((tk, 2, 6))]
    g = rng.standard_normal((tq, 4, 6))
    grads = ref.attend_grad(*x, g, seqs, 0.4)
    for i in range(3):
        for _ in range(12):
            at = tuple(rng.integers(0, s) for s in x[i].shape)
            step = []
            for e in (1e-6, -1e-6):
                y = [a.copy() for a in x]
                y[i][at] += e
                step.append(np.sum(g * ref.attend(*y, seqs, 0.4)[0]))
            assert abs((step[0] - step[1]) / 2e-6 - grads[i][at]) < 1e-7


@pytest.mark.parametrize("half", [True, False])
def test_reference_rotation_and_norm(half):
    rng = np.random.default_rng(2)
    pos = rng.integers(-50, 50, (6, 2))
    ang = ref.angles(pos, [1.0, 0.3, 0.05], [2, 1])
    assert ang[4, 1] == pos[4, 0] * 0.3 and ang[4, 2] == pos[4, 1] * 0.05
    x, g, w = rng.standard_normal((6, 3, 10)), rng.standard_normal((6, 3, 10)), rng.standard_normal(10)
    y = ref.rotate(x, ang, half)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1)) and np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(ref.rotate(y, -ang, half), x)  # the transpose is the inverse
    # scores of rotated rows depend on the distance alone
    p = ref.angles(pos + 7, [1.0, 0.3, 0.05], [2, 1])
    far = ref.rotate(x, p, half)
    assert np.allclose((y[0] * y[5]).sum(-1), (far[0] * far[5]).sum(-1))
    dx, dw = ref.rms_norm_grad(x, w, 0.01, g)
    for _ in range(10):
        at = tuple(rng.integers(0, s) for s in x.shape)
        d = np.zeros_like(x)
        d[at] = 1e-6
        num = np.sum(g * (ref.rms_norm(x + d, w, 0.01) - ref.rms_norm(x - d, w, 0.01))) / 2e-6
        assert abs(num - dx[at]) < 1e-7
        e = np.zeros(10)
        e[at[2]] = 1e-6
        num = np.sum(g * (ref.rms_norm(x, w + e, 0.01) - ref.rms_norm(x, w - e, 0.01))) / 2e-6
        assert abs(num - dw[at[2]]) < 1e-6


# ---------------------------------------------------------------- frequencies
def test_fixed_point_frequencies_give_the_angle_at_any_position():
    freqs, _ = zl.rotary_frequencies(128)
    out = (ctypes.c_uint64 * 64)()
    assert zl.load_library().zl_rope_frequencies((ctypes.c_double * 64)(*freqs), 64, out) == zl.ZL_OK
    for t in (0, 1, -1, 4097, -131071, 2 ** 31 - 1, -2 ** 31):
        for f, x in zip(freqs, out):
            turn = (t * x % 2 ** 64) / 2.0 ** 64  # what the kernel forms, before its top 32 bits
            # 53 bits of the frequency times the position, plus one step of 2^-64 a position
            assert abs(math.remainder(2 * math.pi * turn - math.remainder(t * f, 2 * math.pi), 2 * math.pi)) \
                < 2e-15 * (1 + abs(t * f)) + 1e-12


def test_frequencies_of_whole_turns_negative_and_bad_ones(lib):
    out = (ctypes.c_uint64 * 2)()
    assert lib.zl_rope_frequencies((ctypes.c_double * 2)(0.0, -math.pi), 2, out) == zl.ZL_OK
    assert out[0] == 0 and out[1] == 2 ** 63
    # a negative frequency too small for its fraction: 1 - tiny rounds to a whole turn, which is none
    assert lib.zl_rope_frequencies((ctypes.c_double * 1)(-1e-300), 1, out) == zl.ZL_OK and out[0] == 0
    for bad in (math.inf, math.nan):
        assert lib.zl_rope_frequencies((ctypes.c_double * 1)(bad), 1, out) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_rope_frequencies(None, 1, out) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_rope_frequencies(None, 0, None) == zl.ZL_OK


def test_scaled_frequencies():
    plain, one = zl.rotary_frequencies(64, 10000.0)
    assert one == 1.0 and plain[0] == 1.0 and plain[1] == 10000.0 ** (-2 / 64)
    linear, _ = zl.rotary_frequencies(64, scaling="linear", factor=8)
    assert linear == [f / 8 for f in plain]
    ntk, _ = zl.rotary_frequencies(64, scaling="ntk", factor=8)
    assert ntk[0] == 1.0 and abs(ntk[-1] / plain[-1] * 8 - 1) < 1e-12
    yarn, amp = zl.rotary_frequencies(64, scaling="yarn", factor=8, original_len=4096)
    assert amp == 0.1 * math.log(8) + 1 and yarn[0] == plain[0] and abs(yarn[-1] / plain[-1] * 8 - 1) < 1e-12
    assert all(f / 8 <= y <= f for f, y in zip(plain, yarn))
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(rot_dim=8, base=0.0), dict(rot_dim=8, scaling="other"),
                dict(rot_dim=8, scaling="yarn", factor=0.5), dict(rot_dim=8, scaling="yarn", slow=4, fast=4)):
        with pytest.raises(ValueError):
            zl.rotary_frequencies(**bad)


def test_rotary_table_checks_its_arguments():
    assert zl.rotary_table([1.0, 0.5], device="cpu").rot_dim == 4
    for bad in (dict(layout="other"), dict(axis_pairs=[1]), dict(axis_pairs=[3, -1]), dict(axis_pairs=[1, 1, 0, 0])):
        with pytest.raises(ValueError):
            zl.rotary_table([1.0, 0.5], device="cpu", **bad)
    with pytest.raises(zl.ZlError):
        zl.rotary_table([math.nan], device="cpu")


# ---------------------------------------------------------------- schedule
def _plan(seqs, hq, hk, d):
    return zl.zl_plan_causal(seqs, hq, hk, d, max([s[0] + s[1] for s in seqs] + [0]),
                             max([s[2] + s[3] for s in seqs] + [0]), zl.ZL_PLAN_HOST_ONLY)


def _check_schedule(seqs, hq, hk, d):
    plan, tb = _plan(seqs, hq, hk, d), 128 // (hq // hk)
    spans, parts = {}, set()
    for s, h, b, lo, hi, part, _ in plan.tiles(0):
        assert 0 <= lo <= hi
        if part >= 0:
            assert part not in parts
            parts.add(part)
        for w in (0, 1):
            spans.setdefault((s, h, b + w), []).append((lo, hi))
    for i, (_, n, _, m) in enumerate(seqs):
        for h in range(hk):
            for b in range(-(-n // tb)):
                seen = max(0, m - n + min(n, (b + 1) * tb))
                at = 0
                for lo, hi in sorted(spans[(i, h, b)]):  # every key block the rows see, once
                    assert lo == at
                    at = hi
                assert at >= -(-seen // 128)
    walks, slots = {}, []
    for s, h, b, lo, hi, part, _ in plan.tiles(1):
        walks.setdefault((s, h, b), []).append((lo, hi, part))
        slots += [part] if part >= 0 else []
    assert sorted(walks) == [(i, h, b) for i, s in enumerate(seqs) for h in range(hk) for b in range(-(-s[3] // 128))]
    for (i, _, b), w in walks.items():  # from the first query block that sees one of the keys to the last, once
        _, n, _, m = seqs[i]
        nqb = -(-n // tb)
        at = min(nqb, max(0, b * 128 - (m - n)) // tb)
        assert all((part >= 0) == (len(w) > 1) for _, _, part in w)
        for lo, hi, _ in sorted(w):
            assert lo == at
            at = hi
        assert at == nqb
    assert sorted(slots) == list(range(len(slots)))
    rows = plan.q_tokens * hq * 4
    assert plan.bwd_workspace_bytes == -(-rows // 256) * 256 + sum(-(-s[1] // tb) for s in seqs) * hk * 128 * d * 4 \
        + len(slots) * 2 * 128 * d * 4
    assert plan.fwd_workspace_bytes == len(parts) * 256 * (d + 1) * 4
    assert len(parts) == 0 or sorted(parts) == list(range(len(parts)))
    return plan


def test_schedule_covers_every_visible_block_once():
    rng = random.Random(1)
    for _ in range(150):
        hk, group = rng.choice([1, 2, 3]), rng.choice([1, 2, 3, 5, 7, 8, 24, 100, 128])
        seqs, q0, k0 = [], 0, 0
        for _ in range(rng.randint(0, 6)):
            n, m = rng.choice([0, 1, 2, 5, 127, 128, 129, 300]), rng.choice([0, 1, 3, 127, 128, 129, 500, 2900])
            seqs.append((q0, n, k0, m))
            q0, k0 = q0 + n + rng.randint(0, 3), k0 + m + rng.randint(0, 3)
        _check_schedule(seqs, hk * group, hk, rng.choice([64, 128]))


def test_long_key_ranges_of_few_rows_are_split_and_many_rows_are_not():
    one = _check_schedule([(0, 1, 0, 32760)], 32, 8, 128)
    assert one.fwd_workspace_bytes > 0 and len({t[6] for t in one.tiles(0)}) > 140
    assert _check_schedule(zl.causal_seqs([16384]), 32, 4, 128).fwd_workspace_bytes == 0
    assert _check_schedule(zl.causal_seqs([100, 64]), 4, 2, 64).fwd_workspace_bytes == 0
    assert any(t[5] >= 0 for t in _check_schedule(zl.causal_seqs([2048, 100]), 24, 8, 64).tiles(1))
    assert all(t[5] < 0 for t in _check_schedule(zl.causal_seqs([4096] * 30), 24, 8, 64).tiles(1))


def test_schedule_is_balanced():
    tiles = _plan(zl.causal_seqs([16384]), 32, 4, 128).tiles(0)
    load = {}
    for _, _, _, lo, hi, _, bin_ in tiles:
        load[bin_] = load.get(bin_, 0) + hi - lo
    assert len(load) == 152 and max(load.values()) < 1.05 * sum(load.values()) / 152


# ---------------------------------------------------------------- refusals
@pytest.mark.parametrize("seqs,heads,status", [
    ([(0, 5, 0, 5)], (4, 3, 64), zl.ZL_ERR_INVALID_ARG),       # heads not a multiple
    ([(0, 5, 0, 5)], (4, 0, 64), zl.ZL_ERR_INVALID_ARG),
    ([(0, 5, 0, 5)], (4, 4, 96), zl.ZL_ERR_UNSUPPORTED),
    ([(0, 5, 0, 5)], (129, 1, 64), zl.ZL_ERR_UNSUPPORTED),     # over 128 query heads a key head
    ([(0, 11, 0, 5)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),      # past the query rows
    ([(0, 5, 0, 11)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),      # past the key rows
    ([(6, 5, 0, 5)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),
    ([(2 ** 62, 5, 0, 5)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),
    ([(-1, 5, 0, 5)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),
    ([(0, -5, 0, 5)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),
    ([(0, 5, 0, 5), (4, 2, 5, 2)], (4, 2, 64), zl.ZL_ERR_INVALID_ARG),  # two sequences write row 4
])
def test_bad_sequences_are_refused(seqs, heads, status):
    with pytest.raises(zl.ZlError) as e:
        zl.zl_plan_causal(seqs, *heads, 10, 10, zl.ZL_PLAN_HOST_ONLY)
    assert e.value.status == status


def test_plan_limits(lib):
    for flags in (4, 8, 16, 64, 1 << 31):
        with pytest.raises(zl.ZlError):
            zl.zl_plan_causal([], 4, 2, 64, 0, 0, flags | zl.ZL_PLAN_HOST_ONLY)
    with pytest.raises(zl.ZlError) as e:  # coordinates of the tiles' loads are 32-bit
        zl.zl_plan_causal([], 4, 2, 64, 2 ** 31 - 100, 0, zl.ZL_PLAN_HOST_ONLY)
    assert e.value.status == zl.ZL_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        zl.zl_plan_causal([(0, 2 ** 31, 0, 1)], 4, 2, 64, 2 ** 31, 1, zl.ZL_PLAN_HOST_ONLY)
    empty = zl.zl_plan_causal([], 4, 2, 64, 0, 0, zl.ZL_PLAN_HOST_ONLY)
    assert empty.tiles(0) == [] and empty.tiles(1) == []
    n = ctypes.c_int64()
    assert lib.zl_causal_plan_tiles(empty.handle, 2, None, 0, ctypes.byref(n)) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_causal_plan_tiles(None, 0, None, 0, ctypes.byref(n)) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_causal_plan_workspace(None, None, None) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_plan_causal(None, 1, 4, 2, 64, 9, 9, 1, ctypes.byref(ctypes.c_void_p())) == zl.ZL_ERR_INVALID_ARG
    assert lib.zl_plan_causal(None, 0, 4, 2, 64, 9, 9, 1, None) == zl.ZL_ERR_INVALID_ARG
    lib.zl_causal_plan_destroy(None)


def test_launches_refuse_missing_and_host_only_plans(lib):
    plan = _plan([(0, 5, 0, 5)], 4, 2, 64)
    for h in (None, plan.handle):
        assert lib.zl_causal_attn_fwd(h, 16, 256, 16, 128, 16, 128, 16, 16, None, 0.1, None) == zl.ZL_ERR_INVALID_ARG
        assert lib.zl_causal_attn_bwd(h, 16, 256, 16, 128, 16, 128, 16, 16, 16, 16, 256, 16, 128, 16, 128, 16, 0.1,
                                      None) == zl.ZL_ERR_INVALID_ARG
        assert lib.zl_causal_get_device_status(h, None, ctypes.byref(ctypes.c_int32())) == zl.ZL_ERR_INVALID_ARG


def _desc(**kw):
    d = dict(n_tokens=3, n_q_heads=4, n_kv_heads=2, head_dim=64, norm=1, eps=1e-6, rot_dim=64, half_layout=1, n_axes=1,
             axis_pairs=(32, 0, 0), amplitude=1.0)
    d.update(kw)
    d["axis_pairs"] = (ctypes.c_int32 * 3)(*d["axis_pairs"])
    return zl.zl_qk_rope_desc(**d)


BAD_DESCS = [
    (dict(head_dim=96), zl.ZL_ERR_UNSUPPORTED), (dict(n_tokens=-1), zl.ZL_ERR_INVALID_ARG),
    (dict(n_q_heads=0, n_kv_heads=0), zl.ZL_ERR_INVALID_ARG), (dict(n_q_heads=-4), zl.ZL_ERR_INVALID_ARG),
    (dict(norm=2), zl.ZL_ERR_INVALID_ARG), (dict(eps=-1.0), zl.ZL_ERR_INVALID_ARG), (dict(eps=math.nan), zl.ZL_ERR_INVALID_ARG),
    (dict(rot_dim=66, axis_pairs=(33, 0, 0)), zl.ZL_ERR_INVALID_ARG),
    (dict(rot_dim=24, axis_pairs=(12, 0, 0)), zl.ZL_ERR_INVALID_ARG),   # half layout: not a multiple of 16
    (dict(rot_dim=7, half_layout=0, axis_pairs=(3, 0, 0)), zl.ZL_ERR_INVALID_ARG),
    (dict(half_layout=2), zl.ZL_ERR_INVALID_ARG), (dict(n_axes=0), zl.ZL_ERR_INVALID_ARG), (dict(n_axes=4), zl.ZL_ERR_INVALID_ARG),
    (dict(axis_pairs=(31, 0, 0)), zl.ZL_ERR_INVALID_ARG), (dict(n_axes=2, axis_pairs=(33, -1, 0)), zl.ZL_ERR_INVALID_ARG),
    (dict(amplitude=math.inf), zl.ZL_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,status", BAD_DESCS)
def test_bad_rope_descriptors_are_refused(lib, kw, status):
    d = ctypes.byref(_desc(**kw))
    n = ctypes.c_int64()
    assert lib.zl_qk_rope_workspace(d, ctypes.byref(n)) == status
    assert lib.zl_qk_rope_fwd(d, 16, 256, 16, 128, None, None, 16, 16, 16, 256, 16, 128, None) == status
    assert lib.zl_qk_rope_bwd(d, 16, 256, 16, 128, None, None, 16, 16, 16, 256, 16, 128, 16, 256, 16, 128, None, None, None,
                              None) == status


def test_bad_rope_pointers_are_refused_before_any_launch(lib):
    good = [16, 256, 16, 128, 16, 16, 16, 16, 16, 256, 16, 128, None]
    d = _desc()

    def fwd(**kw):
        a = list(good)
        for i, x in kw.items():
            a[int(i[1:])] = x
        return lib.zl_qk_rope_fwd(ctypes.byref(d), *a)

    inv, al = zl.ZL_ERR_INVALID_ARG, zl.ZL_ERR_ALIGN
    assert lib.zl_qk_rope_fwd(None, *good) == inv
    for i in ("_0", "_2", "_6", "_7", "_8", "_10"):  # q, k, positions, frequencies, outputs
        assert fwd(**{i: None}) == inv
    for i in ("_1", "_3", "_9", "_11"):
        assert fwd(**{i: 64}) == inv  # a stride below heads * d
        assert fwd(**{i: 1001}) == al
    for i in ("_0", "_2", "_8", "_10"):
        assert fwd(**{i: 24}) == al
    d = _desc(norm=0)
    assert fwd() == inv  # weights without norm
    d = _desc()
    bwd = [16, 256, 16, 128, 16, 16, 16, 16, 16, 256, 16, 128, 16, 256, 16, 128, 16, 16, 16, None]

    def back(i, x):
        a = list(bwd)
        a[i] = x
        return lib.zl_qk_rope_bwd(ctypes.byref(d), *a)

    for i in (0, 2, 4, 5, 6, 7, 8, 10, 12, 14, 18):  # 4, 5: a weight's gradient without the weight
        assert back(i, None) == inv
    for i in (0, 2, 8, 10, 12, 14, 18):
        assert back(i, 24) == al
    for i in (9, 11):  # an output on its input at another stride (backward 13, 15: on its gradient)
        assert fwd(**{f"_{i}": 512}) == inv and back(i + 4, 512) == inv
    # no tokens: nothing to do, whatever the pointers
    d = _desc(n_tokens=0)
    assert lib.zl_qk_rope_fwd(ctypes.byref(d), None, 0, None, 0, None, None, None, None, None, 0, None, 0, None) == zl.ZL_OK


def test_a_rotary_table_is_not_changed_but_replaced():
    import dataclasses
    table = zl.rotary_table([1.0, 0.5], "interleaved", device="cpu")
    with pytest.raises(dataclasses.FrozenInstanceError):
        table.amplitude = 2.0
    table.last[0] = ("key", "descriptor")
    other = dataclasses.replace(table, amplitude=2.0, freq=table.freq.clone())
    assert other.last == [(None, None)] and other.ptr == other.freq.data_ptr() != table.ptr and other.axis_pairs == (2,)


def test_host_tensors_are_refused():
    import torch
    x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((TypeError, AssertionError, RuntimeError)):
        zl.zl_qk_rope_fwd(x, None, x, None, None, None)
    plan = _plan([(0, 3, 0, 3)], 4, 4, 64)
    with pytest.raises(TypeError):
        zl.zl_causal_attn_fwd(plan, x, x, x, x, torch.zeros(3, 4), torch.zeros(16, dtype=torch.uint8), 0.1)


def test_forward_only_plans_have_no_backward():
    seqs = [(0, 1, 0, 5000), (1, 3, 5000, 900)]
    both, fwd = (zl.zl_plan_causal(seqs, 8, 2, 128, 4, 5900, zl.ZL_PLAN_HOST_ONLY | f) for f in (0, zl.ZL_PLAN_FORWARD_ONLY))
    assert fwd.tiles(0) == both.tiles(0) and fwd.fwd_workspace_bytes == both.fwd_workspace_bytes
    assert fwd.tiles(1) == [] and fwd.bwd_workspace_bytes == 0 and len(both.tiles(1)) > 0


def test_row_masks_of_ranges():
    assert zl._row_mask([(2, 3), (0, 0), (7, 1), (4, 2)], 9).tolist() == [0, 0, 1, 1, 1, 1, 0, 1, 0]
    assert zl._row_mask([], 2).tolist() == [0, 0]


def test_norm_is_of_the_sides_that_have_a_weight():
    assert zl._sides(None, None) == ((True, True, False),) and zl._sides(1, 2) == ((True, True, True),)
    assert zl._sides(1, None) == ((True, False, True), (False, True, False))
    assert zl._sides(None, 1) == ((True, False, False), (False, True, True))


def test_a_rotary_table_holds_a_number_for_every_pair():
    """The kernels read rot_dim / 2 of them: a table whose tensor is shorter, or of another type or layout, is refused."""
    import dataclasses
    import torch
    table = zl.rotary_table([1.0, 0.5, 0.25, 0.125], "interleaved", device="cpu")
    for bad in (dict(rot_dim=16), dict(rot_dim=16, axis_pairs=(8,)), dict(freq=table.freq[:3]),
                dict(freq=torch.arange(8)[::2]), dict(freq=table.freq.int()), dict(freq=table.freq.double()),
                dict(freq=[1, 2, 3, 4]), dict(freq=None)):
        with pytest.raises((TypeError, ValueError)):
            dataclasses.replace(table, **bad)
    assert dataclasses.replace(table, axis_pairs=(2, 2)).axis_pairs == (2, 2)
    assert dataclasses.replace(table, rot_dim=4, axis_pairs=(2,)).rot_dim == 4  # its first pairs alone


def test_rope_numbers_off_their_alignment_are_refused(lib):
    """Weights, positions and frequencies are read number by number: a pointer off their type's alignment would fault."""
    d = ctypes.byref(_desc())
    fwd = [16, 256, 16, 128, 16, 16, 16, 16, 16, 256, 16, 128, None]
    bwd = [16, 256, 16, 128, 16, 16, 16, 16, 16, 256, 16, 128, 16, 256, 16, 128, 16, 16, 16, None]
    for i, off in ((4, 18), (5, 17), (6, 18), (7, 20)):  # weights, positions, frequencies
        for fn, args in ((lib.zl_qk_rope_fwd, fwd), (lib.zl_qk_rope_bwd, bwd)):
            assert fn(d, *args[:i], off, *args[i + 1:]) == zl.ZL_ERR_ALIGN
    for i in (16, 17):  # weights' gradients
        assert lib.zl_qk_rope_bwd(d, *bwd[:i], 18, *bwd[i + 1:]) == zl.ZL_ERR_ALIGN


def test_yarn_ramps_over_the_pairs():
    """As released checkpoints do.  128 channels, base 10 000, 4096 positions: 128 ln(4096 / (2 pi 32)) / (2 ln 10 000) = 20.9,
    with 1 for 32 turns 45.03: pairs to 20 kept, from 46 on divided, 1 / 26 a pair between."""
    plain, _ = zl.rotary_frequencies(128)
    yarn, amp = zl.rotary_frequencies(128, scaling="yarn", factor=16.0, original_len=4096)
    assert abs(amp - 1.2772588722239782) < 1e-15
    kept = [(y / f - 1 / 16) / (15 / 16) for f, y in zip(plain, yarn)]
    assert all(abs(k - 1) < 1e-12 for k in kept[:21]) and all(abs(k) < 1e-12 for k in kept[46:])
    assert all(abs(kept[20 + i] - (1 - i / 26)) < 1e-12 for i in range(27))
    # 64 channels, base 500 000, 8192 positions, factor 8: pairs 9.04 -> 9 to 17.50 -> 18
    plain, _ = zl.rotary_frequencies(64, base=500000.0)
    yarn, _ = zl.rotary_frequencies(64, base=500000.0, scaling="yarn", factor=8.0, original_len=8192)
    kept = [(y / f - 1 / 8) / (7 / 8) for f, y in zip(plain, yarn)]
    assert abs(kept[9] - 1) < 1e-12 and abs(kept[10] - 8 / 9) < 1e-12 and abs(kept[17] - 1 / 9) < 1e-12 and abs(kept[18]) < 1e-12
    # a context so short that the first pair already turns too seldom: divided from pair 0 (or 1) on, nothing negative
    yarn, _ = zl.rotary_frequencies(16, scaling="yarn", factor=2.0, original_len=4)
    assert all(abs(y * 2 / f - 1) < 1e-12 for f, y in list(zip(zl.rotary_frequencies(16)[0], yarn))[1:])
    # no pair turns 0 times: the ramp ends past the last pair, at 127 (the channels less one)
    open_end, _ = zl.rotary_frequencies(128, scaling="yarn", factor=16.0, original_len=4096, slow=0.0)
    plain, _ = zl.rotary_frequencies(128)
    assert abs((open_end[63] / plain[63] - 1 / 16) / (15 / 16) - (1 - 43 / 107)) < 1e-12
    for bad in (dict(base=1.0), dict(slow=-2.0, fast=-1.0)):
        with pytest.raises(ValueError):
            zl.rotary_frequencies(16, scaling="yarn", **bad)
