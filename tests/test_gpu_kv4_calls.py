"""The 4-bit cache on the GPU: calls that the documentation allows, one after another, at once and with state that goes on."""
import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import kv4 as ref
from tests._lib import ensure_library
from tests.test_gpu_kv4 import F, f64, make_cache, many, reference, run_attention, starts_of, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


@pytest.mark.parametrize("d,page,lens,weights", [(128, 16, [33, 500, 1, 130], False), (64, 64, [200] * 24, True), (128, 256, [250] * 200, False)])
def test_short_calls_one_after_another(d, page, lens, weights):
    """Clusters of every size, launch behind launch, each with outputs of its own: every one of them the first one's."""
    import torch
    c, data, pages = make_cache(lens, 2, d, page, 70)
    n, times = len(lens), 200
    want = run_attention(c, data, pages, lens, [1] * n, 4, 71, no_starts=True)
    q = torch.randn(n, 8, d, generator=torch.Generator().manual_seed(71)).bfloat16().cuda()[:, 4:]
    o, lse = torch.full((times, n, 4, d), 7.0, dtype=torch.bfloat16).cuda(), torch.full((times, n, 4), 7.0).cuda()
    w = torch.zeros((times, *c.slot_shape)).cuda() if weights else [None] * times
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 4, 1, weights), dtype=torch.uint8).cuda()
    for i in range(times):
        zl.zl_kv4_attn_fwd(c, q, o[i], lse[i], ws, d ** -0.5, weights_out=w[i])
    assert zl.zl_kv4_get_device_status(c) == 0
    first = (o[0], lse[0]) if weights else want
    assert all(torch.equal(x, first[0]) for x in o) and all(torch.equal(x, first[1]) for x in lse)
    assert not weights or all(torch.equal(x, w[0]) for x in w)


# ---------------------------------------------------------------- what P in fp16 holds
def one_hot_cache(scores, v, d, page, table=0):
    """A sequence of one head whose slot s has the key scores[s] e0 (held exactly) and the value v[s] in every channel."""
    import torch
    n = len(scores)
    c = zl.allocate_kv4(1, max(-(-n // page), table), 1, d, page=page)
    k, x = np.zeros((n, 1, d)), np.repeat(np.asarray(v, float)[:, None, None], d, 2)
    k[:, 0, 0] = scores
    c.lens.fill_(n)
    zl.zl_kv4_write(c, torch.from_numpy(k).bfloat16().cuda(), torch.from_numpy(x).bfloat16().cuda(), torch.tensor([0, n], dtype=torch.int32).cuda())
    data, pages = c.data.cpu().numpy(), c.pages.cpu().numpy()
    kk, vv = ref.sequence(data, pages, 0, 0, n)
    assert np.array_equal(kk, k[:, 0]) and np.array_equal(vv, x[:, 0])
    return c, data, pages


def attend_one_hot(c, rows, n_new, scale, size=1.0):
    """n_new tokens of rows / n_new heads whose queries are size e0."""
    import torch
    d, hq = c.token_shape[1], rows // n_new
    q = torch.zeros(n_new, hq, d)
    q[..., 0] = size
    q = q.bfloat16().cuda()
    o, lse = torch.empty_like(q), torch.empty(n_new, hq).cuda()
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, hq, n_new), dtype=torch.uint8).cuda()
    zl.zl_kv4_attn_fwd(c, q, o, lse, ws, scale, torch.tensor([0, n_new], dtype=torch.int32).cuda(), n_new)
    assert zl.zl_kv4_get_device_status(c) == 0
    return f64(q), f64(o), f64(lse)


# rows, new tokens, slots of the table: by clusters, dealt out, by the kernel for many rows
FORMS = [(1, 1, 0), (12, 1, 0), (4, 1, 20000), (40, 1, 160000), (96, 3, 70000)]


@pytest.mark.parametrize("rows,new,table", FORMS)
@pytest.mark.parametrize("d", [64, 128])
def test_far_smaller_weights_add_up(rows, new, table, d):
    """31 weights of 2^-25.5 for each of the largest, whose value is 0.  The bound is that of test_gpu_kv4.py, with half a step of
    fp16's smallest numbers at 2^-32 of the row's maximum; scores' products are exact but for their last factor's rounding."""
    n, below = 8192, 25.5
    scores, v = np.zeros(n), np.full(n, 3.0)
    scores[::32], v[::32] = 12.0, 0.0
    c, data, pages = one_hot_cache(scores, v, d, 256, -(-table // 256))
    scale = below * np.log(2) / 12
    q, o, lse = attend_one_hot(c, rows, new, scale)
    k, vv = ref.sequence(data, pages, 0, 0, n)
    for h in range(rows // new):
        p, want, wl = ref.attend_head(q[:, h], k, vv, scale)
        es = scale * 12 * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * es + 2.0 ** -20 + 2.0 ** -22 * below + n * F) * (p @ np.abs(vv)) + \
            2.0 ** -32 * 3.0 * n * p.max(1, keepdims=True)
        assert (np.abs(o[:, h] - want) <= tol).all(), (o[0, 0, 0], want[0, 0])
        assert np.abs(lse[:, h] - wl).max() <= 2 * es + 2.0 ** -20 * (1 + np.abs(wl).max()) + n * F


@pytest.mark.parametrize("rows,new,table", FORMS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("step", [0.5, 1.0, 1.8, 3.0])
def test_scores_that_rise_slowly(rows, new, table, d, step):
    n = 4096
    scores = 0.75 * (8 + np.arange(n) // 96 % 9)  # nine levels, `step` apart to base 2
    v = np.random.default_rng(3).choice([0.0, 0.75, 1.5, 3, 6, 12], n)
    c, data, pages = one_hot_cache(scores, v, d, 256, -(-table // 256))
    scale = step * np.log(2) / 0.75
    q, o, lse = attend_one_hot(c, rows, new, scale)
    k, vv = ref.sequence(data, pages, 0, 0, n)
    for h in range(rows // new):
        p, want, wl = ref.attend_head(q[:, h], k, vv, scale)
        es = scale * 12 * 2.0 ** -22
        tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * es + 2.0 ** -20 + 2.0 ** -22 * 12 * scale + n * F) * (p @ np.abs(vv)) + 2.0 ** -32 * 6 * n
        assert (np.abs(o[:, h] - want) <= tol).all()
        assert np.abs(lse[:, h] - wl).max() <= 2 * es + 2.0 ** -20 * (1 + np.abs(wl).max()) + n * F


@pytest.mark.parametrize("rows,new,table", FORMS)
@pytest.mark.parametrize("power", [12, 17, 20, 21, 22, 24, 26, 27])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(rows, new, table, power, sign):
    """Two equal scores that leave the others nothing: their values' mean, exactly."""
    n = 700
    scores, v = np.full(n, 2.25 * sign), np.full(n, 6.0)
    scores[[3, 650]] = 3.0 if sign > 0 else -1.5
    v[[3, 650]] = 0.75, 2.25
    c, data, pages = one_hot_cache(scores, v, 64, 64, -(-table // 64))
    q, o, lse = attend_one_hot(c, rows, new, 0.3, 2.0 ** power)
    top = 2.0 ** power * 0.3 * (3.0 if sign > 0 else -1.5)
    assert (o == 1.5).all() and (np.abs(lse / top - 1) < 2.0 ** -20 + 1 / abs(top)).all()
