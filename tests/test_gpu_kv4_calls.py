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


@pytest.mark.parametrize("d,page,lens,weights", [
    (128, 16, [33, 500, 1, 130], False), (64, 64, [200] * 24, True), (128, 256, [250] * 200, False)])
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
    zl.zl_kv4_write(c, torch.from_numpy(k).bfloat16().cuda(), torch.from_numpy(x).bfloat16().cuda(),
                    torch.tensor([0, n], dtype=torch.int32).cuda())
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
        tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -32 * 12 * n + \
            (2.0 ** -11 + 2 * es + 2.0 ** -20 + 2.0 ** -22 * 12 * scale + n * F) * (p @ np.abs(vv))
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


# ---------------------------------------------------------------- state that goes on from call to call
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_a_prompt_without_keep_then_steps_on_a_budget(shared, graph):
    """Prompts in several calls, steps on a budget behind them, and a row that becomes another sequence's: what eviction goes by
    comes from the calls alone."""
    import torch
    heads, hq, d, keep, recent = 2, 4, 64, 24, 8
    c = zl.allocate_kv4(2, 4, heads, d, page=16)
    step = zl.allocate_kv4_attention(c, 12, hq, 6, evicts=True)
    prompt = zl.allocate_kv4_attention(c, 20, hq, 10, state=step) if shared else step
    T = {None: 10 if shared else 6, keep: 6}
    g = torch.Generator().manual_seed(60)
    table = zl.rotary_table(zl.rotary_frequencies(d)[0])
    data, pages = c.data.cpu().numpy(), c.pages.cpu().numpy()
    w, pos = np.zeros(c.slot_shape), np.zeros(c.slot_shape, int)
    lens, at = np.zeros(2, int), np.zeros(2, int)
    calls = {}

    def call(k):
        n = T[k]
        if k not in calls:
            inputs = (torch.empty(2 * n, hq + 2 * heads, d, dtype=torch.bfloat16).cuda(),
                      torch.zeros(2 * n, dtype=torch.int32).cuda(), starts_of([n, n])[1])
            calls[k] = [inputs, None]
        (qkv, positions, ds), captured = calls[k]
        qkv.copy_(torch.randn(qkv.shape, generator=g))
        positions.copy_(torch.from_numpy(np.concatenate([at[b] + np.arange(n) for b in range(2)])))

        def body():
            c.lens.add_(n)
            zl.qkv_attention_cached(c, qkv, positions, table, d ** -0.5, prompt if k is None else step, starts=ds, max_new=n,
                                    keep=k, recent=recent)

        if not graph:
            body()
        else:
            if captured is None:
                held = [x.clone() for x in (c.data, c.lens, step["weights"], step["positions"])]
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(side):
                    body()
                torch.cuda.current_stream().wait_stream(side)
                for x, y in zip((c.data, c.lens, step["weights"], step["positions"]), held):
                    x.copy_(y)
                captured = calls[k][1] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(captured):
                    body()
            captured.replay()
        return qkv, prompt if k is None else step

    for turn in range(12):
        if turn == 7:  # the second row is another sequence's from here on
            lens[1] = at[1] = 0
            c.lens.copy_(torch.from_numpy(lens).int())
        k = None if turn < 3 or turn == 7 else keep
        n = T[k]
        qkv, bufs = call(k)
        starts = [0, n, 2 * n]
        lens, at = lens + n, at + n
        ref.write(data, pages, lens, starts, f64(bufs["k"]), f64(qkv[:, hq + heads:]))
        want, tol = reference(f64(bufs["q"]), data, pages, lens, starts, d ** -0.5, w)
        within(f64(bufs["o"]), want["o"], tol["o"], "o")
        within(f64(bufs["lse"]), want["lse"], tol["lse"], "lse")
        for b in range(2):
            pos[b, :, lens[b] - n:lens[b]] = at[b] - n + np.arange(n)
            w[b, :, lens[b] - n:lens[b]] = 0
        if k is not None:
            w = np.where(np.isnan(want["weights"]), w, want["weights"])
            for b in range(2):
                for h in range(heads):
                    for a, to in ref.evict_moves(w[b, h, :lens[b]], pos[b, h, :lens[b]], keep, recent):
                        ref.put_row(data, pages, b, h, to, ref.get_row(data, pages, b, h, a))
                        w[b, h, to], pos[b, h, to] = w[b, h, a], pos[b, h, a]
            lens = np.minimum(lens, keep)
        got_w, got_pos = f64(step["weights"]), step["positions"].cpu().numpy()
        for b in range(2):
            m = lens[b]
            assert np.array_equal(got_pos[b, :, :m], pos[b, :, :m]), turn
            off = np.abs(got_w[b, :, :m] - w[b, :, :m])
            assert off.max() <= (2 * tol["weights"].max() if k is not None else 0), turn
            w[b, :, :m] = got_w[b, :, :m]
        assert np.array_equal(c.lens.cpu().numpy(), lens)
    assert zl.zl_kv4_get_device_status(c) == 0


def test_buffers_with_state_want_one_position_a_token_and_the_cache_s_sizes():
    import torch
    c = zl.allocate_kv4(2, 2, 2, 64, page=16)
    c.lens.fill_(1)
    bufs = zl.allocate_kv4_attention(c, 2, 4, evicts=True)
    other = zl.allocate_kv4(2, 3, 2, 64, page=16)
    with pytest.raises(ValueError):
        zl.allocate_kv4_attention(other, 2, 4, state=bufs)
    more = zl.allocate_kv4_attention(c, 2, 4, state=bufs)
    assert more["weights"] is bufs["weights"] and more["positions"] is bufs["positions"]
    qkv, table = torch.ones(2, 8, 64).bfloat16().cuda(), zl.rotary_table(zl.rotary_frequencies(64)[0])
    with pytest.raises(ValueError):
        zl.qkv_attention_cached(c, qkv, torch.zeros(1, dtype=torch.int32).cuda(), table, 0.1, bufs)


# ---------------------------------------------------------------- status
def test_the_status_of_a_call_under_way_on_another_stream():
    import torch
    c, _, _ = make_cache([40, 40], 2, 64, 16, 72)
    c.pages[1, 0] = -1
    q, o, lse = torch.ones(2, 4, 64).bfloat16().cuda(), torch.empty(2, 4, 64).bfloat16().cuda(), torch.empty(2, 4).cuda()
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 4), dtype=torch.uint8).cuda()
    zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1)
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_PAGE
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1, stream=side)
        assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_PAGE
        assert zl.zl_kv4_get_device_status(c) == 0


# ---------------------------------------------------------------- eviction
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,keep,table", [(64, 61, 0), (64, 40, 0), (700, 300, 0), (64, 62, 640)])
@pytest.mark.parametrize("d", [64, 128])
def test_eviction_leaves_out_whole_moves_of_bad_pages(lens, keep, table, d, in_place):
    import torch
    c, data, pages = make_cache([lens], 2, d, 16, 73, extra_pages=table // 16)
    bad = [1, (lens - 1) // 16]
    pages[0, bad] = -1, 10 ** 6
    c.pages.copy_(torch.from_numpy(pages).int())
    rng = np.random.default_rng(74)
    w, pos = rng.random(c.slot_shape).astype(np.float32), np.argsort(rng.random(c.slot_shape), -1)
    w[0, :, 16:32] *= 1e-3  # slots given up, in a page that is not there
    w[0, :, lens - 5:lens] += 1
    dw, dp = torch.from_numpy(w).cuda(), torch.from_numpy(pos).int().cuda()
    wo, po = (dw, dp) if in_place else (torch.full_like(dw, 7.0), torch.full_like(dp, 7))
    zl.zl_kv4_evict(c, dw, dp, keep, 0, torch.empty(zl.zl_kv4_evict_workspace_bytes(c), dtype=torch.uint8).cuda(), wo, po)
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_PAGE
    want, ww, wp = data.copy(), np.full_like(w, 7.0), np.full_like(pos, 7)
    if in_place:
        ww, wp = w.copy(), pos.copy()
    ww[..., :keep], wp[..., :keep] = w[..., :keep], pos[..., :keep]
    left_out = 0
    for h in range(2):
        for a, to in ref.evict_moves(w[0, h, :lens], pos[0, h, :lens], keep, 0):
            if a // 16 in bad or to // 16 in bad:
                left_out += 1
                continue
            ref.put_row(want, pages, 0, h, to, ref.get_row(data, pages, 0, h, a))
            ww[0, h, to], wp[0, h, to] = w[0, h, a], pos[0, h, a]
    assert left_out > 0
    assert np.array_equal(c.data.cpu().numpy(), want)
    assert np.array_equal(wo.cpu().numpy(), ww) and np.array_equal(po.cpu().numpy(), wp)


# ---------------------------------------------------------------- refusals
def test_a_refused_step_leaves_everything_as_it_was():
    import torch
    heads, hq, d, n = 2, 4, 64, 3
    c = zl.allocate_kv4(n, 2, heads, d, page=16)
    c.lens.fill_(5)
    bufs = zl.allocate_kv4_attention(c, n, hq, evicts=True)
    bufs["weights"].fill_(3.0)
    qkv, at = torch.ones(n, hq + 2 * heads, d).bfloat16().cuda(), torch.full((n,), 4, dtype=torch.int32).cuda()
    table = zl.rotary_table(zl.rotary_frequencies(d)[0])
    held = (c.data, c.lens, bufs["weights"], bufs["positions"])
    before = [x.clone() for x in held]
    ok = dict(cache=c, qkv=qkv, positions=at, table=table, scale=0.1, bufs=bufs, keep=4)
    for bad in (dict(keep=0), dict(keep=-3), dict(recent=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=1e-40),
                dict(decay=float("inf")), dict(max_new=0), dict(max_new=5000), dict(max_new=64), dict(bufs={**bufs, "o": bufs["o"][:2]}),
                dict(bufs={**bufs, "lse": bufs["lse"].half()}), dict(bufs={**bufs, "workspace": bufs["workspace"][:64]}),
                dict(bufs={**bufs, "weights": bufs["weights"][:1]}), dict(bufs={**bufs, "positions": bufs["positions"].long()}),
                dict(starts=torch.zeros(3, dtype=torch.int32).cuda()), dict(keep=2 ** 31), dict(keep=2 ** 32 + 4),
                dict(recent=2 ** 31), dict(keep=None, scale=-1.0), dict(keep=None, max_new=0), dict(keep=None, bufs={**bufs, "o": bufs["o"].float()})):
        with pytest.raises((zl.ZlError, TypeError, ValueError)):
            zl.qkv_attention_cached(**{**ok, **bad})
        assert all(torch.equal(x, y) for x, y in zip(held, before)), bad
    zl.qkv_attention_cached(**ok)
    assert (c.lens == 4).all()
    for bad in (dict(keep=2 ** 32 + 4), dict(keep=0), dict(recent=2 ** 32)):
        with pytest.raises(zl.ZlError):
            zl.zl_kv4_evict(**{**dict(cache=c, weights=bufs["weights"], positions=bufs["positions"], keep=3, recent=1,
                                      workspace=bufs["workspace"]), **bad})


# ---------------------------------------------------------------- starts, workspaces, streams
def test_a_write_with_descending_starts_changes_the_rows_of_the_range_that_is_there():
    import torch
    c, data, pages = make_cache([32, 32, 32], 1, 64, 16, 28)
    x = torch.randn(4, 1, 64, generator=torch.Generator().manual_seed(75)).bfloat16().cuda()
    zl.zl_kv4_write(c, x, -x, torch.tensor([0, 5, 1, 4], dtype=torch.int32).cuda())
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_STARTS
    want = data.copy()
    ref.write(want, pages[2:], [32], [0, 3], f64(x[1:]), -f64(x[1:]))
    got = c.data.cpu().numpy()
    for s in range(32):
        for a, b in zip(ref.get_row(got, pages, 2, 0, s), ref.get_row(want, pages, 2, 0, s)):
            assert np.array_equal(np.where(a == 8, 0, a) if len(a) == 64 else a, np.where(b == 8, 0, b) if len(b) == 64 else b)
    keep = np.ones(len(data), bool)
    keep[pages[2]] = False
    assert np.array_equal(got[keep], data[keep])


@pytest.mark.parametrize("lens,rows", [([300, 64], 0), ([300, 64], 48), ([5000, 9000], 0)])
def test_one_workspace_serves_smaller_calls(lens, rows):
    import torch
    new = [12, 9]
    c, data, pages = many(lens, 2, 64, 16, 53, rows) if rows else make_cache(lens, 2, 64, 16, 53)
    ws = torch.empty(max(zl.zl_kv4_attn_workspace_bytes(c, 8, 16), zl.zl_kv4_attn_workspace_bytes(c, 8, 12, True)),
                     dtype=torch.uint8).cuda()
    g = torch.Generator().manual_seed(76)
    w_in = torch.rand(c.slot_shape, generator=g).cuda()
    for now, weights in (([12, 9], False), ([2, 1], False), ([12, 9], True), ([1, 1], True), ([5, 0], False), ([9, 9], False),
                         ([1, 2], True)):
        starts, ds = starts_of(now)
        q = torch.randn(sum(now), 8, 64, generator=g).bfloat16().cuda()
        o, lse, w = torch.empty_like(q), torch.empty(sum(now), 8).cuda(), torch.zeros(c.slot_shape).cuda()
        kw = dict(weights=w_in, weights_out=w) if weights else {}
        zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.125, ds, max(now), **kw)
        want, tol = reference(f64(q), data, pages, lens, starts, 0.125, f64(w_in) if weights else None)
        within(f64(o), want["o"], tol["o"], "o")
        within(f64(lse), want["lse"], tol["lse"], "lse")
        if weights:
            within(f64(w), want["weights"], tol["weights"], "weights")
    assert zl.zl_kv4_get_device_status(c) == 0


@pytest.mark.parametrize("rows", [0, 64])
def test_calls_that_cut_items_on_other_streams_at_once(rows):
    import torch
    lens, new = [9000, 10, 3000], ([16, 10, 3] if rows else [1, 1, 1])
    c, data, pages = many(lens, 2, 128, 64, 77, rows) if rows else make_cache(lens, 2, 128, 64, 77)
    assert c.slots > 8192
    starts, ds = starts_of(new)
    outs, g = [], torch.Generator().manual_seed(78)
    for _ in range(6):
        q = torch.randn(sum(new), 8, 128, generator=g).bfloat16().cuda()
        ws = torch.full((zl.zl_kv4_attn_workspace_bytes(c, 8, max(new)),), 255, dtype=torch.uint8).cuda()
        outs.append((q, torch.empty_like(q), torch.empty(sum(new), 8).cuda(), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, o, lse, ws, stream in outs:
            zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1, ds, max(new), stream=stream)
    torch.cuda.synchronize()
    assert zl.zl_kv4_get_device_status(c) == 0
    for q, o, lse, _, _ in outs:
        want, tol = reference(f64(q), data, pages, lens, starts, 0.1)
        within(f64(o), want["o"], tol["o"], "o")
        within(f64(lse), want["lse"], tol["lse"], "lse")


@pytest.mark.parametrize("keep", [None, 8])
def test_steps_without_tokens_and_on_streams_of_either_kind(keep):
    """No sequence brings a token: nothing but a decay of the weights; then a step on a stream given as an object, as a number, or not."""
    import torch
    heads, hq, d, n = 2, 4, 64, 3
    table = zl.rotary_table(zl.rotary_frequencies(d)[0])
    g = torch.Generator().manual_seed(79)
    qkv, at = torch.randn(n, hq + 2 * heads, d, generator=g).bfloat16().cuda(), torch.full((n,), 6, dtype=torch.int32).cuda()
    results = []
    for stream in (None, torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        c = zl.allocate_kv4(n, 2, heads, d, page=16)
        bufs = zl.allocate_kv4_attention(c, n, hq, evicts=True)
        none = zl.allocate_kv4_attention(c, 0, hq, evicts=True, state=bufs)
        c.lens.fill_(6)
        bufs["weights"].fill_(2.0)
        torch.cuda.synchronize()
        zl.qkv_attention_cached(c, qkv[:0], at[:0], table, 0.1, none, starts=torch.zeros(n + 1, dtype=torch.int32).cuda(), keep=keep,
                                recent=2, decay=0.5, stream=stream)
        torch.cuda.synchronize()
        assert (bufs["weights"][:, :, :6] == (2.0 if keep is None else 1.0)).all() and (c.lens == 6).all()
        with torch.cuda.stream(None if stream is None else stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream)):
            c.lens.add_(1)
        zl.qkv_attention_cached(c, qkv, at, table, 0.1, bufs, keep=keep, recent=2, stream=stream)
        assert zl.zl_kv4_get_device_status(c) == 0
        assert (bufs["positions"][:, :, 6] == 6).all() and (c.lens == 7).all()
        assert keep is not None or (bufs["weights"][:, :, 6] == 0).all()
        results.append([bufs[x].clone() for x in ("o", "lse", "weights", "positions")] + [c.data])
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))


def test_a_sequence_whose_tokens_do_not_fit_keeps_its_weights_and_positions():
    import torch
    heads, hq, d = 2, 4, 64
    c = zl.allocate_kv4(2, 2, heads, d, page=16)
    bufs = zl.allocate_kv4_attention(c, 4, hq, max_new=9, evicts=True)
    bufs["weights"].fill_(2.0)
    bufs["positions"].fill_(5)
    c.lens.fill_(20)
    qkv, at = torch.ones(4, hq + 2 * heads, d).bfloat16().cuda(), torch.arange(4, dtype=torch.int32).cuda()
    starts = torch.tensor([0, 2, 9], dtype=torch.int32).cuda()
    zl.qkv_attention_cached(c, qkv, at, zl.rotary_table(zl.rotary_frequencies(d)[0]), 0.1, bufs, starts=starts, max_new=9)
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_STARTS
    w, pos = bufs["weights"].cpu(), bufs["positions"].cpu()
    assert (w[1] == 2.0).all() and (pos[1] == 5).all()
    assert (w[0, :, 18:20] == 0).all() and (w[0, :, :18] == 2.0).all() and (w[0, :, 20:] == 2.0).all()
    assert (pos[0, :, 18:20] == torch.tensor([0, 1])).all() and (pos[0, :, :18] == 5).all()
