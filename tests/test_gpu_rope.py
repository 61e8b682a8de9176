"""Rotary positions and head norms on the GPU against the 64-bit reference.

Tolerances.  A bf16 result is off by at most half a step, 2^-8 of its value.  The fp32 arithmetic before it: a
rotated value is a sum of two products, each within a few 2^-24 of its operands (sine and cosine to 2^-22,
angle to 2^-25 turns), so 2^-18 of the row's largest term covers it; the norm's factor is one fp32 scalar to a
few 2^-24.  A weight's gradient is a sum over tokens and heads of terms each within 2^-20 of |g|max |n| in fp32,
summed in short fp32 runs: 2^-17 of the sum of the terms' absolute values."""
import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import causal as ref
from tests._lib import ensure_library

pytestmark = pytest.mark.gpu
HALF_STEP = 2.0 ** -8
EPS = 1e-6


def near(got, want, slack):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape
    err = np.abs(got - want)
    assert (err <= HALF_STEP * np.abs(want) + slack).all(), (err - HALF_STEP * np.abs(want)).max()


def inputs(n, hq, hk, d, axes, seed, far=1000):
    import torch
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(n, hq + 2 * hk, d, generator=g) * 2).bfloat16()
    pos = torch.randint(-far, far, (n, axes), generator=g).int()
    w = 1 + 0.3 * torch.randn(2, d, generator=g)
    go = torch.randn(n, hq + hk, d, generator=g).bfloat16()
    return qkv, pos, w, go


def run(n, hq, hk, d, rot, half, axis_pairs, norm, weights=True, seed=0, far=1000, amplitude=1.0, radians=None):
    """Forward and backward through strided views; everything against the reference."""
    import torch
    ensure_library()
    qkv, pos, w, go = inputs(n, hq, hk, d, len(axis_pairs), seed, far)
    radians = radians if radians is not None else zl.rotary_frequencies(rot)[0] if rot else []
    table = zl.rotary_table(radians, "half" if half else "interleaved", axis_pairs, amplitude) if rot else None
    dev = qkv.cuda()
    q, k = dev[:, :hq], dev[:, hq:hq + hk]
    posd, wd, god = pos.cuda(), w.cuda(), go.cuda()
    out = torch.full_like(dev, float("nan"))
    qo, ko = out[:, :hq], out[:, hq:hq + hk]
    qw, kw = (wd[0], wd[1]) if norm and weights else (None, None)
    none_q, none_k = hq == 0, hk == 0
    a = lambda x, none: None if none else x  # noqa: E731
    zl.zl_qk_rope_fwd(a(q, none_q), a(k, none_k), a(qo, none_q), a(ko, none_k), posd, table, norm, a(qw, none_q), a(kw, none_k), EPS)
    din = torch.full_like(dev, float("nan"))
    dw = torch.full((2, d), float("nan"), device="cuda")
    ws = torch.empty(zl.zl_qk_rope_workspace_bytes(n, hq, hk, d), dtype=torch.uint8, device="cuda")
    use_w = norm and weights
    zl.zl_qk_rope_bwd(a(q, none_q), a(k, none_k), a(god[:, :hq], none_q), a(god[:, hq:], none_k), a(din[:, :hq], none_q),
                      a(din[:, hq:hq + hk], none_k), posd, table, norm, a(qw, none_q), a(kw, none_k),
                      a(dw[0], none_q or not use_w), a(dw[1], none_k or not use_w), ws, EPS)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, hq + hk:].float()).all() and torch.isnan(din[:, hq + hk:].float()).all()  # values untouched
    ang = ref.angles(pos.numpy(), radians, axis_pairs) if rot else np.zeros((n, 0))
    for t, (lo, hi) in enumerate(((0, hq), (hq, hq + hk))):
        if lo == hi or n == 0:
            continue
        x, g = qkv[:, lo:hi].double().numpy(), go[:, lo:hi].double().numpy()
        weight = w[t].double().numpy() if use_w else np.ones(d)
        y = ref.rms_norm(x, weight, EPS) if norm else x
        near(out[:, lo:hi], ref.rotate(y, ang, half, amplitude),
             2.0 ** -18 * abs(amplitude) * np.abs(y).max(-1, keepdims=True) + 1e-30)
        dy = ref.rotate(g, -ang, half, amplitude)
        if not norm:
            near(din[:, lo:hi], dy, 2.0 ** -18 * abs(amplitude) * np.abs(g).max(-1, keepdims=True))
            continue
        dx, dweight = ref.rms_norm_grad(x, weight, EPS, dy)
        r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        size = r * np.abs(dy * weight).max(-1, keepdims=True) * (1 + np.abs(x * r).max(-1, keepdims=True))
        near(din[:, lo:hi], dx, 2.0 ** -17 * size)
        if use_w:
            terms = np.abs(g).max(-1, keepdims=True) * abs(amplitude) * np.abs(x * r)
            assert (np.abs(dw[t].double().cpu().numpy() - dweight) <= 2.0 ** -17 * terms.sum((0, 1)) + 1e-12).all()


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,rot,axis_pairs", [
    (1, 1, 1, 64, 64, [32]), (3, 4, 2, 64, 64, [32]), (7, 5, 1, 128, 128, [64]), (33, 24, 8, 64, 32, [16]),
    (5, 3, 3, 128, 96, [16, 24, 8]), (2, 7, 0, 128, 16, [8]), (2, 0, 5, 64, 48, [4, 20]), (301, 9, 2, 128, 128, [0, 64, 0]),
    (4, 6, 2, 64, 0, [0]), (5000, 4, 2, 64, 64, [32]),
    (64, 16, 2, 128, 128, [64]), (128, 8, 8, 64, 64, [32]), (129, 4, 4, 128, 64, [32]), (9, 200, 40, 64, 32, [16])])
def test_parity(n, hq, hk, d, rot, axis_pairs, half, norm):
    run(n, hq, hk, d, rot, half, axis_pairs, norm, seed=n + rot)


def test_interleaved_parts_that_end_inside_a_lane():
    for rot in (2, 6, 10, 62):
        run(9, 3, 2, 64, rot, False, [rot // 2], True, seed=rot)


@pytest.mark.parametrize("half", [False, True])
def test_far_positions_and_amplitude(half):
    radians, amp = zl.rotary_frequencies(128, scaling="yarn", factor=16.0)
    run(40, 4, 2, 128, 128, half, [64], True, seed=3, far=2 ** 31 - 1, amplitude=amp, radians=radians)
    run(40, 4, 2, 64, 64, half, [32], False, seed=4, far=10 ** 6, amplitude=-0.5)


def test_norm_without_weights_and_one_sided_weights():
    import torch
    run(11, 4, 2, 128, 128, True, [64], True, weights=False)
    qkv, pos, w, go = inputs(11, 4, 2, 128, 1, 5)
    dev, wd, posd = qkv.cuda(), w.cuda(), pos.cuda()
    table = zl.rotary_table(zl.rotary_frequencies(128)[0])
    both = [torch.empty(11, h, 128, dtype=torch.bfloat16, device="cuda") for h in (4, 2)]
    zl.zl_qk_rope_fwd(dev[:, :4], dev[:, 4:6], *both, posd, table, True, wd[0], None, EPS)
    ones = [torch.empty_like(x) for x in both]
    zl.zl_qk_rope_fwd(dev[:, :4], dev[:, 4:6], *ones, posd, table, True, wd[0], torch.ones(128, device="cuda"), EPS)
    assert all(torch.equal(x, y) for x, y in zip(both, ones))


def test_in_place_and_no_tokens():
    import torch
    ensure_library()
    qkv, pos, w, go = inputs(77, 6, 3, 64, 1, 9)
    dev, wd, posd, god = qkv.cuda(), w.cuda(), pos.cuda(), go.cuda()
    table = zl.rotary_table(zl.rotary_frequencies(64)[0])
    out = torch.empty_like(dev)
    zl.zl_qk_rope_fwd(dev[:, :6], dev[:, 6:9], out[:, :6], out[:, 6:9], posd, table, True, wd[0], wd[1], EPS)
    same = dev.clone()
    zl.zl_qk_rope_fwd(same[:, :6], same[:, 6:9], same[:, :6], same[:, 6:9], posd, table, True, wd[0], wd[1], EPS)
    assert torch.equal(same[:, :9], out[:, :9]) and torch.equal(same[:, 9:], dev[:, 9:])
    g2, dw, ws = god.clone(), torch.empty(2, 64, device="cuda"), torch.empty(1 << 21, dtype=torch.uint8, device="cuda")
    args = (posd, table, True, wd[0], wd[1], dw[0], dw[1], ws, EPS)
    zl.zl_qk_rope_bwd(dev[:, :6], dev[:, 6:9], god[:, :6], god[:, 6:], out[:, :6], out[:, 6:9], *args)
    zl.zl_qk_rope_bwd(dev[:, :6], dev[:, 6:9], g2[:, :6], g2[:, 6:], g2[:, :6], g2[:, 6:], *args)
    assert torch.equal(g2, out[:, :9])
    dw.fill_(7.0)
    none = dev[:0]
    zl.zl_qk_rope_bwd(none[:, :6], none[:, 6:9], god[:0, :6], god[:0, 6:], out[:0, :6], out[:0, 6:9], posd[:0], table, True,
                      wd[0], wd[1], dw[0], dw[1], ws, EPS)
    assert (dw == 0).all()  # empty sums
    zl.zl_qk_rope_fwd(none[:, :6], none[:, 6:9], out[:0, :6], out[:0, 6:9], posd[:0], table)


def test_weight_gradients_repeat_bit_for_bit_and_replay():
    """Fixed order of the sums; a captured backward replayed on new data equals an eager one."""
    import torch
    ensure_library()
    n, hq, hk, d = 3001, 8, 2, 128
    table = zl.rotary_table(zl.rotary_frequencies(d)[0])
    sets = [[x.cuda() for x in inputs(n, hq, hk, d, 1, s)] for s in (1, 2)]
    state = [x.clone() for x in sets[0]]
    dx, dw = torch.empty(n, hq + hk, d, dtype=torch.bfloat16, device="cuda"), torch.empty(2, d, device="cuda")
    ws = torch.empty(zl.zl_qk_rope_workspace_bytes(n, hq, hk, d), dtype=torch.uint8, device="cuda")

    def step():
        qkv, pos, w, go = state
        zl.zl_qk_rope_bwd(qkv[:, :hq], qkv[:, hq:hq + hk], go[:, :hq], go[:, hq:], dx[:, :hq], dx[:, hq:], pos, table, True,
                          w[0], w[1], dw[0], dw[1], ws, EPS)

    eager = []
    for s in sets:
        for dst, src in zip(state, s):
            dst.copy_(src)
        step()
        first = (dx.clone(), dw.clone())
        step()
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
        eager.append(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s, want in zip(sets, eager):
        for dst, src in zip(state, s):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_launches_in_a_row_see_the_latest_writes():
    """Kernels that are set up while the one before them runs: the same buffers, inputs that change from call to call,
    nothing awaited in between, equal the same calls each awaited."""
    import torch
    ensure_library()
    n, hq, hk, d = 200, 8, 2, 128
    table = zl.rotary_table(zl.rotary_frequencies(d)[0])
    sets = [[x.cuda() for x in inputs(n, hq, hk, d, 1, s)] for s in (3, 4, 5)]
    state = [x.clone() for x in sets[0]]
    out, dx = (torch.empty(n, hq + hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    dw = torch.empty(2, d, device="cuda")
    ws = torch.empty(zl.zl_qk_rope_workspace_bytes(n, hq, hk, d), dtype=torch.uint8, device="cuda")

    def calls(wait):
        got = []
        for i in range(24):
            for dst, src in zip(state, sets[i % 3]):
                dst.copy_(src)
            qkv, pos, w, _ = state
            for _ in range(2):
                zl.zl_qk_rope_fwd(qkv[:, :hq], qkv[:, hq:hq + hk], out[:, :hq], out[:, hq:], pos, table, True, w[0], w[1], EPS)
                wait()
                zl.zl_qk_rope_bwd(qkv[:, :hq], qkv[:, hq:hq + hk], out[:, :hq], out[:, hq:], dx[:, :hq], dx[:, hq:], pos,
                                  table, True, w[0], w[1], dw[0], dw[1], ws, EPS)
                wait()
                # in place: the result is the next call's input
                zl.zl_qk_rope_fwd(dx[:, :hq], dx[:, hq:], qkv[:, :hq], qkv[:, hq:hq + hk], pos, table)
                wait()
            got += [out.clone(), dx.clone(), dw.clone()]
        torch.cuda.synchronize()
        return got

    for x, y in zip(calls(lambda: None), calls(torch.cuda.synchronize)):
        assert torch.equal(x, y)


def test_calls_on_two_streams_at_once():
    import torch
    ensure_library()
    table = zl.rotary_table(zl.rotary_frequencies(64)[0])
    work = []
    for s, n in ((1, 5000), (2, 3333)):
        qkv, pos, w, _ = (x.cuda() for x in inputs(n, 6, 3, 64, 1, s))
        work.append((qkv, pos, w, torch.empty_like(qkv), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(8):
        for qkv, pos, w, out, st in work:
            zl.zl_qk_rope_fwd(qkv[:, :6], qkv[:, 6:9], out[:, :6], out[:, 6:9], pos, table, True, w[0], w[1], EPS, stream=st)
    torch.cuda.synchronize()
    for qkv, pos, w, out, _ in work:
        want = torch.empty_like(qkv)
        zl.zl_qk_rope_fwd(qkv[:, :6], qkv[:, 6:9], want[:, :6], want[:, 6:9], pos, table, True, w[0], w[1], EPS)
        assert torch.equal(out[:, :9], want[:, :9])


def test_python_refusals():
    import torch
    ensure_library()
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    table = zl.rotary_table(zl.rotary_frequencies(64)[0])
    ok = dict(q=x, k=x.clone(), q_out=x.clone(), k_out=x.clone(), positions=pos, table=table)
    zl.zl_qk_rope_fwd(**ok)
    zl.zl_qk_rope_fwd(**{**ok, "positions": pos[:, 0]})  # one axis may be flat
    for bad in (dict(q=x.float()), dict(q=x[:3]), dict(q=x.transpose(0, 1)), dict(q=x[:, :, ::2]), dict(positions=pos.long()),
                dict(positions=pos[:3]), dict(positions=None), dict(q_out=None), dict(q_out=x[:, :1]),
                dict(q=None, k=None), dict(norm=True, q_weight=torch.ones(32, device="cuda")),
                dict(norm=True, q_weight=torch.ones(64, device="cuda").half()), dict(q=x[0]),
                dict(norm=False, q_weight=torch.ones(64, device="cuda"))):
        with pytest.raises((TypeError, ValueError, zl.ZlError)):
            zl.zl_qk_rope_fwd(**{**ok, **bad})
    odd = torch.zeros(4 * 2 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:513].view(4, 2, 64)
    with pytest.raises(zl.ZlError) as e:
        zl.zl_qk_rope_fwd(**{**ok, "q": odd})
    assert e.value.status == zl.ZL_ERR_ALIGN
    w, dw = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):  # a workspace too small
        zl.zl_qk_rope_bwd(x, x, x.clone(), x.clone(), x.clone(), x.clone(), pos, table, True, w, w, dw, dw,
                          torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,hq,hk,d,norm,eps", [
    (5, 3, 2, 64, True, EPS), (5, 3, 2, 64, True, 0.0), (700, 5, 1, 128, True, EPS), (700, 5, 1, 128, False, EPS),
    (5000, 4, 2, 64, True, 0.0)])
def test_tokens_without_a_gradient(n, hq, hk, d, norm, eps, half):
    """Tokens marked as of no sequence: zero gradients, nothing in the weights', whatever their rows hold.  Equal, bit for
    bit, to the call on rows of ones with zero gradients there, whose terms are exact zeros."""
    import torch
    ensure_library()
    qkv, pos, w, go = inputs(n, hq, hk, d, 1, n)
    g = torch.Generator().manual_seed(n + 1)
    live = [(torch.rand(n, generator=g) < 0.7).to(torch.uint8) for _ in range(2)]
    live[0][0], live[1][-1] = 0, 0
    table = zl.rotary_table(zl.rotary_frequencies(d)[0], "half" if half else "interleaved")
    heads = (slice(0, hq), slice(hq, hq + hk))
    dirty, clean = (qkv.clone(), go.clone()), (qkv.clone(), go.clone())
    for s, rows in zip(heads, live):
        for x in dirty:
            x[:, s][rows == 0] = float("nan")
        clean[0][:, s][rows == 0] = 1.0
        clean[1][:, s][rows == 0] = 0.0
    wd, posd = w.cuda(), pos.cuda()
    ws = torch.empty(zl.zl_qk_rope_workspace_bytes(n, hq, hk, d), dtype=torch.uint8, device="cuda")

    def back(x, grad, rows):
        x, grad = x.cuda(), grad.cuda()
        out, dw = torch.full_like(grad, float("nan")), torch.full((2, d), float("nan"), device="cuda")
        weights = (wd[0], wd[1], dw[0], dw[1]) if norm else (None,) * 4
        zl.zl_qk_rope_bwd(x[:, heads[0]], x[:, heads[1]], grad[:, heads[0]], grad[:, heads[1]], out[:, heads[0]], out[:, heads[1]],
                          posd, table, norm, *weights, ws, eps, q_rows=rows[0], k_rows=rows[1])
        return out, dw

    got, got_w = back(*dirty, [r.cuda() for r in live])
    want, want_w = back(*clean, (None, None))
    assert torch.equal(got, want) and (not norm or torch.equal(got_w, want_w))
    for s, rows in zip(heads, live):
        assert (got[:, s][rows.cuda() == 0] == 0).all()
    one, _ = back(dirty[0], clean[1], (live[0].cuda(), None))  # queries alone
    assert torch.equal(one[:, heads[0]], want[:, heads[0]])
    for bad in (live[0], live[0].cuda()[:-1], live[0].cuda().int()):
        with pytest.raises((TypeError, ValueError)):
            back(*dirty, (bad, None))


@pytest.mark.parametrize("half,rots", [(True, (0, 16, 32, 48)), (False, (0, 2, 6, 32, 62))])
@pytest.mark.parametrize("d", [64, 128])
def test_channels_past_the_rotated_ones_pass_through(half, rots, d):
    """Inf, NaN and -0 there stay what they are, bit for bit, and reach no other channel; forward and gradient."""
    import torch
    ensure_library()
    n, h = 37, 5
    x = inputs(n, h, 1, d, 1, 2)[0][:, :h]
    pos = torch.arange(n).int()[:, None].cuda()
    bits = lambda t: t.cpu().view(torch.int16)  # noqa: E731
    for rot in rots:
        table = zl.rotary_table(zl.rotary_frequencies(rot)[0], "half" if half else "interleaved", amplitude=1.5) if rot else None
        dirty = x.clone()
        for i, bad in enumerate((float("inf"), float("-inf"), float("nan"), -0.0)):
            dirty[i::5, i::3, rot + 1 + 3 * i::11] = bad
        outs = {}
        for name, y in (("clean", x), ("dirty", dirty)):
            y = y.cuda()
            outs[name] = [torch.empty_like(y), torch.empty_like(y)]
            zl.zl_qk_rope_fwd(y, None, outs[name][0], None, pos, table)
            zl.zl_qk_rope_bwd(None, None, y, None, outs[name][1], None, pos, table)
        for c, o in zip(outs["clean"], outs["dirty"]):
            assert torch.equal(bits(o)[..., rot:], dirty.view(torch.int16)[..., rot:])
            assert torch.equal(bits(o)[..., :rot], bits(c)[..., :rot])
        # norm: an Inf makes 1 / rms zero, and NaN of itself alone
        lone = x.clone()
        lone[:, :, rot + 1] = float("inf")
        o = torch.empty_like(lone.cuda())
        zl.zl_qk_rope_fwd(lone.cuda(), None, o, None, pos, table, True, None, None, EPS)
        o = o.cpu()
        assert torch.isnan(o[:, :, rot + 1]).all()
        o[:, :, rot + 1] = 0.0
        assert (o == 0).all()
