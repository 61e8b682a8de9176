"""Causal attention with grouped heads on the GPU against the 64-bit reference.

Tolerances are bounds by arithmetic, element by element, with a = 2^-8 the half step of bf16 relative to a value:
  scores     a dot of d bf16 products summed in fp32: e_s = d 2^-24 scale |q|.|k|; P is off by e_s + 2^-20, relative
  O          P rounded to bf16 (a) and off by that much, O rounded (a):   a |O| + (a + e_P) P |V|
  LSE        max e_s + 2^-20 (1 + |LSE|)
  D          dO . O with the O that the forward stored:                   |dO| . tol(O) + d 2^-24 |dO|.|O|
  dS         P (dP - D):                 e_P |dS| + P (tol(D) + d 2^-24 |dO|.|V|), then rounded to bf16 (a)
  dV, dK, dQ the products of those with |dO|, |Q|, |K|, and rounded (a)
Normwise, the same roundings are independent of one another and each is a / sqrt(3) of its value at most in the root
mean square, so the expected square of the error is at most (b = a^2 / 3, c the group's rows)
  O   b (O^2 + P^2 V^2)      D   dO^2 . that      dV  b (dV^2 + P^2' dO^2)
  dQ  b (dQ^2 + scale^2 dS^2 K^2) + var(D) (scale P K)^2      dK  b dK^2 + scale^2 (b dS^2 + P^2 var(D))' Q^2
(D's error is one number a row: its terms add up along j before they are squared).  The norm of n rows' errors stays
within 4 / sqrt(n) of its expectation; fp32 adds under a tenth.
"""
import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import causal as ref
from tests._lib import ensure_library

pytestmark = pytest.mark.gpu
A, F = 2.0 ** -8, 2.0 ** -24


def f64(x):
    return x.double().cpu().numpy()


def inputs(tq, tk, hq, hk, d, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(*s, generator=g).bfloat16() for s in ((tq, hq, d), (tk, hk, d), (tk, hk, d), (tq, hq, d))]


def bounds(q, k, v, do, seqs, scale):
    """Reference results and their element-wise bounds; rows of no sequence are NaN."""
    hq, hk, d = q.shape[1], k.shape[1], q.shape[2]
    want = dict(zip(("o", "lse"), ref.attend(q, k, v, seqs, scale)))
    want.update(zip(("dq", "dk", "dv"), ref.attend_grad(q, k, v, do, seqs, scale)))
    tol = {n: np.zeros_like(x) for n, x in want.items()}
    var = {n: np.zeros_like(x) for n, x in want.items()}
    b = A * A / 3
    for q0, n, k0, m in seqs:
        for h in range(hq):
            c = h // (hq // hk)
            Q, K, V, G = q[q0:q0 + n, h], k[k0:k0 + m, c], v[k0:k0 + m, c], do[q0:q0 + n, h]
            p, o, lse = ref.attend_head(Q, K, V, scale)
            vis = ref.visible(n, m)
            es = d * F * scale * (np.abs(Q) @ np.abs(K).T) * vis
            es_row = es.max(1, initial=0.0, keepdims=True)
            ep = es + es_row + 2.0 ** -20
            t_o = A * np.abs(o) + ((A + ep) * p) @ np.abs(V)
            tol["o"][q0:q0 + n, h] = t_o
            with np.errstate(invalid="ignore"):
                tol["lse"][q0:q0 + n, h] = np.where(np.isfinite(lse), es_row[:, 0] + 2.0 ** -20 * (1 + np.abs(lse)), 0.0)
            dp, dd = G @ V.T, np.sum(G * o, 1, keepdims=True)
            t_d = np.sum(np.abs(G) * (t_o + d * F * np.abs(o)), 1, keepdims=True)
            ds = p * (dp - dd)
            t_ds = (A + ep) * np.abs(ds) + p * (1 + A) * (t_d + d * F * (np.abs(G) @ np.abs(V).T))
            tol["dv"][k0:k0 + m, c] += ((A + ep) * p).T @ np.abs(G)
            tol["dk"][k0:k0 + m, c] += scale * t_ds.T @ np.abs(Q)
            tol["dq"][q0:q0 + n, h] = scale * t_ds @ np.abs(K)
            var["o"][q0:q0 + n, h] = b * (o ** 2 + p ** 2 @ V ** 2)
            var_d = np.sum(G ** 2 * var["o"][q0:q0 + n, h], 1, keepdims=True)
            var["dv"][k0:k0 + m, c] += b * (p ** 2).T @ G ** 2
            var["dk"][k0:k0 + m, c] += scale ** 2 * (b * ds ** 2 + p ** 2 * var_d).T @ Q ** 2
            var["dq"][q0:q0 + n, h] = b * scale ** 2 * ds ** 2 @ K ** 2 + var_d * (scale * p @ K) ** 2
    for name in ("dq", "dk", "dv"):  # fp32 sums over up to some thousand rows, and the rounding
        with np.errstate(invalid="ignore"):
            tol[name] = tol[name] * (1 + 2.0 ** -10) + A * np.abs(np.nan_to_num(want[name])) + 1e-30
            var[name] += b * np.nan_to_num(want[name]) ** 2
    return want, tol, var


class Case:
    def __init__(self, seqs, hq, hk, d, seed=0, tq=None, tk=None, scale=None, poison=False, ins=None):
        import torch
        ensure_library()
        self.seqs, self.scale = seqs, scale or d ** -0.5
        tq = tq if tq is not None else max([s[0] + s[1] for s in seqs] + [0])
        tk = tk if tk is not None else max([s[2] + s[3] for s in seqs] + [0])
        self.ins = ins or inputs(tq, tk, hq, hk, d, seed)
        self.in_q, self.in_k = np.zeros(tq, bool), np.zeros(tk, bool)
        for q0, n, k0, m in seqs:
            self.in_q[q0:q0 + n], self.in_k[k0:k0 + m] = True, True
        if poison:  # tokens of no sequence hold NaN in every input
            for x, used in zip(self.ins, (self.in_q, self.in_k, self.in_k, self.in_q)):
                x[torch.from_numpy(~used)] = float("nan")
        self.dev = [x.cuda() for x in self.ins]
        self.plan = zl.zl_plan_causal(seqs, hq, hk, d, tq, tk)
        self.bufs = zl.allocate_causal(self.plan, "cuda", backward=True)
        for n, b in self.bufs.items():
            b.fill_(255 if n == "workspace" else float("nan"))  # 255: NaN in every workspace word

    def forward(self, stream=None):
        b, (q, k, v, _) = self.bufs, self.dev
        zl.zl_causal_attn_fwd(self.plan, q, k, v, b["o"], b["lse"], b["workspace"], self.scale, stream)
        return self

    def backward(self, stream=None):
        b, (q, k, v, do) = self.bufs, self.dev
        zl.zl_causal_attn_bwd(self.plan, q, k, v, b["o"], do, b["lse"], b["dq"], b["dk"], b["dv"], b["workspace"],
                              self.scale, stream)
        return self

    def check(self, names=("o", "lse", "dq", "dk", "dv")):
        import torch
        torch.cuda.synchronize()
        assert zl.zl_causal_get_device_status(self.plan) == 0
        want, tol, var = bounds(*(f64(x) for x in self.ins), self.seqs, self.scale)
        for n in names:
            got, used = f64(self.bufs[n]), self.in_k if n in ("dk", "dv") else self.in_q
            assert np.isnan(got[~used]).all(), f"{n}: a row of no sequence was written"
            got, w, t = got[used], want[n][used], tol[n][used]
            fin = np.isfinite(w)
            assert np.array_equal(got[~fin], w[~fin]), n  # LSE = -inf
            assert np.isfinite(got[fin]).all(), n
            over = np.abs(got[fin] - w[fin]) - t[fin]
            assert over.size == 0 or over.max() <= 0, f"{n}: {over.max():.3e} over its bound"
            if n != "lse" and over.size:
                rms = np.sqrt(var[n][used].sum())
                most = 1.1 + 4 / np.sqrt(got.shape[0] * got.shape[1])
                off = np.linalg.norm(got[fin] - w[fin])
                assert off <= most * rms + 1e-30, f"{n}: {off / rms:.2f} times the expected error"
        return self


def packed(*lens):
    return zl.causal_seqs(lens)


@pytest.mark.parametrize("seqs,hq,hk,d", [
    (packed(1), 1, 1, 64), (packed(1, 2, 0, 3), 4, 2, 64), (packed(128), 2, 2, 128), (packed(129, 127), 4, 4, 64),
    (packed(300, 1, 64), 8, 1, 128), (packed(257), 6, 2, 64), (packed(200, 131), 5, 1, 128), (packed(140), 7, 1, 64),
    (packed(77, 400), 12, 1, 64), (packed(9, 33), 128, 1, 64), (packed(40), 100, 2, 64), (packed(513, 256), 16, 2, 128),
    ([(0, 5, 0, 300), (5, 64, 300, 64), (69, 1, 364, 129)], 8, 2, 128),          # chunks and a token behind cached keys
    ([(0, 9, 0, 3), (9, 200, 3, 150), (209, 4, 153, 0)], 6, 2, 64),              # queries that see no key
    ([(40, 70, 10, 70), (0, 30, 100, 30), (115, 0, 90, 5), (116, 3, 140, 260)], 4, 2, 64),  # gaps, any order, no queries
])
def test_parity(seqs, hq, hk, d):
    Case(seqs, hq, hk, d, seed=hq + d, tq=max(s[0] + s[1] for s in seqs) + 3, tk=max(s[2] + s[3] for s in seqs) + 2,
         poison=True).forward().backward().check()


@pytest.mark.parametrize("lens", [(1,), (127, 128), (1, 130, 255, 31), (700,)])
@pytest.mark.parametrize("hq,hk,d", [(4, 4, 64), (3, 1, 128), (8, 2, 128), (14, 2, 64)])
def test_lengths_by_heads(lens, hq, hk, d):
    Case(packed(*lens), hq, hk, d, seed=sum(lens)).forward().backward().check()


@pytest.mark.parametrize("hq,hk,d,seqs", [
    (8, 2, 128, [(0, 1, 0, 9001)]), (4, 4, 64, [(0, 1, 0, 5000), (1, 3, 5000, 4097), (4, 1, 9097, 1)]),
    (3, 1, 64, [(0, 20, 0, 3001)]), (16, 1, 128, [(0, 2, 0, 2600), (2, 7, 2600, 3)])])
def test_split_key_ranges(hq, hk, d, seqs):
    c = Case(seqs, hq, hk, d, seed=5)
    assert c.plan.fwd_workspace_bytes > 0 and any(t[5] >= 0 for t in c.plan.tiles(0))
    c.forward().check(("o", "lse"))
    c.backward().check()


def test_peaked_scores_and_other_scales():
    import torch
    ins = inputs(333, 333, 6, 2, 128, 11)
    ins[0] *= 6  # scores up to some 60: sharp rows, maxima that keep growing
    Case(packed(300, 33), 6, 2, 128, ins=[x.clone() for x in ins]).forward().backward().check()
    Case(packed(300, 33), 6, 2, 128, ins=ins, scale=1e-3).forward().backward().check()
    huge = inputs(200, 200, 2, 1, 64, 12)
    huge[1][150:] *= 1000  # growth past the lazy rescale's threshold many times over
    Case(packed(200), 2, 1, 64, ins=huge).forward().check(("o", "lse"))
    assert torch.isfinite(huge[1].float()).all()


def test_non_finite_keys_do_not_reach_rows_that_do_not_see_them():
    import torch
    for bad in (float("nan"), float("inf"), float("-inf")):
        ins = inputs(300, 300, 4, 2, 64, 13)
        clean = Case(packed(300), 4, 2, 64, ins=[x.clone() for x in ins]).forward()
        ins[1][200:] = bad
        dirty = Case(packed(300), 4, 2, 64, ins=ins).forward()
        torch.cuda.synchronize()
        assert torch.equal(clean.bufs["o"][:200], dirty.bufs["o"][:200])
        assert torch.equal(clean.bufs["lse"][:200], dirty.bufs["lse"][:200])


def test_views_of_a_fused_projection_give_the_same_bits():
    import torch
    seqs, hq, hk, d = packed(260, 33, 1), 6, 2, 128
    c = Case(seqs, hq, hk, d, seed=3).forward().backward()
    fused = torch.cat([x for x in c.dev[:3]], 1).contiguous()
    grads = torch.full_like(fused, float("nan"))
    v = Case(seqs, hq, hk, d, seed=3)
    cut = lambda x: [x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]]  # noqa: E731
    v.dev[:3] = cut(fused)
    v.bufs["dq"], v.bufs["dk"], v.bufs["dv"] = cut(grads)
    v.forward().backward()
    torch.cuda.synchronize()
    for n in ("o", "lse", "dk", "dv"):
        assert torch.equal(c.bufs[n], v.bufs[n].contiguous()), n
    v.check()


def test_key_gradients_and_outputs_repeat_bit_for_bit():
    import torch
    c = Case(packed(1500, 700, 1), 8, 2, 64, seed=8).forward().backward()
    first = {n: b.clone() for n, b in c.bufs.items()}
    for _ in range(3):
        c.forward().backward()
        torch.cuda.synchronize()
        for n in ("o", "lse", "dk", "dv"):
            assert torch.equal(first[n], c.bufs[n]), n


def test_one_plan_on_two_streams_and_in_captured_graphs():
    """The plan holds no state of a launch: two calls at once, and graphs replayed in any order."""
    import torch
    seqs, hq, hk, d = [(0, 1, 0, 9000), (1, 40, 9000, 40)], 8, 2, 128
    cases = [Case(seqs, hq, hk, d, seed=s) for s in (1, 2)]
    cases[1].plan = cases[0].plan
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(cases, streams):
            c.forward(s).backward(s)
    torch.cuda.synchronize()
    for c in cases:
        c.check()
    graphs = []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.forward().backward()
        graphs.append(g)
    for c in cases:
        for n in ("o", "lse", "dq", "dk", "dv"):
            c.bufs[n].fill_(float("nan"))
    for g in (graphs[1], graphs[0], graphs[1]):
        g.replay()
    torch.cuda.synchronize()
    for c in cases:
        c.check()


@pytest.mark.parametrize("d", [64, 128])
def test_launches_in_a_row_see_the_latest_writes(d):
    """Kernels that are set up while the one before them runs: split ranges in one workspace, inputs that change from
    call to call, nothing awaited in between, equal the same calls each awaited (dQ within the order of its fp32 sums)."""
    import torch
    seqs = [(0, 1, 0, 4000), (1, 2, 4000, 2500), (3, 300, 6500, 300)]
    c = Case(seqs, 8, 2, d, seed=21)
    sets = [[x.cuda() for x in inputs(303, 6800, 8, 2, d, s)] for s in (22, 23, 24)]
    assert c.plan.fwd_workspace_bytes > 0

    def calls(wait):
        got = []
        for i in range(12):
            for dst, src in zip(c.dev, sets[i % 3]):
                dst.copy_(src)
            for _ in range(2):
                c.forward()
                wait()
                c.backward()
                wait()
                c.dev[0].copy_(c.bufs["o"])  # the result is the next call's input
                wait()
            got.append({n: c.bufs[n].clone() for n in ("o", "lse", "dq", "dk", "dv")})
        torch.cuda.synchronize()
        return got

    for x, y in zip(calls(lambda: None), calls(torch.cuda.synchronize)):
        for n in ("o", "lse", "dk", "dv"):
            assert torch.equal(x[n], y[n]), n
        # an fp32 sum in another order moves a value over a rounding boundary of bf16 here and there: one step, 2^-7
        a, b = x["dq"].float(), y["dq"].float()
        assert ((a - b).norm() <= 2.0 ** -7 * b.norm()).item()
    assert zl.zl_causal_get_device_status(c.plan) == 0


def test_keys_beyond_32_bit_offsets():
    """A cache of 2.2 million rows (2^31 elements and more): the last rows' keys and values are found."""
    import torch
    ensure_library()
    rows, hk, hq, d = 2_200_000, 8, 16, 128
    seqs = [(0, 3, rows - 1400, 1399), (3, 1, 5, 200), (4, 1, rows - 1, 1)]
    q, _, _, _ = inputs(5, 1, hq, 1, d, 4)
    cache = torch.zeros(2, rows, hk, d, dtype=torch.bfloat16, device="cuda")
    small = inputs(1, 1600, 1, hk, d, 6)[1:3]
    for i in range(2):
        cache[i, rows - 1400:] = small[i][:1400].cuda()
        cache[i, 5:205] = small[i][1400:].cuda()
    plan = zl.zl_plan_causal(seqs, hq, hk, d, 5, rows)
    b = zl.allocate_causal(plan)
    zl.zl_causal_attn_fwd(plan, q.cuda(), cache[0], cache[1], b["o"], b["lse"], b["workspace"], d ** -0.5)
    near = [(0, 3, 0, 1399), (3, 1, 1400, 200), (4, 1, 1399, 1)]
    c = Case(near, hq, hk, d, ins=[q, small[0], small[1], q.clone()], tq=5, tk=1600)
    c.bufs["o"].copy_(b["o"])
    c.bufs["lse"].copy_(b["lse"])
    c.check(("o", "lse"))


def test_shared_keys_have_a_forward_and_no_backward():
    seqs = [(0, 3, 0, 200), (3, 2, 0, 100)]
    c = Case(seqs, 4, 2, 64, seed=2).forward().check(("o", "lse"))
    with pytest.raises(zl.ZlError) as e:
        c.backward()
    assert e.value.status == zl.ZL_ERR_INVALID_ARG
    c = Case([(0, 3, 0, 200), (3, 2, 200, 100)], 4, 2, 64, seed=3)
    c.plan = zl.zl_plan_causal(c.seqs, 4, 2, 64, 5, 300, zl.ZL_PLAN_FORWARD_ONLY)
    c.forward().check(("o", "lse"))
    with pytest.raises(zl.ZlError) as e:
        c.backward()
    assert e.value.status == zl.ZL_ERR_INVALID_ARG


def test_no_keys_no_queries_no_sequences():
    import torch
    c = Case([(0, 4, 0, 0)], 4, 2, 64, tk=0).forward().backward()
    torch.cuda.synchronize()
    assert (c.bufs["o"] == 0).all() and (c.bufs["lse"] == -float("inf")).all() and (c.bufs["dq"] == 0).all()
    c = Case([(0, 0, 0, 130)], 4, 2, 64, tq=0).forward().backward()
    torch.cuda.synchronize()
    assert (c.bufs["dk"] == 0).all() and (c.bufs["dv"] == 0).all()
    c = Case([], 4, 2, 64, tq=3, tk=3).forward().backward()
    torch.cuda.synchronize()
    assert all(torch.isnan(c.bufs[n].float()).all() for n in ("o", "lse", "dq", "dk", "dv"))


def test_gradient_against_differences():
    """<dO, O> moves by the gradient times the step, on fp32 sums of the forward's own outputs: the step is large (a
    bf16 input moves by whole steps) and the difference of two forwards carries their rounding, so the bound
    is on the directional derivative along the gradient itself."""
    import torch
    c = Case(packed(90, 40), 4, 2, 64, seed=21).forward().backward()
    torch.cuda.synchronize()
    want = dict(zip(("dq", "dk", "dv"), ref.attend_grad(*(f64(x) for x in c.ins), c.seqs, c.scale)))
    for i, n in enumerate(("dq", "dk", "dv")):
        g = f64(c.bufs[n])
        unit = g / np.linalg.norm(g)
        step = 1e-4
        moved = []
        for sign in (1, -1):
            x = [f64(y) for y in c.ins]
            x[i] = x[i] + sign * step * unit
            moved.append(np.sum(x[3] * ref.attend(x[0], x[1], x[2], c.seqs, c.scale)[0]))
        slope = (moved[0] - moved[1]) / (2 * step)
        assert abs(slope - np.sum(want[n] * unit)) <= 1e-5 * abs(slope)
        # the kernel's gradient against the differences: <g, g_exact> / |g| within its normwise error
        assert abs(slope - np.linalg.norm(g)) <= 1.2 * A * np.linalg.norm(g)


def test_withheld_load_reports_timeout_and_context_survives():
    import torch
    ensure_library()
    seqs, hq, hk, d = packed(200, 30), 4, 2, 128
    good = Case(seqs, hq, hk, d, seed=6).forward()
    bad = zl.zl_plan_causal(seqs, hq, hk, d, 230, 230, zl.ZL_PLAN_TEST_WITHHOLD_LOAD)
    b, (q, k, v, do) = zl.allocate_causal(bad, backward=True), good.dev
    zl.zl_causal_attn_fwd(bad, q, k, v, b["o"], b["lse"], b["workspace"], good.scale)
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(bad) == zl.ZL_ERR_TIMEOUT
    assert zl.zl_causal_get_device_status(bad) == 0
    zl.zl_causal_attn_bwd(bad, q, k, v, good.bufs["o"], do, good.bufs["lse"], b["dq"], b["dk"], b["dv"], b["workspace"], good.scale)
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(bad) == zl.ZL_ERR_TIMEOUT
    good.backward().check()


def test_launch_refusals():
    import torch
    c = Case(packed(30), 4, 2, 64)
    q, k, v, do = c.dev
    b = c.bufs
    fwd = dict(q=q, k=k, v=v, o=b["o"], lse=b["lse"], workspace=b["workspace"], scale=0.125)
    for bad in (dict(q=q.float()), dict(q=q[:29]), dict(k=k[:, :1]), dict(v=v.transpose(1, 2)), dict(o=None), dict(lse=b["lse"].half()),
                dict(o=b["o"].view(30, 2, 128)), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(scale=1e-42), dict(q=q.cpu())):
        with pytest.raises((TypeError, ValueError, zl.ZlError)):
            zl.zl_causal_attn_fwd(c.plan, **{**fwd, **bad})
    odd = torch.zeros(30 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:30 * 4 * 64 + 1].view(30, 4, 64)
    with pytest.raises(zl.ZlError) as e:
        zl.zl_causal_attn_fwd(c.plan, **{**fwd, "q": odd})
    assert e.value.status == zl.ZL_ERR_ALIGN
    c.forward()
    bwd = dict(q=q, k=k, v=v, o=b["o"], d_o=do, lse=b["lse"], dq=b["dq"], dk=b["dk"], dv=b["dv"], workspace=b["workspace"],
               scale=0.125)
    for bad in (dict(d_o=do[:, :2]), dict(dq=None), dict(dk=b["dk"].float()), dict(workspace=b["workspace"][:64]), dict(scale=0.0)):
        with pytest.raises((TypeError, ValueError, zl.ZlError)):
            zl.zl_causal_attn_bwd(c.plan, **{**bwd, **bad})
    small = zl.zl_plan_causal([(0, 1, 0, 9000)], 8, 2, 128, 1, 9000)
    with pytest.raises((TypeError, ValueError, zl.ZlError)):  # a split plan needs its workspace
        x = torch.zeros(9000, 2, 128, dtype=torch.bfloat16, device="cuda")
        o = torch.zeros(1, 8, 128, dtype=torch.bfloat16, device="cuda")
        zl.zl_causal_attn_fwd(small, o, x, x, o.clone(), torch.zeros(1, 8, device="cuda"), None, 0.1)


def test_projection_to_output_and_back():
    """Norm, rotation, attention and their gradients in one run, from a projection's output to its gradient,
    against the composition in 64 bits.  Normwise bound: each of the chain's stored tensors (q, k rotated; P; O; dS;
    dq, dk before the norm's gradient; the result) is rounded to bf16, at most 0.58 a root mean square each; six of
    them in a row, independent, stay under 1.5 a; the scores move by scale |q||k| a / 8 ~ a with q and k's
    rounding, once more for P and once for dS: 3 a in all."""
    import torch
    ensure_library()
    lens, hq, hk, d = (150, 1, 64), 8, 2, 128
    t = sum(lens)
    g = torch.Generator().manual_seed(0)
    qkv = (2 * torch.randn(t, hq + 2 * hk, d, generator=g)).bfloat16()
    do = torch.randn(t, hq, d, generator=g).bfloat16()
    w = 1 + 0.2 * torch.randn(2, d, generator=g)
    pos = torch.cat([torch.arange(n) for n in lens]).int()[:, None]
    radians, amp = zl.rotary_frequencies(d)
    seqs, scale = zl.causal_seqs(lens), d ** -0.5
    plan = zl.zl_plan_causal(seqs, hq, hk, d, t, t)
    bufs = zl.allocate_qkv_attention(plan, "cuda", backward=True)
    table = zl.rotary_table(radians, amplitude=amp)
    dev, wd = qkv.cuda(), w.cuda()
    dqkv = torch.full_like(dev, float("nan"))
    zl.qkv_attention_forward(plan, dev, pos.cuda(), table, scale, bufs, wd[0], wd[1])
    zl.qkv_attention_backward(plan, dev, do.cuda(), dqkv, pos.cuda(), table, scale, bufs, wd[0], wd[1])
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(plan) == 0
    x, wn, ang = f64(qkv), f64(w), ref.angles(pos.numpy(), radians, [d // 2])
    parts = [x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]]
    turned = [ref.rotate(ref.rms_norm(parts[i], wn[i], 1e-6), ang, True) for i in range(2)]
    o, lse = ref.attend(*turned, parts[2], seqs, scale)
    grads = ref.attend_grad(*turned, parts[2], f64(do), seqs, scale)
    want = [o, None, None, grads[2]]
    back = [ref.rms_norm_grad(parts[i], wn[i], 1e-6, ref.rotate(grads[i], -ang, True)) for i in range(2)]
    got = f64(dqkv)

    def close(a, b):
        assert np.linalg.norm(a - b) <= 3 * A * np.linalg.norm(b), np.linalg.norm(a - b) / np.linalg.norm(b)

    close(f64(bufs["o"]), want[0])
    close(got[:, :hq], back[0][0])
    close(got[:, hq:hq + hk], back[1][0])
    close(got[:, hq + hk:], grads[2])
    close(f64(bufs["dq_weight"]), back[0][1])
    close(f64(bufs["dk_weight"]), back[1][1])
    # the same queries and keys through the engine's bidirectional attention: the rotated tensors are its layout
    # (equal head counts), so the operators stand in front of it as well
    full = zl.zl_plan_worklist([zl.zl_work_item(0, t, 0, t, 0, hk, 0, t, 0, -1, -1)], hk, d, t)
    k = bufs["k"]
    fb = zl.forward(full, k, k, dev[:, hq + hk:].contiguous(), scale)
    torch.cuda.synchronize()
    kk, vv = f64(k), parts[2]
    for h in range(hk):
        s = scale * kk[:, h] @ kk[:, h].T
        p = np.exp(s - s.max(1, keepdims=True))
        close(f64(fb["o"])[:t * hk * d].reshape(t, hk, d)[:, h], p / p.sum(1, keepdims=True) @ vv[:, h])


def projection_reference(qkv, do, pos, w, radians, seqs, scale, hq, hk, eps=1e-6):
    """In 64 bits: o, the gradient of qkv and the weights' gradients of norm (where w has a weight), rotation and attention
    over seqs; rows of no sequence have gradient zero."""
    d = qkv.shape[2]
    x, g, ang = f64(qkv), np.nan_to_num(f64(do)), ref.angles(pos.numpy(), radians, [d // 2])
    parts = [np.nan_to_num(y) for y in (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:])]
    normed = [parts[i] if w[i] is None else ref.rms_norm(parts[i], f64(w[i]), eps) for i in range(2)]
    turned = [ref.rotate(y, ang, True) for y in normed]
    o, _ = ref.attend(*turned, parts[2], seqs, scale)
    grads = [np.nan_to_num(y) for y in ref.attend_grad(*turned, parts[2], g, seqs, scale)]
    dqkv, dw = np.zeros_like(x), [None, None]
    for i, cols in enumerate((slice(0, hq), slice(hq, hq + hk))):
        dy = ref.rotate(grads[i], -ang, True)
        if w[i] is None:
            dqkv[:, cols] = dy
        else:
            dqkv[:, cols], dw[i] = ref.rms_norm_grad(parts[i], f64(w[i]), eps, dy)
    dqkv[:, hq + hk:] = grads[2]
    return o, dqkv, dw


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("seqs,t", [
    ([(0, 90, 0, 90), (90, 41, 90, 41)], 160),                 # rows behind the last sequence
    ([(3, 70, 3, 70), (100, 1, 100, 1), (128, 130, 128, 130)], 300),  # sequences padded to a common stride
    ([(20, 50, 0, 80), (150, 30, 120, 20)], 200),              # rows that are keys alone, queries alone, neither
])
def test_projection_of_padded_batches(seqs, t, norm):
    """Rows of no sequence hold NaN everywhere, outputs and scratch included: the gradient there is zero, and the weights'
    gradients are those of the sequences' rows.  Bound as in test_projection_to_output_and_back, 3 a normwise."""
    import torch
    ensure_library()
    hq, hk, d = 8, 2, 64
    g = torch.Generator().manual_seed(t)
    qkv = ((2 if norm else 1) * torch.randn(t, hq + 2 * hk, d, generator=g)).bfloat16()  # scores of size 1 either way
    do = torch.randn(t, hq, d, generator=g).bfloat16()
    w = 1 + 0.2 * torch.randn(2, d, generator=g)
    pos = torch.randint(0, 500, (t, 1), generator=g).int()
    in_q, in_k = np.zeros(t, bool), np.zeros(t, bool)
    for q0, n, k0, m in seqs:
        in_q[q0:q0 + n], in_k[k0:k0 + m] = True, True
    qkv[:, :hq][torch.from_numpy(~in_q)] = float("nan")
    qkv[:, hq:][torch.from_numpy(~in_k)] = float("nan")
    do[torch.from_numpy(~in_q)] = float("nan")
    radians, _ = zl.rotary_frequencies(d)
    plan = zl.zl_plan_causal(seqs, hq, hk, d, t, t)
    bufs = zl.allocate_qkv_attention(plan, "cuda", backward=True)
    for n, b in bufs.items():
        b.fill_(255 if n.endswith("workspace") else float("nan"))
    dev, wd = qkv.cuda(), [w[0].cuda(), w[1].cuda()] if norm else [None, None]
    dqkv = torch.full_like(dev, float("nan"))
    args = (pos.cuda(), zl.rotary_table(radians))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        zl.qkv_attention_forward(plan, dev, *args, d ** -0.5, bufs, *wd, stream=stream)
        zl.qkv_attention_backward(plan, dev, do.cuda(), dqkv, *args, d ** -0.5, bufs, *wd, stream=stream)
        torch.cuda.synchronize()
        assert zl.zl_causal_get_device_status(plan) == 0
        o, want, dw = projection_reference(qkv, do, pos, [w[0], w[1]] if norm else [None, None], radians, seqs, d ** -0.5, hq, hk)
        got = f64(dqkv)

        def close(a, b):
            assert np.linalg.norm(a - b) <= 3 * A * np.linalg.norm(b), np.linalg.norm(a - b) / np.linalg.norm(b)

        close(f64(bufs["o"])[in_q], o[in_q])
        assert (got[:, :hq][~in_q] == 0).all() and (got[:, hq:][~in_k] == 0).all()
        for cols in (slice(0, hq), slice(hq, hq + hk), slice(hq + hk, None)):
            close(got[:, cols], want[:, cols])
        if norm:
            close(f64(bufs["dq_weight"]), dw[0])
            close(f64(bufs["dk_weight"]), dw[1])
        leaf = torch.full_like(dev, float("nan")).requires_grad_()  # a buffer that autograd knows is written like any other
        zl.qkv_attention_backward(plan, dev, do.cuda(), leaf, *args, d ** -0.5, bufs, *wd, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(leaf.detach()[:, hq + hk:], dqkv[:, hq + hk:])
        dqkv.fill_(float("nan"))


@pytest.mark.parametrize("side", [0, 1])
def test_projection_with_one_weight_norms_that_side_alone(side):
    """A weight for the queries alone (or the keys alone): the other tensor is rotated as it is.  Its heads are far from
    unit size, so that a norm there would show; bound as in test_projection_to_output_and_back."""
    import torch
    ensure_library()
    seqs, t, hq, hk, d = [(0, 90, 0, 90), (95, 40, 95, 40)], 140, 6, 2, 128
    g = torch.Generator().manual_seed(side)
    qkv = torch.randn(t, hq + 2 * hk, d, generator=g)
    qkv[:, hq:hq + hk] *= 0.5 if side == 0 else 1.0
    qkv[:, :hq] *= 0.5 if side == 1 else 1.0
    qkv, do = qkv.bfloat16(), torch.randn(t, hq, d, generator=g).bfloat16()
    w = [None, None]
    w[side] = 1 + 0.2 * torch.randn(d, generator=g)
    pos = torch.randint(0, 500, (t, 1), generator=g).int()
    radians, _ = zl.rotary_frequencies(d)
    plan = zl.zl_plan_causal(seqs, hq, hk, d, t, t)
    bufs = zl.allocate_qkv_attention(plan, "cuda", backward=True)
    for b in (bufs["dq_weight"], bufs["dk_weight"]):
        b.fill_(7.0)
    dev, wd = qkv.cuda(), [None if x is None else x.cuda() for x in w]
    dqkv = torch.full_like(dev, float("nan"))
    args = (pos.cuda(), zl.rotary_table(radians), d ** -0.5, bufs, *wd)
    zl.qkv_attention_forward(plan, dev, *args)
    zl.qkv_attention_backward(plan, dev, do.cuda(), dqkv, *args)
    torch.cuda.synchronize()
    o, want, dw = projection_reference(qkv, do, pos, w, radians, seqs, d ** -0.5, hq, hk)
    used = np.r_[0:90, 95:135]

    def close(a, b):
        assert np.linalg.norm(a - b) <= 3 * A * np.linalg.norm(b), np.linalg.norm(a - b) / np.linalg.norm(b)

    close(f64(bufs["o"])[used], o[used])
    for cols in (slice(0, hq), slice(hq, hq + hk), slice(hq + hk, None)):
        close(f64(dqkv)[:, cols], want[:, cols])
    close(f64(bufs[("dq_weight", "dk_weight")[side]]), dw[side])
    assert (bufs[("dk_weight", "dq_weight")[side]] == 7.0).all()  # not wanted: left as it was


def test_gradient_far_behind_the_query():
    """128 query heads of one token over more than 2^24 keys: the distance times the group passes 2^31.  The keys are zero, so
    every weight is 1 / m and dV is the same row for every key; a few values at both ends make dK.  Bounds as at the
    head of this file."""
    import torch
    ensure_library()
    m, hq, d, ends = 2 ** 24 + 200, 128, 64, 300
    scale = d ** -0.5
    q, _, v, do = inputs(1, 2 * ends, hq, 1, d, 31)
    big = torch.zeros(2, m, 1, d, dtype=torch.bfloat16, device="cuda")
    big[1, :ends], big[1, -ends:] = v[:ends].cuda(), v[ends:].cuda()
    plan = zl.zl_plan_causal([(0, 1, 0, m)], hq, 1, d, 1, m)
    b = zl.allocate_causal(plan, backward=True)
    for n in ("dk", "dv"):
        b[n].fill_(float("nan"))
    zl.zl_causal_attn_fwd(plan, q.cuda(), big[0], big[1], b["o"], b["lse"], b["workspace"], scale)
    zl.zl_causal_attn_bwd(plan, q.cuda(), big[0], big[1], b["o"], do.cuda(), b["lse"], b["dq"], b["dk"], b["dv"], b["workspace"], scale)
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(plan) == 0
    Q, V, G = f64(q)[0], f64(v)[:, 0], f64(do)[0]
    p, ep = 1 / m, 2.0 ** -20 * (2 + np.log(m))
    assert np.abs(f64(b["lse"])[0] - np.log(m)).max() <= 2.0 ** -20 * (1 + np.log(m))
    o, t_o = p * V.sum(0), A * p * np.abs(V.sum(0)) + (A + ep) * p * np.abs(V).sum(0)
    dv = p * G.sum(0)
    got = f64(b["dv"][0, 0])
    assert (np.abs(got - dv) <= (A + ep) * p * np.abs(G).sum(0) * (1 + 2.0 ** -10) + A * np.abs(dv)).all()
    assert torch.equal(b["dv"], b["dv"][:1].expand_as(b["dv"]))
    dd, t_d = G @ o, np.abs(G) @ (t_o + d * F * np.abs(o))
    ds = p * (G @ V.T - dd[:, None])  # [heads, keys of both ends]
    t_ds = (A + ep) * np.abs(ds) + p * (1 + A) * (t_d[:, None] + d * F * np.abs(G) @ np.abs(V).T)
    dk, t_dk = scale * ds.T @ Q, scale * t_ds.T @ np.abs(Q)
    got = np.concatenate([f64(b["dk"][:ends, 0]), f64(b["dk"][-ends:, 0])])
    assert (np.abs(got - dk) <= t_dk * (1 + 2.0 ** -10) + A * np.abs(dk) + 1e-30).all()
    assert (b["dq"] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_launches_behind_one_that_gave_up_are_right(d):
    """Blocks that gave up a wait have handed back their products, copies and tensor memory: the launches behind them in
    the stream, on the same SMs, are right."""
    seqs, hq, hk = packed(400, 130, 70), 8, 2
    good = Case(seqs, hq, hk, d, seed=6)
    bad = zl.zl_plan_causal(seqs, hq, hk, d, 600, 600, zl.ZL_PLAN_TEST_WITHHOLD_LOAD)
    b, (q, k, v, do) = zl.allocate_causal(bad, backward=True), good.dev
    for _ in range(3):
        zl.zl_causal_attn_fwd(bad, q, k, v, b["o"], b["lse"], b["workspace"], good.scale)
        good.forward()
        zl.zl_causal_attn_bwd(bad, q, k, v, good.bufs["o"], do, good.bufs["lse"], b["dq"], b["dk"], b["dv"], b["workspace"], good.scale)
        good.backward()
        assert zl.zl_causal_get_device_status(bad) == zl.ZL_ERR_TIMEOUT
    good.check()


def test_tiles_that_take_longer_than_a_wait_may():
    """152 tiles of 256 rows over 2^26 keys each: no range is split, and a tile takes longer (0.7 s) than a wait between two
    steps may.  Keys and values are zero, so O = 0 and LSE = ln of the keys seen."""
    import torch
    ensure_library()
    n, m, d = 152 * 256, 2 ** 26, 64
    plan = zl.zl_plan_causal([(0, n, 0, m)], 1, 1, d, n, m, zl.ZL_PLAN_FORWARD_ONLY)
    tiles = plan.tiles(0)
    assert all(t[5] < 0 for t in tiles) and len({t[6] for t in tiles}) == len(tiles) == 152
    zeros = torch.zeros(m, 1, d, dtype=torch.bfloat16, device="cuda")
    b = zl.allocate_causal(plan)
    b["o"].fill_(float("nan"))
    b["lse"].fill_(float("nan"))
    zl.zl_causal_attn_fwd(plan, zeros[:n], zeros, zeros, b["o"], b["lse"], b["workspace"], 0.125)
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(plan) == 0
    want = np.log(m - n + 1 + np.arange(n))
    assert (b["o"] == 0).all() and np.abs(f64(b["lse"])[:, 0] - want).max() <= 2.0 ** -20 * (1 + want.max())


def test_a_graph_outlives_its_plan():
    """A captured forward and gradient is replayed after its plan is gone and others have taken its place in memory; the
    plan goes once before the capture's end, once after."""
    import gc
    import torch
    seqs, hq, hk, d = [(0, 1, 0, 9000), (1, 40, 9000, 40)], 8, 2, 128
    for early in (False, True):
        c = Case(seqs, hq, hk, d, seed=12)
        c.forward().backward()  # whatever a kernel sets up at its first launch
        never_launched = zl.zl_plan_causal(seqs, hq, hk, d, 41, 9040)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.forward()
            never_launched.destroy()  # frees its memory at once, which must not spoil the capture
            c.backward()
            if early:
                c.plan.destroy()
        if not early:
            c.plan.destroy()
        for n in ("o", "lse", "dq", "dk", "dv"):
            c.bufs[n].fill_(float("nan"))
        others = [zl.zl_plan_causal(packed(*range(k, k + 40)), hq, hk, d, 4000, 4000) for k in range(1, 20)]
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        c.plan = zl.zl_plan_causal(seqs, hq, hk, d, 41, 9040)
        c.check()
        del g, others
        gc.collect()


def test_tables_of_graphs_and_plans_that_are_gone_are_freed():
    import gc
    import torch
    seqs, d = [(0, 1, 0, 2 ** 22)], 64  # 32 768 key tiles, tables of 1.6 MB
    k = torch.zeros(2 ** 22, 1, d, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(1, 1, d, dtype=torch.bfloat16, device="cuda")

    def once():
        plan = zl.zl_plan_causal(seqs, 1, 1, d, 1, 2 ** 22)
        b = zl.allocate_causal(plan)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            zl.zl_causal_attn_fwd(plan, q, k, k, b["o"], b["lse"], b["workspace"], 0.125)
        del plan
        g.replay()
        torch.cuda.synchronize()

    free = []
    for i in range(120):
        once()
        gc.collect()
        if i in (40, 119):
            torch.cuda.synchronize()
            torch.cuda.empty_cache()
            zl.zl_plan_causal([], 1, 1, d, 0, 0)
            free.append(torch.cuda.mem_get_info()[0])
    assert free[0] - free[1] < 32 * 2 ** 20  # 79 plans of 2 MB and more came and went


def test_rows_beyond_32_bit_offsets():
    """Queries, outputs and gradients behind 2^31 elements, in views of a fused projection: the same rows at offset 0 give
    the same bits (dQ within its bound), and the rows in front stay as they were; the rotation of all of them as well."""
    import torch
    lens, hq, hk, d, rows = (300, 1, 77), 16, 2, 128, 1_060_000
    c = Case(packed(*lens), hq, hk, d, seed=41).forward().backward()
    t, at = sum(lens), rows - sum(lens)
    assert at * hq * d > 2 ** 31
    fused = torch.full((rows, hq + 2 * hk, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    grads = torch.full_like(fused, float("nan"))
    o, do = (torch.full((rows, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cut = lambda x: [x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]]  # noqa: E731
    for dst, src in zip([*cut(fused), do], c.dev):
        dst[at:] = src
    plan = zl.zl_plan_causal([(q0 + at, n, k0 + at, m) for q0, n, k0, m in c.seqs], hq, hk, d, rows, rows)
    lse = torch.full((rows, hq), float("nan"), device="cuda")
    ws = torch.empty(max(plan.fwd_workspace_bytes, plan.bwd_workspace_bytes), dtype=torch.uint8, device="cuda")
    zl.zl_causal_attn_fwd(plan, *cut(fused), o, lse, ws, c.scale)
    zl.zl_causal_attn_bwd(plan, *cut(fused), o, do, lse, *cut(grads), ws, c.scale)
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(plan) == 0
    far = dict(zip(("o", "lse", "dq", "dk", "dv"), (o, lse, *cut(grads))))
    for n, x in far.items():
        assert n == "dq" or torch.equal(x[at:], c.bufs[n]), n
        assert all(torch.isnan(y).all() for y in x[:at].split(100_000)), n
        c.bufs[n].copy_(x[at:])
    c.check()
    table = zl.rotary_table(zl.rotary_frequencies(d)[0])
    pos = torch.arange(rows, device="cuda").int()[:, None]
    w = 1 + 0.2 * torch.randn(2, d, device="cuda")
    q, k, _ = cut(fused)
    gq, gk, _ = cut(grads)
    zl.zl_qk_rope_fwd(q, k, gq, gk, pos, table, True, w[0], w[1])
    near = torch.empty_like(fused[at:])
    zl.zl_qk_rope_fwd(q[at:], k[at:], *cut(near)[:2], pos[at:], table, True, w[0], w[1])
    assert torch.equal(grads[at:, :hq + hk], near[:, :hq + hk])
    zl.zl_qk_rope_bwd(q, k, gq, gk, gq, gk, pos, table, True, w[0], w[1])
    zl.zl_qk_rope_bwd(q[at:], k[at:], *cut(near)[:2], *cut(near)[:2], pos[at:], table, True, w[0], w[1])
    assert torch.equal(grads[at:, :hq + hk], near[:, :hq + hk])


@pytest.mark.parametrize("lens,hq,hk,d", [
    ((5000, 3000, 4100, 2900), 16, 8, 128), ((2600, 5000, 3000, 4100, 2600, 4999, 5001, 3000), 8, 8, 64)])
def test_large_batches(lens, hq, hk, d):
    """Batches that are launched plainly (100 us and more), whose tiles are taken sequence by sequence and many to a thread
    block, against the reference: all rows of some key heads."""
    import torch
    ensure_library()
    t, group, seqs, scale = sum(lens), hq // hk, packed(*lens), d ** -0.5
    ins = inputs(t, t, hq, hk, d, t)
    dev = [x.cuda() for x in ins]
    plan = zl.zl_plan_causal(seqs, hq, hk, d, t, t)
    for which in (0, 1):
        tiles = plan.tiles(which)
        per = [[x[4] - x[3] for x in tiles if x[6] == b] for b in range(152)]
        assert min(len(p) for p in per) >= 3 and all(x[5] < 0 for x in tiles)
        assert any(p != sorted(p, reverse=True) for p in per)  # not longest first over all
    b = zl.allocate_causal(plan, backward=True)
    zl.zl_causal_attn_fwd(plan, *dev[:3], b["o"], b["lse"], b["workspace"], scale)
    zl.zl_causal_attn_bwd(plan, *dev[:3], b["o"], dev[3], b["lse"], b["dq"], b["dk"], b["dv"], b["workspace"], scale)
    torch.cuda.synchronize()
    assert zl.zl_causal_get_device_status(plan) == 0
    for s, c in ((0, 0), (1, hk - 1), (len(lens) - 1, hk // 2)):
        q0, n, _, _ = seqs[s]
        hs, ks = slice(c * group, (c + 1) * group), slice(c, c + 1)
        part = [f64(x[q0:q0 + n, h]) for x, h in zip(ins, (hs, ks, ks, hs))]
        want, tol, var = bounds(*part, [(0, n, 0, n)], scale)
        for name in ("o", "lse", "dq", "dk", "dv"):
            got = f64(b[name][q0:q0 + n, ks if name in ("dk", "dv") else hs])
            over = np.abs(got - want[name]) - tol[name]
            assert over.max() <= 0, f"{name}: {over.max():.3e} over its bound"
            if name != "lse":
                off, rms = np.linalg.norm(got - want[name]), np.sqrt(var[name].sum())
                assert off <= (1.1 + 4 / np.sqrt(got.shape[0] * got.shape[1])) * rms, f"{name}: {off / rms:.2f} times the expected error"
