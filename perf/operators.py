"""Operators of causal sequences beside the coalesced attention engine, as measured cases.

Three operators, each in its directions:

  rope        rotary positions of queries and keys: interleaved or half layout, the whole head or
              its first part, one to three position axes, frequencies scaled for long contexts
  norm_rope   the same with an RMS norm of every head in the same pass (weights for queries and keys)
  attend      causal attention over packed sequences of different lengths with grouped heads, a
              prompt's chunk or a single token behind cached keys included; attend_step is the
              forward and its gradient

listed() and draw() give cases, prepare() the inputs, run() one pass: the framework's calls where
`own` is true, elementary torch operations where it is false.  exact() is the same in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------- cases
def _rope(op, tokens, q_heads, kv_heads, head_dim, rot_dim, layout, axes=1, scaling="none", far=0, grad=False):
    return {"op": op, "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rot_dim": rot_dim, "layout": layout, "axes": axes, "scaling": scaling, "far": far, "grad": grad}


def _attend(op, lens, q_heads, kv_heads, head_dim, past="", room=0):
    return {"op": op, "lens": lens, "past": past, "room": room, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim}


def listed():
    return [
        # one step of serving 16 sequences: their new tokens' queries and keys, far into a context whose
        # frequencies are scaled; latency is what counts
        {"name": "rope_serving_step", **_rope("rope", 16, 32, 8, 128, 128, "half", scaling="yarn", far=120000)},
        # a video clip's tokens (6 latent frames of 30x52 patches) turned by frame, row and column
        {"name": "rope_video", **_rope("rope", 9360, 20, 20, 128, 128, "interleaved", axes=3)},
        # a short prompt through the head norms and the rotation
        {"name": "norm_rope_short", **_rope("norm_rope", 100, 16, 2, 128, 128, "half")},
        # the token count of the mixed image and video batch, grouped heads
        {"name": "norm_rope_batch", **_rope("norm_rope", 49144, 32, 8, 128, 128, "half")},
        # gradient at an odd token count, small heads, a part of the head rotated
        {"name": "norm_rope_grad_odd", **_rope("norm_rope", 1025, 24, 8, 64, 32, "interleaved", grad=True)},
        # gradient of the video batch's norms and rotation by frame, row and column
        {"name": "norm_rope_grad_batch", **_rope("norm_rope", 49144, 20, 20, 128, 128, "interleaved", axes=3, grad=True)},
        # a handful of short sequences, one of a single token: latency
        {"name": "attend_short", **_attend("attend", "64,100,1,7", 4, 2, 64)},
        # packed sequences of the image batch's lengths and a one-token one
        {"name": "attend_packed", **_attend("attend", "256*8,1024*4,4096*2,1", 32, 8, 128)},
        # one new token for each of 64 sequences over caches of very different lengths
        {"name": "attend_single_tokens",
         **_attend("attend", "1*64", 32, 8, 128, past="16383*8,9001*16,4095*24,255*15,0", room=16384)},
        # one long prompt
        {"name": "attend_long", **_attend("attend", "16384", 32, 4, 128)},
        # a training step's attention, forward and gradient, over ragged lengths and small heads
        {"name": "attend_step_ragged", **_attend("attend_step", "1000,250,777,2048,33,1", 24, 8, 64)},
        # a training step's attention over long sequences
        {"name": "attend_step_long", **_attend("attend_step", "8192,4096,6007,8192", 16, 2, 128)},
    ]


HEADS = [(4, 4, 64), (4, 2, 64), (24, 8, 64), (20, 4, 64), (16, 2, 128), (8, 8, 128), (20, 20, 128), (28, 4, 128),
         (32, 4, 128), (32, 8, 128), (10, 1, 128), (6, 2, 128)]


def _log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    q_heads, kv_heads, head_dim = rng.choice(HEADS)
    op = rng.choice(["rope", "norm_rope", "norm_rope", "attend", "attend", "attend_step"])
    if op in ("rope", "norm_rope"):
        axes = rng.choice([1, 1, 3])
        parts = [head_dim, head_dim, head_dim // 2, head_dim // 4 * 3, head_dim // 4]
        return _rope(op, _log_size(rng, 1, 49144), q_heads, kv_heads, head_dim, rng.choice(parts),
                     rng.choice(["half", "interleaved"]), axes, "none" if axes == 3 else rng.choice(["none", "linear", "yarn"]),
                     0 if axes == 3 else _log_size(rng, 1, 1000000), rng.random() < 0.5)
    if op == "attend" and rng.random() < 0.6:  # new tokens behind cached ones
        batch = _log_size(rng, 1, 64)
        longest = _log_size(rng, 16, 16000)
        past = [rng.randint(0, longest) for _ in range(batch)]
        new = [1] * batch if rng.random() < 0.6 else [_log_size(rng, 1, 256) for _ in range(batch)]
        room = max(a + b for a, b in zip(past, new)) + rng.randint(0, 64)
        return _attend(op, ",".join(map(str, new)), q_heads, kv_heads, head_dim, ",".join(map(str, past)), room)
    # packed whole sequences; the padded plain form's scores stay below 2^32 bytes times four
    count = _log_size(rng, 1, 24)
    top = int(math.sqrt((2 ** 32 if op == "attend" else 2 ** 31) / (count * q_heads)))
    lens = [_log_size(rng, 1, min(top, 8192)) for _ in range(count)]
    if op == "attend_step":  # a lone token has no gradient but dv: a training batch holds at least one longer sequence
        lens[rng.randrange(count)] = _log_size(rng, 64, min(top, 8192))
    return _attend(op, ",".join(map(str, lens)), q_heads, kv_heads, head_dim)


def _numbers(text):
    out = []
    for part in text.split(","):
        if part:
            n, _, times = part.partition("*")
            out += [int(n)] * int(times or 1)
    return out


def _sequences(case):
    """[(first query row, queries, first key row, keys)] and the rows of queries and of keys."""
    lens = _numbers(case["lens"])
    past = _numbers(case["past"]) or [0] * len(lens)
    seqs, q0, k0 = [], 0, 0
    for n, p in zip(lens, past):
        seqs.append((q0, n, k0, n + p))
        q0 += n
        k0 += case["room"] or n + p
    return seqs, q0, k0


def _axis_pairs(case):
    pairs = case["rot_dim"] // 2
    if case["axes"] == 1:
        return [pairs]
    side = pairs * 3 // 8
    return [pairs - 2 * side, side, side]


def _frequencies(case):
    """Radians per position of every pair, in 64 bits, and the factor on the rotated values."""
    freqs = []
    for pairs in _axis_pairs(case):
        freqs += [BASE ** (-i / pairs) for i in range(pairs)]
    if case["scaling"] == "linear":  # positions pressed together eightfold
        freqs = [f / 8 for f in freqs]
    amplitude = 1.0
    if case["scaling"] == "yarn":
        # frequencies that turn less than once in the original 4096 positions are divided by the factor, those
        # that turn more than 32 times are kept, the ones between are blended
        factor, original, slow, fast = 16.0, 4096, 1.0, 32.0
        scaled = []
        for f in freqs:
            turns = original * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            scaled.append(f * keep + f / factor * (1 - keep))
        freqs, amplitude = scaled, 0.1 * math.log(factor) + 1
    return freqs, amplitude


def work(case):
    d, hq, hk = case["head_dim"], case["q_heads"], case["kv_heads"]
    if case["op"] in ("rope", "norm_rope"):
        values = case["tokens"] * (hq + hk) * d
        tensors = 3 if case["grad"] and case["op"] == "norm_rope" else 2
        flops = values * ((10 if case["grad"] else 4) if case["op"] == "norm_rope" else 0)
        return {"bytes": 2 * tensors * values + 4 * case["tokens"] * case["axes"],
                "flops": flops + 3 * case["tokens"] * (hq + hk) * case["rot_dim"]}
    seqs, tq, _ = _sequences(case)
    pairs, keys = 0, 0
    for _, n, _, m in seqs:
        pairs += n * m - n * (n - 1) // 2 if n <= m else m * (m + 1) // 2
        keys += m
    q, kv = 2 * tq * hq * d, 2 * 2 * keys * hk * d
    if case["op"] == "attend":
        return {"bytes": 2 * q + kv + 4 * tq * hq, "flops": 4 * d * hq * pairs}
    return {"bytes": 4 * q + 2 * kv + 4 * tq * hq, "flops": 14 * d * hq * pairs}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    d, hq, hk = case["head_dim"], case["q_heads"], case["kv_heads"]
    s = {"case": case}
    if case["op"] in ("rope", "norm_rope"):
        n = case["tokens"]
        # a projection's output: queries, keys and values of a token side by side, channels of unlike size
        qkv = (normal(n, hq + 2 * hk, d) * (0.5 + 1.5 * torch.rand(hq + 2 * hk, d, generator=g, device=DEVICE))).bfloat16()
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        if case["axes"] == 3:  # frames of 30 x 52 patches
            i = torch.arange(n, device=DEVICE)
            s["positions"] = torch.stack([i // 1560, i % 1560 // 52, i % 52], 1).int()
        else:
            first = torch.randint(0, case["far"] + 1, (), generator=g, device=DEVICE)
            s["positions"] = (first + torch.arange(n, device=DEVICE)).int()[:, None].contiguous()
        s["freqs"], s["amplitude"] = _frequencies(case)
        s["freqs64"] = torch.tensor(s["freqs"], dtype=torch.float64, device=DEVICE)
        s["pair_axis"] = torch.tensor([a for a, n_pairs in enumerate(_axis_pairs(case)) for _ in range(n_pairs)], device=DEVICE)
        if case["op"] == "norm_rope":
            s["q_weight"], s["k_weight"] = 1 + 0.2 * normal(d), 1 + 0.2 * normal(d)
        if case["grad"]:
            s["dq_out"], s["dk_out"] = normal(n, hq, d).bfloat16(), normal(n, hk, d).bfloat16()
        if own:
            from coalesced_packed_attention_gb300 import zl
            s["table"] = zl.rotary_table(s["freqs"], layout=case["layout"], axis_pairs=_axis_pairs(case),
                                         amplitude=s["amplitude"], device=DEVICE)
            s["q_res"], s["k_res"] = (torch.empty(n, h, d, dtype=torch.bfloat16, device=DEVICE) for h in (hq, hk))
            if case["grad"] and case["op"] == "norm_rope":
                s["dq_weight"], s["dk_weight"] = torch.empty(d, device=DEVICE), torch.empty(d, device=DEVICE)
                s["workspace"] = torch.empty(zl.zl_qk_rope_workspace_bytes(n, hq, hk, d), dtype=torch.uint8, device=DEVICE)
        return s
    seqs, tq, tk = _sequences(case)
    s["scale"] = d ** -0.5
    s["q"] = normal(tq, hq, d).bfloat16()
    if case["room"]:  # a cache: rows behind each sequence's last key are whatever was there
        s["k"], s["v"] = normal(tk, hk, d).bfloat16(), normal(tk, hk, d).bfloat16()
    else:  # rotated keys of their own, values still side by side with the projection's queries and keys
        s["k"] = normal(tk, hk, d).bfloat16()
        s["v"] = normal(tk, hq + 2 * hk, d).bfloat16()[:, hq + hk:]
    if case["op"] == "attend_step":
        s["d_o"] = normal(tq, hq, d).bfloat16()
    # rows of the padded batch, and each token's place in it
    n_most, m_most = max(x[1] for x in seqs), max(x[3] for x in seqs)
    q0, n, k0, m = (torch.tensor(x, device=DEVICE) for x in zip(*seqs))
    s["n"], s["m"] = n, m
    s["q_rows"] = (q0[:, None] + torch.arange(n_most, device=DEVICE)).clamp(max=tq - 1)
    s["k_rows"] = (k0[:, None] + torch.arange(m_most, device=DEVICE)).clamp(max=tk - 1)
    s["q_seq"] = torch.repeat_interleave(torch.arange(len(seqs), device=DEVICE), n)
    s["q_at"] = torch.arange(tq, device=DEVICE) - q0[s["q_seq"]]
    s["k_seq"] = torch.repeat_interleave(torch.arange(len(seqs), device=DEVICE), m)
    s["k_at"] = torch.cat([torch.arange(x[3], device=DEVICE) for x in seqs])
    if own:
        from coalesced_packed_attention_gb300 import zl
        s["plan"] = zl.zl_plan_causal(seqs, hq, hk, d, tq, tk)
        s["bufs"] = zl.allocate_causal(s["plan"], DEVICE, backward=case["op"] == "attend_step")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] in ("rope", "norm_rope"):
        return _plain_rope(s, case)
    return _plain_attend(s, case)


def _run_own(s, case):
    from coalesced_packed_attention_gb300 import zl
    if case["op"] == "rope":
        if case["grad"]:
            zl.zl_qk_rope_bwd(None, None, s["dq_out"], s["dk_out"], s["q_res"], s["k_res"], s["positions"], s["table"])
        else:
            zl.zl_qk_rope_fwd(s["q"], s["k"], s["q_res"], s["k_res"], s["positions"], s["table"])
        return {"q": s["q_res"], "k": s["k_res"]}
    if case["op"] == "norm_rope":
        if case["grad"]:
            zl.zl_qk_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["q_res"], s["k_res"], s["positions"], s["table"],
                              norm=True, q_weight=s["q_weight"], k_weight=s["k_weight"], dq_weight=s["dq_weight"],
                              dk_weight=s["dk_weight"], workspace=s["workspace"], eps=EPS)
            return {"q": s["q_res"], "k": s["k_res"], "q_weight": s["dq_weight"], "k_weight": s["dk_weight"]}
        zl.zl_qk_rope_fwd(s["q"], s["k"], s["q_res"], s["k_res"], s["positions"], s["table"], norm=True,
                          q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
        return {"q": s["q_res"], "k": s["k_res"]}
    b = s["bufs"]
    zl.zl_causal_attn_fwd(s["plan"], s["q"], s["k"], s["v"], b["o"], b["lse"], b["workspace"], s["scale"])
    if case["op"] == "attend":
        return {"o": b["o"], "lse": b["lse"]}
    zl.zl_causal_attn_bwd(s["plan"], s["q"], s["k"], s["v"], b["o"], s["d_o"], b["lse"], b["dq"], b["dk"], b["dv"],
                          b["workspace"], s["scale"])
    return {"o": b["o"], "lse": b["lse"], "dq": b["dq"], "dk": b["dk"], "dv": b["dv"]}


def _turn(x, cos, sin, rot, half):
    """The first `rot` values of every head turned pair by pair; cos and sin are [tokens, 1, rot / 2]."""
    head, rest = x[..., :rot], x[..., rot:]
    if half:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = head[..., 0::2], head[..., 1::2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _plain_rope(s, case):
    rot, half = case["rot_dim"], case["layout"] == "half"
    # angles in 64 bits: a far position times a frequency has no fraction left in 32
    angle = s["positions"][:, s["pair_axis"]].double() * s["freqs64"]
    cos = (angle.cos() * s["amplitude"]).float()[:, None]
    sin = (angle.sin() * s["amplitude"]).float()[:, None]
    if not case["grad"]:
        out = {}
        for name in ("q", "k"):
            x = s[name].float()
            if case["op"] == "norm_rope":
                x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s[name + "_weight"]
            out[name] = _turn(x, cos, sin, rot, half).bfloat16()
        return out
    out = {}
    for name in ("q", "k"):
        dy = _turn(s["d" + name + "_out"].float(), cos, -sin, rot, half)
        if case["op"] == "rope":
            out[name] = dy.bfloat16()
            continue
        x = s[name].float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        normed = x * r
        out[name + "_weight"] = (dy * normed).sum((0, 1))
        dn = dy * s[name + "_weight"]
        out[name] = (r * (dn - normed * (dn * normed).mean(-1, keepdim=True))).bfloat16()
    return out


def _plain_attend(s, case):
    hk, d = case["kv_heads"], case["head_dim"]
    group = case["q_heads"] // hk
    batch, n_most = s["q_rows"].shape
    m_most = s["k_rows"].shape[1]

    def queries(x):  # [sequences, key heads, queries * group, d]
        return x[s["q_rows"]].float().view(batch, n_most, hk, group, d).transpose(1, 2).reshape(batch, hk, n_most * group, d)

    def tokens(x):  # the packed rows of a padded [sequences, key heads, queries * group, e]
        e = x.shape[-1]
        x = x.view(batch, hk, n_most, group, e)[s["q_seq"], :, s["q_at"]]
        return x.reshape(len(s["q_at"]), hk * group, e)

    q, k, v = queries(s["q"]), s["k"][s["k_rows"]].float().transpose(1, 2), s["v"][s["k_rows"]].float().transpose(1, 2)
    # query i of n sees the keys up to m - n + i
    last = s["m"] - s["n"] + torch.arange(n_most, device=DEVICE)[:, None]
    unseen = torch.arange(m_most, device=DEVICE) > last.T[:, :, None]
    p = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(batch, hk, n_most, group, m_most)
    p.masked_fill_(unseen[:, None, :, None], -math.inf)
    p = p.view(batch, hk, n_most * group, m_most)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    lse = top + total.log()
    o = p @ v
    out = {"o": tokens(o).bfloat16(), "lse": tokens(lse)[..., 0]}
    if case["op"] == "attend":
        return out
    # queries that pad the batch have no gradient
    there = torch.arange(n_most, device=DEVICE) < s["n"][:, None]
    do = queries(s["d_o"]) * there[:, None, :, None].expand(batch, hk, n_most, group).reshape(batch, hk, -1, 1)
    dv = p.transpose(-1, -2) @ do
    ds = do @ v.transpose(-1, -2)
    ds.sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = ds @ k * s["scale"]
    dk = ds.transpose(-1, -2) @ q * s["scale"]
    out["dq"] = tokens(dq).bfloat16()
    out["dk"], out["dv"] = (x.transpose(1, 2)[s["k_seq"], s["k_at"]].bfloat16() for x in (dk, dv))
    return out


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s, case) if case["op"] in ("rope", "norm_rope") else _exact_attend(s, case)


def _exact_rope(s, case):
    rot, d = case["rot_dim"], case["head_dim"]
    # the rotation of a token as a d x d matrix acting on a head's values
    n = case["tokens"]
    first = torch.arange(rot // 2, device=DEVICE)
    a, b = (first, first + rot // 2) if case["layout"] == "half" else (2 * first, 2 * first + 1)
    out = {}
    sums = {"q": 0, "k": 0}
    parts = {"q": [], "k": []}
    for lo in range(0, n, 4096):
        hi = min(n, lo + 4096)
        angle, at = torch.empty(hi - lo, rot // 2, dtype=torch.float64, device=DEVICE), 0
        for axis, pairs in enumerate(_axis_pairs(case)):
            angle[:, at:at + pairs] = s["positions"][lo:hi, axis:axis + 1].double() * s["freqs64"][at:at + pairs]
            at += pairs
        turn = torch.zeros(hi - lo, d, d, dtype=torch.float64, device=DEVICE)
        rest = torch.arange(rot, d, device=DEVICE)
        turn[:, rest, rest] = 1
        turn[:, a, a] = turn[:, b, b] = torch.cos(angle) * s["amplitude"]
        turn[:, a, b] = -torch.sin(angle) * s["amplitude"]
        turn[:, b, a] = torch.sin(angle) * s["amplitude"]
        for name in ("q", "k"):
            x = s[name][lo:hi].double()
            if case["op"] == "norm_rope":
                w = s[name + "_weight"].double()
                mean = (x * x).sum(-1, keepdim=True) / d + EPS
                unit = x / mean.sqrt()
            if not case["grad"]:
                y = unit * w if case["op"] == "norm_rope" else x
                parts[name].append(y @ turn.transpose(1, 2))
                continue
            dy = s["d" + name + "_out"][lo:hi].double() @ turn
            if case["op"] == "norm_rope":
                sums[name] = sums[name] + (dy * unit).sum((0, 1))
                dy = dy * w
                dy = dy / mean.sqrt() - x * (dy * x).sum(-1, keepdim=True) / (d * mean ** 1.5)
            parts[name].append(dy)
    for name in ("q", "k"):
        out[name] = torch.cat(parts[name])
        if case["grad"] and case["op"] == "norm_rope":
            out[name + "_weight"] = sums[name]
    return out


def _exact_attend(s, case):
    seqs, tq, _ = _sequences(case)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    group, step = hq // hk, case["op"] == "attend_step"
    if 4 * d * hq * sum(x[1] * x[3] for x in seqs) * (3.5 if step else 1) > 1.2e13:
        return None  # more than some 20 seconds of products in 64 bits
    keys = sum(x[3] for x in seqs)
    o = torch.zeros(tq, hq, d, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(tq, hq, dtype=torch.float64, device=DEVICE)
    dq = torch.zeros_like(o) if step else None
    dk, dv = (torch.zeros(keys, hk, d, dtype=torch.float64, device=DEVICE) if step else None for _ in range(2))
    at = 0
    for q0, n, k0, m in seqs:
        for h in range(hk):
            k, v = s["k"][k0:k0 + m, h].double(), s["v"][k0:k0 + m, h].double()
            for c in range(h * group, (h + 1) * group):
                for lo in range(0, n, 8192):  # rows of queries at a time
                    hi = min(n, lo + 8192)
                    q = s["q"][q0 + lo:q0 + hi, c].double()
                    rows = torch.arange(lo, hi, device=DEVICE)[:, None]
                    scores = torch.where(torch.arange(m, device=DEVICE) <= m - n + rows, q @ k.T * s["scale"], -math.inf)
                    z = torch.logsumexp(scores, 1)
                    p = torch.exp(scores - torch.where(z == -math.inf, 0.0, z)[:, None])
                    lse[q0 + lo:q0 + hi, c] = z
                    o[q0 + lo:q0 + hi, c] = p @ v
                    if step:
                        do = s["d_o"][q0 + lo:q0 + hi, c].double()
                        dp = do @ v.T
                        ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                        dq[q0 + lo:q0 + hi, c] = ds @ k
                        dk[at:at + m, h] += ds.T @ q
                        dv[at:at + m, h] += p.T @ do
        at += m
    out = {"o": o, "lse": lse}
    if step:
        out.update(dq=dq, dk=dk, dv=dv)
    return out
