"""Operators of a key-value cache held in 4 bits, as measured cases.

Three paths, each over a paged cache whose rows are blocks of 16 channels with one scale:

  chunk    new keys and values enter the cache, and all that its sequences hold is read back as
           bf16 rows, as a prompt's next chunk needs it before its attention
  attend   attention of the newest tokens (one, or a few drafted ones) over the cache with grouped
           heads; with weights, what every slot received of it is added to its running sum
  evict    every head of a sequence keeps its most attended slots and its newest ones: survivors from
           behind move into the slots given up; then the rows kept are read

listed() and draw() give cases, prepare() the inputs, run() one pass: the framework's calls where
`own` is true, elementary torch operations where it is false.  exact() is the same in 64 bits.

The cache is uint8 [pages, key heads, page / 16, 18 d]: a tile of 16 slots holds the keys' codes
[16, d / 2], the values' codes, the keys' scales [16, d / 16], the values' scales.  A code is a sign, two
bits of exponent and one of mantissa (0, .5, 1, 1.5, 2, 3, 4, 6), channel 2j in the low half of a byte.
A scale has five bits of exponent and three of mantissa, no sign: the nearest to the block's
largest magnitude over 6.
"""
import math

import torch

own = False

DEVICE = "cuda"
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------- cases
def _case(op, lens, kv_heads, head_dim, page, new="", q_heads=0, weights=False, keep=0, recent=0):
    return {"op": op, "lens": lens, "new": new, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "weights": weights, "keep": keep, "recent": recent}


def listed():
    return [
        # the first tokens behind short prompts of 16 sequences: latency
        {"name": "chunk_short", **_case("chunk", "64*8,17*4,100*2,1*2", 2, 64, 16, new="1*16")},
        # the third chunk of two prompts and the whole of a short one, odd sizes
        {"name": "chunk_ragged", **_case("chunk", "1537,1025,33", 8, 64, 32, new="513,1,33")},
        # a packed batch of prompts (lengths of the image batch) entering an empty cache
        {"name": "chunk_batch", **_case("chunk", "256*8,1024*4,4096*2", 8, 128, 64, new="256*8,1024*4,4096*2")},
        # a chunk of four long prompts, most of each cached already
        {"name": "chunk_long", **_case("chunk", "16384*4", 8, 128, 128, new="1024*4")},
        # drafted tokens of a handful of sequences, one of which brings none: latency
        {"name": "attend_short", **_case("attend", "17,300,1,2049", 2, 64, 16, new="1,3,0,5", q_heads=4)},
        # one new token for each of 64 sequences over caches of very different lengths
        {"name": "attend_mixed",
         **_case("attend", "16384*8,9002*16,4096*24,256*15,1", 8, 128, 64, new="1*64", q_heads=32)},
        # one new token behind a very long context
        {"name": "attend_far", **_case("attend", "131071", 8, 128, 128, new="1", q_heads=32)},
        # a step of 48 sequences that live on a budget of slots, with the weights that eviction goes by
        {"name": "attend_budget", **_case("attend", "2049*48", 8, 128, 16, new="1*48", q_heads=32, weights=True)},
        # the last 16 tokens of ragged prompts look back: what eviction after a prompt goes by
        {"name": "attend_window", **_case("attend", "8192,3001,777,16,5000", 8, 64, 32, new="16*5", q_heads=24, weights=True)},
        # a step's eviction: one slot a head
        {"name": "evict_step", **_case("evict", "1025*8", 8, 128, 16, keep=1024, recent=128)},
        # one long prompt goes down to its budget
        {"name": "evict_prompt", **_case("evict", "16384", 4, 128, 64, keep=2048, recent=256)},
        # ragged prompts, some of which fit
        {"name": "evict_batch", **_case("evict", "8192*12,5000*9,2047*4,100*7", 8, 64, 64, keep=2048, recent=512)},
    ]


HEADS = [(4, 2, 64), (24, 8, 64), (20, 4, 64), (16, 2, 128), (8, 8, 128), (20, 20, 128), (28, 4, 128), (32, 4, 128),
         (32, 8, 128), (10, 1, 128), (6, 2, 128), (6, 6, 64)]


def _log_size(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    q_heads, kv_heads, head_dim = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128, 256])
    op = rng.choice(["chunk", "chunk", "attend", "attend", "attend", "evict"])
    # padded, the plain form holds every sequence at the longest one's size
    rows = {"chunk": 500000, "attend": 4000000, "evict": 1500000}[op] // kv_heads * 64 // head_dim
    batch = _log_size(rng, 1, 64)
    longest = _log_size(rng, 16, min(65536, max(16, rows // batch)))
    lens = [rng.choice([longest, rng.randint(1, longest), _log_size(rng, 1, longest)]) for _ in range(batch)]
    text = ",".join(map(str, lens))
    if op == "chunk":
        new = [rng.choice([m, rng.randint(0, m), min(m, 1)]) for m in lens]
        new[rng.randrange(batch)] = min(lens)  # at least one row
        return _case(op, text, kv_heads, head_dim, page, new=",".join(map(str, new)))
    if op == "attend":
        most = rng.choice([1, 1, 1, 4, 16])
        new = [min(m, rng.randint(1, most)) for m in lens]
        return _case(op, text, kv_heads, head_dim, page, new=",".join(map(str, new)), q_heads=q_heads,
                     weights=rng.random() < 0.4)
    keep = _log_size(rng, 8, longest)
    return _case(op, text, kv_heads, head_dim, page, keep=keep, recent=rng.randint(0, keep // 2))


def _numbers(text):
    out = []
    for part in text.split(","):
        if part:
            n, _, times = part.partition("*")
            out += [int(n)] * int(times or 1)
    return out


def work(case):
    d, hk, hq = case["head_dim"], case["kv_heads"], case["q_heads"]
    lens, new = _numbers(case["lens"]), _numbers(case["new"])
    held, plain = d + d // 8, 4 * d  # bytes of a head's key and value: codes and scales, bf16
    if case["op"] == "chunk":
        return {"bytes": hk * (sum(new) * (plain + held + 4) + (sum(lens) - sum(new)) * held + sum(lens) * plain),
                "flops": hk * d * (4 * sum(new) + 2 * sum(lens))}
    if case["op"] == "attend":
        pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(new, lens))
        extra = hk * (2 * sum(lens) - sum(new)) * 4 if case["weights"] else 0
        return {"bytes": hk * sum(lens) * held + sum(new) * hq * (4 * d + 4) + extra, "flops": 4 * d * hq * pairs}
    kept = [min(m, case["keep"]) for m in lens]
    # weights and positions in and out, what stays read out; the rows that move depend on the weights
    return {"bytes": hk * (8 * sum(lens) + 8 * sum(kept) + sum(kept) * (held + plain)), "flops": hk * (sum(lens) + 2 * d * sum(kept))}


# ---------------------------------------------------------------- the cache's format
def _scales(x):
    """The scale of every block of 16: x is fp32 [..., blocks, 16]."""
    q = x.abs().amax(-1, keepdim=True) / 6
    _, exponent = torch.frexp(q)
    # three bits behind the leading one, down to steps of 2^-17
    step = torch.ldexp(torch.ones_like(q), (exponent - 4).clamp(min=-17))
    return (torch.round(q / step) * step).clamp(max=8192.0)


def _levels(x, scales):
    """Index of the level nearest to |x| / scale, ties to the even one."""
    y = x.abs() / torch.where(scales == 0, 1.0, scales)
    at = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    for i in range(7):
        border = (LEVELS[i] + LEVELS[i + 1]) / 2
        at += (y >= border) if i % 2 else (y > border)
    return at * (scales != 0)


def _pack(k, v):
    """Rows of keys and values [tiles, 16, d] as the cache's tiles, uint8 [tiles, 18 d]."""
    codes, bits = [], []
    for x in (k, v):
        n, _, d = x.shape
        x = x.float().view(n, 16, d // 16, 16)
        s = _scales(x)
        c = (_levels(x, s) + 8 * (x < 0)).view(n, 16, d).to(torch.uint8)
        codes.append((c[..., 0::2] + 16 * c[..., 1::2]).reshape(n, -1))
        m, e = torch.frexp(s[..., 0])
        normal = 8 * (e + 14) + (m * 16).int() - 8
        bits.append(torch.where(s[..., 0] < 2.0 ** -14, (s[..., 0] * 2.0 ** 17).int(), normal).to(torch.uint8).reshape(n, -1))
    return torch.cat(codes + bits, 1)


def _unpack(tiles, d, table_type=torch.float32):
    """Keys and values [..., 16, d] of tiles [..., 18 d]."""
    level = torch.tensor(LEVELS + [-x for x in LEVELS], dtype=table_type, device=tiles.device)
    u = torch.arange(256, device=tiles.device)
    scale = torch.where(u < 8, (u * 2.0 ** -17).to(table_type), torch.ldexp((8 + u % 8).to(table_type), u // 8 - 18))
    lead, out = tiles.shape[:-1], []
    for i in range(2):
        codes = tiles[..., i * 8 * d:(i + 1) * 8 * d].view(*lead, 16, d // 2)
        bits = tiles[..., 16 * d + i * d:16 * d + (i + 1) * d].view(*lead, 16, d // 16, 1)
        x = torch.stack([level[(codes & 15).int()], level[(codes >> 4).int()]], -1)
        out.append((x.view(*lead, 16, d // 16, 16) * scale[bits.int()]).view(*lead, 16, d))
    return out


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    d, hq, hk, page = case["head_dim"], case["q_heads"], case["kv_heads"], case["page"]
    lens = _numbers(case["lens"])
    new = _numbers(case["new"]) or [0] * len(lens)
    batch = len(lens)
    s = {"case": case, "lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE)}
    # a pool of pages that is larger than what is used; every sequence's lie anywhere in it
    used = [-(-m // page) for m in lens]
    most = max(used)
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=g, device=DEVICE).int()
    table = torch.full((batch, most), -1, dtype=torch.int32, device=DEVICE)
    owner = torch.repeat_interleave(torch.arange(batch, device=DEVICE), torch.tensor(used, device=DEVICE))
    first = torch.tensor([sum(used[:b]) for b in range(batch)], device=DEVICE)
    index = torch.arange(sum(used), device=DEVICE)
    table[owner, index - first[owner]] = order[:sum(used)]
    s["pages"], s["slots"] = table, most * page
    s["data"] = torch.empty(n_pages, hk, page // 16, 18 * d, dtype=torch.uint8, device=DEVICE)
    tiles = s["data"].view(-1, 18 * d)
    size = 0.5 + 1.5 * torch.rand(2, d, generator=g, device=DEVICE)  # channels of unlike size
    for lo in range(0, tiles.shape[0], 32768):
        n = min(32768, tiles.shape[0] - lo)
        tiles[lo:lo + n] = _pack(normal(n, 16, d) * size[0], normal(n, 16, d) * size[1])
    n_new = sum(new)
    s["starts"] = torch.tensor([sum(new[:b]) for b in range(batch + 1)], dtype=torch.int32, device=DEVICE)
    s["token_seq"] = torch.repeat_interleave(torch.arange(batch, device=DEVICE), torch.tensor(new, device=DEVICE))
    s["token_at"] = torch.arange(n_new, device=DEVICE) - s["starts"].long()[s["token_seq"]]
    s["token_slot"] = s["lens"].long()[s["token_seq"]] - torch.tensor(new, device=DEVICE)[s["token_seq"]] + s["token_at"]
    if case["op"] == "attend":
        s["scale"] = d ** -0.5
        s["q"] = (normal(n_new, hq, d) * (0.5 + torch.rand(hq, d, generator=g, device=DEVICE))).bfloat16()
        s["max_new"], s["new"] = max(new), torch.tensor(new, device=DEVICE)
        s["q_rows"] = (s["starts"].long()[:-1, None] + torch.arange(max(new), device=DEVICE)).clamp(max=n_new - 1)
        if case["weights"]:
            s["weights"] = torch.exp(1.5 * normal(batch, hk, s["slots"]))
            s["weights_out"] = torch.zeros_like(s["weights"])
        if own:
            from coalesced_packed_attention_gb300 import zl
            s["cache"] = zl.Kv4Cache(s["data"], s["pages"], s["lens"])
            s["o"] = torch.empty(n_new, hq, d, dtype=torch.bfloat16, device=DEVICE)
            s["lse"] = torch.empty(n_new, hq, dtype=torch.float32, device=DEVICE)
            s["workspace"] = torch.empty(zl.zl_kv4_attn_workspace_bytes(s["cache"], hq, max_new=s["max_new"], weights=case["weights"]),
                                         dtype=torch.uint8, device=DEVICE)
        return s
    if case["op"] == "chunk":
        # keys of their own, values side by side with a projection's queries and keys
        s["k"] = (normal(n_new, hk, d) * size[0]).bfloat16()
        s["v"] = (normal(n_new, 3 * hk, d) * size[1]).bfloat16()[:, 2 * hk:]
        s["token_positions"] = s["token_slot"].int()
        s["positions"] = torch.zeros(batch, hk, s["slots"], dtype=torch.int32, device=DEVICE)
        kept = lens
    else:
        # some slots were never attended to
        w = torch.exp(2 * normal(batch, hk, s["slots"]))
        s["weights"] = torch.where(torch.rand(batch, hk, s["slots"], generator=g, device=DEVICE) < 0.1, 0.0, w)
        # earlier evictions left the older slots in any order
        s["positions"] = torch.rand(batch, hk, s["slots"], generator=g, device=DEVICE).argsort(-1).int()
        s["weights_out"], s["positions_out"] = torch.zeros_like(s["weights"]), torch.zeros_like(s["positions"])
        kept = [min(m, case["keep"]) for m in lens]
    s["row_starts"] = torch.tensor([sum(kept[:b]) for b in range(batch)], dtype=torch.int64, device=DEVICE)
    s["row_seq"] = torch.repeat_interleave(torch.arange(batch, device=DEVICE), torch.tensor(kept, device=DEVICE))
    s["row_slot"] = torch.arange(sum(kept), device=DEVICE) - s["row_starts"][s["row_seq"]]
    if own:
        from coalesced_packed_attention_gb300 import zl
        s["cache"] = zl.Kv4Cache(s["data"], s["pages"], s["lens"])
        s["k_rows"], s["v_rows"] = (torch.empty(sum(kept), hk, d, dtype=torch.bfloat16, device=DEVICE) for _ in range(2))
        if case["op"] == "evict":
            s["kept_lens"] = torch.empty_like(s["lens"])
            s["kept"] = zl.Kv4Cache(s["data"], s["pages"], s["kept_lens"])
            s["workspace"] = torch.empty(zl.zl_kv4_evict_workspace_bytes(s["cache"]), dtype=torch.uint8, device=DEVICE)
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"chunk": _plain_chunk, "attend": _plain_attend, "evict": _plain_evict}[case["op"]](s, case)


def _run_own(s, case):
    from coalesced_packed_attention_gb300 import zl
    if case["op"] == "chunk":
        zl.zl_kv4_write(s["cache"], s["k"], s["v"], starts=s["starts"], positions=s["token_positions"], slot_positions=s["positions"])
        zl.zl_kv4_read(s["cache"], s["k_rows"], s["v_rows"], s["row_starts"])
        return {"k": s["k_rows"], "v": s["v_rows"], "positions": s["positions"]}
    if case["op"] == "attend":
        if not case["weights"]:
            zl.zl_kv4_attn_fwd(s["cache"], s["q"], s["o"], s["lse"], s["workspace"], s["scale"], starts=s["starts"],
                               max_new=s["max_new"])
            return {"o": s["o"], "lse": s["lse"]}
        zl.zl_kv4_attn_fwd(s["cache"], s["q"], s["o"], s["lse"], s["workspace"], s["scale"], starts=s["starts"],
                           max_new=s["max_new"], weights=s["weights"], weights_out=s["weights_out"])
        return {"o": s["o"], "lse": s["lse"], "weights": s["weights_out"]}
    zl.zl_kv4_evict(s["cache"], s["weights"], s["positions"], case["keep"], case["recent"], s["workspace"],
                    weights_out=s["weights_out"], positions_out=s["positions_out"])
    torch.clamp(s["lens"], max=case["keep"], out=s["kept_lens"])
    zl.zl_kv4_read(s["kept"], s["k_rows"], s["v_rows"], s["row_starts"])
    return {"k": s["k_rows"], "v": s["v_rows"], "weights": s["weights_out"], "positions": s["positions_out"]}


def _held(s, case, type_=torch.float32):
    """Keys and values of every sequence, padded: [sequences, key heads, slots, d]."""
    d, hk = case["head_dim"], case["kv_heads"]
    tiles = s["data"][s["pages"].long().clamp(min=0)].transpose(1, 2)  # [sequences, key heads, pages, tiles, bytes]
    return [x.reshape(x.shape[0], hk, -1, d) for x in _unpack(tiles, d, type_)]


def _plain_chunk(s, case):
    d, hk, page = case["head_dim"], case["kv_heads"], case["page"]
    # the new tokens' rows as the cache will hold them
    out = {}
    held = _held(s, case)
    for name, old in zip(("k", "v"), held):
        x = s[name].float().view(-1, hk, d // 16, 16)
        scales = _scales(x)
        level = torch.tensor(LEVELS, device=DEVICE)[_levels(x, scales).int()]
        old[s["token_seq"], :, s["token_slot"]] = (torch.where(x < 0, -level, level) * scales).view(-1, hk, d)
        out[name] = old[s["row_seq"], :, s["row_slot"]].bfloat16()
    positions = s["positions"].clone()
    positions[s["token_seq"], :, s["token_slot"]] = s["token_positions"][:, None].expand(-1, hk)
    out["positions"] = positions
    return out


def _plain_attend(s, case):
    hk, d, hq = case["kv_heads"], case["head_dim"], case["q_heads"]
    group = hq // hk
    batch, n_most = s["q_rows"].shape
    k, v = _held(s, case)
    q = s["q"][s["q_rows"]].float().view(batch, n_most, hk, group, d).transpose(1, 2).reshape(batch, hk, n_most * group, d)
    # query i of n sees the slots up to len - n + i
    last = (s["lens"] - s["new"])[:, None] + torch.arange(n_most, device=DEVICE)
    unseen = torch.arange(s["slots"], device=DEVICE) > last[:, :, None]
    p = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(batch, hk, n_most, group, -1)
    p.masked_fill_(unseen[:, None, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    lse = top + total.log()
    o = p.view(batch, hk, n_most * group, -1) @ v
    o = o.view(batch, hk, n_most, group, d)[s["token_seq"], :, s["token_at"]]
    out = {"o": o.reshape(-1, hq, d).bfloat16(), "lse": lse[s["token_seq"], :, s["token_at"]].reshape(-1, hq)}
    if case["weights"]:
        there = torch.arange(n_most, device=DEVICE) < s["new"][:, None]
        got = (p * there[:, None, :, None, None]).sum((2, 3))
        slot = torch.arange(s["slots"], device=DEVICE)
        older = slot < (s["lens"] - s["new"])[:, None]  # a new token's slot begins with nothing
        w = torch.where(older[:, None], s["weights"], 0.0) + got
        out["weights"] = torch.where((slot < s["lens"][:, None])[:, None], w, 0.0)
    return out


def _plain_evict(s, case):
    keep, recent = case["keep"], case["recent"]
    slot = torch.arange(s["slots"], device=DEVICE)
    there = (slot < s["lens"][:, None])[:, None].expand_as(s["weights"])
    at = torch.where(there, s["positions"], -2 ** 31).long()
    newest = at.amax(-1, keepdim=True)
    # the newest positions first, then the largest weights, then the lowest slots
    w = torch.where(there, s["weights"], -math.inf)
    by_weight = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank_of = ((at > newest - recent) & there).long() * 2 + there.long()
    order = by_weight.gather(-1, torch.sort(rank_of.gather(-1, by_weight), dim=-1, descending=True, stable=True).indices)
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand_as(order).contiguous())
    kept = (rank < keep) & there
    # the slots given up in front take the survivors from behind, both in order
    hole = ~kept & (slot < keep) & there
    mover = kept & (slot >= keep)
    nth_hole, nth_mover = hole.long().cumsum(-1) - 1, mover.long().cumsum(-1) - 1
    movers = torch.zeros_like(order).scatter_(-1, torch.where(mover, nth_mover, s["slots"] - 1), torch.where(mover, slot, 0))
    source = torch.where(hole, movers.gather(-1, nth_hole.clamp(min=0)), slot)
    left = (slot < s["lens"].clamp(max=keep)[:, None])[:, None]
    out = {"weights": torch.where(left, s["weights"].gather(-1, source), 0.0),
           "positions": torch.where(left, s["positions"].gather(-1, source), 0)}
    for name, x in zip(("k", "v"), _held(s, case)):
        x = x.gather(2, source[..., None].expand_as(x))
        out[name] = x[s["row_seq"], :, s["row_slot"]].bfloat16()
    return out


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](s, case)


def _value64(bits, exponents, mantissas, bias):
    """The number that small unsigned floats stand for."""
    e, m = (bits >> mantissas) & (2 ** exponents - 1), (bits & (2 ** mantissas - 1)).double() / 2 ** mantissas
    return torch.where(e == 0, m * 2.0 ** (1 - bias), (1 + m) * torch.pow(2.0, (e - bias).double()))


def _sequence64(s, case, b, h):
    """Keys and values of one head of a sequence in 64 bits, from their bits."""
    d, m = case["head_dim"], int(s["lens"][b])
    rows = s["data"][s["pages"][b, :-(-m // case["page"])].long(), h].reshape(-1, 18 * d).long()
    out = []
    for i in range(2):
        codes = rows[:, 8 * d * i:8 * d * (i + 1)].reshape(-1, d // 2)
        nibbles = torch.empty(codes.shape[0], d, dtype=torch.long, device=DEVICE)
        nibbles[:, 0::2], nibbles[:, 1::2] = codes % 16, codes // 16
        size = _value64(nibbles % 8, 2, 1, 1) * torch.where(nibbles >= 8, -1.0, 1.0)
        scale = _value64(rows[:, 16 * d + i * d:16 * d + (i + 1) * d].reshape(-1, d // 16), 5, 3, 15)
        out.append((size * scale.repeat_interleave(16, 1))[:m])
    return out


def _nearest64(x):
    """Rows [tokens, heads, d] as the cache holds them, from the definition."""
    x = x.double().unflatten(-1, (-1, 16))
    want = x.abs().amax(-1) / 6
    scales = _value64(torch.arange(225, device=DEVICE), 5, 3, 15)  # ascending, up to 2^13

    def pick(values, table):  # nearest, ties to the even index
        hi = torch.searchsorted(table, values.contiguous()).clamp(1, len(table) - 1)
        lo = hi - 1
        below, above = values - table[lo], table[hi] - values
        return torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)

    scale = scales[pick(want, scales)][..., None]
    levels = _value64(torch.arange(8, device=DEVICE), 2, 1, 1)
    level = levels[pick(x.abs() / torch.where(scale == 0, math.inf, scale), levels)]
    return (torch.sign(x) * level * scale).flatten(-2)


def _exact_chunk(s, case):
    new = _numbers(case["new"])
    rows = {"k": [], "v": []}
    fresh = {"k": _nearest64(s["k"]), "v": _nearest64(s["v"])}
    positions, at = s["positions"].clone(), 0
    for b, n in enumerate(new):
        m = int(s["lens"][b])
        held = [_sequence64(s, case, b, h) for h in range(case["kv_heads"])]
        for i, name in enumerate(("k", "v")):
            x = torch.stack([kv[i] for kv in held], 1)
            x[m - n:] = fresh[name][at:at + n]
            rows[name].append(x)
        positions[b, :, m - n:m] = s["token_positions"][at:at + n]
        at += n
    return {"k": torch.cat(rows["k"]), "v": torch.cat(rows["v"]), "positions": positions}


def _exact_attend(s, case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    group, new, at = hq // hk, _numbers(case["new"]), 0
    o = torch.zeros(sum(new), hq, d, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(sum(new), hq, dtype=torch.float64, device=DEVICE)
    weights = torch.zeros(len(new), hk, s["slots"], dtype=torch.float64, device=DEVICE) if case["weights"] else None
    for b, n in enumerate(new):
        m = int(s["lens"][b])
        unseen = torch.arange(m, device=DEVICE) > m - n + torch.arange(n, device=DEVICE)[:, None]
        for h in range(hk):
            k, v = _sequence64(s, case, b, h)
            if weights is not None:
                weights[b, h, :m - n] = s["weights"][b, h, :m - n].double()
            for c in range(h * group, (h + 1) * group):
                scores = (s["q"][at:at + n, c].double() @ k.T * s["scale"]).masked_fill(unseen, -math.inf)
                z = torch.logsumexp(scores, 1)
                p = torch.exp(scores - z[:, None])
                o[at:at + n, c], lse[at:at + n, c] = p @ v, z
                if weights is not None:
                    weights[b, h, :m] += p.sum(0)
        at += n
    out = {"o": o, "lse": lse}
    if weights is not None:
        out["weights"] = weights
    return out


def _exact_evict(s, case):
    keep, recent, hk = case["keep"], case["recent"], case["kv_heads"]
    weights = torch.zeros(s["weights"].shape, dtype=torch.float64, device=DEVICE)
    positions = torch.zeros_like(s["positions"])
    rows = {"k": [], "v": []}
    for b, m in enumerate(_numbers(case["lens"])):
        heads = {"k": [], "v": []}
        for h in range(hk):
            w, at = s["weights"][b, h, :m].tolist(), s["positions"][b, h, :m].tolist()
            newest = max(at)
            ranked = sorted(range(m), key=lambda i: (at[i] <= newest - recent, -w[i], i))
            stays = set(ranked[:keep])
            movers = sorted(i for i in stays if i >= keep)
            source = [i if i in stays else movers.pop(0) for i in range(min(m, keep))]
            source = torch.tensor(source, device=DEVICE)
            n = len(source)
            weights[b, h, :n] = s["weights"][b, h, source].double()
            positions[b, h, :n] = s["positions"][b, h, source]
            for name, x in zip(("k", "v"), _sequence64(s, case, b, h)):
                heads[name].append(x[source])
        for name in heads:
            rows[name].append(torch.stack(heads[name], 1))
    return {"k": torch.cat(rows["k"]), "v": torch.cat(rows["v"]), "weights": weights, "positions": positions}
