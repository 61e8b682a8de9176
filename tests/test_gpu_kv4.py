"""The 4-bit cache on the GPU against the 64-bit reference.

Rows in and out are exact: codes and scales are those of exact arithmetic, and code * scale has six bits.
Attention, with the cache's values as given (F = 2^-24, q scaled by a power of two so that its row's largest is below 2):
  scores   d products in fp32, q in fp16 (exact but for what is below 2^-24 of the row's largest, half a step of that):
           e_s = scale (d F |q|.|k| + 2^-25 max|q| sum|k|);  P is off by e_p = e_s + max e_s + 2^-20 + 2^-22 |s|, relative
  O        P rounded to fp16 (2^-11, and 2^-25 of the row's maximum below its range) and off by that, m F of a sum over m slots,
           O rounded to bf16 (2^-8):   2^-8 |O| + (2^-11 + e_p + m F) P |V| + 2^-25 sum|V| / sum exp(s - max)
  LSE      max e_s + 2^-20 (1 + |LSE|) + m F
  weights  (rows + 1) F (|w| + sum P) + sum over rows of P (e_p + 2^-20 (1 + |LSE|) + m F): the product with decay and one addition
           a row, in any order, each off by F of a partial sum that |w| + sum P bounds (2^-22 |w| would be four of them:
           16 rows have 17)
"""
import numpy as np
import pytest

from coalesced_packed_attention_gb300 import zl
from oracle import kv4 as ref
from tests._lib import ensure_library

pytestmark = pytest.mark.gpu
F = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_library()


def f64(x):
    return x.double().cpu().numpy()


def make_cache(lens, heads, d, page, seed, spare=2, fill=True, extra_pages=0):
    """A cache whose sequences' pages lie anywhere, filled with rows of the format; numbers past a sequence's last slot are what
    no number is (scales of all ones)."""
    import torch
    rng = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    most = max(used + [1]) + extra_pages
    n_pages = sum(used) + spare
    order, at = rng.permutation(n_pages), 0
    pages = np.full((len(lens), most), -1, np.int64)
    for b, n in enumerate(used):
        pages[b, :n] = order[at:at + n]
        at += n
    data = np.full((n_pages, heads, page // 16, 18 * d), 255, np.uint8)
    if fill:
        tiles = rng.integers(0, 256, data.shape, np.uint8)
        tiles[..., 16 * d:] = rng.integers(12 * 8, 17 * 8, tiles[..., 16 * d:].shape)  # scales 2^-3 to 4
        for b, n in enumerate(lens):
            for s in range(0, n, 16):
                p, t, _ = ref.where(pages, page, b, s)
                data[p, :, t] = tiles[p, :, t]
            if n % 16:  # slots behind the last one of its tile
                p, t, _ = ref.where(pages, page, b, n - 1)
                for i in range(2):
                    data[p, :, t, 16 * d + i * d + n % 16 * (d // 16): 16 * d + (i + 1) * d] = 255
    c = zl.Kv4Cache(torch.from_numpy(data.copy()).cuda(), torch.from_numpy(pages).int().cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    return c, data, pages


def starts_of(new):
    import torch
    s = np.concatenate([[0], np.cumsum(new)])
    return s, torch.from_numpy(s).int().cuda()


# ---------------------------------------------------------------- rows in
@pytest.mark.parametrize("heads,d,page,lens,new", [
    (1, 64, 16, [1], [1]), (2, 128, 16, [16, 17, 15, 3], [16, 1, 15, 0]), (3, 64, 32, [100, 5, 64, 33], [37, 5, 64, 2]),
    (8, 128, 64, [130, 1, 257], [130, 1, 200]), (5, 128, 256, [300, 40], [299, 7]), (20, 128, 128, [129], [129])])
def test_write(heads, d, page, lens, new):
    import torch
    c, data, pages = make_cache(lens, heads, d, page, 1)
    starts, dstarts = starts_of(new)
    n = int(starts[-1])
    g = torch.Generator().manual_seed(2)
    # a projection's output: queries, keys and values of a token side by side; blocks of very different sizes
    qkv = torch.randn(n + 2, 4 * heads, d, generator=g) * torch.exp(3 * torch.randn(n + 2, 4 * heads, d // 16, generator=g)).repeat_interleave(16, 2)
    qkv = qkv.bfloat16().cuda()
    k, v = qkv[:, heads:2 * heads], qkv[:, 3 * heads:]
    pos = torch.arange(n + 2, dtype=torch.int32).cuda() * 7 - 3
    slot_pos = torch.full(c.slot_shape, -77, dtype=torch.int32).cuda()
    zl.zl_kv4_write(c, k, v, dstarts, pos, slot_pos)
    want = data.copy()
    ref.write(want, pages, lens, starts, f64(k), f64(v))
    got = c.data.cpu().numpy()
    assert np.array_equal(got[..., 16 * d:], want[..., 16 * d:])
    # codes: equal, but for the sign of 0
    for shift in (0, 4):
        a, b = got[..., :16 * d] >> shift & 15, want[..., :16 * d] >> shift & 15
        assert ((a == b) | ((a & 7 == 0) & (b & 7 == 0))).all()
    wp = np.full(c.slot_shape, -77)
    for b in range(len(lens)):
        for i in range(new[b]):
            wp[b, :, lens[b] - new[b] + i] = (starts[b] + i) * 7 - 3
    assert np.array_equal(slot_pos.cpu().numpy(), wp) and zl.zl_kv4_get_device_status(c) == 0


def test_write_ties_zeros_tiny_large_and_no_numbers():
    import torch
    d, rows = 64, []
    for s in (2.0 ** -17, 2.0 ** -15 * 1.125, 2.0 ** -9, 0.375, 1.0, 1.875, 2.0 ** 10, 2.0 ** 13):
        x = np.zeros(d)
        x[:16] = s * np.array([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -6, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5])
        x[16:32] = s * 6 * (1 + np.arange(16) / 16) / 2  # the scale's own borders
        x[32] = s * 6 * 17 / 16                          # a tie between two scales
        x[33:48] = s
        rows.append(x)
    for y in (2.0 ** -20, 2.0 ** -100, 1e30, -3e38, np.inf, -np.inf, np.nan):
        x = np.full(d, y)
        x[5], x[20] = 1.0, 0.0
        rows.append(x)
    x = torch.from_numpy(np.stack(rows)).bfloat16()[:, None].cuda()
    n = len(rows)
    c, data, pages = make_cache([n], 1, d, 16, 3)
    starts, dstarts = starts_of([n])
    zl.zl_kv4_write(c, x, x.flip(0), dstarts)
    want = data.copy()
    with np.errstate(invalid="ignore"):
        ref.write(want, pages, [n], starts, f64(x), f64(x.flip(0)))
    for s in range(n):
        for a, b in zip(ref.get_row(c.data.cpu().numpy(), pages, 0, 0, s), ref.get_row(want, pages, 0, 0, s)):
            assert np.array_equal(np.where(a == 8, 0, a) if len(a) == d else a, np.where(b == 8, 0, b) if len(b) == d else b), s


def test_write_every_quotient():
    """Every pair of a scale's and a channel's leading digits that bf16 has, at normal and at the smallest scales; every
    largest magnitude."""
    import torch
    rows = []
    for e in (0, -9, -14, -15, -17):
        for m in range(8, 16):
            s = m / 8 * 2.0 ** e
            if s * 2 ** 17 != np.floor(s * 2 ** 17):
                continue  # the smallest scales have fewer digits
            x = np.concatenate([np.arange(128, 256) / 128 * 2.0 ** (e + i) for i in range(-4, 3)])
            x = x[x <= 6 * s]
            x = np.concatenate([x, np.zeros(-len(x) % 15)]).reshape(-1, 15)
            rows.append(np.concatenate([np.full((len(x), 1), 6 * s), x], 1))
    blocks = np.concatenate(rows)
    top = np.arange(1, 0x7F80, dtype=np.uint32) << 16  # every bf16 number as a block's largest
    top = top.view(np.float32).astype(np.float64)
    more = np.zeros((len(top), 16))
    more[:, 3], more[:, 7] = -top, top / 2
    blocks = np.concatenate([blocks, more])
    blocks = np.concatenate([blocks, np.zeros((-len(blocks) % 4, 16))]).reshape(-1, 64)
    x = torch.from_numpy(blocks).bfloat16()[:, None].cuda()
    n = len(blocks)
    c = zl.allocate_kv4(1, -(-n // 256), 1, 64, page=256)
    c.lens.fill_(n)
    zl.zl_kv4_write(c, x, -x, torch.tensor([0, n], dtype=torch.int32).cuda())
    codes, bits = ref.encode(f64(x)[:, 0])
    tiles = c.data.cpu().numpy().reshape(-1, 18 * 64)
    got_bits = np.concatenate([tiles[:, 16 * 64 + i * 64:16 * 64 + (i + 1) * 64].reshape(-1, 4)[:n] for i in range(2)])
    assert np.array_equal(got_bits, np.concatenate([bits, bits]))
    k, v = torch.empty_like(x), torch.empty_like(x)
    zl.zl_kv4_read(c, k, v, torch.zeros(1, dtype=torch.int64).cuda())
    want = ref.decode(codes, bits)
    assert np.array_equal(f64(k)[:, 0], want) and np.array_equal(f64(v)[:, 0], -want)


def test_write_one_token_each_without_starts_and_odd_lengths():
    import torch
    lens = [1, 16, 17, 0, 48]  # a sequence of no slots has none for its token
    c, data, pages = make_cache(lens, 2, 128, 16, 4)
    x = torch.randn(5, 2, 128, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    zl.zl_kv4_write(c, x, -x)
    want = data.copy()
    ref.write(want, pages, lens, range(6), f64(x), -f64(x))
    got = c.data.cpu().numpy()
    for b, n in enumerate(lens):
        for h in range(2):
            for y, z in zip(ref.sequence(got, pages, b, h, n), ref.sequence(want, pages, b, h, n)):
                assert np.array_equal(y, z)
    assert zl.zl_kv4_get_device_status(c) == 0


# ---------------------------------------------------------------- rows out
@pytest.mark.parametrize("heads,d,page,lens", [
    (1, 64, 16, [1]), (2, 128, 16, [16, 17, 0, 3]), (3, 64, 32, [100, 0, 64, 33]), (8, 128, 64, [130, 1, 257]), (5, 128, 256, [300, 40]),
    (2, 64, 16, [3] * 300)])
def test_read(heads, d, page, lens):
    import torch
    c, data, pages = make_cache(lens, heads, d, page, 6)
    order = np.random.default_rng(7).permutation(len(lens))
    row, at = np.zeros(len(lens), np.int64), 1
    for b in order:  # sequences in any order, rows between them
        row[b] = at
        at += lens[b] + 1
    wide = torch.full((at, 3 * heads, d), 7.0, dtype=torch.bfloat16).cuda()
    k, v = wide[:, :heads], torch.full((at, heads, d), 7.0, dtype=torch.bfloat16).cuda()
    zl.zl_kv4_read(c, k, v, torch.from_numpy(row).cuda())
    wk, wv = np.full((at, heads, d), 7.0), np.full((at, heads, d), 7.0)
    for b, n in enumerate(lens):
        for h in range(heads):
            wk[row[b]:row[b] + n, h], wv[row[b]:row[b] + n, h] = ref.sequence(data, pages, b, h, n)
    assert np.array_equal(f64(k), wk) and np.array_equal(f64(v), wv)
    assert (wide[:, heads:] == 7.0).all() and zl.zl_kv4_get_device_status(c) == 0


def test_every_scale_and_code_reads_as_what_it_stands_for():
    import torch
    data = np.zeros((14, 1, 1, 18 * 64), np.uint8)
    codes = np.arange(16, dtype=np.uint8)
    tile = data[:, 0, 0]
    tile[:, :16 * 64] = np.tile(codes[0::2] + 16 * codes[1::2], 128)
    tile[:, 16 * 64:] = np.arange(14 * 128).reshape(14, 128) % 225
    pages = np.arange(14)[None]
    c = zl.Kv4Cache(torch.from_numpy(data).cuda(), torch.from_numpy(pages).int().cuda(), torch.tensor([224], dtype=torch.int32).cuda())
    k, v = torch.empty(224, 1, 64, dtype=torch.bfloat16).cuda(), torch.empty(224, 1, 64, dtype=torch.bfloat16).cuda()
    zl.zl_kv4_read(c, k, v, torch.zeros(1, dtype=torch.int64).cuda())
    wk, wv = ref.sequence(data, pages, 0, 0, 224)
    assert np.array_equal(f64(k)[:, 0], wk) and np.array_equal(f64(v)[:, 0], wv)


# ---------------------------------------------------------------- attention
def reference(q, data, pages, lens, starts, scale, w_in=None, decay=1.0):
    """Expected o, lse, weights and their bounds; rows of no sequence are NaN."""
    hq, heads, d = q.shape[1], data.shape[1], q.shape[2]
    group = hq // heads
    out = {"o": np.full(q.shape, np.nan), "lse": np.full(q.shape[:2], np.nan)}
    tol = {n: np.zeros_like(x) for n, x in out.items()}
    if w_in is not None:
        out["weights"], tol["weights"] = np.full(w_in.shape, np.nan), np.zeros(w_in.shape)
    for b, m in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        n = hi - lo
        for h in range(heads):
            k, v = ref.sequence(data, pages, b, h, m)
            k0, v0 = np.nan_to_num(k), np.nan_to_num(v)
            w = np.zeros(m)
            tw = np.zeros(m)
            if w_in is not None:
                w[:max(0, m - n)] = decay * w_in[b, h, :max(0, m - n)]
            start = np.abs(w)
            for c in range(h * group, (h + 1) * group):
                Q = q[lo:hi, c]
                p, o, lse = ref.attend_head(Q, k, v, scale)
                es = scale * (d * F * np.abs(Q) @ np.abs(k0).T + 2.0 ** -25 * np.abs(Q).max(1, initial=0, keepdims=True) * np.abs(k0).sum(1))
                es_row = es.max(1, initial=0.0, keepdims=True)
                s = np.abs(Q @ k0.T * scale)
                ep = es + es_row + 2.0 ** -20 + 2.0 ** -22 * s
                size = np.where(np.isfinite(lse), 1 + np.abs(np.where(np.isfinite(lse), lse, 0)), 0)
                out["o"][lo:hi, c], out["lse"][lo:hi, c] = o, lse
                top = p.max(1, initial=0.0)  # = 1 / sum exp(s - max)
                tol["o"][lo:hi, c] = 2.0 ** -8 * np.abs(o) + ((2.0 ** -11 + ep + m * F) * p) @ np.abs(v0) + \
                    2.0 ** -25 * top[:, None] * np.abs(v0).sum(0)
                tol["lse"][lo:hi, c] = es_row[:, 0] + 2.0 ** -20 * size + m * F
                w += p.sum(0)
                tw += (p * (ep + 2.0 ** -22 + (2.0 ** -20 * size)[:, None] + m * F)).sum(0)
            if w_in is not None:
                out["weights"][b, h, :m] = w
                tol["weights"][b, h, :m] = tw + (n * group + 1) * F * (start + np.abs(w) + start)
    return out, tol


def within(got, want, tol, what):
    seen = ~np.isnan(want)
    inf = np.isinf(want) & seen
    assert np.array_equal(got[inf], want[inf]), what
    seen &= ~inf
    off = np.abs(got[seen] - want[seen]) - tol[seen]
    assert np.isfinite(got[seen]).all() and (off <= 1e-30).all(), f"{what}: {off.max()} beyond its bound"


def run_attention(c, data, pages, lens, new, hq, seed, weights=False, decay=1.0, size=1.0, in_place=False, no_starts=False, lead=1):
    """One call and its check; rows before the first sequence's and behind the last one's stay as they were."""
    import torch
    d = c.token_shape[1]
    lead = 0 if no_starts else lead
    starts, _ = starts_of(new)
    starts = starts + lead
    total = int(starts[-1]) + 2 * (lead > 0)
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(total, 2 * hq, d, generator=g) * size).bfloat16().cuda()[:, hq:]  # a view: stride of two tensors
    o, lse = torch.full((total, hq, d), 7.0, dtype=torch.bfloat16).cuda(), torch.full((total, hq), 7.0).cuda()
    most, kw, w_in = max(new + [1]), {}, None
    if weights:
        w_in = torch.randn(c.slot_shape, generator=g).cuda()
        kw = dict(weights=w_in, weights_out=w_in.clone() if in_place else torch.full(c.slot_shape, 7.0).cuda(), decay=decay)
        if in_place:
            kw["weights"] = kw["weights_out"]
    ws = torch.full((zl.zl_kv4_attn_workspace_bytes(c, hq, most, weights),), 255, dtype=torch.uint8).cuda()
    ds = None if no_starts else torch.from_numpy(starts).int().cuda()
    scale = d ** -0.5
    zl.zl_kv4_attn_fwd(c, q, o, lse, ws, scale, ds, most, **kw)
    want, tol = reference(f64(q), data, pages, lens, starts, scale, f64(w_in) if weights else None, decay)
    assert zl.zl_kv4_get_device_status(c) & ~zl.ZL_KV4_BAD_PAGE == 0
    for name, x in (("o", o), ("lse", lse)):
        within(f64(x), want[name], tol[name], name)
        assert (f64(x)[np.isnan(want[name])] == 7.0).all(), name
    if weights:
        got = f64(kw["weights_out"])
        within(got, want["weights"], tol["weights"], "weights")
        left = np.isnan(want["weights"])
        assert np.array_equal(got[left], (f64(w_in) if in_place else np.full(got.shape, 7.0))[left])
    return o, lse


SHAPES = [(2, 1, 64), (4, 4, 64), (6, 2, 128), (8, 1, 128), (10, 1, 64), (16, 1, 128), (20, 4, 64), (7, 7, 128)]


@pytest.mark.parametrize("hq,heads,d", SHAPES)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attention_single_tokens(hq, heads, d, page):
    lens = [1, 15, 16, 17, 31, 33, 64, 200, 1000]
    c, data, pages = make_cache(lens, heads, d, page, 8)
    run_attention(c, data, pages, lens, [1] * len(lens), hq, 9, weights=page == 64, no_starts=page == 16)


@pytest.mark.parametrize("hq,heads,d", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_attention_several_tokens(hq, heads, d, weights):
    lens, new = [5, 40, 16, 300, 0, 3, 700], [5, 3, 0, 9, 0, 1, 6]
    c, data, pages = make_cache(lens, heads, d, 32, 10)
    run_attention(c, data, pages, lens, new, hq, 11, weights=weights, decay=0.5)


# Tables of up to 8192 slots and few items: a cluster of blocks takes an item.  Wider ones (entries past a sequence's slots are not
# read): units dealt out.
@pytest.mark.parametrize("hq,heads,d", SHAPES)
@pytest.mark.parametrize("weights", [False, True])
def test_attention_dealt_out(hq, heads, d, weights):
    lens, new = [5, 40, 16, 300, 0, 3, 700, 1500], [3, 3, 0, 2, 0, 1, 1, 1]
    c, data, pages = make_cache(lens, heads, d, 256, 54, extra_pages=33)
    assert c.slots > 8192
    run_attention(c, data, pages, lens, new, hq, 55, weights=weights, decay=0.5)


@pytest.mark.parametrize("hq,heads,d,n", [(4, 1, 128, 3), (8, 2, 64, 40), (16, 1, 64, 100), (9, 3, 128, 80), (2, 2, 128, 200), (6, 3, 64, 500)])
def test_attention_by_clusters_of_every_size(hq, heads, d, n):
    rng = np.random.default_rng(56)  # 8, 4 and 2 blocks an item, one, one for more items than there are blocks
    lens, new = [int(x) for x in rng.integers(0, 900, n)], [int(x) for x in rng.integers(0, 3, n)]
    c, data, pages = make_cache(lens, heads, d, 64, 57)
    a = run_attention(c, data, pages, lens, new, hq, 58, weights=n % 2 == 1)
    b = run_attention(c, data, pages, lens, new, hq, 58, weights=n % 2 == 1)
    import torch
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # bit for bit


@pytest.mark.parametrize("hq,heads,d,n", [(4, 1, 128, 30), (8, 2, 64, 60), (16, 1, 128, 200), (6, 3, 64, 300)])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_by_clusters_of_every_size(hq, heads, d, n, in_place):
    rng = np.random.default_rng(59)  # sequences without new tokens among them, whose sums decay all the same
    lens, new = [int(x) for x in rng.integers(0, 500, n)], [int(x) for x in rng.integers(0, 2 if hq > 8 else 3, n)]
    c, data, pages = make_cache(lens, heads, d, 16, 60)
    run_attention(c, data, pages, lens, new, hq, 61, weights=True, decay=0.75, in_place=in_place)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_more_queries_than_slots_and_none(d):
    lens, new = [0, 2, 0, 1], [2, 7, 1, 3]
    c, data, pages = make_cache(lens, 2, d, 16, 12)
    run_attention(c, data, pages, lens, new, 8, 13, weights=True)


@pytest.mark.parametrize("hq,heads,new", [(8, 2, [70, 1, 33]), (3, 1, [100, 40, 0])])
def test_attention_chunks_of_a_prompt(hq, heads, new):
    lens = [90, 500, 33]
    c, data, pages = make_cache(lens, heads, 128, 64, 14)
    run_attention(c, data, pages, lens, new, hq, 15, weights=True)


@pytest.mark.parametrize("d,weights", [(128, False), (64, True)])
def test_attention_one_long_sequence_is_cut_between_blocks(d, weights):
    lens = [20011]
    c, data, pages = make_cache(lens, 2, d, 128, 16)
    run_attention(c, data, pages, lens, [1], 8, 17, weights=weights, in_place=weights)
    run_attention(c, data, pages, lens, [5], 8, 18)


def test_attention_many_short_sequences():
    rng = np.random.default_rng(19)
    lens = [int(x) for x in rng.integers(0, 70, 700)]
    c, data, pages = make_cache(lens, 1, 64, 16, 20)
    run_attention(c, data, pages, lens, [1] * 700, 2, 21, no_starts=True)


@pytest.mark.parametrize("size", [1e-30, 30.0, 1e4])
def test_attention_scores_far_apart_and_queries_of_any_size(size):
    lens = [50, 333]
    c, data, pages = make_cache(lens, 2, 128, 16, 22)
    run_attention(c, data, pages, lens, [1, 2], 4, 23, size=size, weights=True)


def test_a_table_without_pages():
    import torch
    c = zl.Kv4Cache(torch.zeros(0, 2, 1, 18 * 64, dtype=torch.uint8).cuda(), torch.zeros(2, 0, dtype=torch.int32).cuda(),
                    torch.zeros(2, dtype=torch.int32).cuda())
    q, o, lse = torch.ones(2, 4, 64).bfloat16().cuda(), torch.full((2, 4, 64), 7.0).bfloat16().cuda(), torch.empty(2, 4).cuda()
    w = torch.empty(c.slot_shape).cuda()
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 4, 1, True), dtype=torch.uint8).cuda()
    zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1, weights_out=w)
    assert (o == 0).all() and (lse == -np.inf).all()
    k = torch.ones(2, 2, 64).bfloat16().cuda()
    zl.zl_kv4_write(c, k, k)
    zl.zl_kv4_read(c, k, k, torch.zeros(2, dtype=torch.int64).cuda())
    zl.zl_kv4_evict(c, w, w.int(), 3, 1, torch.empty(16, dtype=torch.uint8).cuda())
    assert zl.zl_kv4_get_device_status(c) == 0 and (k == 1).all()


def test_attention_repeats_bit_for_bit():
    import torch
    lens = [5000, 1, 777]
    c, data, pages = make_cache(lens, 2, 128, 64, 24)
    a = run_attention(c, data, pages, lens, [1, 1, 1], 8, 25)
    b = run_attention(c, data, pages, lens, [1, 1, 1], 8, 25)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_attention_leaves_out_bad_pages_and_says_so():
    import torch
    lens = [100, 64, 40]
    c, data, pages = make_cache(lens, 2, 64, 16, 26)
    pages[0, 2], pages[1, :], pages[2, 1] = -5, 10 ** 6, data.shape[0]  # the second sequence has no page at all
    c.pages.copy_(torch.from_numpy(pages).int())
    run_attention(c, data, pages, lens, [1, 1, 3], 4, 27, weights=True)
    c.status.zero_()
    q, o, lse = torch.ones(3, 4, 64).bfloat16().cuda(), torch.empty(3, 4, 64).bfloat16().cuda(), torch.empty(3, 4).cuda()
    zl.zl_kv4_attn_fwd(c, q, o, lse, torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 4), dtype=torch.uint8).cuda(), 0.1)
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_PAGE
    assert zl.zl_kv4_get_device_status(c) == 0 and (o[1] == 0).all() and (lse[1] == -np.inf).all()


# Many rows: from 33 rows a key head on, and rows x key heads x slots that the table has room for of 3 x 2^21 on, another kernel runs.
def many(lens, heads, d, page, seed, rows):
    """A cache whose table is wide enough for it (entries past a sequence's slots are not read)."""
    width = -(-3 * 2 ** 21 // (rows * heads * len(lens) * page))
    return make_cache(lens, heads, d, page, seed, extra_pages=max(0, width - max([-(-n // page) for n in lens] + [1])))


@pytest.mark.parametrize("hq,heads,d,new", [
    (8, 2, 64, [9, 1, 0, 16, 3, 2, 16, 5]), (7, 1, 128, [5, 3, 1, 0, 2, 4, 5, 1]), (3, 3, 128, [33, 1, 40, 7, 0, 2, 39, 31]),
    (32, 2, 64, [3, 0, 1, 2, 3, 1, 2, 3]), (6, 2, 128, [43, 1, 86, 20, 85, 3, 70, 128]), (128, 1, 64, [1] * 8), (100, 1, 128, [2] * 8)])
@pytest.mark.parametrize("page", [16, 128])
def test_attention_of_many_rows(hq, heads, d, new, page):
    lens = [300, 1, 128, 127, 0, 129, 700, 255]
    c, data, pages = many(lens, heads, d, page, 40, hq // heads * max(new))
    run_attention(c, data, pages, lens, new, hq, 41, no_starts=new == [1] * 8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [17, 64])
def test_attention_of_many_rows_of_one_long_sequence(d, new):
    import torch
    lens = [20011]  # cut between blocks; with 64 tokens in two tiles of rows
    c, data, pages = many(lens, 2, d, 64, 42, 4 * new)
    a = run_attention(c, data, pages, lens, [new], 8, 43)
    b = run_attention(c, data, pages, lens, [new], 8, 43)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # bit for bit


def test_attention_of_many_rows_of_many_sequences():
    rng = np.random.default_rng(44)
    lens, new = [int(x) for x in rng.integers(0, 400, 300)], [int(x) for x in rng.integers(0, 12, 300)]
    c, data, pages = many(lens, 1, 64, 16, 45, 4 * 11)
    run_attention(c, data, pages, lens, new, 4, 46)


@pytest.mark.parametrize("size", [1e-30, 30.0, 1e4])
def test_attention_of_many_rows_and_queries_of_any_size(size):
    lens, new = [50, 333, 4], [20, 7, 10]
    c, data, pages = many(lens, 2, 128, 16, 47, 40)
    run_attention(c, data, pages, lens, new, 4, 48, size=size)


def test_attention_of_many_rows_leaves_out_bad_pages_and_says_so():
    import torch
    lens, new = [300, 64, 140], [12, 9, 3]
    c, data, pages = many(lens, 2, 64, 16, 49, 48)
    pages[0, 2], pages[0, 8:16], pages[1, :], pages[2, 1] = -5, 10 ** 6, 10 ** 6, data.shape[0]
    c.pages.copy_(torch.from_numpy(pages).int())
    o, lse = run_attention(c, data, pages, lens, new, 8, 50)
    assert (o[13:22] == 0).all() and (lse[13:22] == -np.inf).all()  # the second sequence, which has no page at all


def test_attention_of_many_rows_captured_and_replayed_with_other_lengths():
    import torch
    lens, new = [513, 200, 130], [16, 11, 16]
    c, data, pages = many(lens, 2, 128, 64, 51, 64)
    starts, ds = starts_of(new)
    q = torch.randn(43, 8, 128, generator=torch.Generator().manual_seed(52)).bfloat16().cuda()
    o, lse = torch.empty_like(q), torch.empty(43, 8).cuda()
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 8, 16), dtype=torch.uint8).cuda()
    zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1, ds, 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1, ds, 16)
    for now in (lens, [257, 129, 16], [16, 0, 128]):
        c.lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        want, tol = reference(f64(q), data, pages, now, starts, 0.1)
        within(f64(o), want["o"], tol["o"], "o")
        within(f64(lse), want["lse"], tol["lse"], "lse")


def test_workspace_of_more_tokens_or_with_weights_serves_fewer_and_without():
    lens, new = [300, 64], [12, 9]
    c, data, pages = many(lens, 2, 64, 16, 53, 48)
    for more, weights in ((16, False), (12, True), (2000, False)):
        assert zl.zl_kv4_attn_workspace_bytes(c, 8, more, weights) >= zl.zl_kv4_attn_workspace_bytes(c, 8, 12)
    for most in (1, 4, 8, 9, 16):
        assert zl.zl_kv4_attn_workspace_bytes(c, 8, most) <= zl.zl_kv4_attn_workspace_bytes(c, 8, most + 1)


def test_bad_lengths_and_starts_are_left_out():
    import torch
    c, data, pages = make_cache([32, 32, 32], 1, 64, 16, 28)
    before = c.data.clone()
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 1, 2), dtype=torch.uint8).cuda()

    def outputs(n):
        return torch.full((n, 1, 64), 7.0, dtype=torch.bfloat16).cuda(), torch.full((n, 1), 7.0).cuda()

    x = torch.ones(4, 1, 64).bfloat16().cuda()
    for starts in ([0, 1, 9, 4], [-1, 0, 0, 0], [3, 1, 1, 1], [0, 3, 3, 3], [2 ** 31 - 1] * 4):
        o, lse = outputs(4)
        s = torch.tensor(starts, dtype=torch.int32).cuda()
        zl.zl_kv4_attn_fwd(c, x, o, lse, ws, 0.1, s, 2)
        if starts != [2 ** 31 - 1] * 4:
            assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_STARTS
        assert (o[2:] == 7.0).all()
    c.status.zero_()
    zl.zl_kv4_write(c, x, x, torch.tensor([0, 5, 1, 4], dtype=torch.int32).cuda())
    assert zl.zl_kv4_get_device_status(c) in (0, zl.ZL_KV4_BAD_STARTS)
    c.data.copy_(before)
    # lengths: as the nearest that there is
    c.lens.copy_(torch.tensor([-3, 10 ** 6, 32], dtype=torch.int32))
    o, lse = outputs(3)
    zl.zl_kv4_attn_fwd(c, x[:3], o, lse, ws, 0.1)
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_LEN
    want, tol = reference(f64(x[:3]), data, pages, [0, 32, 32], range(4), 0.1)
    within(f64(o), want["o"], tol["o"], "o")
    within(f64(lse), want["lse"], tol["lse"], "lse")
    k, v = torch.full((40, 1, 64), 7.0).bfloat16().cuda(), torch.full((40, 1, 64), 7.0).bfloat16().cuda()
    zl.zl_kv4_read(c, k, v, torch.tensor([0, 30, -1]).cuda())  # the second and third do not fit their rows
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_LEN | zl.ZL_KV4_BAD_STARTS and (k == 7.0).all()


# ---------------------------------------------------------------- eviction
def check_eviction(lens, heads, d, page, keep, recent, weights, positions, seed, in_place, table=0):
    import torch
    c, data, pages = make_cache(lens, heads, d, page, seed, extra_pages=max(0, table - max(-(-n // page) for n in lens)))
    w, pos = torch.from_numpy(weights).float().cuda(), torch.from_numpy(positions).int().cuda()
    wo, po = torch.full_like(w, 7.0), torch.full_like(pos, 7)
    if in_place:
        wo, po = w.clone(), pos.clone()
        w, pos = wo, po
    ws = torch.full((zl.zl_kv4_evict_workspace_bytes(c),), 255, dtype=torch.uint8).cuda()
    zl.zl_kv4_evict(c, w, pos, keep, recent, ws, wo, po)
    assert zl.zl_kv4_get_device_status(c) == 0
    want, want_w, want_p = data.copy(), np.full(weights.shape, 7.0, np.float32), np.full(positions.shape, 7)
    if in_place:
        want_w, want_p = weights.copy(), positions.copy()
    for b, n in enumerate(lens):
        for h in range(heads):
            m = min(n, keep)
            want_w[b, h, :m], want_p[b, h, :m] = weights[b, h, :m], positions[b, h, :m]
            if n == 0:
                continue
            for a, to in ref.evict_moves(weights[b, h, :n], positions[b, h, :n], keep, recent):
                ref.put_row(want, pages, b, h, to, ref.get_row(data, pages, b, h, a))
                want_w[b, h, to], want_p[b, h, to] = weights[b, h, a], positions[b, h, a]
    assert np.array_equal(wo.cpu().numpy(), want_w, equal_nan=True)
    assert np.array_equal(po.cpu().numpy(), want_p)
    assert np.array_equal(c.data.cpu().numpy(), want)
    if not in_place:  # once more leaves the same
        zl.zl_kv4_evict(c, w, pos, keep, recent, ws, wo, po)
        assert np.array_equal(c.data.cpu().numpy(), want) and np.array_equal(po.cpu().numpy(), want_p)


@pytest.mark.parametrize("heads,d,page,lens,keep,recent", [
    (1, 64, 16, [1], 1, 0), (2, 128, 16, [17, 16, 15, 1, 0], 16, 4), (3, 64, 32, [100, 33, 64], 32, 31), (2, 128, 64, [500, 129], 128, 0),
    (4, 64, 128, [3000], 777, 100), (1, 128, 256, [5000, 257], 1, 1), (2, 64, 16, [200], 64, 500), (2, 64, 16, [40, 50], 1000, 3)])
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("in_place", [False, True])
def test_eviction(heads, d, page, lens, keep, recent, kind, in_place):
    rng = np.random.default_rng(30)
    slots = max(1, -(-max(lens) // page)) * page
    shape = (len(lens), heads, slots)
    w = rng.exponential(size=shape).astype(np.float32)
    if kind == "ties":
        w = np.round(w * 2) / 2
    if kind == "odd":
        w = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-45, -1e-45, 3.0, -3.0], np.float32), shape)
    pos = np.argsort(rng.random(shape), -1)
    check_eviction(lens, heads, d, page, keep, recent, w.astype(np.float32), pos, 31, in_place)


@pytest.mark.parametrize("slots,keep", [(20011, 5003), (60000, 200), (230000, 129)])
def test_eviction_of_long_sequences(slots, keep):
    """Eight blocks a head; past 196 608 slots a run does not fit a block's shared memory."""
    rng = np.random.default_rng(47)
    lens = [slots, slots // 7, keep + 2]
    shape = (3, 1, -(-slots // 256) * 256)
    w = np.round(rng.exponential(size=shape) * 64).astype(np.float32)
    pos = np.argsort(rng.random(shape), -1)
    check_eviction(lens, 1, 64, 256, keep, 50, w, pos, 48, False)


@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("keep,recent", [(64, 0), (64, 5), (64, 64), (64, 100), (2, 1)])
def test_eviction_of_a_few_slots(kind, keep, recent):
    """One to six more than are kept, in a table with and without room for many moves."""
    rng = np.random.default_rng(45)
    lens = [keep + i for i in (1, 2, 3, 4, 5, 6, 0)]
    for slots, in_place in ((80, False), (80, True), (640, False)):
        shape = (len(lens), 2, slots)
        w = rng.exponential(size=shape)
        if kind == "ties":
            w = np.round(w)
        if kind == "odd":
            w = rng.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 3.0, -3.0]), shape)
        pos = np.argsort(rng.random(shape), -1) - 40
        check_eviction(lens, 2, 64, 16, keep, recent, w.astype(np.float32), pos, 46, in_place, table=slots // 16)


def test_eviction_among_equal_weights_and_extreme_positions():
    w = np.zeros((1, 1, 64), np.float32)
    pos = np.arange(64)[None, None] * 1000 - 2 ** 31
    check_eviction([64], 1, 64, 16, 20, 2 ** 31 - 1, w, pos, 32, False)  # all are recent: the lowest slots
    pos[0, 0, 10] = 2 ** 31 - 1
    check_eviction([64], 1, 64, 16, 20, 5, w, pos, 33, False)
    check_eviction([64], 1, 64, 16, 63, 0, w, pos, 34, True)


def test_eviction_of_bad_pages_moves_no_rows_of_them():
    import torch
    c, data, pages = make_cache([64], 1, 64, 16, 35)
    pages[0, 3] = -1
    c.pages.copy_(torch.from_numpy(pages).int())
    w, pos = torch.arange(64.).view(1, 1, 64).cuda(), torch.arange(64, dtype=torch.int32).view(1, 1, 64).cuda()
    zl.zl_kv4_evict(c, w, pos, 40, 0, torch.empty(zl.zl_kv4_evict_workspace_bytes(c), dtype=torch.uint8).cuda())
    assert zl.zl_kv4_get_device_status(c) == zl.ZL_KV4_BAD_PAGE
    want = data.copy()
    for a, to in ref.evict_moves(np.arange(64.), np.arange(64), 40, 0):
        if a < 48:
            ref.put_row(want, pages, 0, 0, to, ref.get_row(data, pages, 0, 0, a))
    assert np.array_equal(c.data.cpu().numpy(), want)


# ---------------------------------------------------------------- together, graphs, streams
def test_steps_on_a_budget_as_one_captured_graph():
    """Write, attend and evict, replayed as lengths grow and are cut back, against the same steps by the reference."""
    import torch
    heads, hq, d, page, keep, recent, B = 2, 8, 64, 16, 40, 8, 3
    lens = [38, 5, 40]
    c, data, pages = make_cache(lens, heads, d, page, 36, extra_pages=2)
    pages[:] = np.arange(pages.size).reshape(pages.shape)
    big = np.zeros((pages.size, *data.shape[1:]), np.uint8)
    big[...] = np.random.default_rng(37).integers(0, 256, big.shape, np.uint8)
    big[..., 16 * d:] = 15 * 8
    c = zl.Kv4Cache(torch.from_numpy(big).cuda(), torch.from_numpy(pages).int().cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    k, v, q = (torch.empty(B, h, d, dtype=torch.bfloat16).cuda() for h in (heads, heads, hq))
    at = torch.tensor(lens, dtype=torch.int32).cuda()
    w, pos = torch.rand(c.slot_shape).cuda(), torch.arange(c.slots, dtype=torch.int32).expand(c.slot_shape).contiguous().cuda()
    o, lse = torch.empty(B, hq, d, dtype=torch.bfloat16).cuda(), torch.empty(B, hq).cuda()
    ws = torch.empty(max(zl.zl_kv4_attn_workspace_bytes(c, hq, 1, True), zl.zl_kv4_evict_workspace_bytes(c)), dtype=torch.uint8).cuda()

    def step():
        c.lens.add_(1)
        zl.zl_kv4_write(c, k, v, positions=at, slot_positions=pos)
        zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.125, weights=w, weights_out=w)
        zl.zl_kv4_evict(c, w, pos, keep, recent, ws)
        c.lens.clamp_(max=keep)
        at.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [x.clone() for x in (c.data, c.lens, at, w, pos)]
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((c.data, c.lens, at, w, pos), state):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    g = torch.Generator().manual_seed(38)
    for i in range(6):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g))
        before = c.data.cpu().numpy()
        old_lens, old_at = c.lens.cpu().numpy(), at.cpu().numpy()
        old_w, old_pos = w.cpu().numpy(), pos.cpu().numpy()
        graph.replay()
        torch.cuda.synchronize()
        n = old_lens + 1
        ref.write(before, pages, n, range(B + 1), f64(k), f64(v))
        want, tol = reference(f64(q), before, pages, n, range(B + 1), 0.125, old_w.astype(np.float64))
        within(f64(o), want["o"], tol["o"], "o")
        within(f64(lse), want["lse"], tol["lse"], "lse")
        # eviction goes by the weights that the step left: from the kernel's own where its order is the reference's
        for b in range(B):
            old_pos[b, :, n[b] - 1] = old_at[b]
            for h in range(heads):
                moves = ref.evict_moves(want["weights"][b, h, :n[b]], old_pos[b, h, :n[b]], keep, recent)
                exp_w, exp_p = want["weights"][b, h, :n[b]].copy(), old_pos[b, h, :n[b]].copy()
                rows = [ref.sequence(before, pages, b, h, n[b])]
                kk, vv = rows[0]
                for a, to in moves:
                    exp_w[to], exp_p[to], kk[to], vv[to] = exp_w[a], exp_p[a], kk[a], vv[a]
                m = min(n[b], keep)
                assert np.array_equal(pos.cpu().numpy()[b, h, :m], exp_p[:m]), (i, b, h)
                assert np.abs(w.cpu().numpy()[b, h, :m] - exp_w[:m]).max() <= 2 * tol["weights"][b, h, :n[b]].max()
                gk, gv = ref.sequence(c.data.cpu().numpy(), pages, b, h, m)
                assert np.array_equal(gk, kk[:m]) and np.array_equal(gv, vv[:m])
        assert np.array_equal(c.lens.cpu().numpy(), np.minimum(n, keep))
    assert zl.zl_kv4_get_device_status(c) == 0


def test_prompt_through_the_cache_and_the_causal_attention():
    """A prompt's chunks enter the cache, are read back and attended as rows; the last tokens' attention over the cache
    itself is the same."""
    import torch
    heads, hq, d = 2, 8, 128
    c = zl.allocate_kv4(2, 8, heads, d, page=32)
    chunks = [[40, 100], [60, 7]]
    g = torch.Generator().manual_seed(39)
    total = [0, 0]
    for new in chunks:
        n = sum(new)
        q, k, v = (torch.randn(n, h, d, generator=g).bfloat16().cuda() for h in (hq, heads, heads))
        total = [a + b for a, b in zip(total, new)]
        c.lens.copy_(torch.tensor(total, dtype=torch.int32))
        s, ds = starts_of(new)
        zl.zl_kv4_write(c, k, v, ds)
        rows = torch.tensor([0, total[0]])
        seqs = [(int(s[b]), new[b], int(rows[b]), total[b]) for b in range(2)]
        plan = zl.zl_plan_causal(seqs, hq, heads, d, n, sum(total), zl.ZL_PLAN_FORWARD_ONLY)
        bufs = zl.allocate_causal(plan)
        kr, vr = (torch.empty(sum(total), heads, d, dtype=torch.bfloat16).cuda() for _ in range(2))
        zl.zl_kv4_read(c, kr, vr, rows.cuda())
        zl.zl_causal_attn_fwd(plan, q, kr, vr, bufs["o"], bufs["lse"], bufs["workspace"], d ** -0.5)
        o, lse = torch.empty_like(bufs["o"]), torch.empty_like(bufs["lse"])
        ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, hq, max(new)), dtype=torch.uint8).cuda()
        zl.zl_kv4_attn_fwd(c, q, o, lse, ws, d ** -0.5, ds, max(new))
        data, pages = c.data.cpu().numpy(), c.pages.cpu().numpy()
        want, tol = reference(f64(q), data, pages, total, s, d ** -0.5)
        within(f64(o), want["o"], tol["o"], "o")
        within(f64(lse), want["lse"], tol["lse"], "lse")
        # P is bf16 there: half a step more of every weight
        assert np.abs(f64(bufs["o"]) - want["o"]).max() <= (tol["o"] + 2.0 ** -8 * np.abs(v.float().cpu().numpy()).max() * 2).max()
        assert np.abs(f64(bufs["lse"]) - want["lse"]).max() <= 1e-4


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("on_stream", [False, True])
def test_projection_to_output_through_the_cache(norm, on_stream):
    """Three steps from a projection's output, the last on a budget, against the operators one by one in 64 bits."""
    import torch
    from oracle import causal
    heads, hq, d, page, B = 2, 6, 64, 16, 3
    c = zl.allocate_kv4(B, 5, heads, d, page=page)
    freqs, amplitude = zl.rotary_frequencies(d)
    table = zl.rotary_table(freqs, amplitude=amplitude)
    g = torch.Generator().manual_seed(50)
    qw, kw = ((1 + 0.1 * torch.randn(d, generator=g)).cuda() if norm else None for _ in range(2))
    total = np.zeros(B, int)
    data, pages = c.data.cpu().numpy(), c.pages.cpu().numpy()
    stream = torch.cuda.Stream() if on_stream else None
    w = np.zeros(c.slot_shape)
    for new, keep in (([20, 37, 5], None), ([1, 1, 0], None), ([3, 1, 2], 30)):
        n = sum(new)
        s, ds = starts_of(new)
        qkv = torch.randn(n, hq + 2 * heads, d, generator=g).bfloat16().cuda()
        total = total + new
        pos = np.concatenate([np.arange(total[b] - new[b], total[b]) for b in range(B)])
        bufs = zl.allocate_kv4_attention(c, n, hq, max(new), evicts=keep is not None)
        if keep is not None:
            bufs["positions"].copy_(torch.arange(c.slots, dtype=torch.int32))
            bufs["weights"].copy_(torch.rand(c.slot_shape, generator=g))
            w = f64(bufs["weights"])
        c.lens.copy_(torch.from_numpy(total).int())
        dpos = torch.from_numpy(pos).int().cuda()
        torch.cuda.synchronize()
        zl.qkv_attention_cached(c, qkv, dpos, table, d ** -0.5, bufs, qw, kw, starts=ds, max_new=max(new), keep=keep, recent=4,
                                stream=stream)
        torch.cuda.synchronize()
        # rotation within its own rounding; from there on with the rows that it left
        ang = causal.angles(pos[:, None], freqs, [d // 2])
        for x, y, weight in ((qkv[:, :hq], bufs["q"], qw), (qkv[:, hq:hq + heads], bufs["k"], kw)):
            want = f64(x)
            if norm:
                want = causal.rms_norm(want, f64(weight), 1e-6)
            want = causal.rotate(want, ang, True) * amplitude
            assert np.abs(f64(y) - want).max() <= 2.0 ** -7 * (1 + np.abs(want).max())
        ref.write(data, pages, total, s, f64(bufs["k"]), f64(qkv[:, hq + heads:]))
        want, tol = reference(f64(bufs["q"]), data, pages, total, s, d ** -0.5, w if keep is not None else None)
        within(f64(bufs["o"]), want["o"], tol["o"], "o")
        within(f64(bufs["lse"]), want["lse"], tol["lse"], "lse")
        if keep is not None:
            for b in range(B):
                for h in range(heads):
                    order = want["weights"][b, h, :total[b]]
                    for a, to in ref.evict_moves(order, np.arange(total[b]), keep, 4):
                        ref.put_row(data, pages, b, h, to, ref.get_row(data, pages, b, h, a))
            assert np.array_equal(c.lens.cpu().numpy(), np.minimum(total, keep))
        got = c.data.cpu().numpy()
        for b in range(B):
            for h in range(heads):
                m = total[b] if keep is None else min(total[b], keep)
                for y, z in zip(ref.sequence(got, pages, b, h, m), ref.sequence(data, pages, b, h, m)):
                    assert np.array_equal(y, z)
    assert zl.zl_kv4_get_device_status(c) == 0
    with pytest.raises(ValueError):
        zl.qkv_attention_cached(c, qkv[:, :2 * heads], dpos, table, 0.1, bufs)
    with pytest.raises(ValueError):
        zl.qkv_attention_cached(c, qkv, dpos, table, 0.1, zl.allocate_kv4_attention(c, n, hq, 3), starts=ds, max_new=3, keep=3)


def test_calls_on_other_streams_at_once():
    import torch
    lens = [3000, 10]
    c, data, pages = make_cache(lens, 2, 128, 64, 40)
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(41)).bfloat16().cuda()
    outs = []
    torch.cuda.synchronize()
    for _ in range(4):
        s = torch.cuda.Stream()
        o, lse = torch.empty(2, 8, 128, dtype=torch.bfloat16).cuda(), torch.empty(2, 8).cuda()
        ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 8), dtype=torch.uint8).cuda()
        torch.cuda.synchronize()
        outs.append((o, lse, s, ws))
    for o, lse, s, ws in outs:
        zl.zl_kv4_attn_fwd(c, q, o, lse, ws, 0.1, stream=s)
    torch.cuda.synchronize()
    want, tol = reference(f64(q), data, pages, lens, range(3), 0.1)
    for o, lse, _, _ in outs:
        within(f64(o), want["o"], tol["o"], "o")
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_offsets_past_32_bits():
    """Pages behind 2^32 bytes of the cache, and rows behind 2^31 elements of what is read."""
    import torch
    d, heads, page = 128, 8, 256
    n_pages = 2 ** 33 // (heads * page // 16 * 18 * d) + 8
    data = torch.empty(n_pages, heads, page // 16, 18 * d, dtype=torch.uint8, device="cuda")
    pages = torch.tensor([[n_pages - 1, 0], [n_pages - 3, n_pages - 2]], dtype=torch.int32).cuda()
    lens = [300, 290]
    c = zl.Kv4Cache(data, pages, torch.tensor(lens, dtype=torch.int32).cuda())
    k = torch.randn(590, heads, d, generator=torch.Generator().manual_seed(42)).bfloat16().cuda()
    s, ds = starts_of(lens)
    zl.zl_kv4_write(c, k, -k, ds)
    rows = 2 ** 31 // (heads * d) + 700
    ko, vo = (torch.empty(rows, heads, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    first = torch.tensor([rows - 300, rows - 640])
    zl.zl_kv4_read(c, ko, vo, first.cuda())
    for b, n in enumerate(lens):
        want = ref.decode(*ref.encode(f64(k[s[b]:s[b + 1]])))
        assert np.array_equal(f64(ko[first[b]:first[b] + n]), want) and np.array_equal(f64(vo[first[b]:first[b] + n]), -want)
    q = torch.randn(2, 8, d, generator=torch.Generator().manual_seed(43)).bfloat16().cuda()
    o, lse = torch.empty_like(q), torch.empty(2, 8).cuda()
    zl.zl_kv4_attn_fwd(c, q, o, lse, torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 8), dtype=torch.uint8).cuda(), 0.1)
    small = c.data[[n_pages - 1, 0, n_pages - 3, n_pages - 2]].cpu().numpy()
    want, tol = reference(f64(q), small, np.array([[0, 1], [2, 3]]), lens, range(3), 0.1)
    within(f64(o), want["o"], tol["o"], "o")
    within(f64(lse), want["lse"], tol["lse"], "lse")
    assert zl.zl_kv4_get_device_status(c) == 0


def test_tensors_that_are_not_the_cache_s_are_refused():
    import torch
    c, _, _ = make_cache([32, 32], 2, 64, 16, 44)
    q, o, lse = torch.ones(2, 4, 64).bfloat16().cuda(), torch.empty(2, 4, 64).bfloat16().cuda(), torch.empty(2, 4).cuda()
    ws = torch.empty(zl.zl_kv4_attn_workspace_bytes(c, 4), dtype=torch.uint8).cuda()
    w, p = torch.zeros(c.slot_shape).cuda(), torch.zeros(c.slot_shape, dtype=torch.int32).cuda()
    ok = lambda **kw: zl.zl_kv4_attn_fwd(**{**dict(cache=c, q=q, o=o, lse=lse, workspace=ws, scale=0.1), **kw})  # noqa: E731
    ok()
    for bad, error in ((dict(q=q.float()), TypeError), (dict(q=q[:1]), ValueError), (dict(o=o[:1]), ValueError), (dict(lse=lse.half()), TypeError),
                       (dict(workspace=ws[:100]), ValueError), (dict(weights=w), ValueError), (dict(weights=w[:1], weights_out=w), ValueError),
                       (dict(weights_out=w), ValueError), (dict(starts=torch.zeros(2, dtype=torch.int32).cuda()), ValueError),
                       (dict(starts=torch.zeros(3, dtype=torch.int64).cuda()), TypeError), (dict(q=q.cpu()), TypeError),
                       (dict(scale=-1.0), zl.ZlError), (dict(max_new=0), zl.ZlError)):
        with pytest.raises(error):
            ok(**bad)
    k = torch.ones(2, 2, 64).bfloat16().cuda()
    for bad, error in ((dict(k=k[:, :1]), ValueError), (dict(v=k[:1]), ValueError), (dict(positions=p[0, 0, :2].contiguous()), TypeError),
                       (dict(k=k[:1], v=k[:1]), zl.ZlError)):
        with pytest.raises(error):
            zl.zl_kv4_write(**{**dict(cache=c, k=k, v=k), **bad})
    ew = torch.empty(zl.zl_kv4_evict_workspace_bytes(c), dtype=torch.uint8).cuda()
    for bad, error in ((dict(weights=w[:, :1]), ValueError), (dict(positions=p.long()), TypeError), (dict(keep=0), zl.ZlError),
                       (dict(workspace=ew[:16]), ValueError), (dict(weights_out=w.cpu()), TypeError)):
        with pytest.raises(error):
            zl.zl_kv4_evict(**{**dict(cache=c, weights=w, positions=p, keep=3, recent=1, workspace=ew), **bad})
    with pytest.raises(ValueError):
        zl.zl_kv4_read(c, k, k, torch.zeros(1, dtype=torch.int64).cuda())
    with pytest.raises(ValueError):
        zl.Kv4Cache(c.data[..., :100], c.pages, c.lens)
