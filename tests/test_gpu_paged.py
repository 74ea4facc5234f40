"""The paged-cache operators against float64: kv_append_paged, attn_paged,
softmax_rows and spec_verify, one by one and run together as a step of
speculative decoding."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import status

pytestmark = pytest.mark.gpu

SCALE = float(np.float32(1.0 / math.sqrt(128.0)))


@pytest.fixture(scope="module")
def inv():
    from invariant_numerics_b200 import invnum
    assert invnum.inv_get_device_status() == invnum.INV_OK
    return invnum


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(inv, n_pages, hkv, page, seed):
    """A cache of random codes (every INT16 value may occur) and scales over a factor of 100."""
    g = gen(seed)
    shape = (n_pages, hkv, page, 128)
    codes = lambda: torch.randint(-32768, 32768, shape, generator=g, device="cuda").to(torch.int16)
    scale = lambda: torch.exp(torch.rand(shape[:3], generator=g, device="cuda") * math.log(100.0)) * 1e-5
    return inv.PagedKVCache(codes(), codes(), scale(), scale())


def batch(lens, news, page, seed, spare=3):
    """Descriptors of a ragged batch over pages in random order; table entries behind a sequence's last page are -1."""
    per = max(1, max(-(-n // page) for n in lens)) + 1
    table = torch.full((len(lens), per), -1, dtype=torch.int32)
    n_pages = sum(-(-n // page) for n in lens) + spare
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    for i, n in enumerate(lens):
        for j in range(-(-n // page)):
            table[i, j] = order.pop()
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    return n_pages, table.cuda(), i32(start.tolist()), i32(list(lens))


def keys_of(cache, table, i, length, h):
    """Float64 keys and values 0 .. length - 1 of kv head h of sequence i."""
    page = cache.page_size
    pg = table[i, :-(-length // page)].long()
    f = lambda c, s: (c[pg, h].double() * s[pg, h].double()[..., None]).flatten(0, 1)[:length]
    return f(cache.k, cache.k_scale), f(cache.v, cache.v_scale)


def attend64(q, cache, table, start, lens, scale=SCALE):
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // cache.n_kv_heads
    st, ln = start.tolist(), lens.tolist()
    for i, n in enumerate(ln):
        m = st[i + 1] - st[i]
        if m == 0:
            continue
        for h in range(cache.n_kv_heads):
            k, v = keys_of(cache, table, i, n, h)
            t = torch.einsum("rgd,kd->rgk", q[st[i]:st[i + 1], h * G:(h + 1) * G].double(), k) * scale
            late = torch.arange(n, device="cuda")[None] > torch.arange(n - m, n, device="cuda")[:, None]
            w = torch.softmax(t.masked_fill(late[:, None], -math.inf), -1)
            out[st[i]:st[i + 1], h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", w, v)
    return out


def attend_bound(q, cache, table, start, lens, scale=SCALE):
    """Per output element, what the arithmetic may cost.

    A product x c of a fp32 value x (a query value, a weight) and a code c is formed from two binary16 parts of each:
    x up to 2^-22 |x|, c exactly, and the product of the low parts (2^-11 each) is dropped; 24 accumulations at 2^-24
    of the sum of |x c|: below 2^-19 together.  A score's error moves its weight by that relative amount (2^-18 for
    the exponential, the scalings and the joins), and the normaliser by the weighted mean of them.

    A weight p_j s_j is split after a scaling 2^E with 2^E s in [2^13, 2^14) for the largest scale s among the row's
    keys, so its low part is a multiple of 2^-24 and off by up to 2^-25 where the weight is far below the largest: by
    2^-25 2^-E <= 2^-38 s, times |code_j|, over a normaliser of at least 1 - 2^-18 (the largest p is 1): 2^-37 s
    sum_j |code_j|.  It shows where the keys that carry the weight have code 0."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    G = q.shape[1] // cache.n_kv_heads
    st, ln = start.tolist(), lens.tolist()
    for i, n in enumerate(ln):
        m = st[i + 1] - st[i]
        if m == 0:
            continue
        for h in range(cache.n_kv_heads):
            k, v = keys_of(cache, table, i, n, h)
            qq = q[st[i]:st[i + 1], h * G:(h + 1) * G].double()
            late = torch.arange(n, device="cuda")[None] > torch.arange(n - m, n, device="cuda")[:, None]
            t = torch.einsum("rgd,kd->rgk", qq, k).mul(scale).masked_fill(late[:, None], -math.inf)
            err = scale * 2.0 ** -19 * torch.einsum("rgd,kd->rgk", qq.abs(), k.abs()) + 2.0 ** -18
            w = torch.softmax(t, -1)
            e = (w * err).sum(-1, keepdim=True)
            pg = table[i, :-(-n // cache.page_size)].long()
            s = cache.v_scale[pg, h].double().flatten()[:n].cummax(0).values[n - m:]
            c = cache.v[pg, h].double().abs().flatten(0, 1)[:n].cumsum(0)[n - m:]
            out[st[i]:st[i + 1], h * G:(h + 1) * G] = 2.0 ** -37 * (s[:, None] * c)[:, None] + torch.einsum(
                "rgk,kd->rgd", w * (err + e + 2.0 ** -19), v.abs())
    return out


def check_attend(inv, q, cache, table, start, lens, out, scale=SCALE, rows=None):
    r = slice(0, int(start[-1])) if rows is None else rows
    want = attend64(q, cache, table, start, lens, scale)[r]
    bound = attend_bound(q, cache, table, start, lens, scale)[r]
    d = (out.double()[r] - want).abs()
    assert torch.isfinite(out[r]).all()
    worst = (d / bound.clamp_min(1e-300)).max().item()
    assert worst <= 1.0, worst


ATTEND = [
    # lens, new tokens, hq, hkv, page
    ([1], [1], 8, 2, 16),
    ([2], [2], 4, 4, 16),
    ([127, 128, 129, 1], [1, 1, 1, 1], 8, 2, 64),
    ([511, 512, 513, 1025], [1, 2, 1, 2], 8, 2, 16),
    ([300, 0, 17, 640], [5, 0, 17, 3], 32, 8, 16),
    ([1000, 77], [9, 4], 16, 1, 32),
    ([260, 33], [3, 2], 6, 2, 128),
    ([700, 300], [1, 1], 24, 8, 256),
    ([1300, 90, 2050], [200, 90, 1], 8, 2, 32),
    ([400], [333], 16, 4, 128),
    ([129, 600], [129, 70], 3, 3, 64),
    ([1111], [600], 20, 2, 16),
    ([1700, 900, 40, 77], [1200, 900, 1, 5], 32, 8, 64),
]


@pytest.mark.parametrize("lens,news,hq,hkv,page", ATTEND)
def test_attn_paged_against_float64(inv, lens, news, hq, hkv, page):
    n_pages, table, start, ln = batch(lens, news, page, seed=len(lens) + page)
    cache = pool(inv, n_pages, hkv, page, seed=hq)
    q = torch.randn(sum(news), hq, 128, generator=gen(5), device="cuda") * 0.7
    out, hi, lo = inv.attn_paged(q, cache, table, start, ln, SCALE, want_split=True)
    assert status() == inv.INV_OK
    check_attend(inv, q, cache, table, start, ln, out)
    rh, rl = inv.heal_split(out.view(-1, 128))
    assert torch.equal(rh, hi.view(-1, 128)) and torch.equal(rl, lo.view(-1, 128))
    # tight host bounds change nothing
    again = inv.attn_paged(q, cache, table, start, ln, SCALE, max_q_bound=max(news), max_len_bound=max(lens))
    assert torch.equal(out, again)


@pytest.mark.parametrize("hq,hkv,page", [(8, 2, 16), (32, 8, 64), (6, 2, 32)])
def test_attn_paged_rows_do_not_depend_on_the_batch(inv, hq, hkv, page):
    """One sequence of 1500 positions: all rows in one call, in chunks, and one by one, alone and among others."""
    n, first = 1500, 1100
    lens = [n, 40, 700]
    n_pages, table, start, ln = batch(lens, [n - first, 40, 1], page, seed=3)
    cache = pool(inv, n_pages, hkv, page, seed=4)
    q = torch.randn(int(start[-1]), hq, 128, generator=gen(6), device="cuda")
    full = inv.attn_paged(q, cache, table, start, ln, SCALE)
    one = lambda a, b: inv.attn_paged(q[a - first:b - first], cache, table[:1], i32([0, b - a]), i32([b]), SCALE)
    for a, b in ((1100, 1101), (1100, 1107), (1103, 1120), (1150, 1290), (1279, 1281), (1499, 1500), (1100, 1500)):
        assert torch.equal(one(a, b), full[a - first:b - first]), (a, b)
    assert torch.equal(inv.attn_paged(q[-1:], cache, table[2:], i32([0, 1]), i32([700]), SCALE), full[-1:])
    # the same keys in pages of another size
    for ps in (16, 128):
        per = -(-n // ps)
        other = inv.PagedKVCache.empty(per, hkv, ps)
        for h in range(hkv):
            for src, dst in ((cache.k, other.k), (cache.v, other.v), (cache.k_scale, other.k_scale),
                             (cache.v_scale, other.v_scale)):
                rows = src[table[0, :-(-n // page)].long(), h].flatten(0, 1)[:n]
                pad = torch.zeros((per * ps,) + rows.shape[1:], dtype=rows.dtype, device="cuda")
                pad[:n] = rows
                dst[:, h] = pad.view((per, ps) + rows.shape[1:])
        t2 = torch.arange(per, dtype=torch.int32, device="cuda")[None]
        got = inv.attn_paged(q[:n - first], other, t2, i32([0, n - first]), i32([n]), SCALE)
        assert torch.equal(got, full[:n - first])
    assert status() == inv.INV_OK


def test_attn_paged_large_batch_equals_its_parts(inv):
    """A call whose tiles fill the GPU (each tile folds its own segments) against calls of few rows and of one tile
    (segments joined by another kernel): the same bits."""
    lens, news, hq, hkv, page = [1500, 1203, 30, 1100], [1500, 900, 1, 6], 32, 8, 32
    n_pages, table, start, ln = batch(lens, news, page, seed=51)
    cache = pool(inv, n_pages, hkv, page, seed=52)
    q = torch.randn(int(start[-1]), hq, 128, generator=gen(53), device="cuda")
    full = inv.attn_paged(q, cache, table, start, ln, SCALE)
    st = start.tolist()
    for i, first, count in ((0, 0, 1), (0, 1499, 1), (0, 700, 7), (0, 511, 2), (0, 1024, 33), (1, 0, 20), (1, 899, 1),
                            (1, 300, 300), (2, 0, 1), (3, 0, 6), (3, 3, 2)):
        a = st[i] + first
        n = lens[i] - news[i] + first + count
        got = inv.attn_paged(q[a:a + count], cache, table[i:i + 1], i32([0, count]), i32([n]), SCALE)
        assert torch.equal(got, full[a:a + count]), (i, first, count)
    again = inv.attn_paged(q, cache, table, start, ln, SCALE)
    assert torch.equal(again, full) and status() == inv.INV_OK


@pytest.mark.parametrize("hq,hkv,page,long", [(32, 8, 16, 1400), (32, 8, 64, 500), (16, 1, 32, 1100)])
def test_attn_paged_mixed_token_counts(inv, hq, hkv, page, long):
    """More work items than fit the GPU at once, sequences of 1, 2, .. new tokens in turn: each as if alone."""
    news = [1 + i % 9 for i in range(45)]
    r = np.random.default_rng(long)
    lens = [int(n + r.integers(0, long)) for n in news]
    n_pages, table, start, ln = batch(lens, news, page, seed=61)
    cache = pool(inv, n_pages, hkv, page, seed=62)
    q = torch.randn(int(start[-1]), hq, 128, generator=gen(63), device="cuda")
    few = [i for i in range(45) if news[i] <= 8]  # without the sequences of 9 tokens too
    st = start.tolist()
    rows = torch.cat([torch.arange(st[i], st[i + 1]) for i in few]).cuda()
    full = inv.attn_paged(q, cache, table, start, ln, SCALE)
    part = inv.attn_paged(q[rows], cache, table[few].contiguous(),
                          i32(np.concatenate([[0], np.cumsum([news[i] for i in few])]).tolist()),
                          i32([lens[i] for i in few]), SCALE, max_q_bound=8)
    assert torch.equal(part, full[rows])
    for i in range(0, 45, 4):
        got = inv.attn_paged(q[st[i]:st[i + 1]], cache, table[i:i + 1], i32([0, news[i]]), ln[i:i + 1], SCALE)
        assert torch.equal(got, full[st[i]:st[i + 1]]), (i, news[i])
    check_attend(inv, q, cache, table, start, ln, full)
    assert status() == inv.INV_OK


def test_attn_paged_unused_memory_does_not_matter(inv):
    """What lies behind a sequence's last key (codes, infinite and NaN scales), and rows of no sequence."""
    lens, news, page, hq, hkv = [130, 21], [2, 21], 64, 8, 2
    n_pages, table, start, ln = batch(lens, news, page, seed=8)
    cache = pool(inv, n_pages, hkv, page, seed=9)
    q = torch.randn(30, hq, 128, generator=gen(7), device="cuda")
    out = torch.full_like(q, 7.5)
    inv.attn_paged(q, cache, table, start, ln, SCALE, out=out)
    assert (out[23:] == 7.5).all()
    for i, n in enumerate(lens):
        tail = n % page
        pg = int(table[i, n // page])
        for s, bad in ((cache.k_scale, math.nan), (cache.v_scale, math.inf)):
            s[pg, :, tail:] = bad
        cache.k[pg, :, tail:] = -32768
        cache.v[pg, :, tail:] = 32767
    used = set(table[table >= 0].tolist())
    for p in set(range(n_pages)) - used:
        cache.k_scale[p] = math.nan
        cache.v_scale[p] = math.nan
    out2 = torch.full_like(q, -3.0)
    inv.attn_paged(q, cache, table, start, ln, SCALE, out=out2)
    assert torch.equal(out[:23], out2[:23]) and (out2[23:] == -3.0).all()
    assert status() == inv.INV_OK


def test_attn_paged_extreme_values(inv):
    """Queries and scales far from 1, zero queries, zero scales, equal keys, sigma 0."""
    hq, hkv, page, n = 8, 2, 32, 700
    n_pages, table, start, ln = batch([n], [3], page, seed=1)
    cache = pool(inv, n_pages, hkv, page, seed=2)
    q = torch.randn(3, hq, 128, generator=gen(3), device="cuda")
    base = inv.attn_paged(q, cache, table, start, ln, SCALE)
    # q times 2^20 with sigma 2^-20: exact, so the same bits
    assert torch.equal(inv.attn_paged(q * 2.0 ** 20, cache, table, start, ln, SCALE * 2.0 ** -20), base)
    # values scaled by a power of two
    up = inv.PagedKVCache(cache.k, cache.v, cache.k_scale, cache.v_scale * 2.0 ** 30)
    assert torch.equal(inv.attn_paged(q, up, table, start, ln, SCALE), base * 2.0 ** 30)
    # zero queries, and sigma 0: the mean of the visible values
    for qq, sg in ((torch.zeros_like(q), SCALE), (q, 0.0)):
        check_attend(inv, qq, cache, table, start, ln, inv.attn_paged(qq, cache, table, start, ln, sg), sg)
    # values whose scales differ by 10^6, and values of scale 0
    wide = inv.PagedKVCache(cache.k, cache.v, cache.k_scale,
                            cache.v_scale * 10.0 ** (torch.rand(cache.v_scale.shape, generator=gen(4), device="cuda") * 6))
    check_attend(inv, q, wide, table, start, ln, inv.attn_paged(q, wide, table, start, ln, SCALE))
    none = inv.PagedKVCache(cache.k, cache.v, cache.k_scale, cache.v_scale * 0)
    assert (inv.attn_paged(q, none, table, start, ln, SCALE) == 0).all()
    # one score far above the rest: that key's value
    sharp = q * 300.0
    check_attend(inv, sharp, cache, table, start, ln, inv.attn_paged(sharp, cache, table, start, ln, SCALE))
    assert status() == inv.INV_OK


def test_attn_paged_strided_q_graph_and_streams(inv):
    hq, hkv, page = 8, 2, 16
    lens, news = [600, 35], [4, 2]
    n_pages, table, start, ln = batch(lens, news, page, seed=11)
    cache = pool(inv, n_pages, hkv, page, seed=12)
    wide = torch.randn(6, (hq + 2 * hkv) * 128, generator=gen(13), device="cuda")
    q = wide[:, :hq * 128].view(6, hq, 128)
    want = inv.attn_paged(q.contiguous(), cache, table, start, ln, SCALE)
    assert torch.equal(inv.attn_paged(q, cache, table, start, ln, SCALE), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = inv.attn_paged(q, cache, table, start, ln, SCALE, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    # a graph whose lengths and rows are rewritten between replays (padded to 6 rows)
    ws = torch.empty(inv.attn_paged_workspace_size(6, 2, hq, hkv, 4, 640), dtype=torch.uint8, device="cuda")
    out = torch.zeros(6, hq, 128, device="cuda")
    st, l2 = start.clone(), ln.clone()
    call = lambda: inv.attn_paged(q, cache, table, st, l2, SCALE, max_q_bound=4, max_len_bound=640, out=out, workspace=ws)
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for news2, lens2 in (([4, 2], [600, 35]), ([1, 1], [598, 35]), ([0, 3], [0, 20]), ([2, 4], [513, 33])):
        st.copy_(i32([0, news2[0], sum(news2)]))
        l2.copy_(i32(lens2))
        out.fill_(9.0)
        g.replay()
        m = sum(news2)
        check = inv.attn_paged(q[:m], cache, table, st, l2, SCALE)
        assert torch.equal(out[:m], check) and (out[m:] == 9.0).all()
    assert status() == inv.INV_OK


def test_attn_paged_bad_descriptors_are_recorded(inv):
    hq, hkv, page = 4, 2, 16
    n_pages, table, start, ln = batch([40, 50, 20], [2, 2, 2], page, seed=14)
    cache = pool(inv, n_pages, hkv, page, seed=15)
    q = torch.randn(6, hq, 128, generator=gen(16), device="cuda")
    want = inv.attn_paged(q, cache, table, start, ln, SCALE)
    for bad in ([40, 1, 20], [40, 10 ** 6, 20], [40, -5, 20]):
        out = torch.full_like(q, 5.0)
        inv.attn_paged(q, cache, table, start, i32(bad), SCALE, out=out)
        assert status() == inv.INV_ERR_INVALID_ARG
        assert torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:]) and (out[2:4] == 5.0).all()
    for page_id in (-1, n_pages, 2 ** 31 - 1):
        t2 = table.clone()
        t2[1, 1] = page_id
        out = inv.attn_paged(q, cache, t2, start, ln, SCALE)
        assert status() == inv.INV_ERR_INVALID_ARG
        assert torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:]) and torch.isfinite(out).all()
    assert torch.equal(inv.attn_paged(q, cache, table, start, ln, SCALE), want) and status() == inv.INV_OK


# ------------------------------------------------------------------ append ---

def tables(inv, max_pos=2048):
    return inv.rope_tables(max_pos)


def append64(x, hq, hkv, cos, sin, pos, gains, eps):
    """Float64 heads after norm and rotation: q, k, v."""
    y = x.double().view(x.shape[0], hq + 2 * hkv, 128)
    parts = []
    for a, b, g in ((0, hq, gains[0]), (hq, hq + hkv, gains[1])):
        z = y[:, a:b]
        if g is not None:
            z = z / (z.square().mean(-1, keepdim=True) + eps).sqrt() * g.double()
        c, s = cos[pos].double()[:, None], sin[pos].double()[:, None]
        lo, hi = z[..., :64], z[..., 64:]
        parts.append(torch.cat([lo * c - hi * s, hi * c + lo * s], -1))
    return parts[0], parts[1], y[:, hq + hkv:]


@pytest.mark.parametrize("lens,news,hq,hkv,page,norm", [
    ([1], [1], 8, 2, 16, "qk"), ([33, 16, 0, 700], [5, 16, 0, 1], 32, 8, 16, "qk"), ([300], [300], 6, 3, 64, ""),
    ([64, 65], [64, 1], 8, 8, 128, "k"), ([90] * 70, [1] * 70, 4, 1, 32, "q"), ([257], [200], 16, 4, 256, "qk")])
def test_kv_append_paged_against_float64(inv, lens, news, hq, hkv, page, norm):
    n_pages, table, start, ln = batch(lens, news, page, seed=page)
    T = sum(news)
    g = gen(T)
    wide = torch.randn(T + 2, (hq + 2 * hkv) * 128 + 12, generator=g, device="cuda")
    x = wide[:, :(hq + 2 * hkv) * 128]
    x[0, :128] = 0  # a zero head
    gains = [torch.rand(128, generator=g, device="cuda") + 0.5 if n in norm else None for n in "qk"]
    cos, sin = tables(inv)
    cache = pool(inv, n_pages, hkv, page, seed=21)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    q_out = torch.full((T + 2, hq, 128), 4.25, device="cuda")
    inv.kv_append_paged(x, cache, table, start, ln, cos, sin, q_gain=gains[0], k_gain=gains[1], eps=1e-6, q_out=q_out)
    assert status() == inv.INV_OK
    assert (q_out[T:] == 4.25).all()  # rows of no sequence
    seq = np.repeat(np.arange(len(lens)), news)
    off = np.arange(T) - start.cpu().numpy()[seq]
    pos = torch.tensor(np.array(lens)[seq] - np.array(news)[seq] + off, device="cuda")
    q, k, v = append64(x[:T], hq, hkv, cos, sin, pos, gains, 1e-6)
    # three roundings of the norm and two of a rotated value, 2^-24 each of |a| + |b|, at most sqrt(2) times the
    # rotated pair's |a'| + |b'|: 7.1
    pair = lambda z: (z.abs() + z.roll(64, -1).abs())
    assert ((q_out[:T].double() - q).abs() <= 8 * 2.0 ** -24 * pair(q).clamp_min(1e-30)).all()
    where = table[torch.tensor(seq, device="cuda"), (pos // page)].long()
    touched = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    touched[where, pos % page] = True
    for z, codes, scale in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        c, s = codes[where, :, pos % page].double(), scale[where, :, pos % page].double()
        amax = z.abs().amax(-1)
        # the largest value's error (its pair is at most twice as large: 14.2) and the quotient's rounding
        assert ((s - amax / 32767).abs() <= 16 * 2.0 ** -24 * amax / 32767 + 1e-45).all()
        # half a step of the grid, the value's error (2^-20 of the largest) and its quotient's (2^-24 of 32767 steps)
        assert ((c * s[..., None] - z).abs() <= (0.5 * s + 2.0 ** -19 * amax)[..., None] + 1e-45).all()
    # nothing else of the cache is written
    for now, old in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), before):
        keep = ~touched
        assert torch.equal(now.transpose(1, 2)[keep], old.transpose(1, 2)[keep])


def test_kv_append_paged_matches_the_slot_cache_quantiser(inv):
    """Without gains: V exactly kv_quant_int16's codes, K those of the rotated rows, whatever the batch."""
    hq, hkv, page, T = 8, 2, 32, 50
    n_pages, table, start, ln = batch([T], [T], page, seed=31)
    x = torch.randn(T, (hq + 2 * hkv) * 128, generator=gen(32), device="cuda")
    cos, sin = tables(inv)
    cache = inv.PagedKVCache.empty(n_pages, hkv, page)
    q = inv.kv_append_paged(x, cache, table, start, ln, cos, sin)
    slot = inv.KVCache(n_slots=1, n_kv_heads=hkv, max_len=64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    y = x.view(T, -1, 128)
    lo, hi = y[:, :hq + hkv, :64], y[:, :hq + hkv, 64:]
    c, s = cos[:T, None], sin[:T, None]
    rot = torch.cat([lo * c - hi * s, hi * c + lo * s], -1)
    inv.kv_quant_int16(rot[:, hq:].contiguous(), torch.zeros_like(pos), pos, slot, "k")
    inv.kv_quant_int16(y[:, hq + hkv:].contiguous(), torch.zeros_like(pos), pos, slot, "v")
    assert torch.equal(q, rot[:, :hq])
    pg = table[0, :-(-T // page)].long()
    for a, b in ((cache.k, slot.k), (cache.v, slot.v), (cache.k_scale, slot.k_scale), (cache.v_scale, slot.v_scale)):
        assert torch.equal(a[pg].transpose(0, 1).flatten(1, 2)[:, :T], b[0, :, :T])
    # row by row, the same bits
    other = inv.PagedKVCache.empty(n_pages, hkv, page)
    gains = [torch.rand(128, generator=gen(33), device="cuda") + 0.5 for _ in range(2)]
    inv.kv_append_paged(x, cache, table, start, ln, cos, sin, *gains)
    for t in range(T):
        inv.kv_append_paged(x[t:t + 1], other, table, i32([0, 1]), i32([t + 1]), cos, sin, *gains)
    assert torch.equal(cache.k[pg], other.k[pg]) and torch.equal(cache.k_scale[pg], other.k_scale[pg])
    assert status() == inv.INV_OK


def test_kv_append_paged_bad_descriptors_are_recorded(inv):
    hq, hkv, page = 4, 2, 16
    n_pages, table, start, ln = batch([40, 50], [2, 2], page, seed=41)
    x = torch.randn(4, (hq + 2 * hkv) * 128, generator=gen(42), device="cuda")
    cos, sin = tables(inv, 48)  # positions 48 and 49 have no angles
    cache = pool(inv, n_pages, hkv, page, seed=43)
    old = cache.k.clone()
    q = torch.full((4, hq, 128), 2.0, device="cuda")
    inv.kv_append_paged(x, cache, table, start, ln, cos, sin, q_out=q)
    assert status() == inv.INV_ERR_INVALID_ARG and (q[2:] == 2.0).all() and not (q[:2] == 2.0).any()
    cache.k.copy_(old)
    t2 = table.clone()
    t2[0, 2] = n_pages
    inv.kv_append_paged(x, cache, t2, start, i32([40, 1]), cos, sin, q_out=q)
    assert status() == inv.INV_ERR_INVALID_ARG and torch.equal(cache.k, old)


# ----------------------------------------------------- softmax, verification ---

@pytest.mark.parametrize("rows,n,it", [(1, 1, 1.0), (3, 7, 0.5), (2, 1000, 1.0), (5, 4096, 2.0), (4, 4099, 1 / 0.7),
                                       (2, 8192, 1.0), (2, 32003, 1.0), (3, 65536, 1.0),
                                       (3, 65537, 0.9), (2, 262144, 1.0), (2, 300001, 1.0)])
def test_softmax_rows_against_float64(inv, rows, n, it):
    x = torch.randn(rows, n, generator=gen(n), device="cuda") * 5
    x[:, ::13] = -math.inf
    if n > 1:
        x[-1] = -math.inf  # nothing allowed
    if n == 1:
        x[:] = 3.0
    y = inv.softmax_rows(x, it)
    it32 = float(np.float32(it))
    t = x.double() * it32
    want = torch.softmax(t, -1).nan_to_num(0.0)
    # in units of 2^-24: the exponent's two roundings (of up to |t - max|, in one or two pieces), exp's 2 ulp (4, twice
    # where a row has parts), the factor's and the product's (3); the same of the sum's terms, and its additions
    span = (t.amax(-1, keepdim=True) - t).nan_to_num(0.0, posinf=0.0)
    depth = n // 4096 + 32  # additions one term passes through
    rel = 2.0 ** -24 * (2 * span + 11) + 2.0 ** -24 * (2 * (want * span).sum(-1, keepdim=True) + 9 + depth)
    assert ((y.double() - want).abs() <= rel * want + 1e-38).all()
    assert (y[:, ::13] == 0).all() if n > 1 else (y == 1).all()
    wide = torch.full((rows, n + 5), 1.0, device="cuda")
    wide[:, :n] = x
    assert torch.equal(inv.softmax_rows(wide[:, :n], it), y)          # another row stride, the same bits
    assert torch.equal(inv.softmax_rows(x[:1].contiguous(), it), y[:1])  # a row alone
    z = x.clone()
    assert inv.softmax_rows(z, it, out=z) is z and torch.equal(z, y)  # in place
    assert status() == inv.INV_OK


def verify64(target, draft, tokens, u, us, n_draft):
    B, m1, V = target.shape
    out = np.full((B, m1), -1, np.int32)
    acc = np.zeros(B, np.int32)
    p, x = target.double().cpu().numpy(), tokens.cpu().numpy()
    q = None if draft is None else draft.double().cpu().numpy()
    u, us = u.double().cpu().numpy(), us.double().cpu().numpy()
    for b in range(B):
        m = m1 - 1 if n_draft is None else int(n_draft[b])
        k = 0
        while k < m and u[b, k] * (1.0 if q is None else q[b, k, x[b, k]]) < p[b, k, x[b, k]]:
            out[b, k] = x[b, k]
            k += 1
        w = p[b, k].copy()
        if k < m and q is not None:
            w = np.maximum(w - q[b, k], 0)
        elif k < m:
            w[x[b, k]] = 0
        if not w.sum() > 0:
            w = p[b, k].copy()
        c = np.cumsum(w)
        hit = np.nonzero((c > us[b] * c[-1]) & (w > 0))[0]
        out[b, k] = hit[0] if len(hit) else -1
        acc[b] = k
    return out, acc


@pytest.mark.parametrize("B,m,V,probs", [(1, 0, 5, True), (1, 1, 1, True), (3, 4, 1000, True), (2, 7, 32003, False),
                                         (9, 40, 257, True), (4, 3, 131072, True), (64, 5, 4001, False),
                                         (2, 2, 4096, True), (3, 2, 32768, False), (3, 2, 32769, True), (2, 2, 131073, True),
                                         (2, 1, 131075, False)])
def test_spec_verify_against_float64(inv, B, m, V, probs):
    g = gen(B * 100 + m)
    logits = torch.randn(B, m + 1, V, generator=g, device="cuda") * 3
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :m] + 0.5 * torch.randn(B, m, V, generator=g, device="cuda"), -1)
    pick = draft / -torch.log(torch.rand(B, m, V, generator=g, device="cuda").clamp_min(1e-20))
    tokens = pick.argmax(-1).to(torch.int32)
    u, us = torch.rand(B, m, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    us[0] = 0.0
    us[-1] = 1.0 - 2.0 ** -24
    for n_draft in (None, torch.randint(0, m + 1, (B,), generator=g, device="cuda").to(torch.int32)):
        got, acc = inv.spec_verify(target, draft if probs else None, tokens, u, us, n_draft=n_draft)
        want, wacc = verify64(target, draft if probs else None, tokens, u, us, n_draft)
        assert np.array_equal(acc.cpu().numpy(), wacc)
        assert np.array_equal(got.cpu().numpy(), want)
    one, a1 = inv.spec_verify(target[-1:].contiguous(), draft[-1:].contiguous() if probs else None,
                              tokens[-1:].contiguous(), u[-1:].contiguous(), us[-1:].contiguous())
    both, a2 = inv.spec_verify(target, draft if probs else None, tokens, u, us)
    assert torch.equal(one[0], both[-1]) and int(a1[0]) == int(a2[-1])
    assert status() == inv.INV_OK


def test_spec_verify_edges(inv):
    V = 6
    f = lambda rows: torch.tensor(rows, dtype=torch.float32, device="cuda")
    # draft and target equal: always accepted; target 0 at the draft: rejected even with u = 0
    p = [[0.5, 0.25, 0.25, 0, 0, 0]]
    t, a = inv.spec_verify(f([p + p]), f([p]), i32([[1]]), f([[0.999]]), f([0.5]))
    assert a.tolist() == [1] and t.tolist() == [[1, 1]]  # 0.5 of the total is not exceeded by the first half
    t, a = inv.spec_verify(f([p + p]), f([[[0, 0, 0, 1, 0, 0]]]), i32([[3]]), f([[0.0]]), f([0.75]))
    assert a.tolist() == [0] and t.tolist() == [[2, -1]]
    # residual without positive weight: the target's own weights
    t, a = inv.spec_verify(f([p + p]), f([[[0.5, 0.5, 0.25, 0, 0, 0]]]), i32([[1]]), f([[0.9]]), f([0.1]))
    assert a.tolist() == [0] and t.tolist() == [[0, -1]]
    # a lookup draft that is rejected is not drawn again
    t, a = inv.spec_verify(f([p + p]), None, i32([[0]]), f([[0.6]]), f([0.0]))
    assert a.tolist() == [0] and t.tolist() == [[1, -1]]
    # the same in long rows, in every form of the kernel
    for n in (5000, 40000, 140000):
        row = torch.zeros(1, 2, n, device="cuda")
        row[0, :, n - 7] = 0.75
        row[0, :, 3] = 0.25
        t, a = inv.spec_verify(row, row[:, :1].contiguous() * 2, i32([[3]]), f([[0.9]]), f([0.3]))
        assert a.tolist() == [0] and t.tolist() == [[n - 7, -1]]
        t, a = inv.spec_verify(row, None, i32([[3]]), f([[0.9]]), f([0.999]))
        assert a.tolist() == [0] and t.tolist() == [[n - 7, -1]]
        t, a = inv.spec_verify(row * 0, None, i32([[3]]), f([[0.9]]), f([0.999]))
        assert a.tolist() == [0] and t.tolist() == [[-1, -1]]
    # no weight at all
    z = [[0.0] * V]
    t, a = inv.spec_verify(f([z + z]), None, i32([[0]]), f([[0.0]]), f([0.3]))
    assert a.tolist() == [0] and t.tolist() == [[-1, -1]]
    assert status() == inv.INV_OK
    # a draft token outside the vocabulary
    t, a = inv.spec_verify(f([p + p, p + p]), None, i32([[V], [0]]), f([[0.1], [0.1]]), f([0.3, 0.6]))
    assert status() == inv.INV_ERR_INVALID_ARG
    assert a.tolist() == [0, 1] and t.tolist() == [[-1, -1], [0, 1]]
    t, a = inv.spec_verify(f([p + p]), None, i32([[0]]), f([[0.1]]), f([0.3]), n_draft=i32([2]))
    assert status() == inv.INV_ERR_INVALID_ARG and a.tolist() == [0] and t.tolist() == [[-1, -1]]


# -------------------------------------------------------- the operators together ---

def test_speculative_step_equals_one_token_at_a_time(inv):
    """Three conversations draft 4 tokens; append + attend + head + softmax + verify of the drafts in one call give
    the bits of feeding the same tokens one by one, and the next step writes over the rejected positions."""
    hq, hkv, page, V, H = 8, 2, 16, 640, 256
    g = gen(77)
    B, m = 3, 4
    lens = [37, 130, 515]  # context before the step
    total = [n + m + 1 for n in lens]
    n_pages, table, _, _ = batch(total, [1] * B, page, seed=78)
    cos, sin = tables(inv, 1024)
    gains = [torch.rand(128, generator=g, device="cuda") + 0.5 for _ in range(2)]
    emb = torch.randn(V, H, generator=g, device="cuda")
    w_qkv = inv.heal_pack_weight(torch.randn(H, (hq + 2 * hkv) * 128, generator=g, device="cuda") * 0.1)
    w_o = inv.heal_pack_weight(torch.randn(hq * 128, H, generator=g, device="cuda") * 0.05)
    head = inv.heal_pack_weight(torch.randn(H, V, generator=g, device="cuda") * 0.1)

    def model(cache, ids, start, ln):
        x = inv.embed_gather(emb, ids)
        qkv = inv.comp_gemm(*inv.heal_split(x), *w_qkv)
        q = inv.kv_append_paged(qkv, cache, table, start, ln, cos, sin, *gains)
        _, hi, lo = inv.attn_paged(q, cache, table, start, ln, SCALE, want_split=True)
        y = inv.comp_gemm(hi.view(-1, hq * 128), lo.view(-1, hq * 128), *w_o, residual=x)
        return inv.comp_gemm(*inv.heal_split(y), *head)

    def filled():
        cache = inv.PagedKVCache.empty(n_pages, hkv, page)
        r = np.random.default_rng(5)
        ids = [r.integers(0, V, n) for n in lens]
        start = i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
        model(cache, i32(np.concatenate(ids).tolist()), start, i32(lens))
        return cache

    # last sampled token and the drafts behind it: m + 1 new tokens a conversation
    new = torch.randint(0, V, (B, m + 1), generator=g, device="cuda").to(torch.int32)
    together, apart = filled(), filled()
    start = i32([0, m + 1, 2 * m + 2, 3 * m + 3])
    logits = model(together, new.reshape(-1), start, i32(total)).view(B, m + 1, V)
    single = torch.stack([model(apart, new[:, j].contiguous(), i32([0, 1, 2, 3]), i32([n + j + 1 for n in lens]))
                          for j in range(m + 1)], 1)
    assert torch.equal(logits, single)
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(together, name), getattr(apart, name))
    probs = inv.softmax_rows(logits.view(-1, V), 0.8).view(B, m + 1, V)
    u, us = torch.rand(B, m, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    drafts = new[:, 1:].contiguous()
    tok, acc = inv.spec_verify(probs, None, drafts, u, us)
    want, wacc = verify64(probs, None, drafts, u, us, None)
    assert np.array_equal(tok.cpu().numpy(), want) and np.array_equal(acc.cpu().numpy(), wacc)
    # go on behind the accepted prefix: the same as a cache that never saw the rejected drafts
    k = acc.tolist()
    nxt = torch.stack([tok[b, k[b]] for b in range(B)]).to(torch.int32)
    ln2 = [n + 1 + kk + 1 for n, kk in zip(lens, k)]
    got = model(together, nxt, i32([0, 1, 2, 3]), i32(ln2))
    clean = filled()
    keep = [1 + kk for kk in k]
    ids = torch.cat([new[b, :keep[b]] for b in range(B)])
    model(clean, ids, i32(np.concatenate([[0], np.cumsum(keep)]).tolist()), i32([n + kk for n, kk in zip(lens, keep)]))
    assert torch.equal(model(clean, nxt, i32([0, 1, 2, 3]), i32(ln2)), got)
    assert status() == inv.INV_OK


def test_binding_refuses_wrong_tensors(inv):
    """Types, shapes and strides the operators do not take."""
    n_pages, table, start, ln = batch([20], [2], 16, seed=1)
    cache = pool(inv, n_pages, 2, 16, seed=2)
    q = torch.zeros(2, 4, 128, device="cuda")
    ok = lambda **kw: inv.attn_paged(**{**dict(q=q, cache=cache, page_table=table, q_start=start, lens=ln,
                                               softmax_scale=SCALE), **kw})
    ok()
    for bad in (dict(q=q.half()), dict(q=q[:, :, :64]), dict(q=q.transpose(0, 1)), dict(page_table=table.long()),
                dict(page_table=table[0]), dict(q_start=start[:1]), dict(lens=ln.float()), dict(out=q[:1]),
                dict(lens=ln.cpu())):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(inv.InvError):
        ok(q=torch.zeros(2, 3, 128, device="cuda"))  # 3 heads over 2 kv heads
    with pytest.raises(inv.InvError):
        ok(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"), max_len_bound=0, page_table=table.repeat(1, 40))
    with pytest.raises(ValueError):
        inv.PagedKVCache(cache.k.float(), cache.v, cache.k_scale, cache.v_scale)
    with pytest.raises(ValueError):
        inv.kv_append_paged(torch.zeros(2, 500, device="cuda"), cache, table, start, ln, *tables(inv, 64))
    with pytest.raises(ValueError):
        inv.softmax_rows(torch.zeros(4, 6, device="cuda").t())
    with pytest.raises(ValueError):
        inv.spec_verify(torch.zeros(1, 3, 5, device="cuda"), None, i32([[1]]), torch.zeros(1, 1, device="cuda"),
                        torch.zeros(1, device="cuda"))
    assert status() == inv.INV_OK


def test_the_index_checking_build_agrees(inv):
    """These tests on the build that checks every index: nothing leaves its buffer."""
    import os
    import subprocess
    import sys
    from invariant_numerics_b200 import build
    if inv.inv_debug_bounds_enabled():
        return  # this is that run
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, INVNUM_LIBRARY=build.build(debug_bounds=True))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", __file__],
                       cwd=root, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-4000:] + r.stderr[-2000:]
