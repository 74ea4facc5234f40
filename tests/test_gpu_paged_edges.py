"""Calls of the paged-cache operators at the edges of what their documentation
allows: contradicting descriptors, values that are not numbers, workspaces of
other calls, lengths next to 2^31."""
import math

import numpy as np
import pytest
import torch

from gpu_helpers import status
from test_gpu_paged import SCALE, batch, check_attend, gen, i32, inv, pool, tables  # noqa: F401

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------- descriptors ---

Q_START = [  # q_start of 3 sequences over 6 rows, the sequences it contradicts, rows that are still right
    ([0, 2, 4, 7], [2], [0, 1, 2, 3]),
    ([-1, 2, 4, 6], [0], [2, 3, 4, 5]),
    ([-9, -9, 4, 6], [0, 1], [4, 5]),
    ([0, 2, 4, 2 ** 31 - 1], [2], [0, 1, 2, 3]),
    ([-2 ** 31, 2, 4, 6], [0], [2, 3, 4, 5]),
    ([0, 2, 2, 0], [2], []),
    ([0, 4, 2, 6], [1], []),
    ([6, 4, 2, 0], [0, 1, 2], []),
    ([0, 2, 9, 9], [1, 2], [0, 1]),
]


@pytest.mark.parametrize("q_start,wrong,right", Q_START)
def test_q_start_that_contradicts_the_call_is_recorded(inv, q_start, wrong, right):  # noqa: F811
    hq, hkv, page = 4, 2, 16
    lens, news = [40, 50, 20], [2, 2, 2]
    n_pages, table, start, ln = batch(lens, news, page, seed=71)
    cache = pool(inv, n_pages, hkv, page, seed=72)
    q = torch.randn(6, hq, 128, generator=gen(73), device="cuda")
    want = inv.attn_paged(q, cache, table, start, ln, SCALE)
    assert status() == inv.INV_OK
    bad = i32(q_start)
    for mq in (None, 2):
        out = torch.full_like(q, 5.0)
        inv.attn_paged(q, cache, table, bad, ln, SCALE, max_q_bound=mq, out=out)
        assert status() == inv.INV_ERR_INVALID_ARG
        assert torch.equal(out[right], want[right])
        if right:  # nothing overlaps: the other rows are of no sound sequence
            rest = [r for r in range(6) if r not in right]
            assert (out[rest] == 5.0).all()
    # append: the same rows, and nothing but these rows' places in the cache
    x = torch.randn(6, (hq + 2 * hkv) * 128, generator=gen(74), device="cuda")
    cos, sin = tables(inv, 64)
    old = cache.k.clone(), cache.v.clone()
    good_q = inv.kv_append_paged(x, cache, table, start, ln, cos, sin)
    good = cache.k.clone(), cache.v.clone()
    assert status() == inv.INV_OK
    cache.k.copy_(old[0]), cache.v.copy_(old[1])
    qo = torch.full_like(q, 5.0)
    inv.kv_append_paged(x, cache, table, bad, ln, cos, sin, q_out=qo)
    assert status() == inv.INV_ERR_INVALID_ARG
    assert torch.equal(qo[right], good_q[right])
    if right:
        rest = [r for r in range(6) if r not in right]
        assert (qo[rest] == 5.0).all()
    written = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    may = torch.zeros_like(written)
    for i in range(3):
        for t in range(max(0, lens[i] - 6), lens[i]):
            may[int(table[i, t // page]), t % page] = True
    for r in right:
        i, t = r // 2, lens[r // 2] - 2 + r % 2
        written[int(table[i, t // page]), t % page] = True
    for now, was, full in zip((cache.k, cache.v), old, good):
        now, was, full = now.transpose(1, 2), was.transpose(1, 2), full.transpose(1, 2)
        keep = ~(written if right else may)  # rows of overlapping sequences may land at any of their last places
        assert torch.equal(now[keep], was[keep]) and torch.equal(now[written], full[written])


def test_q_start_that_descends_in_a_long_batch(inv):  # noqa: F811
    """Tiles and partial results of sequences whose rows overlap, beside sound ones; more sequences than rows."""
    hq, hkv, page = 8, 2, 32
    q = torch.randn(300, hq, 128, generator=gen(75), device="cuda")
    lens = [700, 650, 400, 300]
    n_pages, table, _, ln = batch(lens, [1] * 4, page, seed=76)
    cache = pool(inv, n_pages, hkv, page, seed=77)
    for st in ([0, 300, 100, 200, 300], [300, 0, 300, 0, 300], [0, 100, 300, 10, 20], [250, 10, 5, 260, 40]):
        wide = torch.full((900, hq, 128), 5.0, device="cuda")
        inv.attn_paged(q, cache, table, i32(st), ln, SCALE, out=wide[300:600])
        assert status() == inv.INV_ERR_INVALID_ARG
        assert (wide[:300] == 5.0).all() and (wide[600:] == 5.0).all()
    # 40 sequences over 3 rows: what is wrong stands behind the row count
    n = 40
    table1 = table[:1].expand(n, -1).contiguous()
    st = [0, 3] + [3] * (n - 1)
    x = torch.randn(3, (hq + 2 * hkv) * 128, generator=gen(78), device="cuda")
    cos, sin = tables(inv, 1024)
    ln1 = i32([700] * n)
    inv.kv_append_paged(x, cache, table1, i32(st), ln1, cos, sin)
    assert status() == inv.INV_OK
    st[30] = 2
    inv.kv_append_paged(x, cache, table1, i32(st), ln1, cos, sin)
    assert status() == inv.INV_ERR_INVALID_ARG
    inv.attn_paged(q[:3], cache, table1, i32(st), ln1, SCALE)
    assert status() == inv.INV_ERR_INVALID_ARG


@pytest.mark.parametrize("hq,hkv,page,lens,news", [(8, 2, 16, [300, 700], [1, 3]), (4, 2, 64, [640, 90], [8, 1]),
                                                   (8, 2, 256, [1100, 300], [2, 1]), (8, 2, 32, [900, 200], [300, 40]),
                                                   (32, 8, 64, [1300, 700], [1290, 2])])
def test_a_bad_page_counts_as_zeros(inv, hq, hkv, page, lens, news):  # noqa: F811
    """A page number outside the cache: the bits of a page of zeros in its place, whatever page 0 holds."""
    n_pages, table, start, ln = batch(lens, news, page, seed=81)
    cache = pool(inv, n_pages + 2, hkv, page, seed=82)
    cache.k_scale[0], cache.v_scale[0] = math.nan, math.inf  # of no sequence
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t[n_pages + 1] = 0
    table = torch.where(table >= 0, table + 1, table)
    q = torch.randn(sum(news), hq, 128, generator=gen(83), device="cuda")
    for bad, spots in ((-1, [(0, 0)]), (n_pages + 2, [(0, 1), (1, 0)]), (2 ** 31 - 1, [(0, lens[0] // page // 2)]),
                       (-2 ** 31, [(0, (lens[0] - 1) // page), (1, (lens[1] - 1) // page)]),
                       (-7, [(1, j) for j in range(-(-lens[1] // page))])):
        wrong, zeros = table.clone(), table.clone()
        for i, j in spots:
            wrong[i, j], zeros[i, j] = bad, n_pages + 1
        want = inv.attn_paged(q, cache, zeros, start, ln, SCALE)
        assert status() == inv.INV_OK and torch.isfinite(want).all()
        got = inv.attn_paged(q, cache, wrong, start, ln, SCALE)
        assert status() == inv.INV_ERR_INVALID_ARG
        assert torch.equal(got, want)
        if bad == -7:  # all pages of sequence 1
            assert (got[int(start[1]):] == 0).all()


# ---------------------------------------------------------------- workspace ---

@pytest.mark.parametrize("hq,hkv,page,most", [(32, 8, 64, 2500), (8, 1, 16, 5000)])
def test_attn_paged_workspace_of_a_larger_call(inv, hq, hkv, page, most):  # noqa: F811
    """One workspace, sized for the largest chunk of a prompt, for its chunks down to one token: the same bits as with
    each call's own, and nothing behind it is written."""
    n = most + 100
    n_pages, table, _, ln = batch([n], [1], page, seed=84)
    cache = pool(inv, n_pages, hkv, page, seed=85)
    q = torch.randn(most, hq, 128, generator=gen(86), device="cuda")
    size = inv.attn_paged_workspace_size(most, 1, hq, hkv, most, n)
    least = min(most, 32 * hkv // hq) * hq * -(-n // 512) * 520
    assert size >= least and max(inv.attn_paged_workspace_size(t, 1, hq, hkv, t, n) for t in (64, 300, 700)) > size
    big = torch.full((size + 4096,), 7, dtype=torch.uint8, device="cuda")
    small = torch.full((least + 4096,), 7, dtype=torch.uint8, device="cuda")
    for T in (1, 3, 32 * hkv // hq, 32 * hkv // hq + 1, 33, 64, 300, 700, 1100, most):
        start = i32([0, T])
        want = inv.attn_paged(q[:T], cache, table, start, ln, SCALE, max_len_bound=n)
        for ws in (big[:size], small[:least]):
            got = inv.attn_paged(q[:T], cache, table, start, ln, SCALE, max_len_bound=n, workspace=ws)
            assert torch.equal(got, want), T
    assert (big[size:] == 7).all() and (small[least:] == 7).all()
    # a batch padded far beyond its tokens: partial results by (sequence, token)
    pad = q[:400]
    ws = torch.full((least + 4096,), 7, dtype=torch.uint8, device="cuda")
    got = inv.attn_paged(pad, cache, table, i32([0, 3]), ln, SCALE, max_q_bound=3, max_len_bound=n, workspace=ws[:least])
    assert torch.equal(got[:3], inv.attn_paged(q[:3], cache, table, i32([0, 3]), ln, SCALE))
    assert (ws[least:] == 7).all() and status() == inv.INV_OK


def test_attn_paged_mixed_batch_in_a_small_workspace(inv):  # noqa: F811
    """Sequences of few and of many tokens where the split does not fit: few rows have partial results, by row and by
    sequence, the others none."""
    hq, hkv, page = 8, 2, 32
    for lens, news in (([900, 1400, 700, 60], [40, 3, 1, 60]), ([1300, 800], [6, 9]), ([1500, 700, 800], [300, 2, 8])):
        n_pages, table, start, ln = batch(lens, news, page, seed=87)
        cache = pool(inv, n_pages, hkv, page, seed=88)
        T, n = sum(news), max(lens)
        q = torch.randn(T, hq, 128, generator=gen(89), device="cuda")
        want = inv.attn_paged(q, cache, table, start, ln, SCALE, max_len_bound=n)
        least = min(T, 8 * len(lens)) * hq * -(-n // 512) * 520
        ws = torch.full((least + 4096,), 7, dtype=torch.uint8, device="cuda")
        got = inv.attn_paged(q, cache, table, start, ln, SCALE, max_len_bound=n, workspace=ws[:least])
        assert torch.equal(got, want) and (ws[least:] == 7).all()
        check_attend(inv, q, cache, table, start, ln, got)
        with pytest.raises(inv.InvError):
            inv.attn_paged(q, cache, table, start, ln, SCALE, max_len_bound=n, workspace=ws[:least - 16])
    assert status() == inv.INV_OK


def test_lengths_next_to_two_to_the_31(inv):  # noqa: F811
    """A page table of 2^31 positions: short sequences are attended, a length that a segment's end would carry beyond
    int32 is recorded."""
    hq = hkv = 1
    cache = pool(inv, 3, hkv, 256, seed=90)
    table = torch.zeros(1, 1 << 23, dtype=torch.int32, device="cuda")
    table[0, 1] = 2
    q = torch.randn(2, hq, 128, generator=gen(91), device="cuda")
    want = inv.attn_paged(q[:1], cache, table[:, :4].contiguous(), i32([0, 1]), i32([400]), SCALE)
    for bound in (None, 400, 2 ** 31, 2 ** 40):
        got = inv.attn_paged(q[:1], cache, table, i32([0, 1]), i32([400]), SCALE, max_len_bound=bound)
        assert torch.equal(got, want)
    assert status() == inv.INV_OK
    for n in (2 ** 31 - 1, 2 ** 31 - 511):
        out = torch.full_like(q, 5.0)
        inv.attn_paged(q[:1], cache, table, i32([0, 1]), i32([n]), SCALE, out=out[:1])
        assert status() == inv.INV_ERR_INVALID_ARG and (out == 5.0).all()


def test_long_contexts_at_the_end_of_a_large_cache(inv):  # noqa: F811
    """Contexts of 33000 and 40003 positions in pages whose codes lie beyond element 2^31 of the cache, rows before the
    first sequence: float64, and the bits of the same pages in a small cache; what append writes too."""
    hq, hkv, page = 16, 8, 256
    lens, news, skip = [40003, 33000, 36000], [1, 70, 3], 2
    n_pages, table, start, ln = batch(lens, news, page, seed=94)
    small = pool(inv, n_pages, hkv, page, seed=95)
    total = 8200 + n_pages  # 8192 pages hold 2^31 codes
    shape = (total, hkv, page, 128)
    large = inv.PagedKVCache(*(torch.empty(shape, dtype=torch.int16, device="cuda") for _ in range(2)),
                             *(torch.full(shape[:3], math.nan, device="cuda") for _ in range(2)))
    names = ("k", "v", "k_scale", "v_scale")
    for name in names:
        getattr(large, name)[total - n_pages:] = getattr(small, name)
    far = torch.where(table >= 0, table + (total - n_pages), table)
    start = start + skip
    T = int(start[-1])
    x = torch.randn(T, (hq + 2 * hkv) * 128, generator=gen(96), device="cuda")
    cos, sin = tables(inv, 40960)
    q = inv.kv_append_paged(x, small, table, start, ln, cos, sin)
    q2 = inv.kv_append_paged(x, large, far, start, ln, cos, sin)
    assert torch.equal(q[skip:], q2[skip:])
    for name in names:
        assert torch.equal(getattr(large, name)[total - n_pages:], getattr(small, name))
        if "scale" in name:
            assert torch.isnan(getattr(large, name)[:total - n_pages]).all()
    q = torch.where(torch.isfinite(q), q, torch.zeros_like(q)) * 0.3
    q[:skip] = math.nan  # rows of no sequence
    out, out2 = torch.full_like(q, 3.0), torch.full_like(q, 3.0)
    inv.attn_paged(q, small, table, start, ln, SCALE, max_len_bound=40960, out=out)
    inv.attn_paged(q, large, far, start, ln, SCALE, out=out2)
    assert torch.equal(out, out2) and (out[:skip] == 3.0).all()
    check_attend(inv, q, small, table, start, ln, out, rows=slice(skip, T))
    assert status() == inv.INV_OK


# ------------------------------------------------------------------ softmax ---

@pytest.mark.parametrize("n", [1, 5, 1000, 8192, 8193, 16385, 65536, 65537, 131073, 262144, 262145, 300001])
def test_softmax_rows_with_nan_and_infinity(inv, n):  # noqa: F811
    """NaN or +inf anywhere makes the row NaN, as the formula does; rows without are as in a call of their own."""
    part = 32 * (256 if n <= 65536 else 512 if n <= 131072 else 1024)  # elements of a CTA
    base = torch.randn(n, generator=gen(n), device="cuda") * 4
    base[::7] = -math.inf
    base[n // 2] = 1.5
    places = sorted({0, 1, n // 3, n - 1, min(part, n) - 1, min(part, n - 1)} & set(range(n)))
    rows, is_nan = [base], [False]
    for bad in (math.nan, -math.nan, math.inf):
        for at in places:
            x = base.clone()
            x[at] = bad
            rows.append(x), is_nan.append(True)
            y = torch.full_like(base, -math.inf)  # nothing finite beside it
            y[at] = bad
            rows.append(y), is_nan.append(True)
    nothing = torch.full_like(base, -math.inf)
    rows += [nothing * -1, torch.full_like(base, math.nan), nothing]
    is_nan += [True, True, False]
    for a in range(0, n, part):  # one part of nothing but NaN
        x = base.clone()
        x[a:a + part] = math.nan
        rows.append(x), is_nan.append(True)
    x = torch.stack(rows)
    y = inv.softmax_rows(x, 0.9)
    is_nan = torch.tensor(is_nan, device="cuda")
    assert torch.isnan(y[is_nan]).all() and not torch.isnan(y[~is_nan]).any()
    # the formula's NaN rows (torch has NaN for a row of nothing but -inf too)
    lowest = (x == -math.inf).all(1)
    assert torch.equal(torch.isnan(torch.softmax(x.double(), -1)).all(1), is_nan | lowest)
    assert int((lowest & ~is_nan).sum()) == 1 and (y[lowest] == 0).all()
    # two exponents of at most 40 (two roundings each), exp, the factor and n / 4096 + 32 additions: 290 2^-24
    want = torch.softmax(base.double() * float(np.float32(0.9)), -1)
    assert ((y[0].double() - want).abs() <= 290 * 2.0 ** -24 * want + 1e-38).all()
    assert torch.equal(inv.softmax_rows(x[:1].contiguous(), 0.9), y[:1])
    assert status() == inv.INV_OK


def test_the_longest_rows(inv):  # noqa: F811
    """Rows of 2^31 - 1 elements: the last step of the kernels' loops ends behind them."""
    n = 2 ** 31 - 1
    x = torch.full((1, n), -math.inf, device="cuda")
    at = [0, 2 ** 30 + 5, n - 1025, n - 2, n - 1]
    x[0, at] = 2.0
    inv.softmax_rows(x, 1.5, out=x)
    assert (x[0, at] == float(np.float32(1.0) / np.float32(5.0))).all() and int((x != 0).sum()) == 5
    none = lambda dtype: torch.empty(1, 0, dtype=dtype, device="cuda")
    for u, want in ((0.0, 0), (0.3, 2 ** 30 + 5), (0.5, n - 1025), (0.7, n - 2), (0.999, n - 1)):
        t, a = inv.spec_verify(x.view(1, 1, n), None, none(torch.int32), none(torch.float32),
                               torch.tensor([u], device="cuda"))
        assert t.tolist() == [[want]] and a.tolist() == [0]
    t, a = inv.spec_verify(x.zero_().view(1, 1, n), None, none(torch.int32), none(torch.float32),
                           torch.tensor([0.5], device="cuda"))
    assert t.tolist() == [[-1]] and status() == inv.INV_OK


@pytest.mark.parametrize("V", [500, 5000, 40000, 140000])
def test_spec_verify_with_nan(inv, V):  # noqa: F811
    """In every form of the kernel: a NaN accepts nothing and weighs nothing."""
    p = torch.zeros(4, 2, V, device="cuda")
    p[:, :, 7], p[:, :, V - 3] = 0.25, 0.75
    q = torch.zeros(4, 1, V, device="cuda")
    q[:, :, 7] = 1.0
    p[0, 0] = math.nan   # a target row of nothing else
    q[1, 0, 7] = math.nan  # at the draft: rejected; no residual there, and q is 0 at V - 3
    q[2, 0] = math.nan   # no residual at all: the target's own weights
    p[3, 0, 7] = math.nan  # rejected, without weight
    x = torch.full((4, 1), 7, dtype=torch.int32, device="cuda")
    zero, low = torch.zeros(4, 1, device="cuda"), torch.full((4,), 0.1, device="cuda")
    t, a = inv.spec_verify(p, q, x, zero, low)
    assert a.tolist() == [0] * 4 and t.tolist() == [[-1, -1], [V - 3, -1], [7, -1], [V - 3, -1]]
    t, a = inv.spec_verify(p, None, x, zero, low)  # looked-up drafts: accepted with u = 0 where p is a number
    assert a.tolist() == [0, 1, 1, 0] and t.tolist() == [[-1, -1], [7, 7], [7, 7], [V - 3, -1]]
    assert status() == inv.INV_OK


def test_kv_append_paged_with_nan(inv):  # noqa: F811
    """NaN in a key or value row: the codes and scales of kv_quant_int16; in a query: NaN."""
    hq, hkv, page, T = 4, 2, 16, 3
    n_pages, table, start, ln = batch([T], [T], page, seed=92)
    x = torch.randn(T, (hq + 2 * hkv) * 128, generator=gen(93), device="cuda")
    x[0, 5] = x[1, hq * 128 + 9] = x[2, (hq + hkv) * 128 + 100] = math.nan
    x[2, (hq + hkv + 1) * 128:] = math.nan  # a whole value row
    cos, sin = torch.ones(8, 64, device="cuda"), torch.zeros(8, 64, device="cuda")
    cache, slot = inv.PagedKVCache.empty(n_pages, hkv, page), inv.KVCache(n_slots=1, n_kv_heads=hkv, max_len=16)
    q = inv.kv_append_paged(x, cache, table, start, ln, cos, sin)
    assert torch.isnan(q[0, 0, [5, 69]]).all() and int(torch.isnan(q).sum()) == 2
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    y = x.view(T, -1, 128)
    k = y[:, hq:hq + hkv].clone()
    k[1, 0, 9] = k[1, 0, 73] = math.nan  # the rotated pair: x 1 - NaN 0
    inv.kv_quant_int16(k.contiguous(), torch.zeros_like(pos), pos, slot, "k")
    inv.kv_quant_int16(y[:, hq + hkv:].contiguous(), torch.zeros_like(pos), pos, slot, "v")
    pg = int(table[0, 0])
    bits = lambda t: t.view(torch.int32) if t.dtype == torch.float32 else t
    for a, b in ((cache.k, slot.k), (cache.v, slot.v), (cache.k_scale, slot.k_scale), (cache.v_scale, slot.v_scale)):
        assert torch.equal(bits(a)[pg, :, :T], bits(b)[0, :, :T])
    # fmax keeps the number beside a NaN, and a NaN of two
    assert torch.isnan(cache.v_scale[pg, 1, 2]) and int(torch.isnan(cache.v_scale).sum()) == 1
    assert not torch.isnan(cache.k_scale).any() and status() == inv.INV_OK


def test_the_index_checking_build_agrees_at_the_edges(inv):  # noqa: F811
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
