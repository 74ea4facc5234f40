"""Host-side argument checks of the paged-cache operators (CPU only): every
call below returns its status before touching the GPU."""
import ctypes as C

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
PTR = C.c_void_p(0x100000)  # aligned dummy device address
ODD = C.c_void_p(0x100004)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def inv():
    from invariant_numerics_b200 import invnum
    return invnum


def cache(inv, n_pages=10, hkv=8, page=16, d=128, k=PTR.value):
    return inv.PagedKVCacheStruct(k, PTR.value, PTR.value, PTR.value, n_pages, hkv, page, d)


def append(inv, **kw):
    a = dict(qkv=PTR, ld=48 * 128, T=4, hq=32, c=cache(inv), table=PTR, ld_table=5, n=2, start=PTR, lens=PTR, cos=PTR,
             sin=PTR, max_pos=100, qg=None, kg=None, eps=1e-6, out=PTR)
    a.update(kw)
    c = a["c"]
    return inv.lib.kv_append_paged(a["qkv"], a["ld"], a["T"], a["hq"], None if c is None else C.byref(c), a["table"],
                                   a["ld_table"], a["n"], a["start"], a["lens"], a["cos"], a["sin"], a["max_pos"],
                                   a["qg"], a["kg"], a["eps"], a["out"], None)


def attend(inv, **kw):
    a = dict(q=PTR, ld=32 * 128, T=4, hq=32, c=cache(inv), table=PTR, ld_table=50, n=2, start=PTR, lens=PTR, mq=0,
             mlb=0, sigma=0.1, out=PTR, hi=None, lo=None, ws=PTR, nb=10 ** 12)
    a.update(kw)
    c = a["c"]
    return inv.lib.attn_paged(a["q"], a["ld"], a["T"], a["hq"], None if c is None else C.byref(c), a["table"],
                              a["ld_table"], a["n"], a["start"], a["lens"], a["mq"], a["mlb"], a["sigma"], a["out"],
                              a["hi"], a["lo"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("call", [append, attend])
def test_what_both_refuse(inv, call):
    assert call(inv, T=0) == OK and call(inv, n=0) == OK
    assert call(inv, c=None) == INVALID
    assert call(inv, T=-1) == INVALID and call(inv, n=-1) == INVALID and call(inv, ld_table=-1) == INVALID
    assert call(inv, hq=0) == INVALID
    for name in ("table", "start", "lens", "out"):
        assert call(inv, **{name: None}) == INVALID, name
    for c, want in ((cache(inv, d=64), UNSUPPORTED), (cache(inv, page=8), UNSUPPORTED), (cache(inv, page=48), UNSUPPORTED),
                    (cache(inv, page=512), UNSUPPORTED), (cache(inv, n_pages=0), INVALID), (cache(inv, hkv=0), INVALID),
                    (cache(inv, hkv=5), UNSUPPORTED), (cache(inv, n_pages=1 << 27), UNSUPPORTED),
                    (cache(inv, k=None), INVALID), (cache(inv, k=ODD.value), INVALID)):
        assert call(inv, c=c) == want


def test_append_refusals(inv):
    assert append(inv, ld=48 * 128 - 4) == INVALID and append(inv, ld=48 * 128 + 2) == INVALID
    assert append(inv, qkv=None) == INVALID and append(inv, qkv=ODD) == INVALID
    assert append(inv, cos=None) == INVALID and append(inv, sin=None) == INVALID and append(inv, max_pos=0) == INVALID
    assert append(inv, eps=-1e-6) == INVALID and append(inv, eps=NAN) == INVALID
    for name in ("qg", "kg", "out", "cos"):
        assert append(inv, **{name: ODD}) == INVALID, name


def test_attend_refusals(inv):
    assert attend(inv, ld=32 * 128 - 4) == INVALID and attend(inv, ld=32 * 128 + 2) == INVALID
    assert attend(inv, q=None) == INVALID and attend(inv, q=ODD) == INVALID and attend(inv, out=ODD) == INVALID
    assert attend(inv, hi=PTR) == INVALID and attend(inv, lo=PTR) == INVALID
    assert attend(inv, hi=ODD, lo=PTR) == INVALID
    for s in (-0.1, INF, NAN):
        assert attend(inv, sigma=s) == INVALID
    assert attend(inv, hq=17 * 8, ld=17 * 8 * 128) == UNSUPPORTED
    need = inv.lib.attn_paged_workspace_size(4, 2, 32, 8, 4, 800)
    assert need > 0 and attend(inv, nb=need - 1) == WORKSPACE and attend(inv, ws=ODD) == INVALID
    assert attend(inv, nb=0) == WORKSPACE and attend(inv, ws=None) == INVALID


def test_workspace_size(inv):
    f = inv.lib.attn_paged_workspace_size
    for bad in ((0, 2, 32, 8, 4, 800), (4, 0, 32, 8, 4, 800), (4, 2, 0, 8, 4, 800), (4, 2, 32, 0, 4, 800),
                (4, 2, 32, 8, 4, 0)):
        assert f(*bad) == 0
    assert f(4, 2, 32, 8, 4, 8192) >= f(4, 2, 32, 8, 4, 4096) >= f(4, 2, 32, 8, 4, 513)


def test_softmax_refusals(inv):
    f = inv.lib.softmax_rows
    assert f(PTR, 0, 10, 10, 1.0, PTR, 10, None) == OK
    assert f(PTR, -1, 10, 10, 1.0, PTR, 10, None) == INVALID
    assert f(PTR, 2, 0, 10, 1.0, PTR, 10, None) == INVALID
    assert f(PTR, 2, 10, 9, 1.0, PTR, 10, None) == INVALID and f(PTR, 2, 10, 10, 1.0, PTR, 9, None) == INVALID
    for t in (0.0, -1.0, INF, NAN):
        assert f(PTR, 2, 10, 10, t, PTR, 10, None) == INVALID
    assert f(None, 2, 10, 10, 1.0, PTR, 10, None) == INVALID and f(PTR, 2, 10, 10, 1.0, None, 10, None) == INVALID
    assert f(PTR, 2, 10, 12, 1.0, PTR, 10, None) == INVALID  # in place with another stride


def test_verify_refusals(inv):
    f = inv.lib.spec_verify
    ok = [PTR, 100, PTR, 100, 2, 3, 100, PTR, None, PTR, PTR, PTR, PTR]
    call = lambda **kw: f(*[kw.get(f"a{i}", x) for i, x in enumerate(ok)], None)
    assert call(a4=0) == OK
    assert call(a4=-1) == INVALID and call(a5=-1) == INVALID and call(a6=0) == INVALID
    assert call(a1=99) == INVALID and call(a3=99) == INVALID
    for i in (0, 7, 9, 10, 11, 12):
        assert call(**{f"a{i}": None}) == INVALID, i


def test_binding_refuses_cpu_tensors_and_wrong_shapes(inv):
    import torch
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        inv.PagedKVCache(z(2, 1, 16, 128, dtype=torch.int16), z(2, 1, 16, 128, dtype=torch.int16), z(2, 1, 16), z(2, 1, 16))
    with pytest.raises(ValueError, match="paged cache"):
        inv.PagedKVCache(z(2, 1, 16, 128, dtype=torch.int16), z(2, 1, 16, 64, dtype=torch.int16), z(2, 1, 16), z(2, 1, 16))
    with pytest.raises(ValueError, match="CUDA"):
        inv.softmax_rows(z(2, 5))
    with pytest.raises(ValueError, match="CUDA"):
        inv.spec_verify(z(1, 2, 5), None, z(1, 1, dtype=torch.int32), z(1, 1), z(1))


def test_the_largest_bounds(inv):
    """Bounds next to 2^31 keep their sizes positive, and what no launch can hold is refused."""
    # 4 rows of 32 heads, 2^22 segments of 512 keys, 128 sums and (m, l) each
    assert inv.lib.attn_paged_workspace_size(4, 2, 32, 8, 0, 2 ** 31 - 1) == 4 * 32 * 2 ** 22 * (128 * 4 + 8)
    assert attend(inv, ld_table=1 << 40, nb=0) == WORKSPACE
    assert attend(inv, ld_table=0) == INVALID and attend(inv, ld_table=0, T=0) == OK
    assert attend(inv, hq=70000, ld=70000 * 128, c=cache(inv, hkv=70000)) == UNSUPPORTED


@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 1), (8, 8), (24, 8)])
@pytest.mark.parametrize("n_seqs", [1, 3, 40])
@pytest.mark.parametrize("bound", [300, 8192, 131072])
def test_a_workspace_serves_every_smaller_call(inv, hq, hkv, n_seqs, bound):
    """The size for T tokens lets calls of fewer tokens, sequences and keys through, whatever plan these prefer; and the
    least that is documented is what a call takes."""
    size = inv.lib.attn_paged_workspace_size
    c = cache(inv, hkv=hkv)
    few, S = 32 * hkv // hq, -(-bound // 512)

    def passes(nb, T, n=n_seqs, mq=0, mlb=bound):
        # without a pointer: INVALID once the size will do (OK is not reached on a CPU), WORKSPACE before
        rc = attend(inv, T=T, n=n, hq=hq, ld=hq * 128, c=c, ld_table=1 << 14, mq=mq, mlb=mlb, ws=None, nb=nb)
        assert rc in (INVALID, WORKSPACE)
        return rc == INVALID

    tokens = [1, 2, few, few + 1, 2 * few, 33, 64, 100, 300, 512, 700, 1000, 1100, 1152, 2000, 3000, 8192]
    for T in tokens:
        mq = T if S == 1 and T * hq <= 32 * hkv else 0
        if mq:
            assert size(T, n_seqs, hq, hkv, mq, bound) == 0
            continue
        least = min(T, n_seqs * few) * hq * S * 520
        assert passes(least, T) and not passes(least - 1, T)
        nb = size(T, n_seqs, hq, hkv, T, bound)
        assert nb >= least
        for fewer in tokens:
            if fewer <= T and not (S == 1 and fewer <= few):
                assert passes(nb, fewer) and passes(nb, fewer, n=1)
                assert bound < 1000 or passes(nb, fewer, mlb=bound // 2 + 1)


def test_the_longest_sequence(inv):
    """Lengths end at 2^31 - 512, whatever the page table could hold and the bound says: 2^22 - 1 segments."""
    c = cache(inv, hkv=8)
    least = 8 * 520 * (2 ** 22 - 1)
    for ld_table, mlb in ((1 << 40, 0), (1 << 40, 2 ** 31 - 1), (2 ** 27, 0), (2 ** 27, 2 ** 31 - 512)):
        call = lambda nb: attend(inv, T=1, n=1, hq=8, ld=1024, c=c, ld_table=ld_table, mlb=mlb, ws=None, nb=nb)
        assert call(least) == INVALID and call(least - 1) == WORKSPACE  # (no pointer: INVALID once the size will do)


def test_verify_refuses_more_drafts_than_its_counters_hold(inv):
    f = inv.lib.spec_verify
    for m, want in ((2 ** 31 - 1, INVALID), (2 ** 30 + 1, INVALID), (2 ** 30, OK)):
        assert f(PTR, 100, None, 0, 0, m, 100, PTR, None, PTR, PTR, PTR, PTR, None) == want


def test_the_index_checking_build_covers_the_operators(inv):
    """Every kernel of the paged-cache operators and of verification asks before it reads or writes a caller's buffer,
    descriptors and page tables included."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_numerics_b200", "csrc")
    text = {n: re.sub(r"//.*", "", open(os.path.join(csrc, n)).read())
            for n in ("paged.cuh", "kv_append.cu", "attn_paged.cu", "sampling.cu")}
    for name, needs in (("kv_append.cu", ["kv_append_kernel"]),
                        ("attn_paged.cu", ["attn_few_kernel", "attn_many_kernel", "attn_fold_kernel"]),
                        ("sampling.cu", ["softmax_kernel", "softmax_long_kernel", "accepted_prefix", "write_prefix",
                                         "rows_in_bounds"]),
                        ("paged.cuh", ["start_of", "len_of", "page_of"])):
        for f in needs:
            body = re.search(r"\b%s\([^;{]*\{.*?\n\}" % f, text[name], re.S).group(0)
            assert "_IN_BOUNDS(" in body, f
    for f in ("spec_verify_kernel", "spec_verify_long_kernel"):
        body = re.search(r"\b%s\([^;{]*\{.*?\n\}" % f, text["sampling.cu"], re.S).group(0)
        assert all(g + "(a, b" in body for g in ("accepted_prefix", "write_prefix", "rows_in_bounds")), f
    # the descriptors are read in these places only
    for n in ("kv_append.cu", "attn_paged.cu"):
        assert not re.search(r"\brb\.(q_start|len|page_table)\s*\[", text[n]), n
