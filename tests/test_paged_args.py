"""Paged cache on the host: refusals of the C entry points and of the Python
binding before anything is launched, and the plain statements that the GPU
tests compare with.  No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

import paged_ref


@pytest.fixture(scope="module")
def sa():
    import sparse_graph_causal_b200 as m
    return m


# addresses that are never touched: the calls below are refused on the host
BUF = ctypes.create_string_buffer(4096)
A = (ctypes.addressof(BUF) + 255) // 256 * 256
OK, INVALID, UNSUPPORTED = 0, 1, 3


def _step(sa, **change):
    f = dict(B=4, max_pages=8, page_size=16, capacity=32, n_stack=64)
    f.update({n: A for n in ("len", "n_new", "block_table", "free_pages", "free_count", "len_out",
                             "free_count_out", "cu_new", "slot", "pos", "row", "status")})
    f.update(change)
    d = sa.SaPagedStep()
    for k, v in f.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("change, status", [
    (dict(B=0), INVALID), (dict(B=8193), UNSUPPORTED), (dict(max_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(capacity=0), INVALID), (dict(n_stack=0), INVALID),
    (dict(capacity=1 << 31), UNSUPPORTED), (dict(capacity=(1 << 30) + 1), UNSUPPORTED), (dict(n_stack=1 << 31), UNSUPPORTED),
    (dict(max_pages=1 << 30, page_size=2), UNSUPPORTED),
    (dict(max_pages=1, page_size=1 << 31), UNSUPPORTED),
    (dict(len=None), INVALID), (dict(n_new=None), INVALID), (dict(block_table=None), INVALID),
    (dict(free_pages=None), INVALID), (dict(free_count=None), INVALID),
    (dict(len_out=None), INVALID), (dict(free_count_out=None), INVALID),
    (dict(cu_new=None), INVALID), (dict(slot=None), INVALID), (dict(pos=None), INVALID),
    (dict(row=None), INVALID), (dict(status=None), INVALID),
    (dict(len=A + 4), INVALID), (dict(slot=A + 4), INVALID), (dict(row=A + 2), INVALID),
    (dict(block_table=A + 1), INVALID),
], ids=str)
def test_plan_refusals(sa, change, status):
    d = _step(sa, **change)
    assert sa._lib.sparse_attn_paged_plan(ctypes.byref(d), None) == status
    assert sa._lib.sparse_attn_paged_plan(None, None) == INVALID


def _cache(sa, **change):
    f = dict(k=A, v=A, k_scale=None, v_scale=None, dtype=sa.SA_BF16, n_pages=8, Hkv=2,
             page_size=16, D=64)
    f.update(change)
    d = sa.SaPagedCache()
    for k, v in f.items():
        setattr(d, k, v)
    return d


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=A + 8), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(n_pages=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(page_size=0), INVALID), (dict(D=0), INVALID),
    (dict(D=96), UNSUPPORTED), (dict(k_scale=A), INVALID), (dict(v_scale=A), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=2, k_scale=A), INVALID),
    (dict(dtype=2, k_scale=A + 2, v_scale=A), INVALID),
    (dict(n_pages=1 << 31), UNSUPPORTED), (dict(Hkv=(1 << 24) + 1), UNSUPPORTED), (dict(page_size=1 << 31), UNSUPPORTED),
]


def _append(sa, cache, k=None, v=None, ks=128, vs=128, slot=A):
    k = k or sa.SaTensor(A, sa.SA_BF16, 4, 2, 1, 64)
    v = v or sa.SaTensor(A, sa.SA_BF16, 4, 2, 1, 64)
    return sa._lib.sparse_attn_paged_append(ctypes.byref(k), ks, ctypes.byref(v), vs, slot,
                                            ctypes.byref(cache), None)


@pytest.mark.parametrize("change, status", BAD_CACHES, ids=str)
def test_cache_refusals(sa, change, status):
    c = _cache(sa, **change)
    assert _append(sa, c) == status
    q, o = (sa.SaTensor(A, sa.SA_BF16, 4, 4, 1, 64) for _ in range(2))
    g = ctypes.c_void_p(A)   # not looked at before the cache is
    assert sa._lib.sparse_attn_paged_decode(
        ctypes.byref(q), ctypes.byref(c), A, 4, 8, None, A, g, 1.0, ctypes.byref(o), A, A, 4096,
        None) == status
    assert sa._lib.sparse_attn_paged_decode_workspace_size(ctypes.byref(q), ctypes.byref(c), g) == 0


def test_append_refusals(sa):
    T = sa.SaTensor
    c = _cache(sa)
    bad = [
        dict(k=T(A, 0, 4, 3, 1, 64)), dict(k=T(A, 0, 4, 2, 2, 64)), dict(k=T(A, 0, 4, 2, 1, 32)),
        dict(k=T(A, 1, 4, 2, 1, 64)), dict(k=T(A + 8, 0, 4, 2, 1, 64)), dict(k=T(A, 0, 0, 2, 1, 64)),
        dict(k=T(None, 0, 4, 2, 1, 64)), dict(v=T(A, 0, 5, 2, 1, 64)), dict(v=T(A, 1, 4, 2, 1, 64)),
        dict(ks=127), dict(ks=120), dict(vs=132), dict(vs=-128), dict(slot=None), dict(slot=A + 4),
    ]
    for x in bad:
        assert _append(sa, c, **x) == INVALID, x
    # an 8-bit cache takes bf16 rows only
    c8 = _cache(sa, dtype=2, k_scale=A, v_scale=A)
    r = T(A, sa.SA_FP32, 4, 2, 1, 64)
    assert _append(sa, c8, k=r, v=r) == INVALID
    assert sa._lib.sparse_attn_paged_append(None, 128, None, 128, A, ctypes.byref(c), None) == INVALID


def test_decode_refusals(sa):
    T = sa.SaTensor
    h = ctypes.c_void_p()

    def call(q=None, o=None, table=A, rows=4, M=8, row=None, pos=A, g=ctypes.c_void_p(A), scale=1.0,
             lse=A):
        q, o = q or T(A, 0, 4, 4, 1, 64), o or T(A, 0, 4, 4, 1, 64)
        c = _cache(sa)
        return sa._lib.sparse_attn_paged_decode(
            ctypes.byref(q), ctypes.byref(c), table, rows, M, row, pos, g, scale, ctypes.byref(o),
            lse, A, 1 << 30, None)

    for x in (dict(g=h), dict(q=T(A, 0, 4, 3, 1, 64)), dict(q=T(A, 0, 4, 4, 2, 64)),
              dict(q=T(A, 1, 4, 4, 1, 64)), dict(o=T(A, 0, 4, 2, 1, 64)), dict(o=T(A, 1, 4, 4, 1, 64)),
              dict(o=T(A + 2, 0, 4, 4, 1, 64)), dict(table=None), dict(table=A + 2), dict(rows=0),
              dict(rows=3), dict(M=0), dict(row=A + 2), dict(pos=None), dict(pos=A + 4),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(lse=None), dict(lse=A + 4)):
        assert call(**x) == INVALID, x
    assert call(M=1 << 27) == UNSUPPORTED        # 2^27 pages of 16 rows
    assert call(M=(1 << 26) + 1) == UNSUPPORTED  # more than 2^30 positions
    assert call(rows=1 << 31) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_types(sa):
    x = torch.zeros(2, 1, 16, 64)
    with pytest.raises(ValueError):
        sa.PagedCache(x, x)
    i = torch.zeros(4, 8, dtype=torch.int32)
    with pytest.raises(ValueError):
        sa.sparse_attn_paged_plan(i, i, i, i, i, 16, None)


# ------------------------------------------------- the plain statements

def test_plan_statement_by_hand():
    """Three requests with pages of 4: one finishes, one grows over a page
    border, one does not fit."""
    table = np.array([[7, 5, -1], [3, -1, -1], [-1, -1, -1]], np.int32)
    stack = np.array([9, 8, -1, -1, -1], np.int32)
    r = paged_ref.plan([6, 3, 0], [-1, 2, 12], table, stack, 2, 4, 16)
    # pages 7, 5 come back: 9 8 7 5; request 1 takes 5; request 2 needs 3: 7 8 9
    assert r["stack"].tolist() == [9, 8, 7, 5, -1]
    assert r["table"].tolist() == [[7, 5, -1], [3, 5, -1], [7, 8, 9]]
    assert r["length"].tolist() == [0, 5, 12] and r["count"] == 0
    assert r["cu_new"].tolist() == [0, 0, 2, 14] and r["status"].tolist() == [0, 0, 0]
    assert r["slot"].tolist()[:4] == [15, 20, 28, 29] and r["slot"][14:].tolist() == [-1, -1]
    assert r["pos"].tolist()[:4] == [3, 4, 0, 1]
    r = paged_ref.plan([6, 3, 0], [0, 2, 12], table, stack, 2, 4, 16)
    assert r["status"].tolist() == [0, 0, 1] and r["count"] == 1
    assert r["length"].tolist() == [6, 5, 0] and set(r["slot"][2:]) == {-1}


def test_e4m3_statement_agrees_with_the_type():
    y = np.linspace(-448, 448, 30001).astype(np.float32)
    y = np.concatenate([y, y * 2.0 ** -9, y * 2.0 ** -14]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(paged_ref.e4m3_round(y.astype(np.float64)), want)


def _rounded(num, den):
    """num / den > 0 to 24 significant bits, halves to even: (significand, exponent)."""
    e = num.bit_length() - den.bit_length() - 24
    while True:
        n, d = (num << -e, den) if e < 0 else (num, den << e)
        q, r = divmod(n, d)
        if 1 << 23 <= q < 1 << 24:
            q += 2 * r > d or (2 * r == d and q & 1)
            return (q, e) if q < 1 << 24 else (q >> 1, e + 1)
        e += 1 if q >> 24 else -1


def _code(m, e):
    """m * 2^e rounded to e4m3, as a multiple of 2^-9."""
    step = max(m.bit_length() + e - 1, -6) - 3
    shift = step - e
    if shift > 0:
        q, r, half = m >> shift, m & ((1 << shift) - 1), 1 << (shift - 1)
        m = q + (r > half or (r == half and q & 1))
    else:
        m <<= -shift
    return m << (step + 9)


def test_quotients_off_by_2_to_the_minus_45_have_the_same_codes():
    """The rounding of 8-bit rows divides with one correction step, whose result is the rounding
    of a quotient off by at most 2^-45: over all significands of a bf16 value and of its row's
    largest magnitude, the code is that of the correctly rounded quotient, and so is the scale."""
    lo, hi = (1 << 45) - 1, (1 << 45) + 1
    for A in range(128, 256):
        S, e = _rounded(A, 448)
        assert {_rounded(A * lo, 448 << 45), _rounded(A * hi, 448 << 45)} == {(S, e)}
        for X in range(128, 256):
            for j in range(24):                      # x = X 2^-j, amax = A
                if X <= A << j:
                    num, den = X << -e, S << j       # e < 0
                    code = _code(*_rounded(num, den))
                    assert _code(*_rounded(num * lo, den << 45)) == code
                    assert _code(*_rounded(num * hi, den << 45)) == code


def test_attend_statement_by_hand():
    q = np.array([[1.0, 0.0]])
    k = np.array([[0.0, 5.0], [np.log(3.0), 1.0]])
    v = np.array([[4.0, 0.0], [0.0, 8.0]])
    out, lse, _, _ = paged_ref.attend(q, k, v, 1.0)
    assert np.allclose(out, [[1.0, 6.0]]) and np.allclose(lse, [np.log(4.0)])
    out, lse, _, _ = paged_ref.attend(q, k[:0], v[:0], 1.0)
    assert not out.any() and np.isneginf(lse).all()
