"""8-bit rows of the paged cache over the whole range of fp32 scales, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_ref

pytestmark = pytest.mark.gpu

D, PAGE = 64, 16
# half of bf16's smallest step: what the rounding of an output below 2^-126 may be off by
SMALLEST = 2.0 ** -134
# A value's scale goes into its weight by its logarithm: of size up to 149, off by 2^-22 of that
# (lg2.approx's bound), in up to four sums below 256, each rounded by at most 2^-17.
LOG = math.log(2) * (149 * 2.0 ** -22 + 4 * 2.0 ** -17)


@pytest.fixture(scope="module")
def sa():
    import sparse_graph_causal_b200 as m
    return m


def _pages(t):
    """Rows [T, Hkv, ...] in order as pages [n, Hkv, PAGE, ...]."""
    return t.view(-1, PAGE, *t.shape[1:]).transpose(1, 2).contiguous()


def _decode(sa, q, cache, T, W):
    table = torch.arange(T // PAGE, device="cuda", dtype=torch.int32)[None]
    g = sa.sparse_attn_graph_build_structured(T, W, [])
    out, lse = sa.sparse_attn_paged_decode(q, cache, table, torch.tensor([T - 1], device="cuda"), g,
                                           0.125)
    sa.sparse_attn_check_device()
    return out[0, :, 0].double().cpu().numpy(), lse[0].double().cpu().numpy()


def _check(out, lse, q, k, v, Hkv):
    """k, v: rows [T, Hkv, D] in 64 bits (numpy)."""
    G = q.shape[1] // Hkv
    for h in range(Hkv):
        heads = slice(h * G, h * G + G)
        o, l, size, vmax = paged_ref.attend(q[0, heads, 0].double().cpu().numpy(), k[:, h], v[:, h],
                                            0.125)
        t_lse, t_out, rel = paged_ref.tolerances(len(k), D, size, vmax, torch.bfloat16)
        assert (np.abs(lse[heads] - l) <= t_lse + 2.0 ** -24 * np.abs(l)).all()
        off = np.abs(out[heads] - o) - (t_out + LOG * vmax + rel * np.abs(o) + SMALLEST)
        # Sums are held in 32 bits and divided at the end, with the largest probability as 1:
        # sum_j p_j |v_j| has to stay in fp32's range, as the header says (a column whose sum
        # passes 2^127 may come out infinite).
        s = 0.125 * (q[0, heads, 0].double().cpu().numpy() @ k[:, h].T)
        fits = np.exp(s - s.max(1, keepdims=True)) @ np.abs(v[:, h]) < 2.0 ** 127
        assert (off[fits] <= 0).all(), (h, off[fits].max(), np.abs(o).max())


@pytest.mark.parametrize("H, Hkv", [(2, 2), (24, 2)])
@pytest.mark.parametrize("T", [16, 208, 30000])
@pytest.mark.parametrize("e", [100, 0, -80, -100, -108, -116, -122, -126])
def test_append_then_decode_of_values_of_any_size(sa, e, T, H, Hkv):
    """Values of about 2^e, written in 8 bits and read back: rows of one CTA and rows cut over the
    GPU, both tile widths."""
    gen = torch.Generator("cuda")
    gen.manual_seed(e + T)
    k, v = (torch.empty((T, Hkv, D), device="cuda", dtype=torch.float64).normal_(generator=gen)
            for _ in range(2))
    k, v = k.bfloat16(), (v * 2.0 ** e).bfloat16()
    q = torch.empty((1, H, 1, D), device="cuda").normal_(generator=gen).bfloat16()
    n = T // PAGE
    codes = [torch.zeros((n, Hkv, PAGE, D), device="cuda").to(torch.float8_e4m3fn) for _ in "kv"]
    scales = [torch.zeros((n, Hkv, PAGE), device="cuda") for _ in "kv"]
    cache = sa.PagedCache(*codes, *scales)
    sa.sparse_attn_paged_append(k, v, cache, torch.arange(T, device="cuda"))
    rows = []
    for x, c, s in zip((k, v), codes, scales):
        y, unit = paged_ref.quantise(x.float().cpu().numpy())
        rows.append(y * unit.astype(np.float64)[..., None])
        got = c.transpose(1, 2).reshape(T, Hkv, D).double().cpu().numpy()
        assert np.array_equal(got, y)
        assert np.array_equal(s.transpose(1, 2).reshape(T, Hkv).cpu().numpy(), unit)
    out, lse = _decode(sa, q, cache, T, T)
    _check(out, lse, q, *rows, Hkv)


@pytest.mark.parametrize("T", [208, 30000])
@pytest.mark.parametrize("lo, hi", [(-149, -140), (-135, -120), (-149, 118), (-30, 118)])
def test_decode_of_value_scales_of_any_size(sa, lo, hi, T):
    """Scales of any size side by side: the large ones decide, and alone the small ones count."""
    Hkv, H = 1, 4
    gen = torch.Generator("cuda")
    gen.manual_seed(T + lo)
    rng = np.random.default_rng(T + hi)
    scale = np.ldexp(1.0, rng.integers(lo, hi + 1, (T, Hkv))).astype(np.float32)
    code = torch.randint(0, 0x7f, (2, T, Hkv, D), device="cuda", generator=gen, dtype=torch.uint8)
    code |= torch.randint(0, 2, code.shape, device="cuda", generator=gen, dtype=torch.uint8) << 7
    code = code.view(torch.float8_e4m3fn)
    unit = torch.full((T, Hkv), 2.0 ** -8, device="cuda")
    cache = sa.PagedCache(*(_pages(c) for c in code), _pages(unit),
                          _pages(torch.from_numpy(scale).cuda()))
    q = torch.empty((1, H, 1, D), device="cuda").normal_(generator=gen).bfloat16()
    k, v = code.double().cpu().numpy()
    out, lse = _decode(sa, q, cache, T, T)
    _check(out, lse, q, k * 2.0 ** -8, v * scale.astype(np.float64)[..., None], Hkv)


def test_one_key_of_each_size(sa):
    """A row of one key: the output is its value, code * scale, rounded once."""
    T = 16
    q = torch.ones((1, 1, 1, D), device="cuda", dtype=torch.bfloat16)
    code = torch.arange(D, device="cuda", dtype=torch.uint8).add(0x3f).view(torch.float8_e4m3fn)
    code = code.expand(1, 1, PAGE, D).contiguous()
    unit = torch.zeros((1, 1, PAGE), device="cuda")
    for e in range(-149, 119):
        scale = torch.full((1, 1, PAGE), math.ldexp(1.0, e), device="cuda")
        out, lse = _decode(sa, q, sa.PagedCache(code, code, unit, scale), T, 1)
        v = code[0, 0, 0].double().cpu().numpy() * math.ldexp(1.0, e)
        _, t_out, rel = paged_ref.tolerances(1, D, 0.0, np.abs(v), torch.bfloat16)
        assert (np.abs(out[0] - v) <= t_out + (LOG + rel) * np.abs(v) + SMALLEST).all(), e
        assert abs(lse[0]) <= 2.0 ** -20
