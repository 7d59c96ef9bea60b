"""Which of its two ways the paged decode goes: one CTA to a row (one launch) or equal shares of all
rows and a join (two)."""
import numpy as np
import pytest
import torch

import paged_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    import sparse_graph_causal_b200 as m
    return m


def _call(sa, N, Hkv, D, W, links, T, page=32, G=1):
    """A bf16 cache of N requests at random positions beyond a window; (launches, check)."""
    rng = np.random.default_rng(W + links + N)
    gen = torch.Generator("cuda")
    gen.manual_seed(W + N)
    pos = rng.integers(W, T, N)
    M = -(-T // page)
    need = np.zeros((N, M), bool)
    keys = []
    for n, p in enumerate(pos):
        far = [p - (1 << x) for x in range(links) if W <= 1 << x <= p]
        keys.append(np.array(sorted(far) + list(range(max(0, p - W + 1), p + 1))))
        need[n, keys[n] // page] = True
    table = np.full((N, M), -1, np.int32)
    n_pages = int(need.sum())
    table[need] = rng.permutation(n_pages)
    k, v = (torch.empty((n_pages, Hkv, page, D), device="cuda",
                        dtype=torch.bfloat16).normal_(generator=gen) for _ in range(2))
    q = torch.empty((N, Hkv * G, 1, D), device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    g = sa.sparse_attn_graph_build_structured(T, W, list(range(links)))
    args = (q, sa.PagedCache(k, v), torch.from_numpy(table).cuda(), torch.from_numpy(pos).cuda(), g)
    before = sa.sparse_attn_launch_count()
    out, lse = sa.sparse_attn_paged_decode(*args, 0.125)
    launches = sa.sparse_attn_launch_count() - before
    sa.sparse_attn_check_device()
    for n in range(0, N, 5):
        for h in range(0, Hkv, 3):
            at = torch.from_numpy(table[n, keys[n] // page]), h, torch.from_numpy(keys[n] % page)
            heads = slice(h * G, h * G + G)
            o, l, size, vmax = paged_ref.attend(q[n, heads, 0].double().cpu().numpy(),
                                                *(x[at].double().cpu().numpy() for x in (k, v)),
                                                0.125)
            t_lse, t_out, rel = paged_ref.tolerances(len(keys[n]), D, size, vmax, torch.bfloat16)
            assert (np.abs(lse[n, heads].double().cpu().numpy() - l)
                    <= t_lse + 2.0 ** -24 * np.abs(l)).all()
            assert (np.abs(out[n, heads, 0].double().cpu().numpy() - o)
                    <= t_out + rel * np.abs(o)).all()
    return launches


@pytest.mark.parametrize("N", [14, 16, 18])
def test_windows_of_neighbouring_lengths_go_one_way(sa, N):
    """A few keys or links more, or rows more or fewer, change nothing in how a batch of equal
    windows is shared out."""
    ways = {_call(sa, N, 8, 128, W, links, 20000)
            for W, links in ((4000, 0), (4096, 0), (4097, 0), (4096, 15), (4200, 15))}
    assert ways == {1}


def test_long_windows_go_in_shares(sa):
    assert _call(sa, 16, 8, 128, 5400, 0, 22000) == 2
    assert _call(sa, 2, 8, 128, 4096, 0, 20000) == 2      # few rows
