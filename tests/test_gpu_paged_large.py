"""A cache of more than 2^31 rows: slots, pages and offsets beyond 32 bits."""
import numpy as np
import pytest
import torch

import paged_ref

pytestmark = pytest.mark.gpu


def test_slots_above_31_bits():
    import sparse_graph_causal_b200 as sa
    D, page = 32, 1024
    n_pages = (1 << 31) // page + 40
    if torch.cuda.mem_get_info()[0] < 1.1 * n_pages * page * (D + 4):
        pytest.skip("not enough device memory")
    # (keys and values are the same rows: one tensor serves as both)
    pool = torch.empty((n_pages, 1, page, D), device="cuda", dtype=torch.float8_e4m3fn)
    scale = torch.empty((n_pages, 1, page), device="cuda")
    cache = sa.PagedCache(pool, pool, scale, scale)
    T = 3 * page
    gen = torch.Generator("cuda")
    gen.manual_seed(1)
    x = torch.empty((T, 1, D), device="cuda").normal_(generator=gen).bfloat16()
    table = torch.tensor([[n_pages - 1, (1 << 31) // page - 1, (1 << 31) // page + 7]],
                         dtype=torch.int32, device="cuda")
    at = torch.arange(T, device="cuda")
    slot = table[0].long()[at // page] * page + at % page
    assert int(slot.min()) < 1 << 31 < int(slot.max())
    sa.sparse_attn_paged_append(x, x, cache, slot)
    sa.sparse_attn_check_device()
    y, unit = paged_ref.quantise(x.float().cpu().numpy())
    rows = pool.view(torch.uint8)[table[0].long(), 0].view(T, D).view(pool.dtype)
    assert np.array_equal(rows.double().cpu().numpy(), y[:, 0])
    assert np.array_equal(scale[table[0].long(), 0].view(T).cpu().numpy(), unit[:, 0])
    # one past the end, and far past it
    bad = torch.tensor([n_pages * page, (1 << 40) + 3, -1], device="cuda")
    sa.sparse_attn_paged_append(x[:3], x[:3], cache, bad)
    with pytest.raises(sa.SparseAttentionError):
        sa.sparse_attn_check_device()
    q = torch.empty((1, 2, 1, D), device="cuda").normal_(generator=gen).bfloat16()
    kv = (y * unit.astype(np.float64)[..., None])[:, 0]
    for W in (100, T):
        g = sa.sparse_attn_graph_build_structured(T, W, [])
        out, lse = sa.sparse_attn_paged_decode(q, cache, table, torch.tensor([T - 1], device="cuda"),
                                               g, 0.2)
        sa.sparse_attn_check_device()
        o, l, size, vmax = paged_ref.attend(q[0, :, 0].double().cpu().numpy(), kv[T - W:],
                                            kv[T - W:], 0.2)
        t_lse, t_out, rel = paged_ref.tolerances(W, D, size, vmax, torch.bfloat16)
        assert (np.abs(out[0, :, 0].double().cpu().numpy() - o) <= t_out + rel * np.abs(o)).all()
        assert (np.abs(lse[0].double().cpu().numpy() - l) <= t_lse + 2.0 ** -24 * np.abs(l)).all()
