"""Finished requests whose pages do not all fit on the stack, written out by hand: the page plan's
plain statement on the CPU, the kernel on the GPU."""
import numpy as np
import pytest
import torch

import paged_ref

OK, NO_PAGES, REFUSED = 0, 1, 2


def _case():
    """Pages of 4 rows, 12 to a request.  Requests: two finished pages, a running one, ten finished
    pages, three finished pages, one that is finished and holds nothing, one finished page, a prompt."""
    length = [8, 5, 40, 12, 0, 3, 0]
    n_new = [-1, 1, -1, -1, -1, -1, 9]
    table = np.full((7, 12), -1, np.int32)
    at = 100
    for b, L in enumerate(length):
        for p in range(-(-L // 4)):
            table[b, p] = at = at + 1
    stack = np.array([10, 11, 12, -1, -1, -1, -1, -1], np.int32)   # three pages, room for five
    return np.array(length), np.array(n_new, np.int32), table, stack, 3, 4, 12


def _want(table):
    """2 pages go on the stack and leave room for 3; the 10 do not fit; the 3 behind them would, and
    so would the 1, but none overtakes.  The prompt takes 3 pages from the top."""
    first = table[0, :2].tolist()
    after = table.copy()
    after[6, :3] = [first[1], first[0], 12]
    return dict(status=[OK, OK, REFUSED, REFUSED, OK, REFUSED, OK], length=[0, 6, 40, 12, 0, 3, 9],
                count=2, stack=[10, 11, 12, *first, -1, -1, -1], table=after,
                cu_new=[0, 0, 1, 1, 1, 1, 1, 10],
                row=[1] + [6] * 9 + [-1] * 2, pos=[5, *range(9), -1, -1],
                slot=[int(table[1, 1]) * 4 + 1]
                + [int(after[6, j // 4]) * 4 + j % 4 for j in range(9)] + [-1, -1])


def _check(got, want):
    for k, w in want.items():
        assert np.array_equal(np.asarray(got[k]), np.asarray(w)), (k, got[k], w)


def test_statement():
    length, n_new, table, stack, count, page, capacity = _case()
    _check(paged_ref.plan(length, n_new, table, stack, count, page, capacity), _want(table))


@pytest.mark.gpu
@pytest.mark.parametrize("capacity", [12, 3000, 40000])   # one CTA, eight, sixteen
def test_kernel(capacity):
    import sparse_graph_causal_b200 as sa
    length, n_new, table, stack, count, page, _ = _case()
    put = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to("cuda", t)  # noqa: E731
    dl, dt, ds = put(length, torch.int64), put(table, torch.int32), put(stack, torch.int32)
    dc = torch.tensor([count], device="cuda")
    b = sa.sparse_attn_paged_plan(dl, put(n_new, torch.int32), dt, ds, dc, page,
                                  sa.PagedBatch(len(length), capacity))
    got = {k: t.cpu().numpy() for k, t in dict(
        length=dl, table=dt, stack=ds, cu_new=b.cu_new, slot=b.slot, pos=b.pos, row=b.row,
        status=b.status).items()}
    got["count"] = int(dc)
    for k in ("slot", "pos", "row"):
        assert (got[k][12:] == -1).all()
        got[k] = got[k][:12]
    _check(got, _want(table))
