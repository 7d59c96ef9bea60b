"""The paged decode's equal shares of all rows (two launches: the shares and the join), at sizes
where that way is taken whatever the limits of the other one: the longest row that the graph allows
is above 2.5 MB.  Every test asserts that it was taken."""
import numpy as np
import pytest
import torch

import paged_ref
from test_gpu_paged import TYPES, Case, _gpu, _server

pytestmark = pytest.mark.gpu

BYTES = {"bf16": 2, "fp32": 4, "e4m3": 1}


@pytest.fixture(scope="module")
def sa():
    import sparse_graph_causal_b200 as m
    return m


def _long(D, dtype):
    """A sequence length whose whole row has more than 2.5 MB of keys and values."""
    return 2_700_000 // (2 * D * BYTES[dtype]) + 7


def _in_shares(sa, call):
    before = sa.sparse_attn_launch_count()
    got = call()
    assert sa.sparse_attn_launch_count() - before == 2
    return got


# --------------------------------------------- more tokens than a CTA has threads

def _positions(kind, N, T, rng):
    if kind == "short":           # at most 200 keys, a tenth padded
        pos = rng.integers(0, 200, N)
        pos[rng.random(N) < 0.1] = -1
        return pos
    if kind == "ragged":          # a few rows reach far, one to the end
        pos = rng.integers(-1, 150, N)
        pos[rng.integers(0, N, 4)] = rng.integers(1000, T // 2, 4)
        pos[rng.integers(0, N)] = T - 1
        return pos
    if kind == "ends":            # long rows first and last, nothing but padding between
        pos = np.full(N, -1)
        pos[0], pos[-1] = T - 1, T // 3
        return pos
    pos = np.full(N, -1)          # "one": a single token, somewhere
    pos[N * 2 // 3] = 77
    return pos


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D, H, Hkv", [(32, 2, 1), (64, 4, 2), (128, 3, 1), (32, 12, 1),
                                       (128, 16, 1)])
@pytest.mark.parametrize("N, kind", [(257, "short"), (385, "ragged"), (400, "ends"), (700, "ragged"),
                                     (1025, "short"), (1025, "one")])
def test_more_tokens_than_threads(sa, N, kind, D, H, Hkv, dtype):
    rng = np.random.default_rng(N + D + H)
    T = _long(D, dtype)
    pos = _positions(kind, N, T, rng)
    c = Case(pos, H, Hkv, D, 64, dtype, T, T, seed=N)
    assert sa.sparse_attn_paged_decode_workspace_size(c.q, c.cache(sa), c.graph(sa)) > 0
    out, lse = _in_shares(sa, lambda: c.run(sa))
    sa.sparse_attn_check_device()
    far = set(np.argsort(pos)[-6:])
    look = far | set(range(0, N, 23)) | {N - 1}
    c.check(out, lse, skip=set(range(N)) - look)
    assert not out[torch.from_numpy(pos < 0)].any()
    assert torch.isneginf(lse[torch.from_numpy(pos < 0)]).all()
    assert torch.isfinite(lse[torch.from_numpy(pos >= 0)]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_tokens_of_requests_beyond_the_threads(sa, dtype):
    """A step of prompts: 900 tokens of 5 requests, each with its row and its place."""
    T, D = _long(64, dtype), 64
    first, count = [0, 500, 3000, 0, 1], [300, 250, 200, 149, 1]
    row = np.repeat(np.arange(5), count)
    pos = np.concatenate([f + np.arange(n) for f, n in zip(first, count)])
    c = Case(pos, 4, 2, D, 32, dtype, T, T, row=row)
    out, lse = _in_shares(sa, lambda: c.run(sa))
    sa.sparse_attn_check_device()
    c.check(out, lse, skip=set(range(900)) - set(range(0, 900, 29)))
    # each token as if it were alone
    for n in (0, 299, 300, 555, 700, 899):
        one = Case.__new__(Case)
        one.__dict__.update(c.__dict__, pos=c.pos[n:n + 1], row=c.row[n:n + 1], q=c.q[n:n + 1], N=1,
                            keys=[c.keys[n]])
        o, l = sa.sparse_attn_paged_decode(
            one.q, c.cache(sa), _gpu(c.table, torch.int32), _gpu(one.pos, torch.int64), c.graph(sa),
            c.scale, row=_gpu(one.row, torch.int32))
        one.check(o, l)


# -------------------------------------------------------------- flags and scales

@pytest.mark.parametrize("dtype", list(TYPES))
def test_bad_positions_rows_and_pages(sa, dtype):
    T = _long(64, dtype)
    c = Case([T - 1, 1234, 50, 2500, T - 100, 999], 4, 2, 64, 16, dtype, T, T)
    n_pages = c.pool[0][0].shape[0]
    c.pos[1], c.pos[2] = T, -2
    c.keys[1] = c.keys[2] = np.zeros(0, np.int64)
    c.table[3, 2500 // 16] = -1
    c.table[4, 5000 // 16] = n_pages
    for n, p in ((3, 2500 // 16), (4, 5000 // 16)):
        c.keys[n] = c.keys[n][c.keys[n] // 16 != p]
    out, lse = _in_shares(sa, lambda: sa.sparse_attn_paged_decode(
        c.q, c.cache(sa), _gpu(c.table, torch.int32), _gpu(c.pos, torch.int64), c.graph(sa),
        c.scale, row=_gpu(np.array([0, 1, 2, 3, 4, 6]), torch.int32)))
    with pytest.raises(sa.SparseAttentionError):
        sa.sparse_attn_check_device()
    c.check(out, lse, skip=(5,))
    assert not out[5].any() and torch.isneginf(lse[5]).all()    # row 6 of 6
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("H, Hkv, D", [(8, 2, 64), (12, 1, 128), (2, 1, 32)])
def test_value_scales_of_all_sizes(sa, H, Hkv, D):
    """Scales from 2^-40 to 2^40 in rows cut over the GPU: the parts' weights have units of their
    own and are joined in a common one."""
    T = _long(D, "e4m3")
    c = Case([T - 1, 1111, T // 2], H, Hkv, D, 32, "e4m3", T, T)
    gen = torch.Generator("cuda")
    gen.manual_seed(2)
    codes, s = c.pool[1]
    size = torch.randint(-40, 41, s.shape, device="cuda", generator=gen)
    for lo, hi in ((-40, 41), (-40, -30), (30, 41)):
        c.pool[1] = (codes, s * torch.exp2(size.clamp(lo, hi).float()))
        c.check(*_in_shares(sa, lambda: c.run(sa)))
    # a span of pages far above the others, so that some parts see it and others do not
    big = torch.zeros(s.shape[0], dtype=torch.bool, device="cuda")
    big[torch.from_numpy(c.table[0, 100:110].astype(np.int64))] = True
    c.pool[1] = (codes, s * torch.where(big, 2.0 ** 60, 2.0 ** -60)[:, None, None])
    c.check(*_in_shares(sa, lambda: c.run(sa)))
    c.pool[1] = (codes, torch.where(s.isnan(), s, 0.0))
    out, lse = _in_shares(sa, lambda: c.run(sa))
    assert not out.any() and torch.isfinite(lse).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("dtype", list(TYPES))
def test_serving_loop(sa, dtype):
    """Prompts, then a few tokens at a time, one request finishing on the way, every earlier key:
    each step equals the dense computation over the whole sequences so far."""
    B, H, Hkv, D, page = 5, 4, 2, 64, 16
    T = _long(D, dtype)
    M = 60
    s = _server(sa, dtype, B=B, M=M, page=page, Hkv=Hkv, D=D)
    g = sa.sparse_attn_graph_build_structured(T, T, [])
    qt = torch.float32 if dtype == "fp32" else torch.bfloat16
    gen = torch.Generator("cuda")
    gen.manual_seed(3)
    history = [[np.zeros((Hkv, 0, D)) for _ in range(2)] for _ in range(B)]
    capacity = 800
    batch = sa.PagedBatch(B, capacity)
    for n_new in ([400, 37, 0, 1, 300], [1, 1, 16, 1, 1], [1, 1, 1, 1, -1], [100, 1, 1, 1, 333],
                  [5, 0, 1, 15, 1], [1, 1, 1, -1, 1]):
        new = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        sa.sparse_attn_paged_plan(s["length"], new, s["table"], s["stack"], s["count"], page, batch)
        qkv = torch.empty((capacity, H + 2 * Hkv, D), device="cuda").normal_(generator=gen).to(qt)
        k, v = qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        q = qkv[:, :H].contiguous().view(capacity, H, 1, D)
        sa.sparse_attn_paged_append(k, v, s["cache"], batch.slot)
        out, lse = _in_shares(sa, lambda: sa.sparse_attn_paged_decode(
            q, s["cache"], s["table"], batch.pos, g, 0.125, row=batch.row))
        sa.sparse_attn_check_device()
        assert not batch.status.any()
        total = sum(max(n, 0) for n in n_new)
        assert not out[total:].any() and torch.isneginf(lse[total:]).all()
        t = 0
        for b, n in enumerate(n_new):
            if n == -1:
                history[b] = [np.zeros((Hkv, 0, D)) for _ in range(2)]
                continue
            for i, x in enumerate((k, v)):
                rows = x[t:t + n].double().cpu().numpy()
                if dtype == "e4m3":
                    y, unit = paged_ref.quantise(rows)
                    rows = y * unit.astype(np.float64)[..., None]
                history[b][i] = np.concatenate([history[b][i], rows.transpose(1, 0, 2)], 1)
            for x in sorted({0, n // 2, n - 1} & set(range(n))):
                keys = np.arange(history[b][0].shape[1] - n + x + 1)
                for h in range(Hkv):
                    heads = slice(2 * h, 2 * h + 2)
                    o, l, size, vmax = paged_ref.attend(
                        q[t + x, heads, 0].double().cpu().numpy(), history[b][0][h][keys],
                        history[b][1][h][keys], 0.125)
                    t_lse, t_out, rel = paged_ref.tolerances(len(keys), D, size, vmax, qt)
                    got = out[t + x, heads, 0].double().cpu().numpy()
                    assert (np.abs(got - o) <= t_out + rel * np.abs(o)).all(), (n_new, b, x, h)
                    got = lse[t + x, heads].double().cpu().numpy()
                    assert (np.abs(got - l) <= t_lse + 2.0 ** -24 * np.abs(l)).all()
            t += n


@pytest.mark.parametrize("dtype", list(TYPES))
def test_captured_step_advances(sa, dtype):
    """plan, append and decode in one captured graph, replayed, give what separate calls give."""
    B, H, Hkv, D, page = 6, 4, 2, 64, 16
    g = sa.sparse_attn_graph_build_structured(_long(D, dtype), _long(D, dtype), [])
    qt = torch.float32 if dtype == "fp32" else torch.bfloat16
    gen = torch.Generator("cuda")
    gen.manual_seed(8)
    steps = [torch.empty((B, H + 2 * Hkv, D), device="cuda").normal_(generator=gen).to(qt)
             for _ in range(30)]
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    prompt = torch.tensor([900, 3, 0, 411, 64, 1], dtype=torch.int32, device="cuda")
    x = torch.empty((1400, 2 * Hkv, D), device="cuda").normal_(generator=gen).to(qt)

    def make():
        s = _server(sa, dtype, B=B, M=80, page=page, Hkv=Hkv, D=D)
        b = sa.PagedBatch(B, 1400)
        sa.sparse_attn_paged_plan(s["length"], prompt, s["table"], s["stack"], s["count"], page, b)
        sa.sparse_attn_paged_append(x[:, :Hkv], x[:, Hkv:], s["cache"], b.slot)
        s["batch"] = sa.PagedBatch(B, B)
        s["qkv"] = torch.zeros_like(steps[0])
        s["q"] = torch.zeros((B, H, 1, D), device="cuda", dtype=qt)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((B, H), device="cuda")
        n = sa.sparse_attn_paged_decode_workspace_size(s["q"], s["cache"], g)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
        return s

    def step(s):
        sa.sparse_attn_paged_plan(s["length"], ones, s["table"], s["stack"], s["count"], page,
                                  s["batch"])
        s["q"].copy_(s["qkv"][:, :H, None])
        sa.sparse_attn_paged_append(s["qkv"][:, H:H + Hkv], s["qkv"][:, H + Hkv:], s["cache"],
                                    s["batch"].slot)
        _in_shares(sa, lambda: sa.sparse_attn_paged_decode(
            s["q"], s["cache"], s["table"], s["batch"].pos, g, 0.125, row=s["batch"].row,
            out=s["out"], lse=s["lse"], workspace=s["ws"]))

    a, b = make(), make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    for x in steps:
        a["qkv"].copy_(x)
        b["qkv"].copy_(x)
        step(a)
        graph.replay()
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    assert torch.isfinite(a["lse"]).all() and a["out"].abs().max() < 10
    assert torch.equal(a["length"], b["length"]) and int(a["length"][0]) == 900 + len(steps)
    sa.sparse_attn_check_device()
