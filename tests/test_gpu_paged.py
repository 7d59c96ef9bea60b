"""Paged key-value cache on the GPU: the page plan of a step, the writing of
new rows and the attention of new tokens, each against its plain statement
(paged_ref, 64 bits), then together as a serving loop uses them."""
import math

import numpy as np
import pytest
import torch

import paged_ref
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sa():
    import sparse_graph_causal_b200 as m
    return m


def _gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


# ------------------------------------------------------------------- plan

def _plan_case(B, M, page, rng, kinds=(0.5, 0.3, 0.2), most=None):
    """Requests with distinct pages; n_new 0..most, or -1 with kinds[2]."""
    kind = rng.choice(3, B, p=kinds)
    length = rng.integers(0, M * page + 1, B)
    room = M * page - length
    n = np.where(kind == 0, np.minimum(1, room),
                 np.where(kind == 1, np.minimum(rng.integers(0, (most or M * page) + 1, B), room),
                          -1))
    used = -(-length // page)
    ids = rng.permutation(int(used.sum()) + B * M + 8).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    table[np.arange(M)[None] < used[:, None]] = ids[: used.sum()]
    stack = ids[used.sum():].copy()
    return length, n, table, stack


def _run_plan(sa, length, n, table, stack, count, page, capacity, in_place):
    dev = dict(length=_gpu(length, torch.int64), table=_gpu(table, torch.int32),
               stack=_gpu(stack, torch.int32),
               count=torch.tensor([count], dtype=torch.int64, device="cuda"))
    nn = _gpu(n, torch.int32)
    batch = sa.PagedBatch(len(length), capacity)
    for t in (batch.cu_new, batch.slot, batch.pos, batch.row, batch.status):
        t.fill_(-77)
    if in_place:
        out = dict(length_out=None, free_count_out=None)
    else:
        out = dict(length_out=torch.full_like(dev["length"], -77),
                   free_count_out=torch.full_like(dev["count"], -77))
    got = sa.sparse_attn_paged_plan(dev["length"], nn, dev["table"], dev["stack"], dev["count"],
                                    page, batch, **out)
    assert got is batch
    if not in_place:
        assert np.array_equal(dev["length"].cpu().numpy(), np.asarray(length))
        assert int(dev["count"]) == count
    new_len = dev["length"] if in_place else out["length_out"]
    new_count = dev["count"] if in_place else out["free_count_out"]
    assert np.array_equal(nn.cpu().numpy(), np.asarray(n))
    return dict(length=new_len, count=new_count, table=dev["table"], stack=dev["stack"],
                cu_new=batch.cu_new, slot=batch.slot, pos=batch.pos, row=batch.row,
                status=batch.status)


def _check_plan(got, want):
    for k, w in want.items():
        g = got[k].cpu().numpy()
        g = int(g[0]) if k == "count" else g
        assert np.array_equal(g, w), (k, g, w)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B, M, page, enough, capacity", [
    (1, 1, 1, 1.0, 1), (1, 5, 16, 1.0, 200), (3, 4, 7, 1.0, 100), (64, 12, 16, 0.5, 5000),
    (300, 6, 17, 0.8, 20000), (1024, 3, 8, 0.9, 9000), (1025, 3, 8, 0.9, 9001),
    (2500, 2, 32, 0.6, 60000), (8192, 2, 4, 1.0, 33333), (40, 5, 24, 0.0, 2048),
    (40, 5, 24, 1.0, 37), (900, 4, 16, 0.7, 50001), (2000, 3, 16, 0.7, 70000),
])
def test_plan(sa, B, M, page, enough, capacity, in_place):
    rng = np.random.default_rng(B * 1000 + M + page)
    length, n, table, stack = _plan_case(B, M, page, rng)
    need = int((-(-(length + np.maximum(n, 0)) // page) - -(-length // page)).sum())
    back = int((-(-length // page))[n == -1].sum())
    count = min(max(0, int(need * enough) - back), len(stack) - back)
    stack[count:] = -5
    want = paged_ref.plan(length, n, table, stack, count, page, capacity)
    _check_plan(_run_plan(sa, length, n, table, stack, count, page, capacity, in_place), want)


@pytest.mark.parametrize("change", ["len_negative", "len_long", "n_odd", "n_long", "count_negative",
                                    "count_long", "stack_full", "holes"])
def test_plan_refuses_requests(sa, change):
    """What the device alone can see: the request is refused, nothing outside the arrays is
    touched, the others are served."""
    rng = np.random.default_rng(5)
    B, M, page = 50, 6, 16
    length, n, table, stack = _plan_case(B, M, page, rng, most=40)
    count = len(stack) // 2
    big = np.iinfo(np.int32).max
    if change == "len_negative":
        length[[3, 9, 20]] = [-1, -(1 << 40), -7]
    elif change == "len_long":
        length[[3, 9, 20]] = [M * page + 1, 1 << 62, 1 << 31]
    elif change == "n_odd":
        n[[3, 9, 20]] = [-2, -big - 1, -100]
    elif change == "n_long":
        n[[3, 9]] = [M * page + 1, big]
    elif change == "count_negative":
        count = -1
    elif change == "count_long":
        count = len(stack) + 1
    elif change == "stack_full":
        n[10:30] = -1
        count = len(stack) - int((-(-length // page))[10:15].sum())
    elif change == "holes":
        table[5:20, 0] = -1
    guard = np.concatenate([stack, np.full(64, -9, np.int32)])
    want = paged_ref.plan(length, n, table, stack, count, page, 4096)
    dev = _gpu(guard, torch.int32)
    got = None
    batch = sa.PagedBatch(B, 4096)
    dl, dt = _gpu(length, torch.int64), _gpu(table, torch.int32)
    dc = torch.tensor([count], dtype=torch.int64, device="cuda")
    sa.sparse_attn_paged_plan(dl, _gpu(n, torch.int32), dt, dev[:len(stack)], dc, page, batch)
    got = dict(length=dl, count=dc, table=dt, stack=dev[:len(stack)], cu_new=batch.cu_new,
               slot=batch.slot, pos=batch.pos, row=batch.row, status=batch.status)
    _check_plan(got, want)
    assert (dev[len(stack):] == -9).all()


# ----------------------------------------------------------------- append

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _pages(shape, dtype, seed):
    """Pages with recognisable contents (any bytes) and their scales."""
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    n = math.prod(shape) * torch.empty((), dtype=TYPES[dtype]).element_size()
    x = torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=gen)
    x = x.view(TYPES[dtype]).view(shape)
    if dtype != "e4m3":
        return x, None
    return x, torch.empty(shape[:3], device="cuda").normal_(generator=gen)


@pytest.mark.parametrize("wide", [False, True], ids=["plain", "slices"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N, Hkv, D, page", [
    (1, 1, 32, 1), (1, 2, 64, 16), (7, 3, 128, 17), (64, 2, 64, 16), (333, 5, 32, 24),
    (1000, 8, 128, 32), (4099, 1, 64, 100),
])
def test_append(sa, N, Hkv, D, page, dtype, wide):
    gen = torch.Generator("cuda")
    gen.manual_seed(N + D)
    rng = np.random.default_rng(N)
    src = torch.float32 if dtype == "fp32" else torch.bfloat16
    if wide:
        x = torch.empty((N, 4 * Hkv, D), device="cuda", dtype=src).normal_(generator=gen)
        k, v = x[:, Hkv:2 * Hkv], x[:, 3 * Hkv:]
    else:
        k, v = (torch.empty((N, Hkv, 1, D), device="cuda", dtype=src).normal_(generator=gen)
                for _ in range(2))
    # magnitudes over the whole range, and rows that have no scale
    size = torch.exp2(torch.randint(-130, 120, (N, Hkv), device="cuda", generator=gen).float())
    for t in (k, v):
        t.mul_(size.to(src).view(N, Hkv, *([1] * (t.dim() - 2))))
    if N > 6:
        k[1, 0], k[2, 0, ..., 3], v[3, 0, ..., 5] = 0.0, math.inf, math.nan
        v[4, 0, ..., 0] = -math.inf
        k[5, 0, ..., ::2] = -0.0
    n_pages = -(-N // page) + 3
    slot = rng.permutation(n_pages * page)[:N].astype(np.int64)
    if N > 2:
        slot[rng.random(N) < 0.1] = -1
        slot[2] = -(1 << 40)
    (kp, ks), (vp, vs) = (_pages((n_pages, Hkv, page, D), dtype, s) for s in (1, 2))
    cache = sa.PagedCache(kp, vp, ks, vs)
    want = []
    for pool, scale, new in ((kp, ks, k), (vp, vs, v)):
        pool, new = pool.clone(), new.reshape(N, Hkv, D)
        keep = slot >= 0
        pg, at = torch.from_numpy(slot[keep] // page), torch.from_numpy(slot[keep] % page)
        rows = new[torch.from_numpy(keep)]
        if dtype == "e4m3":
            scale = scale.clone()
            y, s = paged_ref.quantise(rows.float().cpu().numpy())
            pool.view(torch.uint8)[pg, :, at] = torch.from_numpy(y).to(
                torch.float8_e4m3fn).view(torch.uint8).cuda()
            scale[pg, :, at] = torch.from_numpy(s).cuda()
        else:
            pool[pg, :, at] = rows
        want.append((pool, scale))
    sa.sparse_attn_paged_append(k, v, cache, _gpu(slot, torch.int64))
    sa.sparse_attn_check_device()
    for (pool, scale), p, s in zip(want, (kp, vp), (ks, vs)):
        g, w = _bytes(p), _bytes(pool)
        if dtype == "e4m3":  # the sign of a zero code is free
            g, w = np.where(g == 128, 0, g), np.where(w == 128, 0, w)
            a, b = s.cpu().numpy(), scale.cpu().numpy()
            assert np.array_equal(a, b, equal_nan=True)
        assert np.array_equal(g, w)


def test_append_rounds_like_division(sa):
    """Codes are the 8-bit roundings of correctly rounded 32-bit quotients: rows whose quotients
    fall on the midpoints between codes, next to them, and everywhere else."""
    N, Hkv, D, page = 8192, 2, 128, 64
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, N, Hkv, D)).astype(np.float32)
    x *= np.exp2(rng.integers(-20, 20, (2, N, Hkv, 1))).astype(np.float32)
    codes = paged_ref.E4M3
    mids = np.concatenate([(codes[1:] + codes[:-1]) / 2, codes]).astype(np.float32)
    half = x[:, : N // 2]
    top = np.abs(half).max(-1, keepdims=True)
    top = np.where(rng.random(top.shape) < 0.5, np.exp2(np.round(np.log2(top))) * 448, top)
    half[:] = rng.choice(mids, half.shape) * rng.choice([-1, 1], half.shape) * top / 448
    half[..., 0] = top[..., 0]
    x = torch.from_numpy(x).bfloat16()
    k, v = x.cuda()
    shape = (N // page, Hkv, page, D)
    kv = [torch.zeros(shape, device="cuda").to(TYPES["e4m3"]) for _ in range(2)]
    scales = [torch.zeros(shape[:3], device="cuda") for _ in range(2)]
    sa.sparse_attn_paged_append(k, v, sa.PagedCache(*kv, *scales),
                                torch.arange(N, device="cuda"))
    for new, pool, scale in zip(x, kv, scales):
        y, s = paged_ref.quantise(new.float().numpy())
        got = pool.transpose(1, 2).reshape(N, Hkv, D).float().cpu().numpy()
        assert np.array_equal(scale.transpose(1, 2).reshape(N, Hkv).cpu().numpy(), s)
        assert np.array_equal(got, y)


def test_append_flags_slots_outside_the_cache(sa):
    n_pages, Hkv, page, D = 4, 2, 16, 64
    kp, vp = (torch.zeros((n_pages, Hkv, page, D), device="cuda", dtype=torch.bfloat16)
              for _ in range(2))
    k, v = (torch.ones((3, Hkv, D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    slot = torch.tensor([n_pages * page, 5, (1 << 62) + 3], device="cuda")
    sa.sparse_attn_paged_append(k, v, sa.PagedCache(kp, vp), slot)
    with pytest.raises(sa.SparseAttentionError):
        sa.sparse_attn_check_device()
    want = torch.zeros_like(kp)
    want[0, :, 5] = 1
    assert torch.equal(kp, want) and torch.equal(vp, want)
    sa.sparse_attn_check_device()


def test_append_of_nothing(sa):
    kp, vp = (torch.zeros((2, 1, 8, 32), device="cuda") for _ in range(2))
    x = torch.zeros((0, 1, 32), device="cuda")
    sa.sparse_attn_paged_append(x, x, sa.PagedCache(kp, vp),
                                torch.zeros(0, dtype=torch.int64, device="cuda"))


# ----------------------------------------------------------------- decode

def _keys(p, T, W, links, csr):
    if csr is not None:
        rp, ci = csr
        return ci[rp[p]:rp[p + 1]].astype(np.int64)
    far = [p - (1 << x) for x in links if W <= 1 << x <= p]
    return np.array(sorted(far) + list(range(max(0, p - W + 1), p + 1)), np.int64)


class Case:
    """A paged cache whose rows outside the keys of its tokens hold NaN."""

    def __init__(self, pos, H, Hkv, D, page, dtype, T, W=0, links=(), csr=None, row=None, seed=1,
                 q_size=1.0, slack=0):
        rng = np.random.default_rng(seed)
        self.pos, self.N, self.H, self.Hkv, self.D = np.asarray(pos, np.int64), len(pos), H, Hkv, D
        self.page, self.dtype, self.T, self.W, self.links, self.csr = page, dtype, T, W, links, csr
        self.row = np.arange(self.N) if row is None else np.asarray(row)
        self.scale = 1.0 / math.sqrt(D)
        rows = int(self.row.max()) + 1 + slack
        M = -(-T // page) + slack
        self.keys = [_keys(p, T, W, links, csr) if p >= 0 else np.zeros(0, np.int64)
                     for p in self.pos]
        self.table = np.full((rows, M), -1, np.int32)
        used = [set() for _ in range(rows)]
        for r, ks in zip(self.row, self.keys):
            used[r].update((ks // page).tolist())
        n_pages = sum(len(u) for u in used) + 3
        ids = rng.permutation(n_pages)
        at = 0
        for r, u in enumerate(used):
            for p in sorted(u):
                self.table[r, p] = ids[at]
                at += 1
        live = np.zeros((n_pages, page), bool)
        for r, ks in zip(self.row, self.keys):
            live[self.table[r, ks // page], ks % page] = True
        gen = torch.Generator("cuda")
        gen.manual_seed(seed)
        live = torch.from_numpy(live).cuda()[:, None, :, None]
        self.pool = []
        for _ in range(2):
            x = torch.empty((n_pages, Hkv, page, D), device="cuda").normal_(generator=gen)
            if dtype == "e4m3":
                s = torch.exp2(torch.empty(x.shape[:3], device="cuda").uniform_(
                    -14, -6, generator=gen))
                c = (x * 64).clamp(-448, 448).to(TYPES[dtype]).view(torch.uint8)
                c = torch.where(live, c, torch.full_like(c, 0x7f)).view(TYPES[dtype])
                self.pool.append((c, torch.where(live[..., 0], s, torch.nan)))
            else:
                self.pool.append((torch.where(live, x, torch.nan).to(TYPES[dtype]), None))
        qt = torch.float32 if dtype == "fp32" else torch.bfloat16
        self.q = (torch.empty((self.N, H, 1, D), device="cuda").normal_(generator=gen)
                  * q_size).to(qt)

    def graph(self, sa):
        if self.csr is not None:
            return sa.sparse_attn_graph_build_csr(_gpu(self.csr[0], torch.int64),
                                                  _gpu(self.csr[1], torch.int32), 0)
        return sa.sparse_attn_graph_build_structured(self.T, self.W, list(self.links))

    def cache(self, sa):
        (k, ks), (v, vs) = self.pool
        return sa.PagedCache(k, v, ks, vs)

    def run(self, sa, **kw):
        row = None if np.array_equal(self.row, np.arange(self.N)) else _gpu(self.row, torch.int32)
        out, lse = sa.sparse_attn_paged_decode(
            self.q, self.cache(sa), _gpu(self.table, torch.int32), _gpu(self.pos, torch.int64),
            self.graph(sa), self.scale, row=row, **kw)
        return out, lse

    def values(self, n, h):
        """Rows of cache head h at the keys of token n, in 64 bits (numpy)."""
        ks = self.keys[n]
        pg = self.table[self.row[n], ks // self.page]
        got = []
        for x, s in self.pool:
            y = x.view(torch.uint8)[pg, h, ks % self.page].view(x.dtype) if s is not None else \
                x[pg, h, ks % self.page]
            y = y.double()
            if s is not None:
                y = y * s[pg, h, ks % self.page].double()[:, None]
            got.append(y.cpu().numpy())
        return got

    def check(self, out, lse, skip=()):
        G = self.H // self.Hkv
        assert out.dtype == self.q.dtype and out.shape == self.q.shape
        out, lse = out.double().cpu().numpy()[:, :, 0], lse.double().cpu().numpy()
        q = self.q.double().cpu().numpy()[:, :, 0]
        for n in range(self.N):
            if n in skip:
                continue
            for h in range(self.Hkv):
                k, v = self.values(n, h)
                g = slice(h * G, h * G + G)
                o, l, size, vmax = paged_ref.attend(q[n, g], k, v, self.scale)
                if len(k) == 0:
                    assert not out[n, g].any() and np.isneginf(lse[n, g]).all(), (n, h)
                    continue
                t_lse, t_out, t_rel = paged_ref.tolerances(len(k), self.D, size, vmax,
                                                           self.q.dtype)
                t_lse += 2.0 ** -24 * np.abs(l).max()
                assert np.abs(lse[n, g] - l).max() <= t_lse, (n, h, np.abs(lse[n, g] - l).max())
                bad = np.abs(out[n, g] - o) - (t_out + t_rel * np.abs(o))
                assert bad.max() <= 0, (n, h, bad.max(), t_out)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("H, Hkv", [(1, 1), (2, 2), (6, 3), (8, 2), (8, 1), (9, 1), (16, 1),
                                    (34, 2)])
def test_decode_heads(sa, H, Hkv, D, dtype):
    """Short and ragged rows of a window with links; every group size."""
    c = Case([0, 1, 15, 16, 46, 700, 999, -1, 63], H, Hkv, D, 16, dtype, 1000, 32, range(11))
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("page", [1, 7, 8, 17, 64, 100, 4096])
def test_decode_pages(sa, page, dtype):
    c = Case([3000, 77, 0, 1500, 2047], 4, 2, 64, page, dtype, 3001, 1500, range(12), seed=page)
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pos, H, Hkv, D, T", [
    ([20000], 4, 1, 128, 20001),                               # one row over the whole GPU
    ([9999, 0, 31, -1, 12345, 1, 4095, 4096], 8, 2, 64, 16384),  # ragged
    ([5000] * 9, 3, 3, 32, 5001),
    ([511, 512, 513, 8191, 8192] * 8, 2, 1, 128, 8193),
])
def test_decode_full_causal(sa, pos, H, Hkv, D, T, dtype):
    """Every earlier key: rows are cut over the GPU and joined."""
    c = Case(pos, H, Hkv, D, 32, dtype, T, T)
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("H, Hkv, D, pos", [
    (8, 2, 128, [60000, 12, 45001, 59999]), (32, 2, 64, [52345, -1, 60000]),
    (12, 1, 32, [60000, 59000, 0, 33333, 60000, 45000]), (4, 4, 64, [59999, 3, 40000]),
])
def test_decode_rows_over_many_ctas(sa, H, Hkv, D, pos, dtype):
    c = Case(pos, H, Hkv, D, 64, dtype, 60001, 60001)
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("seed", range(8))
def test_decode_batches_of_any_shape(sa, seed, dtype):
    """Rows of all lengths in one batch, windows that cut some of them, heads of all groups: the
    shares' borders fall anywhere."""
    rng = np.random.default_rng(100 + seed)
    N = int(np.exp(rng.uniform(0, np.log(60))))
    T = int(rng.integers(3000, 30000))
    pos = np.exp(rng.uniform(0, np.log(T), N)).astype(np.int64) - 1
    pos[rng.integers(N)] = T - 1
    D, Hkv = int(rng.choice([32, 64, 128])), int(rng.choice([1, 2, 3]))
    G, page = int(rng.choice([1, 2, 5, 8, 12, 20])), int(rng.integers(5, 80))
    W = T if seed % 2 else int(rng.integers(2000, T))
    c = Case(pos, Hkv * G, Hkv, D, page, dtype, T, W, range(15), seed=seed)
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_decode_window_rows_fill_the_gpu(sa, dtype):
    """120 windows of equal length: one row for each SM."""
    rng = np.random.default_rng(9)
    c = Case(rng.integers(2500, 9000, 60), 4, 2, 64, 16, dtype, 9000, 2100)
    c.check(*c.run(sa), skip=set(range(60)) - set(range(0, 60, 7)))


@pytest.mark.parametrize("dtype", list(TYPES))
def test_decode_many_tokens(sa, dtype):
    rng = np.random.default_rng(2)
    pos = rng.integers(-1, 600, 700)
    c = Case(pos, 4, 2, 32, 16, dtype, 600, 600)
    c.check(*c.run(sa), skip=set(range(700)) - set(range(0, 700, 9)))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("H, Hkv, D", [(2, 2, 64), (8, 2, 128), (4, 4, 32)])
def test_decode_csr(sa, H, Hkv, D, dtype):
    T = 1500
    rp, ci = synth.csr_random_rows(T, seed=21)
    rows = [np.unique(ci[rp[i]:rp[i + 1]]) for i in range(T)]
    rows[70] = rows[70][:0]                   # a token that attends to nothing
    rows[71] = np.array([3])
    rows[1400] = np.arange(1401)              # and one to every key
    rp = np.concatenate([[0], np.cumsum([len(r) for r in rows])]).astype(np.int64)
    ci = np.concatenate(rows).astype(np.int32)
    c = Case([0, 70, 71, 1499, 1400, 800], H, Hkv, D, 24, dtype, T, csr=(rp, ci))
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [40, 5000])
def test_decode_several_tokens_of_a_request(sa, W, dtype):
    """Tokens name their block-table rows; rows may be longer than the graph."""
    c = Case([100, 101, 102, 4000, 4001, -1], 4, 2, 64, 16, dtype, 5000, W, range(13),
             row=[2, 2, 2, 0, 0, 1], slack=3)
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W, q_size", [(64, 40.0), (3000, 40.0), (3000, 1e-3)])
def test_decode_sharp_and_flat_scores(sa, W, q_size, dtype):
    c = Case([2999, 1234, 50], 8, 2, 64, 16, dtype, 3000, W, range(12), q_size=q_size)
    c.check(*c.run(sa))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [64, 3000])
def test_decode_flags_bad_positions_rows_and_pages(sa, W, dtype):
    c = Case([2999, 1234, 50, 2500, 2000, 999], 4, 2, 64, 16, dtype, 3000, W,
             row=[0, 1, 2, 3, 4, 5])
    tab = c.table.copy()
    n_pages = c.pool[0][0].shape[0]
    c.pos[1], c.pos[2] = 3000, -2
    c.keys[1] = c.keys[2] = np.zeros(0, np.int64)
    c.table[3, 2500 // 16] = -1                # its last page
    c.table[4, 1990 // 16] = n_pages
    for n, p in ((3, 2500 // 16), (4, 1990 // 16)):
        c.keys[n] = c.keys[n][c.keys[n] // 16 != p]
    row = np.array([0, 1, 2, 3, 4, 6])
    out, lse = sa.sparse_attn_paged_decode(
        c.q, c.cache(sa), _gpu(c.table, torch.int32), _gpu(c.pos, torch.int64), c.graph(sa),
        c.scale, row=_gpu(row, torch.int32))
    with pytest.raises(sa.SparseAttentionError):
        sa.sparse_attn_check_device()
    c.check(out, lse, skip=(5,))
    assert not out[5].any() and torch.isneginf(lse[5]).all()    # row 6 of 6
    # the flag is down again, and sound tokens alone raise none
    c.table = tab
    c.pos[1] = c.pos[2] = c.pos[5] = -1
    c.keys[3] = _keys(2500, 3000, W, (), None)
    c.keys[4] = _keys(2000, 3000, W, (), None)
    c.keys[5] = c.keys[5][:0]
    c.check(*c.run(sa))
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [64, 3000])
def test_decode_infinities(sa, W, dtype):
    """An infinite value reaches the output of its column alone, a NaN one too; an infinite
    score of -inf has no weight; a row of such scores is empty."""
    c = Case([2999, 2000, 1000], 2, 1, 64, 16, dtype, 3000, W)
    (k, _), (v, _) = c.pool
    clean, clean_lse = c.run(sa)

    def at(n, j):
        return int(c.table[n, j // 16]), 0, j % 16

    v[at(0, 2990) + (3,)] = math.inf
    v[at(0, 2991) + (4,)] = -math.inf
    v[at(0, 2992) + (5,)] = math.nan
    out, lse = c.run(sa)
    assert torch.equal(lse, clean_lse)
    assert (out[0, :, 0, 3] == math.inf).all() and (out[0, :, 0, 4] == -math.inf).all()
    assert out[0, :, 0, 5].isnan().all()
    same = torch.ones(64, dtype=torch.bool)
    same[3:6] = False
    assert torch.equal(out[0][..., same], clean[0][..., same])
    assert torch.equal(out[1:], clean[1:])
    # scores of -inf: query 1 for one key, query 2 for all of its keys
    c.q[1:, :, 0, 7] = 1.0
    k[at(1, 1999) + (7,)] = -math.inf
    for j in c.keys[2]:
        k[at(2, int(j)) + (7,)] = -math.inf
    out, lse = c.run(sa)
    c.keys[1] = c.keys[1][c.keys[1] != 1999]
    c.check(out, lse, skip=(0, 2))
    assert not out[2].any() and torch.isneginf(lse[2]).all()
    # a NaN key makes its row NaN, no other
    k[at(1, 1998) + (0,)] = math.nan
    out, lse = c.run(sa)
    assert out[1].isnan().all() and lse[1].isnan().all()
    assert not out[2].any() and torch.isneginf(lse[2]).all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_decode_repeats_bit_for_bit(sa, dtype):
    c = Case([9999, 5000, 77], 8, 2, 64, 16, dtype, 10000, 10000)
    g, cache = c.graph(sa), c.cache(sa)
    need = sa.sparse_attn_paged_decode_workspace_size(c.q, cache, g)
    runs = []
    for fill in (0, 255):
        ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda")
        runs.append(sa.sparse_attn_paged_decode(
            c.q, cache, _gpu(c.table, torch.int32), _gpu(c.pos, torch.int64), g, c.scale,
            workspace=ws))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])


def test_decode_of_nothing(sa):
    c = Case([5], 2, 1, 64, 16, "bf16", 100, 100)
    out, lse = sa.sparse_attn_paged_decode(
        c.q[:0], c.cache(sa), _gpu(c.table, torch.int32), _gpu(c.pos[:0], torch.int64),
        c.graph(sa), c.scale)
    assert out.shape == (0, 2, 1, 64) and lse.shape == (0, 2)


# --------------------------------------------------------------- together

def _server(sa, dtype, B=5, M=40, page=16, Hkv=2, D=64, T=640):
    n_pages = B * M
    shape = (n_pages, Hkv, page, D)
    scales = [torch.full(shape[:3], math.nan, device="cuda") for _ in range(2)] \
        if dtype == "e4m3" else [None, None]
    kv = [torch.full(shape, math.nan, device="cuda").to(TYPES[dtype]) for _ in range(2)]
    return dict(cache=sa.PagedCache(*kv, *scales), page=page,
                length=torch.zeros(B, dtype=torch.int64, device="cuda"),
                table=torch.full((B, M), -1, dtype=torch.int32, device="cuda"),
                stack=torch.arange(n_pages, dtype=torch.int32, device="cuda").flip(0).contiguous(),
                count=torch.tensor([n_pages], device="cuda"))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [32, 640])
def test_serving_loop(sa, W, dtype):
    """Prompts, then token by token, one request finishing on the way: every step's attention
    equals the dense computation over the whole sequences so far."""
    B, H, Hkv, D, T, page = 5, 4, 2, 64, 640, 16
    s = _server(sa, dtype)
    g = sa.sparse_attn_graph_build_structured(T, W, list(range(10)))
    qt = torch.float32 if dtype == "fp32" else torch.bfloat16
    gen = torch.Generator("cuda")
    gen.manual_seed(3)
    history = [[np.zeros((Hkv, 0, D)) for _ in range(2)] for _ in range(B)]
    steps = [[100, 37, 0, 1, 300], [1, 1, 16, 1, 1], [1, 1, 1, 1, -1], [1, 1, 1, 1, 33],
             [5, 0, 1, 15, 1], [1, 1, 1, -1, 1]]
    capacity = 512
    batch = sa.PagedBatch(B, capacity)
    for n_new in steps:
        new = torch.tensor(n_new, dtype=torch.int32, device="cuda")
        sa.sparse_attn_paged_plan(s["length"], new, s["table"], s["stack"], s["count"], page, batch)
        qkv = torch.empty((capacity, H + 2 * Hkv, D), device="cuda").normal_(generator=gen).to(qt)
        k, v = qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        q = qkv[:, :H].contiguous().view(capacity, H, 1, D)
        sa.sparse_attn_paged_append(k, v, s["cache"], batch.slot)
        out, lse = sa.sparse_attn_paged_decode(q, s["cache"], s["table"], batch.pos, g, 0.125,
                                               row=batch.row)
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
                p = history[b][0].shape[1] - n + x
                keys = _keys(p, T, W, range(10), None)
                for h in range(Hkv):
                    qd = q[t + x, 2 * h:2 * h + 2, 0].double().cpu().numpy()
                    o, l, size, vmax = paged_ref.attend(qd, history[b][0][h][keys],
                                                        history[b][1][h][keys], 0.125)
                    t_lse, t_out, rel = paged_ref.tolerances(len(keys), D, size, vmax, qt)
                    got = out[t + x, 2 * h:2 * h + 2, 0].double().cpu().numpy()
                    assert (np.abs(got - o) <= t_out + rel * np.abs(o)).all(), (n_new, b, x, h)
                    got = lse[t + x, 2 * h:2 * h + 2].double().cpu().numpy()
                    assert (np.abs(got - l) <= t_lse + 2.0 ** -24 * np.abs(l)).all()
            t += n
    assert int(s["count"]) == B * 40 - sum(-(-int(x) // page) for x in s["length"])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [32, 640])
def test_captured_step_advances(sa, W, dtype):
    """plan, append and decode in one captured graph, replayed: the lengths advance in place, and
    each replay gives what separate calls give."""
    B, H, Hkv, D, T, page = 5, 4, 2, 64, 640, 16
    g = sa.sparse_attn_graph_build_structured(T, W, list(range(10)))
    qt = torch.float32 if dtype == "fp32" else torch.bfloat16
    gen = torch.Generator("cuda")
    gen.manual_seed(8)
    steps = [torch.empty((B, H + 2 * Hkv, D), device="cuda").normal_(generator=gen).to(qt)
             for _ in range(40)]
    ones = torch.ones(B, dtype=torch.int32, device="cuda")

    def make():
        s = _server(sa, dtype)
        s["batch"] = sa.PagedBatch(B, B)
        s["qkv"] = torch.zeros_like(steps[0])
        s["q"] = torch.zeros((B, H, 1, D), device="cuda", dtype=qt)
        s["out"], s["lse"] = torch.zeros_like(s["q"]), torch.zeros((B, H), device="cuda")
        n = sa.sparse_attn_paged_decode_workspace_size(s["q"], s["cache"], g)
        s["ws"] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        return s

    def step(s):
        sa.sparse_attn_paged_plan(s["length"], ones, s["table"], s["stack"], s["count"], page,
                                  s["batch"])
        s["q"].copy_(s["qkv"][:, :H, None])
        sa.sparse_attn_paged_append(s["qkv"][:, H:H + Hkv], s["qkv"][:, H + Hkv:], s["cache"],
                                    s["batch"].slot)
        sa.sparse_attn_paged_decode(s["q"], s["cache"], s["table"], s["batch"].pos, g, 0.125,
                                    row=s["batch"].row, out=s["out"], lse=s["lse"],
                                    workspace=s["ws"])

    a, b = make(), make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(b)
    assert int(b["length"].sum()) == 0      # a capture runs nothing
    for x in steps:
        a["qkv"].copy_(x)
        b["qkv"].copy_(x)
        step(a)
        graph.replay()
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    assert torch.equal(a["length"], b["length"]) and int(a["length"][0]) == len(steps)
    assert torch.equal(a["table"], b["table"]) and torch.equal(a["count"], b["count"])
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [32, 6000])
def test_calls_in_a_row_wait_for_one_another(sa, W, dtype):
    """Each call is launched while the one before it runs.  Every step reads what the step before
    wrote (lengths, pages, cache rows, and its outputs as the next keys, values and queries): the
    same bits as with a synchronisation after every call, on the current stream and on a given one."""
    B, H, Hkv, D, page, M, steps = 4, 4, 2, 64, 16, 400, 60
    g = sa.sparse_attn_graph_build_structured(M * page, W, list(range(13)))
    qt = torch.float32 if dtype == "fp32" else torch.bfloat16
    ones = torch.ones(B, dtype=torch.int32, device="cuda")

    def run(after, stream):
        s = _server(sa, dtype, B=B, M=M, page=page)
        gen = torch.Generator("cuda")
        gen.manual_seed(4)
        lens = torch.tensor([3000, 17, 5900, 1], dtype=torch.int32, device="cuda")
        first, batch = sa.PagedBatch(B, 9000), sa.PagedBatch(B, B)
        x = torch.empty((9000, 2 * Hkv, D), device="cuda").normal_(generator=gen).to(qt)
        q = torch.empty((B, H, 1, D), device="cuda").normal_(generator=gen).to(qt)
        torch.cuda.synchronize()
        n = sa.sparse_attn_paged_decode_workspace_size(q, s["cache"], g)
        ws = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        outs = []
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            given = dict(stream=stream) if stream else {}
            sa.sparse_attn_paged_plan(s["length"], lens, s["table"], s["stack"], s["count"], page,
                                      first, **given)
            after()
            sa.sparse_attn_paged_append(x[:, :Hkv], x[:, Hkv:], s["cache"], first.slot, **given)
            after()
            for _ in range(steps):
                sa.sparse_attn_paged_plan(s["length"], ones, s["table"], s["stack"], s["count"],
                                          page, batch, **given)
                after()
                rows = q[:, :, 0]
                sa.sparse_attn_paged_append(rows[:, :Hkv], rows[:, Hkv:], s["cache"], batch.slot,
                                            **given)
                after()
                out, lse = sa.sparse_attn_paged_decode(q, s["cache"], s["table"], batch.pos, g, 0.2,
                                                       row=batch.row, workspace=ws, **given)
                after()
                outs.append((out, lse))
                q = torch.roll(out, 1, 3) + q
        torch.cuda.synchronize()
        return outs

    want = run(torch.cuda.synchronize, None)
    for stream in (None, torch.cuda.Stream()):
        for (o, l), (o2, l2) in zip(want, run(lambda: None, stream)):
            assert torch.equal(o, o2) and torch.equal(l, l2)
    assert torch.isfinite(want[-1][1]).all()
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_captured_decode_of_long_rows(sa, dtype):
    """Rows cut over the GPU in a captured graph: replays follow the positions in place."""
    c = Case([20000, 15000, 77], 8, 2, 64, 16, dtype, 20001, 20001)
    g, cache, table = c.graph(sa), c.cache(sa), _gpu(c.table, torch.int32)
    need = sa.sparse_attn_paged_decode_workspace_size(c.q, cache, g)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    pos = _gpu(c.pos, torch.int64)
    out, lse = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.sparse_attn_paged_decode(c.q, cache, table, pos, g, c.scale, out=out, lse=lse,
                                    workspace=ws)
    for p in ([20000, 15000, 77], [5, 15000, -1], [19999, 0, 76]):
        pos.copy_(torch.tensor(p))
        graph.replay()
        o, l = sa.sparse_attn_paged_decode(c.q, cache, table, pos, g, c.scale)
        assert torch.equal(out, o) and torch.equal(lse, l)
    c.pos = np.array(p)
    c.keys = [_keys(x, 20001, 20001, (), None) for x in p]
    c.check(out, lse)
    sa.sparse_attn_check_device()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_cache_of_more_than_32_bits(sa, dtype):
    """Rows whose offsets, in elements, are above 2^32: written by append, read by decode."""
    Hkv, page, D = 8, 64, 128
    n_pages = (1 << 32) // (Hkv * page * D) + 70
    if torch.cuda.mem_get_info()[0] < 3 * n_pages * Hkv * page * D * (4 if dtype == "fp32" else 2):
        pytest.skip("not enough device memory")
    kv = [torch.empty((n_pages, Hkv, page, D), device="cuda", dtype=TYPES[dtype])
          for _ in range(2)]
    scales = [torch.empty((n_pages, Hkv, page), device="cuda") if dtype == "e4m3" else None
              for _ in range(2)]
    cache = sa.PagedCache(*kv, *scales)
    T, qt = 4000, torch.float32 if dtype == "fp32" else torch.bfloat16
    M = -(-T // page)
    table = torch.arange(n_pages - M, n_pages, dtype=torch.int32, device="cuda").flip(0)[None]
    table = table.contiguous()
    gen = torch.Generator("cuda")
    gen.manual_seed(6)
    k, v = (torch.empty((T, Hkv, D), device="cuda").normal_(generator=gen).to(qt)
            for _ in range(2))
    at = torch.arange(T, device="cuda")
    slot = table[0].long()[at // page] * page + at % page
    assert int(slot.min()) * D * Hkv > 1 << 32
    sa.sparse_attn_paged_append(k, v, cache, slot)
    q = torch.empty((1, 8, 1, D), device="cuda").normal_(generator=gen).to(qt)
    pos = torch.tensor([T - 1], device="cuda")
    for W in (200, T):
        g = sa.sparse_attn_graph_build_structured(T, W, [])
        out, lse = sa.sparse_attn_paged_decode(q, cache, table, pos, g, 0.125)
        sa.sparse_attn_check_device()
        for h in range(Hkv):
            rows = []
            for x in (k, v):
                x = x[T - W:, h].double().cpu().numpy()
                if dtype == "e4m3":
                    y, unit = paged_ref.quantise(x)
                    x = y * unit.astype(np.float64)[..., None]
                rows.append(x)
            qd = q[0, h:h + 1, 0].double().cpu().numpy()
            o, l, size, vmax = paged_ref.attend(qd, *rows, 0.125)
            t_lse, t_out, rel = paged_ref.tolerances(W, D, size, vmax, qt)
            assert (np.abs(out[0, h].double().cpu().numpy() - o) <= t_out + rel * np.abs(o)).all()
            assert abs(float(lse[0, h]) - l[0]) <= t_lse + 2.0 ** -24 * abs(l[0])


@pytest.mark.parametrize("W", [32, 3000])
def test_decode_scales_of_all_sizes(sa, W):
    """Value scales from 2^-40 to 2^40 in one row: the weights keep their own range."""
    c = Case([2999, 1111], 8, 2, 64, 16, "e4m3", 3000, W, range(12))
    gen = torch.Generator("cuda")
    gen.manual_seed(2)
    codes, s = c.pool[1]
    size = torch.randint(-40, 41, s.shape, device="cuda", generator=gen)
    for lo, hi in ((-40, 41), (-40, -30), (30, 41)):
        c.pool[1] = (codes, s * torch.exp2(size.clamp(lo, hi).float()))
        c.check(*c.run(sa))
    # rows of zeros have scale 0; a row of NaN scale reaches the tokens that see it
    c.pool[1] = (codes, torch.where(s.isnan(), s, 0.0))
    out, lse = c.run(sa)
    assert not out.any() and torch.isfinite(lse).all()


def test_decode_flags_positions_past_the_table(sa):
    c = Case([400, 99], 2, 1, 64, 16, "bf16", 1000, 32)
    table = _gpu(c.table[:, :25], torch.int32)          # 25 pages: positions below 400
    out, lse = sa.sparse_attn_paged_decode(c.q, c.cache(sa), table, _gpu(c.pos, torch.int64),
                                           c.graph(sa), c.scale)
    with pytest.raises(sa.SparseAttentionError):
        sa.sparse_attn_check_device()
    assert not out[0].any() and torch.isneginf(lse[0]).all()
    c.check(out, lse, skip=(0,))


def test_decode_on_two_streams_at_once(sa):
    """Calls that overlap, each with its own workspace."""
    cases = [Case([9999, 5000, 77], 8, 2, 64, 16, "bf16", 10000, 10000, seed=s) for s in (1, 2)]
    args = []
    for c in cases:
        g, cache = c.graph(sa), c.cache(sa)
        need = sa.sparse_attn_paged_decode_workspace_size(c.q, cache, g)
        args.append((c, cache, _gpu(c.table, torch.int32), _gpu(c.pos, torch.int64), g,
                     torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for x, (c, cache, table, pos, g, ws) in enumerate(args):
            with torch.cuda.stream(streams[x]):
                outs[x].append(sa.sparse_attn_paged_decode(c.q, cache, table, pos, g, c.scale,
                                                           workspace=ws))
    torch.cuda.synchronize()
    for x, c in enumerate(cases):
        c.check(*outs[x][0])
        for o, l in outs[x][1:]:
            assert torch.equal(o, outs[x][0][0]) and torch.equal(l, outs[x][0][1])


def test_binding_refusals(sa):
    """Shapes, types and devices that the binding refuses before the library is called."""
    c = Case([5, 6], 4, 2, 64, 16, "bf16", 100, 100)
    cache, g = c.cache(sa), c.graph(sa)
    table, pos = _gpu(c.table, torch.int32), _gpu(c.pos, torch.int64)

    def bad(**kw):
        a = dict(q=c.q, table=table, pos=pos)
        rest = {k: v for k, v in kw.items() if k not in a}
        a.update({k: v for k, v in kw.items() if k in a})
        with pytest.raises((ValueError, sa.SparseAttentionError)):
            sa.sparse_attn_paged_decode(a["q"], cache, a["table"], a["pos"], g, 0.125, **rest)

    bad(q=c.q.cpu())
    bad(q=c.q.float())
    bad(q=c.q[:, :3].contiguous())
    bad(q=c.q[..., :32].contiguous())
    bad(q=c.q[:1])
    bad(table=table.long())
    bad(table=table.cpu())
    bad(table=table[:1])
    bad(table=table.t())
    bad(pos=pos.int())
    bad(pos=pos[:1])
    bad(pos=pos.cpu())
    bad(row=pos)
    bad(row=torch.zeros(3, dtype=torch.int32, device="cuda"))
    bad(out=torch.empty_like(c.q, dtype=torch.float32))
    bad(out=torch.empty_like(c.q[:1]))
    bad(lse=torch.empty((2, 2), device="cuda"))
    wide = sa.sparse_attn_paged_decode_workspace_size(c.q, cache, g)
    if wide:
        bad(workspace=torch.empty(wide - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises((ValueError, sa.SparseAttentionError)):
        sa.sparse_attn_paged_decode(c.q, cache, table, pos, g, math.nan)
    k = torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16)
    slot = torch.zeros(2, dtype=torch.int64, device="cuda")
    for kk, vv, ss in ((k.float(), k, slot), (k[:, :1], k, slot), (k, k[:1], slot),
                       (k, k, slot.int()), (k, k, slot[:1]), (k.cpu(), k, slot),
                       (k[..., :32], k, slot), (k[:, :, ::2], k, slot),
                       (torch.zeros((2, 2, 68), device="cuda", dtype=k.dtype)[..., :64], k, slot)):
        with pytest.raises((ValueError, sa.SparseAttentionError)):
            sa.sparse_attn_paged_append(kk, vv, cache, ss)
    x = torch.zeros((2, 2, 16, 64), device="cuda", dtype=torch.bfloat16)
    s = torch.zeros((2, 2, 16), device="cuda")
    for a in ((x, x[:1]), (x, x.float()), (x.half(), x.half()), (x, x, s, s),
              (x.to(torch.float8_e4m3fn),) * 2, (x[0], x[0]), (x, x.transpose(1, 2))):
        with pytest.raises(ValueError):
            sa.PagedCache(*a)
    with pytest.raises(ValueError):
        sa.PagedCache(*(x.to(torch.float8_e4m3fn),) * 2, s, s.double())
