"""Cases of the paged key-value cache: the page plan of a step, the writing of new rows and the
attention of new tokens over the sparse graph.

Three operators, as a serving loop calls them one after the other:
  plan    block tables, slot maps and the free-page stack from request lengths
  append  new key and value rows into their slots (bf16, fp32, or e4m3 with a scale per row)
  decode  softmax over N(pos) of a graph, keys and values read through the block table

`run` computes them in plain torch operations in 32 bits, or, with `own` set, by the library's
entry points.  `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}


def listed():
    return [
        # the bookkeeping of one decode step of 64 sequences with 16K caches
        dict(name="plan_step_64", op="plan", B=64, page=16, max_pages=1024, tokens=0),
        # a scheduler's large mixed step: prompts of all lengths, running and finished requests
        dict(name="plan_mixed_2000", op="plan", B=2000, page=32, max_pages=512, tokens=60000),
        # the keys and values of one decode step (64 sequences, 2 cache heads)
        dict(name="append_step_64", op="append", N=64, Hkv=2, D=64, page=16, dtype="bf16",
             wide=True),
        # the prompts of a prefill step, cached in 8 bits
        dict(name="append_16k_e4m3", op="append", N=16384, Hkv=8, D=128, page=32, dtype="e4m3",
             wide=True),
        # odd sizes: 3 heads of 32 columns, pages of 24 rows, fp32
        dict(name="append_odd_fp32", op="append", N=5003, Hkv=3, D=32, page=24, dtype="fp32",
             wide=False),
        # a long document's prompt at once
        dict(name="append_131k_bf16", op="append", N=131072, Hkv=8, D=128, page=64, dtype="bf16",
             wide=False),
        # 64 sequences on the 16K layer's graph (window 32 and links 2^k): 46 keys a token
        dict(name="decode_16k", op="decode", N=64, H=8, Hkv=2, D=64, T=16384, W=32, links=14,
             page=16, dtype="bf16", spread="upper", csr=False),
        # a 4,096-key window in 32K caches, 32 query heads over 8
        dict(name="decode_window_4k", op="decode", N=16, H=32, Hkv=8, D=128, T=32768, W=4096,
             links=0, page=32, dtype="bf16", spread="upper", csr=False),
        # one sequence of 131,072 tokens, every earlier key: a single row over the whole GPU
        dict(name="decode_full_131k", op="decode", N=1, H=32, Hkv=8, D=128, T=131072, W=131072,
             links=0, page=64, dtype="bf16", spread="last", csr=False),
        # a ragged batch, from one token to 32K, padded rows among them, cached in 8 bits
        dict(name="decode_ragged_e4m3", op="decode", N=48, H=8, Hkv=2, D=128, T=32768, W=32768,
             links=0, page=16, dtype="e4m3", spread="ragged", csr=False),
        # odd sizes in fp32: heads in pairs, pages of 17 rows, window and links
        dict(name="decode_odd_fp32", op="decode", N=7, H=6, Hkv=3, D=32, T=5000, W=1000, links=13,
             page=17, dtype="fp32", spread="ragged", csr=False),
        # the graph view: CSR rows of a window of 64, 16 shared and 16 random earlier keys
        dict(name="decode_csr_64k", op="decode", N=32, H=8, Hkv=8, D=64, T=65536, W=64, links=0,
             page=32, dtype="bf16", spread="upper", csr=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "decode", "decode"])
    page = rng.choice([8, 16, 32, 64, rng.randint(9, 100)])
    if op == "plan":
        B = _log(rng, 1, 2000)
        return dict(op=op, B=B, page=page, max_pages=_log(rng, 64, 2048),
                    tokens=rng.choice([0, _log(rng, max(B, 16), 60000)]))
    Hkv, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp32", "e4m3"])
    if op == "append":
        most = 131072 * 8 * 128 // (2 if dtype == "fp32" else 1) // (Hkv * D)
        return dict(op=op, N=_log(rng, 1, min(131072, most)), Hkv=Hkv, D=D, page=page,
                    dtype=dtype, wide=rng.random() < 0.5)
    T, group = _log(rng, 64, 131072), rng.choice([1, 2, 3, 4, 8, 16])
    W = min(T, rng.choice([32, _log(rng, 1, T), T]))
    links = rng.choice([0, T.bit_length()])
    N = _log(rng, 1, 256)
    csr = W <= 512 and T <= 65536 and rng.random() < 0.4
    N = max(1, min(N, (1 << 27) // ((W + 32) * Hkv * D), (1 << 29) // (T * Hkv * D)))
    return dict(op=op, N=N, H=Hkv * group, Hkv=Hkv, D=D, T=T, W=W, links=0 if csr else links,
                page=page, dtype=dtype, spread=rng.choice(["upper", "ragged"]), csr=csr)


def _pages(n, page):
    return -(-n // page)


def _quantise(x):
    """Rows of x in e4m3 and one scale for each row, the largest magnitude at 448."""
    x = x.float()
    amax = x.abs().amax(-1)
    scale = torch.where(torch.isfinite(amax), amax / 448.0, torch.nan)
    y = torch.where(scale[..., None] > 0, x / scale[..., None], 0.0)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _pool(gen, shape, dtype):
    """Key or value pages of a cache in use, and their scales."""
    x = torch.empty(shape, device=DEV, dtype=torch.float32 if dtype == "fp32" else torch.bfloat16)
    x.normal_(generator=gen)
    return _quantise(x) if dtype == "e4m3" else (x, None)


def _prepare_plan(case, gen, rng):
    B, page, M = case["B"], case["page"], case["max_pages"]
    length = rng.integers(1, M * page // 2 + 1, B)
    if case["tokens"]:
        # a mixed step: running requests, prompts of all lengths, finished and idle ones
        kind = rng.choice(4, B, p=[0.55, 0.3, 0.1, 0.05])
        weight = np.exp(rng.uniform(0.0, 5.0, B)) * (kind == 1)
        prompt = np.maximum(1, (weight / max(weight.sum(), 1e-9) * case["tokens"])).astype(np.int64)
        prompt = np.minimum(prompt, M * page)
        n_new = np.select([kind == 0, kind == 1, kind == 2], [1, prompt, -1], 0)
        length = np.where(kind == 1, 0, length)
    else:
        n_new = np.ones(B, dtype=np.int64)
    used = _pages(length, page)
    need = int((_pages(length + np.maximum(n_new, 0), page) - used).sum())
    # pages enough for nearly all of a mixed step: its last requests are refused
    spare = max(1, need if not case["tokens"] else int(need * 0.9))
    pool = B * (M // 2 + 2) + case["tokens"] // page + 1
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    table[np.arange(M)[None] < used[:, None]] = ids[: used.sum()]
    capacity = B + case["tokens"]
    stack = np.full(pool, -1, np.int32)
    stack[:spare] = ids[used.sum():used.sum() + spare]
    put = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(DEV, t)  # noqa: E731
    s = dict(length=put(length, torch.int64), n_new=put(n_new, torch.int32),
             table=put(table, torch.int32), stack=put(stack, torch.int32),
             count=torch.tensor([spare], device=DEV), capacity=capacity,
             length_out=torch.zeros(B, dtype=torch.int64, device=DEV),
             count_out=torch.zeros(1, dtype=torch.int64, device=DEV))
    if own:
        import sparse_graph_causal_b200 as sa
        s["batch"] = sa.PagedBatch(B, capacity, DEV)
    return s


def _prepare_append(case, gen, rng):
    N, Hkv, D, page = case["N"], case["Hkv"], case["D"], case["page"]
    n_pages = _pages(N, page) + 4
    kp, ks = _pool(gen, (n_pages, Hkv, page, D), case["dtype"])
    vp, vs = _pool(gen, (n_pages, Hkv, page, D), case["dtype"])
    src = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    if case["wide"]:  # slices of a fused projection: query heads, then keys, then values
        x = torch.empty((N, 6 * Hkv, D), device=DEV, dtype=src).normal_(generator=gen)
        k, v = x[:, 4 * Hkv:5 * Hkv], x[:, 5 * Hkv:]
    else:
        k, v = (torch.empty((N, Hkv, D), device=DEV, dtype=src).normal_(generator=gen)
                for _ in range(2))
    # pages in a pool's random order, rows in order inside each page; a padded row now and then
    order = torch.from_numpy(rng.permutation(n_pages)).to(DEV)
    at = torch.arange(N, device=DEV)
    slot = order[at // page] * page + at % page
    slot[N // 2:N // 2 + N // 64] = -1
    s = dict(k=k, v=v, kp=kp, vp=vp, ks=ks, vs=vs, slot=slot)
    if own:
        import sparse_graph_causal_b200 as sa
        s["cache"] = sa.PagedCache(kp, vp, ks, vs)
    return s


def _csr(T, W, gen):
    """Rows of a window, the first 16 keys and 16 random earlier ones, sorted, repeats removed."""
    i = torch.arange(T, device=DEV)[:, None]
    j = torch.cat([i - torch.arange(W, device=DEV), torch.arange(16, device=DEV).expand(T, 16),
                   (torch.rand((T, 16), device=DEV, generator=gen) * i).long()], 1)
    j = torch.where((j >= 0) & (j <= i), j, T).sort(1).values
    keep = j < T
    keep[:, 1:] &= j[:, 1:] != j[:, :-1]
    rowptr = torch.zeros(T + 1, dtype=torch.int64, device=DEV)
    rowptr[1:] = keep.sum(1).cumsum(0)
    return rowptr, j[keep].int()


def _deltas(case):
    """Distances of the keys of a structured row: the window, then the links beyond it."""
    links = [1 << k for k in range(case["links"]) if case["W"] <= 1 << k < case["T"]]
    return torch.cat([torch.arange(case["W"], device=DEV),
                      torch.tensor(links, dtype=torch.int64, device=DEV)])


def _prepare_decode(case, gen, rng):
    N, H, Hkv, D, T, page = (case[k] for k in ("N", "H", "Hkv", "D", "T", "page"))
    if case["spread"] == "ragged":
        pos = np.exp(rng.uniform(0.0, math.log(T), N)).astype(np.int64).clip(1, T) - 1
        pos[rng.integers(0, N)] = T - 1
        pos[rng.random(N) < 0.05] = -1
    else:
        pos = rng.integers(T // 2, T, N) if case["spread"] == "upper" else np.full(N, T - 1)
    M = _pages(T, page)
    used = _pages(pos + 1, page)
    n_pages = int(used.sum()) + 3
    table = np.full((N, M), -1, np.int32)
    table[np.arange(M)[None] < used[:, None]] = rng.permutation(n_pages)[: used.sum()]
    kp, ks = _pool(gen, (n_pages, Hkv, page, D), case["dtype"])
    vp, vs = _pool(gen, (n_pages, Hkv, page, D), case["dtype"])
    qt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    s = dict(q=torch.empty((N, H, 1, D), device=DEV, dtype=qt).normal_(generator=gen),
             kp=kp, vp=vp, ks=ks, vs=vs, table=torch.from_numpy(table).to(DEV),
             pos=torch.from_numpy(pos).to(DEV), scale=D ** -0.5, page=page)
    if case["csr"]:
        s["rowptr"], s["colidx"] = _csr(T, case["W"], gen)
        s["widest"] = int((s["rowptr"][1:] - s["rowptr"][:-1]).max())
    else:
        s["deltas"] = _deltas(case)
    if own:
        import sparse_graph_causal_b200 as sa
        if case["csr"]:
            s["graph"] = sa.sparse_attn_graph_build_csr(s["rowptr"], s["colidx"], case["W"])
        else:
            s["graph"] = sa.sparse_attn_graph_build_structured(T, case["W"],
                                                               list(range(case["links"])))
        s["cache"] = sa.PagedCache(kp, vp, ks, vs)
        s["workspace"] = torch.empty(
            sa.sparse_attn_paged_decode_workspace_size(s["q"], s["cache"], s["graph"]),
            dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((N, H), device=DEV)
    return s


def prepare(case, seed):
    gen = torch.Generator(DEV)
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    s = {"plan": _prepare_plan, "append": _prepare_append,
         "decode": _prepare_decode}[case["op"]](case, gen, rng)
    s["case"] = case
    return s


def _plan(s):
    page, capacity, table, stack = s["case"]["page"], s["capacity"], s["table"], s["stack"]
    length, n = s["length"], s["n_new"].long()
    B, M = table.shape
    index = torch.arange(M, device=DEV)
    tokens = n.clamp(min=0)
    cu = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    cu[1:] = tokens.cumsum(0)
    used = (length + page - 1) // page
    # finished requests give their pages back, on top of the stack
    gone = n == -1
    back = torch.where(gone, used, 0).cumsum(0)
    freed = gone[:, None] & (index < used[:, None])
    top = s["count"] + back[-1]
    place = torch.where(freed, (s["count"] + back - used)[:, None] + index, stack.numel())
    stack = torch.cat([stack, stack[:1]]).scatter_(0, place.reshape(-1), table.reshape(-1))[:-1]
    # the others take theirs from the top, in order, as long as there are enough
    total = (length + tokens + page - 1) // page
    fits = ~gone & (n >= 0) & (length + tokens <= M * page) & (cu[1:] <= capacity)
    need = torch.where(fits, total - used, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= top))
    taken = torch.where(ok, need, 0).sum()
    fresh = ok[:, None] & (index >= used[:, None]) & (index < total[:, None])
    which = top - 1 - (upto - need)[:, None] - (index - used[:, None])
    table = torch.where(fresh, stack[which.clamp(0, stack.numel() - 1)], table)
    # the tokens' places
    t = torch.arange(capacity, device=DEV)
    row = torch.searchsorted(cu[1:], t, right=True)
    real = (t < cu[-1])
    r = row.clamp(max=B - 1)
    pos = length[r] + t - cu[r]
    good = real & ok[r]
    p = torch.where(good, pos, 0)
    slot = table[r, p // page].long() * page + p % page
    status = torch.where(ok | gone, 0, torch.where(fits, 1, 2)).int()
    return dict(length=torch.where(gone, 0, torch.where(ok, length + tokens, length)),
                count=top - taken, table=table, stack=stack, cu_new=cu, status=status,
                slot=torch.where(good, slot, -1), pos=torch.where(good, pos, -1),
                row=torch.where(good, r, -1).int())


def _append(s):
    page, slot = s["case"]["page"], s["slot"]
    keep = torch.where(slot >= 0)[0]
    at = slot[keep]
    for_page, for_row = at // page, at % page
    out = {}
    if s["ks"] is None:
        s["kp"][for_page, :, for_row] = s["k"][keep]
        s["vp"][for_page, :, for_row] = s["v"][keep]
        return dict(k=s["kp"], v=s["vp"])
    kq, ks = _quantise(s["k"][keep])
    vq, vs = _quantise(s["v"][keep])
    s["kp"].view(torch.uint8)[for_page, :, for_row] = kq.view(torch.uint8)
    s["vp"].view(torch.uint8)[for_page, :, for_row] = vq.view(torch.uint8)
    s["ks"][for_page, :, for_row] = ks
    s["vs"][for_page, :, for_row] = vs
    return dict(k=s["kp"], v=s["vp"], k_scale=s["ks"], v_scale=s["vs"])


def _keys(s):
    """Key positions of each token's row and which of them are there: [N, width]."""
    pos = s["pos"][:, None]
    if s["case"]["csr"]:
        first = s["rowptr"][pos.clamp(min=0)]
        e = torch.arange(s["widest"], device=DEV)
        there = (pos >= 0) & (e < s["rowptr"][pos + 1] - first)
        return s["colidx"][torch.where(there, first + e, 0)].long(), there
    j = pos - s["deltas"]
    return j, j >= 0


def _rows(pool, scale, page, at):
    x = pool.view(torch.uint8)[page, :, at].view(pool.dtype) if scale is not None else \
        pool[page, :, at]
    return x.float() * scale[page, :, at][..., None] if scale is not None else x.float()


def _decode(s):
    q = s["q"]
    N, H, _, D = q.shape
    Hkv = s["kp"].shape[1]
    j, there = _keys(s)
    j = torch.where(there, j, 0)
    page = s["table"].gather(1, j // s["page"]).long()
    page, at = torch.where(there, page, 0), j % s["page"]
    k = _rows(s["kp"], s["ks"], page, at).transpose(1, 2)       # [N, Hkv, width, D]
    score = q.float().view(N, Hkv, H // Hkv, D) @ k.transpose(2, 3) * s["scale"]
    del k
    score = torch.where(there[:, None, None], score, -torch.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(torch.isfinite(m), m, 0.0)
    p = torch.exp(score - m)
    total = p.sum(-1, keepdim=True)
    v = _rows(s["vp"], s["vs"], page, at).transpose(1, 2)
    v = torch.where(there[:, None, :, None], v, 0.0)
    out = torch.where(total > 0, p @ v / total, 0.0)
    lse = (m + torch.log(total)).view(N, H)
    return dict(out=out.view(N, H, 1, D).to(q.dtype), lse=lse)


def run(s):
    op = s["case"]["op"]
    if own:
        import sparse_graph_causal_b200 as sa
        if op == "plan":
            b = s["batch"]
            sa.sparse_attn_paged_plan(s["length"], s["n_new"], s["table"], s["stack"], s["count"],
                                      s["case"]["page"], b, length_out=s["length_out"],
                                      free_count_out=s["count_out"])
            return dict(length=s["length_out"], count=s["count_out"], table=s["table"],
                        stack=s["stack"], cu_new=b.cu_new, status=b.status, slot=b.slot, pos=b.pos,
                        row=b.row)
        if op == "append":
            c = s["cache"]
            sa.sparse_attn_paged_append(s["k"], s["v"], c, s["slot"])
            if s["ks"] is None:
                return dict(k=c.k, v=c.v)
            return dict(k=c.k, v=c.v, k_scale=c.k_scale, v_scale=c.v_scale)
        out, lse = sa.sparse_attn_paged_decode(s["q"], s["cache"], s["table"], s["pos"],
                                               s["graph"], s["scale"], out=s["out"],
                                               lse=s["lse"], workspace=s["workspace"])
        return dict(out=out, lse=lse)
    return {"plan": _plan, "append": _append, "decode": _decode}[op](s)


def work(case):
    """Bytes read once and written once, and the operations on them."""
    if case["op"] == "plan":
        B, tokens = case["B"], case["tokens"] or case["B"]
        # lengths and counts in, lengths, offsets and states out; a token's three numbers; new pages
        return dict(bytes=32 * B + 20 * tokens + 8 * (tokens // case["page"] + 1), flops=0)
    size = {"bf16": 2, "fp32": 4, "e4m3": 1}[case["dtype"]]
    if case["op"] == "append":
        n = 2 * case["N"] * case["Hkv"]
        new = 2 if case["dtype"] == "e4m3" else size
        return dict(bytes=n * (case["D"] * (new + size) + (4 if size == 1 else 0)) + 8 * case["N"],
                    flops=2 * n * case["D"] if size == 1 else 0)
    # the keys of a row at its mean position
    T, N = case["T"], case["N"]
    x = {"upper": 0.75 * T, "last": T, "ragged": T / max(math.log(T), 1.0)}[case["spread"]]
    keys = case["W"] + 32 if case["csr"] else min(case["W"], x)
    keys += sum(case["W"] <= 1 << k < x for k in range(case["links"]))
    row = 2 * case["D"] * size + (8 if size == 1 else 0)
    io = case["H"] * (2 * case["D"] * (4 if size == 4 else 2) + 4)
    return dict(bytes=N * (keys * case["Hkv"] * row + io),
                flops=4 * N * keys * case["H"] * case["D"])


def exact(case, seed):
    def append(s):
        page, got = s["case"]["page"], {}
        slot = s["slot"].cpu().numpy()
        keep = np.nonzero(slot >= 0)[0]
        at = torch.from_numpy(slot[keep]).to(DEV)
        for name, new, pool, scale in (("k", "k", "kp", "ks"), ("v", "v", "vp", "vs")):
            x = s[new].double()[torch.from_numpy(keep).to(DEV)]
            flat = s[pool].double().transpose(1, 2).reshape(-1, *x.shape[1:])
            if s[scale] is not None:
                unit = x.abs().max(-1).values / 448
                x = x / unit[..., None]
                every = s[scale].double().transpose(1, 2).reshape(-1, unit.shape[1])
                every[at] = unit
                every = every.view(-1, page, unit.shape[1]).transpose(1, 2)
                got[name + "_scale"] = every.contiguous()
            flat[at] = x
            got[name] = flat.view(-1, page, *x.shape[1:]).transpose(1, 2).contiguous()
        return got

    def decode(s):
        case, q = s["case"], s["q"].double()
        N, H, _, D = q.shape
        group, page = H // case["Hkv"], case["page"]
        out = torch.zeros_like(q)
        lse = torch.full((N, H), -math.inf, device=DEV, dtype=torch.float64)
        for n, p in enumerate(s["pos"].tolist()):
            if p < 0:
                continue
            if case["csr"]:
                a, b = s["rowptr"][p:p + 2].tolist()
                keys = s["colidx"][a:b].long()
            else:
                far = [p - (1 << x) for x in range(case["links"]) if 1 << x >= case["W"]]
                far = [j for j in far if j >= 0]
                keys = torch.cat([torch.tensor(far, dtype=torch.int64, device=DEV),
                                  torch.arange(max(0, p - case["W"] + 1), p + 1, device=DEV)])
            where = s["table"][n].long()[keys // page]
            for h in range(case["Hkv"]):
                k, v = (s[x][where, h, keys % page].double() if s[y] is None else
                        s[x].view(torch.uint8)[where, h, keys % page].view(s[x].dtype).double()
                        * s[y][where, h, keys % page].double()[:, None]
                        for x, y in (("kp", "ks"), ("vp", "vs")))
                z = q[n, h * group:(h + 1) * group, 0] @ k.T / math.sqrt(D)
                total = torch.logsumexp(z, 1)
                lse[n, h * group:(h + 1) * group] = total
                out[n, h * group:(h + 1) * group, 0] = torch.exp(z - total[:, None]) @ v
        return dict(out=out, lse=lse)

    if case["op"] == "plan":  # whole numbers: nothing is rounded
        return None
    s = prepare(case, seed)
    return append(s) if case["op"] == "append" else decode(s)
