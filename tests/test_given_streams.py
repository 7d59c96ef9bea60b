"""Memory that a call makes for itself (outputs, workspaces) when it is given a stream that is not
the current one.  The allocator hands freed memory on in the order of the stream it was made on, so
it has to be made on the stream that the call's kernels run on."""
import ctypes
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def sa():
    import sparse_graph_causal_b200 as m
    return m


class _Library:
    """Every entry point answers 0 (no error, no bytes)."""

    def __getattr__(self, name):
        return lambda *args: 0


def _calls(sa):
    x = torch.zeros((2, 4, 8, 32))
    lse, q1 = torch.zeros((2, 4, 8)), torch.zeros((2, 4, 1, 32))
    pos = SimpleNamespace(dtype=torch.int64, is_cuda=True, numel=lambda: 2, data_ptr=lambda: 0)
    a = torch.zeros((2, 4, 8, 3))
    g = SimpleNamespace(handle=ctypes.c_void_p(1), T=8)
    cache = SimpleNamespace(_index=-1, _address=0, _ref=None, device="cpu")
    return dict(
        fwd=(2, lambda **kw: sa.sparse_attn_fwd(x, x, x, g, 1.0, **kw)),
        bwd=(4, lambda **kw: sa.sparse_attn_bwd(x, x, x, x, lse, x, g, 1.0, **kw)),
        bwd_noalloc=(3, lambda **kw: sa.sparse_attn_bwd_noalloc(x, x, x, x, lse, x, g, 1.0, **kw)),
        decode=(2, lambda **kw: sa.sparse_attn_decode(q1, x, x, pos, g, 1.0, **kw)),
        paged_decode=(3, lambda **kw: sa.sparse_attn_paged_decode(q1, cache, x, pos, g, 1.0, **kw)),
        dist_fwd=(2, lambda **kw: sa.sparse_attn_dist_fwd(a, a, x, g, 1.0, **kw)),
        dist_bwd=(4, lambda **kw: sa.sparse_attn_dist_bwd(a, a, x, x, lse, x, g, 1.0, **kw)),
        graph_export=(4, lambda **kw: sa.sparse_attn_graph_export(g, device="cpu", **kw)))


@pytest.mark.parametrize("name", ["fwd", "bwd", "bwd_noalloc", "decode", "paged_decode", "dist_fwd",
                                  "dist_bwd", "graph_export"])
def test_memory_is_made_on_the_given_stream(sa, monkeypatch, name):
    entered, made = [], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)

        def __exit__(self, *exc):
            entered.pop()

    def recorded(real):
        def make(*args, **kw):
            made.append(entered[-1] if entered else None)
            return real(*args, **kw)
        return make

    count, call = _calls(sa)[name]
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, recorded(getattr(torch, f)))
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(sa, "_lib", _Library())
    monkeypatch.setattr(sa, "_paged", _Library())
    monkeypatch.setattr(sa, "_tensor", lambda t, n: sa.SaTensor())
    monkeypatch.setattr(sa, "_coords", lambda t, n: sa.SaTensor())
    monkeypatch.setattr(sa, "sparse_attn_paged_decode_workspace_size", lambda *args: 64)
    call(stream=4096)
    assert made == [4096] * count and not entered
    # the legacy default stream has two handles
    for handle in (0, 1):
        made.clear()
        call(stream=handle)
        assert made == [0] * count and not entered


# ------------------------------------------------------------------ on the GPU

def _busy(stream):
    """Some ten milliseconds of waiting on a stream."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


def _overwrite(sizes):
    """New memory of these sizes, on the current stream, filled over and over."""
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    for _ in range(30):
        for x in junk:
            x.fill_(255)


def _same_on_a_busy_stream(call, sizes, raw):
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(3):
        _busy(stream)
        got = call(stream.cuda_stream if raw else stream)
        _overwrite([*sizes, *(t.nbytes for t in got)])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    got = call(0)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_paged_decode_on_a_given_stream(sa, raw):
    """Rows cut over the GPU: the workspace is written by one kernel and read by the next, long
    after the call has returned."""
    T, H, Hkv, D, page = 20000, 8, 2, 64, 16
    gen = torch.Generator("cuda")
    gen.manual_seed(1)
    M = -(-T // page)
    k, v = (torch.empty((2 * M, Hkv, page, D), device="cuda",
                        dtype=torch.bfloat16).normal_(generator=gen) for _ in range(2))
    q = torch.empty((2, H, 1, D), device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    table = torch.randperm(2 * M, device="cuda", generator=gen).int().view(2, M)
    pos = torch.tensor([T - 1, T // 3], device="cuda")
    cache, g = sa.PagedCache(k, v), sa.sparse_attn_graph_build_structured(T, T, [])
    need = sa.sparse_attn_paged_decode_workspace_size(q, cache, g)
    assert need > 0
    _same_on_a_busy_stream(
        lambda s: sa.sparse_attn_paged_decode(q, cache, table, pos, g, 0.125, stream=s), [need], raw)
    sa.sparse_attn_check_device()


@pytest.mark.gpu
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_attention_on_a_given_stream(sa, raw):
    T, W = 1024, 32
    gen = torch.Generator("cuda")
    gen.manual_seed(2)
    q, k, v, do = (torch.empty((2, 4, T, 64), device="cuda",
                               dtype=torch.bfloat16).normal_(generator=gen) for _ in range(4))
    a, c = (torch.empty((2, 4, T, 3), device="cuda").normal_(generator=gen) for _ in range(2))
    g = sa.sparse_attn_graph_build_structured(T, W, list(range(10)))

    def call(s):
        out, lse = sa.sparse_attn_fwd(q, k, v, g, 0.125, stream=s)
        grads = sa.sparse_attn_bwd(q, k, v, out, lse, do, g, 0.125, stream=s)
        y, l = sa.sparse_attn_dist_fwd(a, c, v, g, 0.5, stream=s)
        return (out, lse, *grads, y, l, *sa.sparse_attn_dist_bwd(a, c, v, y, l, do, g, 0.5, stream=s))

    sizes = [sa.sparse_attn_bwd_workspace_size(q, g), sa.sparse_attn_dist_bwd_workspace_size(v, g)]
    _same_on_a_busy_stream(call, sizes, raw)
    sa.sparse_attn_check_device()
