"""Calls that are given a stream and make their own outputs: the memory has to
be the stream's.  A block that the current stream has freed may still be in use
by work queued there; on another stream it would be written too early.

The values are copied or compared with the same call's on the current stream,
bit for bit."""
import contextlib
import types

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from paged_kv_decode_flash_b200 import binding as B
from paged_kv_decode_flash_b200 import inputs as gen
import test_pages as TP
import test_shared_prefix as TS


# ---------------------------------------------------------------------------
# without a GPU: where the allocations are made
# ---------------------------------------------------------------------------
class FakeStream:
    cuda_stream, device = 64, None


@pytest.fixture
def log(monkeypatch):
    """Every allocation of an output with the stream that is current, on a
    library that does nothing."""
    at = types.SimpleNamespace(current="default", made=[], recorded=[])

    @contextlib.contextmanager
    def stream(s):
        before, at.current = at.current, s
        yield
        at.current = before

    def logged(f):
        def call(*a, **kw):
            at.made.append(at.current)
            kw.pop("device", None)
            return f(*a, **kw)
        return call

    nothing = types.SimpleNamespace(**{n: lambda *a: 0 for n in (
        "paged_attn_resize", "paged_attn_compact", "paged_attn_decode_shared", "paged_attn_decode",
        "paged_attn_decode_partial", "paged_attn_trace", "paged_attn_merge")})
    monkeypatch.setattr(B, "lib", lambda: nothing)
    monkeypatch.setattr(B, "_on", lambda index, s, call: call(64))
    monkeypatch.setattr(B, "_stream_ptr", lambda s: 64)
    monkeypatch.setattr(B, "_dptr", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: at.current)
    monkeypatch.setattr(torch, "empty", logged(torch.empty))
    monkeypatch.setattr(torch, "empty_like", logged(torch.empty_like))
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: at.recorded.append(s))
    return at


def pool_on_the_host():
    from paged_kv_decode_flash_b200.pages import PagePool
    pool = object.__new__(PagePool)
    pool.device = torch.device("cpu")
    pool.dims = B.Dims(4, 1, 1, 128, 16, 4, 20, None, 0)
    for name, n in (("block_table", 16), ("context_lens", 4), ("ref_counts", 20)):
        setattr(pool, name, torch.zeros(n, dtype=torch.int32))
    return pool


def decoder_on_the_host(cls):
    dec = object.__new__(cls)
    dec.n_query, dec.prefix_blocks = 1, 7
    dec.dims = B.Dims(2, 4, 2, 128, 16, 10, 25, None, 0)
    dec.workspace = torch.zeros(64, dtype=torch.uint8)
    dec._caches = {0: (torch.float16, (25, 2, 16, 128))}
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    half = lambda *s: torch.zeros(s, dtype=torch.float16)
    return dec, (half(2, 1, 4, 128), half(25, 2, 16, 128), half(25, 2, 16, 128), i32(2, 10), i32(2)), i32


def calls():
    from paged_kv_decode_flash_b200.shared_prefix import SharedPrefixDecode
    kw = dict(causal=1, window=0, scale=0.1, kv_dtype=0)

    def resize(stream):
        rows = torch.zeros(2, dtype=torch.int32)
        pool_on_the_host().resize(rows, rows, stream=stream)

    def compact(stream):
        pool_on_the_host().compact(stream=stream)

    def shared(stream):
        dec, args, i32 = decoder_on_the_host(SharedPrefixDecode)
        dec(*args, i32(7), i32(1), stream=stream, **kw)

    def plain(stream):
        dec, args, _ = decoder_on_the_host(B.PagedDecode)
        dec(*args, stream=stream, **kw)

    def partial(stream):
        dec, args, i32 = decoder_on_the_host(B.PagedDecode)
        dec.partial(*args, i32(2), i32(2), stream=stream, **kw)

    def trace(stream):
        dec, args, _ = decoder_on_the_host(B.PagedDecode)
        dec.trace(*args, stream=stream, **kw)

    def merge(stream):
        B.merge(torch.zeros(3, 5, 128), torch.zeros(3, 5), stream=stream)

    return dict(resize=resize, compact=compact, shared=shared, plain=plain, partial=partial, trace=trace,
                merge=merge)


@pytest.mark.parametrize("name", list(calls()))
def test_outputs_are_allocated_on_the_stream_that_writes_them(log, name):
    s = FakeStream()
    calls()[name](s)
    assert log.made and all(c is s for c in log.made), log.made
    assert len(log.recorded) >= 1 and set(log.recorded) == {"default"}  # where the caller may use them
    log.made.clear()
    log.recorded.clear()
    calls()[name](None)
    assert log.made and set(log.made) == {"default"} and not log.recorded


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import build
    build.build()  # no-op when the in-tree library is up to date
    return B.lib()


def beside_a_busy_stream(call, like):
    """call(stream) while the current stream still has to write and read
    tensors like these, which are freed already.  Returns its outputs."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    temporaries = [torch.full_like(t, 77) for t in like]
    used = [t.clone() for t in temporaries]
    del temporaries
    got = call(s)
    s.synchronize()
    with torch.cuda.stream(s):
        copies = [t.clone() for t in got]
    torch.cuda.synchronize()
    assert all((t == 77).all() for t in used)
    for t, c in zip(got, copies):
        assert torch.equal(t, c)
    return got


@pytest.mark.gpu
def test_page_lists_beside_a_busy_stream(lib):
    from paged_kv_decode_flash_b200 import pages
    books = TP.Books(6, 20, 90, 16)
    books.resize([0], [37])
    books.fork([0] * 3, [1, 2, 3])
    pool = TP.pool_of(pages, books)
    rows, new = TP.dev([1, 2, 3, 0, 4]), TP.dev([38, 50, 38, 0, 100])
    want = books.resize(rows.tolist(), new.tolist())
    got = beside_a_busy_stream(lambda s: pool.resize(rows, new, stream=s), (rows, rows))
    assert (got[0].tolist(), got[1].tolist()) == want[:2]
    TP.same(pool, books)
    want = books.compact()
    lists = torch.empty(2 * 45 + 1 + 90, dtype=torch.int32, device="cuda")

    def compact(s):
        m = pool.compact(stream=s)
        return [m.src, m.dst, m.count, m.remap]

    src, dst, count, remap = beside_a_busy_stream(compact, (lists,))
    assert (src.tolist(), dst.tolist(), count.item()) == want[:3]
    assert np.array_equal(remap.cpu().numpy(), want[3])
    TP.same(pool, books)
    assert pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [gen.KV_FP16, gen.KV_Q8_0, gen.KV_INT8_ROW])
def test_attention_beside_a_busy_stream(lib, dt):
    from paged_kv_decode_flash_b200 import shared_prefix
    case = TS.shared_case(512, (9, 40, 100), n_query=2, num_q_heads=8, num_kv_heads=2, kv_dtype=dt)
    dec, args, kw = TS.prepared(shared_prefix, case, 512)
    want = dec(*args, **kw)
    assert torch.equal(beside_a_busy_stream(lambda s: [dec(*args, stream=s, **kw)], (want,))[0], want)
    plain = B.PagedDecode.for_case(case)
    full = [*args[:3], torch.from_numpy(case.block_table).cuda(), args[4]]
    want = plain(*full, **kw)
    assert torch.equal(beside_a_busy_stream(lambda s: [plain(*full, stream=s, **kw)], (want,))[0], want)
    begin, count = TP.dev([0, 0, 0]), TP.dev([256, 256, 256])
    want = plain.partial(*full, begin, count, **kw)
    got = beside_a_busy_stream(lambda s: plain.partial(*full, begin, count, stream=s, **kw), want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    parts, lses = torch.stack([want[0].view(-1, 128)] * 2), torch.stack([want[1].view(-1)] * 2)
    want = B.merge(parts, lses)
    got = beside_a_busy_stream(lambda s: B.merge(parts, lses, stream=s), want)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert dec.get_error() == 0 and plain.get_error() == 0


# ---------------------------------------------------------------------------
# the context-parallel call: partial, gather and merge in one order
# ---------------------------------------------------------------------------
def test_the_gather_of_partials_runs_on_the_stream_that_makes_them(log, monkeypatch):
    from paged_kv_decode_flash_b200 import context_parallel as CP
    dec, args, i32 = decoder_on_the_host(B.PagedDecode)
    cp = object.__new__(CP.ContextParallelDecode)
    cp.B, cp.dec = B, dec
    at = []

    def exchange(po, pl, dist):
        at.append(log.current)
        return po[None], pl[None]

    monkeypatch.setattr(CP, "exchange", exchange)
    s = FakeStream()
    kw = dict(causal=1, window=0, scale=0.1, kv_dtype=0)
    cp(None, *args, i32(2), i32(2), stream=s, **kw)
    cp(None, *args, i32(2), i32(2), **kw)
    assert at == [s, "default"]
