"""Calls on several streams at once, each with a workspace of its own: shared
and plain decodes of different cache types and page operations.  Every result
is what the same call gives alone, bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_pages as TP
import test_shared_prefix as TS
from paged_kv_decode_flash_b200 import inputs as gen


@pytest.mark.gpu
def test_streams_do_not_disturb_each_other():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding as B, build, pages, shared_prefix
    build.build()  # no-op when the in-tree library is up to date
    jobs = []
    for seed, (dt, prefix, own, nq, G, Hkv) in enumerate((
            (gen.KV_FP16, 8192, (20, 400, 77, 9) * 6, 2, 4, 8),
            (gen.KV_Q8_0, 2048, (5, 130, 60) * 10, 4, 4, 4),
            (gen.KV_INT8_ROW, 4096, (33, 900) * 4, 4, 6, 4),
            (gen.KV_FP16, 64, tuple(range(2, 152)), 1, 2, 2))):
        case = TS.shared_case(prefix, own, seed=seed, n_query=nq, num_q_heads=G * Hkv, num_kv_heads=Hkv, kv_dtype=dt)
        dec, args, kw = TS.prepared(shared_prefix, case, prefix)
        out = torch.empty_like(args[0])
        jobs.append((lambda st, d=dec, a=args, k=kw, o=out: d(*a, out=o, stream=st, **k), out, dec))
        plain = B.PagedDecode.for_case(case)
        full = [*args[:3], torch.from_numpy(case.block_table).cuda(), args[4]]
        out = torch.empty_like(args[0])
        jobs.append((lambda st, d=plain, a=full, k=kw, o=out: d(*a, out=o, stream=st, **k), out, plain))
    alone = []
    for call, out, dec in jobs:
        call(None)
        assert dec.get_error() == 0
        alone.append(out.clone())
        out.zero_()
    books = TP.Books(40, 30, 3000, 16)
    pool = TP.pool_of(pages, books)
    rng = np.random.default_rng(5)
    steps = [([int(x) for x in rng.permutation(40)], [int(x) for x in rng.integers(0, 480, 40)]) for _ in range(25)]
    requests = [(TP.dev(r), TP.dev(n)) for r, n in steps]
    streams = [torch.cuda.Stream() for _ in jobs]
    paging = torch.cuda.Stream()
    torch.cuda.synchronize()
    for rows, new in requests:
        for (call, _, _), st in zip(jobs, streams):
            call(st)
        pool.resize(rows, new, stream=paging)
    torch.cuda.synchronize()
    for (_, out, dec), want in zip(jobs, alone):
        assert dec.get_error() == 0
        assert torch.equal(out, want)
    for rows, new in steps:
        books.resize(rows, new)
    TP.same(pool, books)
    assert pool.get_error() == 0
