"""Resize on both sides of the number of requests up to which one plan is made
by every CTA, on one pool, exactly."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import test_pages as TP


@pytest.mark.gpu
@pytest.mark.parametrize("rows,entries,blocks,bs", [(255, 9, 1500, 16), (256, 9, 1500, 32), (257, 9, 1500, 16),
                                                    (600, 5, 2500, 48)])
def test_random_walk_around_the_form_that_plans_in_every_cta(rows, entries, blocks, bs):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import pages
    TP.test_random_walk(pages, rows, rows, entries, blocks, bs)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [256, 257])
def test_every_row_in_one_call(n):
    """All rows grown, forked pages written in common, all given up."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import pages
    books = TP.Books(n, 30, 6000, 16)
    pool = TP.pool_of(pages, books)
    rng = np.random.default_rng(n)
    half = n // 2
    steps = [(list(range(half)), [int(x) for x in rng.integers(0, 300, half)]),
             None,
             (list(range(n)), [int(x) for x in rng.integers(0, 480, n)]),
             (list(range(n))[::-1], [int(x) for x in rng.integers(0, 480, n)]),
             (list(range(n)), [0] * n)]
    for step in steps:
        if step is None:
            books.fork(list(range(half)), list(range(half, 2 * half)))
            pool.fork(TP.dev(list(range(half))), TP.dev(list(range(half, 2 * half))))
            continue
        src, dst, errors = books.resize(*step)
        got = pool.resize(TP.dev(step[0]), TP.dev(step[1]))
        assert (got[0].tolist(), got[1].tolist()) == (src, dst)
        TP.same(pool, books)
        assert pool.get_error() == TP.worst(errors)
    assert not books.refs.any()
