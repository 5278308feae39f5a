"""Resize and compact on books with damaged entries, in both forms of the
resize kernel (pools up to 32768 pages, and larger ones): a shorter length is
carried out for the entries that name a held page, the others are reported."""
import pytest

torch = pytest.importorskip("torch")

import test_pages as TP
from test_pages import BAD_BLOCK, BAD_REQUEST, dev


@pytest.fixture(scope="module")
def PG():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding, build, pages
    build.build()  # no-op when the in-tree library is up to date
    binding.lib()
    return pages


def test_the_header_says_so():
    import os
    import re
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(here, "include", "pagedattn.h")) as f:
        text = re.sub(r"\s*\n \*\s*", " ", f.read())
    assert "A shorter length is carried out whatever the row's entries hold" in text


@pytest.mark.gpu
@pytest.mark.parametrize("blocks", [50, 32768, 32769])
def test_a_shorter_length_over_damaged_entries(PG, blocks):
    def fresh():
        books = TP.Books(4, 12, blocks, 16)
        books.resize([0, 1, 2], [100, 128, 40])  # pages 0..6, 7..14, 15..17
        books.fork([1], [3])
        return books, TP.pool_of(PG, books)

    for entry, page in ((5, -3), (5, blocks), (5, 1 << 30), (0, -1)):
        books, pool = fresh()
        pool.block_table[1, entry] = page
        pool.resize(dev([1, 0]), dev([33, 10]))
        kept = entry < 3  # entries 0..2 stay, 3..7 are given up
        assert pool.get_error() == (0 if kept else BAD_BLOCK)
        refs = books.refs.copy()
        refs[1:7] -= 1
        refs[10:15] -= 1  # row 1's pages 10..14
        if not kept:
            refs[7 + entry] += 1  # ... but the one that it no longer names
        assert pool.ref_counts.tolist() == refs.tolist()
        assert pool.context_lens.tolist() == [10, 33, 40, 128]
    # a page whose count is 0 already: the other pages of the row are given up
    books, pool = fresh()
    pool.ref_counts[16] = 0
    pool.free(dev([2, 0]))
    assert pool.get_error() == BAD_REQUEST
    refs = books.refs.copy()
    refs[:7] = 0
    refs[15:18] = 0
    assert pool.ref_counts.tolist() == refs.tolist()
    assert pool.context_lens.tolist() == [0, 128, 0, 128]


@pytest.mark.gpu
@pytest.mark.parametrize("blocks,entries", [(50, 12), (50, 10000)])  # tables rewritten by one launch, by two
def test_compact_over_damaged_entries(PG, blocks, entries):
    books = TP.Books(4, entries, blocks, 16)
    books.resize([0, 1, 2], [100, 128, 40])
    books.resize([0], [0])
    for page, error in ((-5, BAD_BLOCK), (blocks, BAD_BLOCK), (40, BAD_REQUEST)):
        want = books.copy()
        pool = TP.pool_of(PG, books)
        pool.block_table[1, 2] = page
        want.compact()
        pool.compact()
        assert pool.get_error() == error
        want.table[1, 2] = page
        TP.same(pool, want)
