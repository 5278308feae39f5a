"""The page operations (fork, resize, compact, copy) against a plain sequential
implementation on the host, exactly: every value is a whole number or bytes."""
import ctypes
import dataclasses

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
from paged_kv_decode_flash_b200 import inputs as gen

DTYPES = (gen.KV_FP16, gen.KV_Q8_0, gen.KV_INT8_ROW)
BAD_BLOCK, BAD_LEN, BAD_REQUEST, NO_PAGES = -5, -6, -8, -9


# ---------------------------------------------------------------------------
# the plain implementation
# ---------------------------------------------------------------------------
class Books:
    def __init__(self, rows, entries, blocks, bs):
        self.table = np.full((rows, entries), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        self.refs = np.zeros(blocks, np.int32)
        self.bs = bs

    def copy(self):
        b = Books(*self.table.shape, len(self.refs), self.bs)
        b.table, b.lens, b.refs = self.table.copy(), self.lens.copy(), self.refs.copy()
        return b

    def held(self, n):
        return -(-int(n) // self.bs)

    def row_ok(self, r):
        return 0 <= r < len(self.lens)

    def len_ok(self, n):
        return 0 <= n <= self.table.shape[1] * self.bs

    def fork(self, parents, children):
        before, error = self.copy(), set()
        for i, (p, c) in enumerate(zip(parents, children)):
            if not self.row_ok(p) or not self.row_ok(c) or p in children or c in children[:i] or before.lens[c] != 0:
                error.add(BAD_REQUEST)
                continue
            n = self.held(before.lens[p])
            self.table[c, :n] = before.table[p, :n]
            for page in before.table[p, :n]:
                self.refs[page] += 1
            self.lens[c] = before.lens[p]
        return error

    def resize(self, rows, new):
        before, error = self.copy(), set()
        free = [b for b in range(len(self.refs)) if before.refs[b] == 0]
        src, dst = [-1] * len(rows), [-1] * len(rows)
        stands, ragged = [], []
        for i, (r, n) in enumerate(zip(rows, new)):
            ok = self.row_ok(r) and self.len_ok(n) and r not in [q for q, s in zip(rows[:i], stands) if s]
            if not self.row_ok(r):
                error.add(BAD_REQUEST)
            elif not self.len_ok(n):
                error.add(BAD_LEN)
            elif not ok:
                error.add(BAD_REQUEST)
            stands.append(ok)
            old = before.lens[r] if ok else 0
            ragged.append(int(before.table[r, old // self.bs]) if ok and n > old and old % self.bs else -1)
        used, out_of_pages = 0, False
        for i, (r, n) in enumerate(zip(rows, new)):
            if not stands[i]:
                continue
            old = int(before.lens[r])
            if n <= old:
                for b in range(self.held(n), self.held(old)):
                    self.refs[before.table[r, b]] -= 1
                self.lens[r] = n
                continue
            page = ragged[i]
            split = page >= 0 and before.refs[page] > 1
            if split and ragged.count(page) == before.refs[page] and page not in ragged[i + 1:]:
                split = False
            need = self.held(n) - self.held(old) + split
            used += need
            if used > len(free):
                out_of_pages = True
            if out_of_pages:
                error.add(NO_PAGES)
                continue
            fresh = free[used - need:used]
            if split:
                f = fresh.pop(0)
                src[i], dst[i] = page, f
                self.table[r, old // self.bs] = f
                self.refs[f] = 1
                self.refs[page] -= 1
            for b, f in zip(range(self.held(old), self.held(n)), fresh):
                self.table[r, b] = f
                self.refs[f] = 1
            self.lens[r] = n
        return src, dst, error

    def compact(self):
        n = len(self.refs)
        live = [b for b in range(n) if self.refs[b] > 0]
        gaps = [b for b in range(len(live)) if self.refs[b] == 0]
        high = [b for b in live if b >= len(live)]
        remap = np.full(n, -1, np.int32)
        remap[live] = live
        remap[high] = gaps
        refs = np.zeros_like(self.refs)
        for b in live:
            refs[remap[b]] = self.refs[b]
        self.refs = refs
        for r in range(len(self.lens)):
            for b in range(self.held(self.lens[r])):
                self.table[r, b] = remap[self.table[r, b]]
        room = max(1, n // 2)
        fill = [-1] * (room - len(high))
        return high + fill, gaps + fill, len(high), remap


def test_the_plain_implementation():
    """Hand-worked: a prompt of 5 tokens in pages of 2, two answers."""
    b = Books(3, 8, 10, 2)
    assert b.resize([0], [5]) == ([-1], [-1], set())
    assert list(b.table[0, :3]) == [0, 1, 2] and list(b.refs[:4]) == [1, 1, 1, 0]
    assert b.fork([0, 0], [1, 2]) == set()
    assert list(b.refs[:4]) == [3, 3, 3, 0] and list(b.lens) == [5, 5, 5]
    # all three grow out of page 2: two copies, the last request keeps it
    src, dst, e = b.resize([1, 2, 0], [6, 7, 6])
    assert (src, dst, e) == ([2, 2, -1], [3, 4, -1], set())
    assert list(b.table[2, :4]) == [0, 1, 4, 5] and list(b.refs) == [3, 3, 1, 1, 1, 1, 0, 0, 0, 0]
    b.resize([0], [0])
    assert list(b.refs) == [2, 2, 0, 1, 1, 1, 0, 0, 0, 0]
    src, dst, n, remap = b.compact()
    assert (src[:n], dst[:n], n) == ([5], [2], 1)
    assert list(b.table[2, :4]) == [0, 1, 4, 2] and list(b.refs[:6]) == [2, 2, 1, 1, 1, 0]


# ---------------------------------------------------------------------------
# without a GPU: sizes and refusals
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    from paged_kv_decode_flash_b200 import build
    build.build()
    from paged_kv_decode_flash_b200 import binding
    return binding.lib()


def dims(**kw):
    from paged_kv_decode_flash_b200.binding import Dims
    d = dict(num_seqs=6, num_q_heads=8, num_kv_heads=8, head_dim=128, block_size=16,
             max_blocks_per_seq=30, num_blocks=100, workspace=4096, workspace_bytes=1 << 20)
    d.update(kw)
    return Dims(**d)


def test_workspace_size(L):
    size = lambda d: L.paged_attn_pages_workspace_size(ctypes.byref(d))
    n = size(dims())
    assert n > 256 and n % 256 == 0
    assert size(dims(num_blocks=100000)) >= 100000 * 12
    for bad in (dims(block_size=8), dims(num_seqs=0), dims(head_dim=64), dims(num_blocks=0)):
        assert size(bad) == 0
    assert L.paged_attn_pages_workspace_size(None) == 0


def test_refusals_on_the_host(L):
    from paged_kv_decode_flash_b200 import binding as b
    p, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 2)  # never dereferenced
    calls = {
        "fork": (L.paged_attn_fork, [p, p, p, p, p, 2], (0, 1, 2, 3, 4), 5, 6),
        "resize": (L.paged_attn_resize, [p, p, p, p, p, 2, p, p], (0, 1, 2, 3, 6, 7), 5, 6),
        "compact": (L.paged_attn_compact, [p, p, p, p, p, p, p], range(7), None, None),
        "copy": (L.paged_attn_copy_blocks, [p, p, 2, None, 0, p, p], (0, 1, 5, 6), 2, 100),
    }
    for name, (f, args, pointers, n_at, n_most) in calls.items():
        def call(d, change=None, value=None):
            a = list(args)
            if change is not None:
                a[change] = value
            return f(ctypes.byref(d) if d is not None else None, *a, None)
        assert call(None) == b.PA_ERR_INVALID_ARG, name
        for at in pointers:
            assert call(dims(), at, None) == b.PA_ERR_INVALID_ARG, (name, at)
            assert call(dims(), at, odd) == b.PA_ERR_INVALID_ARG, (name, at)
        if n_at is not None:
            assert call(dims(), n_at, -1) == b.PA_ERR_INVALID_ARG, name
            assert call(dims(), n_at, n_most + 1) == b.PA_ERR_INVALID_ARG, name
            assert call(dims(), n_at, 0) == b.PA_OK, name  # nothing to do, nothing enqueued
        assert call(dims(head_dim=64)) == b.PA_ERR_UNSUPPORTED, name
        assert call(dims(workspace=None)) == b.PA_ERR_WORKSPACE, name
        assert call(dims(workspace=4100)) == b.PA_ERR_WORKSPACE, name
        assert call(dims(workspace_bytes=256)) == b.PA_ERR_WORKSPACE, name
    assert L.paged_attn_resize(ctypes.byref(dims()), p, p, p, p, odd, 2, p, p, None) == b.PA_ERR_INVALID_ARG
    assert L.paged_attn_copy_blocks(ctypes.byref(dims()), p, p, 2, odd, 0, p, p, None) == b.PA_ERR_INVALID_ARG
    assert L.paged_attn_copy_blocks(ctypes.byref(dims()), p, p, 2, None, 5, p, p, None) == b.PA_ERR_INVALID_ARG
    assert L.paged_attn_pages_workspace_init(ctypes.byref(dims(workspace=None)), None) == b.PA_ERR_WORKSPACE
    assert L.paged_attn_pages_workspace_init(None, None) == b.PA_ERR_INVALID_ARG
    for code in (-8, -9):
        assert L.paged_attn_status_string(code) != b"unknown status"


def test_a_workspace_elsewhere_is_refused(L):
    from paged_kv_decode_flash_b200 import pages
    with pytest.raises(ValueError, match="workspace"):
        pages.PagePool(num_seqs=3, num_kv_heads=1, head_dim=128, block_size=16, max_blocks_per_seq=4,
                       num_blocks=20, device="cuda:0", workspace=torch.empty(4096, dtype=torch.uint8))


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def PG():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding, build, pages
    build.build()  # no-op when the in-tree library is up to date
    binding.lib()
    return pages


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def pool_of(PG, books, heads=2):
    rows, entries = books.table.shape
    return PG.PagePool(num_seqs=rows, num_kv_heads=heads, head_dim=128, block_size=books.bs,
                       max_blocks_per_seq=entries, num_blocks=len(books.refs),
                       block_table=dev(books.table), context_lens=dev(books.lens),
                       ref_counts=dev(books.refs))


def same(pool, books, what=""):
    assert np.array_equal(pool.block_table.cpu().numpy(), books.table), what
    assert np.array_equal(pool.context_lens.cpu().numpy(), books.lens), what
    assert np.array_equal(pool.ref_counts.cpu().numpy(), books.refs), what


def worst(errors):
    """What get_error reports of several."""
    return next((e for e in (BAD_BLOCK, BAD_LEN, BAD_REQUEST, NO_PAGES) if e in errors), 0)


@pytest.mark.gpu
@pytest.mark.parametrize("seed,rows,entries,blocks,bs", [
    (0, 5, 12, 30, 16), (1, 40, 60, 700, 16), (2, 300, 8, 1500, 48), (3, 17, 200, 20000, 32),
    (4, 1, 3, 2, 16), (5, 9, 5, 1, 16), (6, 1300, 4, 9000, 16), (7, 60, 30, 333, 112)])
def test_random_walk(PG, seed, rows, entries, blocks, bs):
    """Steps of every kind on one pool, with bad requests mixed in, compared
    after each."""
    rng = np.random.default_rng(seed)
    books = Books(rows, entries, blocks, bs)
    pool = pool_of(PG, books)
    pick = lambda k: [int(x) for x in rng.permutation(rows)[:k]]
    for step in range(14):
        kind = int(rng.integers(0, 5))
        if kind == 4:
            want = books.compact()
            got = pool.compact()
            assert got.src.tolist() == want[0] and got.dst.tolist() == want[1], step
            assert got.count.item() == want[2] and np.array_equal(got.remap.cpu().numpy(), want[3]), step
            errors = set()
        elif kind == 3:
            k = max(1, rows // 3)
            parents, children = pick(k), pick(k)
            if step % 2:
                parents[0], children[-1] = -1, children[0]
            errors = books.fork(parents, children)
            pool.fork(dev(parents), dev(children))
        else:
            k = int(rng.integers(1, rows + 1))
            which = pick(k)
            most = entries * bs
            new = [int(books.lens[r]) + int(rng.integers(1, 2 * bs)) if rng.random() < 0.5 else
                   int(rng.integers(0, most + 1)) if rng.random() < 0.3 else int(books.lens[r]) // 2 for r in which]
            new = [min(n, most) for n in new]
            if step % 3 == 0 and k > 2:
                which[1], new[2], which[-1] = rows, most + 1, which[0]
            src, dst, errors = books.resize(which, new)
            got = pool.resize(dev(which), dev(new))
            assert got[0].tolist() == src and got[1].tolist() == dst, step
        same(pool, books, f"step {step} kind {kind}")
        assert pool.get_error() == worst(errors), (step, kind, errors)


@pytest.mark.gpu
def test_out_of_pages_leaves_the_requests_behind_it(PG):
    books = Books(6, 10, 8, 16)
    pool = pool_of(PG, books)
    for rows, new in (([0, 1, 2, 3], [40, 33, 90, 1]), ([0, 4, 5], [0, 30, 65]), ([5, 4, 0], [160, 10, 16])):
        src, dst, errors = books.resize(rows, new)
        got = pool.resize(dev(rows), dev(new))
        assert (got[0].tolist(), got[1].tolist()) == (src, dst)
        same(pool, books)
        assert pool.get_error() == worst(errors)


@pytest.mark.gpu
def test_shared_ragged_page(PG):
    """Holders of one ragged page: some grow, all grow, one truncates while
    another grows, and a row cut back into a page that others hold."""
    for rows, new in (([1, 2], [38, 38]), ([0, 1, 2, 3], [38, 60, 38, 39]), ([3, 0, 2, 1], [38] * 4),
                      ([0, 1], [0, 38]), ([1], [20]), ([1, 1, 0], [38, 39, 40])):
        books = Books(4, 6, 40, 16)
        books.resize([0], [37])
        books.fork([0, 0, 0], [1, 2, 3])
        pool = pool_of(PG, books)
        src, dst, errors = books.resize(rows, new)
        got = pool.resize(dev(rows), dev(new))
        assert (got[0].tolist(), got[1].tolist()) == (src, dst), rows
        same(pool, books, rows)
        if rows == [1]:  # the row now ends inside a page that the others hold in full
            src, dst, errors = books.resize([1], [21])
            assert src == [books.table[0, 1]]
            got = pool.resize(dev([1]), dev([21]))
            assert (got[0].tolist(), got[1].tolist()) == (src, dst)
            same(pool, books)
        assert pool.get_error() == worst(errors)


@pytest.mark.gpu
def test_freed_rows_and_bad_pages(PG):
    books = Books(5, 8, 50, 16)
    books.resize([0, 1, 2], [100, 128, 5])
    books.fork([1], [3])
    pool = pool_of(PG, books)
    pool.free(dev([3, 0, 4]))
    books.resize([3, 0, 4], [0, 0, 0])
    same(pool, books)
    assert pool.get_error() == 0
    # a page index out of range in a row: nothing is dereferenced
    pool.block_table[1, 3] = 1 << 29
    before = pool.block_table.clone(), pool.ref_counts.clone()
    pool.fork(dev([1]), dev([4]))
    assert pool.get_error() == BAD_BLOCK
    assert torch.equal(pool.block_table, before[0]) and torch.equal(pool.ref_counts, before[1])
    assert pool.context_lens.tolist() == [0, 128, 5, 0, 0]
    pool.free(dev([1]))
    assert pool.get_error() == BAD_BLOCK
    assert pool.ref_counts.sum().item() == 2  # row 2's page, and the one row 1 no longer names
    pool.block_table[2, 0] = -7
    pool.resize(dev([2]), dev([6]))
    assert pool.get_error() == BAD_BLOCK
    assert pool.context_lens[2].item() == 5
    pool.compact()
    assert pool.get_error() == BAD_BLOCK


@pytest.mark.gpu
def test_a_page_given_up_twice_is_told(PG):
    """Books that do not add up: the count stays at 0 and the call says so."""
    books = Books(2, 4, 10, 16)
    books.resize([0, 1], [16, 16])
    books.table[1, 0] = books.table[0, 0]
    pool = pool_of(PG, books)
    pool.free(dev([0, 1]))
    assert pool.get_error() == BAD_REQUEST
    assert pool.ref_counts[0].item() == 0 and pool.ref_counts.min().item() == 0


def random_cache(rng, dt, blocks, heads, bs):
    if dt == gen.KV_FP16:
        return rng.integers(0, 1 << 16, (blocks, heads, bs, 128)).astype(np.uint16).view(np.float16)
    return rng.integers(0, 256, (blocks, heads, gen.cache_tile_bytes(dt, bs, 128))).astype(np.uint8)


def as_bytes(t):
    return t.cpu().contiguous().view(torch.uint8).numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("blocks,heads,bs,n", [(9, 1, 16, 1), (64, 2, 16, 30), (400, 3, 48, 200),
                                               (90, 8, 112, 40), (9000, 1, 16, 4500)])
def test_copy(PG, dt, blocks, heads, bs, n):
    rng = np.random.default_rng(n)
    k, v = (random_cache(rng, dt, blocks, heads, bs) for _ in range(2))
    order = rng.permutation(blocks)
    src, dst = order[:n].astype(np.int32), order[n:2 * n].astype(np.int32)
    src[::5] = -1  # fillers
    pool = PG.PagePool(num_seqs=1, num_kv_heads=heads, head_dim=128, block_size=bs,
                       max_blocks_per_seq=1, num_blocks=blocks)
    gk, gv = torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda()
    count = max(1, n - 3)
    for limit in (count, None):
        c = None if limit is None else dev([limit])
        pool.copy(gk, gv, dev(src), dev(dst), kv_dtype=dt, count=c)
        for i in range(n if limit is None else limit):
            if src[i] >= 0:
                k[dst[i]], v[dst[i]] = k[src[i]], v[src[i]]
        assert np.array_equal(as_bytes(gk), np.ascontiguousarray(k).view(np.uint8))
        assert np.array_equal(as_bytes(gv), np.ascontiguousarray(v).view(np.uint8))
    assert pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("many", [0, 3000])
def test_copy_refuses_pairs_that_would_race(PG, many):
    """One target twice (the lowest pair stands), a source that is a target, a
    page onto itself, pages out of range; the rest is carried out."""
    rng = np.random.default_rng(1)
    blocks = 40 + 2 * many
    k = random_cache(rng, gen.KV_FP16, blocks, 1, 16)
    pairs = [(0, 10), (1, 10), (2, 11), (11, 12), (3, 3), (4, 13), (5, blocks), (blocks + 7, 14), (6, -1),
             (-1, 15), (7, 16)]
    pairs += [(40 + i, 40 + many + i) for i in range(many)]
    stand = [(0, 10), (2, 11), (4, 13), (7, 16)] + pairs[11:]
    pool = PG.PagePool(num_seqs=1, num_kv_heads=1, head_dim=128, block_size=16, max_blocks_per_seq=1,
                       num_blocks=blocks)
    gk = torch.from_numpy(k).cuda()
    gv = torch.from_numpy(k.copy()).cuda()
    pool.copy(gk, gv, dev([s for s, _ in pairs]), dev([d for _, d in pairs]), kv_dtype=0)
    assert pool.get_error() == BAD_BLOCK
    want = k.copy()
    for s, d in stand:
        want[d] = k[s]
    assert np.array_equal(as_bytes(gk), want.view(np.uint8))
    assert np.array_equal(as_bytes(gv), want.view(np.uint8))
    pool.copy(gk, gv, dev([1, 2]), dev([20, 20]), kv_dtype=0)
    assert pool.get_error() == BAD_REQUEST
    for count in (-4, 0):
        pool.copy(gk, gv, dev([1, 2]), dev([30, 31]), kv_dtype=0, count=dev([count]))
    want[20] = want[1]
    assert np.array_equal(as_bytes(gk), want.view(np.uint8))


@pytest.mark.gpu
def test_binding_refuses_wrong_tensors(PG):
    pool = PG.PagePool(num_seqs=3, num_kv_heads=1, head_dim=128, block_size=16, max_blocks_per_seq=4,
                       num_blocks=20)
    good = dev([0, 1])
    with pytest.raises(ValueError, match="parents"):
        pool.fork(dev([0]), good)
    with pytest.raises(ValueError, match="rows"):
        pool.resize(good.long(), good)
    with pytest.raises(ValueError, match="new_lens"):
        pool.resize(good, good.cpu())
    with pytest.raises(ValueError, match="contiguous"):
        pool.resize(dev([0, 9, 1, 9])[::2], good)
    from paged_kv_decode_flash_b200 import binding as b
    with pytest.raises(b.PagedAttnError):
        pool.resize(dev([0, 1, 2, 0]), dev([1, 1, 1, 1]))  # more requests than rows
    k = torch.empty(20, 1, 16, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="v_cache"):
        pool.copy(k, k[:19], good, good, kv_dtype=0)
    with pytest.raises(ValueError, match="kv_dtype"):
        pool.copy(k, k, good, good, kv_dtype=9)
    with pytest.raises(ValueError, match="context_lens"):
        PG.PagePool(num_seqs=3, num_kv_heads=1, head_dim=128, block_size=16, max_blocks_per_seq=4,
                    num_blocks=20, context_lens=dev([0, 0]))
    pool.fork(dev([]), dev([]))
    pool.resize(dev([]), dev([]))
    pool.copy(k, k, dev([]), dev([]), kv_dtype=0)
    assert pool.get_error() == 0


@pytest.mark.gpu
def test_capture_and_replay(PG):
    """A captured step (grow, copy) reads its requests and the books at replay."""
    books = Books(4, 20, 60, 16)
    books.resize([0], [37])
    pool = pool_of(PG, books)
    rows, new = dev([1, 0]), dev([1, 38])
    parents, children = dev([0]), dev([1])
    k = torch.randn(60, 2, 16, 128, device="cuda").half()
    v = torch.randn_like(k)
    src, dst = dev([0, 0]), dev([0, 0])
    pool.resize(dev([2]), dev([1]))  # warm: modules loaded before the capture
    books.resize([2], [1])
    pool.copy(k, v, dev([-1]), dev([-1]), kv_dtype=0)
    pool.fork(dev([]), dev([]))
    pool.fork(dev([3]), dev([3]))
    pool.get_error()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.fork(parents, children)
        pool.resize(rows, new, copy_src=src, copy_dst=dst)
        pool.copy(k, v, src, dst, kv_dtype=0)
    for (p, c), r, n in (((0, 1), [1, 0], [38, 39]), ((0, 3), [3, 1], [50, 60])):
        parents.copy_(dev([p]))
        children.copy_(dev([c]))
        rows.copy_(dev(r))
        new.copy_(dev(n))
        g.replay()
        books.fork([p], [c])
        ws, wd, _ = books.resize(r, n)
        assert (src.tolist(), dst.tolist()) == (ws, wd)
        same(pool, books)
        for s, d in zip(ws, wd):
            if s >= 0:
                assert torch.equal(k[s], k[d]) and torch.equal(v[s], v[d])
    assert pool.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_a_prompt_with_several_answers(PG, dt):
    """The calls together, as a serving loop makes them: a prompt is written,
    forked, each answer grows and is written, the batch attends with the
    prompt's pages shared, one answer ends, the pool is closed up, and the
    rest attend again.  Every step's output against the oracle on a host copy
    of the cache that is written token by token."""
    from paged_kv_decode_flash_b200 import binding as B
    from paged_kv_decode_flash_b200.shared_prefix import SharedPrefixDecode
    orc = oracle.load()
    rng = np.random.default_rng(3)
    heads, G, bs, rows, entries, blocks, prompt = 2, 4, 16, 5, 12, 64, 100
    books = Books(rows, entries, blocks, bs)
    pool = pool_of(PG, books, heads)
    dtype, shape = B.cache_shape(dt, blocks, heads, bs, 128)
    k = torch.zeros(shape, dtype=dtype, device="cuda")
    v = torch.zeros_like(k)
    half = lambda *s: rng.standard_normal(s).astype(np.float16)
    history = {r: [] for r in range(rows)}  # per row: (k, v) fp16 rows of its tokens

    def write(which, n):
        """n new tokens into rows `which` (all rows are passed, the others are empty)."""
        w = B.PagedDecode(num_seqs=1, num_q_heads=heads * G, num_kv_heads=heads, head_dim=128,
                          block_size=bs, max_blocks_per_seq=entries, num_blocks=blocks, n_query=n)
        for r in which:
            kn, vn = half(1, n, heads, 128), half(1, n, heads, 128)
            w.cache_write(torch.from_numpy(kn).cuda(), torch.from_numpy(vn).cuda(),
                          pool.block_table[r:r + 1], pool.context_lens[r:r + 1], kv_dtype=dt,
                          k_cache=k, v_cache=v)
            history[r] += [(kn[0, i], vn[0, i]) for i in range(n)]
        assert w.get_error() == 0

    def grow(which, n):
        new = [len(history[r]) + n for r in which]
        src, dst = pool.resize(dev(which), dev(new))
        pool.copy(k, v, src, dst, kv_dtype=dt)
        write(which, n)

    def one_row(case, s, n):
        """Row s alone, with its n tokens as the new ones."""
        return dataclasses.replace(case, num_seqs=1, n_query=n,
                                   q=np.zeros((1, n, heads * G, 128), np.float16),
                                   block_table=case.block_table[s:s + 1],
                                   context_lens=case.context_lens[s:s + 1])

    def attend(which, n, prefix):
        q = half(len(which), n, heads * G, 128)
        dec = SharedPrefixDecode(num_seqs=len(which), num_q_heads=heads * G, num_kv_heads=heads,
                                 head_dim=128, block_size=bs, max_blocks_per_seq=entries,
                                 num_blocks=blocks, n_query=n, prefix_blocks=entries)
        out = dec(torch.from_numpy(q).cuda(), k, v, pool.block_table[which], pool.context_lens[which],
                  pool.block_table[which[0]], dev([prefix]), causal=1, window=0, scale=128 ** -0.5,
                  kv_dtype=dt)
        assert dec.get_error() == 0
        # the oracle on a cache of its own: row after row, unshared
        most = max(len(history[r]) for r in which)
        case = gen.make_case(context_lens=tuple(len(history[r]) for r in which), n_query=n,
                             num_q_heads=heads * G, num_kv_heads=heads, kv_dtype=dt, poison=False,
                             max_blocks_per_seq=-(-most // bs))
        case.q = q
        for s, r in enumerate(which):
            case.k_cache, case.v_cache, rc = orc.cache_write(
                one_row(case, s, len(history[r])), np.stack([a for a, _ in history[r]])[None],
                np.stack([b for _, b in history[r]])[None])
            assert rc == 0
        ref, _ = orc.attend(case)
        assert_parity(out.cpu().numpy(), ref, f"rows {which}")

    for _ in range(prompt // 10):
        grow([0], 10)
    pool.fork(dev([0] * 4), dev([1, 2, 3, 4]))
    for r in range(1, rows):
        history[r] = list(history[0])
    everyone = [0, 1, 2, 3, 4]
    attend(everyone, 1, 96)
    for n in (1, 3):
        grow(everyone, n)
        attend(everyone, n, 96)
    pool.free(dev([0, 3]))
    history[0], history[3] = [], []
    rest = [1, 2, 4]
    live = int((pool.ref_counts > 0).sum())
    moved = pool.compact()
    pool.copy(k, v, moved.src, moved.dst, kv_dtype=dt, count=moved.count)
    assert int((pool.ref_counts[:live] > 0).sum()) == live
    attend(rest, 3, 96)
    grow(rest, 8)
    attend(rest, 8, 96)
    assert pool.get_error() == 0
