"""Shared-prefix decode and page operations where their work is cut otherwise:
more sequences than a CTA has threads, row parts, references that rise all the
way, caches past 32-bit offsets, workspaces that two graphs share.

Tolerance: as in test_shared_prefix.py (tests/parity.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
import pins
import test_pages as TP
import test_shared_prefix as TS
from paged_kv_decode_flash_b200 import inputs as gen

DTYPES = TS.DTYPES
PREFIX = 3024


@pytest.fixture(scope="module")
def orc():
    return oracle.load()


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding, build, shared_prefix
    build.build()  # no-op when the in-tree library is up to date
    binding.lib()
    return shared_prefix


def test_a_plan_never_outgrows_the_workspace():
    """The workspace of any cache type holds what the largest grid writes; more
    sequences, tokens and query heads only ever need more."""
    import ctypes
    from paged_kv_decode_flash_b200 import binding as b, build
    build.build()
    L = b.lib()

    def size(seqs, hq, hkv, nq):
        d = b.Dims(seqs, hq, hkv, 128, 16, 40, 1000, None, 0)
        return L.paged_attn_shared_workspace_size(ctypes.byref(d), nq, 16)

    for hkv, g in ((1, 1), (2, 3), (8, 4), (8, 8)):
        last = 0
        for seqs, nq in ((1, 1), (2, 1), (16, 1), (16, 8), (64, 8), (300, 8), (1000, 12)):
            n = size(seqs, g * hkv, hkv, nq)
            # a partial for every row at least, and one of 128 rows for every CTA
            assert n >= 516 * (seqs * nq * g * hkv + 148 * min(128, seqs * nq * g)), (hkv, g, seqs, nq)
            assert n > last
            last = n


def test_lengths_at_the_end_of_the_int_range_are_refused():
    import ctypes
    from paged_kv_decode_flash_b200 import binding as b, build
    build.build()
    for entries, blocks, ok in (((1 << 31) // 16 - 17, 4, True), ((1 << 31) // 16 - 1, 4, False),
                                (4, (1 << 31) // 16 - 17, True), (4, (1 << 31) // 16 - 1, False)):
        d = b.Dims(1, 8, 2, 128, 16, entries, 1000, None, 0)
        assert (b.lib().paged_attn_shared_workspace_size(ctypes.byref(d), 1, blocks) > 0) == ok


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("nseq,prefix", [(385, 320), (641, 0), (1500, 96)])
def test_more_sequences_than_threads(S, orc, dt, nseq, prefix):
    """Some have no keys of their own, some many; a bad length in each third."""
    own = [(s * 7) % 60 + 1 if s % 5 else 0 for s in range(nseq)]
    if prefix == 0:
        own = [max(1, n) for n in own]
    own[nseq - 2] = 700
    case = TS.shared_case(prefix, own, num_q_heads=4, num_kv_heads=2, kv_dtype=dt)
    ref, _ = orc.attend(case)
    dec, args, kw = TS.prepared(S, case, prefix)
    out = dec(*args, **kw)
    assert dec.get_error() == 0
    assert_parity(out.cpu().numpy(), ref, "all")
    bad = [3, nseq // 2, nseq - 1]
    args[4][bad] = -1
    out = dec(*args, **kw).cpu().numpy()
    assert dec.get_error() == -6
    assert not out[bad].any()
    good = [s for s in range(nseq) if s not in bad]
    assert_parity(out[good], ref[good], "the others")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("nq,G,own", [(33, 4, (40, 300, 33)), (100, 3, (100, 129)), (128, 8, (130,)),
                                      (128, 1, (500, 128))])
def test_sequences_with_many_rows(S, orc, dt, nq, G, own):
    """More than 128 rows of a sequence on a KV head: several row parts."""
    case = TS.shared_case(480, own, seed=nq, n_query=nq, num_q_heads=2 * G, num_kv_heads=2, kv_dtype=dt,
                          block_size=48)
    TS.check(S, orc, case, 480, "row parts")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("nseq,G,prefix", [(32, 4, 16), (64, 4, 144), (67, 5, 272), (40, 4, 1040)])
def test_short_prefixes_under_many_sequences(S, orc, dt, nseq, G, prefix):
    """The starts of segments are most of the work: row tiles of 128 and 256
    rows (a last one of 79), one to nine tiles of the prefix."""
    own = [1 + (s * 37) % 150 for s in range(nseq)]
    case = TS.shared_case(prefix, own, seed=nseq, num_q_heads=8 * G, num_kv_heads=8, kv_dtype=dt)
    TS.check(S, orc, case, prefix, "short prefix")


def ramp(case, prefix, top):
    """Keys that grow along the prefix: every later tile has larger scores.
    Values above 0.5: with scores up to 1400 (log2 units) their fp32 sums are
    good to 1400 * 2^-22 = 3e-4, which an output near 0 would show beside a
    tolerance of 1e-5 and one above 0.5 does not beside 5e-3."""
    case.q[:] = np.abs(case.q) + np.float16(0.25)
    case.v_cache[:] = np.abs(case.v_cache) + np.float16(0.5)
    f = np.linspace(0.05, top, prefix, dtype=np.float32)
    for j in range(prefix):
        b, slot = case.block_table[0, j // case.block_size], j % case.block_size
        case.k_cache[b, :, slot, :] = (np.abs(case.k_cache[b, :, slot, :].astype(np.float32)) * f[j]).astype(np.float16)
    return case


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("own", [(9, 40), (5,) * 30])
@pytest.mark.parametrize("top", [0.3, 3.0, 100.0])
def test_references_that_rise_all_the_way(S, orc, dt, own, top):
    """Scores that rise along the prefix by 0.1, 0.9 and 28 (log2 units) a step
    of 64 keys: the last by more than fp16's range within a step."""
    case = TS.shared_case(PREFIX, own, seed=3, n_query=2, num_q_heads=16, num_kv_heads=2)
    ramp(case, PREFIX, top)
    if dt != gen.KV_FP16:
        k, v = case.k_cache.astype(np.float32), case.v_cache.astype(np.float32)
        bs = case.block_size

        def packed(x):
            blocks, heads = x.shape[:2]
            x = np.where(np.isnan(x), 0, x)
            if dt == gen.KV_Q8_0:
                g = x.reshape(blocks, heads, bs, 4, 32)
                d = (np.abs(g).max(-1) / 127).astype(np.float16)
                q = np.round(g / np.maximum(d.astype(np.float32), 1e-30)[..., None])
            else:
                d = (np.abs(x).max(-1) / 127).astype(np.float32)
                q = np.round(x / np.maximum(d, 1e-30)[..., None])
            q = np.clip(q, -127, 127).astype(np.int8).reshape(blocks, heads, -1).view(np.uint8)
            return np.concatenate([q, np.ascontiguousarray(d).reshape(blocks, heads, -1).view(np.uint8)], -1)

        case.k_cache, case.v_cache, case.kv_dtype = packed(k), packed(v), dt
    ref, _ = orc.attend(pins.zero_nans(case))
    assert_parity(TS.run(S, case, PREFIX), ref, "rising")


def poison_key(case, seq, key, head):
    """NaN in the key (not the value) of one position of one KV head."""
    block, slot = case.block_table[seq, key // case.block_size], key % case.block_size
    if case.kv_dtype == gen.KV_FP16:
        case.k_cache[block, head, slot, :] = np.float16(np.nan)
    else:
        width = 8 if case.kv_dtype == gen.KV_Q8_0 else 4
        nan = np.full(4, np.nan, np.float16) if width == 8 else np.full(1, np.nan, np.float32)
        at = case.block_size * 128 + slot * width
        case.k_cache[block, head, at: at + width] = nan.view(np.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("G,own", [(4, (5, 40, 9)), (8, (7,) * 20)])
def test_scores_that_are_not_finite_show(S, orc, dt, G, own):
    """A row that sees a NaN key, or whose query holds one, is NaN, as the
    formula has it, and no other row is touched."""
    prefix, nq = 640, 3
    case = TS.shared_case(prefix, own, n_query=nq, num_q_heads=2 * G, num_kv_heads=2, kv_dtype=dt)
    ref, _ = orc.attend(case)
    ref = np.asarray(ref)
    dec, args, kw = TS.prepared(S, case, prefix)
    shape = dec(*args, **kw).shape
    assert shape == ref.shape == (len(own), nq, 2 * G, 128)

    def check(nan, what):
        out = TS.run(S, case, prefix)
        assert np.isnan(out[nan]).all(), what
        assert_parity(out[~nan], ref[~nan], what)

    nan = np.zeros((len(own), nq, 2 * G), bool)
    L = prefix + own[1]
    poison_key(case, 1, L - 2, 0)  # seen by the last two of sequence 1's new tokens
    nan[1, 1:, :G] = True
    check(nan, "own key")
    case.q[0, 0, 2 * G - 1, 5] = np.float16(np.nan)
    nan[0, 0, 2 * G - 1] = True
    check(nan, "query")
    case.q[2, 2, 0, :] = np.float16(np.inf)
    nan[2, 2, 0] = True
    check(nan, "infinite query")
    poison_key(case, 0, 70, 1)  # seen by every row of its KV head
    nan[:, :, G:] = True
    check(nan, "prefix key")


@pytest.mark.gpu
def test_row_scales_of_every_size(S, orc):
    """int8 rows whose scales lie 80 powers of two apart, key by key: V's are
    folded into the weights, whose fp16 range they must not leave."""
    case = TS.shared_case(1024, (20, 300, 7), n_query=2, num_q_heads=8, num_kv_heads=2,
                          kv_dtype=gen.KV_INT8_ROW)
    bs = case.block_size
    rng = np.random.default_rng(4)
    for cache, spread in ((case.v_cache, 40), (case.k_cache, 2)):
        sc = cache[:, :, bs * 128:].copy().view(np.float32)
        sc *= np.exp2(rng.integers(-spread, 1, sc.shape)).astype(np.float32)
        sc[rng.random(sc.shape) < 0.1] = 0
        sc[rng.random(sc.shape) < 0.1] *= -1
        cache[:, :, bs * 128:] = sc.view(np.uint8).reshape(cache[:, :, bs * 128:].shape)
    ref, _ = orc.attend(pins.zero_nans(case))
    assert_parity(TS.run(S, case, 1024), ref, "scales")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_caches_past_32_bit_offsets(S, dt):
    """The pages at the end of a cache of more than 4 GB give the bits that the
    same pages give in a small one."""
    from paged_kv_decode_flash_b200 import binding as B, pages
    small = TS.shared_case(512, (70, 9, 33), n_query=2, num_q_heads=8, num_kv_heads=2, kv_dtype=dt, poison=False)
    dec, args, kw = TS.prepared(S, small, 512)
    want = dec(*args, **kw)
    used = small.num_blocks
    tile = {gen.KV_FP16: 4096, gen.KV_Q8_0: 2176, gen.KV_INT8_ROW: 2112}[dt]
    blocks = (1 << 32) // (2 * tile) + used + 40
    dtype, shape = B.cache_shape(dt, blocks, 2, 16, 128)
    k, v = (torch.zeros(shape, dtype=dtype, device="cuda") for _ in range(2))
    shift = blocks - used
    k[shift:], v[shift:] = args[1], args[2]
    far = S.SharedPrefixDecode(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
                               max_blocks_per_seq=small.max_blocks_per_seq, num_blocks=blocks, n_query=2,
                               prefix_blocks=32)
    table = torch.from_numpy(small.block_table).cuda() + shift
    got = far(args[0], k, v, table, args[4], args[5][:32] + shift, args[6], **kw)
    assert far.get_error() == 0
    assert torch.equal(got, want)
    pool = pages.PagePool(num_seqs=1, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=1,
                          num_blocks=blocks)
    n = min(used, shift)
    pool.copy(k, v, torch.arange(shift, shift + n, dtype=torch.int32, device="cuda"),
              torch.arange(n, dtype=torch.int32, device="cuda"), kv_dtype=dt)
    assert pool.get_error() == 0
    assert torch.equal(k[:n], args[1][:n]) and torch.equal(v[:n], args[2][:n])
    assert torch.equal(k[shift:], args[1])


@pytest.mark.gpu
def test_two_graphs_share_a_workspace(S, orc):
    """Captured one after the other, replayed in turn; an eager call between."""
    one = TS.shared_case(1024, (40, 90, 20), n_query=2, num_q_heads=8, num_kv_heads=2)
    two = TS.shared_case(2048, (7, 300, 2), seed=9, n_query=2, num_q_heads=8, num_kv_heads=2,
                         max_blocks_per_seq=one.max_blocks_per_seq + 100)
    from paged_kv_decode_flash_b200 import binding as B
    dims = dict(num_seqs=3, num_q_heads=8, num_kv_heads=2, head_dim=128, block_size=16, n_query=2)
    a = S.SharedPrefixDecode(max_blocks_per_seq=one.max_blocks_per_seq, num_blocks=one.num_blocks,
                             prefix_blocks=64, **dims)
    need = S.SharedPrefixDecode(max_blocks_per_seq=two.max_blocks_per_seq, num_blocks=two.num_blocks,
                                prefix_blocks=128, **dims)
    ws = torch.empty(max(a.workspace_bytes, need.workspace_bytes), dtype=torch.uint8, device="cuda")
    decs, graphs, outs, refs = [], [], [], []
    for case, prefix in ((one, 1024), (two, 2048)):
        dec = S.SharedPrefixDecode(max_blocks_per_seq=case.max_blocks_per_seq, num_blocks=case.num_blocks,
                                   prefix_blocks=prefix // 16, workspace=ws, **dims)
        _, args, kw = TS.prepared(S, case, prefix, dec=dec)
        out = torch.empty_like(args[0])
        dec(*args, **kw, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dec(*args, **kw, out=out)
        decs.append((dec, args, kw))
        graphs.append(g)
        outs.append(out)
        refs.append(orc.attend(case)[0])
    for turn in range(4):
        for g, out, ref in zip(graphs, outs, refs):
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert_parity(out.cpu().numpy(), ref, f"replay {turn}")
        dec, args, kw = decs[turn % 2]
        assert_parity(dec(*args, **kw).cpu().numpy(), refs[turn % 2], "between")
    assert all(d.get_error() == 0 for d, _, _ in decs)


@pytest.mark.gpu
@pytest.mark.parametrize("seed,rows,entries,blocks,bs", [(21, 30, 40, 40000, 16), (22, 1200, 5, 33000, 16),
                                                         (23, 1024, 6, 32768, 16), (24, 1025, 4, 5000, 32)])
def test_random_walk_on_large_pools(seed, rows, entries, blocks, bs):
    """On both sides of the sizes up to which one plan is made by every CTA."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import pages
    TP.test_random_walk(pages, seed, rows, entries, blocks, bs)


@pytest.mark.gpu
@pytest.mark.parametrize("blocks", [600, 40000])
def test_a_long_row_is_grown_and_given_up(blocks):
    """Hundreds of pages in one request, shared by a fork, given up by both."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import pages
    books = TP.Books(4, 520, blocks, 16)
    pool = TP.pool_of(pages, books)
    dev = TP.dev
    for rows, new in (([2], [520 * 16 - 5]), ([0, 3], [900, 17])):
        src, dst, errors = books.resize(rows, new)
        got = pool.resize(dev(rows), dev(new))
        assert (got[0].tolist(), got[1].tolist()) == (src, dst)
        TP.same(pool, books)
        assert pool.get_error() == TP.worst(errors) == 0
    books.fork([2], [1])
    pool.fork(dev([2]), dev([1]))
    for rows, new in (([1], [400 * 16 + 1]), ([2, 1], [3, 0]), ([2, 0, 3], [0, 0, 0])):
        src, dst, errors = books.resize(rows, new)
        got = pool.resize(dev(rows), dev(new))
        assert (got[0].tolist(), got[1].tolist()) == (src, dst)
        TP.same(pool, books)
        assert pool.get_error() == TP.worst(errors) == 0
    assert not books.refs.any()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2047, 2048, 2049])
def test_copies_on_both_sides_of_the_self_check(n):
    """Pairs that clash at the ends of lists that the copy kernel looks over
    itself, and of longer ones."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import pages
    blocks = 2 * n + 8
    rng = np.random.default_rng(n)
    k = rng.integers(0, 256, (blocks, 1, 16 * 132), dtype=np.uint8)
    order = rng.permutation(blocks).astype(np.int32)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    dst[-1] = dst[0]           # the lowest stands
    src[-2] = dst[5]           # a source that is a target
    src[1] = -1
    pool = pages.PagePool(num_seqs=1, num_kv_heads=1, head_dim=128, block_size=16, max_blocks_per_seq=1,
                          num_blocks=blocks)
    gk, gv = torch.from_numpy(k).cuda(), torch.from_numpy(k[::-1].copy()).cuda()
    pool.copy(gk, gv, TP.dev(src), TP.dev(dst), kv_dtype=gen.KV_INT8_ROW)
    assert pool.get_error() == TP.BAD_REQUEST
    wk, wv = k.copy(), k[::-1].copy()
    for i in range(n - 2):
        if src[i] >= 0:
            wk[dst[i]], wv[dst[i]] = k[src[i]], k[::-1][src[i]]
    assert np.array_equal(gk.cpu().numpy(), wk) and np.array_equal(gv.cpu().numpy(), wv)
