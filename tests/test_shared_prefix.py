"""Shared-prefix decode (paged_attn_decode_shared) against the fp64 oracle.

The oracle computes ordinary decode attention over tables whose rows begin
with the same blocks; the call under test gets tables whose entries for the
prefix are out of range (they must not be read) and the prefix's blocks apart.

Tolerance: tests/parity.py (max-abs 2e-3 and max-rel 1e-2 against
max(|oracle|, 1e-3)).  What the arithmetic may lose: q, K and V enter exactly
or to 2^-21, weights to 2^-21, fp32 sums over L keys of relative error below
L * 2^-24 / 2 (random signs: sqrt(L) * 2^-24), each join weight 2^-22, and the
fp16 output half a step, 2^-11 relative and 2^-25 absolute: together below
1e-3 relative to the largest |v| that matters and below 1e-5 absolute on
outputs near zero at the sizes used here.
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
from paged_kv_decode_flash_b200 import inputs as gen

DTYPES = (gen.KV_FP16, gen.KV_Q8_0, gen.KV_INT8_ROW)
NOT_READ = 1 << 30  # a block index no pool has


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
    d = dict(num_seqs=4, num_q_heads=32, num_kv_heads=8, head_dim=128, block_size=16,
             max_blocks_per_seq=300, num_blocks=1000, workspace=None, workspace_bytes=0)
    d.update(kw)
    return Dims(**d)


def test_workspace_size(L):
    size = lambda d, nq, pb: L.paged_attn_shared_workspace_size(ctypes.byref(d), nq, pb)
    n = size(dims(), 1, 256)
    assert n > L.paged_attn_workspace_size(ctypes.byref(dims()), 1)
    assert n % 256 == 0
    assert size(dims(), 8, 256) >= n
    assert size(dims(), 1, 1) > 0
    for bad in (dims(num_q_heads=30), dims(block_size=8), dims(head_dim=64), dims(num_seqs=0)):
        assert size(bad, 1, 256) == 0
    assert size(dims(), 0, 256) == 0
    assert size(dims(), 129, 256) == 0
    assert size(dims(), 1, 0) == 0
    assert size(dims(), 1, -5) == 0
    assert size(dims(), 1, (1 << 31) // 16) == 0  # more than 2^31 - 1 keys
    assert L.paged_attn_shared_workspace_size(None, 1, 4) == 0


def test_refusals_on_the_host(L):
    from paged_kv_decode_flash_b200 import binding as b
    d = dims(workspace=4096, workspace_bytes=1 << 34)
    p = ctypes.c_void_p(1 << 20)  # never dereferenced: checks fail first

    def call(dd, **kw):
        a = dict(dict(q=p, k=p, v=p, bt=p, cl=p, pt=p, pl=p, pb=64, nq=1, causal=1, window=0,
                      scale=0.088, dt=0, out=p), **kw)
        return L.paged_attn_decode_shared(
            ctypes.byref(dd) if dd is not None else None, a["q"], a["k"], a["v"], a["bt"], a["cl"],
            a["pt"], a["pl"], a["pb"], a["nq"], a["causal"], a["window"], a["scale"], a["dt"],
            a["out"], None)

    assert call(None) == b.PA_ERR_INVALID_ARG
    for name in ("q", "k", "v", "bt", "cl", "pt", "pl", "out"):
        assert call(d, **{name: None}) == b.PA_ERR_INVALID_ARG, name
    odd = ctypes.c_void_p((1 << 20) + 2)
    for name in ("q", "k", "v", "bt", "cl", "pt", "pl", "out"):
        assert call(d, **{name: odd}) == b.PA_ERR_INVALID_ARG, name
    assert call(d, pb=0) == b.PA_ERR_INVALID_ARG
    assert call(d, pb=-1) == b.PA_ERR_INVALID_ARG
    assert call(d, pb=(1 << 31) // 16) == b.PA_ERR_UNSUPPORTED
    assert call(d, nq=0) == b.PA_ERR_INVALID_ARG
    assert call(d, nq=129) == b.PA_ERR_INVALID_ARG
    assert call(d, causal=2) == b.PA_ERR_INVALID_ARG
    assert call(d, window=-1) == b.PA_ERR_INVALID_ARG
    assert call(d, dt=3) == b.PA_ERR_INVALID_ARG
    assert call(d, scale=float("inf")) == b.PA_ERR_INVALID_ARG
    assert call(dims(head_dim=64, workspace=4096, workspace_bytes=1 << 34)) == b.PA_ERR_UNSUPPORTED
    assert call(dims(workspace=None)) == b.PA_ERR_WORKSPACE
    assert call(dims(workspace=4100, workspace_bytes=1 << 34)) == b.PA_ERR_WORKSPACE


def test_binding_refuses_wrong_prefix_tensors():
    from paged_kv_decode_flash_b200 import binding as b
    from paged_kv_decode_flash_b200.shared_prefix import SharedPrefixDecode
    dec = object.__new__(SharedPrefixDecode)  # no device: the checks only
    dec.n_query, dec.prefix_blocks = 1, 7
    dec.dims = b.Dims(2, 16, 4, 128, 16, 10, 25, None, 0)
    dec.workspace = torch.empty(1024, dtype=torch.uint8)
    i32 = torch.int32
    table, n = torch.empty(7, dtype=i32), torch.empty(1, dtype=i32)
    dec.check_shared(table, n)
    for bad in (torch.empty(6, dtype=i32), torch.empty(7, dtype=torch.int64), torch.empty(1, 7, dtype=i32)):
        with pytest.raises(ValueError, match="prefix_table"):
            dec.check_shared(bad, n)
    for bad in (torch.empty(2, dtype=i32), torch.empty(1, dtype=torch.int64), torch.empty((), dtype=i32)):
        with pytest.raises(ValueError, match="prefix_len"):
            dec.check_shared(table, bad)
    with pytest.raises(TypeError):
        dec.check_shared(None, n)


# ---------------------------------------------------------------------------
# on the GPU
# ---------------------------------------------------------------------------
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


def shared_case(prefix, own, *, seed=0, **kw):
    """A case whose rows begin with the same prefix / block_size blocks."""
    case = gen.make_case(seed=seed, context_lens=tuple(prefix + n for n in own), **kw)
    nb = prefix // case.block_size
    case.block_table[1:, :nb] = case.block_table[0, :nb]
    return case


def poison(case, block, slot):
    """NaN in one key and value of every KV head."""
    for c in (case.k_cache, case.v_cache):
        if case.kv_dtype == gen.KV_FP16:
            c[block, :, slot, :] = np.float16(np.nan)
        else:
            values = case.block_size * 128
            width = 8 if case.kv_dtype == gen.KV_Q8_0 else 4
            nan = np.full(4, np.nan, np.float16) if width == 8 else np.full(1, np.nan, np.float32)
            c[block, :, values + slot * width: values + (slot + 1) * width] = nan.view(np.uint8)


def prepared(S, case, prefix, extra_blocks=0, dec=None):
    """(decoder, tensors, keywords); the tables' entries of the prefix are out
    of range, and so are the prefix table's entries behind it."""
    nb = prefix // case.block_size
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    table = case.block_table.copy()
    table[:, :nb] = NOT_READ
    ptable = np.full(max(1, nb + extra_blocks), NOT_READ, dtype=np.int32)
    ptable[:nb] = case.block_table[0, :nb]
    if dec is None:
        dec = S.SharedPrefixDecode(
            num_seqs=case.num_seqs, num_q_heads=case.num_q_heads, num_kv_heads=case.num_kv_heads,
            head_dim=128, block_size=case.block_size, max_blocks_per_seq=case.max_blocks_per_seq,
            num_blocks=case.num_blocks, n_query=case.n_query, prefix_blocks=len(ptable))
    args = [t(case.q), t(case.k_cache), t(case.v_cache), t(table), t(case.context_lens), t(ptable),
            torch.tensor([prefix], dtype=torch.int32, device="cuda")]
    kw = dict(causal=case.causal, window=case.window, scale=case.scale, kv_dtype=case.kv_dtype)
    return dec, args, kw


def run(S, case, prefix, **kw):
    dec, args, k = prepared(S, case, prefix, **kw)
    out = dec(*args, **k)
    torch.cuda.synchronize()
    assert dec.get_error() == 0
    return out.cpu().numpy()


def check(S, orc, case, prefix, what, **kw):
    ref, _ = orc.attend(case)
    assert_parity(run(S, case, prefix, **kw), ref, what)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("prefix,own,nq,G,Hkv,bs", [
    (1024, (5, 40, 1, 17), 1, 4, 8, 16),       # four answers, one token each
    (16, (1,), 1, 1, 1, 16),                   # one sequence, one block, one row
    (48, (3, 100), 3, 2, 2, 48),               # odd page size
    (1120, (9, 30, 300), 4, 6, 4, 112),        # 24 rows a sequence, pages that end inside a tile
    (2000, (130, 8, 64, 11, 9), 8, 4, 2, 16),  # ragged last tile, 160 rows
    (640, (20,) * 16, 1, 8, 1, 32),            # 128 rows
    (640, (20,) * 43, 1, 3, 2, 32),            # 129 rows
    (384, (6,) * 37, 5, 7, 1, 64),             # 1295 rows
    (5008, (700, 2), 2, 1, 3, 16),             # 4 rows
])
def test_shapes(S, orc, dt, prefix, own, nq, G, Hkv, bs):
    case = shared_case(prefix, [max(n, nq) for n in own], seed=prefix + nq, n_query=nq,
                       num_q_heads=G * Hkv, num_kv_heads=Hkv, block_size=bs, kv_dtype=dt,
                       spike_frac=0.01, spike_gain=4.0, spare_blocks=2)
    check(S, orc, case, prefix, "shapes", extra_blocks=3)


def _sweep():
    rng = np.random.default_rng(77)
    for t in range(36):
        nq = int(rng.choice([1, 2, 3, 4, 8, 12]))
        G = int(rng.choice([1, 2, 4, 6, 8]))
        Hkv = int(rng.choice([1, 2, 4]))
        bs = int(16 * rng.choice([1, 2, 3, 7]))
        nseq = int(rng.choice([1, 2, 5, 9, 33]))
        prefix = bs * int(rng.integers(0, 2500 // bs))
        own = [int(x) for x in rng.integers(nq, nq + int(rng.choice([2, 60, 400])), size=nseq)]
        yield dict(prefix=prefix, own=own, nq=nq, G=G, Hkv=Hkv, bs=bs, dt=DTYPES[t % 3],
                   causal=int(rng.integers(0, 2)), window=int(rng.choice([0, 0, 1, 90, 700])), seed=t)


@pytest.mark.gpu
@pytest.mark.parametrize("c", list(_sweep()), ids=lambda c: f"P{c['prefix']}_B{len(c['own'])}_nq{c['nq']}_G{c['G']}_w{c['window']}_dt{c['dt']}")
def test_sweep(S, orc, c):
    case = shared_case(c["prefix"], c["own"], seed=c["seed"], n_query=c["nq"],
                       num_q_heads=c["G"] * c["Hkv"], num_kv_heads=c["Hkv"], block_size=c["bs"],
                       kv_dtype=c["dt"], causal=c["causal"], window=c["window"])
    check(S, orc, case, c["prefix"], "sweep")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_long_prefix_with_spikes(S, orc, dt):
    """Many key tiles per CTA, references raised after the first tile."""
    case = shared_case(40000, (50, 3, 200, 77, 12, 31), seed=5, n_query=4, num_q_heads=12,
                       num_kv_heads=2, kv_dtype=dt, spike_frac=0.002, spike_gain=8.0)
    check(S, orc, case, 40000, "long")


@pytest.mark.gpu
@pytest.mark.parametrize("nseq", [3, 24])
@pytest.mark.parametrize("dt", DTYPES)
def test_no_prefix_and_nothing_but_prefix(S, orc, dt, nseq):
    """P = 0 is a plain decode; P = L leaves a sequence no keys of its own
    (its new tokens lie inside the prefix)."""
    case = shared_case(0, [20 + 3 * s for s in range(nseq)], n_query=2, num_q_heads=4,
                       num_kv_heads=1, kv_dtype=dt)
    check(S, orc, case, 0, "no prefix", extra_blocks=4)
    case = shared_case(320, [0] * nseq, n_query=2, num_q_heads=4, num_kv_heads=1, kv_dtype=dt)
    check(S, orc, case, 320, "only prefix")
    case = shared_case(320, [s % 4 for s in range(nseq)], n_query=8, num_q_heads=8, num_kv_heads=2,
                       kv_dtype=dt)
    check(S, orc, case, 320, "new tokens in the prefix")


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("window", [3, 130, 500])
def test_window_reaches_into_the_prefix(S, orc, dt, causal, window):
    """Keys that no row sees are NaN, key by key; some sequences see none of
    the prefix, some part of it."""
    own = [4, 100, 300, 700, 9]
    case = shared_case(960, own, seed=window, n_query=4, num_q_heads=8, num_kv_heads=2,
                       causal=causal, window=window, kv_dtype=dt, block_size=48)
    first = [960 + n - (4 if causal else 1) - window + 1 for n in own]
    for j in range(min(960, max(0, min(first)))):
        poison(case, case.block_table[0, j // 48], j % 48)
    out = run(S, case, 960)
    import pins
    ref, _ = orc.attend(pins.zero_nans(case))
    assert_parity(out, ref, "window")


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.07, 0.0])
def test_negative_and_zero_scale(S, orc, scale):
    case = shared_case(500 * 16, (9, 30), n_query=2, num_q_heads=8, num_kv_heads=2, scale=scale)
    check(S, orc, case, 500 * 16, "scale")


@pytest.mark.gpu
def test_more_sequences_than_one_queue_launch(S, orc):
    case = shared_case(256, [1 + s % 40 for s in range(300)], num_q_heads=4, num_kv_heads=1)
    check(S, orc, case, 256, "300 sequences")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_repeats_are_bit_identical_and_sequences_independent(S, dt):
    case = shared_case(4096, [10, 300, 77, 5, 50], n_query=3, num_q_heads=16, num_kv_heads=4,
                       kv_dtype=dt)
    dec, args, kw = prepared(S, case, 4096)
    a = dec(*args, **kw).clone()
    for _ in range(3):
        assert torch.equal(a, dec(*args, **kw))
    args[0] = args[0].clone()
    args[0][1:] = torch.randn_like(args[0][1:])  # the others' queries
    assert torch.equal(a[0], dec(*args, **kw)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("P", [7, -16, 16 * 21])
def test_bad_prefix_length(S, dt, P):
    """Not whole blocks, negative, more than the prefix table: rows of 0."""
    case = shared_case(320, [30, 60], kv_dtype=dt)
    dec, args, kw = prepared(S, case, 320)
    args[6].fill_(P)
    out = dec(*args, **kw)
    assert dec.get_error() == -6
    assert not out.any()
    args[6].fill_(320)
    dec(*args, **kw)
    assert dec.get_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("bad", [0, 100, 319, 1 << 20, -3])
def test_sequence_shorter_than_the_prefix(S, orc, dt, bad):
    """That sequence's rows are 0, the others as ever."""
    case = shared_case(320, [30, 60, 9], kv_dtype=dt)
    ref, _ = orc.attend(case)
    dec, args, kw = prepared(S, case, 320)
    args[4][1] = bad
    out = dec(*args, **kw).cpu().numpy()
    assert dec.get_error() == -6
    assert not out[1].any()
    assert_parity(out[[0, 2]], ref[[0, 2]], "the others")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("index", [-1, 1 << 29])
def test_bad_blocks(S, orc, dt, index):
    """A bad block of the prefix zeroes the rows that see it, a bad block of a
    sequence that sequence's rows; nothing is dereferenced."""
    case = shared_case(640, [30, 400, 9], kv_dtype=dt, window=300)
    ref, _ = orc.attend(case)
    dec, args, kw = prepared(S, case, 640)
    good = args[5].clone()
    args[5][25] = index  # keys 400..415: sequence 0 sees from 370 on, 2 from 349, 1 none
    out = dec(*args, **kw).cpu().numpy()
    assert dec.get_error() == -5
    assert not out[0].any() and not out[2].any()
    assert_parity(out[1], ref[1], "the row that does not see it")
    args[5].copy_(good)
    args[3][2, 40] = index
    out = dec(*args, **kw).cpu().numpy()
    assert dec.get_error() == -5
    assert not out[2].any()
    assert_parity(out[:2], ref[:2], "the others")
    out = dec(*args[:3], torch.from_numpy(case.block_table).cuda(), *args[4:], **kw)
    assert dec.get_error() == 0
    assert_parity(out.cpu().numpy(), ref, "good again")


@pytest.mark.gpu
def test_plain_and_shared_calls_on_one_workspace(S, orc):
    case = shared_case(1024, [10, 200], n_query=2, num_q_heads=16, num_kv_heads=4)
    ref, _ = orc.attend(case)
    dec, args, kw = prepared(S, case, 1024)
    full = torch.from_numpy(case.block_table).cuda()
    for _ in range(2):
        assert_parity(dec(*args, **kw).cpu().numpy(), ref, "shared")
        assert_parity(dec(*args[:3], full, args[4], **kw).cpu().numpy(), ref, "plain")
    assert dec.get_error() == 0
    # a row of the table as the prefix table
    dec2 = S.SharedPrefixDecode(num_seqs=2, num_q_heads=16, num_kv_heads=4, head_dim=128,
                                block_size=16, max_blocks_per_seq=case.max_blocks_per_seq,
                                num_blocks=case.num_blocks, n_query=2,
                                prefix_blocks=case.max_blocks_per_seq)
    assert_parity(dec2(*args[:3], full, args[4], full[1], args[6], **kw).cpu().numpy(), ref, "row")


@pytest.mark.gpu
def test_graph_replay_reads_new_lengths_and_another_stream(S, orc):
    """Captured once; the lengths, the prefix length and the tables are read
    at replay."""
    case = shared_case(2048, [40, 90, 20], n_query=2, num_q_heads=8, num_kv_heads=2)
    dec, args, kw = prepared(S, case, 2048)
    out = torch.empty_like(args[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    dec(*args, **kw, out=out, stream=st)
    st.synchronize()
    assert_parity(out.cpu().numpy(), orc.attend(case)[0], "another stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dec(*args, **kw, out=out)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert_parity(out.cpu().numpy(), orc.attend(case)[0], "replay")
    case.context_lens[:] = [2048 + 7, 2048 + 90, 2048 + 2]
    args[4].copy_(torch.from_numpy(case.context_lens))
    args[6].fill_(1024)
    args[3].copy_(torch.from_numpy(case.block_table))
    g.replay()
    torch.cuda.synchronize()
    assert dec.get_error() == 0
    import pins
    assert_parity(out.cpu().numpy(), orc.attend(pins.zero_nans(case))[0], "shorter prefix")


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
def test_waits_that_time_out_leave_the_workspace_usable(S, orc, dt):
    from paged_kv_decode_flash_b200 import binding as b
    case = shared_case(16384, [40] * 24, n_query=2, num_q_heads=16, num_kv_heads=2, kv_dtype=dt)
    dec, args, kw = prepared(S, case, 16384)
    try:
        b.set_wait_limit(1)  # nanoseconds: no copy is that fast
        dec(*args, **kw)
        torch.cuda.synchronize()
        assert dec.get_error() in (0, -7)
    finally:
        b.set_wait_limit(0)
    out = dec(*args, **kw)
    torch.cuda.synchronize()
    assert dec.get_error() == 0
    assert_parity(out.cpu().numpy(), orc.attend(case)[0], "after a timeout")
