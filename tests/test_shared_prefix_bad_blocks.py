"""Shared-prefix decode with a block out of range in a table, while block 0,
which belongs to nobody, holds NaN: rows that do not see the bad block's keys
are what they are without it.

Tolerance: as in test_shared_prefix.py (tests/parity.py)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
import test_shared_prefix as TS

DTYPES = TS.DTYPES


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


def block_0_is_nobodys(case):
    """Exchanges block 0 with a spare one and fills it with NaN."""
    used = set()
    for row, n in zip(case.block_table, case.context_lens):
        used |= set(int(b) for b in row[:-(-int(n) // case.block_size)])
    spare = max(b for b in range(case.num_blocks) if b not in used)
    for cache in (case.k_cache, case.v_cache):
        cache[[0, spare]] = cache[[spare, 0]]
    case.block_table[:] = np.where(case.block_table == 0, spare, case.block_table)
    for slot in range(case.block_size):
        TS.poison(case, 0, slot)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("index", [-1, 1 << 29])
@pytest.mark.parametrize("G,nseq", [(2, 3), (4, 9)])  # 48 rows a KV head, and 288 (two row tiles)
def test_rows_that_do_not_see_a_bad_block(S, orc, dt, index, G, nseq):
    nq = 8
    own = [20, 400, 30, 60, 12, 40, 9, 100, 75][:nseq]
    case = TS.shared_case(640, own, n_query=nq, num_q_heads=2 * G, num_kv_heads=2, kv_dtype=dt, spare_blocks=4)
    block_0_is_nobodys(case)
    ref = np.asarray(orc.attend(case)[0])
    dec, args, kw = TS.prepared(S, case, 640)
    assert_parity(dec(*args, **kw).cpu().numpy(), ref, "without")
    # a sequence's own block: keys 656 .. 671, of which new tokens 652 .. 655 see none
    args[3][0, 41] = index
    out = dec(*args, **kw).cpu().numpy()
    assert dec.get_error() == -5
    assert not out[0, 4:].any()
    assert_parity(out[0, :4], ref[0, :4], "the tokens before it")
    assert_parity(out[1:], ref[1:], "the other sequences")
    # a block of the prefix behind some windows: sequence 1 sees from 1032 - 300 on
    case = TS.shared_case(640, own, n_query=nq, num_q_heads=2 * G, num_kv_heads=2, kv_dtype=dt, spare_blocks=4,
                          window=300)
    block_0_is_nobodys(case)
    ref = np.asarray(orc.attend(case)[0])
    dec, args, kw = TS.prepared(S, case, 640)
    args[5][25] = index  # keys 400 .. 415
    out = dec(*args, **kw).cpu().numpy()
    assert dec.get_error() == -5
    sees = np.array([[max(0, 640 + n - nq + i - 299) <= 415 for i in range(nq)] for n in own])
    assert not out[sees].any() and sees.any()
    assert_parity(out[~sees], ref[~sees], "rows that do not see it")
