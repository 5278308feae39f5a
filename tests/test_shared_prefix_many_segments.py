"""Shared-prefix decode where a CTA runs through many short segments, so that
the slots of the segments' descriptions are filled again and again while the
roles of the kernel are at different segments.

Tolerance: as in test_shared_prefix.py (tests/parity.py); repeats are compared
bit for bit."""
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


@pytest.mark.gpu
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("prefix,nseq", [(0, 700), (64, 520)])
def test_slots_are_not_read_once_they_are_given_back(S, orc, dt, prefix, nseq):
    """About ten segments a CTA, of one tile and of several in turn: a lane that
    read a slot's tile count too late would lose the ring's phase for all that
    follow."""
    own = [1 + (s * 7) % 90 if s % 3 else 150 + s % 400 for s in range(nseq)]
    case = TS.shared_case(prefix, own, seed=nseq, num_q_heads=6, num_kv_heads=2, kv_dtype=dt)
    dec, args, kw = TS.prepared(S, case, prefix)
    first = dec(*args, **kw)
    for _ in range(12):
        assert torch.equal(first, dec(*args, **kw))
    assert dec.get_error() == 0
    assert_parity(first.cpu().numpy(), orc.attend(case)[0], "many segments")
