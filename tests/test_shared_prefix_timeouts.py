"""Shared-prefix decode whose waits run out (a limit set by the host, so short
that the copies cannot keep it): a call that gave up says so, and what it
writes is zero or right, never what an earlier call left in the workspace."""
import pytest

torch = pytest.importorskip("torch")

import test_shared_prefix as TS

DTYPES = TS.DTYPES
TIMEOUT = -7


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
@pytest.mark.parametrize("prefix,own,G", [(16384, (40,) * 24, 8), (0, tuple(range(2, 300)), 3), (320, (9, 700), 4)])
def test_rows_of_a_call_that_gave_up_are_zero_or_right(S, dt, prefix, own, G):
    """Long segments, many short ones, few rows."""
    from paged_kv_decode_flash_b200 import binding as b
    case = TS.shared_case(prefix, own, n_query=2, num_q_heads=2 * G, num_kv_heads=2, kv_dtype=dt)
    dec, args, kw = TS.prepared(S, case, prefix)
    want = dec(*args, **kw)
    assert dec.get_error() == 0
    good = want.any(-1)  # [B][nq][Hq]
    assert good.all()
    other = [torch.randn_like(args[0]), *args[1:]]
    told = 0
    for limit in (1, 1, 1000, 5000, 20000, 80000):  # nanoseconds
        left = dec(*other, **kw)  # other partials in every slot
        assert dec.get_error() == 0 and not torch.equal(left, want)
        try:
            b.set_wait_limit(limit)
            out = dec(*args, **kw)
            error = dec.get_error()
        finally:
            b.set_wait_limit(0)
        zero = ~out.any(-1)
        right = (out == want).all(-1)
        assert (zero | right).all(), limit
        assert error in (0, TIMEOUT), limit
        assert error == TIMEOUT or right.all(), limit
        told += error == TIMEOUT
    assert told > 0
    assert torch.equal(dec(*args, **kw), want)
    assert dec.get_error() == 0
