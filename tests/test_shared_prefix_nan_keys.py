"""Shared-prefix decode over the int8 caches with a key of NaN among the second
32 keys of a segment's first 64: the rows that see it have the first 32 keys'
weights read back and written again, the others keep theirs, bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
import test_shared_prefix as TS
import test_shared_prefix_edges as TE
from paged_kv_decode_flash_b200 import inputs as gen


@pytest.fixture(scope="module")
def S():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding, build, shared_prefix
    build.build()  # no-op when the in-tree library is up to date
    binding.lib()
    return shared_prefix


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [gen.KV_Q8_0, gen.KV_INT8_ROW])
@pytest.mark.parametrize("prefix,nseq,G", [(0, 90, 4), (256, 30, 2)])
def test_rows_that_do_not_see_it_keep_their_bits(S, dt, prefix, nseq, G):
    nq, own = 8, 45  # new tokens at own positions 37 .. 44; the key at 41
    case = TS.shared_case(prefix, (own,) * nseq, seed=dt, n_query=nq, num_q_heads=2 * G, num_kv_heads=2,
                          kv_dtype=dt)
    ref = np.asarray(oracle.load().attend(case)[0])
    dec, args, kw = TS.prepared(S, case, prefix)
    want = dec(*args, **kw).cpu()
    assert_parity(want.numpy(), ref, "finite")
    for s in range(0, nseq, 2):
        TE.poison_key(case, s, prefix + 41, s // 2 % 2)
    args[1] = torch.from_numpy(case.k_cache).cuda()
    nan = np.zeros((nseq, nq, 2, G), bool)
    for s in range(0, nseq, 2):
        nan[s, 4:, s // 2 % 2] = True
    nan = nan.reshape(nseq, nq, 2 * G)
    for _ in range(5):
        out = dec(*args, **kw).cpu()
        assert out[torch.from_numpy(nan)].isnan().all()
        assert torch.equal(out[torch.from_numpy(~nan)], want[torch.from_numpy(~nan)])
    assert dec.get_error() == 0
