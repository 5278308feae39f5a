"""Plain decode of batches with far more (sequence, KV head, row part) groups
than CTAs: every CTA completes more groups than it can list in shared memory,
and every output row has to be written.

Tolerance: tests/parity.py, as in test_gpu_parity.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
from paged_kv_decode_flash_b200 import inputs as gen


@pytest.fixture(scope="module")
def B():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding, build
    build.build()  # no-op when the in-tree library is up to date
    binding.lib()
    return binding


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [gen.KV_FP16, gen.KV_Q8_0, gen.KV_INT8_ROW])
@pytest.mark.parametrize("nseq,nq,G,Hkv,longest", [
    (256, 1, 1, 64, 40),    # 16384 groups of one row
    (300, 1, 2, 40, 300),   # two launches, up to three items a group
    (24, 64, 4, 8, 90),     # 256 rows a KV head in parts
])
def test_every_group_is_merged(B, dt, nseq, nq, G, Hkv, longest):
    lens = [nq + (s * 37) % (longest - nq + 1) for s in range(nseq)]
    case = gen.make_case(seed=nseq, context_lens=tuple(lens), n_query=nq, num_q_heads=G * Hkv, num_kv_heads=Hkv,
                         kv_dtype=dt)
    ref, _ = oracle.load().attend(case)
    dec = B.PagedDecode.for_case(case)
    for _ in range(3):
        out = torch.full(case.q.shape, float("nan"), dtype=torch.float16, device="cuda")
        B.decode_case(case, dec=dec, out=out)
        assert dec.get_error() == 0
        rows = torch.isnan(out).any(-1).sum().item()
        assert rows == 0, f"{rows} rows were not written"
        assert_parity(out.cpu().numpy(), ref, "many groups")
    # nothing is left in the workspace for the next call on other lengths
    case.context_lens[:] = nq
    ref, _ = oracle.load().attend(case)
    out, _ = B.decode_case(case, dec=dec)
    assert dec.get_error() == 0
    assert_parity(out.cpu().numpy(), ref, "short ones behind them")
