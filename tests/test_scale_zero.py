"""Decode with scale 0: every visible key has the same weight."""
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
from paged_kv_decode_flash_b200 import inputs as gen


@pytest.mark.gpu
@pytest.mark.parametrize("dt", (gen.KV_FP16, gen.KV_Q8_0, gen.KV_INT8_ROW))
@pytest.mark.parametrize("nseq", [1, 40])
def test_plain_decode_with_scale_zero_is_the_mean(dt, nseq):
    """In the split kernel and in both modes of the segment kernel."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding as b, build
    build.build()
    case = gen.make_case(context_lens=tuple(30 + 7 * s for s in range(nseq)), n_query=2, num_q_heads=8,
                         num_kv_heads=2, scale=0.0, kv_dtype=dt)
    out, dec = b.decode_case(case)
    assert dec.get_error() == 0
    assert_parity(out.cpu().numpy(), oracle.load().attend(case)[0], "scale 0")
