"""Shared-prefix decode over int8 rows whose V scales lie far apart, where the
key that carries the weight is not the one with the large V.

Tolerance: tests/parity.py (max-abs 2e-3 and max-rel 1e-2 against
max(|oracle|, 1e-3)).  What the arithmetic may lose: a key's weight times its V
scale is kept to 2^-21 of the largest such product among the row's keys (fp16
high part and residual, 2^-24 steps at the least, the largest above 2), V's
values and K's are exact, fp32 sums over at most 1500 keys add 1500 * 2^-24.
The outputs here are sums in which the largest product is not cancelled by
more than a factor of some tens: below 1e-3 relative."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from parity import assert_parity
import pins
import test_shared_prefix as TS
from paged_kv_decode_flash_b200 import inputs as gen


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


def scale_of(case, cache):
    """The row scales fp32 [blocks][heads][bs] of a cache, to be written back
    by `store`."""
    return cache[:, :, case.block_size * 128:].copy().view(np.float32)


def store(case, cache, scales):
    cache[:, :, case.block_size * 128:] = np.ascontiguousarray(scales, np.float32).view(np.uint8).reshape(
        cache[:, :, case.block_size * 128:].shape)


def aligned_case(prefix, own, keys, lead, others, light, G=2, heavy=1.0):
    """Every row's weight lies on the keys `keys` of the prefix, whose scores
    lead the others' by `lead` (log2 units); V scales: `light` there, `others`
    elsewhere."""
    case = TS.shared_case(prefix, own, n_query=2, num_q_heads=2 * G, num_kv_heads=2, kv_dtype=gen.KV_INT8_ROW,
                          poison=False)
    rng = np.random.default_rng(len(keys))
    bs = case.block_size
    case.q[:] = (0.5 + rng.random(case.q.shape) / 8).astype(np.float16)
    ks, vs = scale_of(case, case.k_cache), scale_of(case, case.v_cache)
    ks[:] = np.exp2(-20.0)
    vs[:] = others * (0.75 + 0.25 * rng.random(vs.shape))
    for key in keys:
        b, slot = case.block_table[0, key // bs], key % bs
        case.k_cache[b, :, slot * 128:(slot + 1) * 128] = 100
        # sum of q is about 72: lead = scale * log2(e) * 72 * 100 * ks
        ks[b, :, slot] = lead / (case.scale * 1.4427 * 72 * 100)
        vs[b, :, slot] = light
    store(case, case.k_cache, ks)
    store(case, case.v_cache, vs)
    return case


@pytest.mark.gpu
@pytest.mark.parametrize("keys", [[5], [40], [64 + 33], [700], [3, 41, 610, 999]])
@pytest.mark.parametrize("power", [0, 10, 18, 24, 30, 40])
@pytest.mark.parametrize("nseq", [3, 40])  # a single and a dual segment
def test_the_weight_is_not_where_the_large_values_are(S, orc, keys, power, nseq):
    """V scales 2^power apart; the weights of the large ones are 2^-(power + 25)."""
    case = aligned_case(1008, [20 + s % 7 * 30 for s in range(nseq)], keys, power + 25.0, 2.0 ** power / 127, 1 / 127)
    ref, _ = orc.attend(case)
    assert np.abs(ref).max() > 0.3
    assert_parity(TS.run(S, case, 1008), ref, f"2^{power}")


@pytest.mark.gpu
@pytest.mark.parametrize("lead", [10.0, 90.0, 200.0])
@pytest.mark.parametrize("light", [0.0, 2.0 ** -100])
def test_the_weight_is_on_a_value_of_zero(S, orc, lead, light):
    """The row's sum of weights grows where its values do not."""
    case = aligned_case(1008, (20, 150, 9), [41, 640], lead, 1 / 127, light)
    ref, _ = orc.attend(case)
    assert_parity(TS.run(S, case, 1008), ref, f"{lead}")


@pytest.mark.gpu
def test_scales_that_rise_and_fall_along_the_keys(S, orc):
    """Each tile's V scales are 2^8 off the last one's, up and down again, with
    scores that make up for it: all tiles count."""
    prefix = 2048
    case = TS.shared_case(prefix, (9, 200, 33), n_query=2, num_q_heads=8, num_kv_heads=2, kv_dtype=gen.KV_INT8_ROW,
                          poison=False)
    bs = case.block_size
    rng = np.random.default_rng(11)
    case.q[:] = (0.5 + rng.random(case.q.shape) / 8).astype(np.float16)
    ks, vs = scale_of(case, case.k_cache), scale_of(case, case.v_cache)
    for key in range(prefix):
        b, slot = case.block_table[0, key // bs], key % bs
        t = key // 128
        power = 8 * min(t, 15 - t)
        case.k_cache[b, :, slot * 128:(slot + 1) * 128] = 100
        ks[b, :, slot] = (64 - power) / (case.scale * 1.4427 * 72 * 100)
        vs[b, :, slot] = 2.0 ** power / 127
    store(case, case.k_cache, ks)
    store(case, case.v_cache, vs)
    ref, _ = orc.attend(pins.zero_nans(case))
    assert_parity(TS.run(S, case, prefix), ref, "rise and fall")
