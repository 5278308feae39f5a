"""Batches whose tables reach far: the partials of one group, which a CTA
merges through shared memory, stay as many as fit there."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def L():
    from paged_kv_decode_flash_b200 import build
    build.build()
    from paged_kv_decode_flash_b200 import binding
    return binding.lib()


@pytest.mark.parametrize("kv_heads", [1, 8])
def test_partials_of_a_group_are_bounded(L, kv_heads):
    """A partial of a row takes 516 bytes of workspace and, while it is merged,
    20 of about 200,000 bytes of shared memory."""
    from paged_kv_decode_flash_b200.binding import Dims

    def slots(tokens):
        d = Dims(64, kv_heads, kv_heads, 128, 16, tokens // 16, 1000, None, 0)
        n = L.paged_attn_workspace_size(ctypes.byref(d), 1)
        assert n > 0
        return n / (64 * kv_heads * 516)

    last = 0
    for tokens in (1 << 12, 1 << 16, 1 << 20, 1 << 22, 1 << 24, 1 << 27, (1 << 31) - 16):
        n = slots(tokens)
        assert n < 4200, tokens
        if tokens <= 1 << 22:  # an item of 2048 keys each
            assert n >= tokens / 2048
            assert n >= last
        last = n


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [0, 1, 2])
def test_a_batch_behind_a_long_table(L, dt):
    """Twelve million keys a sequence, all in the same few blocks, against the
    same keys weighed by how often they come."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_decode_flash_b200 import binding as B
    import numpy as np
    rng = np.random.default_rng(dt)
    bs, blocks, heads, nseq = 16, 8, 8, 5  # 40 groups: the queue's form
    entries = 750_000 + 3
    lens = [12_000_000, 12_000_005, 300, 16, 11_000_000]
    dtype, shape = B.cache_shape(dt, blocks, heads, bs, 128)
    if dt == 0:
        k, v = (torch.randn(shape, device="cuda").half() for _ in range(2))
        kf, vf = k.double(), v.double()
    else:
        def quant():
            q = torch.randint(-127, 128, (blocks, heads, bs, 128), device="cuda", dtype=torch.int8)
            n = 4 if dt == 1 else 1
            d = (0.005 + torch.rand(blocks, heads, bs, n, device="cuda") / 60).to(torch.float16 if dt == 1 else torch.float32)
            raw = torch.cat([q.reshape(blocks, heads, -1).view(torch.uint8),
                             d.reshape(blocks, heads, -1).contiguous().view(torch.uint8)], -1).contiguous()
            return raw, q.double() * d.double().repeat_interleave(128 // n, -1)
        (k, kf), (v, vf) = quant(), quant()
    table = torch.randint(0, blocks, (nseq, entries), device="cuda", dtype=torch.int32)
    q = torch.randn(nseq, 1, heads, 128, device="cuda").half()
    dec = B.PagedDecode(num_seqs=nseq, num_q_heads=heads, num_kv_heads=heads, head_dim=128, block_size=bs,
                        max_blocks_per_seq=entries, num_blocks=blocks, n_query=1)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = dec(q, k, v, table, ctx, causal=1, window=0, scale=128 ** -0.5, kv_dtype=dt)
    assert dec.get_error() == 0
    for s, n in enumerate(lens):
        whole, rest = divmod(n, bs)
        times = torch.bincount(table[s, :whole].long(), minlength=blocks).double().view(blocks, 1).repeat(1, bs)
        if rest:
            times[table[s, whole].long(), :rest] += 1
        for h in range(heads):
            z = (kf[:, h].reshape(-1, 128) @ q[s, 0, h].double()) * 128 ** -0.5
            w = torch.exp(z - z.max()) * times.reshape(-1)
            ref = (w @ vf[:, h].reshape(-1, 128)) / w.sum()
            # fp16 rounding of the output, 2^-11, and the tensor cores' sums, cut off at 2^-23 each of the up to 400
            # additions of an item of 3000 keys: together below 6e-4
            err = (out[s, 0, h].double() - ref).abs()
            assert (err <= 2e-3 * ref.abs().clamp_min(ref.abs().mean())).all(), (s, h, err.max().item())
