"""Decoders whose tensors are not on the current device, on the host with a
library and a device that only tell what they were asked: every call has to be
made with the workspace's device current, on that device's current stream."""
import types

import pytest

torch = pytest.importorskip("torch")

from paged_kv_decode_flash_b200 import binding as B
import test_outputs_on_streams as TO


@pytest.fixture
def asked(monkeypatch):
    """(device index, stream) of every launch."""
    seen = []

    def on(index, stream, call):
        seen.append((index, stream))
        return call(64)

    names = ("paged_attn_decode", "paged_attn_decode_partial", "paged_attn_trace", "paged_attn_merge",
             "paged_attn_cache_write", "paged_attn_get_error", "paged_attn_workspace_init",
             "paged_attn_decode_shared")
    nothing = types.SimpleNamespace(**{n: lambda *a: 0 for n in names})
    nothing.paged_attn_workspace_size = nothing.paged_attn_shared_workspace_size = lambda *a: 64
    monkeypatch.setattr(B, "lib", lambda: nothing)
    monkeypatch.setattr(B, "_on", on)
    monkeypatch.setattr(B, "_dptr", lambda t: 0)

    def not_this_way(stream):
        raise AssertionError("the stream of whatever device is current")

    monkeypatch.setattr(B, "_stream_ptr", not_this_way)
    return seen


@pytest.mark.parametrize("shared", [False, True])
def test_calls_go_to_the_workspaces_device(asked, shared):
    from paged_kv_decode_flash_b200.shared_prefix import SharedPrefixDecode
    dec, args, i32 = TO.decoder_on_the_host(SharedPrefixDecode if shared else B.PagedDecode)
    kw = dict(causal=1, window=0, scale=0.1, kv_dtype=0)
    new = torch.zeros(2, 1, 2, 128, dtype=torch.float16)
    calls = [lambda: dec(*args, **kw), lambda: dec.partial(*args, i32(2), i32(2), **kw),
             lambda: dec.trace(*args, **kw), lambda: dec.get_error(),
             lambda: dec.cache_write(new, new, *args[3:], kv_dtype=0, k_cache=args[1], v_cache=args[2]),
             lambda: B.merge(torch.zeros(3, 5, 128), torch.zeros(3, 5))]
    if shared:
        calls.append(lambda: dec(*args, i32(7), i32(1), **kw))
    for n, call in enumerate(calls):
        call()
        assert asked == [(dec.workspace.device.index, None)] * (n + 1)


def made_on(monkeypatch, make):
    """The devices that a constructor asks memory of."""
    devices = []
    empty = torch.empty

    def logged(*a, **kw):
        devices.append(kw.pop("device", None))
        return empty(*a, **kw)

    monkeypatch.setattr(torch, "empty", logged)
    monkeypatch.setattr(torch.cuda, "device", lambda d: __import__("contextlib").nullcontext())
    make()
    return devices


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("device,want", [(0, 0), (1, 1), (None, "cuda"), ("cuda:0", "cuda:0")])
def test_device_0_is_a_device(asked, monkeypatch, shared, device, want):
    """Whatever device is current; nothing is asked of "cuda" where one is named."""
    from paged_kv_decode_flash_b200.shared_prefix import SharedPrefixDecode
    dims = dict(num_seqs=2, num_q_heads=4, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=10,
                num_blocks=25, n_query=1)
    make = ((lambda: SharedPrefixDecode(prefix_blocks=7, device=device, **dims)) if shared else
            (lambda: B.PagedDecode(device=device, **dims)))
    assert made_on(monkeypatch, make) == [want]
