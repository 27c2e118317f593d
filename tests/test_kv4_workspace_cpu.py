"""The binding's workspace sizes for the 4-bit cache's attention: they depend on the device's number of SMs, and the binding keeps
them for the device they are of."""
import types

import torch

import ternary_weight_bit_b200 as tb
from ternary_weight_bit_b200 import _native


def test_sizes_are_kept_for_their_own_device(monkeypatch):
    # two devices with different numbers of SMs, in place of the library and of torch's
    current, sms, asked = [0], [148, 160], []

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *_):
            current[0] = self.before

    def size(T, q_heads, heads, dim, batch):
        asked.append(current[0])
        return 1000 * sms[current[0]] + T

    monkeypatch.setattr(_native, "load", lambda: types.SimpleNamespace(bitnet_kv4_attention_workspace_bytes=size))
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    kept = [getattr(tb, n, None) for n in ("_kv4_workspace_bytes", "bitnet_kv4_attention_workspace_bytes")]
    clear = [f.cache_clear for f in kept if hasattr(f, "cache_clear")]
    for f in clear:
        f()
    try:
        args = (5, 8, 4, 128, 2)
        for _ in range(2):
            assert tb.bitnet_kv4_attention_workspace_bytes(*args) == 148005
            current[0] = 1
            assert tb.bitnet_kv4_attention_workspace_bytes(*args) == 160005  # not what device 0 was told
            assert tb.bitnet_kv4_attention_workspace_bytes(*args, device=0) == 148005 and current[0] == 1
            assert tb.bitnet_kv4_attention_workspace_bytes(*args, device=torch.device("cuda", 1)) == 160005
            current[0] = 0
        assert asked == [0, 1]  # each asked for once, with its own device current
    finally:
        for f in clear:
            f()
