"""Q4Cache without a GPU: what it hands to the calls."""
import pytest
import torch

from kv_cache_eviction_02_gb300 import _build, api


@pytest.fixture
def calls(monkeypatch):
    _build.build()
    seen = []
    for name in ("q4_pack", "q4_attention", "q4_unpack"):
        monkeypatch.setattr(api, name, lambda *a, name=name: seen.append((name, a)))
    return seen


def test_every_layer_keeps_its_own_lengths(calls):
    pb = api.Q4Problem(2, 1, 4, 2, 32, 40, 16, 4, 2, 2, 1, api.KVE_BF16, 32)
    c = api.Q4Cache(pb, 3, "cpu")
    K = torch.zeros(2, 2, 40, 32, dtype=torch.bfloat16)
    few, other = torch.tensor([7, 0], dtype=torch.int32), torch.tensor([40, 12], dtype=torch.int32)
    c.pack(0, K, K, few)
    c.pack(1, K, K)
    c.pack(2, K, K, other)
    want = [few, None, other]
    assert [a[3] for n, a in calls if n == "q4_pack"] == want
    calls.clear()
    for layer in (2, 0, 1):
        c.attend(layer, None, None)
        c.unpack(layer, K, K, prompts=True)
        (n0, attend), (n1, unpack) = calls
        assert (n0, n1) == ("q4_attention", "q4_unpack")
        assert attend[3] is want[layer] and unpack[3] is want[layer] and unpack[2] is None
        for cache in (attend[2], unpack[1]):
            assert cache.data_ptr() == c.prefix[layer].data_ptr()
        calls.clear()
    c.pack(0, K, K, other)  # after another eviction
    c.attend(0, None, None)
    assert calls[-1][1][3] is other
