"""Cache in 4 bits without a GPU: what Q4Cache hands to the calls, and values of the oracle worked out by hand."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import _build, api
from oracle import cache4


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


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_a_group_of_ones_beside_one_that_holds_no_number(dtype):
    """1 / 15 lies between the numbers of four bits 8 / 128 and 9 / 128; 128 / 9 is nearest to 14."""
    x = np.ones((2, 32))
    x[0, 5] = np.inf
    v, s = cache4.hold(x, 32, cache4.LARGEST[dtype])
    assert np.isnan(v[0]).all() and (v[1] == 14 * 9 / 128).all() and (s[1] == 9 / 128).all()
