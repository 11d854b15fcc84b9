"""PgProblem as a value, without a GPU."""
import copy
import pickle

import pytest


@pytest.mark.parametrize("way", ["pickle", "deepcopy", "copy"])
@pytest.mark.parametrize("used", [False, True])
def test_a_problem_can_be_copied_and_sent(way, used):
    """Also after a call has made the C struct of it, whose address stays with the object that owns it."""
    from kv_cache_eviction_02_gb300 import api
    pb = api.PgProblem(2, 3, 8, 2, 64, 100, 16, 40, 5, 20, 7, api.KVE_BF16)
    if used:
        assert pb.c_address and pb.requests == 6 and pb.torch_dtype and pb.pool_elements
    twin = {"pickle": lambda x: pickle.loads(pickle.dumps(x)), "deepcopy": copy.deepcopy,
            "copy": copy.copy}[way](pb)
    assert twin == pb and hash(twin) == hash(pb) and twin.requests == 6
    address = pb.c_address
    assert twin.c_address != address
    assert twin.c_shape.contents.page_size == 16 and twin.c_shape.contents.dtype == api.KVE_BF16
