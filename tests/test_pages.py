"""Shared-prompt decoding without a GPU: pins of the fp64 oracle, refusals of the C-ABI and of the
binding (everything here returns before a CUDA call)."""
import ctypes
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import shared_prompt as sp


@pytest.fixture(scope="module")
def api():
    from kv_cache_eviction_02_gb300 import _build, api as a
    _build.build()
    a.lib()
    return a


def _pb(api, **kw):
    base = dict(n_prompts=2, fan=3, n_q_heads=8, n_kv_heads=2, d_head=64, n_prefix=100,
                page_size=16, n_pages=40, max_pages=5, n_rows=20, max_new=7, dtype=1)
    base.update(kw)
    return api.PgProblem(**base)


# ---- the oracle ------------------------------------------------------------------------------------
def test_a_page_is_never_held_twice_and_none_is_lost():
    """Random steps (rows, idle, finished, requests too long, an empty pool): every page is either in
    one table or in the ring, and a request's slots are its pages' rows in order."""
    rng = np.random.default_rng(0)
    R, page, n_pages, max_pages, max_new, n_rows = 7, 4, 19, 6, 9, 30
    lens, pool = np.zeros(R, int), np.array([0, n_pages, 0, 0])
    free, table = np.arange(n_pages), np.full((R, max_pages), -1)
    refused = finished = 0
    for _ in range(400):
        new = rng.choice([-1, 0, 1, 2, 5, 9, 11], R)
        o = sp.pg_plan(new, lens, pool, free, table, page, max_new, n_rows)
        for r in range(R):
            for i in np.flatnonzero(o["row_req"] == r):
                p = o["row_pos"][i]
                assert o["slot_map"][i] == o["block_table"][r, p // page] * page + p % page
            assert (o["row_req"] == r).sum() == max(0, o["len"][r] - lens[r])
        lens, pool, free, table = o["len"], o["pool"], o["free_pages"], o["block_table"]
        held = [p for r in range(R) for p in table[r, :math.ceil(lens[r] / page)]]
        ring = [free[(pool[0] + i) % n_pages] for i in range(pool[1])]
        assert sorted(held + ring) == list(range(n_pages))
        refused += pool[3]
        finished += (new < 0).sum()
    assert refused > 50 and finished > 50


def test_attention_is_one_softmax_over_prompt_and_own_rows():
    """Against a dense softmax with an explicit mask, from one-hot pages laid out by hand."""
    rng = np.random.default_rng(1)
    d, page, fan = 8, 2, 2
    K, V = rng.normal(size=(5, 1, page, d)), rng.normal(size=(5, 1, page, d))
    Kp, Vp = rng.normal(size=(1, 1, 3, d)), rng.normal(size=(1, 1, 3, d))
    q = rng.normal(size=(3, 2, d))
    # request 0: rows in pages 4, 1 (3 rows, 2 of them new); request 1: page 2 (1 row, new)
    o = sp.pg_attention(q, Kp, Vp, [3], K, V, np.array([[4, 1], [2, 0]]), [3, 1], [0, 2, 3], fan)
    k = np.concatenate((Kp[0, 0], K[4, 0], K[1, 0, :1], K[2, 0, :1]))
    v = np.concatenate((Vp[0, 0], V[4, 0], V[1, 0, :1], V[2, 0, :1]))
    sees = np.array([[1, 1, 1, 1, 1, 0, 0], [1, 1, 1, 1, 1, 1, 0], [1, 1, 1, 0, 0, 0, 1]], bool)
    for i, h in itertools.product(range(3), range(2)):
        w = np.where(sees[i], np.exp(k @ q[i, h] / math.sqrt(d)), 0)
        assert np.allclose(o["out"][i, h], w @ v / w.sum(), rtol=1e-12)
        assert np.isclose(o["lse"][i, h], math.log(w.sum()), rtol=1e-12)


def test_equal_keys_average_the_values_and_nothing_gives_zero():
    d = 4
    K, V = np.ones((1, 1, 4, d)), np.arange(4.0)[:, None].repeat(d, 1)[None, None]
    q = np.ones((2, 1, d))
    o = sp.pg_attention(q, np.zeros((1, 1, 0, d)), np.zeros((1, 1, 0, d)), [0], K, V,
                        np.array([[0]]), [2], [0, 2], 1)
    assert np.allclose(o["out"][:, 0, 0], [0.0, 0.5])
    assert np.allclose(o["lse"][:, 0], [2.0, 2.0 + math.log(2)])
    o = sp.pg_attention(q, np.zeros((1, 1, 0, d)), np.zeros((1, 1, 0, d)), [0], K, V,
                        np.array([[0]]), [1], [0, 2], 1)  # the first row sees nothing
    assert (o["out"][0] == 0).all() and np.isneginf(o["lse"][0, 0])


# ---- refusals --------------------------------------------------------------------------------------
BAD = [
    dict(n_prompts=0), dict(fan=0), dict(n_prefix=-1), dict(n_pages=0), dict(max_pages=0),
    dict(n_rows=0), dict(max_new=0),
    dict(n_q_heads=9),                            # not a multiple of n_kv_heads
    dict(n_q_heads=258),                          # 129 query heads per KV head
    dict(d_head=96), dict(dtype=3), dict(dtype=-1),
    dict(page_size=12), dict(page_size=512), dict(page_size=0),
    dict(n_prompts=16385, fan=1),                 # too many requests
    dict(n_prompts=1 << 16, fan=1 << 16),         # their product passes 32 bits
    dict(n_pages=1 << 27),                        # slots beyond 2^30
    dict(max_pages=1 << 27),
    dict(n_rows=1 << 28, n_q_heads=8),            # rows * heads beyond 31 bits
    dict(n_kv_heads=64, n_q_heads=64, n_pages=1 << 22),   # pool rows beyond 31 bits
    dict(n_prompts=2048, fan=1, n_q_heads=64, n_kv_heads=64),  # launch-grid limits
    dict(n_prompts=1, fan=1, n_rows=1, n_q_heads=1 << 17, n_kv_heads=1 << 12),
]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: "-".join(f"{k}{v}" for k, v in b.items()))
def test_invalid_shapes_are_rejected_without_a_gpu(api, bad):
    pb = _pb(api, **bad)
    assert api.pg_workspace_size(pb) == 0
    L, sh, fake = api.lib(), pb.shape(), ctypes.c_void_p(256)
    p = ctypes.byref(sh)
    want = api.KVE_EDTYPE if "dtype" in bad else api.KVE_EINVAL
    assert L.pg_plan(p, *[fake] * 11, None) == want
    assert L.pg_append(p, fake, fake, 1 << 20, 1 << 20, fake, fake, fake, None) == want
    assert L.pg_attention(p, fake, 1 << 20, fake, fake, 1 << 20, 1 << 20, 1 << 10, fake, fake, fake,
                          fake, fake, fake, fake, fake, fake, fake, 1 << 50, None) == want
    assert L.kve_last_error().decode()
    with pytest.raises(api.KveError):
        api.PgCache(pb, 1, "cpu")


def test_null_and_unaligned_arguments_are_rejected_without_a_gpu(api):
    L, sh = api.lib(), _pb(api).shape()
    p, fake, odd = ctypes.byref(sh), ctypes.c_void_p(256), ctypes.c_void_p(264)
    assert L.pg_plan(None, *[fake] * 11, None) == api.KVE_EINVAL
    for i in range(11):
        args = [fake] * 11
        args[i] = None
        assert L.pg_plan(p, *args, None) == api.KVE_EINVAL
    row = 2 * 64
    good = [fake, fake, row, row, fake, fake, fake]
    for i, v in ((0, None), (1, None), (4, None), (5, None), (6, None), (0, odd), (1, odd), (5, odd),
                 (6, odd), (2, row - 8), (3, row - 8), (2, row + 4), (3, row + 4)):
        args = list(good)
        args[i] = v
        assert L.pg_append(p, *args, None) == api.KVE_EINVAL, (i, v)
    head = 100 * 64
    good = [fake, 8 * 64, fake, fake, 2 * head, head, 64, None] + [fake] * 6 + [fake, fake, fake,
                                                                             1 << 40]
    for i, v in ((0, None), (0, odd), (1, 8 * 64 - 8), (1, 8 * 64 + 4), (2, None), (3, None),
                 (2, odd), (3, odd), (4, 4), (5, head + 4), (6, 60), (6, 32), (6, 1 << 40),
                 (8, None), (8, odd), (9, None), (9, odd), (10, None), (11, None), (12, None),
                 (13, None), (14, None), (14, odd)):
        args = list(good)
        args[i] = v
        assert L.pg_attention(p, *args, None) == api.KVE_EINVAL, (i, v)
    args = list(good)
    args[16] = None
    assert L.pg_attention(p, *args, None) == api.KVE_EWORKSPACE
    args[16], args[17] = fake, api.pg_workspace_size(_pb(api)) - 1
    assert L.pg_attention(p, *args, None) == api.KVE_EWORKSPACE
    args[16], args[17] = odd, 1 << 40
    assert L.pg_attention(p, *args, None) == api.KVE_EINVAL


def test_injected_failures_reach_every_call(api):
    pb = _pb(api)
    api.kve_inject_failure(api.KVE_ECUDA, 3)
    L, sh, fake = api.lib(), pb.shape(), ctypes.c_void_p(256)
    p = ctypes.byref(sh)
    assert L.pg_plan(p, *[fake] * 11, None) == api.KVE_ECUDA
    assert L.pg_append(p, fake, fake, 128, 128, fake, fake, fake, None) == api.KVE_ECUDA
    assert L.pg_attention(p, fake, 512, fake, fake, 12800, 6400, 64, *[fake] * 10, 1 << 40,
                          None) == api.KVE_ECUDA
    api.kve_inject_failure(0, 0)


def test_workspace_holds_a_partial_result_per_split(api):
    pb = _pb(api)
    ws = api.pg_workspace_size(pb)
    assert ws % 256 == 0 and ws >= 2 * pb.n_rows * pb.n_q_heads * (pb.d_head + 2) * 4
    assert api.pg_workspace_size(_pb(api, n_rows=40)) > ws


def test_binding_checks_tensors_against_the_shape(api):
    pb = _pb(api)
    R, n = pb.requests, pb.n_rows
    i = lambda k: torch.zeros(k, dtype=torch.int32)  # noqa: E731
    plan = [i(R), i(R), i(4), i(pb.n_pages), i(R * pb.max_pages), i(R), i(4), i(R + 1), i(n), i(n),
            i(n)]
    for k in range(len(plan)):
        args = [1] * len(plan)
        args[k] = plan[k][:-1]
        with pytest.raises(ValueError, match="elements"):
            api.pg_plan(pb, *args)
        args[k] = plan[k].long()
        with pytest.raises(ValueError, match="dtype"):
            api.pg_plan(pb, *args)
        args[k] = plan[k]
        with pytest.raises(ValueError, match="CUDA"):
            api.pg_plan(pb, *args)
    bf = torch.bfloat16
    pool = torch.zeros(pb.pool_elements, dtype=bf)
    new = torch.zeros(n, 6, 64, dtype=bf)[:, 2:4]
    with pytest.raises(ValueError, match="dtype"):
        api.pg_append(pb, new.float(), new, i(n), pool, pool)
    with pytest.raises(ValueError, match="elements"):
        api.pg_append(pb, new[:-1], new, i(n), pool, pool)
    with pytest.raises(ValueError, match="elements"):
        api.pg_append(pb, 1, 1, 1, pool[1:], pool)
    with pytest.raises(ValueError, match="CUDA"):
        api.pg_append(pb, new, new, i(n), pool, pool)
    q, kp = torch.zeros(n, 8, 64, dtype=bf), torch.zeros(2, 2, 100, 64, dtype=bf)

    def attend(q=1, k=1, v=1, plen=None, pages=1, out=1, lse=None):
        api.pg_attention(pb, q, k, v, plen, pages, 1, 1, 1, 1, 1, out, lse, None)

    for kw, word in ((dict(q=q.half()), "dtype"), (dict(q=q[:-1]), "elements"),
                     (dict(k=kp[:, :, :99]), "elements"), (dict(k=kp[:1]), "elements"),
                     (dict(v=kp.float()), "dtype"), (dict(plen=i(1)), "elements"),
                     (dict(pages=pool[1:]), "elements"), (dict(out=q[:-1]), "elements"),
                     (dict(lse=torch.zeros(n * 8 - 1)), "elements"),
                     (dict(q=q), "CUDA"), (dict(k=kp), "CUDA")):
        with pytest.raises(ValueError, match=word):
            attend(**kw)
