"""Cache in 4 bits without a GPU: pins of the fp64 oracle, sizes, refusals of the C-ABI and of the binding
(everything here returns before a CUDA call)."""
import copy
import ctypes
import itertools
import pickle

import numpy as np
import pytest
import torch

from oracle import cache4


@pytest.fixture(scope="module")
def api():
    from kv_cache_eviction_02_gb300 import _build, api as a
    _build.build()
    a.lib()
    return a


def _pb(api, **kw):
    base = dict(n_prompts=2, fan=3, n_q_heads=8, n_kv_heads=2, d_head=64, n_prefix=100, page_size=16,
                n_pages=40, max_pages=5, n_rows=20, max_new=7, dtype=1, group=32)
    base.update(kw)
    return api.Q4Problem(**base)


# ---- the oracle ------------------------------------------------------------------------------------
def test_a_value_is_the_nearest_that_its_group_has():
    """By trying all 16 values of the group; the step by trying all smaller ones of four bits."""
    rng = np.random.default_rng(0)
    for scale, shift in itertools.product((2.0 ** -130, 1e-3, 1.0, 2.0 ** 100), (0.0, 0.7, 30.0, -30.0)):
        x = (rng.normal(size=(8, 32)) + shift) * scale
        v, s = cache4.hold(x, 32, cache4.LARGEST["f32"])
        for row, val, st in zip(x, v, s[:, 0]):
            lo, hi = min(0, row.min()), max(0, row.max())
            assert 15 * st >= hi - lo
            mant, exp = np.frexp(st)
            assert mant * 16 == round(mant * 16)
            below = np.ldexp((mant * 16 - 1) / 16 if mant > 0.5 else 15 / 32, exp)
            assert st == 2.0 ** -126 or 15 * below < hi - lo
            k = cache4.nearest(-lo / st)
            have = (np.arange(16) - k) * st
            assert (np.abs(val - row) <= np.abs(have[:, None] - row).min(0) * (1 + 1e-12)).all()
            assert np.isin(val, have).all()


def test_steps_zeros_halves_and_the_largest_numbers():
    F = cache4.LARGEST["f16"]
    v, s = cache4.hold(np.zeros((1, 32)), 32, F)
    assert (v == 0).all() and (s == 2.0 ** -126).all()
    x = np.zeros((1, 32))
    x[0, :6] = [15, -0.5, 0.5, 1.5, -0.25, 7.5]  # the step is above 1: 15.5 / 15
    v, s = cache4.hold(x, 32, F)
    assert s[0, 0] == 1.125 and v[0, 0] == 13 * 1.125
    x[0, 1] = x[0, 4] = 0  # now it is 1: halves go toward zero
    v, s = cache4.hold(x, 32, F)
    assert s[0, 0] == 1 and v[0, :6].tolist() == [15, 0, 0, 1, 0, 7]
    x = np.full((1, 32), 65504.0)
    x[0, 1] = -20000
    v, s = cache4.hold(x, 32, F)
    assert (np.abs(v) <= F).all() and s[0, 0] == 6144 and v[0, 0] == 10 * 6144
    x[0, 5] = np.inf
    v, _ = cache4.hold(np.concatenate((x, np.ones((1, 32)))), 32, F)
    assert np.isnan(v[0]).all() and (v[1] == 1).mean() >= 0 and np.isfinite(v[1]).all()


# ---- sizes and refusals ----------------------------------------------------------------------------
@pytest.mark.parametrize("d,group", [(32, 32), (64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_sizes(api, d, group):
    pb = _pb(api, d_head=d, group=group, n_prefix=33, page_size=64)
    tile = 16 * d + 64 * d // group
    assert pb.prefix_bytes == 2 * 2 * 3 * tile and pb.pool_bytes == 40 * 2 * 4 * tile
    assert api.q4_workspace_size(pb) > 0 and api.q4_workspace_size(pb) % 256 == 0
    assert _pb(api, d_head=d, group=group, n_prefix=0).prefix_bytes == 0


BAD = [dict(group=16), dict(group=48), dict(group=0), dict(group=-32), dict(group=128), dict(page_size=8),
       dict(page_size=1), dict(page_size=24), dict(page_size=512), dict(d_head=48), dict(d_head=256),
       dict(n_kv_heads=3), dict(n_prompts=0), dict(n_prefix=-1), dict(n_rows=0), dict(max_new=0), dict(dtype=7)]


@pytest.mark.parametrize("bad", BAD, ids=lambda b: "-".join(f"{k}{v}" for k, v in b.items()))
def test_invalid_shapes_are_rejected_without_a_gpu(api, bad):
    pb = _pb(api, **bad)
    assert api.q4_workspace_size(pb) == 0 and pb.prefix_bytes == 0 and pb.pool_bytes == 0
    L, g, fake = api.lib(), pb.group, ctypes.c_void_p(256)
    p = pb.c_shape
    want = api.KVE_EDTYPE if "dtype" in bad else api.KVE_EINVAL
    assert L.q4_pack(p, g, fake, fake, 1 << 20, 1 << 16, 1 << 10, fake, fake, None) == want
    assert L.q4_append(p, g, fake, fake, 1 << 20, 1 << 20, fake, fake, None) == want
    assert L.q4_unpack(p, g, fake, None, fake, 10, fake, fake, 1 << 20, 1 << 16, 1 << 10, None) == want
    assert L.q4_attention(p, g, fake, 1 << 20, *[fake] * 10, 1 << 50, None) == want
    assert L.kve_last_error().decode()
    with pytest.raises(api.KveError):
        api.Q4Cache(pb, 1, "cpu")


def test_null_and_unaligned_arguments_are_rejected_without_a_gpu(api):
    pb = _pb(api)
    L, p, fake, odd = api.lib(), pb.c_shape, ctypes.c_void_p(256), ctypes.c_void_p(264)

    def refused(f, good, changes):
        for i, v in changes:
            args = list(good)
            args[i] = v
            assert f(*args, None) == api.KVE_EINVAL, (i, v)

    head = 100 * 64
    refused(L.q4_pack, [p, 32, fake, fake, 2 * head, head, 64, None, fake],
            ((0, None), (2, None), (3, None), (8, None), (2, odd), (3, odd), (8, odd), (4, 32), (5, 4), (6, 60),
             (6, 1 << 40)))
    row = 2 * 64
    refused(L.q4_append, [p, 32, fake, fake, row, row, fake, fake],
            ((0, None), (2, None), (3, None), (6, None), (7, None), (2, odd), (3, odd), (7, odd), (4, row - 8),
             (5, row + 4)))
    refused(L.q4_unpack, [p, 32, fake, None, None, 100, fake, fake, 2 * head, head, 64],
            ((0, None), (2, None), (6, None), (7, None), (2, odd), (6, odd), (7, odd), (3, fake), (5, 0), (5, 101),
             (5, -1), (8, 32), (9, head + 4), (10, 32)))
    refused(L.q4_unpack, [p, 32, fake, fake, fake, 80, fake, fake, 2 * head, head, 64], ((4, None), (5, 81)))
    none = _pb(api, n_prefix=0).c_shape
    assert L.q4_pack(none, 32, fake, fake, 128, 64, 64, None, fake, None) == api.KVE_EINVAL
    assert L.q4_unpack(none, 32, fake, None, None, 1, fake, fake, 128, 64, 64, None) == api.KVE_EINVAL
    good = [p, 32, fake, 8 * 64, fake, None] + [fake] * 6 + [None, fake, 1 << 40]
    refused(L.q4_attention, good,
            ((0, None), (2, None), (2, odd), (3, 8 * 64 - 8), (3, 8 * 64 + 4), (4, None), (4, odd), (6, None),
             (6, odd), (7, None), (8, None), (9, None), (10, None), (11, None), (11, odd), (13, odd)))
    for i, v in ((13, None), (14, api.q4_workspace_size(pb) - 1)):
        args = list(good)
        args[i] = v
        assert L.q4_attention(*args, None) == api.KVE_EWORKSPACE


def test_injected_failures_reach_every_call(api):
    pb = _pb(api)
    L, p, fake = api.lib(), pb.c_shape, ctypes.c_void_p(256)
    api.kve_inject_failure(api.KVE_ECUDA, 4)
    assert L.q4_pack(p, 32, fake, fake, 12800, 6400, 64, None, fake, None) == api.KVE_ECUDA
    assert L.q4_append(p, 32, fake, fake, 128, 128, fake, fake, None) == api.KVE_ECUDA
    assert L.q4_unpack(p, 32, fake, None, None, 100, fake, fake, 12800, 6400, 64, None) == api.KVE_ECUDA
    assert L.q4_attention(p, 32, fake, 512, *[fake] * 10, 1 << 40, None) == api.KVE_ECUDA
    api.kve_inject_failure(0, 0)


def test_binding_checks_tensors_against_the_shape(api):
    pb = _pb(api)
    bf, n = torch.bfloat16, pb.n_rows
    i = lambda k: torch.zeros(k, dtype=torch.int32)  # noqa: E731
    u8 = lambda k: torch.zeros(k, dtype=torch.uint8)  # noqa: E731
    kp, new = torch.zeros(2, 2, 100, 64, dtype=bf), torch.zeros(n, 6, 64, dtype=bf)[:, 2:4]
    prefix, pages = u8(pb.prefix_bytes), u8(pb.pool_bytes)
    q, own = torch.zeros(n, 8, 64, dtype=bf), torch.zeros(6, 2, 80, 64, dtype=bf)
    calls = [
        (lambda: api.q4_pack(pb, kp[:, :, :99], kp, None, prefix), "elements"),
        (lambda: api.q4_pack(pb, kp.float(), kp, None, prefix), "dtype"),
        (lambda: api.q4_pack(pb, kp, kp, None, prefix), "CUDA|tensor on"),
        (lambda: api.q4_pack(pb, 16, 16, i(1), 16), "elements"),
        (lambda: api.q4_pack(pb, 16, 16, None, prefix[1:]), "elements"),
        (lambda: api.q4_pack(pb, 16, 16, None, prefix.char()), "dtype"),
        (lambda: api.q4_append(pb, new[:-1], new, i(n), pages), "elements"),
        (lambda: api.q4_append(pb, new.half(), new, i(n), pages), "dtype"),
        (lambda: api.q4_append(pb, 16, 16, i(n - 1), pages), "elements"),
        (lambda: api.q4_append(pb, 16, 16, 16, pages[1:]), "elements"),
        (lambda: api.q4_unpack(pb, prefix[1:], None, None, 16, 16), "elements"),
        (lambda: api.q4_unpack(pb, 16, None, None, kp[:1], kp), "elements"),
        (lambda: api.q4_unpack(pb, 16, 16, i(5), 16, 16), "elements"),
        (lambda: api.q4_unpack(pb, 16, i(6 * 5 - 1), 16, 16, 16), "elements"),
        (lambda: api.q4_unpack(pb, 16, 16, 16, own.float(), own), "dtype"),
        (lambda: api.q4_attention(pb, q[:-1], 16, None, 16, 16, 16, 16, 16, 16, None, None), "elements"),
        (lambda: api.q4_attention(pb, q.half(), 16, None, 16, 16, 16, 16, 16, 16, None, None), "dtype"),
        (lambda: api.q4_attention(pb, 16, prefix[1:], None, 16, 16, 16, 16, 16, 16, None, None), "elements"),
        (lambda: api.q4_attention(pb, 16, 16, i(1), 16, 16, 16, 16, 16, 16, None, None), "elements"),
        (lambda: api.q4_attention(pb, 16, 16, None, pages[1:], 16, 16, 16, 16, 16, None, None), "elements"),
        (lambda: api.q4_attention(pb, 16, 16, None, 16, 16, 16, 16, 16, q[:-1], None, None), "elements"),
    ]
    for call, word in calls:
        with pytest.raises(ValueError, match=word):
            call()
    # K and V of different strides
    wide = torch.zeros(2, 2, 120, 64, dtype=bf)[:, :, :100]
    with pytest.raises(ValueError):
        api.q4_pack(pb, kp, wide, None, prefix)


@pytest.mark.parametrize("way", ["copy", "deepcopy", "pickle"])
def test_a_problem_can_be_copied_and_sent(api, way):
    pb = _pb(api, group=64)
    pb.pool_bytes, pb.c_address  # an address of this object is not carried over
    other = {"copy": copy.copy, "deepcopy": copy.deepcopy,
             "pickle": lambda x: pickle.loads(pickle.dumps(x))}[way](pb)
    assert other == pb and other.group == 64 and other.pool_bytes == pb.pool_bytes
    assert other.c_address != pb.c_address
