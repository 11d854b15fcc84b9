"""Each way through pg_attention by name: the cases say which kernels they are for, the profiling scopes say
which ran, and the results stand against the fp64 oracle within test_gpu_pages' bound (fp32 products of three
tf32 products add 2^-21 of each, 8 2^-24 mag a score, to what that bound counts for the sum of d of them; its
d 2^-24 mag holds the worst case of d roundings of one sign)."""
import dataclasses

import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import api
from test_gpu_pages import DEV, DT, Case, f64, ids

pytestmark = pytest.mark.gpu

# kernels per stage of a call
DIRECT = {"pg_own": 1}                                  # a warp per request and KV head does all
LINE = {"pg_own": 1, "pg_join": 1}                      # prompts and own rows dealt to warps
LINE_TC = {"pg_own": 2, "pg_join": 1}                   # and own rows of many new rows on tcgen05
BESIDE = {"pg_prompt": 1, "pg_join": 1}                 # own rows in the idle warps of the prompt's kernel
SPLIT = {"pg_prompt": 1, "pg_own": 1, "pg_join": 1}     # the prompt on tcgen05, own rows dealt to warps
SPLIT_TC = {"pg_prompt": 1, "pg_own": 2, "pg_join": 1}  # and own rows of many new rows on tcgen05


def way(c):
    """Runs c and returns (kernels per stage, out, lse)."""
    api.kve_profile_report()
    api.kve_profile_enable(True)
    try:
        out, lse = c.run()
    finally:
        api.kve_profile_enable(False)
    return {k: v["kernels"] for k, v in api.kve_profile_report().items()}, out, lse


def some(c, n=24):
    """At most n packed rows, the first and the last among them."""
    rng = np.random.default_rng(0)
    return {0, c.rows - 1} | set(rng.integers(0, c.rows, n).tolist()) if c.rows > n else None


def check(c, want):
    got, out, lse = way(c)
    assert got == want
    ref = c.check(some(c))
    assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    return out, lse


def rows_of_others_stay(c, want):
    """Rows of nobody, and rows whose request is not the one that q_start gives."""
    _, ref, z = way(c)
    keep = c.row_req.copy()
    c.row_req[keep == 1] = -1
    c.row_req[keep == 2] = 0
    got, out, lse = way(c)
    assert got == want
    hit = torch.as_tensor((keep == 1) | (keep == 2) | (keep < 0), device=DEV)
    assert (out[hit] == 3.0).all() and (lse[hit] == 5.0).all()
    assert torch.equal(out[~hit], ref[~hit]) and torch.equal(lse[~hit], z[~hit])


# dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi
OWN_ROWS_BESIDE = [
    ("f16", 2, 4, 16, 16, 128, 3000, 8, 6, 1), ("bf16", 8, 2, 16, 8, 128, 3000, 16, 15, 1),
    ("f16", 1, 2, 4, 1, 128, 5000, 1, 5, 2), ("f16", 1, 5, 64, 1, 128, 20000, 2, 3, 1),
    ("bf16", 2, 3, 8, 2, 64, 9000, 8, 6, 2), ("bf16", 1, 4, 4, 4, 64, 3000, 2, 5, 1),
    ("f16", 4, 4, 32, 8, 64, 8000, 8, 7, 1), ("f16", 3, 2, 6, 3, 64, 7000, 1, 20, 1),
    ("bf16", 8, 4, 16, 8, 32, 3000, 4, 7, 1), ("f16", 1, 6, 4, 4, 32, 4000, 4, 8, 2),
]


@pytest.mark.parametrize("case", OWN_ROWS_BESIDE, ids=ids)
def test_own_rows_in_the_prompt_kernel(case):
    """The lookahead's shape; prompts of no length among the others, requests without rows, strided inputs,
    rows that see nothing of their own, rows of nobody and of another request."""
    check(Case(*case, seed=60), BESIDE)
    c = Case(*case, seed=61, ragged=True, idle=0.2, stride=True)
    c.plen.mul_((torch.arange(case[1], device=DEV) != case[1] // 2).to(torch.int32))
    c.np_plen = c.plen.tolist()
    check(c, BESIDE)
    check(Case(*case, seed=62, nothing=True, ragged=True), BESIDE)
    rows_of_others_stay(Case(*case, seed=63), BESIDE)


PROMPT_TILES = [
    (("bf16", 1, 9, 7, 1, 128, 400, 32, 300, 9), SPLIT_TC),   # 7 query heads per KV head: 18 new rows a tile
    (("f16", 1, 3, 64, 1, 128, 300, 16, 60, 2), SPLIT),       # 64: 2
    (("f16", 1, 2, 128, 1, 32, 300, 2, 30, 2), SPLIT),        # 128: 1, four tiles in pairs
    (("bf16", 1, 2, 128, 1, 128, 290, 16, 70, 1), SPLIT),     # a pair
    (("bf16", 1, 70, 8, 2, 64, 300, 16, 20, 1), SPLIT),       # 4: 280 rows a KV head, three tiles
    (("bf16", 2, 5, 28, 4, 64, 270, 16, 300, 3), SPLIT),
    (("f16", 1, 400, 8, 2, 32, 700, 16, 150, 1), SPLIT),      # 13 tiles in pairs
]


@pytest.mark.parametrize("case,want", PROMPT_TILES, ids=lambda x: ids(x) if isinstance(x, tuple) else "")
def test_tiles_of_any_head_count(case, want):
    check(Case(*case, seed=64), want)
    check(Case(*case, seed=65, ragged=True, idle=0.2, stride=True), want)
    check(Case(*case, seed=66, ragged=True, nothing=True), want)
    rows_of_others_stay(Case(*case, seed=67), want)


SHORT_PROMPTS = [
    (("f16", 1, 3, 64, 1, 128, 140, 16, 60, 2), LINE), (("bf16", 1, 9, 7, 1, 128, 129, 32, 300, 9), LINE_TC),
    (("f16", 1, 64, 4, 2, 128, 164, 16, 100, 1), LINE),
]


@pytest.mark.parametrize("case,want", SHORT_PROMPTS, ids=lambda x: ids(x) if isinstance(x, tuple) else "")
def test_short_prompts_in_line_with_the_own_rows(case, want):
    check(Case(*case, seed=68), want)
    check(Case(*case, seed=69, ragged=True, idle=0.2, stride=True), want)
    rows_of_others_stay(Case(*case, seed=70), want)


@pytest.mark.parametrize("case", [("bf16", 1, 70, 8, 2, 64, 128, 16, 20, 1), ("f16", 1, 2, 128, 1, 32, 100, 2, 30, 2),
                                  ("bf16", 1, 33, 4, 4, 64, 5, 4, 9, 1)], ids=ids)
def test_one_launch(case):
    check(Case(*case, seed=71), DIRECT)
    check(Case(*case, seed=72, ragged=True, idle=0.2, stride=True), DIRECT)
    rows_of_others_stay(Case(*case, seed=73), DIRECT)


@pytest.mark.parametrize("n", [0, 300])
def test_fp32_is_one_line(n):
    check(Case("f32", 2, 5, 10, 2, 64, n, 8, 70, 3, seed=74, ragged=True, idle=0.2), LINE)


@pytest.mark.parametrize("n,want", [(500, SPLIT), (20, DIRECT), (200, LINE)])
def test_rows_of_a_refused_request_in_front_of_the_others(n, want):
    """300 packed rows of a request that was refused, far more than max_new; every other row by the module's
    bound."""
    pad, own = 300, 150 if want is LINE else 90
    c = Case("bf16", 1, 6, 8, 2, 128, n, 16, 20 if want is DIRECT else own, 4, seed=75)
    mine = int((c.row_req == 0).sum())
    c.q = torch.cat((torch.full((pad, 8, 128), float("nan"), dtype=DT["bf16"], device=DEV), c.q))
    c.q_start = np.concatenate(([0], c.q_start[1:] + pad))
    c.row_req = np.concatenate((np.full(pad, -1), np.where(c.row_req == 0, -1, c.row_req)))
    c.lens[0] -= mine
    c.rows, c.n_rows = c.rows + pad, c.n_rows + pad
    c.shape = (c.n_rows, *c.shape[1:])
    c.pb = dataclasses.replace(c.pb, n_rows=c.n_rows)
    c.ws = torch.empty(api.pg_workspace_size(c.pb), dtype=torch.uint8, device=DEV)
    got, out, lse = way(c)
    assert got == want
    c.check(set(range(pad + mine, c.rows)))
    assert (f64(out)[:pad + mine] == 3.0).all() and (f64(lse)[:pad + mine] == 5.0).all()


@pytest.mark.parametrize("case,want", [
    (("bf16", 2, 3, 8, 2, 64, 9000, 8, 6, 2), BESIDE), (("bf16", 2, 5, 28, 4, 64, 270, 16, 300, 3), SPLIT),
    (("bf16", 1, 9, 7, 1, 128, 400, 32, 300, 9), SPLIT_TC), (("bf16", 1, 9, 7, 1, 128, 129, 32, 300, 9), LINE_TC),
    (("bf16", 1, 33, 4, 4, 64, 5, 4, 9, 1), DIRECT), (("f32", 2, 5, 10, 2, 64, 300, 8, 70, 3), LINE),
], ids=lambda x: ids(x) if isinstance(x, tuple) else "")
def test_large_values(case, want):
    """V up to about 2^88: sums of unnormalised weights (2^8 at most) times V stay finite."""
    c = Case(*case, seed=76, ragged=True)
    c.Vp, c.V = c.Vp * 2.0 ** 86, c.V * 2.0 ** 86
    out, _ = check(c, want)
    assert torch.isfinite(out[:c.rows]).all() and out[:c.rows].abs().max() > 2.0 ** 80
