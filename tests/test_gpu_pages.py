"""Shared-prompt decoding on the GPU against the fp64 oracle: the page planner's integers exactly,
the append byte for byte, attention within a bound derived from the roundings of its inputs' type.

Bound of an output component, o = sum_j a_j v_j in exact arithmetic:
  * its own rounding to the type: h |o|, h = finfo.eps / 2 (bf16 2^-8, fp16 2^-11, fp32 2^-24);
  * 16-bit types: each unnormalised weight rounds to the type before it meets V: h sum_j a_j |v_j|;
  * scores: d products summed in fp32 are off by at most d 2^-24 mag (mag = max_j sum_c |q_c k_jc| /
    sqrt d), the scaling to log2 and the subtraction of the running maximum by 4 2^-24 (|s| + |m|)
    <= 8 2^-24 mag, the exponential by 2^-21 relative; a relative error w of every weight moves o by
    at most 2 w sum_j a_j |v_j| (numerator and denominator);
  * sums over n tokens in fp32: 8 sqrt(n) 2^-24 sum_j a_j |v_j| (roundings add like a random walk).
lse: the same w, plus the sum's and its own rounding."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import api, synth
from oracle import shared_prompt as sp
from test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
KD = {"f32": api.KVE_F32, "bf16": api.KVE_BF16, "f16": api.KVE_F16}


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def f64(t):
    return t.double().cpu().numpy()


# ---- planner ---------------------------------------------------------------------------------------
NAMES = ("len", "pool", "q_start", "row_req", "row_pos", "slot_map", "block_table", "free_pages")


def run_plan(pb, new, lens, pool, free, table, in_place=False, stream=None):
    R, n = pb.requests, pb.n_rows
    new, lens, pool, free, table = (i32(x) for x in (new, lens, pool, free, table))
    out = {"len": lens if in_place else torch.full((R,), -7, dtype=torch.int32, device=DEV),
           "pool": pool if in_place else torch.full((4,), -7, dtype=torch.int32, device=DEV)}
    g = {k: Guarded(s, torch.int32) for k, s in (("q_start", (R + 1,)), ("row_req", (n,)),
                                                  ("row_pos", (n,)), ("slot_map", (n,)))}
    api.pg_plan(pb, new, lens, pool, free, table, out["len"], out["pool"],
                *(g[k].t for k in ("q_start", "row_req", "row_pos", "slot_map")), stream=stream)
    assert all(b.intact() for b in g.values())
    out.update({k: b.t for k, b in g.items()}, block_table=table, free_pages=free)
    return {k: out[k].cpu().numpy() for k in NAMES}


def plan_pb(fan, page, n_pages, max_pages, n_rows, max_new, prompts=1):
    return api.PgProblem(prompts, fan, 1, 1, 128, 0, page, n_pages, max_pages, n_rows, max_new,
                         api.KVE_BF16)


def plan_state(rng, R, page, max_pages, old_hi, new, spare):
    """Lengths, a table of distinct pages, and a ring with `spare` more (or fewer) than wanted."""
    lens = rng.integers(0, old_hi + 1, R)
    have = -(-lens // page)
    want = int((-(-(lens + np.maximum(new, 0)) // page) - have).sum())
    n_free = max(0, want + spare)
    n_pages = int(have.sum()) + n_free + 3
    ids = rng.permutation(n_pages)
    table, at = np.full((R, max_pages), -1), 0
    for r in range(R):
        table[r, :have[r]] = ids[at:at + have[r]]
        at += have[r]
    head = int(rng.integers(n_pages))
    free = np.full(n_pages, -1)
    free[(head + np.arange(n_free)) % n_pages] = ids[at:at + n_free]
    return lens, np.array([head, n_free, 0, 0]), free, table, n_pages


@pytest.mark.parametrize("R,page,old_hi,new_hi,spare,finished", [
    (1, 16, 0, 1, 0, 0.0), (4, 16, 7, 1, 3, 0.0), (3, 1, 5, 4, 0, 0.3), (33, 8, 100, 1, 9, 0.2),
    (512, 16, 4095, 1, 5, 0.1), (100, 64, 300, 40, -20, 0.1), (256, 128, 512, 300, 0, 0.0),
    (1500, 16, 60, 3, -100, 0.2), (5000, 32, 33, 2, 50, 0.3), (16384, 16, 20, 1, -3000, 0.1),
    (17, 16, 50, 2500, 2, 0.0),
])
def test_plan_matches_the_oracle(R, page, old_hi, new_hi, spare, finished):
    rng = np.random.default_rng(R)
    new = rng.integers(0, new_hi + 1, R)
    new[rng.random(R) < finished] = -1
    max_pages = -(-(old_hi + new_hi) // page)
    lens, pool, free, table, n_pages = plan_state(rng, R, page, max_pages, old_hi, new, spare)
    n_rows = int(np.maximum(new, 0).sum()) + int(rng.integers(0, 5)) + 1
    pb = plan_pb(R, page, n_pages, max_pages, n_rows, new_hi)
    want = sp.pg_plan(new, lens, pool, free, table, page, min(new_hi, n_rows), n_rows)
    for in_place in (False, True):
        got = run_plan(pb, new, lens, pool, free, table, in_place)
        for k in NAMES:
            assert np.array_equal(got[k], want[k]), (k, in_place)


def test_plan_refusals_leave_the_request_as_it_was():
    """Too many rows, a full table, lengths out of range, rows past n_rows, an empty ring."""
    rng = np.random.default_rng(3)
    page, max_pages, max_new, n_rows = 4, 3, 6, 12
    cases = [
        ([7, 1, 0], [0, 2, 3]), ([2, 5, 1], [8, 8, 8]), ([1, -1, 0], [-1, 13, 13]),
        ([6, 6, 1], [0, 0, 0]), ([2 ** 31 - 1, 1, 1], [0, 0, 0]), ([6, 5, 2 ** 31 - 1], [1, 1, 1]),
        ([1, 1, 1], [2 ** 31 - 1, -2 ** 31, 4]), ([0, 0, 0], [0, 12, 5]),
        ([-1, -2 ** 31, -5], [12, 0, 3]),
    ]
    for new, lens in cases:
        table = rng.permutation(9).reshape(3, 3)
        for free in (0, 1, 5):
            ring, pool = np.arange(9, 16), np.array([6, free, 0, 0])
            ring = np.concatenate((ring, [0, 0]))
            pb = plan_pb(3, page, 9, max_pages, n_rows, max_new)
            want = sp.pg_plan(new, lens, pool, ring % 9, table, page, max_new, n_rows)
            got = run_plan(pb, new, lens, pool, ring % 9, table)
            for k in NAMES:
                assert np.array_equal(got[k], want[k]), (k, new, lens, free)


def test_plan_runs_a_pool_through_many_steps_in_place():
    rng = np.random.default_rng(4)
    R, page, n_pages, max_pages, max_new, n_rows = 40, 8, 100, 6, 9, 128
    pb = plan_pb(R, page, n_pages, max_pages, n_rows, max_new)
    c = api.PgCache(pb, 1, DEV)
    lens, pool = np.zeros(R, int), np.array([0, n_pages, 0, 0])
    free, table = np.arange(n_pages), np.full((R, max_pages), -1)
    for _ in range(60):
        new = rng.choice([-1, 0, 1, 1, 1, 9, 10], R)
        o = sp.pg_plan(new, lens, pool, free, table, page, max_new, n_rows)
        c.plan(i32(new))
        for k, t in (("len", c.lens), ("pool", c.pool), ("block_table", c.block_table),
                     ("free_pages", c.free_pages), ("slot_map", c.slot_map), ("row_req", c.row_req),
                     ("row_pos", c.row_pos), ("q_start", c.q_start)):
            assert np.array_equal(t.cpu().numpy(), o[k]), k
        lens, pool, free, table = o["len"], o["pool"], o["free_pages"], o["block_table"]


# ---- append ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("rows,heads,d,page,dtype,fused", [
    (1, 1, 32, 1, "bf16", False), (5, 3, 64, 8, "f16", True), (33, 8, 128, 16, "bf16", True),
    (700, 4, 128, 64, "f32", False), (1000, 7, 32, 256, "f32", True),
])
def test_append_stores_rows_and_leaves_the_rest(rows, heads, d, page, dtype, fused):
    gen = torch.Generator(device=DEV).manual_seed(rows)
    n_pages = -(-rows // page) + 2
    pb = api.PgProblem(1, 1, heads, heads, d, 0, page, n_pages, n_pages, rows, rows, KD[dtype])
    wide = torch.randn(rows, 3 * heads if fused else heads, d, generator=gen, device=DEV).to(DT[dtype])
    K_new = wide[:, heads:2 * heads] if fused else wide
    V_new = wide[:, 2 * heads:] if fused else wide * 2
    slots = torch.randperm(n_pages * page, generator=gen, device=DEV)[:rows].to(torch.int32)
    slots[::5] = -1
    K, V = (Guarded((n_pages, heads, page, d), DT[dtype]) for _ in range(2))
    K.t.normal_(generator=gen)
    V.t.normal_(generator=gen)
    wantK, wantV = K.t.clone(), V.t.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            wantK[s // page, :, s % page] = K_new[i]
            wantV[s // page, :, s % page] = V_new[i]
    api.pg_append(pb, K_new, V_new, slots, K.t, V.t)
    api.kve_check_device()
    assert torch.equal(K.t, wantK) and torch.equal(V.t, wantV) and K.intact() and V.intact()
    # a slot outside the pool is skipped and reported
    slots[-1] = n_pages * page
    api.pg_append(pb, K_new, V_new, slots, K.t, V.t)
    with pytest.raises(api.KveError, match="slot or page id"):
        api.kve_check_device()
    api.kve_check_device()
    assert torch.equal(K.t, wantK) and torch.equal(V.t, wantV) and K.intact() and V.intact()


# ---- attention -------------------------------------------------------------------------------------
class Case:
    """Inputs of one attention call: random lengths, rows and pages; NaN wherever no row may look."""

    def __init__(self, dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi, ragged=False, seed=0,
                 idle=0.0, nothing=False, stride=False, scale=1.0, new=None):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device=DEV).manual_seed(seed)
        dt, R = DT[dtype], S * F
        self.dtype, self.F = dtype, F
        nq = rng.integers(1, new_hi + 1, R)
        nq[rng.random(R) < idle] = 0
        if new is not None:
            nq = np.asarray(new)
        own = rng.integers(0, own_hi + 1, R)
        lens = own + nq
        if nothing:
            lens = np.minimum(lens, rng.integers(0, 2, R))  # rows without anything to see
        max_pages = max(1, -(-(own_hi + new_hi) // page)) + 1
        have = -(-lens // page)
        n_pages = int(have.sum()) + 2
        ids = rng.permutation(n_pages)
        table = np.full((R, max_pages), 2 ** 31 - 1)  # entries behind a request's pages: anything
        K = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=dt, device=DEV)
        V = K.clone()
        at = 0
        for r in range(R):
            for j in range(have[r]):
                p, cnt = int(ids[at]), int(min(page, lens[r] - j * page))
                table[r, j] = p
                K[p, :, :cnt] = torch.randn(Hkv, cnt, d, generator=gen, device=DEV).to(dt)
                V[p, :, :cnt] = torch.randn(Hkv, cnt, d, generator=gen, device=DEV).to(dt)
                at += 1
        plen = rng.integers(0, n + 1, S) if ragged else np.full(S, n)
        extra = 5 if stride else 0
        self.Kp = torch.full((S, 2 if stride else 1, Hkv, n + extra, d), float("nan"), dtype=dt,
                             device=DEV)
        self.Vp = self.Kp.clone()
        for s in range(S):
            self.Kp[s, 0, :, :plen[s]] = torch.randn(Hkv, int(plen[s]), d, generator=gen,
                                                     device=DEV).to(dt)
            self.Vp[s, 0, :, :plen[s]] = torch.randn(Hkv, int(plen[s]), d, generator=gen,
                                                     device=DEV).to(dt)
        self.Kp, self.Vp = self.Kp[:, 0, :, :n], self.Vp[:, 0, :, :n]
        if not stride:
            self.Kp, self.Vp = self.Kp.contiguous(), self.Vp.contiguous()
        q_start = np.concatenate(([0], nq.cumsum()))
        rows = int(q_start[-1])
        self.rows, self.n_rows = rows, rows + 3
        row_req = np.full(self.n_rows, -1)
        row_req[:rows] = np.repeat(np.arange(R), nq)
        wide = torch.randn(self.n_rows, Hq + (2 * Hkv if stride else 0), d, generator=gen, device=DEV)
        wide *= scale
        wide[rows:] = float("nan")
        self.q = wide.to(dt)[:, :Hq]
        self.K, self.V, self.plen, self.np_plen = K, V, i32(plen) if ragged else None, plen
        self.table, self.lens, self.q_start, self.row_req = table, lens, q_start, row_req
        self.pb = api.PgProblem(S, F, Hq, Hkv, d, n, page, n_pages, max_pages, self.n_rows, new_hi,
                                KD[dtype])
        self.shape = (self.n_rows, Hq, d)
        self.ws = torch.full((api.pg_workspace_size(self.pb),), 0xFF, dtype=torch.uint8, device=DEV)

    def args(self):
        return (self.K, self.V, i32(self.table), i32(self.lens), i32(self.q_start),
                i32(self.row_req))

    def run(self, lse=True, stream=None):
        out, z = Guarded(self.shape, DT[self.dtype]), Guarded(self.shape[:2], torch.float32)
        out.t.fill_(3.0)
        z.t.fill_(5.0)
        ws = Guarded((self.ws.numel(),), torch.uint8)
        ws.t.fill_(0xFF)
        api.pg_attention(self.pb, self.q, self.Kp, self.Vp, self.plen, *self.args(), out.t,
                         z.t if lse else None, ws.t, stream=stream)
        api.kve_check_device(stream)
        assert out.intact() and z.intact() and ws.intact()
        return out.t, z.t

    def oracle(self, rows=None):
        return sp.pg_attention(f64(self.q), f64(self.Kp), f64(self.Vp), self.np_plen, f64(self.K),
                               f64(self.V), np.where(self.table > 2 ** 30, 0, self.table), self.lens,
                               self.q_start, self.F, rows)

    def check(self, rows=None):
        out, lse = self.run()
        ref = self.oracle(rows)
        live = ~np.isnan(ref["lse"])
        assert live.any() or self.rows == 0
        if rows is None:
            assert live[:self.rows].all()
        h = torch.finfo(DT[self.dtype]).eps / 2
        d, n = self.shape[2], self.pb.n_prefix + int(self.lens.max())
        w = (d + 8) * U * ref["mag"] + 2.0 ** -21
        tol = (2 * w + 8 * math.sqrt(n) * U + (h if self.dtype != "f32" else 0))[..., None]
        tol = tol * ref["terms"] * (1 + h) + h * np.abs(ref["out"])
        if self.dtype == "f16":
            tol = tol + 2.0 ** -25  # half a step of the smallest fp16 numbers
        got = f64(out)
        bad = live[..., None] & ~(np.abs(got - ref["out"]) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref["out"])[bad][:5], tol[bad][:5])
        z = f64(lse)
        zt = w + 8 * math.sqrt(n) * U + 4 * U * np.abs(np.where(np.isinf(ref["lse"]), 0, ref["lse"]))
        inf = live & np.isinf(ref["lse"])
        assert np.isneginf(z[inf]).all()
        fin = live & ~inf
        assert (np.abs(z[fin] - ref["lse"][fin]) <= zt[fin]).all()
        # rows of nobody
        assert (got[self.rows:] == 3.0).all() and (z[self.rows:] == 5.0).all()
        return out, lse


SMALL = [
    # dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi
    ("f32", 1, 4, 1, 1, 64, 512, 16, 7, 1),
    ("f32", 2, 3, 6, 2, 128, 77, 8, 40, 5),
    ("f32", 1, 1, 4, 4, 32, 1, 1, 3, 1),
    ("bf16", 1, 4, 8, 2, 128, 1000, 16, 7, 1),
    ("bf16", 2, 5, 10, 2, 128, 300, 16, 150, 1),      # 5 query heads per KV head
    ("bf16", 1, 9, 7, 1, 128, 129, 32, 300, 9),       # 7 per KV head, several new rows
    ("bf16", 1, 70, 8, 2, 64, 128, 16, 20, 1),        # 280 rows a KV head: several tiles of rows
    ("bf16", 3, 2, 4, 1, 32, 260, 64, 33, 3),
    ("f16", 1, 64, 4, 2, 128, 164, 16, 100, 1),
    ("f16", 2, 2, 6, 6, 64, 511, 128, 500, 70),       # one query head per KV head
    ("f16", 1, 3, 64, 1, 128, 140, 16, 60, 2),        # 64 per KV head
    ("f16", 1, 2, 128, 1, 32, 100, 2, 30, 2),         # 128 per KV head
    ("bf16", 1, 33, 4, 4, 64, 5, 4, 9, 1),            # a prompt shorter than any tile
]
ids = lambda c: "-".join(map(str, c))  # noqa: E731


@pytest.mark.parametrize("case", SMALL, ids=ids)
def test_attention_matches_the_oracle(case):
    Case(*case, seed=1).check()


@pytest.mark.parametrize("case", SMALL[1::2], ids=ids)
def test_ragged_prompts_idle_requests_and_strided_inputs(case):
    """Prompts of any length from 0, requests without rows, q out of a wider projection, the prompt
    as a slice of a larger cache; NaN behind every length."""
    for seed in (2, 3):
        Case(*case, seed=seed, ragged=True, idle=0.3, stride=True).check()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("f16", 64), ("bf16", 32)])
def test_a_prompt_stored_row_by_row_with_all_heads(dtype, d):
    """K and V as [prompt][row][head][d]: the head stride is smaller than the row's."""
    c = Case(dtype, 2, 3, 6, 3, d, 333, 16, 20, 2, seed=14, ragged=True)
    ref = c.run()
    c.Kp, c.Vp = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.Kp, c.Vp))
    assert c.Kp.stride(1) < c.Kp.stride(2)
    got = c.check()
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_many_requests_of_very_different_lengths(dtype):
    """700 requests, most without rows or nearly so, a few long: the same rows whichever requests
    stand around them."""
    c = Case(dtype, 1, 700, 4, 2, 64, 40, 16, 12, 2, seed=15, idle=0.5)
    c.check(set(range(0, c.rows, 37)))
    c = Case(dtype, 7, 20, 4, 2, 64, 40, 16, 3000, 1, seed=16, idle=0.8, ragged=True)
    c.check(set(range(0, c.rows, 5)) | {c.rows - 1})


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_that_see_nothing_are_zero(dtype):
    c = Case(dtype, 2, 6, 4, 2, 64, 0, 8, 5, 4, seed=5, nothing=True)
    out, lse = c.check()
    assert torch.isneginf(lse[:c.rows]).any()
    Case(dtype, 3, 4, 4, 2, 128, 40, 8, 5, 4, seed=6, nothing=True, ragged=True).check()
    Case(dtype, 2, 3, 4, 2, 128, 300, 8, 0, 1, seed=7, idle=1.0).run()  # no rows at all


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_peaked_scores(dtype):
    """Queries 12 times as long: the running maximum moves by tens of powers of two on the way."""
    Case(dtype, 1, 6, 8, 2, 128, 700, 16, 300, 2, seed=8, scale=12.0).check()


# requests of one new row beside requests of many: both ways of the own rows in one batch
MANY_NEW = [
    ("bf16", 1, 5, 10, 2, 128, 200, 16, 300, 64), ("f16", 2, 3, 8, 1, 64, 130, 4, 200, 33),
    ("bf16", 1, 4, 4, 1, 32, 90, 1, 40, 50), ("f16", 1, 3, 6, 2, 128, 0, 256, 700, 100),
    ("bf16", 1, 2, 128, 2, 64, 70, 32, 150, 3), ("bf16", 3, 4, 3, 3, 128, 33, 128, 257, 130),
]


@pytest.mark.parametrize("case", MANY_NEW, ids=ids)
def test_many_new_rows_beside_few(case):
    Case(*case, seed=17).check()
    c = Case(*case, seed=18, ragged=True, idle=0.2, stride=True)
    c.check()
    Case(*case, seed=19, nothing=True).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [1, 40])
def test_many_requests_with_several_blocks_of_rows_each(dtype, S):
    """17 to 20 new rows each, without a prompt and behind a short one: every unit has its place."""
    rng = np.random.default_rng(29)
    new = rng.integers(17, 21, 200)
    for n in (0, 7):
        c = Case(dtype, S, 200 // S, 8, 8, 32, n, 16, 5, 20, seed=29, new=new)
        c.check(set(range(0, c.rows, 61)) | {c.rows - 1})


@pytest.mark.parametrize("dtype,n", [("f32", 400), ("bf16", 180), ("f16", 600)])
@pytest.mark.parametrize("new", [1, 5])
def test_prompts_and_requests_without_tokens_between_others(dtype, n, new):
    """A prompt of no length with rows behind it, and requests with rows but nothing in their pages, in the
    middle of the line of work: the results behind them are the right ones."""
    c = Case(dtype, 4, 5, 6, 2, 64, n, 16, 90, new, seed=41, ragged=True)
    c.plen[1] = c.plen[2] = 0
    c.np_plen = c.plen.tolist()
    c.lens[[1, 6, 7, 8, 13]] = 0
    c.check()
    c.plen[:] = 0
    c.np_plen = c.plen.tolist()
    c.check()


# little enough for one warp per request and KV head, which writes the output itself
BRIEF = [
    # dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi
    ("bf16", 1, 9, 32, 8, 128, 20, 16, 15, 1), ("f16", 3, 5, 8, 1, 128, 3, 8, 40, 1),
    ("bf16", 2, 60, 28, 4, 64, 40, 1, 30, 1), ("f16", 1, 33, 16, 16, 32, 100, 2, 20, 7),
    ("bf16", 2, 7, 16, 1, 128, 17, 32, 9, 1),      # 16 query heads per KV head
    ("f16", 1, 30, 10, 2, 64, 0, 4, 60, 3),        # up to 15 query rows, no prompt
    ("bf16", 5, 4, 3, 1, 32, 16, 16, 16, 5),
]


@pytest.mark.parametrize("case", BRIEF, ids=ids)
def test_brief_work(case):
    for seed in (30, 31):
        c = Case(*case, seed=seed, ragged=seed == 31, idle=0.2 if seed == 31 else 0.0,
                 stride=seed == 31)
        out, lse = c.check()
        b, z = c.run()
        assert torch.equal(out, b) and torch.equal(lse, z)
        assert torch.equal(out, c.run(lse=False)[0])
    Case(*case, seed=32, nothing=True).check()
    # rows whose request is not the one that q_start gives, and of nobody, stay
    c = Case(*case, seed=33)
    ref, _ = c.run()
    keep = c.row_req.copy()
    c.row_req[keep == 1] = -1
    c.row_req[keep == 2] = 0
    out, lse = c.run()
    hit = torch.as_tensor((keep == 1) | (keep == 2) | (keep < 0), device=DEV)
    assert (out[hit] == 3.0).all() and (lse[hit] == 5.0).all()
    assert torch.equal(out[~hit], ref[~hit])


@pytest.mark.parametrize("case", [
    ("bf16", 3, 60, 12, 4, 128, 2, 16, 2, 57),      # up to 171 query rows: blocks of 16
    ("f16", 1, 300, 16, 8, 64, 100, 16, 150, 2), ("bf16", 2, 100, 28, 4, 32, 33, 8, 60, 5),
], ids=ids)
def test_brief_work_of_many_requests(case):
    """More warps than the GPU holds at a time, several blocks of rows per request."""
    for kw in (dict(seed=38), dict(seed=39, ragged=True, idle=0.3, stride=True), dict(seed=40, nothing=True)):
        c = Case(*case, **kw)
        out, _ = c.check(set(range(0, c.rows, max(1, c.rows // 25))) | {c.rows - 1})
        assert torch.isfinite(out[:c.rows].float()).all()


@pytest.mark.parametrize("case", [
    ("bf16", 1, 4, 8, 2, 128, 3000, 16, 14, 1), ("f16", 3, 3, 8, 1, 64, 1500, 4, 20, 2),
    ("bf16", 5, 2, 12, 4, 32, 800, 1, 20, 3), ("f16", 2, 4, 16, 16, 128, 700, 8, 12, 1),
], ids=ids)
def test_few_own_rows_behind_long_prompts(case):
    """The lookahead's shape: tables of at most 32 rows; prompts of no length among them, requests
    without rows, rows that see nothing of their own, rows of nobody and of another request."""
    for seed in (34, 35):
        c = Case(*case, seed=seed, ragged=True, idle=0.2, stride=seed == 34)
        assert c.pb.max_pages * c.pb.page_size <= 32
        c.plen.mul_((torch.arange(case[1], device=DEV) != 1).to(torch.int32))
        c.np_plen = c.plen.tolist()
        c.check()
    Case(*case, seed=36, nothing=True, ragged=True).check()
    c = Case(*case, seed=37)
    ref, _ = c.run()
    keep = c.row_req.copy()
    c.row_req[keep == 1] = -1
    c.row_req[keep == 2] = 0
    out, lse = c.run()
    hit = torch.as_tensor((keep == 1) | (keep == 2) | (keep < 0), device=DEV)
    assert (out[hit] == 3.0).all() and (lse[hit] == 5.0).all()
    assert torch.equal(out[~hit], ref[~hit])


LONG = [("bf16", 1, 4, 32, 8, 128, 16384, 16, 7, 1), ("f16", 2, 3, 8, 2, 64, 9001, 16, 5000, 1),
        ("bf16", 1, 2, 5, 1, 128, 3, 256, 20000, 2), ("f32", 1, 2, 4, 2, 64, 4000, 16, 3000, 2),
        ("bf16", 1, 300, 8, 2, 128, 2500, 64, 700, 1), ("bf16", 2, 4, 10, 2, 128, 4100, 32, 600, 64)]


@pytest.mark.parametrize("case", LONG, ids=ids)
def test_long_prompts_and_long_own_rows(case):
    c = Case(*case, seed=9, ragged=True)
    rng = np.random.default_rng(0)
    c.check(set(rng.integers(0, c.rows, 4).tolist()) | {0, c.rows - 1})


def test_attention_without_lse_and_bitwise_repeatable():
    c = Case("bf16", 1, 8, 8, 2, 128, 3000, 16, 600, 2, seed=10)
    a, z = c.run()
    for _ in range(3):
        b, z2 = c.run()
        assert torch.equal(a, b) and torch.equal(z, z2)
    assert torch.equal(a, c.run(lse=False)[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_page_ids_outside_the_pool_are_reported(dtype):
    """Read as page 0, recorded, and the other requests' rows are what they were."""
    c = Case(dtype, 1, 4, 4, 2, 64, 64, 8, 30, 2, seed=11)
    a, _ = c.run()
    c.K[0].nan_to_num_(0.0)
    c.V[0].nan_to_num_(0.0)
    c.table[1, 0] = c.pb.n_pages
    with pytest.raises(api.KveError, match="page id"):
        c.run()
    c.table[1, 0] = -1
    with pytest.raises(api.KveError, match="page id"):
        c.run()
    out = torch.full(c.shape, 3.0, dtype=DT[dtype], device=DEV)
    api.pg_attention(c.pb, c.q, c.Kp, c.Vp, c.plen, *c.args(), out, None, c.ws)
    with pytest.raises(api.KveError):
        api.kve_check_device()
    other = torch.as_tensor(c.row_req != 1, device=DEV)
    assert torch.equal(a[other], out[other])


def test_refused_and_mismatched_rows_are_left_alone():
    """row_req < 0 inside the batch (a refused request that packed more rows than max_new), and a
    row_req that q_start contradicts: those rows stay, the others are right."""
    c = Case("bf16", 1, 6, 8, 2, 128, 500, 16, 90, 4, seed=12)
    ref, _ = c.run()
    keep = c.row_req.copy()
    c.row_req[keep == 2] = -1
    c.row_req[keep == 4] = 3
    out, _ = c.run()
    hit = np.isin(keep, (2, 4))
    assert (f64(out)[hit] == 3.0).all()
    live = torch.as_tensor((keep >= 0) & ~hit, device=DEV)
    assert torch.equal(out[live], ref[live])
    # 300 rows of a refused request in front of the others
    pad = 300
    c2 = Case("bf16", 1, 6, 8, 2, 128, 500, 16, 90, 4, seed=12)
    c2.q = torch.cat((torch.zeros(pad, 8, 128, dtype=torch.bfloat16, device=DEV), c2.q))
    c2.q_start = np.concatenate(([0], c2.q_start[1:] + pad))
    c2.row_req = np.concatenate((np.full(pad, -1), np.where(c2.row_req == 0, -1, c2.row_req)))
    c2.lens[0] -= (keep == 0).sum()
    c2.n_rows += pad
    c2.shape = (c2.n_rows, 8, 128)
    c2.pb = api.PgProblem(1, 6, 8, 2, 128, 500, 16, c2.pb.n_pages, c2.pb.max_pages, c2.n_rows, 4,
                          api.KVE_BF16)
    c2.ws = torch.empty(api.pg_workspace_size(c2.pb), dtype=torch.uint8, device=DEV)
    out, _ = c2.run()
    live = torch.as_tensor(c2.row_req > 0, device=DEV)
    assert (f64(out)[c2.row_req < 0] == 3.0).all()
    got, want = f64(out[live]), f64(ref[live[pad:]])
    assert np.abs(got - want).max() <= 2 ** -6 * np.abs(want).max()  # other splits, same rows


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pad,g", [(7, 1), (40, 3)])
def test_a_refused_request_with_most_of_the_rows(dtype, pad, g):
    """Its rows stand in front of all others' in the packed arrays, more than a step may add for a
    request and more than all others together."""
    c = Case(dtype, 2, 2, 2 * g, 2, 64, 50, 8, 30, 1, seed=20)
    c.q = torch.cat((torch.full_like(c.q[:1], float("nan")).expand(pad, -1, -1), c.q))
    c.q_start = np.concatenate(([0], c.q_start[1:] + pad))
    c.row_req = np.concatenate((np.full(pad + 1, -1), c.row_req[1:]))
    c.lens[0] -= 1
    c.rows, c.n_rows = c.rows + pad, c.n_rows + pad
    c.shape = (c.n_rows, *c.shape[1:])
    c.pb = dataclasses.replace(c.pb, n_rows=c.n_rows)
    c.ws = torch.empty(api.pg_workspace_size(c.pb), dtype=torch.uint8, device=DEV)
    out, lse = c.check(set(range(pad + 1, c.rows)))
    assert (f64(out)[:pad + 1] == 3.0).all() and (f64(lse)[:pad + 1] == 5.0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_one_request_with_most_of_the_rows(dtype):
    """700 new rows of one request among 12: more than four times its even share, of which the
    launches on the tensor cores have places for."""
    new = np.ones(12, int)
    new[3] = 700
    c = Case(dtype, 6, 2, 8, 2, 64, 150, 16, 40, 700, seed=21, new=new)
    c.check({0, 2, 3, 4, 66, 67, 260, 261, 511, 514, 701, 702, 703, 710})


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_requests_that_share_pages(dtype):
    """A fork: both requests' block tables name the same pages, the second up to the middle of one."""
    c = Case(dtype, 1, 4, 4, 2, 128, 60, 8, 60, 3, seed=22)
    c.lens[0] = max(c.lens)
    c.table[0] = c.table[np.argmax(c.lens[1:]) + 1]
    c.table[1], c.lens[1] = c.table[0], max(1, c.lens[0] - 3)
    c.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_most_requests(dtype):
    c = Case(dtype, 64, 256, 4, 2, 32, 20, 4, 2, 2, seed=23, idle=0.96, ragged=True)
    assert c.pb.requests == 16384
    c.check(set(range(0, c.rows, 41)) | {c.rows - 1})


def test_small_fp16_weights_do_not_vanish():
    """One token far above the rest, which have 2^-25.5 of its weight each: rounded to fp16 as they
    are they would all be 0. Bound: the module's, and 2^-32 of the largest weight for each of them
    (half a step of the smallest fp16 numbers, 2^-25, with weights carried 2^7 higher)."""
    n, own, d = 16384, 4096, 64
    c = Case("f16", 1, 1, 1, 1, d, n, 16, own - 1, 1, seed=24)
    c.lens[0] = int(c.lens[0])
    for k, v in ((c.Kp, c.Vp), (c.K, c.V)):
        k.zero_()
        v.fill_(1.0)
    c.q[0] = 0.0
    c.q[0, 0, 0] = 8.0 * math.log(2)  # score: k_0 ln 2
    tops = (c.Kp[0, 0, 0], c.K[int(c.table[0, 0]), 0, 0])
    vals = (c.Vp[0, 0, 0], c.V[int(c.table[0, 0]), 0, 0])
    for k, v in zip(tops, vals):
        k[0] = 25.5
        v.zero_()
    out, _ = c.run()
    ref = c.oracle()
    w = (d + 8) * U * ref["mag"][0, 0] + 2.0 ** -21
    h = 2.0 ** -11
    tol = (2 * w + 8 * math.sqrt(n + own) * U + 2 * h) * ref["terms"][0, 0] * (1 + h)
    tol = tol + 2.0 ** -25 + 2.0 ** -32 * (n + own)
    assert ref["out"][0, 0, 0] > 20 * tol[0]
    assert (np.abs(f64(out[0, 0]) - ref["out"][0, 0]) <= tol).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_that_overlap_on_two_streams(dtype):
    """Each with its own workspace: the results are those of the calls one after the other."""
    cs = [Case(dtype, 1, 8, 8, 2, 128, 2000, 16, 300, 1, seed=25),
          Case(dtype, 2, 3, 8, 2, 128, 700, 16, 100, 20, seed=26)]
    want = [c.run() for c in cs]
    args = [c.args() for c in cs]
    outs = [[torch.full_like(w[0], 3.0) for _ in range(10)] for w in want]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for i in range(10):
        for c, a, o, s in zip(cs, args, outs, streams):
            api.pg_attention(c.pb, c.q, c.Kp, c.Vp, c.plen, *a, o[i], None, c.ws, stream=s)
    api.kve_check_device(streams[0])
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w[0], x) for x in o)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("order", ["falling", "same", "wild"])
def test_row_starts_that_are_no_sums_of_lengths_stay_in_bounds(dtype, order):
    """Nothing behind the arrays is written, and rows whose request is not the one that q_start
    gives stay."""
    c = Case(dtype, 2, 20, 8, 2, 64, 90, 8, 60, 12, seed=27)
    rng = np.random.default_rng(0)
    if order == "falling":
        c.q_start = c.q_start[::-1].copy()
    elif order == "same":  # every request claims all rows
        c.q_start = np.where(np.arange(41) % 2, c.rows, 0)
    else:
        c.q_start = rng.integers(-2 ** 31, 2 ** 31, 41)
    start = np.clip(c.q_start, 0, c.n_rows)
    out, lse = c.run()  # (checks the guards)
    at = np.arange(c.n_rows)
    r = np.maximum(c.row_req, 0)
    left = (c.row_req < 0) | (at < start[r]) | (at - start[r] >= np.minimum(start[r + 1] - start[r], 12))
    assert (f64(out)[left] == 3.0).all() and (f64(lse)[left] == 5.0).all()


def test_addresses_and_tensors_that_do_not_fit():
    """Addresses give what tensors give; a tensor that does not fit the shape is named, and nothing
    is written."""
    c = Case("bf16", 2, 3, 8, 2, 64, 120, 8, 40, 2, seed=28, stride=True)
    ref, lse = c.run()
    qk = (c.q, c.Kp, c.Vp, c.plen, *c.args())
    out = torch.full(c.shape, 3.0, dtype=torch.bfloat16, device=DEV)
    z = torch.full(c.shape[:2], 5.0, device=DEV)
    args = [*qk, out, z, c.ws]
    for i in (4, 5, 6, 7, 8, 9, 10, 11):
        call = list(args)
        call[i] = call[i].data_ptr()
        api.pg_attention(c.pb, *call)
        assert torch.equal(out, ref) and torch.equal(z, lse)
        out.fill_(3.0)
        z.fill_(5.0)
    bad = [(0, c.q.float(), "dtype"), (0, c.q[:-1], "elements"), (0, c.q.transpose(0, 1), "contiguous"),
           (1, c.Kp[:, :, :-1], "elements"), (1, c.Kp[..., :32], "elements"), (1, c.Kp.half(), "dtype"),
           (2, c.Vp.contiguous(), "strides differ"), (4, c.K.view(-1)[1:], "elements"),
           (6, args[6].view(-1)[:-1], "elements"), (7, args[7].long(), "dtype"),
           (8, args[8][:-1], "elements"), (9, args[9].cpu(), "CUDA"),
           (10, torch.empty(*c.shape, 2, dtype=torch.bfloat16, device=DEV)[..., 0], "contiguous"),
           (11, z.double(), "dtype"), (11, z[:-1], "elements"), (12, c.ws.cpu(), "CUDA")]
    for i, t, word in bad:
        call = list(args)
        call[i] = t
        with pytest.raises(ValueError, match=word):
            api.pg_attention(c.pb, *call)
    with pytest.raises(api.KveError, match="workspace"):
        api.pg_attention(c.pb, *args[:12], c.ws[:-256])
    with pytest.raises(api.KveError, match="null"):
        api.pg_attention(c.pb, *args[:10], None, *args[11:])
    api.kve_check_device()
    assert (f64(out) == 3.0).all() and (f64(z) == 5.0).all()


def test_another_stream_and_the_wrong_device(monkeypatch):
    c = Case("bf16", 1, 4, 8, 2, 128, 700, 16, 60, 1, seed=13)
    a, _ = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b, _ = c.run(stream=s)
    assert torch.equal(a, b)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        c.run(stream=s)
    with pytest.raises(ValueError, match="current CUDA device is cuda:1"):
        api.pg_append(c.pb, c.Kp, c.Kp, c.args()[0].int(), c.K, c.V, stream=0)


# ---- together ----------------------------------------------------------------------------------------
def lookahead(dtype, S, M, T, L, Hq, Hkv, d, n, stop=None):
    """T steps of M trajectories behind S prompts through every layer; each step's attention output
    against the oracle over the rows appended so far. Returns the queries as lorekv_score takes them
    and the cache."""
    gen = torch.Generator(device=DEV).manual_seed(T)
    dt, R = DT[dtype], S * M
    pb = api.PgProblem(S, M, Hq, Hkv, d, n, 4, R * -(-T // 4) + 1, -(-T // 4), R + 2, 1, KD[dtype])
    c = api.PgCache(pb, L, DEV)
    K, V = (torch.randn(S, L, Hkv, n, d, generator=gen, device=DEV).to(dt) for _ in range(2))
    Q_look = torch.empty(S, L, Hq, M * T, d, dtype=dt, device=DEV)
    new = torch.ones(R, dtype=torch.int32, device=DEV)
    own = [[np.zeros((2, Hkv, 0, d)) for _ in range(R)] for _ in range(L)]
    h = torch.finfo(dt).eps / 2
    out = torch.empty(R + 2, Hq, d, dtype=dt, device=DEV)
    for t in range(T):
        if t == stop:
            new[R - 1] = -1  # the last trajectory has ended
        c.plan(new)
        new[new < 0] = 0
        for layer in range(L):
            qkv = torch.randn(R + 2, Hq + 2 * Hkv, d, generator=gen, device=DEV).to(dt)
            c.append(layer, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
            c.attend(layer, qkv[:, :Hq], K[:, layer], V[:, layer], out)
            live = R - int((new <= 0).sum())
            got, x = f64(out), f64(qkv)
            for r in range(live):
                s = r // M
                Q_look[s, layer, :, (r % M) * T + t] = qkv[r, :Hq]
                kv = own[layer][r] = np.concatenate(
                    (own[layer][r], x[r, Hq:].reshape(2, Hkv, 1, d)), 2)
                for hq in range(0, Hq, 3):
                    k = np.concatenate((f64(K[s, layer, hq // (Hq // Hkv)]), kv[0, hq // (Hq // Hkv)]))
                    v = np.concatenate((f64(V[s, layer, hq // (Hq // Hkv)]), kv[1, hq // (Hq // Hkv)]))
                    sc = k @ x[r, hq] / math.sqrt(d)
                    a = np.exp(sc - sc.max())
                    a /= a.sum()
                    ref, terms = a @ v, a @ np.abs(v)
                    # module bound with mag <= 6 sqrt(d) for normal inputs
                    w = (d + 8) * U * 6 * math.sqrt(d) + 2.0 ** -21
                    tol = (2 * w + 8 * math.sqrt(n + T) * U + h) * terms * (1 + h) + h * np.abs(ref)
                    assert (np.abs(got[r, hq] - ref) <= tol).all()
    api.kve_check_device()
    return Q_look, c, K, V


def test_lookahead_feeds_the_eviction_pass_and_answers_decode_from_its_cache():
    """The use these calls are for: the lookahead's trajectories decode behind the prompt, their
    queries score it, the cache is compressed, and answers decode from the compressed cache."""
    S, M, T, L, Hq, Hkv, d, n = 1, 4, 8, 2, 8, 2, 128, 1000
    Q_look, c, K, V = lookahead("bf16", S, M, T, L, Hq, Hkv, d, n)
    assert c.lens.tolist() == [T] * M and c.pool.tolist()[1] == 1
    cfg = synth.LorekvConfig("chain", "bf16", S=S, L=L, Hq=Hq, Hkv=Hkv, d=d, d_model=256, n=n,
                             vocab=500)
    inp = {k: v.to(DEV) for k, v in synth.lorekv_inputs(cfg, "cpu").items()}
    inp.update(K=K.contiguous(), V=V.contiguous(), Q_look=Q_look)
    pb = api.LorekvProblem.from_config(cfg)
    Lf = torch.empty(L, Hq, d, d, device=DEV)
    G = torch.empty_like(Lf)
    api.lorekv_prepare_wo(pb, inp["W_O"], Lf, G)
    ev = api.LorekvPass(pb, DEV)
    ev.run(inp, Lf, G)
    api.kve_check_device()
    # the trajectories are dropped: their pages return
    c.plan(torch.full((M,), -1, dtype=torch.int32, device=DEV))
    assert c.lens.tolist() == [0] * M and c.pool.tolist()[1] == c.pb.n_pages
    # three answers of one row each behind the compressed cache
    Kc, Vc = (x.view(S, L, Hkv, ev.cap, d) for x in (ev.K_out, ev.V_out))
    ab = api.PgProblem(S, 3, Hq, Hkv, d, ev.cap, 16, 3, 1, 3, 1, api.KVE_BF16)
    a = api.PgCache(ab, L, DEV)
    a.plan(torch.ones(3, dtype=torch.int32, device=DEV))
    qkv = torch.randn(3, Hq + 2 * Hkv, d, device=DEV).bfloat16()
    out = torch.empty(3, Hq, d, dtype=torch.bfloat16, device=DEV)
    for layer in range(L):
        a.append(layer, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
        a.attend(layer, qkv[:, :Hq], Kc[:, layer], Vc[:, layer], out)
        ref = sp.pg_attention(f64(qkv[:, :Hq]), f64(Kc[:, layer]), f64(Vc[:, layer]), [ev.cap],
                              f64(a.K_pages[layer]), f64(a.V_pages[layer]),
                              a.block_table.cpu().numpy(), [1] * 3, [0, 1, 2, 3], 3)
        w = (d + 8) * U * ref["mag"] + 2.0 ** -21
        tol = (2 * w + 8 * math.sqrt(ev.cap) * U + 2.0 ** -8)[..., None] * ref["terms"] * 1.004
        assert (np.abs(f64(out) - ref["out"]) <= tol + 2.0 ** -8 * np.abs(ref["out"])).all()
    api.kve_check_device()


def test_lookahead_of_several_prompts_in_fp32_with_a_trajectory_that_ends():
    _, c, _, _ = lookahead("f32", 2, 3, 5, 1, 4, 2, 64, 130, stop=3)
    assert c.lens.tolist() == [5] * 5 + [0]


def test_a_captured_step_replays():
    """plan, append and attend in one graph: two replays advance the lengths and give what eager
    steps give; a second cache's graph between them does not disturb it."""
    def make():
        pb = api.PgProblem(1, 4, 8, 2, 128, 600, 4, 20, 4, 4, 1, api.KVE_BF16)
        gen = torch.Generator(device=DEV).manual_seed(1)
        c = api.PgCache(pb, 1, DEV)
        K, V = (torch.randn(1, 2, 600, 128, generator=gen, device=DEV).bfloat16() for _ in range(2))
        return c, K, V, torch.empty(4, 12, 128, dtype=torch.bfloat16, device=DEV), torch.empty(
            4, 8, 128, dtype=torch.bfloat16, device=DEV)

    new = torch.ones(4, dtype=torch.int32, device=DEV)
    rows = [torch.randn(4, 12, 128, device=DEV).bfloat16() for _ in range(6)]

    def step(c, K, V, qkv, out):
        c.plan(new)
        c.append(0, qkv[:, 8:10], qkv[:, 10:])
        c.attend(0, qkv[:, :8], K, V, out)

    eager = make()
    want = []
    for x in rows:
        eager[3].copy_(x)
        step(*eager)
        want.append(eager[4].clone())
    graphs = []
    for _ in range(2):
        st = make()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*st)
        graphs.append((g, st))
    for x, w in zip(rows, want):
        for g, st in graphs:
            st[3].copy_(x)
            g.replay()
        for _, st in graphs:
            assert torch.equal(st[4], w)
    api.kve_check_device()
    assert graphs[0][1][0].lens.tolist() == [6] * 4
