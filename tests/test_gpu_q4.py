"""Cache in 4 bits on the GPU against the fp64 oracle: what is held bit for bit, attention within a bound
derived from the roundings of the call.

Bound of an output component, o = sum_j a_j v_j over the values that the cache holds:
  * its own rounding to the type: h |o|, h = finfo.eps / 2 (bf16 2^-8, fp16 2^-11, fp32 2^-24);
  * 16-bit types: each weight (or weight times step) rounds once, to the type or finer: h sum_j a_j |v_j|;
  * scores are sums of q_c n_c s and, for the zero codes, s k sum q: magnitudes of at most M = max_j sum_c |q_c| 15 s_jc
    / sqrt d each. Queries are off by 2^-22 of themselves at most, the sums of q by 2^-22, and each of the at most 12
    product instructions of a score by 2^-22 of its terms: 2^-18 M in all (fp32: 2^-21 M, its codes being normal
    numbers). With 2^-21 for the exponential, a relative error w of every weight moves o by 2 w sum_j a_j |v_j|;
  * codes and zero codes of V are summed apart and subtracted, each at most 15 in units of weight times step; the
    product instructions of four tiles are off by 2^-22 of their terms, and weights below 2^-31 of the largest are
    lost: 2^-14 sum_j a_j s_j (fp32, whose codes are subtracted before: 2^-18);
  * sums over n tokens in fp32: 8 sqrt(n) 2^-24 sum_j a_j |v_j| (roundings add like a random walk).
lse: the scores' error, the sum's, and the roundings of a reference that stands up to 40 powers of two away."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import api, synth
from oracle import cache4
from oracle import shared_prompt as sp
from test_gpu_canary import Guarded
from test_gpu_pages import DEV, DT, KD, U, Case, f64, i32

pytestmark = pytest.mark.gpu


def held(t, group, dtype):
    return cache4.hold(f64(t), group, cache4.LARGEST[dtype])


# ---- what is held ----------------------------------------------------------------------------------
def rows_of(kind, shape, dtype, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(shape, generator=gen, device=DEV)
    if kind == "wide":     # steps from 2^-40 to 2^12
        x = x * torch.exp2(torch.randint(-40, 12, shape[:-1] + (1,), generator=gen, device=DEV).float())
    elif kind == "halves":  # multiples of half a step: what lies between two codes
        x = torch.randint(-15, 16, shape, generator=gen, device=DEV).float() / 2
    elif kind == "sided":  # all of one sign, constants, zeros
        x = x.abs() + 3
        x[..., 1::5, :] = 0
        x[..., 2::5, :] = -7.25
    elif kind == "edge":   # next to the largest numbers, infinities, NaN
        f = cache4.LARGEST[dtype]
        x = (torch.rand(shape, generator=gen, device=DEV, dtype=torch.float64) * 2 - 1) * f
        x[..., 0::7, :] = f
        x[..., 1::7, 3] = float("inf")
        x[..., 2::7, 9] = float("nan")
        x[..., 3::7, :] *= 2.0 ** -120 if dtype != "f16" else 2.0 ** -20
    return x.to(DT[dtype])


SIZES = [("bf16", 128, 32), ("bf16", 64, 64), ("f16", 128, 64), ("f16", 32, 32), ("f32", 128, 128), ("f32", 64, 32),
         ("bf16", 128, 128), ("f16", 128, 32), ("f32", 32, 32)]


@pytest.mark.parametrize("kind", ["normal", "wide", "halves", "sided", "edge"])
@pytest.mark.parametrize("dtype,d,group", SIZES)
def test_prompts_hold_what_the_definition_says(dtype, d, group, kind):
    S, H, n = 2, 3, 75
    pb = api.Q4Problem(S, 1, H, H, d, n, 16, 1, 1, 1, 1, KD[dtype], group)
    K, V = (rows_of(kind, (S, H, n, d), dtype, s) for s in (1, 2))
    prefix = Guarded((pb.prefix_bytes,), torch.uint8)
    api.q4_pack(pb, K, V, None, prefix.t)
    out = [Guarded((S, H, n, d), DT[dtype]) for _ in range(2)]
    api.q4_unpack(pb, prefix.t, None, None, out[0].t, out[1].t)
    api.kve_check_device()
    assert prefix.intact()
    for x, o in zip((K, V), out):
        want, _ = held(x, group, dtype)
        want = torch.from_numpy(want).to(DT[dtype])  # (only fp16 rounds: below its normal numbers)
        assert o.intact() and torch.equal(o.t.cpu().nan_to_num(12345.0), want.nan_to_num(12345.0))


@pytest.mark.parametrize("dtype,d,group", SIZES[:6])
def test_ragged_strided_prompts_leave_the_rest(dtype, d, group):
    """A layer's slice of a larger cache; lengths of none, one, a tile, all and more; output rows behind them stay."""
    S, H, n = 6, 2, 50
    lens = i32([0, 1, 16, 17, 50, 99])
    gen = torch.Generator(device=DEV).manual_seed(0)
    wide = torch.randn(S, 2, H, n + 3, 2 * d, generator=gen, device=DEV).to(DT[dtype])
    K, V = wide[:, 1, :, :n, :d], wide[:, 1, :, :n, d:]
    pb = api.Q4Problem(S, 1, H, H, d, n, 16, 1, 1, 1, 1, KD[dtype], group)
    prefix = Guarded((pb.prefix_bytes,), torch.uint8)
    prefix.t.fill_(0xA5)
    api.q4_pack(pb, K, V, lens, prefix.t)
    tile = prefix.t.view(S, H, -1, 16 * d + 64 * d // group)
    for s, m in enumerate((0, 1, 16, 17, 50, 50)):
        assert (tile[s, :, -(-m // 16):] == 0xA5).all()
    got = torch.full((S, H, 3, n, 2, d), 7.0, device=DEV, dtype=DT[dtype])
    api.q4_unpack(pb, prefix.t, None, lens, got[:, :, 1, :, 0], got[:, :, 1, :, 1])
    api.kve_check_device()
    assert prefix.intact()
    for i, x in enumerate((K, V)):
        want = torch.from_numpy(held(x, group, dtype)[0]).to(DT[dtype]).to(DEV)
        for s, m in enumerate((0, 1, 16, 17, 50, 50)):
            assert torch.equal(got[s, :, 1, :m, i], want[s, :, :m]) and (got[s, :, 1, m:, i] == 7).all()
    got[:, :, 1] = 7
    assert (got == 7).all()
    few = torch.zeros(S, H, 20, d, device=DEV, dtype=DT[dtype])  # fewer rows than there are
    api.q4_unpack(pb, prefix.t, None, lens, few, few.clone())
    assert torch.equal(few[4], torch.from_numpy(held(K, group, dtype)[0]).to(
        DT[dtype]).to(DEV)[4, :, :20])


@pytest.mark.parametrize("dtype,d,group,page", [("bf16", 128, 32, 16), ("f16", 64, 64, 64), ("f32", 128, 64, 32),
                                                ("bf16", 32, 32, 256), ("f32", 64, 32, 16), ("f16", 128, 128, 128)])
def test_rows_go_into_their_slots_and_nothing_else_changes(dtype, d, group, page):
    """Runs of every length at every offset, scattered rows and rows of nobody, in several calls: values, and every byte
    that belongs to another token."""
    rng = np.random.default_rng(page)
    H, n_pages = 3, 12
    total = n_pages * page
    free = np.ones(total, bool)
    held_K = np.full((total, H, d), np.nan)
    held_V = held_K.copy()
    have = np.zeros(total, bool)
    pages = None
    for call in range(4):
        slots = []
        for _ in range(int(rng.integers(1, 9))):
            run, at = int(rng.choice([1, 2, 15, 16, 17, 33, 48])), int(rng.integers(total))
            if call == 1:
                at &= ~15
            for s in range(at, min(at + run, total)):
                if free[s]:
                    slots.append(s)
                    free[s] = False
        slots += [-1] * int(rng.integers(0, 20))
        if call == 2:
            slots = list(rng.permutation(slots))
        n = max(1, len(slots))
        slots = i32(slots or [-1])
        pb = api.Q4Problem(1, 1, H, H, d, 0, page, n_pages, n_pages, n, n, KD[dtype], group)
        if pages is None:
            pages = Guarded((pb.pool_bytes,), torch.uint8)
            pages.t.copy_(torch.randint(0, 256, (pb.pool_bytes,), dtype=torch.uint8, device=DEV))
        qkv = rows_of("normal", (n, 4 * H, d), dtype, call)
        K, V = qkv[:, H:2 * H], qkv[:, 3 * H:]
        before = pages.t.clone()
        api.q4_append(pb, K, V, slots, pages.t)
        api.kve_check_device()
        assert pages.intact()
        mine = slots.cpu().numpy()
        live = mine >= 0
        held_K[mine[live]] = held(K, group, dtype)[0][live]
        held_V[mine[live]] = held(V, group, dtype)[0][live]
        have[mine[live]] = True
        # bytes that changed: those of the tokens written, half of a code row and 2 bytes per group each
        changed = int((before != pages.t).sum())
        assert changed <= live.sum() * H * (d + 4 * d // group)
        table, lens = i32(np.arange(n_pages)), i32([total])
        out = [torch.zeros(1, H, total, d, device=DEV, dtype=DT[dtype]) for _ in range(2)]
        pb1 = dataclasses.replace(pb, n_rows=1, max_new=1)
        api.q4_unpack(pb1, pages.t, table, lens, *out)
        for o, want in zip(out, (held_K, held_V)):
            got = o[0].transpose(0, 1).cpu()[have]
            assert torch.equal(got, torch.from_numpy(want[have]).to(DT[dtype]))
    # a slot outside the pool is skipped and reported
    before = pages.t.clone()
    pb = api.Q4Problem(1, 1, H, H, d, 0, page, n_pages, n_pages, 1, 1, KD[dtype], group)
    x = rows_of("normal", (1, H, d), dtype)
    api.q4_append(pb, x, x, i32([total]), pages.t)
    with pytest.raises(api.KveError, match="slot or page id"):
        api.kve_check_device()
    api.kve_check_device()
    assert torch.equal(before, pages.t) and pages.intact()


def test_page_ids_outside_the_pool_are_read_as_page_0_and_reported():
    pb = api.Q4Problem(1, 1, 4, 2, 64, 0, 16, 3, 2, 1, 1, api.KVE_BF16, 32)
    x = rows_of("normal", (48, 2, 64), "bf16")
    pages = torch.zeros(pb.pool_bytes, dtype=torch.uint8, device=DEV)
    api.q4_append(dataclasses.replace(pb, n_rows=48, max_new=48), x, x, i32(np.arange(48)), pages)
    good, bad = (torch.zeros(1, 2, 32, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    api.q4_unpack(pb, pages, i32([1, 0]), i32([32]), good, good.clone())
    api.kve_check_device()
    for page in (3, -1, 2 ** 31 - 1, -2 ** 31):
        api.q4_unpack(pb, pages, i32([1, page]), i32([32]), bad, bad.clone())
        with pytest.raises(api.KveError, match="slot or page id"):
            api.kve_check_device()
        assert torch.equal(good, bad)
        q, out = torch.randn(1, 4, 64, device=DEV).bfloat16(), [torch.zeros(1, 4, 64, device=DEV).bfloat16() for _ in range(2)]
        ws = torch.empty(api.q4_workspace_size(pb), dtype=torch.uint8, device=DEV)
        for o, t in zip(out, (page, 0)):
            api.q4_attention(pb, q, None, None, pages, i32([1, t]), i32([32]), i32([0, 1]), i32([0]), o, None, ws)
        with pytest.raises(api.KveError, match="slot or page id"):
            api.kve_check_device()
        assert torch.equal(*out)


# ---- attention -------------------------------------------------------------------------------------
class Q4Case(Case):
    """Case with its prompts and pages in 4 bits; bytes of rows that nobody wrote hold anything, NaN among it."""

    def __init__(self, dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi, group=32, v_scale=1.0, **kw):
        super().__init__(dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi, **kw)
        if v_scale != 1.0:
            self.V, self.Vp = self.V * v_scale, self.Vp * v_scale
        self.group = group
        self.pb = api.Q4Problem(**{f.name: getattr(self.pb, f.name) for f in dataclasses.fields(self.pb)}, group=group)
        self.ws = torch.empty(api.q4_workspace_size(self.pb), dtype=torch.uint8, device=DEV)
        self.pages = torch.full((self.pb.pool_bytes,), 0xFF, dtype=torch.uint8, device=DEV)
        self.prefix = None
        slots = [int(self.table[r, j // page]) * page + j % page for r in range(S * F) for j in range(self.lens[r])]
        if slots:
            at = torch.tensor(slots, device=DEV)
            pb = dataclasses.replace(self.pb, n_rows=len(slots), max_new=len(slots), n_q_heads=Hkv)
            api.q4_append(pb, self.K[at // page, :, at % page].contiguous(), self.V[at // page, :, at % page].contiguous(),
                          i32(slots), self.pages)
        if n:
            self.prefix = torch.full((self.pb.prefix_bytes,), 0xFF, dtype=torch.uint8, device=DEV)
            api.q4_pack(self.pb, self.Kp.contiguous(), self.Vp.contiguous(), self.plen, self.prefix)
        api.kve_check_device()

    def run(self, lse=True, stream=None):
        out, z = Guarded(self.shape, DT[self.dtype]), Guarded(self.shape[:2], torch.float32)
        out.t.fill_(3.0)
        z.t.fill_(5.0)
        ws = Guarded((self.ws.numel(),), torch.uint8)
        ws.t.fill_(0xFF)
        api.q4_attention(self.pb, self.q, self.prefix, self.plen, self.pages, i32(self.table), i32(self.lens),
                         i32(self.q_start), i32(self.row_req), out.t, z.t if lse else None, ws.t, stream=stream)
        api.kve_check_device(stream)
        assert out.intact() and z.intact() and ws.intact()
        return out.t, z.t

    def check(self, rows=None):
        out, lse = self.run()
        (K, Ks), (V, Vs), (Kp, Kps), (Vp, Vps) = (held(x, self.group, self.dtype) for x in (self.K, self.V, self.Kp, self.Vp))
        table = np.where(self.table > 2 ** 30, 0, self.table)

        def attend(q, Kp, Vp, K, V):
            return sp.pg_attention(q, Kp, Vp, self.np_plen, K, V, table, self.lens, self.q_start, self.F, rows)

        q = f64(self.q)
        ref = attend(q, Kp, Vp, K, V)
        S = attend(q, Kp, Vps, K, Vs)["out"]
        M = attend(np.abs(q), 15 * Kps, Vps, 15 * Ks, Vs)["mag"]
        live = ~np.isnan(ref["lse"])
        if rows is None:
            assert live[:self.rows].all()
        fp32 = self.dtype == "f32"
        h = torch.finfo(DT[self.dtype]).eps / 2
        n = self.pb.n_prefix + int(self.lens.max())
        w = 2.0 ** (-21 if fp32 else -18) * M + 2.0 ** -21
        tol = (2 * w + 8 * math.sqrt(n) * U + (0 if fp32 else h))[..., None] * ref["terms"] * (1 + h)
        tol = tol + h * np.abs(ref["out"]) + 2.0 ** (-18 if fp32 else -14) * S
        if self.dtype == "f16":
            tol = tol + 2.0 ** -24  # half a step of the smallest fp16 numbers, of the value and of the output
        got = f64(out)
        bad = live[..., None] & ~(np.abs(got - ref["out"]) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], np.abs(got - ref["out"])[bad][:5], tol[bad][:5])
        z = f64(lse)
        zt = w + 8 * math.sqrt(n) * U + 4 * U * (np.abs(np.where(np.isinf(ref["lse"]), 0, ref["lse"])) + 40)
        inf = live & np.isinf(ref["lse"])
        assert np.isneginf(z[inf]).all()
        fin = live & ~inf
        assert (np.abs(z[fin] - ref["lse"][fin]) <= zt[fin]).all()
        assert (got[self.rows:] == 3.0).all() and (z[self.rows:] == 5.0).all()  # rows of nobody
        return out, lse


def stages(case):
    """The launch groups of a call, by the library's own record."""
    api.kve_profile_enable(True)
    case.run()
    got = set(api.kve_profile_report())
    api.kve_profile_enable(False)
    return got


CASES = [
    # dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi, group
    ("f32", 1, 4, 1, 1, 64, 512, 16, 7, 1, 32),
    ("f32", 2, 3, 6, 2, 128, 77, 16, 40, 5, 128),
    ("f32", 1, 1, 4, 4, 32, 1, 16, 3, 1, 32),
    ("f32", 3, 2, 8, 2, 128, 300, 64, 200, 3, 32),
    ("f32", 9, 1, 4, 2, 64, 0, 32, 300, 20, 64),
    ("bf16", 1, 1, 8, 2, 128, 1000, 16, 7, 1, 32),
    ("bf16", 1, 4, 8, 2, 128, 999, 16, 7, 1, 64),       # 16 query rows a KV head: two units
    ("bf16", 40, 1, 8, 2, 128, 0, 16, 150, 1, 32),      # more requests than lanes, no prompts
    ("bf16", 5, 1, 7, 1, 64, 0, 256, 600, 1, 64),       # 7 query heads per KV head
    ("bf16", 2, 3, 10, 2, 128, 40, 64, 100, 2, 128),    # 5 per KV head
    ("bf16", 1, 2, 16, 16, 32, 33, 32, 40, 3, 32),      # one per KV head
    ("f16", 1, 2, 8, 2, 128, 700, 32, 90, 1, 64),
    ("f16", 33, 1, 6, 6, 64, 0, 16, 60, 9, 32),
    ("f16", 1, 3, 4, 1, 32, 260, 64, 33, 1, 32),
    ("f16", 4, 1, 12, 4, 128, 0, 128, 1000, 2, 128),
    ("f16", 1, 40, 8, 2, 64, 130, 16, 9, 1, 32),        # many rows behind a short prompt
    ("bf16", 2, 9, 4, 1, 32, 5, 16, 9, 2, 32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_attention_by_lines(case):
    c = Q4Case(*case[:10], group=case[10], seed=3)
    assert stages(c) == {"q4_lines", "q4_join"}
    c.check()


TC = [  # one row tile behind a prompt: on tcgen05 from codes
    ("bf16", 1, 5, 8, 2, 128, 700, 16, 20, 1, 32),
    ("bf16", 2, 8, 16, 4, 64, 300, 32, 60, 2, 64),
    ("bf16", 1, 30, 4, 1, 32, 385, 16, 9, 1, 32),
    ("bf16", 1, 3, 40, 5, 128, 257, 64, 50, 2, 128),
    ("f16", 1, 17, 8, 2, 128, 515, 16, 30, 1, 32),
    ("f16", 3, 6, 12, 4, 64, 384, 64, 12, 1, 32),
    ("f16", 1, 1, 128, 1, 128, 260, 16, 40, 1, 128),
    ("f16", 2, 20, 4, 2, 32, 300, 128, 20, 3, 32),
    ("bf16", 2, 5, 8, 2, 64, 1500, 16, 20, 1, 32),
]


@pytest.mark.parametrize("case", TC, ids=lambda c: "-".join(map(str, c)))
def test_attention_of_one_row_tile(case):
    c = Q4Case(*case[:10], group=case[10], seed=4)
    assert "q4_prompt" in stages(c)
    c.check()


WIDE = [  # several row tiles: the prompt is read back first
    ("bf16", 1, 70, 8, 2, 64, 300, 16, 20, 1, 32),
    ("f16", 1, 64, 8, 2, 128, 260, 16, 100, 1, 64),
    ("bf16", 2, 40, 8, 1, 32, 270, 32, 30, 2, 32),
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: "-".join(map(str, c)))
def test_attention_of_several_row_tiles(case):
    c = Q4Case(*case[:10], group=case[10], seed=5)
    assert "q4_prompt" in stages(c)
    c.check()


OWN_TC = [  # many new rows of requests with long own caches
    ("bf16", 16, 1, 32, 8, 128, 0, 64, 500, 40, 32),
    ("f16", 130, 1, 8, 1, 64, 0, 16, 300, 24, 64),
    ("bf16", 8, 2, 64, 8, 32, 60, 32, 600, 60, 32),
    ("f16", 16, 1, 40, 8, 128, 0, 16, 700, 50, 128),
]


@pytest.mark.parametrize("case", OWN_TC, ids=lambda c: "-".join(map(str, c)))
def test_attention_of_many_new_rows(case):
    c = Q4Case(*case[:10], group=case[10], seed=6)
    assert "q4_own" in stages(c)
    rng = np.random.default_rng(0)
    c.check(sorted(set(rng.integers(0, c.rows, 12).tolist()) | {0, c.rows - 1}))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fan,new_hi", [(2, 1), (9, 3), (70, 1)])
@pytest.mark.parametrize("n", [90, 290])
def test_ragged_prompts_idle_requests_and_strided_queries(dtype, fan, new_hi, n):
    Q4Case(dtype, 3, fan, 8, 2, 64, n, 16, 40, new_hi, ragged=True, idle=0.3, stride=True, seed=7).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [0, 20])
def test_rows_that_see_nothing_are_zero(dtype, n):
    Q4Case(dtype, 4, 2, 4, 2, 128, n, 16, 3, 4, ragged=n > 0, nothing=True, seed=8).check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fan", [2, 9, 70])
def test_peaked_scores(dtype, fan):
    Q4Case(dtype, 1, fan, 8, 2, 128, 300, 16, 60, 1, scale=12.0, seed=9).check()


@pytest.mark.parametrize("dtype,power", [("f32", 60), ("bf16", 80), ("f32", -40), ("bf16", -40), ("f16", -8), ("f16", 12)])
@pytest.mark.parametrize("fan", [1, 6, 70])
def test_values_of_any_size(dtype, power, fan):
    """Steps far from 1, of V in the prompt and in the pages alike."""
    Q4Case(dtype, 1, fan, 4, 2, 64, 200, 16, 50, 1, v_scale=2.0 ** power, seed=10).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_tokens_of_very_different_sizes(dtype):
    """The reference of the weights follows weight times step: rows of V a million times larger come late."""
    c = Q4Case(dtype, 1, 1, 4, 1, 64, 400, 16, 60, 1, seed=11)
    size = torch.exp2(torch.arange(400, device=DEV) / 20 - 12).to(DT[dtype])[:, None]
    c.Vp = c.Vp * size
    api.q4_pack(c.pb, c.Kp, c.Vp, None, c.prefix)
    c.check()


def test_a_value_that_is_none_reaches_its_groups_alone():
    """A NaN in V: the channels of its group (bf16: and maybe the head's others), of the requests behind its prompt; in
    K: all of them."""
    for dtype in ("bf16", "f32"):
        c = Q4Case(dtype, 2, 1, 4, 1, 128, 100, 16, 20, 1, seed=12)
        good, _ = c.run()
        c.Vp[1, 0, 37, 70] = float("nan")
        api.q4_pack(c.pb, c.Kp, c.Vp, None, c.prefix)
        out, lse = c.run()
        assert torch.isnan(out[1, :, 64:96]).all() and torch.isfinite(lse[:2]).all()
        if dtype != "bf16":
            assert torch.isfinite(out[1, :, :64]).all() and torch.isfinite(out[1, :, 96:]).all()
        assert torch.equal(out[0], good[0])
        c.Kp[1, 0, 40, 3] = float("inf")
        api.q4_pack(c.pb, c.Kp, c.Vp, None, c.prefix)
        out, lse = c.run()
        assert torch.isnan(out[1]).all() and torch.equal(out[0], good[0])


def test_rows_do_not_see_what_comes_after_them():
    """Later new rows hold NaN: earlier rows of the request are as they were (lines)."""
    c = Q4Case("bf16", 1, 1, 2, 1, 64, 0, 16, 30, 4, new=[4], seed=13)
    good, z = c.run()
    last = int(c.lens[0]) - 1
    x = torch.full((1, 1, 64), float("nan"), device=DEV).bfloat16()
    slot = int(c.table[0, last // 16]) * 16 + last % 16
    api.q4_append(dataclasses.replace(c.pb, n_rows=1, max_new=1), x, x, i32([slot]), c.pages)
    out, lse = c.run()
    assert torch.equal(out[:3], good[:3]) and torch.equal(lse[:3], z[:3]) and torch.isnan(out[3]).all()


@pytest.mark.parametrize("case", [CASES[5], CASES[12], TC[0], WIDE[1], OWN_TC[0], CASES[3]],
                         ids=lambda c: "-".join(map(str, c)))
def test_without_lse_repeatable_and_on_another_stream(case):
    c = Q4Case(*case[:10], group=case[10], seed=14)
    out, lse = c.run()
    again, _ = c.run(lse=False)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        other, z = c.run(stream=st)
    assert torch.equal(out, again) and torch.equal(out, other) and torch.equal(lse, z)


@pytest.mark.parametrize("case", [CASES[5], CASES[0], TC[0], OWN_TC[0]], ids=lambda c: "-".join(map(str, c)))
def test_row_starts_that_are_no_sums_of_lengths_stay_in_bounds(case):
    c = Q4Case(*case[:10], group=case[10], seed=15)
    rng = np.random.default_rng(1)
    for starts in (rng.integers(-5, c.n_rows + 9, len(c.q_start)), np.zeros(len(c.q_start)),
                   np.sort(rng.integers(0, c.n_rows, len(c.q_start))), np.full(len(c.q_start), 2 ** 31 - 1)):
        c.q_start = starts
        c.lens = rng.integers(-3, int(c.pb.max_pages * c.pb.page_size) + 50, len(c.lens)).clip(max=2 ** 31 - 1)
        out, z = Guarded(c.shape, DT[c.dtype]), Guarded(c.shape[:2], torch.float32)
        ws = Guarded((c.ws.numel(),), torch.uint8)
        api.q4_attention(c.pb, c.q, c.prefix, c.plen, c.pages, i32(np.where(c.table > 2 ** 30, 0, c.table)), i32(c.lens),
                         i32(c.q_start), i32(c.row_req), out.t, z.t, ws.t)
        api.kve_check_device()
        assert out.intact() and z.intact() and ws.intact()


@pytest.mark.parametrize("dtype,d,Hkv", [("bf16", 64, 4), ("f16", 128, 4)])
def test_one_request_with_most_of_the_new_rows(dtype, d, Hkv):
    """More row blocks than the launch has places for: a CTA takes several in turn."""
    new = [1] * 31 + [400]
    c = Q4Case(dtype, 32, 1, 4 * Hkv, Hkv, d, 0, 16, 200, 400, new=new, seed=21)
    assert "q4_own" in stages(c)
    c.check([0, 15, 30, 31, 32, 100, 158, 159, 160, 250, 430])


def test_prompts_too_large_to_be_read_back():
    """Above 4 GiB of 16-bit values two row tiles run on codes: as one tile of the same requests does."""
    n, heads, d = 2 ** 20 + 5, 8, 128
    gen = torch.Generator(device=DEV).manual_seed(0)
    K, V = (torch.randn(1, heads, n, d, generator=gen, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    qkv = torch.randn(40, 48, d, generator=gen, device=DEV).bfloat16()
    outs = []
    for fan in (40, 20):
        pb = api.Q4Problem(1, fan, 32, heads, d, n, 16, fan, 1, fan, 1, api.KVE_BF16, 32)
        assert api.q4_workspace_size(pb) < 2 ** 32
        c = api.Q4Cache(pb, 1, DEV)
        c.pack(0, K, V)
        c.plan(i32([1] * fan))
        c.append(0, qkv[:fan, 32:40], qkv[:fan, 40:])
        out, lse = torch.zeros(fan, 32, d, device=DEV).bfloat16(), torch.zeros(fan, 32, device=DEV)
        c.attend(0, qkv[:fan, :32], out, lse)
        api.kve_check_device()
        outs.append((f64(out[:20]), f64(lse[:20])))
        del c
    (a, x), (b, y) = outs
    # each rounds its weights (2^-8, of sums over a million tokens: their random walk) and its output (2^-8)
    assert np.abs(a - b).max() <= 2.0 ** -7 * np.abs(b).max() and np.abs(x - y).max() < 1e-4
    assert np.linalg.norm(a - b) <= 2.0 ** -7 * np.linalg.norm(b)


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 4 GiB: the last pages are written, attended to and read back as the first ones are."""
    pages, heads, d = 240_000, 8, 128
    pb = api.Q4Problem(2, 1, 8, heads, d, 0, 16, pages, 3, 96, 40, api.KVE_BF16, 32)
    assert pb.pool_bytes > 2 ** 32
    pool = torch.zeros(pb.pool_bytes, dtype=torch.uint8, device=DEV)
    table = i32([[0, 1, 2], [pages - 1, pages - 3, pages - 2]])
    x = torch.randn(96, 2 * heads, d, device=DEV).bfloat16()
    x[48:] = x[:48]
    slots = (table.long().repeat_interleave(16, 1).flatten() * 16 + torch.arange(16, device=DEV).repeat(6)).int()
    api.q4_append(pb, x[:, :heads], x[:, heads:], slots, pool)
    back = [torch.zeros(2, heads, 48, d, device=DEV).bfloat16() for _ in range(2)]
    api.q4_unpack(pb, pool, table, i32([48, 48]), *back)
    pb1 = dataclasses.replace(pb, n_rows=2, max_new=1)
    q = torch.randn(1, 8, d, device=DEV).bfloat16().expand(2, 8, d).contiguous()
    out = torch.zeros(2, 8, d, device=DEV).bfloat16()
    ws = torch.empty(api.q4_workspace_size(pb1), dtype=torch.uint8, device=DEV)
    api.q4_attention(pb1, q, None, None, pool, table, i32([48, 48]), i32([0, 1, 2]), i32([0, 1]), out, None, ws)
    api.kve_check_device()
    assert all(torch.equal(b[0], b[1]) and b.abs().max() > 1 for b in back)
    # (the two requests' tiles fall to other warps: their weights round apart)
    assert (out[0] - out[1]).abs().max() <= 2.0 ** -7 * out.abs().max() and out.abs().max() > 0.01


def test_the_most_requests():
    c = Q4Case("bf16", 4096, 1, 2, 1, 32, 0, 16, 2, 1, seed=16)
    rng = np.random.default_rng(2)
    c.check(sorted(rng.integers(0, c.rows, 40).tolist()))


def test_addresses_and_tensors_that_do_not_fit():
    c = Q4Case("bf16", 1, 2, 4, 2, 64, 40, 16, 9, 1, seed=17)
    want, _ = c.run()
    out = torch.zeros_like(want)
    args = [c.q.contiguous(), c.prefix, None, c.pages, i32(c.table), i32(c.lens), i32(c.q_start), i32(c.row_req), out, None,
            c.ws]
    api.q4_attention(c.pb, *[a.data_ptr() if torch.is_tensor(a) and i not in (10,) else a for i, a in enumerate(args)])
    assert torch.equal(out[:c.rows], want[:c.rows])
    for i, bad, word in ((0, args[0].cpu(), "CUDA"), (1, c.prefix[:-1], "elements"), (3, c.pages.int(), "dtype"),
                         (8, out[:, :, :32], "elements")):
        a = list(args)
        a[i] = bad
        with pytest.raises(ValueError, match=word):
            api.q4_attention(c.pb, *a)
    with pytest.raises(api.KveError):
        api.q4_attention(c.pb, *args[:-1], c.ws[:-256])
    with pytest.raises(api.KveError):
        api.q4_attention(c.pb, args[0], None, *args[2:])


def test_a_captured_step_replays():
    """Plan, append and attend of two layers captured once, replayed with other rows: as the same calls one by one."""
    pb = api.Q4Problem(2, 2, 8, 2, 64, 60, 16, 16, 4, 5, 1, api.KVE_BF16, 32)
    gen = torch.Generator(device=DEV).manual_seed(0)
    prompt = [torch.randn(2, 2, 60, 64, generator=gen, device=DEV).bfloat16() for _ in range(4)]
    steps = [torch.randn(5, 12, 64, generator=gen, device=DEV).bfloat16() for _ in range(40)]
    new = i32([1, 1, 1, 1])
    outs = []
    for captured in (False, True):
        c = api.Q4Cache(pb, 2, DEV)
        for layer in range(2):
            c.pack(layer, prompt[2 * layer], prompt[2 * layer + 1])
        qkv, out = torch.zeros_like(steps[0]), torch.zeros(2, 5, 8, 64, dtype=torch.bfloat16, device=DEV)

        def step():
            c.plan(new)
            for layer in range(2):
                c.append(layer, qkv[:, 8:10], qkv[:, 10:])
                c.attend(layer, qkv[:, :8], out[layer])

        if captured:
            st = torch.cuda.Stream()
            state = [t.clone() for t in (c.block_table, c.free_pages, c.pool, c.lens, c.pages)]
            with torch.cuda.stream(st):
                step()
            st.synchronize()
            for t, s in zip((c.block_table, c.free_pages, c.pool, c.lens, c.pages), state):
                t.copy_(s)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        got = []
        for x in steps:
            qkv.copy_(x)
            g.replay() if captured else step()
            got.append(out.clone())
        api.kve_check_device()
        assert c.lens.tolist() == [40] * 4
        outs.append(torch.stack(got))
    assert torch.equal(*outs)


def test_two_calls_at_once_on_two_streams():
    a, b = Q4Case(*CASES[7][:10], group=32, seed=18), Q4Case(*TC[4][:10], group=32, seed=19)
    want = [c.run() for c in (a, b)]
    sts = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for c, st in zip((a, b), sts):
        with torch.cuda.stream(st):
            for _ in range(5):
                o = torch.full(c.shape, 3.0, dtype=DT[c.dtype], device=DEV)
                api.q4_attention(c.pb, c.q, c.prefix, c.plen, c.pages, i32(c.table), i32(c.lens), i32(c.q_start),
                                 i32(c.row_req), o, None, c.ws)
        outs.append(o)
    torch.cuda.synchronize()
    for o, (w, _) in zip(outs, want):
        assert torch.equal(o, w)


def test_without_the_binding_the_same(monkeypatch):
    c = Q4Case("f16", 1, 2, 4, 2, 64, 40, 16, 9, 1, seed=20)
    want = c.run()
    pages, prefix = c.pages.clone(), c.prefix.clone()
    monkeypatch.setattr(api, "_native", api._NoBinding)
    d = Q4Case("f16", 1, 2, 4, 2, 64, 40, 16, 9, 1, seed=20)
    got = d.run()
    assert torch.equal(pages, d.pages) and torch.equal(prefix, d.prefix)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_an_evicted_cache_in_4_bits_answers_and_is_evicted_again():
    """Eviction of a prompt, its compacted rows packed, three decode steps behind them, and the pages and the prompt read
    back: the whole run against the oracle on the same rows."""
    cfg = synth.LOREKV_CONFIGS["tiny"]
    inp = {k: v.to(DEV) for k, v in synth.lorekv_inputs(cfg, "cpu").items()}
    lp = api.LorekvProblem.from_config(cfg)
    Lf = torch.empty(cfg.L, cfg.Hq, cfg.d, cfg.d, device=DEV)
    G = torch.empty_like(Lf)
    api.lorekv_prepare_wo(lp, inp["W_O"], Lf, G)
    run = api.LorekvPass(lp, DEV)
    run.run(inp, Lf, G)
    kept = int(run.kept_len[0])
    K, V = (x.view(1, 1, run.cap, cfg.d) for x in (run.K_out, run.V_out))
    pb = api.Q4Problem(1, 3, 2, 1, cfg.d, run.cap, 16, 12, 3, 6, 2, api.KVE_F32, 32)
    c = api.Q4Cache(pb, 1, DEV)
    c.pack(0, K, V, i32([kept]))
    gen = torch.Generator(device=DEV).manual_seed(1)
    own = {r: ([], []) for r in range(3)}
    F = cache4.LARGEST["f32"]
    hold = lambda x: cache4.hold(f64(x), 32, F)[0]  # noqa: E731
    Kh, Vh = hold(K)[0, 0, :kept], hold(V)[0, 0, :kept]
    for new in ([1, 2, 1], [2, 0, 1], [1, 1, 1]):
        rows = sum(new)
        qkv = torch.randn(6, 4, cfg.d, generator=gen, device=DEV)
        out, lse = torch.zeros(6, 2, cfg.d, device=DEV), torch.zeros(6, 2, device=DEV)
        c.plan(i32(new))
        c.append(0, qkv[:, 2:3], qkv[:, 3:])
        c.attend(0, qkv[:, :2], out, lse)
        api.kve_check_device()
        i = 0
        for r, m in enumerate(new):
            for _ in range(m):
                own[r][0].append(hold(qkv[i, 2]))
                own[r][1].append(hold(qkv[i, 3]))
                k, v = np.concatenate((Kh, own[r][0])), np.concatenate((Vh, own[r][1]))
                s = f64(qkv[i, :2]) @ k.T / math.sqrt(cfg.d)
                z = s.max(1) + np.log(np.exp(s - s.max(1, keepdims=True)).sum(1))
                want = np.exp(s - z[:, None]) @ v
                assert np.abs(f64(out[i]) - want).max() < 2e-5 and np.abs(f64(lse[i]) - z).max() < 2e-5
                i += 1
        assert (out[rows:] == 0).all()
    back = [torch.zeros(3, 1, 48, cfg.d, device=DEV) for _ in range(2)]
    c.unpack(0, *back)
    for r in range(3):
        for b, x in zip(back, own[r]):
            assert np.array_equal(f64(b[r, 0, :len(x)]), np.array(x)) and (b[r, 0, len(x):] == 0).all()
    again = [torch.zeros(1, 1, run.cap, cfg.d, device=DEV) for _ in range(2)]
    c.unpack(0, *again, prompts=True)
    assert np.array_equal(f64(again[0][0, 0, :kept]), Kh) and np.array_equal(f64(again[1][0, 0, :kept]), Vh)
