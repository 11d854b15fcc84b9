"""Cache in 4 bits on the GPU, where it can go wrong: row blocks taken in turn, arrays read as another type, groups of
very different steps, rows that hold no number. Bounds as in test_gpu_q4.py."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import api
from oracle import shared_prompt as sp
from test_gpu_pages import DEV, DT, KD, f64, i32
from test_gpu_q4 import Q4Case, held, stages

pytestmark = pytest.mark.gpu


# ---- row blocks taken in turn ------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_d_head_32_in_the_later_row_blocks_of_a_request(dtype):
    """One request adds most of the rows: 7 blocks of 64 of them for 4 places, so rows 256 and on come in a second turn."""
    new = [1] * 31 + [400]
    c = Q4Case(dtype, 32, 1, 16, 4, 32, 0, 16, 200, 400, new=new, seed=21)
    assert "q4_own" in stages(c)
    c.check([0, 30, 31, 286, 287, 288, 300, 350, 351, 400, 430])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_rows_behind_a_refused_request(dtype, d):
    """A request asks for more rows than max_new and is refused; its rows still count, so the others of its prompt stand in
    row blocks that the launch has no places for."""
    F, Hq, Hkv, n, page = 8, 8, 2, 300, 16
    new = [2, 300, 1, 2, 1, 2, 2, 1]
    pb = api.Q4Problem(1, F, Hq, Hkv, d, n, page, 16, 2, sum(new), 2, KD[dtype], 32)
    gen = torch.Generator(device=DEV).manual_seed(d)
    K, V = (torch.randn(1, Hkv, n, d, generator=gen, device=DEV).to(DT[dtype]) for _ in range(2))
    c = api.Q4Cache(pb, 1, DEV)
    c.pack(0, K, V)
    c.plan(i32(new))
    assert c.pool.tolist()[3] == 1 and c.lens.tolist() == [2, 0, 1, 2, 1, 2, 2, 1]
    qkv = torch.randn(sum(new), Hq + 2 * Hkv, d, generator=gen, device=DEV).to(DT[dtype])
    c.append(0, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
    out = torch.full((sum(new), Hq, d), 3.0, device=DEV, dtype=DT[dtype])
    lse = torch.full((sum(new), Hq), 5.0, device=DEV)
    api.kve_profile_enable(True)
    c.attend(0, qkv[:, :Hq], out, lse)
    api.kve_check_device()
    assert "q4_prompt" in api.kve_profile_report()
    api.kve_profile_enable(False)
    slots, own = c.slot_map.cpu().numpy(), np.zeros((2, 16, Hkv, page, d))
    for i in np.flatnonzero(slots >= 0):
        for x, row in zip(own, (qkv[i, Hq:Hq + Hkv], qkv[i, Hq + Hkv:])):
            x[slots[i] // page, :, slots[i] % page] = held(row, 32, dtype)[0]
    rows = [i for i in range(sum(new)) if not 2 <= i < 302]
    ref = sp.pg_attention(f64(qkv[:, :Hq]), held(K, 32, dtype)[0], held(V, 32, dtype)[0], [n], own[0], own[1],
                          c.block_table.cpu().numpy(), c.lens.tolist(), c.q_start.tolist(), F, rows)
    # weights and outputs round once to the type (h of the terms each); the rest of the bound is far below h
    h = torch.finfo(DT[dtype]).eps / 2
    assert (np.abs(f64(out) - ref["out"])[rows] <= (2.5 * h * ref["terms"] + 2.0 ** -14)[rows]).all()
    assert (np.abs(f64(lse) - ref["lse"])[rows] <= 2.0 ** -14 * (1 + ref["mag"])[rows]).all()
    assert (out[2:302] == 3).all() and (lse[2:302] == 5).all()


# ---- arrays read as another type -----------------------------------------------------------------------
@pytest.mark.parametrize("d,group", [(128, 32), (64, 64), (32, 32)])
@pytest.mark.parametrize("written,read", [("bf16", "f16"), ("f32", "f16"), ("f16", "bf16"), ("f16", "f32"),
                                          ("bf16", "f32"), ("f32", "bf16")])
def test_an_array_written_from_one_type_is_read_as_another(written, read, d, group):
    """The values s m, rounded to the type that reads: zeros stay zeros whatever the step, what is above its largest number
    becomes an infinity, and only groups that hold no number are NaN."""
    n = 96
    gen = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn(1, 2, n, d, generator=gen, device=DEV)
    power = torch.arange(n, device=DEV) - (48 if written != "f16" else 20)  # steps below and above all that fp16 has
    x = x * torch.exp2(power.clamp(max=15 if written == "f16" else 47).float())[:, None]
    x[..., ::3] = 0
    x[:, 1, 5, 1] = float("nan")
    x = x.to(DT[written])
    pb = api.Q4Problem(1, 1, 2, 2, d, n, 16, 1, 1, 1, 1, KD[written], group)
    other = api.Q4Problem(1, 1, 2, 2, d, n, 16, 1, 1, 1, 1, KD[read], group)
    prefix = torch.zeros(pb.prefix_bytes, dtype=torch.uint8, device=DEV)
    api.q4_pack(pb, x, -x, None, prefix)
    out = [torch.full((1, 2, n, d), 7.0, device=DEV, dtype=DT[read]) for _ in range(2)]
    api.q4_unpack(other, prefix, None, None, *out)
    api.kve_check_device()
    for y, o in zip((x, -x), out):
        want = torch.from_numpy(held(y, group, written)[0]).to(DT[read])
        got = o.cpu()
        assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
        if read == "f16" and written != "f16":
            assert want.isinf().any() and ((want == 0) & ~want.isnan()).any()


@pytest.mark.parametrize("fan", [1, 8, 70])
def test_zeros_of_large_groups_do_not_become_nan_in_attention(fan):
    """V of steps of 2^18, written from bf16 and attended to as fp16: the channels that are 0 throughout are 0, by lines, on
    tcgen05 from codes and read back first."""
    n, d = 300, 64
    gen = torch.Generator(device=DEV).manual_seed(fan)
    K = torch.randn(1, 2, n, d, generator=gen, device=DEV)
    V = torch.randn(1, 2, n, d, generator=gen, device=DEV)
    V[..., :32] = 0
    V[..., 3] = 15 * 2.0 ** 18
    pw = api.Q4Problem(1, fan, 8, 2, d, n, 16, fan, 1, fan, 1, api.KVE_BF16, 32)
    pb = api.Q4Problem(1, fan, 8, 2, d, n, 16, fan, 1, fan, 1, api.KVE_F16, 32)
    c = api.Q4Cache(pb, 1, DEV)
    api.q4_pack(pw, K.bfloat16(), V.bfloat16(), None, c.prefix[0])
    c.plan(i32([1] * fan))
    new = torch.randn(fan, 12, d, generator=gen, device=DEV).half()
    new[..., :32] *= 0.125
    c.append(0, new[:, 8:10], torch.zeros_like(new[:, 10:]))
    out = torch.zeros(fan, 8, d, device=DEV).half()
    c.attend(0, new[:, :8], out)
    api.kve_check_device()
    zero = [x for x in range(32) if x != 3]
    assert (out[..., zero] == 0).all() and out[..., 32:].isfinite().all() and out[..., 32:].abs().max() > 0


# ---- layers of different lengths -----------------------------------------------------------------------
def test_layers_of_one_cache_with_lengths_of_their_own():
    """Each layer answers as a cache of its own would."""
    n, fan, d = 60, 3, 64
    pb = api.Q4Problem(2, fan, 8, 2, d, n, 16, 2 * fan, 1, 2 * fan, 1, api.KVE_BF16, 32)
    gen = torch.Generator(device=DEV).manual_seed(0)
    rows = [[torch.randn(2, 2, n, d, generator=gen, device=DEV).bfloat16() for _ in range(2)] for _ in range(3)]
    lens = [i32([17, 60]), None, i32([0, 33])]
    qkv = torch.randn(2 * fan, 12, d, generator=gen, device=DEV).bfloat16()

    def answers(layers):
        c = api.Q4Cache(pb, len(layers), DEV)
        for at, x in enumerate(layers):
            c.pack(at, *rows[x], lens[x])
        c.plan(i32([1] * 2 * fan))
        outs = []
        for at in range(len(layers)):
            out, back = torch.zeros(2 * fan, 8, d, device=DEV).bfloat16(), [torch.zeros_like(rows[0][0]) for _ in range(2)]
            c.append(at, qkv[:, 8:10], qkv[:, 10:])
            c.attend(at, qkv[:, :8], out)
            c.unpack(at, *back, prompts=True)
            outs.append((out, *back))
        api.kve_check_device()
        return outs

    together = answers([0, 1, 2])
    for x in range(3):
        alone = answers([x])[0]
        assert all(torch.equal(a, b) for a, b in zip(together[x], alone))
    assert (together[0][1][0, :, 17:] == 0).all() and (together[1][1][:, :, n - 1] != 0).any()


# ---- rows that hold no number --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,fan,n", [("bf16", 1, 100), ("f32", 1, 100), ("f16", 1, 0), ("bf16", 8, 300),
                                         ("f16", 70, 300), ("f32", 20, 300)])
def test_a_row_that_sees_a_nan_in_k_has_no_log_sum_either(dtype, fan, n):
    """-inf would say that there was nothing to see. By lines, on tcgen05 from codes and read back first."""
    c = Q4Case(dtype, 2, fan, 8, 2, 64, n, 16, 20, 1, seed=12)
    good, z = c.run()
    if n:
        c.Kp[1, 0, 40, 3] = float("nan")
        api.q4_pack(c.pb, c.Kp, c.Vp, None, c.prefix)
        bad = range(fan, 2 * fan)
    else:
        slot = int(c.table[1, 0]) * 16
        x = torch.full((1, 2, 64), float("inf"), device=DEV, dtype=DT[dtype])
        x[:, 1] = 1
        api.q4_append(api.Q4Problem(2, fan, 8, 2, 64, 0, 16, c.pb.n_pages, c.pb.max_pages, 1, 1, KD[dtype], 32), x,
                      torch.ones_like(x), i32([slot]), c.pages)
        bad = [1]
    out, lse = c.run()
    bad = list(bad)
    assert torch.isnan(out[bad][:, :4]).all() and torch.isnan(lse[bad][:, :4]).all()
    assert torch.isfinite(lse[:c.rows][:, 4:]).all() and torch.isfinite(out[:c.rows][:, 4:]).all()
    rest = [i for i in range(fan) if i not in bad]
    assert torch.equal(lse[rest], z[rest]) and torch.equal(out[rest], good[rest])


# ---- groups of very different steps --------------------------------------------------------------------
def refill(c):
    """What Q4Case's pages and prompts hold, from its K and V as they are now."""
    page = c.pb.page_size
    slots = [int(c.table[r, j // page]) * page + j % page for r in range(len(c.lens)) for j in range(c.lens[r])]
    at = torch.tensor(slots, device=DEV)
    pb = api.Q4Problem(1, 1, c.pb.n_kv_heads, c.pb.n_kv_heads, c.pb.d_head, 0, page, c.pb.n_pages, c.pb.max_pages,
                       len(slots), len(slots), c.pb.dtype, c.group)
    api.q4_append(pb, c.K[at // page, :, at % page].contiguous(), c.V[at // page, :, at % page].contiguous(), i32(slots),
                  c.pages)
    if c.pb.n_prefix:
        api.q4_pack(c.pb, c.Kp.contiguous(), c.Vp.contiguous(), c.plen, c.prefix)
    api.kve_check_device()
    return c


def scaled(c, power):
    """V's channels times 2^power, a number per group."""
    f = torch.exp2(torch.tensor(power, device=DEV, dtype=torch.float64).repeat_interleave(c.group))
    c.V, c.Vp = ((x.double() * f).to(x.dtype) for x in (c.V, c.Vp))
    return refill(c)


POWERS = [("bf16", 32, [0, -28, -60, 20]), ("f32", 32, [-34, 0, 12, -70]), ("f16", 32, [12, -9, 0, -8]),
          ("bf16", 64, [-64, 0]), ("f16", 64, [-10, 12]), ("f32", 64, [0, -30]), ("bf16", 128, [-64]), ("f32", 128, [-66]),
          ("bf16", 32, [-90] * 4), ("f32", 32, [-85] * 4), ("bf16", 32, [40, -35, 40, -35])]


@pytest.mark.parametrize("fan,new_hi", [(1, 1), (2, 3), (6, 1)])
@pytest.mark.parametrize("dtype,group,power", POWERS, ids=str)
def test_every_group_of_v_keeps_its_own_bits(dtype, group, power, fan, new_hi):
    """A group's output does not go by the size of its row's other groups, nor by V's size as a whole."""
    scaled(Q4Case(dtype, 2, fan, 4, 2, 128, 200, 16, 50, new_hi, group=group, ragged=True, seed=22), power).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_groups_that_change_their_size_from_token_to_token(dtype, d):
    """Sizes of every group and token for itself, over 2^40 (fp16 2^20), rows without any at all and a NaN that nobody
    sees among them."""
    c = Q4Case(dtype, 1, 2, 4, 1, d, 150, 16, 90, 4, ragged=False, seed=23)
    gen = torch.Generator(device=DEV).manual_seed(d)
    lo, hi = (-14, 6) if dtype == "f16" else (-30, 10)
    for name in ("V", "Vp"):
        x = getattr(c, name)
        e = torch.randint(lo, hi, x.shape[:-1] + (d // 32,), generator=gen, device=DEV)
        e = e.masked_fill(torch.rand(e.shape, generator=gen, device=DEV) < 0.1, -999).double()
        setattr(c, name, (x.double() * torch.exp2(e).repeat_interleave(32, -1)).to(x.dtype))
    refill(c).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_small_v_behind_one_that_is_large_in_another_group(dtype):
    """The first tokens weigh in one group 2^50 times what the later ones do, in the others as much."""
    c = Q4Case(dtype, 1, 1, 4, 1, 128, 400, 16, 60, 1, seed=24)
    c.Vp[:, :, :20, 32:64] = (c.Vp[:, :, :20, 32:64].double() * 2.0 ** 50).to(DT[dtype])
    refill(c).check()
    c.Vp[:, :, 100:110, 96:] = (c.Vp[:, :, 100:110, 96:].double() * 2.0 ** 70).to(DT[dtype])
    refill(c).check()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_channels_that_are_not_used(dtype):
    """A head of 96 channels in 128: the last group is 0 throughout, and stays it."""
    c = Q4Case(dtype, 1, 2, 4, 1, 128, 200, 16, 60, 2, seed=25)
    for x in (c.V, c.Vp):
        x[..., 96:] = torch.where(x[..., 96:].isnan(), x[..., 96:], 0)
    out, _ = refill(c).check()
    assert (out[:c.rows, :, 96:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,group", [(128, 32), (128, 64), (64, 32), (64, 64)])
def test_groups_that_are_zero_at_first(dtype, d, group):
    """The last group is zero for some tokens, then small, then as the others; others are zero for a while, too."""
    for late, size in ((16, -20), (7, -9), (130, 0)):
        c = Q4Case(dtype, 1, 1, 4, 1, d, 200, 16, 90, 3, seed=26)
        for x in (c.V, c.Vp):
            x[..., -group:] *= 2.0 ** size
        c.Vp[:, :, :late, -group:] = 0
        c.Vp[:, :, late + 20:late + 30, :group] = 0
        c.Vp[:, :, 180:, -group:] *= 2.0 ** -size
        refill(c).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_largest_steps_beside_the_smallest(dtype):
    """Near 2^89 and near 2^-90 in one row: all finite, the large group within its bound; and beside zeros."""
    for power in ([83, -90, 83, 0], [83, -9999, 83, 83]):
        c = Q4Case(dtype, 1, 2, 4, 1, 128, 120, 16, 40, 2, seed=27)
        scaled(c, power)
        out, lse = c.run()
        (V, _), (K, _) = held(c.V, 32, dtype), held(c.K, 32, dtype)
        (Vp, _), (Kp, _) = held(c.Vp, 32, dtype), held(c.Kp, 32, dtype)
        ref = sp.pg_attention(f64(c.q), Kp, Vp, c.np_plen, K, V, np.where(c.table > 2 ** 30, 0, c.table), c.lens, c.q_start,
                              c.F)
        got, h = f64(out)[:c.rows], torch.finfo(DT[dtype]).eps / 2
        assert np.isfinite(got).all() and np.isfinite(f64(lse)[:c.rows]).all()
        # weights and output round (h each), codes and zero codes to 2^-12 of a step, of which a term is one at least
        big = [i for i in range(128) if power[i // 32] == 83]
        tol = 2.5 * h * ref["terms"] + 2.0 ** -12 * ref["terms"].max(-1, keepdims=True)
        assert (np.abs(got - ref["out"][:c.rows]) <= tol[:c.rows])[..., big].all()
        assert (np.abs(f64(lse) - ref["lse"])[:c.rows] <= 2.0 ** -12 * (1 + ref["mag"])[:c.rows]).all()


@pytest.mark.parametrize("dtype,fan,n,new,path", [("bf16", 8, 300, 1, "q4_prompt"), ("f16", 70, 300, 1, "q4_prompt"),
                                                  ("bf16", 70, 0, 24, "q4_own"), ("f32", 5, 40, 3, "q4_lines")])
def test_captured_calls_of_every_path_replay_on_other_rows(dtype, fan, n, new, path):
    """Captured once, replayed with other queries, lengths and prompts: as the same calls one by one."""
    c = Q4Case(dtype, 1, fan, 8, 2, 64, n, 16, 600 if new > 20 else 40, new, seed=28)
    assert path in stages(c)
    q, out, lse = c.q.contiguous(), torch.zeros(c.shape, device=DEV, dtype=DT[dtype]), torch.zeros(c.shape[:2], device=DEV)
    plen = i32([n]) if n else None
    args = (c.prefix, plen, c.pages, i32(c.table), i32(c.lens), i32(c.q_start), i32(c.row_req), out, lse, c.ws)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        api.q4_attention(c.pb, q, *args)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        api.q4_attention(c.pb, q, *args)
    gen = torch.Generator(device=DEV).manual_seed(1)
    for step in range(3):
        q.copy_(torch.randn(c.shape, generator=gen, device=DEV))
        if n:
            plen.fill_(n - 37 * step)
            api.q4_pack(c.pb, torch.randn(1, 2, n, 64, generator=gen, device=DEV).to(DT[dtype]),
                        torch.randn(1, 2, n, 64, generator=gen, device=DEV).to(DT[dtype]), None, c.prefix)
        out.fill_(3.0)
        api.q4_attention(c.pb, q, *args)
        want = out.clone(), lse.clone()
        out.fill_(3.0)
        lse.fill_(5.0)
        c.ws.fill_(0xFF)
        g.replay()
        api.kve_check_device()
        assert torch.equal(out, want[0]) and torch.equal(lse[:c.rows], want[1][:c.rows])
        assert (lse[c.rows:] == 5).all()


# ---- strides ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("native", [True, False])
def test_strides_of_dimensions_of_one_entry_do_not_matter(native, monkeypatch):
    """One prompt, one KV head or one row: K and V may come from arrays of different widths."""
    if not native:
        monkeypatch.setattr(api, "_native", api._NoBinding)
    for S, H, n in ((1, 2, 40), (2, 1, 40), (1, 1, 40), (2, 2, 1), (1, 1, 1)):
        d = 64
        K = torch.randn(S, H, n, d, device=DEV).bfloat16()
        V = torch.randn(S, H, n, d, device=DEV).bfloat16()
        apart = [7 * H * n * d if S == 1 else H * n * d, 3 * n * d if H == 1 else n * d, 5 * d if n == 1 else d, 1]
        W = V.as_strided(V.shape, apart)
        pb = api.Q4Problem(S, 1, H, H, d, n, 16, 1, 1, 1, 1, api.KVE_BF16, 32)
        prefix = [torch.zeros(pb.prefix_bytes, dtype=torch.uint8, device=DEV) for _ in range(2)]
        api.q4_pack(pb, K, V, None, prefix[0])
        api.q4_pack(pb, K, W, None, prefix[1])
        assert torch.equal(*prefix)
        a, b = torch.zeros_like(K), torch.zeros_like(V)
        api.q4_unpack(pb, prefix[0], None, None, a, b.as_strided(V.shape, apart))
        api.kve_check_device()
        assert all(torch.equal(y, torch.from_numpy(held(x, 32, "bf16")[0]).to(DEV).bfloat16()) for x, y in ((K, a), (V, b)))
