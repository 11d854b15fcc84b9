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
