"""Shared-prompt calls made the way a program makes them: from several threads at once, in captured steps
behind other work, on arrays beyond 32-bit offsets. Bounds as in test_gpu_pages."""
import dataclasses
import threading

import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import api
from oracle import shared_prompt as sp
from test_gpu_pages import DEV, DT, Case, f64

pytestmark = pytest.mark.gpu


def test_planners_of_two_sizes_from_two_threads():
    """More requests than 48 KB of shared memory hold, so every call sets the kernel's limit, which the
    threads share."""
    faults = []

    def steps(R):
        try:
            s, n = torch.cuda.Stream(), 64
            pb = api.PgProblem(1, R, 1, 1, 128, 0, 16, R, 2, n, 1, api.KVE_BF16)
            new = torch.zeros(R, dtype=torch.int32, device=DEV)
            new[::R // 50] = 1
            back = -new
            c = api.PgCache(pb, 1, DEV)
            torch.cuda.synchronize()
            for k in range(8000):
                c.plan(new, stream=s)
                if k % 16 == 15:
                    c.plan(back, stream=s)
                if k % 256 == 255:
                    s.synchronize()
            c.plan(new, stream=s)
            s.synchronize()
            want = sp.pg_plan(f64(new), np.zeros(R), [0, R, 0, 0], np.arange(R), np.full((R, 2), -1), 16, 1, n)
            assert np.array_equal(c.lens.cpu().numpy(), want["len"])
            assert np.array_equal(c.row_req.cpu().numpy(), want["row_req"])
        except Exception as e:
            faults.append((R, e))

    threads = [threading.Thread(target=steps, args=(R,)) for R in (16384, 5000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not faults


def step_arrays(rows, n, seed=1):
    pb = api.PgProblem(1, 4, 8, 2, 128, n, 4, 4000, 800, rows, max(1, rows // 4), api.KVE_BF16)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    K, V = (torch.randn(1, 2, n, 128, generator=gen, device=DEV).bfloat16() for _ in range(2))
    qkv = torch.randn(rows, 12, 128, generator=gen, device=DEV).bfloat16()
    return api.PgCache(pb, 1, DEV), K, V, qkv, torch.full((rows, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("between", ["copies", "fills", "fork"])
@pytest.mark.parametrize("rows,n", [(4, 600), (6000, 600), (4, 40)])
def test_a_step_captured_behind_other_nodes(rows, n, between):
    """Copies from the host and on the device, fills, and appends on a forked stream between the calls of a
    captured step: two replays give what two eager steps give."""
    host = torch.full((4,), rows // 4, dtype=torch.int32).pin_memory()

    def step(c, K, V, qkv, out, new):
        cur = torch.cuda.current_stream()
        if between == "copies":
            new.copy_(host, non_blocking=True)
        elif between == "fills":
            c.row_pos.zero_()
        c.plan(new)
        if between == "fork":
            s = torch.cuda.Stream()
            s.wait_stream(cur)
            with torch.cuda.stream(s):
                c.append(0, qkv[:, 8:10], qkv[:, 10:])
            out.mul_(2)
            cur.wait_stream(s)
        else:
            c.append(0, qkv[:, 8:10], qkv[:, 10:])
        if between == "copies":
            out.copy_(qkv[:, :8])
        elif between == "fills":
            out.zero_()
        c.attend(0, qkv[:, :8], K, V, out)

    new = host.to(DEV)
    eager = step_arrays(rows, n)
    want = []
    for _ in range(2):
        step(*eager, new)
        want.append(eager[4].clone())
    st = step_arrays(rows, n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*st, new)
    for w in want:
        g.replay()
        assert torch.equal(st[4], w)
    api.kve_check_device()
    assert st[0].lens.tolist() == eager[0].lens.tolist() == [2 * (rows // 4)] * 4


def spread(buffer, at, shape, strides):
    return torch.as_strided(buffer, shape, strides, at)


FAR = [
    # dtype, S, F, Hq, Hkv, d, n, page, own_hi, new_hi
    (("bf16", 2, 4, 8, 2, 128, 20, 16, 15, 1), "direct"), (("f16", 2, 40, 8, 2, 128, 150, 16, 150, 1), "line"),
    (("bf16", 2, 2, 8, 2, 128, 5000, 8, 6, 1), "beside"), (("bf16", 2, 3, 8, 2, 128, 700, 16, 400, 60), "split"),
    (("f32", 2, 3, 8, 2, 128, 300, 16, 200, 5), "fp32"),
]


@pytest.mark.parametrize("case", [c for c, _ in FAR], ids=[w for _, w in FAR])
def test_arrays_beyond_32_bit_offsets(case):
    """Pages, prompts, heads of a prompt and packed rows that lie more than 2^32 elements behind the start of
    their arrays: the results are those of the same values lying close together."""
    c = Case(*case, seed=80, ragged=True)
    ref, lse = c.run()
    S, d, n, page, dt = case[1], case[5], case[6], case[7], DT[case[0]]
    Hkv = c.pb.n_kv_heads
    # the pool: the same pages, from the far end down
    far = 2 ** 32 // (Hkv * page * d) + 16
    slots = torch.as_tensor([far - 1 - p for p in range(c.pb.n_pages)], device=DEV)
    assert int(slots[-1]) * Hkv * page * d > 2 ** 32 - 2 ** 30 and far * Hkv * page < 2 ** 31
    K, V = (torch.empty(far, Hkv, page, d, dtype=dt, device=DEV) for _ in range(2))
    K[slots], V[slots] = c.K, c.V
    c.K, c.V, c.table = K, V, np.where(c.table < 2 ** 30, far - 1 - c.table, c.table)
    c.pb = dataclasses.replace(c.pb, n_pages=far)
    # the prompts: 2^31 elements from head to head, 2^32 from prompt to prompt
    prompt, head = 2 ** 32 + 2 ** 30, 2 ** 31 + 64
    wide = torch.empty(prompt + head + 4 * n * d, dtype=dt, device=DEV)
    Kp = spread(wide, 0, (S, Hkv, n, d), (prompt, head, d, 1)).copy_(c.Kp)
    Vp = spread(wide, 2 * n * d, (S, Hkv, n, d), (prompt, head, d, 1)).copy_(c.Vp)
    c.Kp, c.Vp = Kp, Vp
    # the packed rows
    row = 2 ** 32 // (c.n_rows - 1) // 64 * 64 + 64
    rows = torch.empty(row * (c.n_rows - 1) + c.q[0].numel(), dtype=dt, device=DEV)
    c.q = spread(rows, 0, c.q.shape, (row, d, 1)).copy_(c.q)
    assert c.q.stride(0) * (c.n_rows - 1) >= 2 ** 32
    out, z = c.run()
    assert torch.equal(out, ref) and torch.equal(z, lse)
    # the append: every row of the batch into a page behind the first 2^32 elements or close to them
    K_new = spread(rows, 0, (c.n_rows, Hkv, d), (row, d, 1))
    slot = ((slots[torch.arange(c.n_rows, device=DEV) % len(slots)] * page +
             torch.arange(c.n_rows, device=DEV) // len(slots) % page).to(torch.int32))
    assert len(set(slot.tolist())) == c.n_rows
    K_new.normal_()
    small = K_new.clone()
    api.pg_append(c.pb, K_new, small, slot, K, V)
    api.kve_check_device()
    for pool in (K, V):
        assert torch.equal(pool[slot.long() // page, :, slot.long() % page], small)
    del K, V, wide, rows, c, K_new, pool
    torch.cuda.empty_cache()


TWO = [[("bf16", 1, 8, 8, 2, 128, 2000, 16, 300, 1), ("bf16", 2, 3, 8, 2, 128, 700, 16, 100, 20)],
       [("f32", 1, 8, 8, 2, 64, 900, 16, 300, 1), ("f16", 2, 9, 8, 2, 64, 20, 16, 15, 1)]]


@pytest.mark.parametrize("pair", TWO, ids=["bf16", "mixed"])
def test_two_branches_of_one_graph(pair):
    """Attention of two batches on forked streams of one captured step, each with its own workspace."""
    cs = [Case(*c, seed=81 + i) for i, c in enumerate(pair)]
    want = [c.run()[0] for c in cs]
    args = [c.args() for c in cs]
    outs = [torch.full_like(w, 3.0) for w in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cur = torch.cuda.current_stream()
        side = [torch.cuda.Stream() for _ in cs]
        for _ in range(3):
            for c, a, o, s in zip(cs, args, outs, side):
                s.wait_stream(cur)
                with torch.cuda.stream(s):
                    api.pg_attention(c.pb, c.q, c.Kp, c.Vp, c.plen, *a, o, None, c.ws)
        for s in side:
            cur.wait_stream(s)
    for _ in range(5):
        for o in outs:
            o.fill_(3.0)
        g.replay()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
    api.kve_check_device()


@pytest.mark.parametrize("pair", TWO, ids=["bf16", "mixed"])
def test_attention_from_two_threads(pair):
    cs = [Case(*c, seed=83 + i) for i, c in enumerate(pair)]
    want = [c.run()[0] for c in cs]
    args = [c.args() for c in cs]
    outs = [[torch.full_like(w, 3.0) for _ in range(8)] for w in want]
    faults = []
    torch.cuda.synchronize()

    def calls(c, a, o):
        try:
            s = torch.cuda.Stream()
            for k in range(400):
                api.pg_attention(c.pb, c.q, c.Kp, c.Vp, c.plen, *a, o[k % 8], None, c.ws, stream=s)
            s.synchronize()
        except Exception as e:
            faults.append(e)

    threads = [threading.Thread(target=calls, args=x) for x in zip(cs, args, outs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    api.kve_check_device()
    assert not faults
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)
