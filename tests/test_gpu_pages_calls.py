"""Shared-prompt calls made the way a program makes them: from several threads at once."""
import threading

import numpy as np
import pytest
import torch

from kv_cache_eviction_02_gb300 import api
from oracle import shared_prompt as sp
from test_gpu_pages import DEV, f64

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
