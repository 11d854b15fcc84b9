"""Oracle of shared-prompt decoding in fp64 (test infrastructure only): the page planner step by
step in request order, and the attention of a step's rows by its definition, one row and head at a
time over the rows it sees."""
from __future__ import annotations

import math

import numpy as np


def pg_plan(new_len, lens, pool, free_pages, table, page, max_new, n_rows):
    """One step of the planner: the arrays as pg_plan leaves them (inputs are not changed)."""
    lens, table, ring = list(map(int, lens)), np.array(table), np.array(free_pages)
    R, max_pages = table.shape
    n_pages, head, free = len(ring), int(pool[0]), int(pool[1])
    old_ring = ring.copy()
    taken = back = refused = rows = 0
    dry = False  # a request found too few pages: later ones that need pages find none either
    q_start = [0]
    row = {"row_req": np.full(n_rows, -1), "row_pos": np.full(n_rows, -1),
           "slot_map": np.full(n_rows, -1)}
    for r in range(R):
        new, old = int(new_len[r]), lens[r]
        first = rows
        rows = min(rows + max(new, 0), n_rows + 1)
        q_start.append(min(rows, n_rows))
        if new == 0:
            continue
        if not 0 <= old <= max_pages * page:
            refused += 1
            continue
        have = math.ceil(old / page)
        if new < 0:
            for j in range(have):
                ring[(head + free + back) % n_pages] = table[r, j]
                back += 1
            lens[r] = 0
            continue
        want = math.ceil((old + new) / page) - have
        if new > max_new or rows > n_rows or old + new > max_pages * page:
            refused += 1
            continue
        if want and (dry or taken + want > free):
            refused += 1
            dry = True
            continue
        for j in range(want):
            table[r, have + j] = old_ring[(head + taken) % n_pages]
            taken += 1
        for i in range(new):
            pos = old + i
            row["row_req"][first + i] = r
            row["row_pos"][first + i] = pos
            row["slot_map"][first + i] = table[r, pos // page] * page + pos % page
        lens[r] = old + new
    out = {k: v.astype(np.int32) for k, v in row.items()}
    out.update(len=np.array(lens, np.int32), q_start=np.array(q_start, np.int32),
               block_table=table.astype(np.int32), free_pages=ring.astype(np.int32),
               pool=np.array([(head + taken) % n_pages, free - taken + back, q_start[-1], refused],
                             np.int32))
    return out


def own_rows(pages, table_row, n):
    """The first n own rows of a request, [Hkv][n][d], through its block table."""
    page = pages.shape[2]
    at = np.arange(n)
    ids = np.asarray(table_row)[at // page]
    return pages[ids, :, at % page].transpose(1, 0, 2) if n else np.zeros(
        (pages.shape[1], 0, pages.shape[3]))


def pg_attention(q, K_prefix, V_prefix, prefix_len, K_pages, V_pages, table, lens, q_start, fan,
                 rows=None):
    """out [rows][Hq][d], lse [rows][Hq] in fp64, plus the magnitudes a bound on rounding needs:
    terms = sum_j a_j |v_j| and mag = max_j sum_c |q_c k_jc| / sqrt(d). Rows that no request holds
    are NaN. `rows`: only these packed rows."""
    q = np.asarray(q, np.float64)
    n_rows, Hq, d = q.shape
    Hkv = K_pages.shape[1]
    g = Hq // Hkv
    out = np.full((n_rows, Hq, d), np.nan)
    terms = np.full((n_rows, Hq, d), np.nan)
    lse = np.full((n_rows, Hq), np.nan)
    mag = np.full((n_rows, Hq), np.nan)
    for r in range(len(lens)):
        first, count = int(q_start[r]), int(q_start[r + 1] - q_start[r])
        if count == 0 or (rows is not None and not any(first <= i < first + count for i in rows)):
            continue
        n = int(prefix_len[r // fan])
        k2 = own_rows(K_pages, table[r], int(lens[r])).astype(np.float64)
        v2 = own_rows(V_pages, table[r], int(lens[r])).astype(np.float64)
        k, v = k2, v2
        if n:
            k = np.concatenate((K_prefix[r // fan, :, :n].astype(np.float64), k2), 1)
            v = np.concatenate((V_prefix[r // fan, :, :n].astype(np.float64), v2), 1)
        for i in range(count):
            if rows is not None and first + i not in rows:
                continue
            sees = n + max(0, int(lens[r]) - count + i + 1)
            for h in range(Hq):
                kk, vv = k[h // g, :sees], v[h // g, :sees]
                if sees == 0:
                    out[first + i, h] = terms[first + i, h] = mag[first + i, h] = 0
                    lse[first + i, h] = -np.inf
                    continue
                s = kk @ q[first + i, h] / math.sqrt(d)
                z = s.max() + math.log(np.exp(s - s.max()).sum())
                a = np.exp(s - z)
                out[first + i, h] = a @ vv
                terms[first + i, h] = a @ np.abs(vv)
                lse[first + i, h] = z
                mag[first + i, h] = (np.abs(kk) @ np.abs(q[first + i, h])).max() / math.sqrt(d)
    return {"out": out, "lse": lse, "terms": terms, "mag": mag}
