"""Measured cases of the shared-prompt decoding operators: the page planner, the paged append and
the attention of a batch over one shared prompt cache plus each request's own pages.

Every operator has a plain form here (elementary torch operations in 32 bits) next to the
framework's call; ``own`` selects which one ``run`` computes.

The setting: ``prompts`` cached prompts, each continued by ``fan`` requests (the Monte Carlo
trajectories of the lookahead, or the answers that are decoded from one compressed cache). The
requests of a prompt read its K/V together; what a request adds lies in its own pages.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases ---------------------------------------------------------------------------------------
def _plan(name, fan, old_hi, new_hi, page, idle, tight=False):
    """old lengths 0..old_hi, new rows 1..new_hi; idle: share of requests that add nothing, and a
    quarter of it of requests that have finished; tight: fewer free pages than wanted."""
    return {"name": name, "op": "plan", "fan": fan, "old_hi": old_hi, "new_hi": new_hi,
            "page": page, "idle": idle, "tight": tight}


def _append(name, rows, heads, d, page, dtype):
    return {"name": name, "op": "append", "rows": rows, "heads": heads, "d": d, "page": page,
            "dtype": dtype}


def _attend(name, prompts, fan, hq, hkv, d, n, page, own_lo, own_hi, new_hi, dtype, ragged=False):
    """own_lo..own_hi: rows a request has in its pages, the new ones apart; new_hi: new rows per
    request are 1..new_hi; ragged: prompts of 7/8 n to n rows."""
    return {"name": name, "op": "attend", "prompts": prompts, "fan": fan, "hq": hq, "hkv": hkv,
            "d": d, "n": n, "page": page, "own_lo": own_lo, "own_hi": own_hi, "new_hi": new_hi,
            "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # one step of the lookahead's four trajectories: the smallest call, all latency
        _plan("plan 4 trajectories", 4, 7, 1, 16, 0.0),
        # a decode step of a full batch: some requests wait, some have finished and return pages
        _plan("plan 512 decoding", 512, 4095, 1, 16, 0.125),
        # ragged prompts entered at once
        _plan("plan 256 prompts", 256, 512, 2048, 64, 0.0),
        # the K/V rows of one decode step of a small batch, out of the fused projection's output
        _append("append 32 rows", 32, 8, 128, 16, "bf16"),
        # the K/V rows of a large prompt batch
        _append("append 64K rows", 65536, 8, 128, 64, "bf16"),
        # the small fp32 workload (one head)
        _attend("attend tiny fp32", 1, 4, 1, 1, 64, 512, 16, 0, 7, 1, "f32"),
        # lookahead step over the 16K prompt (32/8 heads)
        _attend("attend lookahead 16K", 1, 4, 32, 8, 128, 16384, 16, 0, 7, 1, "bf16"),
        # lookahead step over the 128K prompt
        _attend("attend lookahead 128K", 1, 4, 32, 8, 128, 131072, 16, 0, 7, 1, "bf16"),
        # lookahead step of four ragged 32K prompts (40/8 heads)
        _attend("attend lookahead 4x32K", 4, 4, 40, 8, 128, 32768, 16, 0, 7, 1, "bf16", True),
        # 64 answers decoded from one compressed cache (sink 4 + 128 kept + window 32 rows)
        _attend("attend 64 answers", 1, 64, 32, 8, 128, 164, 16, 0, 1023, 1, "bf16"),
        # a large serving batch behind one 8K system prompt
        _attend("attend 256 behind 8K", 1, 256, 32, 8, 128, 8192, 64, 0, 1023, 1, "f16"),
        # ragged continuations of two 16K prompts, up to 64 new rows each
        _attend("attend continuations", 2, 8, 40, 8, 128, 16384, 32, 0, 512, 64, "bf16"),
    ]


_MAX_BYTES = 5.0e8
_MAX_FLOPS = 1.7e11


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    what = rng.random()
    if what < 0.2:
        fan = _log(rng, 1, 2048)
        new_hi = _log(rng, 1, 2048) if rng.random() < 0.5 else 1
        new_hi = max(1, min(new_hi, 2 ** 18 // fan))
        c = _plan("", fan, _log(rng, 1, 8192), new_hi, rng.choice((8, 16, 32, 64, 128)),
                  rng.choice((0.0, 0.125, 0.25)), rng.random() < 0.2)
    elif what < 0.4:
        heads, d, dtype = rng.choice((1, 4, 8, 16)), rng.choice((32, 64, 128)), rng.choice(
            ("bf16", "f16", "f32"))
        top = int(_MAX_BYTES / (4 * heads * d * _BYTES[dtype]))
        c = _append("", _log(rng, 1, min(top, 65536)), heads, d, rng.choice((8, 16, 32, 64, 128)),
                    dtype)
    else:
        while True:
            hq, hkv = rng.choice(((32, 8), (40, 8), (28, 4), (16, 16), (8, 1), (12, 4)))
            dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
            prompts = rng.choice((1, 1, 2, 3))
            c = _attend("", prompts, _log(rng, 1, 256), hq, hkv, rng.choice((128, 128, 64, 32)),
                        _log(rng, 1, 131072), rng.choice((8, 16, 32, 64, 128)), 0,
                        _log(rng, 1, 2048), rng.choice((1, 1, 1, _log(rng, 2, 64))), dtype,
                        rng.random() < 0.3)
            w = work(c)
            # the plain form holds the fp32 logits of padded rows and each request's padded rows
            pad = c["prompts"] * c["fan"] * c["new_hi"] * hq
            logits = pad * (c["n"] + c["own_hi"] + 64) * 4
            dense = c["prompts"] * c["fan"] * hkv * (c["own_hi"] + 192) * c["d"] * 4
            flops = _MAX_FLOPS if dtype != "f32" else _MAX_FLOPS / 16
            if w["bytes"] < _MAX_BYTES and w["flops"] < flops and logits < 3e9 and dense < 3e9:
                break
    del c["name"]
    return c


def work(case):
    if case["op"] == "plan":
        rows = _sum(1, case["new_hi"], case["fan"])
        pages = rows * (1 - 1.25 * case["idle"]) / case["page"]  # on average
        # new and old lengths in, lengths and row starts out; every new page is read from the free
        # list and written to its table; three words per row out
        return {"bytes": 16.0 * case["fan"] + 8 * pages + 12 * rows, "flops": 0.0}
    if case["op"] == "append":
        return {"bytes": 2.0 * 2 * case["rows"] * case["heads"] * case["d"] * _BYTES[case["dtype"]]
                + 4 * case["rows"], "flops": 0.0}
    es, d = _BYTES[case["dtype"]], case["d"]
    reqs = case["prompts"] * case["fan"]
    rows = reqs * (case["new_hi"] + 1) / 2
    mine = (case["own_lo"] + case["own_hi"]) / 2 + (case["new_hi"] + 1) / 2
    n = case["n"] * (15 / 16 if case["ragged"] else 1)
    kv = 2.0 * case["hkv"] * d * es * (case["prompts"] * n + reqs * mine)
    return {"bytes": kv + rows * case["hq"] * (2 * d * es + 4) + 4 * reqs * mine / case["page"],
            "flops": 4.0 * rows * case["hq"] * (n + mine) * d}


# ---- inputs --------------------------------------------------------------------------------------
class _State:
    pass


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(lo, hi, n, gen):
    return torch.randint(lo, hi + 1, (n,), device="cuda", generator=gen, dtype=torch.int32)


def _spread(lo, hi, n, gen):
    """n whole numbers evenly spread over lo..hi, in random order: their sum does not go by the
    seed."""
    at = torch.randperm(n, device="cuda", generator=gen)
    return (lo + (2 * at + 1) * (hi - lo + 1) // (2 * n)).to(torch.int32)


def _sum(lo, hi, n):
    return sum(lo + (2 * i + 1) * (hi - lo + 1) // (2 * n) for i in range(n))


def _i32(*shape, fill=-1):
    return torch.full(shape, fill, device="cuda", dtype=torch.int32)


def _ceil(a, b):
    return (a + b - 1) // b


def prepare(case, seed):
    return {"plan": _prepare_plan, "append": _prepare_append, "attend": _prepare_attend}[
        case["op"]](case, _gen(seed))


def _problem(**kw):
    from kv_cache_eviction_02_gb300 import api
    kw["dtype"] = {"f32": api.KVE_F32, "bf16": api.KVE_BF16, "f16": api.KVE_F16}[kw["dtype"]]
    return api.PgProblem(**kw)


def _prepare_plan(case, gen):
    s = _State()
    s.case, fan, page = case, case["fan"], case["page"]
    s.len_in = _spread(0, case["old_hi"], fan, gen)
    s.new = _spread(1, case["new_hi"], fan, gen)
    if case["idle"]:
        u = torch.rand(fan, device="cuda", generator=gen)
        s.new = torch.where(u < 1.25 * case["idle"], 0, s.new)
        s.new = torch.where(u < 0.25 * case["idle"], -1, s.new).to(torch.int32)
    s.max_pages = _ceil(case["old_hi"] + case["new_hi"], page)
    have = _ceil(s.len_in.long(), page)
    wanted = _ceil(s.len_in.long() + s.new.clamp(min=0), page) - have
    used, free = int(have.sum()), int(wanted.sum())
    free = free // 2 if case["tight"] else free + free // 4 + 3
    s.n_pages = (_sum(0, case["old_hi"], fan) + _sum(1, case["new_hi"], fan)) // page + 2 * fan + 8
    free = min(free, s.n_pages - used)
    perm = torch.randperm(s.n_pages, device="cuda", generator=gen).to(torch.int32)
    first = have.cumsum(0) - have
    j = torch.arange(s.max_pages, device="cuda")
    at = (first[:, None] + j).clamp(max=s.n_pages - 1)
    s.table = torch.where(j < have[:, None], perm[at], -1).contiguous()
    # the free pages stand in a ring, from `head` on
    head = int(torch.randint(0, s.n_pages, (1,), device="cuda", generator=gen))
    s.free = _i32(s.n_pages)
    ring = (head + torch.arange(free, device="cuda")) % s.n_pages
    s.free[ring] = perm[used:used + free]
    s.pool_in = torch.tensor([head, free, 0, 0], device="cuda", dtype=torch.int32)
    s.rows = _sum(1, case["new_hi"], fan) + 3  # a batch padded by a few rows
    s.len_out, s.pool_out, s.q_start = _i32(fan), _i32(4), _i32(fan + 1)
    s.row_req, s.row_pos, s.slots = _i32(s.rows), _i32(s.rows), _i32(s.rows)
    if own:
        s.pb = _problem(n_prompts=1, fan=fan, n_q_heads=1, n_kv_heads=1, d_head=128, n_prefix=0,
                        page_size=page, n_pages=s.n_pages, max_pages=s.max_pages, n_rows=s.rows,
                        max_new=case["new_hi"], dtype="bf16")
    return s


def _prepare_append(case, gen):
    s = _State()
    s.case = case
    rows, heads, d, page, dt = (case["rows"], case["heads"], case["d"], case["page"],
                                _DTYPES[case["dtype"]])
    # the fused projection's output: 2 * heads query heads, then K's and V's
    qkv = torch.randn(rows, 4 * heads, d, device="cuda", generator=gen, dtype=dt)
    s.K_new, s.V_new = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
    s.n_pages = _ceil(rows, page) + 7
    perm = torch.randperm(s.n_pages, device="cuda", generator=gen).to(torch.int32)
    i = torch.arange(rows, device="cuda")
    s.slots = (perm[i // page] * page + i % page).to(torch.int32)
    s.slots[rows - rows // 16:] = -1  # a padded batch: the last rows belong to nobody
    s.K_pages = torch.randn(s.n_pages, heads, page, d, device="cuda", generator=gen, dtype=dt)
    s.V_pages = torch.randn(s.n_pages, heads, page, d, device="cuda", generator=gen, dtype=dt)
    if own:
        s.pb = _problem(n_prompts=1, fan=1, n_q_heads=heads, n_kv_heads=heads, d_head=d,
                        n_prefix=0, page_size=page, n_pages=s.n_pages, max_pages=s.n_pages,
                        n_rows=rows, max_new=rows, dtype=case["dtype"])
    return s


def _prepare_attend(case, gen):
    """Keys g + s mu with mu of length 2 per head and s Zipf-like, queries g + 2 mu, values normal:
    the distribution of the eviction workloads."""
    s = _State()
    s.case = case
    S, fan, hq, hkv, d, n, page = (case[k] for k in ("prompts", "fan", "hq", "hkv", "d", "n",
                                                     "page"))
    dt, R, g = _DTYPES[case["dtype"]], S * fan, hq // hkv
    mu = torch.randn(hkv, 1, d, device="cuda", generator=gen)
    mu = 2 * mu / mu.norm(dim=-1, keepdim=True)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=dt)

    def keys(*shape):
        k = normal(*shape, d)
        z = (1 / torch.rand(*shape, 1, device="cuda", generator=gen)).floor().clamp(max=8).to(dt)
        return k.addcmul_(z, mu.to(dt))

    s.K_prefix, s.V_prefix = keys(S, hkv, n), normal(S, hkv, n, d)
    s.prefix_len = _ints(n - n // 8, n, S, gen) if case["ragged"] else None
    nq = _spread(1, case["new_hi"], R, gen)
    s.lens = _spread(case["own_lo"], case["own_hi"], R, gen) + nq
    s.max_pages = _ceil(case["own_hi"] + case["new_hi"], page)
    have = _ceil(s.lens.long(), page)
    s.n_pages = (_sum(case["own_lo"], case["own_hi"], R) + _sum(1, case["new_hi"], R)) // page + R
    perm = torch.randperm(s.n_pages, device="cuda", generator=gen).to(torch.int32)
    first = have.cumsum(0) - have
    j = torch.arange(s.max_pages, device="cuda")
    at = (first[:, None] + j).clamp(max=s.n_pages - 1)
    s.table = torch.where(j < have[:, None], perm[at], 0).contiguous()
    s.K_pages, s.V_pages = keys(s.n_pages, hkv, page), normal(s.n_pages, hkv, page, d)
    s.q_start = _i32(R + 1, fill=0)
    s.q_start[1:] = nq.cumsum(0)
    rows = int(nq.sum())
    s.rows = rows + 3  # a batch padded by a few rows
    s.row_req = _i32(s.rows)
    s.row_req[:rows] = torch.repeat_interleave(torch.arange(R, device="cuda"), nq.long())
    qkv = normal(s.rows, hq + 2 * hkv, d)  # the fused projection's output
    qkv[:, :hq].view(s.rows, hkv, g, d).add_(2 * mu.to(dt))
    s.q = qkv[:, :hq]
    s.out = normal(s.rows, hq, d).mul_(0.02)  # rows that belong to nobody keep what they hold
    s.lse = torch.randn(s.rows, hq, device="cuda", generator=gen)
    if own:
        from kv_cache_eviction_02_gb300 import api
        s.pb = _problem(n_prompts=S, fan=fan, n_q_heads=hq, n_kv_heads=hkv, d_head=d, n_prefix=n,
                        page_size=page, n_pages=s.n_pages, max_pages=s.max_pages, n_rows=s.rows,
                        max_new=case["new_hi"], dtype=case["dtype"])
        s.ws = torch.empty(api.pg_workspace_size(s.pb), device="cuda", dtype=torch.uint8)
    return s


# ---- one pass ------------------------------------------------------------------------------------
def run(s):
    op = s.case["op"]
    if own:
        from kv_cache_eviction_02_gb300 import api
        if op == "plan":
            api.pg_plan(s.pb, s.new, s.len_in, s.pool_in, s.free, s.table, s.len_out, s.pool_out,
                        s.q_start, s.row_req, s.row_pos, s.slots)
        elif op == "append":
            api.pg_append(s.pb, s.K_new, s.V_new, s.slots, s.K_pages, s.V_pages)
        else:
            api.pg_attention(s.pb, s.q, s.K_prefix, s.V_prefix, s.prefix_len, s.K_pages, s.V_pages,
                             s.table, s.lens, s.q_start, s.row_req, s.out, s.lse, s.ws)
    else:
        {"plan": _plan_plain, "append": _append_plain, "attend": _attend_plain}[op](s)
    if op == "plan":
        return {"len": s.len_out, "pool": s.pool_out, "q_start": s.q_start, "row_req": s.row_req,
                "row_pos": s.row_pos, "slots": s.slots, "table": s.table, "free": s.free}
    if op == "append":
        return {"K": s.K_pages, "V": s.V_pages}
    return {"out": s.out, "lse": s.lse}


def _plan_plain(s):
    page, n_pages, dev = s.case["page"], s.n_pages, s.new.device
    old, new = s.len_in.long(), s.new.long()
    head, n_free = s.pool_in[0].long(), s.pool_in[1].long()
    add = new.clamp(min=0)
    have, need = _ceil(old, page), _ceil(old + add, page)
    ends = add.cumsum(0)
    bad = (new > s.case["new_hi"]) | (need > s.max_pages) | (ends > s.rows)
    want = torch.where(bad, 0, need - have)
    upto = want.cumsum(0)
    off = upto - want
    bad = bad | ((want > 0) & (upto > n_free))
    taken = torch.where(bad, 0, want)
    # pages: the i-th wanted page comes from the i-th place behind the ring's head
    j = torch.arange(s.max_pages, device=dev)
    fresh = (j >= have[:, None]) & (j < (have + taken)[:, None])
    page_id = s.free[(head + off[:, None] + j - have[:, None]) % n_pages]
    table = torch.where(fresh, page_id, s.table)
    # finished requests: their pages join the ring's end
    freed = torch.where(new < 0, have, 0)
    freed_upto = freed.cumsum(0)
    i = (torch.arange(n_pages, device=dev) - head - n_free) % n_pages
    who = torch.searchsorted(freed_upto, i, right=True).clamp(max=len(freed) - 1)
    back = (i - (freed_upto - freed)[who]).clamp(0, s.max_pages - 1)
    free = torch.where(i < freed_upto[-1], s.table[who, back], s.free)
    # rows
    row = torch.arange(s.rows, device=dev)
    req = torch.searchsorted(ends, row, right=True)
    live = req < len(new)
    req = req.clamp(max=len(new) - 1)
    live = live & ~bad[req]
    pos = old[req] + row - (ends - add)[req]
    at = (pos // page).clamp(0, s.max_pages - 1)
    slot = table[req, at].long() * page + pos % page
    s.q_start[0] = 0
    s.q_start[1:] = ends.clamp(max=s.rows)
    s.row_req.copy_(torch.where(live, req, -1))
    s.row_pos.copy_(torch.where(live, pos, -1))
    s.slots.copy_(torch.where(live, slot, -1))
    s.len_out.copy_(torch.where(new < 0, 0, torch.where(bad, old, old + add)))
    total = taken.sum()
    s.pool_out.copy_(torch.stack(((head + total) % n_pages, n_free - total + freed.sum(),
                                  ends[-1].clamp(max=s.rows), bad.sum())))
    s.table.copy_(table)
    s.free.copy_(free)


def _append_plain(s):
    page = s.case["page"]
    slots = s.slots.long()
    live = slots >= 0
    # rows of nobody repeat the first row that has a place
    row = torch.where(live, torch.arange(len(slots), device=slots.device), live.int().argmax())
    slot = slots[row]
    s.K_pages[slot // page, :, slot % page] = s.K_new[row]
    s.V_pages[slot // page, :, slot % page] = s.V_new[row]


def _attend_plain(s):
    c = s.case
    S, fan, hq, hkv, d, n, page, T = (c[k] for k in ("prompts", "fan", "hq", "hkv", "d", "n",
                                                     "page", "new_hi"))
    R, g, dev = S * fan, hq // hkv, s.q.device
    nq = s.q_start[1:] - s.q_start[:-1]
    t = torch.arange(T, device=dev)
    q = s.q[(s.q_start[:-1, None] + t).clamp(max=s.rows - 1)].float() / math.sqrt(d)
    q = q.view(S, fan, T, hkv, g, d).permute(0, 3, 1, 2, 4, 5)       # S hkv fan T g d
    a = q.reshape(S, hkv, fan * T * g, d) @ s.K_prefix.float().transpose(-1, -2)
    if s.prefix_len is not None:
        hidden = torch.arange(n, device=dev) >= s.prefix_len[:, None]
        a.masked_fill_(hidden[:, None, None], -math.inf)
    mine = q.transpose(1, 2).reshape(R, hkv, T * g, d)
    ks = s.K_pages[s.table].transpose(1, 2).reshape(R, hkv, -1, d).float()
    vs = s.V_pages[s.table].transpose(1, 2).reshape(R, hkv, -1, d).float()
    b = mine @ ks.transpose(-1, -2)
    last = (s.lens - nq)[:, None] + t                                # R T: the row's own position
    hidden = torch.arange(b.shape[-1], device=dev) > last[..., None]
    b.view(R, hkv, T, g, -1).masked_fill_(hidden[:, None, :, None], -math.inf)

    def by_request(x):  # S hkv fan*T*g ... -> R hkv T*g ...
        return x.reshape(S, hkv, fan, T * g, -1).transpose(1, 2).reshape(R, hkv, T * g, -1)

    def by_prompt(x):
        return x.reshape(S, fan, hkv, T * g, -1).transpose(1, 2).reshape(S, hkv, fan * T * g, -1)

    m = torch.maximum(by_request(a.amax(-1, keepdim=True)), b.amax(-1, keepdim=True))
    a = a.sub_(by_prompt(m)).exp_()
    b = b.sub_(m).exp_()
    total = by_request(a.sum(-1, keepdim=True)) + b.sum(-1, keepdim=True)
    o = (by_request(a @ s.V_prefix.float()) + b @ vs) / total
    lse = m + total.log()
    req = s.row_req.long().clamp(min=0)
    live = (s.row_req >= 0)[:, None]
    i = (torch.arange(s.rows, device=dev) - s.q_start[req]).clamp(0, T - 1)
    o = o.view(R, hkv, T, g, d)[req, :, i].reshape(s.rows, hq, d)
    lse = lse.view(R, hkv, T, g)[req, :, i].reshape(s.rows, hq)
    s.out.copy_(torch.where(live[..., None], o, s.out.float()))
    s.lse.copy_(torch.where(live, lse, s.lse))


# ---- from the definitions, in 64 bits --------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        K, V = s.K_pages.double(), s.V_pages.double()
        at = s.slots.tolist()
        rows = torch.tensor([i for i, x in enumerate(at) if x >= 0], device="cuda",
                            dtype=torch.long)
        p = torch.tensor([x // case["page"] for x in at if x >= 0], device="cuda", dtype=torch.long)
        o = torch.tensor([x % case["page"] for x in at if x >= 0], device="cuda", dtype=torch.long)
        for h in range(case["heads"]):
            K[p, h, o] = s.K_new[rows, h].double()
            V[p, h, o] = s.V_new[rows, h].double()
        return {"K": K, "V": V}
    out, lse = s.out.double(), s.lse.double()
    g, page, fan = case["hq"] // case["hkv"], case["page"], case["fan"]
    starts, lens, table = s.q_start.tolist(), s.lens.tolist(), s.table.tolist()
    ends = s.prefix_len.tolist() if s.prefix_len is not None else [case["n"]] * case["prompts"]
    for r in range(case["prompts"] * fan):
        first, count = starts[r], starts[r + 1] - starts[r]
        pages = table[r][:_ceil(lens[r], page)]
        k2 = s.K_pages[pages].transpose(0, 1).flatten(1, 2)[:, :lens[r]]
        v2 = s.V_pages[pages].transpose(0, 1).flatten(1, 2)[:, :lens[r]]
        k = torch.cat((s.K_prefix[r // fan, :, :ends[r // fan]], k2), 1).double()
        v = torch.cat((s.V_prefix[r // fan, :, :ends[r // fan]], v2), 1).double()
        # row i of the request sees the prompt and its own rows up to itself
        q = s.q[first:first + count].double().view(count, case["hkv"], g, case["d"])
        x = torch.einsum("ihgd,hnd->hign", q, k) / math.sqrt(case["d"])
        sees = ends[r // fan] + lens[r] - count + torch.arange(count, device="cuda")
        x.masked_fill_((torch.arange(k.shape[1], device="cuda") > sees[:, None])[:, None],
                       -math.inf)
        z = torch.logsumexp(x, -1)
        o = torch.einsum("hign,hnd->ihgd", (x - z[..., None]).exp(), v)
        out[first:first + count] = o.reshape(count, case["hq"], case["d"])
        lse[first:first + count] = z.permute(1, 0, 2).reshape(count, case["hq"])
    return {"out": out, "lse": lse}
