"""Measured cases of the 4-bit cache: prompts quantised as a whole, rows quantised as they are written
into pages, both read back, and the attention of a batch over such prompts and pages.

Every operator has a plain form here (elementary torch operations in 32 bits) next to the
framework's call; ``own`` selects which one ``run`` computes.

What a cache holds: a row of a KV head in groups of ``group`` neighbouring channels, each with a step
s and whole numbers m, for the values s m. With lo = min(0, least value), hi = max(0, largest value):
  * s is the smallest number of four significant bits, 2^-126 at least, with 15 s >= hi - lo;
  * M = floor(F / s), F the largest finite number of the rows' type; k = min(M, -lo / s to the nearest);
  * m = x / s to the nearest, no less than -k and no more than min(15 - k, M).
What lies halfway goes toward zero. A group that holds an infinity or a NaN stands for NaN.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases ---------------------------------------------------------------------------------------
def _append(name, reqs, new_hi, heads, d, group, page, dtype):
    """reqs requests write 1..new_hi rows each into their pages, then all of them are read back."""
    return {"name": name, "op": "append", "reqs": reqs, "new_hi": new_hi, "heads": heads, "d": d,
            "group": group, "page": page, "dtype": dtype}


def _pack(name, prompts, heads, n, d, group, dtype, ragged=False):
    """Prompts of n rows (ragged: 7/8 n to n) are quantised, then read back."""
    return {"name": name, "op": "pack", "prompts": prompts, "heads": heads, "n": n, "d": d,
            "group": group, "dtype": dtype, "ragged": ragged}


def _unpack(name, prompts, heads, n, d, group, dtype, ragged=False):
    """Prompts of n rows that lie in 4 bits are read back."""
    return dict(_pack(name, prompts, heads, n, d, group, dtype, ragged), op="unpack")


def _attend(name, prompts, fan, hq, hkv, d, group, n, page, own_lo, own_hi, new_hi, dtype,
            ragged=False):
    """own_lo..own_hi: rows a request has in its pages, the new ones apart; new_hi: new rows per
    request are 1..new_hi; n 0: requests without a prompt before their pages."""
    return {"name": name, "op": "attend", "prompts": prompts, "fan": fan, "hq": hq, "hkv": hkv,
            "d": d, "group": group, "n": n, "page": page, "own_lo": own_lo, "own_hi": own_hi,
            "new_hi": new_hi, "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # the K/V rows of one decode step of a small batch, out of the fused projection's output
        _append("append 32 rows", 32, 1, 8, 128, 32, 16, "bf16"),
        # ragged prompts entered at once
        _append("append 64 prompts", 64, 2000, 8, 128, 64, 64, "f16"),
        # the cache that the small fp32 workload's eviction leaves (sink 4, 128 kept, window 32)
        _pack("pack 164 rows fp32", 1, 1, 164, 64, 32, "f32"),
        # one layer of the 128K prompt (8 KV heads)
        _pack("pack 128K", 1, 8, 131072, 128, 32, "bf16"),
        # one layer of the 16K prompt read back, for the next eviction pass over it
        _unpack("unpack 16K", 1, 8, 16384, 128, 32, "bf16"),
        # one layer of four ragged 32K prompts
        _unpack("unpack 4x32K", 4, 8, 32768, 128, 128, "f16", True),
        # the small fp32 workload (one head)
        _attend("attend tiny fp32", 1, 4, 1, 1, 64, 32, 512, 16, 0, 7, 1, "f32"),
        # a step of four requests behind the 16K prompt (32/8 heads)
        _attend("attend 4 behind 16K", 1, 4, 32, 8, 128, 32, 16384, 16, 0, 7, 1, "bf16"),
        # one answer decoded behind the 128K prompt
        _attend("attend 1 behind 128K", 1, 1, 32, 8, 128, 32, 131072, 16, 0, 511, 1, "bf16"),
        # a decode batch of requests with long caches of their own
        _attend("attend 64 caches", 64, 1, 32, 8, 128, 64, 0, 64, 1, 16384, 1, "bf16"),
        # a large serving batch behind one 8K system prompt
        _attend("attend 256 behind 8K", 1, 256, 32, 8, 128, 32, 8192, 64, 0, 1023, 1, "f16"),
        # ragged continuations of two 16K prompts, up to 64 new rows each
        _attend("attend continuations", 2, 8, 40, 8, 128, 128, 16384, 32, 0, 512, 64, "bf16"),
    ]


_MAX_BYTES = 6.0e8
_MAX_FLOPS = 1.7e11


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    what = rng.random()
    d = rng.choice((128, 128, 64, 32))
    group = rng.choice([x for x in (32, 64, 128) if x <= d])
    page, dtype = rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "f16", "f32"))
    if what < 0.2:
        heads, new_hi = rng.choice((1, 4, 8, 16)), _log(rng, 1, 4096) if rng.random() < 0.7 else 1
        top = int(_MAX_BYTES / (8 * heads * d * _BYTES[dtype]))
        c = _append("", _log(rng, 1, min(1024, max(1, 2 * top // (new_hi + 1)))), new_hi, heads, d,
                    group, page, dtype)
    elif what < 0.5:
        heads, prompts = rng.choice((1, 4, 8, 16)), rng.choice((1, 1, 2, 4))
        top = int(_MAX_BYTES / (6 * prompts * heads * d * _BYTES[dtype]))
        c = (_pack if what < 0.35 else _unpack)("", prompts, heads, _log(rng, 1, min(top, 131072)),
                                                d, group, dtype, rng.random() < 0.3)
    else:
        while True:
            hq, hkv = rng.choice(((32, 8), (40, 8), (28, 4), (16, 16), (8, 1), (12, 4)))
            prompts, fan = rng.choice((1, 1, 2, 3)), _log(rng, 1, 256)
            n, own_hi = _log(rng, 1, 131072), _log(rng, 1, 2048)
            if rng.random() < 0.3:  # requests without a prompt
                prompts, fan, n, own_hi = fan, 1, 0, _log(rng, 1, 16384)
            c = _attend("", prompts, fan, hq, hkv, d, group, n, page, 0, own_hi,
                        rng.choice((1, 1, 1, _log(rng, 2, 64))), dtype, n > 0 and rng.random() < 0.3)
            w = work(c)
            # the plain form holds the fp32 logits of padded rows and each request's padded rows
            pad = c["prompts"] * c["fan"] * c["new_hi"] * hq
            logits = pad * (c["n"] + c["own_hi"] + 64) * 4
            dense = c["prompts"] * c["fan"] * hkv * (c["own_hi"] + 192) * c["d"] * 4
            flops = _MAX_FLOPS if dtype != "f32" else _MAX_FLOPS / 16
            if w["bytes"] < _MAX_BYTES and w["flops"] < flops and logits < 3e9 and dense < 4e9:
                break
    del c["name"]
    return c


def _row_bytes(case):
    """Of a head's row in 4 bits, K or V: codes and 16 bits per group."""
    return case["d"] / 2 + 2 * case["d"] / case["group"]


def work(case):
    es, d, packed = _BYTES[case["dtype"]], case["d"], _row_bytes(case)
    if case["op"] != "attend":
        rows = (_sum(1, case["new_hi"], case["reqs"]) if case["op"] == "append" else
                case["prompts"] * case["n"] * (15 / 16 if case["ragged"] else 1))
        # rows in (not for unpack), 4 bits written and read again, rows out
        ways = 1 if case["op"] == "unpack" else 2
        return {"bytes": 2.0 * rows * case["heads"] * ways * (d * es + packed), "flops": 0.0}
    reqs = case["prompts"] * case["fan"]
    rows = reqs * (case["new_hi"] + 1) / 2
    mine = (case["own_lo"] + case["own_hi"]) / 2 + (case["new_hi"] + 1) / 2
    n = case["n"] * (15 / 16 if case["ragged"] else 1)
    kv = 2.0 * case["hkv"] * packed * (case["prompts"] * n + reqs * mine)
    return {"bytes": kv + rows * case["hq"] * (2 * d * es + 4) + 4 * reqs * mine / case["page"],
            "flops": 4.0 * rows * case["hq"] * (n + mine) * d}


# ---- inputs --------------------------------------------------------------------------------------
class _State:
    pass


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _spread(lo, hi, n, gen):
    """n whole numbers evenly spread over lo..hi, in random order: their sum does not go by the
    seed."""
    at = torch.randperm(n, device="cuda", generator=gen)
    return (lo + (2 * at + 1) * (hi - lo + 1) // (2 * n)).to(torch.int32)


def _sum(lo, hi, n):
    return sum(lo + (2 * i + 1) * (hi - lo + 1) // (2 * n) for i in range(n))


def _ceil(a, b):
    return (a + b - 1) // b


def _keys(shape, mu, dt, gen):
    """Keys g + z mu with mu of length 2 per head and z Zipf-like: the distribution of the eviction
    workloads. mu broadcasts against [*shape][d]."""
    k = torch.randn(*shape, mu.shape[-1], device="cuda", generator=gen, dtype=dt)
    z = (1 / torch.rand(*shape, 1, device="cuda", generator=gen)).floor().clamp(max=8).to(dt)
    return k.addcmul_(z, mu.to(dt))


def _mu(heads, d, gen):
    mu = torch.randn(heads, d, device="cuda", generator=gen)
    return 2 * mu / mu.norm(dim=-1, keepdim=True)


def _prompts(case, mu, gen):
    """Rows [prompts][heads][n][d] of K and V and the prompts' lengths (None: all of n)."""
    S, n, dt = case["prompts"], case["n"], _DTYPES[case["dtype"]]
    K = _keys((S, len(mu), n), mu[:, None], dt, gen)
    V = torch.randn(K.shape, device="cuda", generator=gen, dtype=dt)
    lens = None
    if case["ragged"]:
        lens = torch.randint(n - n // 8, n + 1, (S,), device="cuda", generator=gen,
                             dtype=torch.int32)
    return K, V, lens


def _paged(lens, page, gen, s):
    """Distinct pages in random order for requests of these lengths: table, and the slot of every row
    of every request, request after request."""
    R = len(lens)
    have = _ceil(lens.long(), page)
    s.max_pages, s.n_pages = int(have.max()), int(have.sum()) + 3
    perm = torch.randperm(s.n_pages, device="cuda", generator=gen).to(torch.int32)
    first = have.cumsum(0) - have
    j = torch.arange(s.max_pages, device="cuda")
    at = (first[:, None] + j).clamp(max=s.n_pages - 1)
    s.table = torch.where(j < have[:, None], perm[at], 0).contiguous()
    req = torch.repeat_interleave(torch.arange(R, device="cuda"), lens.long())
    pos = torch.arange(len(req), device="cuda") - (lens.long().cumsum(0) - lens)[req]
    return (s.table[req, pos // page] * page + pos % page).to(torch.int32)


def _problem(s, case, rows, max_new, hq, hkv):
    from kv_cache_eviction_02_gb300 import api
    dtype = {"f32": api.KVE_F32, "bf16": api.KVE_BF16, "f16": api.KVE_F16}[case["dtype"]]
    return api.Q4Problem(n_prompts=case.get("prompts", 1), fan=case.get("fan", case.get("reqs", 1)),
                         n_q_heads=hq, n_kv_heads=hkv, d_head=case["d"], n_prefix=case.get("n", 0),
                         page_size=case.get("page", 16), n_pages=s.n_pages, max_pages=s.max_pages,
                         n_rows=rows, max_new=max_new, dtype=dtype, group=case["group"])


def _bytes(n):
    return torch.zeros(n, device="cuda", dtype=torch.uint8)


def _inputs(case, seed):
    """What a case starts from, before anything is quantised."""
    s, gen = _State(), _gen(seed)
    s.case, d, dt = case, case["d"], _DTYPES[case["dtype"]]
    if case["op"] == "append":
        heads = case["heads"]
        s.lens = _spread(1, case["new_hi"], case["reqs"], gen)
        s.rows = _sum(1, case["new_hi"], case["reqs"])
        # the fused projection's output: 2 * heads query heads, then K's and V's
        qkv = torch.randn(s.rows, 4 * heads, d, device="cuda", generator=gen, dtype=dt)
        s.K, s.V = qkv[:, 2 * heads:3 * heads], qkv[:, 3 * heads:]
        s.K.copy_(_keys((s.rows, heads), _mu(heads, d, gen), dt, gen))
        s.slots = _paged(s.lens, case["page"], gen, s)
        s.n_out = s.max_pages * case["page"]
    elif case["op"] != "attend":
        s.K, s.V, s.lens = _prompts(case, _mu(case["heads"], d, gen), gen)
        s.n_pages = s.max_pages = s.rows = 1
        s.n_out = case["n"]
    else:
        hq, hkv, R = case["hq"], case["hkv"], case["prompts"] * case["fan"]
        mu = _mu(hkv, d, gen)
        s.Kp, s.Vp, s.prefix_len = _prompts(case, mu, gen) if case["n"] else (None, None, None)
        s.nq = _spread(1, case["new_hi"], R, gen)
        s.lens = _spread(case["own_lo"], case["own_hi"], R, gen) + s.nq
        s.slots = _paged(s.lens, case["page"], gen, s)
        s.K = _keys((len(s.slots), hkv), mu, dt, gen)
        s.V = torch.randn(s.K.shape, device="cuda", generator=gen, dtype=dt)
        s.q_start = torch.zeros(R + 1, device="cuda", dtype=torch.int32)
        s.q_start[1:] = s.nq.cumsum(0)
        rows = _sum(1, case["new_hi"], R)
        s.rows = rows + 3  # a batch padded by a few rows
        s.row_req = torch.full((s.rows,), -1, device="cuda", dtype=torch.int32)
        s.row_req[:rows] = torch.repeat_interleave(torch.arange(R, device="cuda"), s.nq.long())
        # the fused projection's output
        qkv = torch.randn(s.rows, hq + 2 * hkv, d, device="cuda", generator=gen, dtype=dt)
        qkv[:, :hq].view(s.rows, hkv, hq // hkv, d).add_(2 * mu[:, None].to(dt))
        s.q = qkv[:, :hq]
        # rows that belong to nobody keep what they hold
        s.out = torch.randn(s.rows, hq, d, device="cuda", generator=gen, dtype=dt).mul_(0.02)
        s.lse = torch.randn(s.rows, hq, device="cuda", generator=gen)
    if case["op"] != "attend":
        shape = (case.get("prompts") or case["reqs"], case["heads"], s.n_out, d)
        s.K_out, s.V_out = (torch.zeros(shape, device="cuda", dtype=dt) for _ in range(2))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "append":
        if own:
            s.pb = _problem(s, case, s.rows, s.rows, case["heads"], case["heads"])
            s.pages = _bytes(s.pb.pool_bytes)
        else:
            s.pages = _empty_plain(s.n_pages, case["heads"], case["page"], case)
    elif case["op"] != "attend":
        if own:
            s.pb = _problem(s, case, 1, 1, case["heads"], case["heads"])
            s.prefix = _bytes(s.pb.prefix_bytes)
        else:
            s.prefix = _empty_plain(case["prompts"], case["heads"], case["n"], case)
        if case["op"] == "unpack":
            _pack_pass(s)
            del s.K, s.V
    else:
        if own:
            from kv_cache_eviction_02_gb300 import api
            # the rows go into the pages as they would over many steps
            total = len(s.slots)
            api.q4_append(pb := _problem(s, case, total, total, case["hkv"], case["hkv"]), s.K, s.V,
                          s.slots, pages := _bytes(pb.pool_bytes))
            s.pb = _problem(s, case, s.rows, case["new_hi"], case["hq"], case["hkv"])
            s.pages, s.prefix = pages, None
            if case["n"]:
                s.prefix = _bytes(s.pb.prefix_bytes)
                api.q4_pack(s.pb, s.Kp, s.Vp, s.prefix_len, s.prefix)
            s.ws = torch.empty(api.q4_workspace_size(s.pb), device="cuda", dtype=torch.uint8)
        else:
            s.pages = _empty_plain(s.n_pages, case["hkv"], case["page"], case)
            _append_plain(s)
            if case["n"]:
                s.prefix = [_quantise(x, case) for x in (s.Kp, s.Vp)]
        del s.K, s.V, s.Kp, s.Vp
    return s


# ---- one pass ------------------------------------------------------------------------------------
def _pack_pass(s):
    if own:
        from kv_cache_eviction_02_gb300 import api
        api.q4_pack(s.pb, s.K, s.V, s.lens, s.prefix)
    else:
        s.prefix = [_quantise(x, s.case) for x in (s.K, s.V)]


def run(s):
    op = s.case["op"]
    if own:
        from kv_cache_eviction_02_gb300 import api
        if op == "append":
            api.q4_append(s.pb, s.K, s.V, s.slots, s.pages)
            api.q4_unpack(s.pb, s.pages, s.table, s.lens, s.K_out, s.V_out)
        elif op == "attend":
            api.q4_attention(s.pb, s.q, s.prefix, s.prefix_len, s.pages, s.table, s.lens, s.q_start,
                             s.row_req, s.out, s.lse, s.ws)
        else:
            if op == "pack":
                _pack_pass(s)
            api.q4_unpack(s.pb, s.prefix, None, s.lens, s.K_out, s.V_out)
    elif op == "append":
        _append_plain(s)
        for to, cache in zip((s.K_out, s.V_out), s.pages):
            _read_plain(to, _gather(cache, s.table), s.lens)
    elif op == "attend":
        _attend_plain(s)
    else:
        if op == "pack":
            _pack_pass(s)
        for to, cache in zip((s.K_out, s.V_out), s.prefix):
            _read_plain(to, _value(cache), s.lens)
    if op == "attend":
        return {"out": s.out, "lse": s.lse}
    return {"K": s.K_out, "V": s.V_out}


# The plain cache: whole numbers m [...][d / group][group] in 8 bits and steps s [...][d / group][1].
def _empty_plain(count, heads, rows, case):
    shape = (count, heads, rows, case["d"] // case["group"])
    return [(torch.zeros(*shape, case["group"], device="cuda", dtype=torch.int8),
             torch.zeros(*shape, 1, device="cuda")) for _ in range(2)]


def _quantise(x, case):
    """Rows [...][d] as (m, s). The quotient of a 16-bit value and a step of four bits is nearer to a
    half than 2^-12 only where it is one, so 32 bits tell them apart; fp32 values take 64."""
    wide = torch.float64 if x.dtype == torch.float32 else torch.float32
    g = x.reshape(*x.shape[:-1], -1, case["group"])
    lo, hi = g.amin(-1, keepdim=True).double().clamp(max=0), g.amax(-1, keepdim=True).double().clamp(min=0)
    need = (hi - lo) / 15
    # rounded up to three bits behind the leading one: the other 49 of a 64-bit number's are cut off
    bits = need.clamp(min=2.0 ** -126).view(torch.int64) + (2 ** 49 - 1)
    s = torch.where(need.isfinite(), (bits >> 49 << 49).view(torch.float64), math.nan)
    most = (torch.finfo(x.dtype).max / s).floor()
    k = torch.minimum((-lo / s - 0.5).ceil(), most)
    top = torch.minimum(15 - k, most).to(wide)
    y = g.to(wide) / s.to(wide)
    m = ((y.abs() - 0.5).ceil() * y.sign()).clamp_(-k.to(wide), top)
    return m.nan_to_num_().to(torch.int8), s.float()


def _value(cache):
    m, s = cache
    return (m.float() * s).flatten(-2)


def _gather(cache, table):
    """Rows [requests][heads][width * page][d] through a table of pages."""
    m, s = (x[table].transpose(1, 2).flatten(2, 3) for x in cache)
    return _value((m, s))


def _read_plain(to, values, lens):
    if lens is None:
        to.copy_(values)
    else:
        there = torch.arange(to.shape[2], device=to.device) < lens[:, None]
        to.copy_(torch.where(there[:, None, :, None], values, to.float()))


def _append_plain(s):
    page, slots = s.case["page"], s.slots.long()
    for (m, step), rows in zip(s.pages, (s.K, s.V)):
        a, b = _quantise(rows, s.case)
        m[slots // page, :, slots % page] = a
        step[slots // page, :, slots % page] = b


def _attend_plain(s):
    c = s.case
    S, fan, hq, hkv, d, n, T = (c[k] for k in ("prompts", "fan", "hq", "hkv", "d", "n", "new_hi"))
    R, g, dev = S * fan, hq // hkv, s.q.device
    t = torch.arange(T, device=dev)
    q = s.q[(s.q_start[:-1, None] + t).clamp(max=s.rows - 1)].float() / math.sqrt(d)
    q = q.view(S, fan, T, hkv, g, d).permute(0, 3, 1, 2, 4, 5)       # S hkv fan T g d
    mine = q.transpose(1, 2).reshape(R, hkv, T * g, d)
    b = mine @ _gather(s.pages[0], s.table).transpose(-1, -2)
    last = (s.lens - s.nq)[:, None] + t                              # R T: the row's own position
    hidden = torch.arange(b.shape[-1], device=dev) > last[..., None]
    b.view(R, hkv, T, g, -1).masked_fill_(hidden[:, None, :, None], -math.inf)
    m = b.amax(-1, keepdim=True)

    def by_request(x):  # S hkv fan*T*g ... -> R hkv T*g ...
        return x.reshape(S, hkv, fan, T * g, -1).transpose(1, 2).reshape(R, hkv, T * g, -1)

    if n:
        a = q.reshape(S, hkv, fan * T * g, d) @ _value(s.prefix[0]).transpose(-1, -2)
        if s.prefix_len is not None:
            hidden = torch.arange(n, device=dev) >= s.prefix_len[:, None]
            a.masked_fill_(hidden[:, None, None], -math.inf)
        m = torch.maximum(by_request(a.amax(-1, keepdim=True)), m)
    b = b.sub_(m).exp_()
    total, o = b.sum(-1, keepdim=True), b @ _gather(s.pages[1], s.table)
    if n:
        a.sub_(m.view(S, fan, hkv, T * g, 1).transpose(1, 2).reshape(S, hkv, fan * T * g, 1)).exp_()
        total = total + by_request(a.sum(-1, keepdim=True))
        o = o + by_request(a @ _value(s.prefix[1]))
    o, lse = o / total, m + total.log()
    req = s.row_req.long().clamp(min=0)
    live = (s.row_req >= 0)[:, None]
    i = (torch.arange(s.rows, device=dev) - s.q_start[req]).clamp(0, T - 1)
    o = o.view(R, hkv, T, g, d)[req, :, i].reshape(s.rows, hq, d)
    lse = lse.view(R, hkv, T, g)[req, :, i].reshape(s.rows, hq)
    s.out.copy_(torch.where(live[..., None], o, s.out.float()))
    s.lse.copy_(torch.where(live, lse, s.lse))


# ---- from the definitions, in 64 bits --------------------------------------------------------------
def _stands_for(rows, group):
    """The values that rows [...][d] are held as: of all multiples that a group has, the nearest, of
    two equally near the one nearer to zero. Steps are found by halving from 2^127 down and then
    taking eighths of a power of two."""
    x = rows.double().unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
    span, largest = hi - lo, torch.finfo(rows.dtype).max
    power = torch.full_like(span, 2.0 ** 127)
    for e in range(126, -127, -1):
        power = torch.where(15 * 2.0 ** e >= span, 2.0 ** e, power)
    s = power  # the smallest power of two that is enough; below it, the eighths of its half
    for eighth in range(15, 8, -1):
        t = power / 2 * (eighth / 8)
        s = torch.where((15 * t >= span) & (t >= 2.0 ** -126), t, s)

    def nearest(y, least, most):
        best, off = torch.zeros_like(y), y.abs()
        for size in range(1, 16):
            for m in (-size, size):
                d = (y - m * s).abs()
                fits = (m >= least) & (m <= most) & (abs(m) * s <= largest) & (d < off)
                best, off = torch.where(fits, float(m), best), torch.where(fits, d, off)
        return best

    k = nearest(-lo, 0, 15)
    v = nearest(x, -k, 15 - k) * s
    return torch.where(x.isfinite().all(-1, keepdim=True), v, math.nan).flatten(-2)


def exact(case, seed):
    s, group = _inputs(case, seed), case["group"]
    if case["op"] != "attend":
        K, V = s.K_out.double(), s.V_out.double()
        lens = s.lens.tolist() if s.lens is not None else [case["n"]] * case["prompts"]
        first = 0
        for r, count in enumerate(lens):
            for h in range(case["heads"]):
                at = (slice(first, first + count), h) if case["op"] == "append" else (r, h, slice(0, count))
                K[r, h, :count] = _stands_for(s.K[at], group)
                V[r, h, :count] = _stands_for(s.V[at], group)
            first += count
        return {"K": K, "V": V}
    out, lse = s.out.double(), s.lse.double()
    g, fan, hkv = case["hq"] // case["hkv"], case["fan"], case["hkv"]
    starts, lens = s.q_start.tolist(), s.lens.tolist()
    ends = s.prefix_len.tolist() if s.prefix_len is not None else [case["n"]] * case["prompts"]
    first = 0
    for r in range(case["prompts"] * fan):
        if r % fan == 0 and case["n"]:
            p = r // fan
            kp, vp = (torch.stack([_stands_for(x[p, h, :ends[p]], group) for h in range(hkv)])
                      for x in (s.Kp, s.Vp))
        k, v = (_stands_for(x[first:first + lens[r]].transpose(0, 1), group) for x in (s.K, s.V))
        first += lens[r]
        if case["n"]:
            k, v = torch.cat((kp, k), 1), torch.cat((vp, v), 1)
        # row i of the request sees the prompt and its own rows up to itself
        at, count = starts[r], starts[r + 1] - starts[r]
        q = s.q[at:at + count].double().view(count, hkv, g, case["d"])
        sees = k.shape[1] - count + torch.arange(count, device="cuda")
        step = max(1, 2 ** 26 // (case["hq"] * k.shape[1]))
        for i in range(0, count, step):
            x = torch.einsum("ihgd,hnd->hign", q[i:i + step], k) / math.sqrt(case["d"])
            x.masked_fill_((torch.arange(k.shape[1], device="cuda") > sees[i:i + step, None])[:, None],
                           -math.inf)
            z = torch.logsumexp(x, -1)
            o = torch.einsum("hign,hnd->ihgd", (x - z[..., None]).exp(), v)
            out[at + i:at + i + len(o)] = o.reshape(-1, case["hq"], case["d"])
            lse[at + i:at + i + len(o)] = z.permute(1, 0, 2).reshape(-1, case["hq"])
    return {"out": out, "lse": lse}
