"""The 4-bit cache operators: writing a paged cache, reading it back, and attention over it.

A cached row of 512 values is held as 256 bytes of e2m1 codes (element 2j in the low nibble of byte j), 32 bytes of
e4m3 scales (one per 16 elements) and one fp32 scale, a power of two, beside the row:

    value_d = s * scale_{d / 16} * e2m1(code_d)

and quantised from x by: s the least power of two with max |x| <= 2688 s (2688 = 448 * 6), scale_b = e4m3(max |x| of
the block / (6 s)), code_d = e2m1(x_d / (s scale_b)), each rounded to nearest even.

``own`` False: the plain forms, elementary torch operations.  ``own`` True: the calls of this package.
Every case is a dict of plain values; ``op`` says which call it times.
"""
import math

import torch

own = False

DIM = 512
ROW_BYTES = 288            # 256 bytes of codes, 32 of block scales
ROPE_DIM = 64
THETA = 10000.0
WINDOW_TOKENS = {"c4a": (8, 4), "c128a": (128, 128)}   # raw tokens of an entry, stride
SM_SCALE = 1.0 / math.sqrt(512.0)


# ---- cases ------------------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode batch appends one row to each request's cache and reads the stored rows back: launch latency
        {"name": "append_decode", "op": "cache", "batch": 32, "rows": 1, "ragged": 0, "extra": 0},
        # the entries of a few ragged prefill chunks, appended at odd starts, read back for a dense pass over them
        {"name": "append_chunks", "op": "cache", "batch": 5, "rows": 2047, "ragged": 1, "extra": 0},
        # the caches of 16 long requests handed over in bf16 by a prefill, stored in 4 bits, then read back
        {"name": "convert_prefixes", "op": "cache", "batch": 16, "rows": 8192, "ragged": 0, "extra": 0},
        # the top-k rows of a decode batch fetched as values (512 scattered rows a request, some lists not full)
        {"name": "read_topk", "op": "read", "batch": 32, "rows": 512, "pool_rows": 16384, "ordered": 0,
         "pads": 3},
        # a whole prefix of one long request read back in order
        {"name": "read_prefix", "op": "read", "batch": 1, "rows": 65535, "pool_rows": 65536, "ordered": 1,
         "pads": 0},
        # one short request of a small layer: latency
        {"name": "decode_one", "op": "decode", "kind": "c4a", "batch": 1, "ctx": 4096, "spread": 1, "heads": 16,
         "k": 512, "window": 128},
        # the decode batch of the layer step: 512 selected entries and the window for each request
        {"name": "decode_batch", "op": "decode", "kind": "c4a", "batch": 32, "ctx": 65536, "spread": 1, "heads": 64,
         "k": 512, "window": 128},
        # requests of very different lengths: some shorter than the window, some with fewer entries than k
        {"name": "decode_mixed", "op": "decode", "kind": "c4a", "batch": 61, "ctx": 65536, "spread": 65536, "heads": 128,
         "k": 512, "window": 128},
        # the layer that reads every entry of a million-token context
        {"name": "decode_dense", "op": "decode", "kind": "c128a", "batch": 16, "ctx": 1048576, "spread": 1, "heads": 64,
         "k": 0, "window": 128},
        # a decode step that stores the new window rows in 4 bits and then attends to them with the rest
        {"name": "append_attend", "op": "step", "kind": "c4a", "batch": 48, "ctx": 32768, "spread": 16, "heads": 32,
         "k": 512, "window": 128},
        # one prefill chunk of a long request
        {"name": "prefill_chunk", "op": "prefill", "kind": "c4a", "batch": 1, "ctx": 65536, "spread": 1, "new": 2048,
         "heads": 64, "k": 512, "window": 128},
        # short ragged prompts from position 0 on: queries that see no entry yet, fewer than k, an odd window
        {"name": "prefill_ragged", "op": "prefill", "kind": "c4a", "batch": 3, "ctx": 700, "spread": 5, "new": 700,
         "heads": 16, "k": 333, "window": 100},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["cache", "read", "decode", "decode", "prefill", "step"])
    if op == "cache":
        batch = _log(rng, 1, 64)
        return {"op": op, "batch": batch, "rows": _log(rng, 1, 131072 // batch),
                "ragged": rng.choice([0, 1]), "extra": rng.choice([0, 0, 7])}
    if op == "read":
        batch = _log(rng, 1, 64)
        pool_rows = _log(rng, 64, 16384)
        return {"op": op, "batch": batch, "rows": _log(rng, 1, min(2048, 65536 // batch)), "pool_rows": pool_rows,
                "ordered": 0, "pads": rng.choice([0, 1, 5])}
    kind = rng.choice(["c4a", "c4a", "c128a"])
    case = {"op": op, "kind": kind, "heads": rng.choice([16, 32, 64, 128]), "window": rng.choice([1, 64, 128, 128, 513])}
    if op == "prefill":
        case["batch"] = _log(rng, 1, 8)
        case["new"] = _log(rng, 1, 1536 // case["batch"])
        case["ctx"] = case["new"] + _log(rng, 1, 32768)
        case["spread"] = rng.choice([1, 3, 50])
        case["k"] = _log(rng, 1, 512)
        return case
    case["batch"] = _log(rng, 1, 64 if kind == "c4a" else 16)
    case["ctx"] = _log(rng, 1, 65536 if kind == "c4a" else 1048576)
    case["spread"] = rng.choice([1, 4, 300])
    case["k"] = 0 if kind == "c128a" else _log(rng, 1, 1024)   # 0: every visible entry
    return case


# ---- sizes of a case ----------------------------------------------------------------------------------------------
def _appended(case):
    """Rows each request appends: the same number, or (ragged) the first the most, every one at least 1."""
    batch, most = case["batch"], case["rows"]
    if not case["ragged"]:
        return [most] * batch
    return [max(1, most - (i * most) // batch - i % 3) for i in range(batch)]


def _lengths(batch, ctx, spread):
    """Context lengths (raw tokens) of the requests: from ctx down to ctx / spread, evenly in their logarithm."""
    if spread <= 1 or batch == 1:
        return [ctx] * batch
    return [max(1, int(ctx * math.exp(-math.log(spread) * i / (batch - 1)))) for i in range(batch)]


def _entries(tokens, kind):
    w, s = WINDOW_TOKENS[kind]
    return 0 if tokens < w else (tokens - w) // s + 1


def _queries(case):
    """(positions, requests) of the query rows: the last token of each request, or its last `new` tokens."""
    lens = _lengths(case["batch"], case["ctx"], case["spread"])
    pos, req = [], []
    for r, t in enumerate(lens):
        n = min(t, case["new"]) if case["op"] == "prefill" else 1
        pos += list(range(t - n, t))
        req += [r] * n
    return lens, pos, req


def work(case):
    if case["op"] == "cache":
        n = sum(_appended(case))
        return {"bytes": n * (1024 + ROW_BYTES + 4 + 8 + 1024), "flops": 0}
    if case["op"] == "read":
        n = case["batch"] * case["rows"]
        return {"bytes": n * (ROW_BYTES + 4 + 8 + 1024), "flops": 0}
    lens, pos, req = _queries(case)
    h, k = case["heads"], case["k"]
    keys, rows = 0, 0
    most = {}
    for m, r in zip(pos, req):
        n = _entries(m + 1, case["kind"])
        win = min(case["window"], m + 1)
        picked = min(n, k) if k else n
        keys += picked + win
        if case["op"] == "prefill":   # rows that several queries read are counted once
            most.setdefault(r, [0, 0])
            most[r][0] = max(most[r][0], min(n, most[r][0] + picked))
            most[r][1] += 1
        else:
            rows += picked + win
    for r, (entries, n) in most.items():
        rows += entries + min(lens[r], n + case["window"] - 1)
    nq = len(pos)
    fresh = case["batch"] * 1024 if case["op"] == "step" else 0
    return {"bytes": rows * (ROW_BYTES + 4) + nq * (h * (1024 + 1024 + 4) + 4 * k) + fresh,
            "flops": 4.0 * DIM * h * keys}


# ---- the format, in elementary operations ---------------------------------------------------------------------------
def _codebook(device):
    mags = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(mags + [-v for v in mags], dtype=torch.float32, device=device)


def _power_of_two(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _to_e4m3_grid(v):
    """Nearest e4m3 value (ties to even) of v >= 0, at most 448, in 64 bits."""
    e = torch.clamp(torch.frexp(v).exponent - 1, min=-6).to(torch.float64)
    step = torch.exp2(e - 3)
    return torch.clamp(torch.round(v / step) * step, max=448.0)


def _to_e2m1_grid(u):
    """Nearest e2m1 value (ties to even), saturating at 6, in 64 bits."""
    a = u.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.clamp(torch.round(a / step) * step, max=6.0) * torch.sign(u)


def _quantise(x):
    """Rows [n, 512] -> (element values on the e2m1 grid, block scales [n, 32], row scale [n]), as float32; the
    borders between two codes are decided in 64 bits."""
    xd = x.to(torch.float64)
    amax = xd.abs().amax(-1)
    m, k = torch.frexp(amax)
    e = torch.clamp(k - 12 + (m > 0.65625).to(k.dtype), min=-126)     # 2688 = 0.65625 * 2^12
    s = torch.where(amax > 0, _power_of_two(e), torch.ones_like(amax, dtype=torch.float32))
    blocks = xd.view(-1, DIM // 16, 16)
    bs = _to_e4m3_grid(blocks.abs().amax(-1) / (6.0 * s.to(torch.float64)[:, None]))
    div = (s.to(torch.float64)[:, None] * bs)[:, :, None]
    u = torch.where(div > 0, blocks / torch.where(div > 0, div, 1.0), 0.0)
    q = _to_e2m1_grid(u).view(-1, DIM)
    return q.to(torch.float32), bs.to(torch.float32), s


def _pack(q, bs):
    """The stored bytes [n, 288] of element values and block scales."""
    mags = q.abs()
    idx = (2 * torch.clamp(mags, max=2.0) + torch.clamp(mags - 2.0, 0.0, 2.0)
           + torch.clamp(mags - 4.0, min=0.0) / 2).round().to(torch.uint8)
    code = idx | ((q < 0).to(torch.uint8) << 3)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    return torch.cat([packed, bs.to(torch.float8_e4m3fn).view(torch.uint8)], dim=1)


def _values(data, scale):
    """Stored rows [..., 288] and row scales [...] as float32 values [..., 512]."""
    codes = data[..., :256]
    both = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    el = _codebook(data.device)[both.to(torch.int32)]
    bs = data[..., 256:].contiguous().view(torch.float8_e4m3fn).to(torch.float32)
    v = el.unflatten(-1, (DIM // 16, 16)) * bs[..., None]
    return v.flatten(-2) * scale[..., None]


# ---- inputs ---------------------------------------------------------------------------------------------------------
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _pool_rows(n, gen):
    """n stored rows of values as a cache holds them: normed rows, their spread differing by row and by channel."""
    data = torch.empty((n, ROW_BYTES), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n,), dtype=torch.float32, device="cuda")
    for lo in range(0, n, 65536):
        m = min(n, lo + 65536) - lo
        x = torch.randn((m, DIM), generator=gen, device="cuda")
        x = x * torch.exp2(torch.randn((m, 1), generator=gen, device="cuda") * 0.5)
        q, bs, s = _quantise(x)
        data[lo:lo + m], scale[lo:lo + m] = _pack(q, bs), s
    return data, scale


def _tables(blocks, gen):
    """A block table [batch, most blocks] over a shuffled pool a little larger than what is mapped; -1: unmapped."""
    total = sum(blocks)
    count = total + max(1, total // 8)
    perm = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    bt = torch.full((len(blocks), max(blocks)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, b in enumerate(blocks):
        bt[r, :b] = perm[at:at + b]
        at += b
    return bt, count


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = _gen(seed)
    if case["op"] == "cache":
        n = _appended(case)
        first = [(37 * i) % 111 for i in range(case["batch"])]
        bt, count = _tables([(a + b + 63) // 64 for a, b in zip(first, n)], gen)
        total = sum(n)
        x = (torch.randn((total + case["extra"], DIM), generator=gen, device="cuda")
             * torch.exp2(torch.randn((total + case["extra"], 1), generator=gen, device="cuda"))).to(torch.bfloat16)
        cu = [0]
        for v in n:
            cu.append(cu[-1] + v)
        req = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
        offset = torch.arange(total, device="cuda") - torch.tensor(cu, device="cuda")[req]
        ids = torch.tensor(first, device="cuda")[req] + offset
        return {"case": case, "x": x, "cu": _ints(cu), "start": _ints(first), "bt": bt, "epb": 64,
                "data": torch.zeros((count * 64, ROW_BYTES), dtype=torch.uint8, device="cuda"),
                "scale": torch.zeros((count * 64,), dtype=torch.float32, device="cuda"),
                "req": req.to(torch.int32), "ids": ids.to(torch.int32), "total": total,
                "out": torch.empty((total, DIM), dtype=torch.bfloat16, device="cuda")}
    if case["op"] == "read":
        b, k, rows = case["batch"], case["rows"], case["pool_rows"]
        bt, count = _tables([(rows + 63) // 64] * b, gen)
        data, scale = _pool_rows(count * 64, gen)
        if case["ordered"]:
            ids = torch.arange(k, device="cuda")[None]
        else:
            ids = torch.randint(0, rows, (b, k), generator=gen, device="cuda").sort(-1).values
        if case["pads"]:
            ids[:, k - min(k - 1, case["pads"]):] = -1
        req = torch.arange(b, device="cuda")[:, None].expand(b, k)
        return {"case": case, "data": data, "scale": scale, "bt": bt, "epb": 64,
                "req": req.reshape(-1).to(torch.int32), "ids": ids.reshape(-1).to(torch.int32),
                "out": torch.empty((b * k, DIM), dtype=torch.bfloat16, device="cuda")}
    return _prepare_attention(case, gen)


def _prepare_attention(case, gen):
    lens, pos, req = _queries(case)
    epb = 256 // WINDOW_TOKENS[case["kind"]][1]
    blocks = [(t + 255) // 256 for t in lens]
    bt, count = _tables(blocks, gen)
    data, scale = _pool_rows(count * epb, gen)
    swa_bt, swa_count = _window_table(case, lens, pos, req, gen)
    swa_data, swa_scale = _pool_rows(swa_count * 256, gen)
    q_pos, q_req = _ints(pos), _ints(req)
    nq, k, h = len(pos), case["k"], case["heads"]
    n_vis = _ints([_entries(m + 1, case["kind"]) for m in pos])
    topk = None
    if k:   # k distinct visible entries in increasing order, -1 behind them where there are fewer
        most = max(1, max(_entries(t, case["kind"]) for t in lens), k)
        topk = torch.empty((nq, k), dtype=torch.int32, device="cuda")
        col = torch.arange(most, device="cuda")
        for lo in range(0, nq, 512):
            score = torch.rand((min(nq, lo + 512) - lo, most), generator=gen, device="cuda")
            score = torch.where(col < n_vis[lo:lo + 512, None], score, -1.0)
            val, idx = score.topk(k, -1)
            idx = torch.where(val >= 0, idx, most).sort(-1).values
            topk[lo:lo + 512] = torch.where(idx == most, -1, idx).to(torch.int32)
    state = {"case": case, "data": data, "scale": scale, "bt": bt, "epb": epb, "swa_data": swa_data,
             "swa_scale": swa_scale, "swa_bt": swa_bt, "q_pos": q_pos, "q_req": q_req, "n_vis": n_vis, "topk": topk,
             "most": max(1, max(_entries(t, case["kind"]) for t in lens)),
             "q": (torch.randn((nq, h, DIM), generator=gen, device="cuda")
                   * torch.exp2(torch.randn((nq, h, 1), generator=gen, device="cuda") * 0.5)).to(torch.bfloat16),
             "out": torch.empty((nq, h, DIM), dtype=torch.bfloat16, device="cuda"),
             "lse": torch.empty((nq, h), dtype=torch.float32, device="cuda"), "workspace": None}
    if case["op"] == "step":
        state["x"] = torch.randn((nq, DIM), generator=gen, device="cuda").to(torch.bfloat16)
        state["cu"] = torch.arange(nq + 1, dtype=torch.int32, device="cuda")
    if own:
        from compressed_sparse_attention_c4a_gb300 import dsa
        keys = (k if k else bt.shape[1] * epb) + case["window"]
        need = dsa.dsa_attn_workspace_size(nq, h, keys)
        state["workspace"] = torch.empty((need,), dtype=torch.uint8, device="cuda") if need else None
    return state


def _window_table(case, lens, pos, req, gen):
    """The window pool's table: only the blocks that some query's window touches are mapped."""
    lo = {}
    for m, r in zip(pos, req):
        lo[r] = min(lo.get(r, m), max(0, m - case["window"] + 1))
    spans = [(lo[r] // 256, (t - 1) // 256) for r, t in enumerate(lens)]
    total = sum(b - a + 1 for a, b in spans)
    count = total + max(1, total // 8)
    perm = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    bt = torch.full((len(lens), max(b for _, b in spans) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, (a, b) in enumerate(spans):
        bt[r, a:b + 1] = perm[at:at + b - a + 1]
        at += b - a + 1
    return bt, count


# ---- one pass -------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own_cache(state) if op == "cache" else _own_read(state) if op == "read" else _own_attention(state)
    if op == "cache":
        _plain_write(state["x"][:state["total"]], state["req"], state["ids"], state["data"], state["scale"],
                     state["bt"], state["epb"])
        return _plain_read(state)
    if op == "read":
        return _plain_read(state)
    if op == "step":
        _plain_write(state["x"], state["q_req"], state["q_pos"], state["swa_data"], state["swa_scale"],
                     state["swa_bt"], 256)
    return _plain_attention(state)


def _own_cache(state):
    from compressed_sparse_attention_c4a_gb300 import dsa
    pool = dsa.pool(state["data"], state["epb"], state["scale"], fmt="fp4_block")
    bt = dsa.block_table(state["bt"])
    dsa.dsa_cache_write(state["cu"], state["start"], state["x"], pool, bt)
    dsa.dsa_cache_read(pool, bt, state["req"], state["ids"], state["out"])
    return state["out"]


def _own_read(state):
    from compressed_sparse_attention_c4a_gb300 import dsa
    pool = dsa.pool(state["data"], state["epb"], state["scale"], fmt="fp4_block")
    dsa.dsa_cache_read(pool, dsa.block_table(state["bt"]), state["req"], state["ids"], state["out"])
    return state["out"]


def _own_attention(state):
    from compressed_sparse_attention_c4a_gb300 import dsa
    case = state["case"]
    main = dsa.pool(state["data"], state["epb"], state["scale"], fmt="fp4_block")
    swa = dsa.pool(state["swa_data"], 256, state["swa_scale"], fmt="fp4_block")
    bt, swa_bt = dsa.block_table(state["bt"]), dsa.block_table(state["swa_bt"])
    if case["op"] == "step":
        dsa.dsa_cache_write(state["cu"], state["q_pos"], state["x"], swa, swa_bt)
    rope = dsa.rope(ROPE_DIM, THETA)
    if case["op"] == "prefill":
        dsa.dsa_sparse_attn_prefill(state["q"], state["q_pos"], state["q_req"], case["kind"], state["topk"], case["k"],
                                    main, bt, swa, swa_bt, case["window"], SM_SCALE, rope, state["out"], state["lse"],
                                    state["workspace"])
    else:
        dsa.dsa_sparse_attn_decode(state["q"], state["q_pos"], case["kind"], state["topk"], case["k"], main, bt, swa,
                                   swa_bt, case["window"], SM_SCALE, rope, state["out"], state["lse"],
                                   state["workspace"])
    return state["out"], state["lse"]


def _physical(bt, req, ids, epb):
    """Pool rows of logical rows (ids >= 0)."""
    ids = ids.long()
    return bt[req.long(), ids // epb].long() * epb + ids % epb


def _plain_write(x, req, ids, data, scale, bt, epb):
    rows = _physical(bt, req, ids, epb)
    q, bs, s = _quantise(x)
    data[rows], scale[rows] = _pack(q, bs), s


def _plain_read(state):
    ids = state["ids"]
    rows = _physical(state["bt"], state["req"], ids.clamp(min=0), state["epb"])
    v = _values(state["data"][rows], state["scale"][rows])
    return torch.where((ids >= 0)[:, None], v, 0.0).to(torch.bfloat16)


def _plain_attention(state):
    case = state["case"]
    q, pos, req = state["q"].to(torch.float32), state["q_pos"].long(), state["q_req"].long()
    if state["topk"] is not None:
        ids = state["topk"].long()
        seen = ids >= 0
    else:
        ids = torch.arange(state["most"], device="cuda")[None].expand(len(pos), -1)
        seen = ids < state["n_vis"][:, None]
    rows = _physical(state["bt"], req[:, None], torch.where(seen, ids, 0), state["epb"])
    win = pos[:, None] - torch.arange(case["window"], device="cuda")[None]
    in_window = win >= 0
    win_rows = _physical(state["swa_bt"], req[:, None], torch.where(in_window, win, pos[:, None]), 256)
    keys = torch.cat([_values(state["data"][rows], state["scale"][rows]),
                      _values(state["swa_data"][win_rows], state["swa_scale"][win_rows])], dim=1)
    mask = torch.cat([seen, in_window], dim=1)[:, None]
    logits = torch.where(mask, torch.matmul(q, keys.transpose(1, 2)) * SM_SCALE, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p / total, keys)
    lse = (top + torch.log(total))[..., 0]
    # out = o with its last 64 dims rotated back by the query's position; the angle in 64 bits
    freq = THETA ** (-2.0 * torch.arange(ROPE_DIM // 2, dtype=torch.float64, device="cuda") / ROPE_DIM)
    ang = (pos.to(torch.float64)[:, None] * freq)[:, None]
    c, s = torch.cos(ang).to(torch.float32), torch.sin(ang).to(torch.float32)
    a, b = o[..., DIM - ROPE_DIM::2], o[..., DIM - ROPE_DIM + 1::2]
    tail = torch.stack([a * c + b * s, b * c - a * s], dim=-1).flatten(-2)
    return torch.cat([o[..., :DIM - ROPE_DIM], tail], dim=-1).to(torch.bfloat16), lse


# ---- the definition in 64 bits ----------------------------------------------------------------------------------------
def _nearest(v, grid):
    """Index of the grid value nearest to each v >= 0 (grid increasing, v within it); a tie goes to the even index."""
    hi = torch.clamp(torch.searchsorted(grid, v), max=len(grid) - 1)
    lo = torch.clamp(hi - 1, min=0)
    dh, dl = (grid[hi] - v).abs(), (v - grid[lo]).abs()
    return torch.where(dh < dl, hi, torch.where(dl < dh, lo, torch.where(hi % 2 == 0, hi, lo)))


def _stored_exactly(x):
    """The values, in 64 bits, that rows of x stand for once stored."""
    e2m1 = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    b = torch.arange(127, device="cuda", dtype=torch.float64)   # e4m3 codes 0 .. 126 in order
    e4m3 = torch.where(b < 8, b / 512, (1 + (b % 8) / 8) * 2.0 ** (torch.floor(b / 8) - 7))
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for lo in range(0, len(x), 16384):
        v = x[lo:lo + 16384].to(torch.float64)
        amax = v.abs().amax(-1)
        s = torch.ones_like(amax)
        for e in range(60, -127, -1):    # the least power of two that still holds the row
            s = torch.where(amax <= 2688 * 2.0 ** e, 2.0 ** e, s)
        s = torch.where(amax > 0, s, 1.0)[:, None, None]
        w = v.view(-1, 32, 16)
        bs = e4m3[_nearest(torch.clamp(w.abs().amax(-1, keepdim=True) / (6 * s), max=448.0), e4m3)]
        unit = torch.where(bs > 0, bs * s, 1.0)
        q = e2m1[_nearest(torch.clamp(w.abs() / unit, max=6.0), e2m1)] * torch.sign(w)
        out[lo:lo + 16384] = torch.where(bs > 0, q * bs * s, 0.0).view(-1, DIM)
    return out


def _held_exactly(data, scale):
    """The values, in 64 bits, of stored rows: each field of the bytes taken apart."""
    codes = torch.stack([data[:, :256] % 16, data[:, :256] // 16], dim=-1).view(len(data), DIM).to(torch.int64)
    e, m = (codes >> 1) & 3, (codes & 1).to(torch.float64)
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1).to(torch.float64))
    el = torch.where(codes >= 8, -mag, mag)
    sb = data[:, 256:].to(torch.int64)
    se, sm = (sb >> 3) & 15, (sb & 7).to(torch.float64)
    bs = torch.where(se == 0, sm / 512, (1 + sm / 8) * 2.0 ** (se - 7).to(torch.float64))
    return el * bs.repeat_interleave(16, dim=1) * scale.to(torch.float64)[:, None]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "cache":
        return _stored_exactly(state["x"][:state["total"]])
    bt, epb = state["bt"].cpu().tolist(), state["epb"]
    if case["op"] == "read":
        ids, req = state["ids"].cpu().tolist(), state["req"].cpu().tolist()
        rows = torch.tensor([bt[r][i // epb] * epb + i % epb if i >= 0 else 0 for r, i in zip(req, ids)], device="cuda")
        v = _held_exactly(state["data"][rows], state["scale"][rows])
        return v * (state["ids"] >= 0)[:, None]
    pos, req = state["q_pos"].cpu().tolist(), state["q_req"].cpu().tolist()
    swa_bt = state["swa_bt"].cpu().tolist()
    picks = state["topk"].cpu().tolist() if state["topk"] is not None else None
    visible = state["n_vis"].cpu().tolist()
    fresh = _stored_exactly(state["x"]) if case["op"] == "step" else None
    out = torch.empty((len(pos), case["heads"], DIM), dtype=torch.float64, device="cuda")
    lse = torch.empty((len(pos), case["heads"]), dtype=torch.float64, device="cuda")
    for j, (m, r) in enumerate(zip(pos, req)):
        ids = [i for i in picks[j] if i >= 0] if picks else list(range(visible[j]))
        rows = torch.tensor([bt[r][i // epb] * epb + i % epb for i in ids], dtype=torch.int64, device="cuda")
        span = range(max(0, m - case["window"] + 1), m + 1)
        wins = torch.tensor([swa_bt[r][p // 256] * 256 + p % 256 for p in span], device="cuda")
        window = _held_exactly(state["swa_data"][wins], state["swa_scale"][wins])
        if fresh is not None:
            window[-1] = fresh[j]
        keys = torch.cat([_held_exactly(state["data"][rows], state["scale"][rows]), window])
        logits = state["q"][j].to(torch.float64) @ keys.T / math.sqrt(512.0)
        lse[j] = torch.logsumexp(logits, -1)
        out[j] = torch.exp(logits - lse[j][:, None]) @ keys
    angles = [[m * THETA ** (-d / ROPE_DIM) for d in range(0, ROPE_DIM, 2)] for m in pos]
    theta = torch.tensor(angles, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(theta), -theta)
    pairs = torch.view_as_complex(out[..., DIM - ROPE_DIM:].unflatten(-1, (-1, 2)).contiguous())
    out[..., DIM - ROPE_DIM:] = torch.view_as_real(pairs * turn[:, None]).flatten(-2)
    return out, lse
