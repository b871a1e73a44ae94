"""The operators around the attention of a layer: the norm in front of its projections, the projections, the rows they append.

Rows in 8 bits are e4m3 codes with one fp32 scale per 128 consecutive values (the last block of a row may be shorter):

    scale_b = max |v| of the block / 448  (1 for a block of zeros),    code_d = e4m3(v_d / scale_{d / 128})

- norm:   h = x + residual,  v = gamma h / sqrt(mean(h^2) + eps), stored as such rows; h itself in bf16
- gemm:   out[m][g][n] = sum_k a[m][g][k] w[g][n][k] over 8-bit rows a (a scale per row and 128 of k) and weights w (a scale
          per 128 of n and 128 of k), stored in fp32, bf16 or as such rows
- append: rows x normed as above, their last 64 dims rotated by the row's position, stored in a paged cache (bf16, or e4m3
          with one scale per row)

``own`` False: the plain forms, elementary torch operations.  ``own`` True: the calls of this package.
Every case is a dict of plain values; ``op`` says which call it times.
"""
import math

import torch

own = False

BLOCK = 128
EPS = 1e-6
ROPE_DIM = 64
THETA = 10000.0
FORMATS = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases ------------------------------------------------------------------------------------------------------
def listed():
    return [
        # the residual stream of a decode batch, a token a request: launch latency
        {"name": "norm_decode", "op": "norm", "rows": 32, "dim": 4096, "residual": 1, "zeros": 0},
        # ragged prompts behind one another, padded with rows of zeros, a width that ends inside a block
        {"name": "norm_ragged", "op": "norm", "rows": 1153, "dim": 1040, "residual": 0, "zeros": 7},
        # a prefill chunk's residual stream
        {"name": "norm_chunk", "op": "norm", "rows": 8192, "dim": 8192, "residual": 1, "zeros": 0},
        # a decode batch appends one row to each request's window cache
        {"name": "append_decode", "op": "append", "batch": 32, "rows": 1, "ragged": 0, "dim": 512, "fmt": "fp8", "norm": 1,
         "far": 65535},
        # a few ragged prefill chunks appended at odd positions, kept in bf16
        {"name": "append_chunks", "op": "append", "batch": 5, "rows": 2047, "ragged": 1, "dim": 512, "fmt": "bf16", "norm": 1,
         "far": 131071},
        # the window caches of 16 long prompts
        {"name": "append_prompts", "op": "append", "batch": 16, "rows": 8192, "ragged": 0, "dim": 512, "fmt": "fp8",
         "norm": 1, "far": 0},
        # one token's indexer weights and gates: latency
        {"name": "project_one", "op": "gemm", "m": 1, "n": 520, "k": 4096, "groups": 1, "out": "f32"},
        # the query projection of a decode batch: 64 heads of 512; the weights' bytes
        {"name": "project_decode", "op": "gemm", "m": 32, "n": 32768, "k": 4096, "groups": 1, "out": "bf16"},
        # the first output projection of a decode batch, eight groups of eight heads, its rows in 8 bits for the second
        {"name": "groups_decode", "op": "gemm", "m": 32, "n": 1024, "k": 4096, "groups": 8, "out": "fp8"},
        # ragged prompts, a width and an inner size that end inside a block
        {"name": "project_ragged", "op": "gemm", "m": 1153, "n": 1000, "k": 1040, "groups": 1, "out": "bf16"},
        # the first output projection of a prefill chunk
        {"name": "groups_chunk", "op": "gemm", "m": 2048, "n": 1024, "k": 4096, "groups": 8, "out": "fp8"},
        # the query projection of a prefill chunk
        {"name": "project_chunk", "op": "gemm", "m": 8192, "n": 32768, "k": 4096, "groups": 1, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "gemm", "gemm"])
    if op == "norm":
        dim = 16 * _log(rng, 4, 512)
        return {"op": op, "rows": _log(rng, 1, min(65536, 8192 * 8192 // dim)), "dim": dim,
                "residual": rng.choice([0, 1]), "zeros": rng.choice([0, 0, 3])}
    if op == "append":
        batch = _log(rng, 1, 64)
        return {"op": op, "batch": batch, "rows": _log(rng, 1, 131072 // batch), "ragged": rng.choice([0, 1]),
                "dim": rng.choice([64, 128, 512, 512]), "fmt": rng.choice(["bf16", "fp8"]), "norm": rng.choice([0, 1, 1]),
                "far": rng.choice([0, 5000, 131071])}
    groups = rng.choice([1, 1, 1, 2, 8])
    k = 16 * _log(rng, 1, 512)
    n = _log(rng, 1, 16384) if rng.random() < 0.5 else 128 * _log(rng, 1, 128)
    return {"op": op, "m": _log(rng, 1, 8192), "n": max(1, n // groups), "k": k, "groups": groups,
            "out": rng.choice(["f32", "bf16", "bf16", "fp8"])}


# ---- sizes of a case ----------------------------------------------------------------------------------------------
def _blocks(n):
    return -(-n // BLOCK)


def _appended(case):
    """Rows each request appends: the same number, or (ragged) the first the most, every one at least 1."""
    batch, most = case["batch"], case["rows"]
    if not case["ragged"]:
        return [most] * batch
    return [max(1, most - (i * most) // batch - i % 3) for i in range(batch)]


def work(case):
    if case["op"] == "norm":
        n, d = case["rows"], case["dim"]
        return {"bytes": n * (d * (7 if case["residual"] else 3) + 4 * _blocks(d)) + 4 * d, "flops": 0}
    if case["op"] == "append":
        d = case["dim"]
        return {"bytes": sum(_appended(case)) * (2 * d + (2 * d if case["fmt"] == "bf16" else d + 4)), "flops": 0}
    m, n, k, g = (case[c] for c in ("m", "n", "k", "groups"))
    out = {"f32": 4 * n, "bf16": 2 * n, "fp8": n + 4 * _blocks(n)}[case["out"]]
    return {"bytes": g * (m * (k + 4 * _blocks(k)) + n * k + 4 * _blocks(n) * _blocks(k) + m * out),
            "flops": 2.0 * m * n * k * g}


# ---- inputs ---------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _hidden(gen, rows, dim):
    """Rows of a residual stream: their sizes differ by row and, more, by channel."""
    return _randn(gen, rows, dim) * torch.exp2(_randn(gen, rows, 1)) * torch.exp2(1.5 * _randn(gen, 1, dim))


def _block_amax(v):
    """max |v| of each 128 values of the last dimension, [..., blocks]."""
    n = v.shape[-1]
    a = v.abs()
    if n % BLOCK:
        a = torch.nn.functional.pad(a, (0, BLOCK - n % BLOCK))
    return a.unflatten(-1, (-1, BLOCK)).amax(-1)


def _spread(s, n):
    """Block scales [..., blocks] as one for each of n values."""
    return s.repeat_interleave(BLOCK, -1)[..., :n]


def _to_rows8(v):
    """The 8-bit rows of float32 values: codes as float8, scales."""
    amax = _block_amax(v)
    scale = torch.where(amax > 0, amax / 448.0, 1.0)
    return (v / _spread(scale, v.shape[-1])).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), scale


def _weights8(gen, groups, n, k):
    """Weights [groups, n, k] in 8 bits with a scale per 128 x 128, their spread differing by output and by input."""
    codes = torch.empty((groups, n, k), dtype=torch.float8_e4m3fn, device="cuda")
    scale = torch.empty((groups, _blocks(n), _blocks(k)), device="cuda")
    for g in range(groups):
        for lo in range(0, n, 4096):
            hi = min(n, lo + 4096)
            v = (_randn(gen, hi - lo, k) * torch.exp2(0.5 * _randn(gen, hi - lo, 1)) * torch.exp2(0.5 * _randn(gen, 1, k))
                 / math.sqrt(k))
            s = _block_amax(_block_amax(v).transpose(0, 1)).transpose(0, 1) / 448.0
            scale[g, lo // BLOCK:_blocks(hi)] = s
            full = _spread(_spread(s, k).transpose(0, 1), hi - lo).transpose(0, 1)
            codes[g, lo:hi] = (v / full).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _tables(blocks, gen):
    """A block table [batch, most blocks] over a shuffled pool a little larger than what is mapped; -1: unmapped."""
    lo, hi = [b[0] for b in blocks], [b[1] for b in blocks]
    total = sum(h - l for l, h in blocks)
    count = total + max(1, total // 8)
    perm = torch.randperm(count, generator=gen, device="cuda").to(torch.int32)
    bt = torch.full((len(blocks), max(hi)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, (a, b) in enumerate(zip(lo, hi)):
        bt[r, a:b] = perm[at:at + b - a]
        at += b - a
    return bt, count


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = _gen(seed)
    return {"norm": _prepare_norm, "append": _prepare_append, "gemm": _prepare_gemm}[case["op"]](case, gen)


def _prepare_norm(case, gen):
    n, d = case["rows"], case["dim"]
    x = _hidden(gen, n, d).to(torch.bfloat16)
    if case["zeros"]:
        x[max(1, n - case["zeros"]):] = 0
    return {"case": case, "x": x, "residual": _hidden(gen, n, d).to(torch.bfloat16) if case["residual"] else None,
            "sum": torch.empty((n, d), dtype=torch.bfloat16, device="cuda") if case["residual"] else None,
            "gamma": 1.0 + 0.2 * _randn(gen, d), "codes": torch.empty((n, d), dtype=torch.uint8, device="cuda"),
            "scale": torch.empty((n, _blocks(d)), device="cuda")}


def _prepare_append(case, gen):
    n = _appended(case)
    first = [max(0, case["far"] - 977 * i) for i in range(case["batch"])]
    bt, count = _tables([(a // 256, (a + b + 255) // 256) for a, b in zip(first, n)], gen)
    total, d = sum(n), case["dim"]
    cu = [0]
    for v in n:
        cu.append(cu[-1] + v)
    req = torch.repeat_interleave(torch.arange(len(n), device="cuda"), torch.tensor(n, device="cuda"))
    pos = torch.tensor(first, device="cuda")[req] + torch.arange(total, device="cuda") - torch.tensor(cu, device="cuda")[req]
    fp8 = case["fmt"] == "fp8"
    return {"case": case, "x": (_randn(gen, total, d) * torch.exp2(_randn(gen, total, 1))).to(torch.bfloat16),
            "gamma": 1.0 + 0.2 * _randn(gen, d) if case["norm"] else None, "cu": _ints(cu), "start": _ints(first), "bt": bt,
            "req": req, "pos": pos,
            "data": torch.zeros((count * 256, d), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda"),
            "scale": torch.zeros((count * 256,), device="cuda") if fp8 else None}


def _prepare_gemm(case, gen):
    m, n, k, g = (case[c] for c in ("m", "n", "k", "groups"))
    a, a_scale = _to_rows8(_randn(gen, m, g, k) * torch.exp2(_randn(gen, m, 1, 1)) * torch.exp2(_randn(gen, 1, g, k)))
    w, w_scale = _weights8(gen, g, n, k)
    fp8 = case["out"] == "fp8"
    return {"case": case, "a": a.view(torch.uint8), "a_scale": a_scale, "w": w, "w_scale": w_scale,
            "out": torch.empty((m, g, n), dtype=torch.uint8 if fp8 else FORMATS[case["out"]], device="cuda"),
            "scale": torch.empty((m, g, _blocks(n)), device="cuda") if fp8 else None}


# ---- one pass -------------------------------------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own_norm(state) if op == "norm" else _own_append(state) if op == "append" else _own_gemm(state)
    return _plain_norm(state) if op == "norm" else _plain_append(state) if op == "append" else _plain_gemm(state)


def _own_norm(state):
    from compressed_sparse_attention_c4a_gb300 import dsa
    dsa.dsa_norm_q8(state["x"], state["gamma"], EPS, state["codes"], state["scale"], residual=state["residual"],
                    sum_out=state["sum"])
    return state["sum"], state["codes"].view(torch.float8_e4m3fn), state["scale"]


def _own_append(state):
    from compressed_sparse_attention_c4a_gb300 import dsa
    pool = dsa.pool(state["data"], 256, state["scale"])
    dsa.dsa_cache_append(state["cu"], state["start"], state["x"], dsa.rope(ROPE_DIM, THETA), pool,
                         dsa.block_table(state["bt"]), norm=bool(state["case"]["norm"]), rms_gamma=state["gamma"], rms_eps=EPS)
    return _stored(state)


def _own_gemm(state):
    from compressed_sparse_attention_c4a_gb300 import dsa
    dsa.dsa_gemm_q8(state["a"], state["a_scale"], state["w"], state["w_scale"], state["out"], out_scale=state["scale"])
    if state["scale"] is None:
        return state["out"]
    return state["out"].view(torch.float8_e4m3fn), state["scale"]


def _stored(state):
    """What a pool holds: bf16 values, or e4m3 values with a scale per row."""
    if state["scale"] is None:
        return state["data"]
    return state["data"].view(torch.float8_e4m3fn), state["scale"]


def _plain_norm(state):
    h = state["x"].to(torch.float32)
    total = None
    if state["residual"] is not None:
        h = h + state["residual"].to(torch.float32)
        total = h.to(torch.bfloat16)
    v = h * (1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)) * state["gamma"]
    codes, scale = _to_rows8(v)
    return total, codes, scale


def _plain_append(state):
    v = state["x"].to(torch.float32)
    if state["case"]["norm"]:
        v = v * (1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)) * state["gamma"]
    # the last 64 dims rotated in pairs by position * theta^(-2j / 64); the angle in 64 bits
    freq = THETA ** (-2.0 * torch.arange(ROPE_DIM // 2, dtype=torch.float64, device="cuda") / ROPE_DIM)
    ang = state["pos"].to(torch.float64)[:, None] * freq
    c, s = torch.cos(ang).to(torch.float32), torch.sin(ang).to(torch.float32)
    d = v.shape[-1]
    a, b = v[:, d - ROPE_DIM::2], v[:, d - ROPE_DIM + 1::2]
    v = torch.cat([v[:, :d - ROPE_DIM], torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)], dim=-1)
    rows = state["bt"][state["req"], state["pos"] // 256].long() * 256 + state["pos"] % 256
    if state["scale"] is None:
        state["data"][rows] = v.to(torch.bfloat16)
    else:
        amax = v.abs().amax(-1)
        scale = torch.where(amax > 0, amax / 448.0, 1.0)
        state["data"][rows] = (v / scale[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        state["scale"][rows] = scale
    return _stored(state)


def _plain_gemm(state):
    n, k = state["case"]["n"], state["case"]["k"]
    a = state["a"].view(torch.float8_e4m3fn).to(torch.float32) * _spread(state["a_scale"], k)
    ws = _spread(_spread(state["w_scale"], k).transpose(1, 2), n).transpose(1, 2)
    w = state["w"].view(torch.float8_e4m3fn).to(torch.float32) * ws
    out = torch.matmul(a.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1)
    if state["scale"] is not None:
        return _to_rows8(out)
    return out.to(state["out"].dtype).contiguous()


# ---- the definition in 64 bits ----------------------------------------------------------------------------------------
def _held(codes):
    """The value, in 64 bits, of each e4m3 byte, its fields taken apart."""
    b = torch.arange(256, device="cuda", dtype=torch.int64)
    e, m = (b >> 3) & 15, (b & 7).to(torch.float64)
    mag = torch.where(e == 0, m / 512, (1 + m / 8) * 2.0 ** (e - 7).to(torch.float64))
    return torch.where(b >= 128, -mag, mag)[codes.to(torch.int32)]


def _unrounded_rows8(v):
    """8-bit rows before their rounding: v / scale and the scales, in 64 bits."""
    n = v.shape[-1]
    at = torch.arange(n, device="cuda") // BLOCK
    amax = torch.zeros((*v.shape[:-1], _blocks(n)), dtype=torch.float64, device="cuda")
    amax = amax.scatter_reduce(-1, at.expand(v.shape), v.abs(), "amax")
    scale = torch.where(amax == 0, 1.0, amax / 448)
    return v / scale[..., at], scale


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "gemm": _exact_gemm}[case["op"]](state)


def _exact_norm(state):
    h = state["x"].to(torch.float64)
    if state["residual"] is not None:
        h = h + state["residual"].to(torch.float64)
    size = torch.linalg.vector_norm(h, dim=1)
    v = h / torch.sqrt(size ** 2 / h.shape[1] + EPS)[:, None] * state["gamma"].to(torch.float64)
    codes, scale = _unrounded_rows8(v)
    return (None if state["residual"] is None else h), codes, scale


def _exact_append(state):
    x = state["x"].to(torch.float64)
    d = x.shape[1]
    if state["case"]["norm"]:
        x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=1) ** 2 / d + EPS)[:, None] * state["gamma"].to(torch.float64)
    turns = [THETA ** (-j / ROPE_DIM) for j in range(0, ROPE_DIM, 2)]
    theta = torch.outer(state["pos"].to(torch.float64), torch.tensor(turns, dtype=torch.float64, device="cuda"))
    pairs = torch.view_as_complex(x[:, d - ROPE_DIM:].unflatten(-1, (-1, 2)).contiguous())
    x = x.clone()
    x[:, d - ROPE_DIM:] = torch.view_as_real(pairs * torch.polar(torch.ones_like(theta), theta)).flatten(-2)
    block = state["bt"][state["req"], torch.div(state["pos"], 256, rounding_mode="floor")].to(torch.int64)
    at = block * 256 + state["pos"].remainder(256)
    data = torch.zeros(state["data"].shape, dtype=torch.float64, device="cuda")
    if state["scale"] is None:
        data[at] = x
        return data
    scale = torch.zeros(len(data), dtype=torch.float64, device="cuda")
    amax = torch.linalg.vector_norm(x, float("inf"), dim=1)
    scale[at] = torch.where(amax == 0, 1.0, amax / 448)
    data[at] = x / scale[at][:, None]
    return data, scale


def _exact_gemm(state):
    m, n, k, groups = (state["case"][c] for c in ("m", "n", "k", "groups"))
    out = torch.empty((m, groups, n), dtype=torch.float64, device="cuda")
    ik, jn = torch.arange(k, device="cuda") // BLOCK, torch.arange(n, device="cuda") // BLOCK
    for g in range(groups):
        a = _held(state["a"][:, g]) * state["a_scale"][:, g].to(torch.float64)[:, ik]
        for lo in range(0, n, 4096):
            rows = slice(lo, min(n, lo + 4096))
            w = _held(state["w"][g, rows]) * state["w_scale"][g].to(torch.float64)[jn[rows]][:, ik]
            out[:, g, rows] = torch.einsum("mk,nk->mn", a, w)
    return _unrounded_rows8(out) if state["scale"] is not None else out
