"""Measured cases of the MXFP4 and grouped-expert operators.

quantise  rows to MXFP4 (e2m1 codes, one e8m0 scale per 32) and back to the values the codes stand for
product   y = x W^T with MXFP4 weights, x in bf16 or MXFP4
group     the routed (token, rank) pairs ordered by expert
grouped   ragged products of each expert's rows with that expert's weights; "up" gathers token rows and
          ends in silu(gate) * up, "down" takes grouped rows and writes one row per pair
combine   the weighted sum of a token's k expert rows

``own`` False computes the operators from elementary torch operations in
32 bits; True calls the library.
"""
import torch

own = False

BLOCK = 32
# magnitudes of the e2m1 codes 0..7
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # hidden states of eight concurrent decode streams on their way into a 4-bit product
        {"name": "quantise-streams", "op": "quantise", "rows": 8, "cols": 2048, "dtype": "bf16"},
        # fp32 checkpoint matrices of sixteen experts converted into the bank format
        {"name": "quantise-banks", "op": "quantise", "rows": 32768, "cols": 4096, "dtype": "f32"},
        # one token through a dense (shared-expert or attention) projection held in 4 bits
        {"name": "product-token", "op": "product", "M": 1, "N": 4096, "K": 4096, "act": "bf16", "out": "bf16"},
        # a short odd prompt: ragged rows and columns, an odd number of scale blocks
        {"name": "product-ragged", "op": "product", "M": 333, "N": 2040, "K": 2080, "act": "bf16", "out": "f32"},
        # a prefill chunk with 4-bit activations
        {"name": "product-chunk", "op": "product", "M": 8192, "N": 4096, "K": 4096, "act": "mxfp4", "out": "bf16"},
        # routing of eight decode streams
        {"name": "group-streams", "op": "group", "T": 8, "k": 8, "E": 128, "zipf": 1.1, "pad": 0},
        # routing of a prefill chunk whose batch is padded at the end
        {"name": "group-chunk", "op": "group", "T": 8192, "k": 8, "E": 256, "zipf": 1.0, "pad": 100},
        # gate/up of eight decode streams over resident bf16 experts
        {"name": "grouped-streams-bf16", "op": "grouped", "dir": "up", "T": 8, "k": 8, "E": 128, "N": 1536,
         "K": 2048, "act": "bf16", "w": "bf16", "out": "bf16", "zipf": 1.1},
        # gate/up of a prefill chunk, weights and activations in 4 bits
        {"name": "grouped-chunk-mxfp4", "op": "grouped", "dir": "up", "T": 8192, "k": 8, "E": 256, "N": 4096,
         "K": 4096, "act": "mxfp4", "w": "mxfp4", "out": "bf16", "zipf": 1.0},
        # down projection of an odd-length prompt over bf16 experts
        {"name": "grouped-prompt-bf16", "op": "grouped", "dir": "down", "T": 4001, "k": 8, "E": 128, "N": 2048,
         "K": 768, "act": "bf16", "w": "bf16", "out": "f32", "zipf": 1.1},
        # merge of eight decode streams
        {"name": "combine-streams", "op": "combine", "T": 8, "k": 8, "H": 2048, "rows": "f32", "out": "bf16"},
        # merge of a prefill chunk
        {"name": "combine-chunk", "op": "combine", "T": 8192, "k": 8, "H": 4096, "rows": "f32", "out": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def _drawn(rng, op):
    if op == "quantise":
        return {"op": op, "rows": _log_int(rng, 1, 65536), "cols": _log_int(rng, 32, 8192, 32),
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "product":
        return {"op": op, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 64, 8192, rng.choice([1, 8, 64])),
                "K": _log_int(rng, 256, 8192, 32), "act": rng.choice(["bf16", "mxfp4"]),
                "out": rng.choice(["bf16", "f32"])}
    if op == "group":
        T = _log_int(rng, 1, 8192)
        return {"op": op, "T": T, "k": rng.choice([1, 2, 4, 6, 8]), "E": rng.choice([8, 16, 60, 128, 256]),
                "zipf": rng.choice([0.0, 1.0, 1.1]), "pad": rng.choice([0, T // 5])}
    if op == "grouped":
        act, w = rng.choice([("bf16", "bf16"), ("bf16", "mxfp4"), ("mxfp4", "mxfp4")])
        return {"op": op, "dir": rng.choice(["up", "down"]), "T": _log_int(rng, 1, 8192),
                "k": rng.choice([1, 2, 4, 8]), "E": rng.choice([8, 16, 60, 128, 256]),
                "N": _log_int(rng, 256, 4096, rng.choice([2, 8, 64])), "K": _log_int(rng, 256, 4096, 32),
                "act": act, "w": w, "out": rng.choice(["bf16", "f32"]), "zipf": rng.choice([0.0, 1.0, 1.1])}
    return {"op": op, "T": _log_int(rng, 1, 8192), "k": rng.choice([1, 2, 4, 6, 8]), "H": _log_int(rng, 64, 4096),
            "rows": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"])}


def draw(rng):
    op = rng.choice(["quantise", "product", "product", "group", "grouped", "grouped", "combine"])
    most = [work(c) for c in listed() if c["op"] == op]
    while True:
        case = _drawn(rng, op)
        w = work(case)
        if all(w[key] <= max(m[key] for m in most) for key in ("bytes", "flops")):
            return case


def work(case):
    op = case["op"]
    if op == "quantise":
        n = case["rows"] * case["cols"]
        b = 4 if case["dtype"] == "f32" else 2
        # values in, codes and scales out, codes and scales in, values out
        return {"bytes": n * (2 * b + 2 * (1 / 2 + 1 / 32)), "flops": 4 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * _bytes(case["act"]) + N * K * _bytes("mxfp4") + M * N * _bytes(case["out"]),
                "flops": 2 * M * N * K}
    if op == "group":
        return {"bytes": 8 * case["T"] * case["k"] + 4 * (case["E"] + 1), "flops": case["T"] * case["k"]}
    if op == "grouped":
        R = case["T"] * case["k"]
        x_rows = case["T"] if case["dir"] == "up" else R
        y_cols = case["N"] // 2 if case["dir"] == "up" else case["N"]
        touched = _expected_touched(case)
        return {"bytes": x_rows * case["K"] * _bytes(case["act"]) + touched * case["N"] * case["K"] * _bytes(case["w"])
                + R * y_cols * _bytes(case["out"]) + 8 * R, "flops": 2 * R * case["N"] * case["K"]}
    R = case["T"] * case["k"]
    return {"bytes": R * case["H"] * _bytes(case["rows"]) + 4 * R + case["T"] * case["H"] * _bytes(case["out"]),
            "flops": 2 * R * case["H"]}


def _bytes(dtype):
    return {"f32": 4, "bf16": 2, "mxfp4": 1 / 2 + 1 / 32}[dtype]


def _popularity(E, zipf):
    p = [(e + 1.0) ** -zipf for e in range(E)]
    s = sum(p)
    return [v / s for v in p]


def _expected_touched(case):
    """Experts that T draws of k experts reach, in expectation (drawn with replacement: a lower bound)."""
    n = case["T"] * case["k"]
    return sum(1 - (1 - p) ** n for p in _popularity(case["E"], case["zipf"]))


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, sigma=1.0):
    return torch.randn(shape, generator=g, device="cuda") * sigma


def _route(g, T, k, E, zipf):
    """k distinct experts per token, drawn by a popularity that falls as rank^-zipf (ranks shuffled)."""
    logp = torch.log(torch.tensor(_popularity(E, zipf), device="cuda"))[torch.randperm(E, generator=g, device="cuda")]
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)
    return torch.topk(logp - torch.log(-torch.log(u)), k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    dev = "cuda"
    op = case["op"]
    if op == "quantise":
        rows, cols = case["rows"], case["cols"]
        x = _normal(g, (rows, cols))
        # magnitudes differ from row to row and some blocks are zero, as in weights and hidden states
        x *= torch.exp2(torch.randint(-8, 9, (rows, 1), generator=g, device=dev).float())
        x.view(rows, cols // BLOCK, BLOCK)[torch.rand((rows, cols // BLOCK), generator=g, device=dev) < 0.01] = 0
        s["x"] = x.to(DTYPES[case["dtype"]])
        s["codes"] = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        s["scales"] = torch.empty((rows, cols // BLOCK), dtype=torch.uint8, device=dev)
        s["y"] = torch.empty_like(s["x"])
    elif op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        s["w"], s["w_scales"] = _quantise(_normal(g, (N, K), 0.02))
        x = _normal(g, (M, K))
        s["x"], s["x_scales"] = _quantise(x) if case["act"] == "mxfp4" else (x.to(torch.bfloat16), None)
        s["y"] = torch.empty((M, N), dtype=DTYPES[case["out"]], device=dev)
    elif op == "group":
        T, k, E = case["T"], case["k"], case["E"]
        s["ids"] = _route(g, T, k, E, case["zipf"])
        if case["pad"]:
            s["ids"][T - case["pad"]:] = -1  # tokens that pad the batch have no expert
        s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=dev)
        s["perm"] = torch.empty(T * k, dtype=torch.int32, device=dev)
        # 256 pairs a chunk and E counters for each: what the library asks for at most
        s["workspace"] = torch.empty(4 * E * (-(-T * k // 256)), dtype=torch.uint8, device=dev)
    elif op == "grouped":
        T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
        up = case["dir"] == "up"
        ids = _route(g, T, k, E, case["zipf"]).reshape(-1).long()
        order = torch.sort(ids, stable=True).indices
        counts = torch.zeros(E, dtype=torch.int64, device=dev).scatter_add_(0, ids, torch.ones_like(ids))
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
        s["perm"] = order.to(torch.int32)
        s["counts"] = counts.tolist()
        x = _normal(g, (T if up else T * k, K))
        s["x"], s["x_scales"] = _quantise(x) if case["act"] == "mxfp4" else (x.to(torch.bfloat16), None)
        s["w_scales"] = None
        if case["w"] == "mxfp4":
            s["w"] = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
            s["w_scales"] = torch.empty((E, N, K // BLOCK), dtype=torch.uint8, device=dev)
            for e in range(E):
                s["w"][e], s["w_scales"][e] = _quantise(_normal(g, (N, K), 0.02))
        else:
            s["w"] = torch.empty((E, N, K), dtype=torch.bfloat16, device=dev)
            for e in range(E):
                s["w"][e] = _normal(g, (N, K), 0.02)
        s["y"] = torch.empty((T * k, N // 2 if up else N), dtype=DTYPES[case["out"]], device=dev)
    else:
        T, k, H = case["T"], case["k"], case["H"]
        s["p"] = _normal(g, (T * k, H)).to(DTYPES[case["rows"]])
        s["w"] = torch.softmax(_normal(g, (T, k)), dim=1)
        s["y"] = torch.empty((T, H), dtype=DTYPES[case["out"]], device=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quantise":
        codes, scales = _quantise(s["x"].float())
        return _values(codes, scales).to(s["x"].dtype)
    if op == "product":
        return (_rows(s["x"], s["x_scales"]) @ _values(s["w"], s["w_scales"]).T).to(s["y"].dtype)
    if op == "group":
        E = s["E"]
        ids = s["ids"].reshape(-1).long()
        ids = torch.where((ids >= 0) & (ids < E), ids, E)
        key, order = torch.sort(ids, stable=True)
        counts = torch.zeros(E + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, ids, torch.ones_like(ids))
        offsets = torch.nn.functional.pad(counts[:E].cumsum(0), (1, 0))
        return offsets.to(torch.int32), torch.where(key < E, order, -1).to(torch.int32)
    if op == "grouped":
        return _grouped(s)
    p = s["p"].float().view(s["T"], s["k"], s["H"])
    return (s["w"][:, :, None] * p).sum(1).to(s["y"].dtype)


def _run_own(s):
    import routed_expert_execution_moe_amd as moe
    op = s["op"]
    if op == "quantise":
        moe.moe_mx_quantize(s["x"], s["codes"], s["scales"])
        moe.moe_mx_dequantize(s["codes"], s["scales"], s["y"])
    elif op == "product":
        moe.moe_mx_gemm(s["x"], s["w"], s["w_scales"], s["y"], x_scales=s["x_scales"])
    elif op == "group":
        moe.moe_group_pairs(s["ids"], s["E"], s["offsets"], s["perm"], workspace=s["workspace"])
        return s["offsets"], s["perm"]
    elif op == "grouped":
        up = s["dir"] == "up"
        moe.moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["y"], x_scales=s["x_scales"], w_scales=s["w_scales"],
                             x_index=s["perm"] if up else None, x_index_div=s["k"] if up else 1,
                             y_index=None if up else s["perm"], glu=up)
    else:
        moe.moe_combine_pairs(s["p"], s["w"], s["y"])
    return s["y"]


def _quantise(x):
    """Rows of fp32 to (codes, scales): exponent floor(log2 amax) - 2, nearest code, ties to the even code."""
    rows, cols = x.shape
    v = x.view(rows, cols // BLOCK, BLOCK)
    amax = v.abs().amax(2)
    e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, 0)
    a = torch.ldexp(v, -e[:, :, None])
    m = a.abs()
    code = torch.zeros_like(v, dtype=torch.uint8)
    # the borders halfway between neighbours of the grid; a tie goes up where the upper code is even
    for border, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (m >= border) if tie_up else (m > border)
    code = torch.where((a < 0) & (code > 0), code + 8, code).view(rows, cols // 2, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """The fp32 values that codes [..., C/2] and scales [..., C/32] stand for."""
    table = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), dim=-1).view(*scales.shape, BLOCK)
    v = torch.ldexp(table[pair.int()], scales[..., None].int() - 127)
    return v.view(*codes.shape[:-1], codes.shape[-1] * 2)


def _rows(x, scales):
    return x.float() if scales is None else _values(x, scales)


def _silu_product(y):
    gate, up = y.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _grouped(s):
    up = s["dir"] == "up"
    order = s["perm"].long()
    x = _rows(s["x"], s["x_scales"])
    x = x[order // s["k"]] if up else x
    y = torch.empty_like(s["y"])
    at = 0
    for e, n in enumerate(s["counts"]):
        if n == 0:
            continue
        w = s["w"][e].float() if s["w_scales"] is None else _values(s["w"][e], s["w_scales"][e])
        part = x[at:at + n] @ w.T
        if up:
            y[at:at + n] = _silu_product(part)
        else:
            y[order[at:at + n]] = part.to(y.dtype)
        at += n
    return y


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return _exact_round_trip(s["x"].double())
    if op == "group":
        return _exact_group(s["ids"], case["E"])
    if op == "product":
        x = s["x"].double() if s["x_scales"] is None else _decode64(s["x"], s["x_scales"])
        return torch.matmul(x, _decode64(s["w"], s["w_scales"]).t())
    if op == "grouped":
        x = s["x"].double() if s["x_scales"] is None else _decode64(s["x"], s["x_scales"])
        perm, offsets = s["perm"].long(), s["offsets"].tolist()
        y = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            rows = perm[offsets[e]:offsets[e + 1]]
            if rows.numel() == 0:
                continue
            w = s["w"][e].double() if s["w_scales"] is None else _decode64(s["w"][e], s["w_scales"][e])
            if case["dir"] == "up":
                z = torch.matmul(x[torch.div(rows, case["k"], rounding_mode="floor")], w.t())
                half = case["N"] // 2
                y[offsets[e]:offsets[e + 1]] = z[:, :half] * torch.sigmoid(z[:, :half]) * z[:, half:]
            else:
                y[rows] = torch.matmul(x[offsets[e]:offsets[e + 1]], w.t())
        return y
    p = s["p"].double().view(case["T"], case["k"], case["H"])
    return torch.bmm(s["w"].double()[:, None, :], p)[:, 0, :]


def _exact_group(ids, E):
    """Pairs by (expert, pair index) as one 64-bit key each; a pair of no expert comes last as -1."""
    ids = ids.flatten().to(torch.int64)
    n = ids.numel()
    expert = torch.where((ids < 0) | (ids >= E), E, ids)
    keys = torch.sort(expert * n + torch.arange(n, device=ids.device)).values
    perm = torch.where(keys >= E * n, -1, keys % n)
    offsets = torch.searchsorted(keys, torch.arange(E + 1, device=ids.device) * n)
    return offsets.to(torch.int32), perm.to(torch.int32)


def _decode64(codes, scales):
    """Sign, exponent and mantissa bits of each e2m1 code times its block's power of two, in fp64."""
    c = torch.empty((*codes.shape, 2), dtype=torch.int32, device=codes.device)
    c[..., 0] = codes.int() % 16
    c[..., 1] = torch.div(codes.int(), 16, rounding_mode="floor")
    c = c.flatten(-2)
    exponent, mantissa = (c // 2) % 4, (c % 2).double()
    size = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * torch.exp2((exponent - 1).double()))
    size = torch.where(c >= 8, -size, size)
    return size * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, dim=-1)


def _exact_round_trip(x):
    """Every value's nearest multiple of its own step on the e2m1 grid under its block's scale."""
    out = torch.empty_like(x)
    for i in range(0, x.shape[0], 4096):
        v = x[i:i + 4096].unflatten(1, (-1, BLOCK))
        top = v.abs().amax(2, keepdim=True)
        power = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
        power = power + (torch.exp2(power + 1) <= top).double() - (torch.exp2(power) > top).double()
        scale = torch.exp2((power - 2).clamp(-127, 127))
        q = v / scale
        # steps of 1/2 below 2, of 1 below 4, of 2 from there; round() takes ties to even
        step = torch.where(q.abs() < 2, 0.5, torch.where(q.abs() < 4, 1.0, 2.0))
        out[i:i + 4096] = ((torch.round(q / step) * step).clamp(-6, 6) * scale).flatten(1)
    return out
