"""Cases of a layer's projections in 8 bits: root-mean-square norm, E4M3
quantisers and the matrix product of codes with a scale for each block of 128.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges,
``prepare`` makes the inputs on the GPU from a seed, ``run`` computes one pass:
in elementary torch operations where ``own`` is false, through the package's
entry points where it is true.  ``exact`` computes the same outputs in 64 bits
and ``work`` counts what a pass cannot do without.

Operators (``op``):
  norm      y = h / rms(h) * weight per row, h = x + residual where there is one
            (rounded to the type and given back); rows are tokens, or the heads
            of a token inside a projection's output.
  norm8     the same, held as E4M3 codes with one float32 scale per 128 elements.
  quant     16-bit rows as such codes: a scale per row and 128 columns (an
            activation), or per 128 x 128 elements (a weight).
  matmul    out = A B^T of codes [M, K] and [N, K], scales of A per row and 128
            columns, of B per 128 x 128; out in 16 or 32 bits.
"""
import math

import torch

own = False

GROUP = 128     # elements of a row that share a scale
EPS = 1e-5
LARGEST = 448.0  # of E4M3
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of a step's feed-forward part, residual stream beside it
        {"name": "norm one step of 64 tokens", "op": "norm", "tokens": 64, "heads": 1, "dim": 8192,
         "dtype": "bf16", "residual": True},
        # norms of the query heads in front of the rotary append, a prompt; the heads are a
        # slice of one projection's output
        {"name": "norm query heads of 8191 tokens", "op": "norm", "tokens": 8191, "heads": 64,
         "dim": 128, "dtype": "bf16", "residual": False},
        # the norm in front of a step's projection
        {"name": "norm8 one step of 64 tokens", "op": "norm8", "tokens": 64, "dim": 8192,
         "dtype": "bf16", "residual": True},
        # the prompts of a batch that shares a system prompt
        {"name": "norm8 prompts of 33098 tokens", "op": "norm8", "tokens": 33098, "dim": 4096,
         "dtype": "fp16", "residual": True},
        # an attention's output on its way to the output projection
        {"name": "quant attention output, 8191 tokens", "op": "quant", "rows": 8191, "dim": 8192,
         "dtype": "bf16", "block": 1},
        # a layer's weights taken over from 16 bits
        {"name": "quant weights 10240 x 8192", "op": "quant", "rows": 10240, "dim": 8192,
         "dtype": "bf16", "block": 128},
        # one token of a small model: one launch, latency
        {"name": "matmul one token, small", "op": "matmul", "m": 1, "n": 768, "k": 512,
         "dtype": "fp16"},
        # a decode step's query, key and value projection, grouped heads
        {"name": "matmul step of 64 tokens", "op": "matmul", "m": 64, "n": 10240, "k": 8192,
         "dtype": "bf16"},
        # the logits of a decode step, kept in 32 bits
        {"name": "matmul logits of 33 tokens", "op": "matmul", "m": 33, "n": 32000, "k": 4096,
         "dtype": "fp32"},
        # a chunk of a prompt beside running requests
        {"name": "matmul chunk of 517 tokens", "op": "matmul", "m": 517, "n": 4096, "k": 4096,
         "dtype": "bf16"},
        # a long prompt's projection, grouped heads
        {"name": "matmul prompt of 8191 tokens", "op": "matmul", "m": 8191, "n": 10240, "k": 8192,
         "dtype": "bf16"},
        # the prompts of a batch, every query head with its own kv head
        {"name": "matmul prompts of 33098 tokens", "op": "matmul", "m": 33098, "n": 12288,
         "k": 4096, "dtype": "fp16"},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["norm", "norm8", "quant", "matmul", "matmul", "matmul"])
    if op == "matmul":
        m, n = _spread(rng, 1, 33098), _spread(rng, 64, 32000)
        if rng.random() < 0.7:
            n = -(-n // 64) * 64            # heads of 64 and 128; else an odd vocabulary
        k = 16 * _spread(rng, 8, 512)
        if rng.random() < 0.7:
            k = -(-k // 128) * 128
        m = max(1, min(m, 33098 * 12288 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["fp16", "bf16", "bf16",
                                                                       "fp32"])}
    case = {"op": op, "dtype": rng.choice(["fp16", "bf16"])}
    if op == "norm" and rng.random() < 0.5:
        dim, heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 5, 7, 8, 16, 32, 64])
        return {**case, "tokens": min(_spread(rng, 1, 33098), 33098 * 32 // heads), "heads": heads,
                "dim": dim, "residual": False}
    dim = 16 * _spread(rng, 4, 1024)
    rows = max(1, min(_spread(rng, 1, 33098), 33098 * 4096 // dim))
    if op == "quant":
        return {**case, "rows": rows, "dim": dim, "block": rng.choice([1, 1, 128])}
    case = {**case, "tokens": rows, "dim": dim, "residual": rng.choice([True, True, False])}
    return {**case, "heads": 1} if op == "norm" else case


# ------------------------------------------------------------------ inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 64 + k)
    return g


def _rows(shape, dtype, seed, k):
    """Activations: N(0, 1) with some channels much larger, as a model's are."""
    x = torch.randn(shape, generator=_gen(seed, k), device="cuda")
    wide = torch.rand(shape[-1], generator=_gen(seed, k + 1), device="cuda")
    return x.mul_(torch.where(wide < 0.02, 12.0, 0.5 + wide)).to(dtype)


def prepare(case, seed):
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "matmul":
        M, N, K = case["m"], case["n"], case["k"]
        a, sa = _codes(_rows((M, K), torch.float16, seed, 0).float(), 1)
        w = torch.randn((N, K), generator=_gen(seed, 2), device="cuda").mul_(K ** -0.5)
        w *= 0.25 + torch.rand((N, 1), generator=_gen(seed, 3), device="cuda")
        b, sb = _codes(w, GROUP)
        return {"case": case, "a": a, "sa": sa, "b": b, "sb": sb,
                "out": torch.zeros((M, N), dtype=dt, device="cuda")}
    if op == "quant":
        R, D, block = case["rows"], case["dim"], case["block"]
        x = _rows((R, D), dt, seed, 0)
        return {"case": case, "x": x, **_buffers(R, D, block)}
    T, D, H = case["tokens"], case["dim"], case.get("heads", 1)
    state = {"case": case, "weight": (1 + 0.2 * torch.randn(
        D, generator=_gen(seed, 4), device="cuda")).to(dt), "residual": None}
    if H > 1:  # the first heads of a projection of H query heads and two kv heads
        state["x"] = _rows((T, H + 2, D), dt, seed, 0)[:, :H]
    else:
        state["x"] = _rows((T, D), dt, seed, 0)
    if case["residual"]:
        state["residual"] = (4 * torch.randn((T, D), generator=_gen(seed, 5), device="cuda")).to(dt)
        state["sum"] = torch.zeros((T, D), dtype=dt, device="cuda")
    if op == "norm":
        state["out"] = torch.zeros(state["x"].shape, dtype=dt, device="cuda")
        return state
    return {**state, **_buffers(T, D, 1)}


def _buffers(rows, dim, block):
    return {"codes": torch.zeros((rows, dim), dtype=torch.uint8, device="cuda").view(F8),
            "scales": torch.zeros((-(-rows // block), -(-dim // GROUP)), device="cuda")}


# ------------------------------------------------------------------ plain forms
def _codes(x, block):
    """E4M3 codes of x [R, D] float32 and their scales, one per `block` rows and
    128 columns: scale = largest / 448, code = x * (448 / largest) rounded."""
    R, D = x.shape
    nr, nd = -(-R // block), -(-D // GROUP)
    g = torch.nn.functional.pad(x, (0, nd * GROUP - D, 0, nr * block - R))
    g = g.view(nr, block, nd, GROUP)
    most = g.abs().amax((1, 3), keepdim=True)
    safe = most.clamp(min=2.0 ** -100)
    scales = torch.where(most > 0, safe / LARGEST, 1.0)
    # (LARGEST / safe would be LARGEST times a reciprocal: two roundings)
    codes = (g * torch.full_like(safe, LARGEST).div(safe)).to(F8).view(torch.uint8).view(nr * block, nd * GROUP)
    return codes[:R, :D].contiguous().view(F8), scales.view(nr, nd)


def _values(codes, scales, block):
    """float32 values of codes [R, D]."""
    R, D = codes.shape
    s = scales.repeat_interleave(GROUP, 1)[:, :D]
    return codes.float() * (s if block == 1 else s.repeat_interleave(block, 0)[:R])


def _plain_norm(st):
    h = st["x"].float()
    if st["residual"] is not None:
        h = (h + st["residual"].float()).to(st["x"].dtype)
    f = h.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * st["weight"].float()
    return (h if st["residual"] is not None else None), y


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    if op == "matmul":
        a, b = _values(state["a"], state["sa"], 1), _values(state["b"], state["sb"], GROUP)
        return torch.matmul(a, b.t()).to(state["out"].dtype)
    if op == "quant":
        codes, scales = _codes(state["x"].float(), state["case"]["block"])
        return {"codes": codes, "scales": scales}
    h, y = _plain_norm(state)
    if op == "norm":
        return {"y": y.to(state["x"].dtype), "sum": h}
    codes, scales = _codes(y, 1)
    return {"codes": codes, "scales": scales, "sum": h}


def _own_norm(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_rms_norm(st["out"], st["x"], st["weight"], EPS, residual=st["residual"],
                     residual_out=st.get("sum"))
    return {"y": st["out"], "sum": st.get("sum")}


def _own_norm8(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_rms_norm_fp8(st["codes"], st["scales"], st["x"], st["weight"], EPS,
                         residual=st["residual"], residual_out=st.get("sum"))
    return {"codes": st["codes"], "scales": st["scales"], "sum": st.get("sum")}


def _own_quant(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_quantise_fp8(st["codes"], st["scales"], st["x"], block_rows=st["case"]["block"])
    return {"codes": st["codes"], "scales": st["scales"]}


def _own_matmul(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_matmul_fp8(st["out"], st["a"], st["sa"], st["b"], st["sb"])
    return st["out"]


_OWN = {"norm": _own_norm, "norm8": _own_norm8, "quant": _own_quant, "matmul": _own_matmul}


# ------------------------------------------------------------------ 64 bits
def _exact_codes(y, block):
    """The same as _codes in 64 bits, codes as the numbers that they are."""
    R, D = y.shape
    scales = torch.empty((-(-R // block), -(-D // GROUP)), dtype=torch.float64, device="cuda")
    codes = torch.empty_like(y)
    for j in range(scales.shape[1]):
        part = y[:, j * GROUP:(j + 1) * GROUP]
        most = part.abs().max(1)[0]
        if block > 1:
            most = torch.nn.functional.pad(most, (0, -R % block)).view(-1, block).max(1)[0]
        scales[:, j] = torch.where(most > 0, most / LARGEST, 1.0)
        v = part / scales[:, j].repeat_interleave(block)[:R, None]
        # three bits behind the leading one, 2^-9 at least
        step = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).double() - 3)
        codes[:, j * GROUP:(j + 1) * GROUP] = torch.round(v / step) * step
    return {"codes": codes, "scales": scales}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "matmul":
        a, b = st["a"].double(), st["b"].double()
        for x, s, block in ((a, st["sa"].double(), 1), (b, st["sb"].double(), GROUP)):
            for j in range(s.shape[1]):
                x[:, j * GROUP:(j + 1) * GROUP] *= s[:, j].repeat_interleave(block)[:len(x), None]
        return torch.mm(a, b.t())
    if case["op"] == "quant":
        return _exact_codes(st["x"].double(), case["block"])
    h = st["x"].double()
    total = None
    if case["residual"]:
        total = h + st["residual"].double()
        h = total.to(st["x"].dtype).double()    # the sum is kept in the type
    y = h / (h.square().sum(-1, keepdim=True) / case["dim"] + EPS).sqrt() * st["weight"].double()
    if case["op"] == "norm":
        return {"y": y, "sum": total}
    return {**_exact_codes(y, 1), "sum": total}


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "matmul":
        M, N, K = case["m"], case["n"], case["k"]
        groups = -(-K // GROUP)
        return {"bytes": (M + N) * K + 4 * groups * (M + -(-N // GROUP))
                + M * N * (4 if case["dtype"] == "fp32" else 2), "flops": 2 * M * N * K}
    if op == "quant":
        n = case["rows"] * case["dim"]
        return {"bytes": 3 * n + 4 * n // (GROUP * case["block"]), "flops": 3 * n}
    n = case["tokens"] * case.get("heads", 1) * case["dim"]
    moved = 2 * n + 2 * case["dim"] + (4 * n if case["residual"] else 0)
    if op == "norm":
        return {"bytes": moved + 2 * n, "flops": 5 * n}
    return {"bytes": moved + n + 4 * n // GROUP, "flops": 8 * n}
