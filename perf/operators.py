"""Cases of the 4-bit cache, the rotary append and the device-side block tables.

``listed()`` names the cases, ``draw(rng)`` makes more of the same ranges,
``prepare`` makes the inputs on the GPU from a seed, ``run`` computes one pass:
in elementary torch operations where ``own`` is false, through the package's
entry points where it is true.  ``exact`` computes the same outputs in 64 bits
and ``work`` counts what a pass cannot do without.

Operators (``op``):
  decode4   single-query attention over a paged cache of 4-bit codes with one
            (scale, zero) pair per 64 elements of a token's K or V row.
  append4   quantise new K/V rows into their slots of that cache and read the
            rows back as the 16-bit values they stand for.
  rope      rotate q and k by positions on one to four axes (time, height,
            width, ...), write K and V to their slots of a 16-bit cache.
  rope4     the same into the 4-bit cache; the rows are read back.
  tables    one serving step's plan: blocks of finished requests go back to the
            free stack, the others' tables grow by their new tokens, and the
            slots, query offsets and positions of those tokens are listed.
"""
import math

import torch

own = False

BLOCK = 16      # tokens per cache block
GROUP = 64      # elements per (scale, zero) pair
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # four short requests of a small model: one launch, latency
        {"name": "decode4 four short requests", "op": "decode4", "batch": 4, "heads": 8,
         "kv_heads": 2, "dim": 64, "dtype": "fp16", "shortest": 1, "longest": 255},
        # a serving batch with grouped heads and ragged contexts
        {"name": "decode4 ragged batch, grouped heads", "op": "decode4", "batch": 64, "heads": 64,
         "kv_heads": 8, "dim": 128, "dtype": "bf16", "shortest": 512, "longest": 8192},
        # a serving batch where every query head has its own kv head
        {"name": "decode4 batch of 4096-token contexts", "op": "decode4", "batch": 32,
         "heads": 32, "kv_heads": 32, "dim": 128, "dtype": "fp16", "shortest": 4096,
         "longest": 4096},
        # four very long documents
        {"name": "decode4 four 131072-token contexts", "op": "decode4", "batch": 4, "heads": 64,
         "kv_heads": 8, "dim": 128, "dtype": "fp16", "shortest": 131072, "longest": 131072},
        # the new tokens of one decode step
        {"name": "append4 one step of 64 requests", "op": "append4", "tokens": 64, "kv_heads": 8,
         "dim": 128, "dtype": "bf16"},
        # the prompts of a batch that shares a system prompt
        {"name": "append4 prompts of 33098 tokens", "op": "append4", "tokens": 33098,
         "kv_heads": 32, "dim": 128, "dtype": "fp16"},
        # one decode step after images: three axes
        {"name": "rope one step of 64 requests", "op": "rope", "tokens": 64, "heads": 64,
         "kv_heads": 8, "dim": 128, "rotary": 128, "axes": 3, "interleaved": False,
         "dtype": "bf16"},
        # prompts with images and video
        {"name": "rope prompts of 33098 tokens", "op": "rope", "tokens": 33098, "heads": 32,
         "kv_heads": 32, "dim": 128, "rotary": 128, "axes": 3, "interleaved": False,
         "dtype": "fp16"},
        # one decode step of text into the 4-bit cache, adjacent pairs, half the row rotated
        {"name": "rope4 one step of 32 requests", "op": "rope4", "tokens": 32, "heads": 8,
         "kv_heads": 2, "dim": 64, "rotary": 32, "axes": 1, "interleaved": True, "dtype": "fp16"},
        # a long prompt with images into the 4-bit cache
        {"name": "rope4 prompt of 8191 tokens", "op": "rope4", "tokens": 8191, "heads": 64,
         "kv_heads": 8, "dim": 128, "rotary": 128, "axes": 3, "interleaved": False,
         "dtype": "bf16"},
        # a decode step: one new token for each running request
        {"name": "tables one step of 64 requests", "op": "tables", "batch": 64, "longest": 8192,
         "most_new": 1, "blocks": 40000},
        # a step that admits prompts beside the running requests
        {"name": "tables 1024 requests with prompts", "op": "tables", "batch": 1024,
         "longest": 4096, "most_new": 512, "blocks": 400000},
    ]


def _spread(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["decode4", "append4", "rope", "rope4", "tables"])
    if op == "tables":
        return {"op": op, "batch": _spread(rng, 1, 1024), "longest": _spread(rng, 16, 8192),
                "most_new": rng.choice([1, _spread(rng, 1, 512)]), "blocks": 600000}
    dim = rng.choice([64, 128])
    kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
    case = {"op": op, "kv_heads": kv, "dim": dim, "dtype": rng.choice(["fp16", "bf16"])}
    if op == "append4":
        return {**case, "tokens": _spread(rng, 1, 33098)}
    group = rng.choice([1, 1, 2, 3, 4, 6, 7, 8, 12, 16])
    heads = kv * group
    if op in ("rope", "rope4"):
        tokens = _spread(rng, 1, 33098)
        tokens = max(1, min(tokens, 33098 * 96 // (heads + 2 * kv)))
        return {**case, "tokens": tokens, "heads": heads,
                "rotary": rng.choice([dim, dim, dim // 2]), "axes": rng.choice([1, 2, 3, 3, 4]),
                "interleaved": rng.choice([False, False, True])}
    # decode4: at most 4 M (token, kv head) pairs and 64 query heads
    while heads > 64:
        group = max(1, group // 2)
        heads = kv * group
        if group == 1:
            break
    batch = _spread(rng, 1, 128)
    most = max(1, min(131072, 4 * 131072 * 8 // (batch * kv * max(1, group // 8))))
    longest = _spread(rng, 1, most)
    return {**case, "heads": heads, "batch": batch, "longest": longest,
            "shortest": rng.choice([longest, 1 + longest // 16])}


# ------------------------------------------------------------------ inputs
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 64 + k)
    return g


def _normal(shape, dtype, seed, k, offset=0.0):
    """N(0, 1) values, and where `offset` is given a bias of that size per channel
    (cached keys have channels far from zero)."""
    g = _gen(seed, k)
    x = torch.randn(shape, generator=g, device="cuda")
    if offset:
        x += offset * torch.randn(shape[-1], generator=g, device="cuda")
    return x.to(dtype)


def _sections(case):
    """Rotary pairs per axis: the first axis takes what the others leave."""
    half, axes = case["rotary"] // 2, case["axes"]
    rest = [3 * half // (2 * (axes + 1)) if axes > 1 else 0] * (axes - 1)
    return [half - sum(rest)] + rest


def prepare(case, seed):
    op = case["op"]
    if op == "tables":
        return _prepare_tables(case, seed)
    kv, D, dt = case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
    groups = D // GROUP
    if op == "decode4":
        B, Hq = case["batch"], case["heads"]
        lens = torch.randint(case["shortest"], case["longest"] + 1, (B,), generator=_gen(seed, 0),
                             device="cuda").to(torch.int32)
        lens[0] = case["longest"]
        per = -(-case["longest"] // BLOCK)
        blocks = -(-lens.long() // BLOCK)
        NB = int(blocks.sum()) + 7
        perm = torch.randperm(NB, generator=_gen(seed, 1), device="cuda").to(torch.int32)
        at = torch.arange(per, device="cuda")[None, :]
        first = (torch.cumsum(blocks, 0) - blocks)[:, None]
        tables = torch.where(at < blocks[:, None], perm[(first + at).clamp(max=NB - 1)], -1)
        kc, ks = _quantise(_normal((NB, kv, BLOCK, D), dt, seed, 2, offset=1.0))
        vc, vs = _quantise(_normal((NB, kv, BLOCK, D), dt, seed, 3))
        q = _normal((B, Hq, D), dt, seed, 4)
        return {"case": case, "q": q, "kc": kc, "vc": vc, "ks": ks, "vs": vs,
                "tables": tables.to(torch.int32).contiguous(), "lens": lens,
                "scale": 1.0 / math.sqrt(D), "out": torch.empty_like(q)}
    T = case["tokens"]
    NB = -(-T // BLOCK) + 5
    slots = torch.randperm(NB * BLOCK, generator=_gen(seed, 0), device="cuda")[:T].to(torch.int32)
    if T > 8:  # a padded batch: some rows are nobody's
        slots[-(T // 8):] = torch.where(
            torch.rand(T // 8, generator=_gen(seed, 1), device="cuda") < 0.25, -1,
            slots[-(T // 8):])
    state = {"case": case, "slots": slots}
    if op in ("append4", "rope4"):
        state["kc"] = torch.zeros((NB, kv, BLOCK, D // 2), dtype=torch.uint8, device="cuda")
        state["vc"] = torch.zeros_like(state["kc"])
        state["ks"] = torch.zeros((NB, kv, BLOCK, groups, 2), dtype=dt, device="cuda")
        state["vs"] = torch.zeros_like(state["ks"])
        state["k_read"] = torch.zeros((T, kv, D), dtype=dt, device="cuda")
        state["v_read"] = torch.zeros_like(state["k_read"])
    else:
        state["kc"] = torch.zeros((NB, kv, BLOCK, D), dtype=dt, device="cuda")
        state["vc"] = torch.zeros_like(state["kc"])
    if op == "append4":
        state["k"] = _normal((T, kv, D), dt, seed, 2, offset=1.0)
        state["v"] = _normal((T, kv, D), dt, seed, 3)
        return state
    # q, k and v are slices of one projection's output
    Hq, R, A = case["heads"], case["rotary"], case["axes"]
    qkv = _normal((T, Hq + 2 * kv, D), dt, seed, 2)
    state["q"], state["k"], state["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + kv], qkv[:, Hq + kv:]
    state["q_out"] = torch.zeros((T, Hq, D), dtype=dt, device="cuda")
    state["cos_sin"] = _cos_sin(R)
    # tokens of frames, rows and columns; text follows the last frame on every axis
    i = torch.arange(T, device="cuda") + 37 * (int(seed) % 1009)
    axes = [i // 256 % ROWS, i // 16 % 16 + i // 4096, i % 16 + i // 2048, i % ROWS]
    if A == 1:
        axes[0] = i % ROWS
    state["positions"] = torch.stack(axes[:A]).to(torch.int32).contiguous()
    state["sections"] = _sections(case)
    state["axis"] = torch.repeat_interleave(torch.arange(A), torch.tensor(state["sections"])).cuda()
    return state


ROWS = 40960  # positions in the table of angles


def _cos_sin(R):
    """[ROWS, R] float32: cos of the R/2 angles, then sin (angles in 64 bits)."""
    inv = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    ang = torch.arange(ROWS, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def _prepare_tables(case, seed):
    B, MB, NB = case["batch"], case["longest"] // BLOCK + case["most_new"] // BLOCK + 2, \
        case["blocks"]
    g = _gen(seed, 0)
    lens = torch.randint(0, case["longest"] + 1, (B,), generator=g, device="cuda")
    kind = torch.rand(B, generator=g, device="cuda")
    finished = (kind < 0.125) & (lens > 0)                # done: their blocks come back
    fresh = (kind > 0.875) & ~finished                    # free places that admit a prompt
    lens = torch.where(fresh, 0, lens)
    new = torch.ones(B, dtype=torch.long, device="cuda")
    if case["most_new"] > 1:
        prompt = torch.randint(1, case["most_new"] + 1, (B,), generator=g, device="cuda")
        new = torch.where(fresh | (kind > 0.5), prompt, new)
    new = torch.where(finished, 0, new)
    blocks = -(-lens // BLOCK)
    perm = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(MB, device="cuda")[None, :]
    first = (torch.cumsum(blocks, 0) - blocks)[:, None]
    tables = torch.where(at < blocks[:, None], perm[(first + at).clamp(max=NB - 1)], -1)
    used = blocks.sum()
    free = torch.roll(perm, -int(used))                   # the free ids, then the used ones
    T = B * case["most_new"] + 3                          # the padded width of the step
    i32 = dict(dtype=torch.int32, device="cuda")
    return {"case": case, "tables": tables.to(torch.int32).contiguous(),
            "lens": lens.to(torch.int32), "new": new.to(torch.int32),
            "finished": finished.to(torch.int32), "free": free.contiguous(),
            "count": (NB - used).reshape(1).to(torch.int32),
            "lens_mid": torch.zeros(B, **i32), "lens_out": torch.zeros(B, **i32),
            "count_mid": torch.zeros(1, **i32), "count_out": torch.zeros(1, **i32),
            "slots": torch.zeros(T, **i32), "starts": torch.zeros(B + 1, **i32),
            "positions": torch.zeros(T, **i32)}


# ------------------------------------------------------------------ plain forms
def _quantise(x):
    """Codes (two to a byte, the even element low) and (scale, zero) pairs of
    x [..., D] in its 16-bit type, one pair per 64 elements."""
    g = x.float().unflatten(-1, (-1, GROUP))
    z = g.amin(-1, keepdim=True)
    s = ((g.amax(-1, keepdim=True) - z) / 15.0).to(x.dtype).float()
    c = torch.where(s > 0, torch.round((g - z) / s).clamp(0, 15), 0.0).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.cat([s, z], -1).to(x.dtype)


def _values(codes, sz):
    """float32 values of packed codes [..., D/2] and pairs [..., D/64, 2]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (-1, GROUP))
    sz = sz.float()
    return (c * sz[..., :1] + sz[..., 1:]).flatten(-2)


def _plain_decode(st):
    q, lens, tables = st["q"], st["lens"], st["tables"].long().clamp(min=0)
    B, Hq, D = q.shape
    kv = st["kc"].shape[1]
    n = tables.shape[1] * BLOCK

    def rows(codes, sz):  # [B, kv, n, D]
        v = _values(codes[tables], sz[tables])
        return v.permute(0, 2, 1, 3, 4).reshape(B, kv, n, D)

    k = rows(st["kc"], st["ks"])
    s = torch.matmul(q.float().view(B, kv, Hq // kv, D), k.transpose(2, 3)) * st["scale"]
    del k
    live = torch.arange(n, device=q.device) < lens[:, None]
    s = s.masked_fill(~live[:, None, None, :], -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p, rows(st["vc"], st["vs"])) / p.sum(-1, keepdim=True)
    return o.view(B, Hq, D).to(q.dtype)


def _write(pool, rows, slots):
    """pool[slot / 16, :, slot % 16] = rows; rows of negative slots are nobody's."""
    live = slots >= 0
    at = slots[live].long()
    pool[at // BLOCK, :, at % BLOCK] = rows[live]


def _plain_append4(st, k):
    v, slots = st["v"], st["slots"]
    read = []
    for x, codes, sz in ((k, st["kc"], st["ks"]), (v, st["vc"], st["vs"])):
        c, p = _quantise(x)
        _write(codes, c, slots)
        _write(sz, p, slots)
        at = slots.long().clamp(min=0)
        val = _values(codes[at // BLOCK, :, at % BLOCK], sz[at // BLOCK, :, at % BLOCK])
        read.append(torch.where((slots >= 0)[:, None, None], val, 0.0).to(x.dtype))
    return read


def _rotate(x, st):
    """x [T, H, D] rotated: products and sums in float32, rounded once."""
    R, half = st["case"]["rotary"], st["case"]["rotary"] // 2
    pos = st["positions"].long()[st["axis"]]               # [half, T]
    col = torch.arange(half, device=x.device)[:, None]
    cos = st["cos_sin"][pos, col].t()[:, None, :]
    sin = st["cos_sin"][pos, half + col].t()[:, None, :]
    f = x.float()
    if st["case"]["interleaved"]:
        a, b = f[..., 0:R:2], f[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, f[..., R:]], -1).to(x.dtype)


def _plain_tables(st):
    tables, lens, free, NB = st["tables"], st["lens"].long(), st["free"], st["free"].shape[0]
    B, MB = tables.shape
    at = torch.arange(MB, device=tables.device)[None, :]
    count = st["count"].long()
    # finished requests push their blocks in request and table order
    back = torch.where(st["finished"] != 0, -(-lens // BLOCK), 0)
    first = (torch.cumsum(back, 0) - back)[:, None]
    dest = torch.where(at < back[:, None], count + first + at, NB)
    ext = torch.cat([free, free[:1]])
    ext = ext.scatter(0, dest.reshape(-1), tables.reshape(-1))
    free = ext[:NB]
    count = count + back.sum()
    lens = torch.where(st["finished"] != 0, 0, lens)
    # the others pop what their new tokens need, in request order
    new = st["new"].long()
    have, want = -(-lens // BLOCK), -(-(lens + new) // BLOCK)
    need = want - have
    first = (torch.cumsum(need, 0) - need)[:, None]
    take = (count - 1 - (first + at - have[:, None])).clamp(0, NB - 1)
    tables = torch.where((at >= have[:, None]) & (at < want[:, None]), free[take], tables)
    starts = torch.cat([torch.zeros_like(count), torch.cumsum(new, 0)])
    t = torch.arange(st["slots"].shape[0], device=tables.device)
    b = torch.searchsorted(starts[1:], t, right=True).clamp(max=B - 1)
    live = t < starts[-1]
    pos = torch.where(live, lens[b] + t - starts[b], 0)
    slot = tables[b, pos // BLOCK].long() * BLOCK + pos % BLOCK
    i32 = torch.int32
    return {"tables": tables, "lens": (lens + new).to(i32), "free": free,
            "count": (count - need.sum()).to(i32), "slots": torch.where(live, slot, -1).to(i32),
            "starts": starts.to(i32), "positions": pos.to(i32)}


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    if op == "decode4":
        return _plain_decode(state)
    if op == "tables":
        return _plain_tables(state)
    if op == "append4":
        k, v = _plain_append4(state, state["k"])
        return {"k": k, "v": v}
    live = (state["slots"] >= 0)[:, None, None]
    q = torch.where(live, _rotate(state["q"], state), 0)
    k = _rotate(state["k"], state)
    if op == "rope4":
        k, v = _plain_append4(state, k)
        return {"q": q, "k": k, "v": v}
    _write(state["kc"], k, state["slots"])
    _write(state["vc"], state["v"], state["slots"])
    return {"q": q, "k": state["kc"], "v": state["vc"]}


def _own_decode(st):
    import pagedattention_decode_kvp_gb300 as kvp
    if "workspace" not in st:  # sized once, kept with the batch's buffers
        B, Hq, D = st["q"].shape
        nbytes = kvp.kvp_decode_workspace_bytes(B, Hq, kvp.cache_desc_int4(st["kc"]),
                                                st["tables"].shape[1], kv_int4=True)
        st["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    kvp.kvp_attention_decode_int4(st["out"], st["q"], st["kc"], st["vc"], st["ks"], st["vs"],
                                  st["tables"], st["lens"], st["scale"],
                                  workspace=st["workspace"])
    return st["out"]


def _own_append4(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_append_int4(st["k"], st["v"], st["kc"], st["vc"], st["ks"], st["vs"], st["slots"])
    kvp.kvp_read_int4(st["k_read"], st["v_read"], st["kc"], st["vc"], st["ks"], st["vs"],
                      st["slots"])
    return {"k": st["k_read"], "v": st["v_read"]}


def _own_rope(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_rope_append(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"],
                        st["cos_sin"], st["positions"], st["slots"], sections=st["sections"],
                        interleaved=st["case"]["interleaved"])
    return {"q": st["q_out"], "k": st["kc"], "v": st["vc"]}


def _own_rope4(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_rope_append_int4(st["q_out"], st["q"], st["k"], st["v"], st["kc"], st["vc"],
                             st["ks"], st["vs"], st["cos_sin"], st["positions"], st["slots"],
                             sections=st["sections"], interleaved=st["case"]["interleaved"])
    kvp.kvp_read_int4(st["k_read"], st["v_read"], st["kc"], st["vc"], st["ks"], st["vs"],
                      st["slots"])
    return {"q": st["q_out"], "k": st["k_read"], "v": st["v_read"]}


def _own_tables(st):
    import pagedattention_decode_kvp_gb300 as kvp
    kvp.kvp_release_tables(st["tables"], st["lens"], st["finished"], st["free"], st["count"],
                           st["lens_mid"], st["count_mid"])
    kvp.kvp_extend_tables(st["tables"], st["lens_mid"], st["new"], st["free"], st["count_mid"],
                          st["lens_out"], st["count_out"], st["slots"], st["starts"],
                          st["positions"])
    return {"tables": st["tables"], "lens": st["lens_out"], "free": st["free"],
            "count": st["count_out"], "slots": st["slots"], "starts": st["starts"],
            "positions": st["positions"]}


_OWN = {"decode4": _own_decode, "append4": _own_append4, "rope": _own_rope, "rope4": _own_rope4,
        "tables": _own_tables}


# ------------------------------------------------------------------ 64 bits
def _exact_values(x):
    """What the 4-bit rows of x [T, kv, D] stand for, in 64 bits."""
    T, kv, D = x.shape
    d = x.double().reshape(T, kv, D // GROUP, GROUP)
    low, high = d.min(-1, keepdim=True)[0], d.max(-1, keepdim=True)[0]
    step = ((high - low) / 15).to(x.dtype).double()
    code = torch.round((d - low) / torch.where(step > 0, step, 1.0)).clamp(0, 15)
    return (low + step * code * (step > 0)).reshape(T, kv, D)


def _exact_rotate(x, case, table, positions, sections):
    y = x.double().clone()
    half = case["rotary"] // 2
    first = 0
    for axis, n in enumerate(sections):
        i = torch.arange(first, first + n, device=x.device)
        rows = table[positions[axis].long()].double()
        c, s = rows[:, None, i], rows[:, None, half + i]
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
        a, b = x[..., lo].double(), x[..., hi].double()
        y[..., lo] = a * c - b * s
        y[..., hi] = a * s + b * c
        first += n
    return y


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers: they are equal or wrong
    st = prepare(case, seed)
    if case["op"] == "decode4":
        B, Hq, D = st["q"].shape
        kv = st["kc"].shape[1]
        out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = int(st["lens"][b])
            ids = st["tables"][b, :-(-n // BLOCK)].long()
            rows = []
            for codes, sz in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
                c = codes[ids].transpose(0, 1).reshape(kv, -1, D // 2)[:, :n]
                p = sz[ids].transpose(0, 1).reshape(kv, -1, D // GROUP, 2)[:, :n].double()
                val = torch.empty(kv, n, D, dtype=torch.float64, device="cuda")
                val[..., 0::2], val[..., 1::2] = (c % 16).double(), (c // 16).double()
                rows.append(val * p[..., 0].repeat_interleave(GROUP, -1)
                            + p[..., 1].repeat_interleave(GROUP, -1))
            w = torch.einsum("kgd,knd->kgn", st["q"][b].double().view(kv, Hq // kv, D), rows[0])
            w = torch.softmax(w * st["scale"], -1)
            out[b] = torch.einsum("kgn,knd->kgd", w, rows[1]).reshape(Hq, D)
        return out
    live = (st["slots"] >= 0)[:, None, None]
    if case["op"] == "append4":
        return {"k": _exact_values(st["k"]) * live, "v": _exact_values(st["v"]) * live}
    turn = [_exact_rotate(st[n], case, st["cos_sin"], st["positions"], st["sections"])
            for n in ("q", "k")]
    if case["op"] == "rope4":
        # the codes are of the rotated rows rounded to the cache's 16-bit type
        return {"q": turn[0] * live, "k": _exact_values(turn[1].to(st["k"].dtype)) * live,
                "v": _exact_values(st["v"]) * live}
    pools = []
    for x in (turn[1], st["v"].double()):
        pool = torch.zeros(st["kc"].shape, dtype=torch.float64, device="cuda")
        at = st["slots"][st["slots"] >= 0].long()
        pool[at // BLOCK, :, at % BLOCK] = x[st["slots"] >= 0]
        pools.append(pool)
    return {"q": turn[0] * live, "k": pools[0], "v": pools[1]}


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "tables":
        B, new = case["batch"], case["batch"] * (1 + case["most_new"]) // 2
        T = B * case["most_new"] + 3
        blocks = new // BLOCK + B // 16
        return {"bytes": 4 * (5 * B + 2 * T + 2 * blocks + B // 8 * case["longest"] // BLOCK),
                "flops": 0}
    kv, D = case["kv_heads"], case["dim"]
    row4 = D // 2 + 4 * (D // GROUP)                      # codes and pairs of one row
    if op == "decode4":
        tokens = case["batch"] * (case["shortest"] + case["longest"]) // 2
        return {"bytes": tokens * kv * 2 * row4 + 4 * case["batch"] * case["heads"] * D
                + tokens // BLOCK * 4, "flops": 4 * D * case["heads"] * tokens}
    T = case["tokens"]
    if op == "append4":                                   # read, hold in 4 bits, give back
        return {"bytes": T * kv * 2 * (2 * D + row4 + 2 * D) + 4 * T, "flops": T * kv * 2 * 5 * D}
    turn = 2 * T * case["heads"] * 2 * D + 4 * T * (1 + case["axes"]) \
        + min(T, ROWS) * 4 * case["rotary"]
    flops = T * (case["heads"] + kv) * 3 * case["rotary"]
    if op == "rope":
        return {"bytes": turn + 2 * T * kv * 2 * 2 * D, "flops": flops}
    return {"bytes": turn + T * kv * 2 * (2 * D + row4 + 2 * D), "flops": flops + T * kv * 10 * D}
