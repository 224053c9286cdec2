"""Plain implementations the GPU tests compare with: loops and library routines
on the CPU, float64 except where a definition fixes float32 (the quantiser and
the rotation).  They share no code with the library."""
import math

import numpy as np
import torch

BLOCK, GROUP = 16, 64


# ------------------------------------------------------------------ 4-bit rows
def quantise4(x):
    """Codes (uint8 [..., D]) and (scale, zero) pairs [..., D/64, 2] of x."""
    g = x.float().unflatten(-1, (-1, GROUP))
    zero = g.amin(-1, keepdim=True)
    scale = ((g.amax(-1, keepdim=True) - zero) / torch.tensor(15.0)).to(x.dtype)
    s = scale.float()
    q = (g - zero) / torch.where(s > 0, s, torch.tensor(1.0))
    code = torch.where(s > 0, torch.round(q).clamp(max=15.0), torch.tensor(0.0))
    return code.to(torch.uint8).flatten(-2), torch.cat([scale, zero.to(x.dtype)], -1)


def pack4(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack4(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def values4(packed, pairs, dtype=torch.float64):
    """code * scale + zero of packed [..., D/2] and pairs [..., D/64, 2]."""
    c = unpack4(packed).to(dtype).unflatten(-1, (-1, GROUP))
    p = pairs.to(dtype)
    return (c * p[..., :1] + p[..., 1:]).flatten(-2)


# ------------------------------------------------------------------ decode
def decode4(q, kc, vc, ks, vs, tables, lens, scale):
    """float64 attention over 4-bit pools, and how far a kernel may be from it.

    The bound adds up, for an output element d of group g with weights w_t:
      * a_t = p_t s_t rounded to fp16, half a step 2^-11, weighted by
        |c - 7.5| <= 7.5 (the codes are centred):    2^-11 sum_t w_t 7.5 s_t;
        weights far below the largest are fp16 subnormals, off by at most 2^-25
        where the largest is at least 8:             n 2^-28 7.5 max_t(w_t s_t);
      * the score in float32: a product chain of at most D / 16 + 8 roundings,
        2^-23 each (a tensor core may truncate), of terms whose magnitudes add up
        to M_t (log2 units); a weight moves by ln 2 of that, and ex2 by 2^-22;
      * the sums over a context in float32, one rounding (2^-23) per 16 tokens
        and 16 for the merges, of terms of magnitude w_t (15 s_t + |z_t|);
      * the output's own rounding, half a step of its type.
    """
    B, Hq, D = q.shape
    kv = kc.shape[1]
    G = Hq // kv
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    tol = torch.zeros(B, Hq, D, dtype=torch.float64)
    half = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        ids = tables[b, :-(-n // BLOCK)].long()

        def rows(pool):  # [kv, n, ...]
            return pool[ids].transpose(0, 1).flatten(1, 2)[:, :n]

        kp, vp = rows(ks).double(), rows(vs).double()
        K, V = values4(rows(kc), kp), values4(rows(vc), vp)
        for h in range(Hq):
            g = h // G
            x = q[b, h].double()
            s = scale * (K[g] @ x)
            w = torch.softmax(s, 0)
            o = w @ V[g]
            # magnitudes
            c = unpack4(rows(kc)[g]).double().unflatten(-1, (-1, GROUP))
            xa = x.abs().unflatten(-1, (-1, GROUP))
            M = ((c * kp[g][..., :1].abs()) * xa).sum((-1, -2)) + \
                (kp[g][..., 1].abs() * xa.sum(-1)).sum(-1)
            dw = (D / 16 + 8) * 2.0 ** -23 * float((scale * M).max()) + 2.0 ** -22
            sv, zv = vp[g][..., 0], vp[g][..., 1]           # [n, groups]
            ws = w[:, None] * sv
            size = (w[:, None] * (15 * sv + zv.abs())).sum(0)
            t = 2.0 ** -11 * 7.5 * ws.sum(0) + n * 2.0 ** -28 * 7.5 * ws.amax(0) + \
                (2 * dw + (n / 16 + 16) * 2.0 ** -23) * size
            out[b, h] = o
            tol[b, h] = t.repeat_interleave(GROUP) * (1 + half) + half * o.abs() + tiny
    return out, tol


# ------------------------------------------------------------------ rotary
def angles(max_position, R):
    inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    a = torch.arange(max_position, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def rotate(x, cos_sin, positions, sections, interleaved, dtype=torch.float32):
    """x [T, H, D] rotated pair by pair; with float32, every product and sum
    rounded by itself (the definition), one rounding to x's type at the end."""
    R = cos_sin.shape[1]
    y = x.to(dtype).clone()
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    assert len(axis) == R // 2
    for i, a in enumerate(axis):
        row = cos_sin[positions[a].long()].to(dtype)
        c, s = row[:, i, None], row[:, R // 2 + i, None]
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        p, q = x[..., lo].to(dtype), x[..., hi].to(dtype)
        y[..., lo] = p * c - q * s
        y[..., hi] = q * c + p * s
    return y if dtype == torch.float64 else y.to(x.dtype)


def scatter(pool, rows, slots):
    """A copy of pool [NB, H, 16, ...] with rows [T, H, ...] at their slots."""
    pool = pool.clone()
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            pool[s // BLOCK, :, s % BLOCK] = rows[t]
    return pool


# ------------------------------------------------------------------ tables
def extend(tables, lens, new, free, count, num_tokens):
    """(tables, lens, count, slots, starts, positions) after one step's growth."""
    tables = [list(r) for r in tables]
    top, slots, positions, starts, after = count, [], [], [0], []
    for b, (n, k) in enumerate(zip(lens, new)):
        for i in range(-(-n // BLOCK), -(-(n + k) // BLOCK)):
            top -= 1
            tables[b][i] = free[top]
        for pos in range(n, n + k):
            slots.append(tables[b][pos // BLOCK] * BLOCK + pos % BLOCK)
            positions.append(pos)
        starts.append(starts[-1] + k)
        after.append(n + k)
    pad = num_tokens - len(slots)
    return tables, after, top, slots + [-1] * pad, starts, positions + [0] * pad


def release(tables, lens, finished, free, count):
    """(lens, free, count) after the finished requests' blocks came back."""
    free, after = list(free), []
    for b, n in enumerate(lens):
        if finished[b]:
            for i in range(-(-n // BLOCK)):
                free[count] = tables[b][i]
                count += 1
        after.append(0 if finished[b] else n)
    return after, free, count
