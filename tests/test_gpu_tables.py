"""Block tables and slot maps made on the GPU, against loops on the host; and a
serving loop of them with the 4-bit rotary append and decode, captured."""
import math
import random

import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import plain64
from test_gpu_int4 import DTYPES, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Plan:
    """A pool of NB blocks, B requests holding `lens` tokens, MB table entries."""

    def __init__(self, lens, MB, NB, seed=0):
        rnd = random.Random(seed)
        ids = list(range(NB))
        rnd.shuffle(ids)
        self.lens, self.MB, self.NB = list(lens), MB, NB
        self.tables = []
        for n in lens:
            k = -(-n // 16)
            self.tables.append([ids.pop() for _ in range(k)] + [-1] * (MB - k))
        self.count = len(ids)
        self.free = ids + [-7] * (NB - len(ids))

    def gpu(self, T):
        B = len(self.lens)
        self.T = T
        self.g = dict(tables=i32(self.tables).view(B, self.MB), lens=i32(self.lens),
                      free=i32(self.free), count=i32([self.count]),
                      lens_out=torch.full((B,), -9, dtype=torch.int32, device="cuda"),
                      count_out=i32([-9]), slots=torch.full((T,), -9, dtype=torch.int32,
                                                            device="cuda"),
                      starts=torch.full((B + 1,), -9, dtype=torch.int32, device="cuda"),
                      pos=torch.full((T,), -9, dtype=torch.int32, device="cuda"),
                      status=i32([0]))
        return self.g

    def extend(self, new, in_place=False, positions=True):
        g = self.g
        lo, co = (g["lens"], g["count"]) if in_place else (g["lens_out"], g["count_out"])
        kvp.kvp_extend_tables(g["tables"], g["lens"], i32(new), g["free"], g["count"], lo, co,
                              g["slots"], g["starts"], g["pos"] if positions else None,
                              status=g["status"])
        return lo, co

    def release(self, finished, in_place=False):
        g = self.g
        lo, co = (g["lens"], g["count"]) if in_place else (g["lens_out"], g["count_out"])
        kvp.kvp_release_tables(g["tables"], g["lens"], i32(finished), g["free"], g["count"], lo,
                               co, status=g["status"])
        return lo, co


SIZES = [(1, 40, 1), (3, 100, 17), (64, 500, 1), (64, 300, 200), (1000, 64, 3), (1025, 50, 40),
         (16384, 20, 2)]


@pytest.mark.parametrize("B,longest,most", SIZES)
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_and_release(B, longest, most, in_place):
    rnd = random.Random(B + most)
    lens = [rnd.choice([0, 16, longest, rnd.randint(0, longest)]) for _ in range(B)]
    new = [rnd.choice([0, 1, most, rnd.randint(0, most)]) for _ in range(B)]
    MB = -(-(longest + most) // 16)
    NB = sum(-(-(n + k) // 16) for n, k in zip(lens, new)) + 2
    p = Plan(lens, MB, NB, seed=B)
    T = sum(new) + 5
    g = p.gpu(T)
    lo, co = p.extend(new, in_place)
    want = plain64.extend(p.tables, p.lens, new, p.free, p.count, T)
    assert kvp.kvp_read_status(g["status"]) == kvp.KVP_OK
    got = (g["tables"].tolist(), lo.tolist(), int(co), g["slots"].tolist(), g["starts"].tolist(),
           g["pos"].tolist())
    for a, b in zip(got, want):
        assert a == b
    assert g["free"].tolist() == p.free
    # every block is held once: by a table or by the stack
    held = [i for t, n in zip(got[0], got[1]) for i in t[:-(-n // 16)]]
    assert sorted(held + p.free[:got[2]]) == list(range(NB))
    # some requests end
    done = [rnd.choice([0, 0, 1, 7]) for _ in range(B)]
    p.tables, p.lens, p.count = got[0], got[1], got[2]
    g = p.gpu(T)
    lo, co = p.release(done, in_place)
    want = plain64.release(p.tables, p.lens, done, p.free, p.count)
    assert kvp.kvp_read_status(g["status"]) == kvp.KVP_OK
    assert (lo.tolist(), g["free"].tolist(), int(co)) == want
    assert g["tables"].tolist() == p.tables


def test_extend_a_prompt_across_clusters():
    """Enough tokens for every CTA of the largest cluster, one request's tokens
    spread over all of them."""
    lens, new = [5, 0, 33], [0, 40001, 1]
    p = Plan(lens, 2600, 2600)
    g = p.gpu(40010)
    lo, co = p.extend(new)
    want = plain64.extend(p.tables, lens, new, p.free, p.count, 40010)
    assert (g["tables"].tolist(), lo.tolist(), int(co), g["slots"].tolist(),
            g["starts"].tolist(), g["pos"].tolist()) == want


@pytest.mark.parametrize("B", [3, 700, 5000])
def test_extend_many_tokens(B):
    """More tokens than the planning launch lists itself: requests without new
    tokens between the others, a request longer than a CTA's share, padding
    behind."""
    rnd = random.Random(B)
    lens = [rnd.randint(0, 40) for _ in range(B)]
    new = [rnd.choice([0, 0, 0, 1, 5, 30000 // B]) for _ in range(B)]
    new[B // 2] = 4000
    T = max(sum(new), 16385) + 1500
    MB = -(-(max(new) + 40) // 16)
    p = Plan(lens, MB, sum(-(-(n + k) // 16) for n, k in zip(lens, new)) + 3, seed=B)
    g = p.gpu(T)
    lo, co = p.extend(new)
    want = plain64.extend(p.tables, lens, new, p.free, p.count, T)
    assert kvp.kvp_read_status(g["status"]) == kvp.KVP_OK
    got = (g["tables"].tolist(), lo.tolist(), int(co), g["slots"].tolist(), g["starts"].tolist(),
           g["pos"].tolist())
    for a, b in zip(got, want):
        assert a == b
    # and nothing of it when a block is missing
    p.count = 0
    g = p.gpu(T)
    lo, co = p.extend(new, in_place=True)
    assert kvp.kvp_read_status(g["status"]) == kvp.KVP_ERR_OOM
    assert lo.tolist() == lens and (g["slots"] == -1).all() and (g["pos"] == 0).all()
    assert (g["starts"] == 0).all() and g["tables"].tolist() == p.tables


def test_extend_long_runs_of_requests_without_new_tokens():
    """A CTA's first and last request lie further apart than it has tokens."""
    B, T = 12000, 17000
    lens, new = [3] * B, [0] * B
    new[1], new[B - 2], new[B - 1] = 700, 700, 15500
    p = Plan(lens, 1000, B + 1100)
    g = p.gpu(T)
    lo, co = p.extend(new)
    want = plain64.extend(p.tables, lens, new, p.free, p.count, T)
    assert g["slots"].tolist() == want[3] and g["pos"].tolist() == want[5]
    assert g["starts"].tolist() == want[4] and lo.tolist() == want[1]


def test_extend_without_positions_or_tokens_or_requests():
    p = Plan([16, 3], 4, 9)
    g = p.gpu(4)
    p.extend([1, 1], positions=False)
    assert (g["pos"] == -9).all() and g["starts"].tolist() == [0, 1, 2]
    p = Plan([16, 3], 4, 9)
    g = p.gpu(0)
    lo, co = p.extend([0, 0])
    assert lo.tolist() == [16, 3] and int(co) == p.count and g["starts"].tolist() == [0, 0, 0]
    p = Plan([], 4, 9)
    g = p.gpu(2)
    lo, co = p.extend([])
    assert int(co) == 9 and g["starts"].tolist() == [0] and g["slots"].tolist() == [-1, -1]
    lo, co = p.release([])
    assert int(co) == 9 and kvp.kvp_read_status(g["status"]) == kvp.KVP_OK


def damage(what, p, new):
    if what == "too few blocks":
        p.count = 1
    elif what == "past the table":
        new[1] = 16 * p.MB - p.lens[1] + 1
    elif what == "negative length":
        p.lens[0] = -1
    elif what == "negative growth":
        new[2] = -1
    elif what == "too many tokens":
        new[0] += 60
    elif what == "stack height":
        p.count = p.NB + 1
    elif what == "negative height":
        p.count = -1
    elif what == "free id":
        p.free[p.count - 2] = p.NB
    elif what == "partly filled block":
        p.tables[0][0] = -1
    return p, new


@pytest.mark.parametrize("what", ["too few blocks", "past the table", "negative length",
                                  "negative growth", "too many tokens", "stack height",
                                  "negative height", "free id", "partly filled block"])
@pytest.mark.parametrize("in_place", [False, True])
def test_extend_is_all_or_nothing(what, in_place):
    p, new = damage(what, Plan([10, 40, 32], 8, 30), [3, 20, 17])
    g = p.gpu(60)
    lo, co = p.extend(new, in_place)
    want = kvp.KVP_ERR_OOM if what == "too few blocks" else kvp.KVP_ERR_BAD_BLOCK
    assert kvp.kvp_read_status(g["status"]) == want
    assert g["tables"].tolist() == p.tables and g["free"].tolist() == p.free
    assert lo.tolist() == p.lens and int(co) == p.count
    assert g["slots"].tolist() == [-1] * 60 and g["starts"].tolist() == [0] * 4
    assert g["pos"].tolist() == [0] * 60


@pytest.mark.parametrize("what,code", [("full", kvp.KVP_ERR_REFCOUNT), ("id", kvp.KVP_ERR_BAD_BLOCK),
                                       ("length", kvp.KVP_ERR_BAD_BLOCK),
                                       ("height", kvp.KVP_ERR_BAD_BLOCK)])
def test_release_is_all_or_nothing(what, code):
    p = Plan([10, 40, 32], 8, 30)
    if what == "full":
        p.count = 28
    elif what == "id":
        p.tables[1][2] = 30
    elif what == "length":
        p.lens[0] = 16 * 8 + 1
    else:
        p.count = -2
    g = p.gpu(1)
    lo, co = p.release([0, 1, 1])
    assert kvp.kvp_read_status(g["status"]) == code
    assert lo.tolist() == p.lens and int(co) == p.count and g["free"].tolist() == p.free


def test_a_table_entry_past_the_requests_blocks_is_never_read():
    p = Plan([16, 32], 6, 20)
    p.tables[0][1:] = [10 ** 9] * 5
    g = p.gpu(3)
    lo, _ = p.extend([1, 1])
    assert kvp.kvp_read_status(g["status"]) == kvp.KVP_OK and lo.tolist() == [17, 33]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("D,R,sections", [(128, 128, (16, 24, 24)), (64, 32, (16,))])
def test_serving_loop_in_a_graph(dtype, D, R, sections):
    """Plan, rotate and append, attend: one captured step, replayed with other
    lengths each time (requests start, grow by one or several tokens, end and
    give their blocks to others), against 64 bits.  The last new token of each
    request is its query."""
    B, MB, NB, T, Hq, kv, A = 5, 12, 40, 90, 8, 2, len(sections)
    f = dict(dtype=dtype, device="cuda")
    z = dict(dtype=torch.int32, device="cuda")
    tables, lens, count = torch.full((B, MB), -1, **z), torch.zeros(B, **z), i32([NB])
    free = torch.randperm(NB, generator=gen(1)).to(torch.int32).cuda()
    new, done = torch.zeros(B, **z), torch.zeros(B, **z)
    slots, starts, pos = torch.zeros(T, **z), torch.zeros(B + 1, **z), torch.zeros(T, **z)
    status = i32([0])
    qkv = torch.zeros((T, (Hq + 2 * kv), D), **f)
    turned, q, out = torch.zeros((T, Hq, D), **f), torch.zeros((B, Hq, D), **f), \
        torch.zeros((B, Hq, D), **f)
    kc = torch.randint(0, 256, (NB, kv, 16, D // 2), dtype=torch.uint8).cuda()
    vc = kc.clone()
    ks = torch.full((NB, kv, 16, D // 64, 2), float("nan"), **f)
    vs = ks.clone()
    cs = plain64.angles(256, R).cuda()
    scale = 1.0 / math.sqrt(D)
    nbytes = kvp.kvp_decode_workspace_bytes(B, Hq, kvp.cache_desc_int4(kc), MB, 2, kv_int4=True)
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda")

    def step():
        kvp.kvp_release_tables(tables, lens, done, free, count, lens, count, status=status)
        kvp.kvp_extend_tables(tables, lens, new, free, count, lens, count, slots, starts, pos,
                              status=status)
        axes = pos.expand(A, T).contiguous()
        kvp.kvp_rope_append_int4(turned, qkv[:, :Hq], qkv[:, Hq:Hq + kv], qkv[:, Hq + kv:], kc, vc,
                                 ks, vs, cs, axes, slots, sections=sections, status=status)
        q.copy_(turned[(starts[1:] - 1).clamp(min=0).long()])
        kvp.kvp_attention_decode_int4(out, q, kc, vc, ks, vs, tables, lens, scale, workspace=ws,
                                      partition_blocks=2, status=status)

    step()  # nothing to do yet
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rnd = random.Random(3)
    h_lens, h_tables, h_free, h_count = [0] * B, tables.tolist(), free.tolist(), NB
    hk = [torch.zeros(0, kv, D, dtype=dtype) for _ in range(B)]
    hv = list(hk)
    for it in range(12):
        fin = [int(n > 0 and rnd.random() < 0.25) for n in h_lens]
        grow = [0 if fin[b] else rnd.randint(1, 25) if h_lens[b] == 0 else rnd.randint(0, 4)
                for b in range(B)]
        grow = [min(k, 16 * MB - n) for k, n in zip(grow, h_lens)]
        x = randn((T, Hq + 2 * kv, D), dtype, 100 + it)
        new.copy_(i32(grow))
        done.copy_(i32(fin))
        qkv.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert kvp.kvp_read_status(status) == kvp.KVP_OK
        h_lens, h_free, h_count = plain64.release(h_tables, h_lens, fin, h_free, h_count)
        before = list(h_lens)
        h_tables, h_lens, h_count, h_slots, h_starts, h_pos = \
            plain64.extend(h_tables, h_lens, grow, h_free, h_count, T)
        assert tables.tolist() == h_tables and lens.tolist() == h_lens
        assert slots.tolist() == h_slots and starts.tolist() == h_starts
        assert free.tolist() == h_free and int(count) == h_count
        p = torch.tensor(h_pos)[None].expand(A, T)
        turn = plain64.rotate(x[:, :Hq + kv], cs.cpu(), p, sections, False)
        live = [b for b in range(B) if grow[b] > 0]
        for b in range(B):
            if before[b] == 0:
                hk[b], hv[b] = hk[b][:0], hv[b][:0]
            a, e = h_starts[b], h_starts[b + 1]
            hk[b] = torch.cat([hk[b], turn[a:e, Hq:]])
            hv[b] = torch.cat([hv[b], x[a:e, Hq + kv:]])
        ck, cv = kc.cpu().clone(), vc.cpu().clone()
        pk, pv = ks.cpu().clone(), vs.cpu().clone()
        for b in range(B):  # the pools hold what was appended
            ids = torch.tensor(h_tables[b])[torch.arange(h_lens[b]) // 16]
            off = torch.arange(h_lens[b]) % 16
            for rows, codes, pairs in ((hk[b], ck, pk), (hv[b], cv, pv)):
                c, s = plain64.quantise4(rows)
                assert torch.equal(codes[ids, :, off], plain64.pack4(c))
                assert torch.equal(pairs[ids, :, off], s)
        want_q = torch.stack([turn[max(h_starts[b + 1] - 1, 0), :Hq] for b in range(B)])
        assert torch.equal(q.cpu()[live], want_q[live])
        ref, tol = plain64.decode4(want_q, ck, cv, pk, pv, torch.tensor(h_tables),
                                   torch.tensor(h_lens), scale)
        for b in live:
            assert ((out[b].cpu().double() - ref[b]).abs() <= tol[b]).all()
