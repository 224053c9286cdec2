"""Arguments of the 4-bit cache, rotary append and table entry points that are
refused on the host, before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import plain64
from pagedattention_decode_kvp_gb300 import _build

A = 1 << 20  # an aligned address that is never dereferenced
INVALID, UNSUPPORTED, OK = kvp.KVP_ERR_INVALID_ARG, kvp.KVP_ERR_UNSUPPORTED, kvp.KVP_OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvp.load_library()


def desc(nb=64, kv=2, bs=16, d=128):
    return kvp.kvp_cache_desc(nb, kv, bs, d)


def test_sizing_of_the_4_bit_decode(lib):
    d = desc(40000, 8)
    # the automatic split is balanced: a number of pieces that the heads alone
    # decide, for each kv head two partial states of 8 heads and a 16-byte note
    per = 8 * (2 * 8 * (128 + 2) * 4 + 16)
    n = kvp.kvp_decode_workspace_bytes(4, 64, d, 8192, kv_int4=True)
    assert n % per == 0 and n > 0
    assert n == kvp.kvp_decode_workspace_bytes(64, 64, d, 512, kv_int4=True)
    run = kvp.kvp_decode_partition_blocks(4, 64, d, 8192, kv_int4=True)
    assert run == -(-4 * 8192 // (n // per))
    # given partitions, and tables short enough for a single pass
    assert kvp.kvp_decode_workspace_bytes(4, 64, d, 8192, 512, kv_int4=True) == \
        4 * 64 * 16 * (128 + 2) * 4
    assert kvp.kvp_decode_workspace_bytes(4, 64, d, 64, kv_int4=True) == 0
    assert kvp.kvp_decode_partition_blocks(4, 64, d, 64, kv_int4=True) == 64
    assert kvp.kvp_decode_workspace_bytes(4, 64, d, 65, kv_int4=True) > 0
    for kind in (3, 5, -1):
        assert lib.kvp_decode_workspace_bytes(4, 64, d, 8192, 0, kind) == 0
        assert lib.kvp_decode_partition_blocks(4, 64, d, 8192, kind) == 0


@pytest.mark.parametrize("name", ["kvp_append_int4", "kvp_read_int4"])
def test_append_and_read_int4(lib, name):
    def call(k=A, v=A, dtype=0, kc=A, vc=A, ks=A, vs=A, slots=A, T=1, d=desc()):
        return getattr(lib, name)(k, v, dtype, kc, vc, ks, vs, slots, T, d, None, None)
    assert call(T=0, k=None, kc=None) == OK
    assert call(d=desc(bs=32)) == UNSUPPORTED and call(d=desc(d=96)) == UNSUPPORTED
    assert call(dtype=2) == INVALID and call(T=-1) == INVALID
    for bad in ("k", "v", "kc", "vc", "ks", "vs", "slots"):
        assert call(**{bad: None}) == INVALID, bad
    for bad in ("k", "v", "kc", "vc", "ks", "vs"):
        assert call(**{bad: A + 8}) == INVALID, bad


def test_copy_blocks_int4(lib):
    def call(kc=A, vc=A, ks=A, vs=A, pairs=A, n=1, d=desc()):
        return lib.kvp_copy_blocks_int4(kc, vc, ks, vs, pairs, n, d, None, None)
    assert call(n=0, pairs=None) == OK and call(n=-1) == INVALID
    assert call(d=desc(d=32)) == UNSUPPORTED
    for bad in ("kc", "vc", "ks", "vs", "pairs"):
        assert call(**{bad: None}) == INVALID, bad


def test_decode_int4(lib):
    def call(out=A, q=A, dtype=0, kc=A, ks=A, tables=A, mb=16, lens=A, batch=2, hq=8, scale=0.1,
             d=desc(), pb=0, ws=None, wsb=0, phases=3):
        return lib.kvp_attention_decode_int4(out, q, dtype, kc, A, ks, A, tables, mb, lens, batch,
                                             hq, scale, d, pb, ws, wsb, phases, None, None)
    assert call(batch=0) == OK and call(batch=-1) == INVALID
    assert call(dtype=2) == INVALID and call(hq=7) == INVALID and call(hq=0) == INVALID
    assert call(scale=float("nan")) == INVALID and call(phases=4) == INVALID
    assert call(d=desc(d=80)) == UNSUPPORTED and call(d=desc(bs=8)) == UNSUPPORTED
    assert call(pb=1025) == INVALID and call(pb=-1) == INVALID
    for bad in ("out", "q", "kc", "ks", "tables", "lens"):
        assert call(**{bad: None}) == INVALID, bad
    for bad in ("out", "q", "kc", "ks"):
        assert call(**{bad: A + 4}) == INVALID, bad
    need = lib.kvp_decode_workspace_bytes(2, 8, desc(), 64, 4, 4)
    assert need == 2 * 8 * 16 * 130 * 4
    assert call(mb=64, pb=4) == INVALID                       # no workspace
    assert call(mb=64, pb=4, ws=A, wsb=need - 1) == INVALID   # too small
    assert call(mb=64, pb=4, ws=A + 4, wsb=need) == INVALID   # misaligned
    assert call(batch=65536) == UNSUPPORTED


def rope(R=128, axes=1, sections=(64,), interleaved=0):
    return kvp.kvp_rope_desc(R, axes, (ctypes.c_int32 * 4)(*sections), interleaved)


@pytest.mark.parametrize("int4", [False, True])
def test_rope_append(lib, int4):
    def call(qo=A, qos=1024, q=A, qs=1024, k=A, ks=256, v=A, vs=256, kc=A, vc=A, ksz=A, vsz=A,
             table=A, maxp=100, pos=A, slots=A, T=3, hq=8, r=rope(), d=desc(), dtype=0):
        pools = (kc, vc, ksz, vsz) if int4 else (kc, vc)
        f = lib.kvp_rope_append_int4 if int4 else lib.kvp_rope_append
        return f(qo, qos, q, qs, k, ks, v, vs, *pools, table, maxp, pos, slots, T, hq, r, d, dtype,
                 None, None)
    assert call(T=0, k=None) == OK and call(T=-1) == INVALID and call(dtype=2) == INVALID
    assert call(d=desc(d=96)) == UNSUPPORTED and call(hq=-1) == INVALID
    assert call(maxp=0) == INVALID
    assert call(r=rope(144, 1, (72,))) == INVALID              # wider than the row
    assert call(r=rope(24, 1, (12,))) == UNSUPPORTED           # not a multiple of 16
    assert call(r=rope(0, 1, (0,))) == UNSUPPORTED
    assert call(r=rope(128, 0, ())) == INVALID and call(r=rope(128, 5, (64,))) == INVALID
    assert call(r=rope(128, 2, (64, 1))) == INVALID            # sections past R / 2
    assert call(r=rope(128, 2, (65, -1))) == INVALID
    assert call(r=rope(128, 1, (32, 32))) == INVALID           # the second axis is not counted
    bad = ["qo", "q", "k", "v", "kc", "vc", "table"] + (["ksz", "vsz"] if int4 else [])
    for name in bad + ["pos", "slots"]:
        assert call(**{name: None}) == INVALID, name
    for name in bad:
        assert call(**{name: A + 8}) == INVALID, name
    for name in ("qs", "qos", "ks", "vs"):
        assert call(**{name: 252}) == INVALID, name            # not whole 16-byte pieces
        assert call(**{name: 0}) == INVALID, name              # tokens would overlap
    assert call(hq=65535) == UNSUPPORTED


def test_tables(lib):
    def ext(tables=A, mb=8, lens=A, new=A, B=2, free=A, count=A, nb=50, lo=A, co=A, slots=A, T=4,
            starts=A):
        return lib.kvp_extend_tables(tables, mb, lens, new, B, free, count, nb, lo, co, slots, T,
                                     starts, None, None, None)

    def rel(tables=A, mb=8, lens=A, fin=A, B=2, free=A, count=A, nb=50, lo=A, co=A):
        return lib.kvp_release_tables(tables, mb, lens, fin, B, free, count, nb, lo, co, None,
                                      None)
    for f in (ext, rel):
        assert f(B=-1) == INVALID and f(mb=0) == INVALID and f(nb=0) == INVALID
        assert f(B=16385) == UNSUPPORTED
        assert f(nb=2 ** 31 // 16) == UNSUPPORTED and f(mb=2 ** 31 // 16) == UNSUPPORTED
        for name in ("tables", "lens", "free", "count", "lo", "co"):
            assert f(**{name: None}) == INVALID, name
    assert ext(new=None) == INVALID and rel(fin=None) == INVALID
    assert ext(slots=None) == INVALID and ext(starts=None) == INVALID and ext(T=-1) == INVALID


def test_sizes_past_32_bit_offsets(lib):
    wide = desc(1, 65536)
    for name in ("kvp_append_int4", "kvp_read_int4"):
        assert getattr(lib, name)(A, A, 0, A, A, A, A, A, 1, wide, None, None) == UNSUPPORTED
    assert lib.kvp_extend_tables(A, 8, A, A, 2, A, A, 50, A, A, A, 2 ** 30 + 1, A, None, None,
                                 None) == UNSUPPORTED


@pytest.mark.parametrize("int4", [False, True])
def test_rope_append_onto_q_with_another_stride(lib, int4):
    pools = (A,) * (4 if int4 else 2)
    f = lib.kvp_rope_append_int4 if int4 else lib.kvp_rope_append
    assert f(A, 1024, A, 1032, A, 256, A, 256, *pools, A, 100, A, A, 3, 8, rope(), desc(), 0, None,
             None) == INVALID


def test_a_decode_that_needs_a_workspace_never_reads_as_single_pass(lib):
    """kvp_decode_partition_blocks at or above the table's width means no workspace."""
    for batch in (1, 3, 57, 1000, 65535):
        for mb in (1, 64, 65, 100, 9000):
            for hq, kv in ((8, 8), (64, 8), (1, 1), (1024, 1024)):
                d = desc(1000, kv)
                single = kvp.kvp_decode_partition_blocks(batch, hq, d, mb, kv_int4=True) >= mb
                assert single == (kvp.kvp_decode_workspace_bytes(batch, hq, d, mb,
                                                                 kv_int4=True) == 0)


class Fake:
    """Just enough of a tensor on some GPU for the binding's checks."""

    def __init__(self, device):
        self._d = device

    def get_device(self):
        return self._d


def test_tensors_of_another_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    with pytest.raises(ValueError, match="one call"):
        kvp._on_one_device(None, Fake(0), None, Fake(1))
    with pytest.raises(ValueError, match="current device"):
        kvp._on_one_device(None, Fake(1), Fake(1))
    with pytest.raises(ValueError, match="CUDA tensors"):
        kvp._on_one_device(None, Fake(0), Fake(-1))

    class S:
        device_index, cuda_stream = 1, 5
    with pytest.raises(ValueError, match="stream"):
        kvp._on_one_device(S, Fake(0))
    S.device_index = 0
    assert kvp._on_one_device(S, Fake(0)) == 5


def test_shapes_types_and_strides_are_refused(monkeypatch):
    """On the CPU the first refusal is the device; past it, the rest."""
    monkeypatch.setattr(kvp, "_on_one_device", lambda stream, *ts: 0)
    f16, u8, i32 = torch.float16, torch.uint8, torch.int32
    kc = torch.zeros(4, 2, 16, 64, dtype=u8)
    ks = torch.zeros(4, 2, 16, 2, 2, dtype=f16)
    x = torch.zeros(3, 2, 128, dtype=f16)
    slots = torch.zeros(3, dtype=i32)
    for f in (kvp.kvp_append_int4, kvp.kvp_read_int4):
        with pytest.raises(TypeError):
            f(x.float(), x, kc, kc, ks, ks, slots)
        with pytest.raises(TypeError):
            f(x.bfloat16(), x, kc, kc, ks, ks, slots)
        with pytest.raises(TypeError):
            f(x, x, kc.to(torch.int8), kc, ks, ks, slots)
        with pytest.raises(TypeError):
            f(x, x, kc, kc, ks, ks, slots.long())
        with pytest.raises(ValueError):
            f(x[:2], x, kc, kc, ks, ks, slots)
        with pytest.raises(ValueError):
            f(x, x, kc, kc[:3], ks, ks, slots)
        with pytest.raises(ValueError):
            f(x, x, kc, kc, ks[..., :1, :], ks, slots)
        with pytest.raises(ValueError):
            f(x.transpose(0, 1), x, kc, kc, ks, ks, slots)
    q = torch.zeros(2, 4, 128, dtype=f16)
    tables, lens = torch.zeros(2, 5, dtype=i32), torch.zeros(2, dtype=i32)
    dec = kvp.kvp_attention_decode_int4
    with pytest.raises(ValueError):
        dec(q[:1], q, kc, kc, ks, ks, tables, lens, 1.0)
    with pytest.raises(ValueError):
        dec(q, q, kc, kc, ks, ks, tables[:1], lens, 1.0)
    with pytest.raises(ValueError):
        dec(q, q[..., :64], kc, kc, ks, ks, tables, lens, 1.0)
    with pytest.raises(TypeError):
        dec(q, q, kc, kc, ks, ks, tables, lens.long(), 1.0)
    pool = torch.zeros(4, 2, 16, 128, dtype=f16)
    cs, pos = torch.zeros(9, 128), torch.zeros(3, 3, dtype=i32)
    qq = torch.zeros(3, 4, 128, dtype=f16)
    rope_append = kvp.kvp_rope_append
    with pytest.raises(ValueError, match="sections"):
        rope_append(qq, qq, x, x, pool, pool, cs, pos, slots)
    with pytest.raises(ValueError, match="go together"):
        rope_append(None, qq, x, x, pool, pool, cs, pos[0], slots)
    with pytest.raises(TypeError):
        rope_append(qq, qq, x, x, pool, pool, cs.double(), pos[0], slots)
    with pytest.raises(ValueError):
        rope_append(qq, qq, x, x, pool, pool, cs, pos[:, :2].contiguous(), slots,
                    sections=(16, 24, 24))
    with pytest.raises(ValueError, match="contiguous"):
        rope_append(qq, qq.transpose(1, 2).contiguous().transpose(1, 2), x, x, pool, pool, cs,
                    pos[0], slots)
    free, one, B1 = torch.zeros(9, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError):
        kvp.kvp_extend_tables(tables, lens, lens, free, one, lens, one, slots, lens)
    with pytest.raises(TypeError):
        kvp.kvp_extend_tables(tables, lens, lens, free, one, lens, one, slots.long(), B1)
    with pytest.raises(ValueError):
        kvp.kvp_release_tables(tables, lens, lens[:1], free, one, lens, one)


# ------------------------------------------------------------------ the plain forms
def test_plain_quantiser_and_rotation():
    """The tests' own references, against closed forms."""
    x = torch.arange(64, dtype=torch.float16)[None] / 63 * 15 - 4
    c, p = plain64.quantise4(x)
    assert p[0, 0, 1] == -4 and p[0, 0, 0] == 1 and int(c.min()) == 0 and int(c.max()) == 15
    assert torch.equal(plain64.unpack4(plain64.pack4(c)), c)
    # rotating by two positions one after the other is rotating by their sum
    cs = plain64.angles(32, 64)
    x = torch.randn(1, 1, 64, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    for inter in (False, True):
        a = plain64.rotate(x, cs, [torch.tensor([5])], (32,), inter, torch.float64)
        b = plain64.rotate(a, cs, [torch.tensor([9])], (32,), inter, torch.float64)
        d = plain64.rotate(x, cs, [torch.tensor([14])], (32,), inter, torch.float64)
        assert (b - d).abs().max() < 1e-5
        assert torch.allclose(a.norm(), x.norm(), rtol=1e-6)


def test_plain_tables_by_hand():
    free = [4, 9, 2, 7, 0]
    t, n, top, slots, starts, pos = plain64.extend([[5, -1], [-1, -1]], [15, 0], [2, 1], free, 5, 4)
    assert t == [[5, 0], [7, -1]] and n == [17, 1] and top == 3
    assert slots == [95, 0, 112, -1] and starts == [0, 2, 3] and pos == [15, 16, 0, 0]
    n, free, top = plain64.release(t, n, [1, 0], free, top)
    assert n == [0, 1] and top == 5 and free == [4, 9, 2, 5, 0]


def test_compiled_calls_leave_cpu_tensors_to_the_checks(lib):
    x, z = torch.zeros(2, 2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    kc, ks = torch.zeros(4, 2, 16, 32, dtype=torch.uint8), \
        torch.zeros(4, 2, 16, 1, 2, dtype=torch.float16)
    c = kvp._calls()
    assert c.append_int4(x, x, kc, kc, ks, ks, z, None) is None
    assert c.read_int4() is None and c.extend_tables(z, z) is None and c.release_tables() is None
    assert c.attention_decode_int4(x) is None and c.rope_append(x, x, x, x) is None
    assert c.rope_append_int4(None) is None
    with pytest.raises(ValueError, match="CUDA tensors"):
        kvp.kvp_append_int4(x, x, kc, kc, ks, ks, z)
    with pytest.raises(TypeError, match="status"):
        kvp._status_ptr(z.long())
