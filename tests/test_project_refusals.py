"""Arguments of the norms, E4M3 quantisers and the block-scaled product that are
refused on the host, before anything is launched (no GPU needed)."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
from pagedattention_decode_kvp_gb300 import _build

A = 1 << 20  # an aligned address that is never dereferenced
INVALID, UNSUPPORTED, OK = kvp.KVP_ERR_INVALID_ARG, kvp.KVP_ERR_UNSUPPORTED, kvp.KVP_OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvp.load_library()


@pytest.mark.parametrize("fp8", [False, True])
def test_norm(lib, fp8):
    def call(out=A, os=1024, scales=A, x=A, xs=1024, r=None, rs=0, ro=None, ros=0, w=A, eps=1e-5,
             T=2, H=1, D=1024, dtype=0):
        if fp8:
            return lib.kvp_rms_norm_fp8(out, os, scales, x, xs, r, rs, ro, ros, w, eps, T, D, dtype,
                                        None)
        return lib.kvp_rms_norm(out, os, x, xs, r, rs, ro, ros, w, eps, T, H, D, dtype, None)
    assert call(T=0, out=None, x=None, w=None) == OK
    assert call(T=-1) == INVALID and call(D=0) == INVALID and call(dtype=2) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(eps=float("inf")) == INVALID
    assert call(D=1004) == UNSUPPORTED and call(D=32768 + 16, xs=2 ** 16, os=2 ** 16) == UNSUPPORTED
    for bad in ("out", "x", "w"):
        assert call(**{bad: None}) == INVALID and call(**{bad: A + 8}) == INVALID, bad
    assert call(xs=1023) == INVALID and call(xs=1016) == INVALID and call(xs=1028) == INVALID
    assert call(os=1020) == INVALID and call(os=1008) == INVALID
    assert call(r=A) == INVALID and call(ro=A) == INVALID          # one without the other
    assert call(r=A, rs=1024, ro=A, ros=1000) == INVALID
    assert call(r=A + 8, rs=1024, ro=A, ros=1024) == INVALID
    if fp8:
        assert call(D=1000, T=0) == UNSUPPORTED and call(scales=None) == INVALID
        assert call(scales=A + 2) == INVALID and call(os=1032) == INVALID
    else:
        assert call(H=0) == INVALID and call(H=2) == INVALID       # strides of one head
        assert call(H=2, D=512, r=A, rs=1024, ro=A, ros=1024) == UNSUPPORTED
        assert call(T=1 << 20, H=1 << 11, D=8, xs=1 << 14, os=1 << 14) == UNSUPPORTED
        assert call(T=1, H=1 << 16, D=32768, xs=1 << 31, os=1 << 31) == UNSUPPORTED


def test_quantise(lib):
    def call(c=A, cs=1024, s=A, x=A, xs=1024, R=2, D=1024, block=1, dtype=0):
        return lib.kvp_quantise_fp8(c, cs, s, x, xs, R, D, block, dtype, None)
    assert call(R=0, c=None, x=None, s=None) == OK
    assert call(R=-1) == INVALID and call(D=0) == INVALID and call(dtype=2) == INVALID
    assert call(D=1000) == UNSUPPORTED
    for block in (0, 2, 64, 256, -1):
        assert call(block=block) == UNSUPPORTED
    for bad in ("c", "x"):
        assert call(**{bad: None}) == INVALID and call(**{bad: A + 8}) == INVALID, bad
    assert call(s=None) == INVALID and call(s=A + 2) == INVALID
    assert call(cs=1000) == INVALID and call(cs=1032) == INVALID and call(xs=1020) == INVALID
    assert call(R=1 << 30, D=256, cs=256, xs=256) == UNSUPPORTED
    assert call(R=1, D=2 ** 31 - 16, cs=2 ** 31, xs=2 ** 31) == UNSUPPORTED


def test_matmul(lib):
    def call(o=A, os=256, dt=1, a=A, as_=512, sa=A, b=A, bs=512, sb=A, M=3, N=256, K=512):
        return lib.kvp_matmul_fp8(o, os, dt, a, as_, sa, b, bs, sb, M, N, K, None, None)
    assert call(M=0, o=None, a=None) == OK
    assert call(M=-1) == INVALID and call(N=0) == INVALID and call(K=0) == INVALID
    assert call(dt=3) == INVALID and call(dt=-1) == INVALID
    assert call(K=500) == UNSUPPORTED and call(K=520) == UNSUPPORTED
    for bad in ("o", "a", "sa", "b", "sb"):
        assert call(**{bad: None}) == INVALID, bad
    for bad in ("a", "b"):
        assert call(**{bad: A + 8}) == INVALID, bad
    assert call(sa=A + 2) == INVALID and call(sb=A + 2) == INVALID
    assert call(o=A + 1) == INVALID and call(o=A + 2, dt=2) == INVALID
    assert call(os=255) == INVALID and call(as_=496) == INVALID and call(bs=520) == INVALID
    assert call(as_=1 << 40) == UNSUPPORTED and call(bs=1 << 40) == UNSUPPORTED
    assert call(M=2 ** 31 - 1) == UNSUPPORTED and call(N=2 ** 31 - 1, os=2 ** 31) == UNSUPPORTED
    assert call(M=2 ** 31 - 300, N=2 ** 31 - 300, os=2 ** 31) == UNSUPPORTED   # tiles


class Stream:
    device_index = 0
    cuda_stream = 7


@pytest.fixture
def checks(monkeypatch):
    """The binding's checks on tensors without a device; the calls themselves succeed."""
    made = []

    class Library:
        def kvp_status_string(self, status):
            return b"status"

        def __getattr__(self, name):
            return lambda *args: made.append((name, args)) or 0

    monkeypatch.setattr(kvp, "load_library", lambda: Library())
    monkeypatch.setattr(kvp, "_on_one_device", lambda stream, *ts: 7)
    return made


def t(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_binding_of_the_norms(checks):
    x, w, F = t(3, 256), t(256), torch.float32
    codes, scales = t(3, 256, dtype=torch.uint8), t(3, 2, dtype=F)
    norm, norm8 = kvp.kvp_rms_norm, kvp.kvp_rms_norm_fp8
    good = dict(stream=Stream)
    for bad in ((t(3, 128), x, w), (t(3, 256, dtype=F), x, w), (t(3, 256), x, t(128)),
                (x, x, t(256, dtype=torch.bfloat16)), (x.t(), x.t(), w), (t(256, 3).t(), x, w),
                (t(3, 512)[:, ::2], x, w), (x, t(3, 256, dtype=F), w), (t(3, 2, 128), x, w),
                (x, t(3, 2, 128), t(128))):
        with pytest.raises((TypeError, ValueError)):
            norm(*bad, 1e-5, **good)
    for kw in (dict(residual=x), dict(residual_out=x), dict(residual=t(3, 128), residual_out=x),
               dict(residual=x, residual_out=t(3, 256, dtype=F))):
        with pytest.raises((TypeError, ValueError)):
            norm(x, x, w, 1e-5, **kw, **good)
        with pytest.raises((TypeError, ValueError)):
            norm8(codes, scales, x, w, 1e-5, **kw, **good)
    heads = t(3, 4, 64)
    with pytest.raises(ValueError):
        norm(heads, heads, t(64), 1e-5, residual=x, residual_out=x, **good)
    with pytest.raises(ValueError):
        norm(t(3, 4, 128)[..., :64], heads, t(64), 1e-5, **good)
    for bad in ((codes.to(torch.int8), scales, x, w), (codes, t(3, 1, dtype=F), x, w),
                (codes, scales.half(), x, w), (codes[:2], scales, x, w),
                (codes, scales, t(3, 2, 128), t(128))):
        with pytest.raises((TypeError, ValueError)):
            norm8(*bad, 1e-5, **good)
    assert not checks
    norm(heads, t(3, 9, 64)[:, :4], t(64), 1e-5, **good)
    norm8(codes, scales, t(3, 512)[:, 256:], w, 1e-5, residual=x, residual_out=x, **good)
    norm8(codes.view(torch.float8_e4m3fn), scales, x, w, 0, **good)
    (_, n), (_, n8), _ = checks
    assert n[1] == 256 and n[3] == 9 * 64 and n[10:14] == (3, 4, 64, kvp.KVP_F16)
    assert n8[1] == 256 and n8[4] == 512 and n8[6] == 256 and n8[11:14] == (3, 256, kvp.KVP_F16)


def test_binding_of_the_codes(checks):
    F, U = torch.float32, torch.uint8
    x, codes = t(130, 272), t(130, 272, dtype=U)
    for bad in ((codes, t(130, 2, dtype=F), x), (codes, t(2, 3, dtype=F), x),
                (codes[:, :256], t(130, 3, dtype=F), x), (codes, t(130, 3, dtype=F), x.float()),
                (codes.t(), t(130, 3, dtype=F), x)):
        with pytest.raises((TypeError, ValueError)):
            kvp.kvp_quantise_fp8(*bad, stream=Stream)
    with pytest.raises(ValueError):
        kvp.kvp_quantise_fp8(codes, t(130, 3, dtype=F), x, block_rows=64, stream=Stream)
    out, a, sa = t(5, 130), t(5, 272, dtype=U), t(5, 3, dtype=F)
    b, sb = codes, t(2, 3, dtype=F)
    for bad in ((t(5, 129), a, sa, b, sb), (out, a[:, :256], sa, b, sb), (out, a, sa[:, :2], b, sb),
                (out, a, sa.t(), b, sb), (out, a, sa, b, t(130, 3, dtype=F)),
                (out.double(), a, sa, b, sb), (out, a.half(), sa, b, sb), (out, a, sa, b.t(), sb),
                (t(130, 5).t(), a, sa, b, sb), (out, a, sa.half(), b, sb)):
        with pytest.raises((TypeError, ValueError)):
            kvp.kvp_matmul_fp8(*bad, stream=Stream)
    with pytest.raises(TypeError):
        kvp.kvp_matmul_fp8(out, a, sa, b, sb, status=t(1), stream=Stream)
    assert not checks
    kvp.kvp_quantise_fp8(codes, t(2, 3, dtype=F), x, block_rows=128, stream=Stream)
    kvp.kvp_matmul_fp8(t(5, 400, dtype=F)[:, 9:139], t(5, 288, dtype=U)[:, :272], sa,
                       b.view(torch.float8_e4m3fn), sb, stream=Stream)
    (_, q), (_, m) = checks
    assert q[5:9] == (130, 272, 128, kvp.KVP_F16)
    assert m[1:3] == (400, kvp.KVP_F32) and m[4] == 288 and m[9:12] == (5, 130, 272)
    many = 2 ** 32 + 5
    for call in (lambda: kvp.kvp_matmul_fp8(t(many, 16), t(many, 16, dtype=U), t(many, 1, dtype=F),
                                            t(16, 16, dtype=U), t(1, 1, dtype=F), stream=Stream),
                 lambda: kvp.kvp_quantise_fp8(t(many, 16, dtype=U), t(many, 1, dtype=F), t(many, 16),
                                              stream=Stream),
                 lambda: kvp.kvp_rms_norm(t(many, 16), t(many, 16), t(16), 0, stream=Stream)):
        with pytest.raises(kvp.KvpError) as e:
            call()
        assert e.value.status == UNSUPPORTED
    assert len(checks) == 2
