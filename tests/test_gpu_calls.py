"""The compiled way into the short entry points: it makes the calls that are in
order, and leaves every other to the checks in Python."""
import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
import plain64
from test_gpu_int4 import DTYPES, bits, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from pagedattention_decode_kvp_gb300 import _build
    _build.build()
    kvp.load_library()


def arguments(dtype, D=64):
    """Arguments of every entry point, in the order of the compiled functions."""
    NB, kv, Hq, T, B, MB = 6, 2, 4, 5, 3, 2
    f, z = dict(dtype=dtype, device="cuda"), dict(dtype=torch.int32, device="cuda")
    pools = [torch.zeros((NB, kv, 16, D // 2), dtype=torch.uint8, device="cuda") for _ in "kv"] + \
        [torch.zeros((NB, kv, 16, D // 64, 2), **f) for _ in "kv"]
    k, v = randn((T, kv, D), dtype, 1).cuda(), randn((T, kv, D), dtype, 2).cuda()
    qkv = randn((T, Hq + 2 * kv, D), dtype, 3).cuda()
    slots = torch.tensor([0, 17, -1, 33, 95], **z)
    tables, lens = torch.tensor([[0, 1], [2, 3], [4, 5]], **z), torch.tensor([0, 20, 32], **z)
    pool16 = [torch.zeros((NB, kv, 16, D), **f) for _ in "kv"]
    cs, pos = plain64.angles(64, D).cuda(), torch.arange(2 * T, **z).view(2, T)
    rope = [torch.zeros((T, Hq, D), **f), qkv[:, :Hq], qkv[:, Hq:Hq + kv], qkv[:, Hq + kv:]]
    place = [cs, pos, slots, (D // 4, D // 4), False]
    status = torch.zeros(1, **z)
    free, count = torch.arange(9, **z), torch.tensor([9], **z)
    lens_out, count_out = torch.zeros(B, **z), torch.zeros(1, **z)
    plan = [tables.clone(), lens, torch.tensor([1, 2, 0], **z), free, count, lens_out, count_out]
    return {
        "append_int4": [k, v, *pools, slots, status],
        "read_int4": [k.clone(), v.clone(), *pools, slots, status],
        "attention_decode_int4": [torch.zeros((B, Hq, D), **f), qkv[:B, :Hq].contiguous(), *pools,
                                  tables, lens, 0.125, None, 0, 3, status],
        "rope_append": [*rope, *pool16, *place, status],
        "rope_append_int4": [*rope, *pools, *place, status],
        "extend_tables": [*plan, torch.zeros(8, **z), torch.zeros(B + 1, **z),
                          torch.zeros(8, **z), status],
        "release_tables": [*plan[:4], torch.tensor([5], **z), *plan[5:], status],
    }


NAMES = ["append_int4", "read_int4", "attention_decode_int4", "rope_append", "rope_append_int4",
         "extend_tables", "release_tables"]


def by_python(name, args):
    """The same call by the public function on an explicit stream, which takes the
    way through Python."""
    args, kw = list(args), dict(status=args[-1], stream=torch.cuda.current_stream())
    del args[-1]
    if name.startswith("rope"):
        kw.update(sections=args[-2], interleaved=args[-1])
        del args[-2:]
    if name == "attention_decode_int4":
        kw.update(workspace=args[-3], partition_blocks=args[-2], phases=args[-1])
        del args[-3:]
    getattr(kvp, {"attention_decode_int4": "kvp_attention_decode_int4"}.get(
        name, "kvp_" + name))(*args, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", NAMES)
def test_both_ways_give_the_same(name, dtype):
    a, b = arguments(dtype)[name], arguments(dtype)[name]
    assert getattr(kvp._calls(), name)(*a) == kvp.KVP_OK
    by_python(name, b)
    torch.cuda.synchronize()
    assert int(a[-1]) == kvp.KVP_OK
    for x, y in zip(a, b):
        if isinstance(x, torch.Tensor):
            assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("name", NAMES)
def test_what_is_not_in_order_is_left_alone(name):
    """Every tensor in turn of another type, on the CPU, one row short, not
    contiguous, or something else altogether: not called, and nothing written."""
    call = getattr(kvp._calls(), name)
    good = arguments(torch.float16)[name]
    before = [x.clone() if isinstance(x, torch.Tensor) else x for x in good]
    rows = {"rope_append": 4, "rope_append_int4": 4}.get(name, 0)  # may be strided over tokens
    for i, x in enumerate(good):
        if not isinstance(x, torch.Tensor):
            continue
        wide = torch.zeros((*x.shape[:-1], 2 * x.shape[-1]), dtype=x.dtype, device="cuda")
        bad = [x.double(), x.cpu(), "x", 3, wide[..., ::2]]
        if x is not good[-1]:
            bad += [x[:-1], x[None], None if not (name == "extend_tables" and i == 9) else 0]
        if i >= rows and x.dim() > 1:
            bad.append(x.transpose(0, 1).contiguous().transpose(0, 1))
        for y in bad:
            if isinstance(y, torch.Tensor) and y.shape == x.shape and y.dtype == x.dtype and \
                    y.is_cuda and y.is_contiguous():
                continue
            # (a free stack, and a table of angles, may have any length)
            any_length = i == 3 if "tables" in name else name.startswith("rope") and x is good[-6]
            if any_length and isinstance(y, torch.Tensor) and y.shape == x[:-1].shape:
                continue
            assert call(*good[:i], y, *good[i + 1:]) is None, (i, getattr(y, "shape", y))
    torch.cuda.synchronize()
    for x, y in zip(good, before):
        if isinstance(x, torch.Tensor):
            assert torch.equal(bits(x), bits(y))


def test_numbers_and_sections_out_of_order():
    good = arguments(torch.float16)
    call, a = kvp._calls().attention_decode_int4, good["attention_decode_int4"]
    for i, bads in ((8, ["1", None]), (10, [1.5, 2 ** 40, None]), (11, [None, "3"])):
        for bad in bads:
            assert call(*a[:i], bad, *a[i + 1:]) is None
    assert call(*a[:11], 4, a[12]) == kvp.KVP_ERR_INVALID_ARG  # the library's own refusals
    with pytest.raises(kvp.KvpError):
        kvp.kvp_attention_decode_int4(*a[:9], phases=4)
    call, a = kvp._calls().rope_append, good["rope_append"]
    for bad in ((), (4,) * 5, (16, 16.0), "ab", 16, (2 ** 40, 0), (32,)):
        assert call(*a[:9], bad, *a[10:]) is None
    assert call(*a[:10], 1, a[11]) is None
    assert call(*a[:9], [16, 16], *a[10:]) == kvp.KVP_OK
    assert call(*a[:9], (16, 15), *a[10:]) == kvp.KVP_ERR_INVALID_ARG


def test_empty_calls():
    z = dict(dtype=torch.int32, device="cuda")
    pools = arguments(torch.float16)["append_int4"][2:6]
    none = torch.zeros((0, 2, 64), dtype=torch.float16, device="cuda")
    e = torch.zeros(0, **z)
    assert kvp._calls().append_int4(none, none, *pools, e, None) == kvp.KVP_OK
    q = torch.zeros((0, 4, 64), dtype=torch.float16, device="cuda")
    assert kvp._calls().attention_decode_int4(q, q, *pools, torch.zeros((0, 3), **z), e, 1.0, None,
                                              0, 3, None) == kvp.KVP_OK


def test_a_tensor_without_data_is_an_error():
    """An exception on the way to the library leaves the interpreter as it was."""
    fake = pytest.importorskip("torch._subclasses.fake_tensor")
    with fake.FakeTensorMode():
        x = torch.empty((2, 2, 64), dtype=torch.float16, device="cuda")
        kc = torch.empty((4, 2, 16, 32), dtype=torch.uint8, device="cuda")
        ks = torch.empty((4, 2, 16, 1, 2), dtype=torch.float16, device="cuda")
        slots = torch.empty(2, dtype=torch.int32, device="cuda")
    for _ in range(3):
        with pytest.raises(Exception):
            kvp.kvp_append_int4(x, x, kc, kc, ks, ks, slots)
    assert sum(range(10)) == 45


def test_two_threads_on_two_streams():
    from threading import Thread
    calls = [arguments(torch.float16) for _ in range(2)]
    want = [arguments(torch.float16) for _ in range(2)]
    for a in want:
        kvp._calls().rope_append_int4(*a["rope_append_int4"])
        kvp._calls().append_int4(*a["append_int4"])
    torch.cuda.synchronize()
    errors = []

    def work(a):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(200):
                    r = a["rope_append_int4"]
                    kvp.kvp_rope_append_int4(*r[:11], sections=r[11], interleaved=r[12],
                                             status=r[13])
                    k = a["append_int4"]
                    kvp.kvp_append_int4(*k[:7], status=k[7])
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [Thread(target=work, args=(a,)) for a in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for a, b in zip(calls, want):
        for name in ("rope_append_int4", "append_int4"):
            for x, y in zip(a[name], b[name]):
                if isinstance(x, torch.Tensor):
                    assert torch.equal(bits(x), bits(y))
