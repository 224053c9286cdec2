"""The Python binding and its build, without a GPU."""
import os

import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp
from pagedattention_decode_kvp_gb300 import _build


class Recorder:
    """A library whose calls are recorded and succeed."""

    def __init__(self):
        self.calls = []

    def kvp_status_string(self, status):
        return b"status"

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


class Stream:
    cuda_stream = 7


def test_read_status_takes_any_tensor(monkeypatch):
    """Whatever an earlier entry point takes as `status` can be read back: the first
    word of any tensor."""
    lib = Recorder()
    monkeypatch.setattr(kvp, "load_library", lambda: lib)
    for dtype in (torch.int32, torch.int64, torch.uint8):
        status = torch.zeros(8, dtype=dtype)
        assert kvp.kvp_read_status(status, Stream) == 0
        assert lib.calls[-1] == ("kvp_read_status", (status.data_ptr(), 7))
    kvp.kvp_read_status(torch.zeros(0, dtype=torch.int32), Stream)
    assert lib.calls[-1][1][0] == 0  # (no word: the library refuses it)
    monkeypatch.setattr(kvp, "_need_cuda", lambda *ts: None)
    status = torch.zeros(1, dtype=torch.int64)
    kvp.kvp_selftest_wait_timeout(status, 100, Stream)
    assert lib.calls[-1] == ("kvp_selftest_wait_timeout", (status.data_ptr(), 100, 7))


class Toolchain:
    """The build in an empty directory, with compilers that only leave a file."""

    def __init__(self, monkeypatch, tmp_path):
        self.compiled, self.linked, self.broken = [], [], ()
        for name, path in (("BUILD_DIR", "build"), ("LIB_DIR", "lib"), ("LIB_PATH", "lib/libkvp.so"),
                           ("CALLS_PATH", "lib/_kvp_calls.so"),
                           ("CALLS_KEY_PATH", "lib/_kvp_calls.key")):
            monkeypatch.setattr(_build, name, str(tmp_path / path))
        monkeypatch.setattr(_build.subprocess, "run", self.run)

    def run(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        (self.compiled if "-c" in cmd else self.linked).append(os.path.basename(out).split(".tmp")[0])
        failed = any(os.path.basename(out).startswith(b) for b in self.broken)
        if not failed:
            open(out, "w").close()
        return _build.subprocess.CompletedProcess(cmd, int(failed), "", "broken" * failed)


@pytest.fixture
def toolchain(monkeypatch, tmp_path):
    return Toolchain(monkeypatch, tmp_path)


def test_the_library_builds_without_torch(toolchain, monkeypatch):
    """A C caller needs nvcc and nothing else."""
    find = _build.importlib.util.find_spec
    monkeypatch.setattr(_build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert _build.build() == _build.LIB_PATH and os.path.exists(_build.LIB_PATH)
    assert toolchain.linked == ["libkvp.so"] and "kvp_calls.cpp.o" not in toolchain.compiled
    assert len(toolchain.compiled) == len(_build.SOURCES)


def test_the_library_builds_where_the_binding_does_not(toolchain):
    toolchain.broken = ("kvp_calls",)
    with pytest.raises(RuntimeError, match="kvp_calls.cpp"):
        _build.build()
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.CALLS_PATH)
    toolchain.broken = ()
    assert _build.build() == _build.LIB_PATH and os.path.exists(_build.CALLS_PATH)
    assert toolchain.linked == ["libkvp.so", "_kvp_calls.so"]
    n = len(toolchain.compiled)
    _build.build()  # and nothing is done twice
    assert len(toolchain.compiled) == n and len(toolchain.linked) == 2


def test_the_binding_is_built_anew_for_another_torch_or_python(toolchain, monkeypatch):
    _build.build()
    toolchain.compiled.clear(), toolchain.linked.clear()
    for change in (lambda: monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda n: "other"),
                   lambda: monkeypatch.setattr(_build, "_torch_dir", lambda: str(other))):
        other = os.path.join(_build.BUILD_DIR, "torch")
        os.makedirs(other, exist_ok=True)
        open(os.path.join(other, "version.py"), "w").write("__version__ = '9'")
        change()
        assert _build.calls_key_built() != _build.calls_key()
        _build.build()
        assert _build.calls_key_built() == _build.calls_key()
        _build.build()
    assert toolchain.compiled == ["kvp_calls.cpp.o"] * 2
    assert toolchain.linked == ["_kvp_calls.so"] * 2
    # one that could not be built is not taken for the present one
    open(os.path.join(other, "version.py"), "w").write("__version__ = '10'")
    toolchain.broken = ("kvp_calls",)
    with pytest.raises(RuntimeError):
        _build.build()
    assert _build.calls_key_built() is None


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    _build.build()
    kvp._calls.cache_clear()
    with monkeypatch.context() as m:
        m.setattr(_build, "calls_key", lambda: "another")
        with pytest.raises(RuntimeError, match="another torch or Python"):
            kvp._calls()
    assert kvp._calls() is not None


def test_counts_past_32_bits_are_refused(monkeypatch):
    """A count that the C interface's int32 cannot hold must not arrive there as its
    low word: 2^32 + 5 slots would be listed as 5."""
    lib = Recorder()
    monkeypatch.setattr(kvp, "load_library", lambda: lib)
    monkeypatch.setattr(kvp, "_on_one_device", lambda stream, *ts: 0)

    def i32(*shape):
        return torch.empty(shape, dtype=torch.int32, device="meta")

    many, one, two = 2 ** 32 + 5, i32(1), i32(2)
    tables = i32(2, 3)

    def refused(f, *args, **kw):
        with pytest.raises(kvp.KvpError) as e:
            f(*args, stream=Stream, **kw)
        assert e.value.status == kvp.KVP_ERR_UNSUPPORTED and lib.calls == []

    refused(kvp.kvp_extend_tables, tables, two, two, i32(9), one, two, one, i32(many), i32(3))
    refused(kvp.kvp_extend_tables, tables, two, two, i32(many), one, two, one, i32(4), i32(3))
    refused(kvp.kvp_extend_tables, i32(2, many), two, two, i32(9), one, two, one, i32(4), i32(3))
    refused(kvp.kvp_release_tables, i32(many, 1), i32(many), i32(many), i32(9), one, i32(many), one)
    refused(kvp.kvp_release_tables, tables, two, two, i32(many), one, two, one)
    f16 = dict(dtype=torch.float16, device="meta")
    codes = torch.empty((many, 1, 16, 32), dtype=torch.uint8, device="meta")
    pairs = torch.empty((many, 1, 16, 1, 2), **f16)
    row = torch.empty((1, 1, 64), **f16)
    refused(kvp.kvp_append_int4, row, row, codes, codes, pairs, pairs, one)
    refused(kvp.kvp_attention_decode_int4, row, row, codes, codes, pairs, pairs, i32(1, 4), one, 1.0)
    small, few = codes[:4], pairs[:4]
    refused(kvp.kvp_copy_blocks_int4, small, small, few, few, i32(many, 2))
    for parts in (2 ** 32, -2 ** 31 - 1):
        refused(kvp.kvp_attention_decode_int4, row, row, small, small, few, few, i32(1, 4), one, 1.0,
                partition_blocks=parts)
    refused(kvp.kvp_attention_decode_int4, row, row, small, small, few, few, i32(1, 4), one, 1.0,
            phases=2 ** 32 + 3)
    pool = torch.empty((4, 1, 16, 64), **f16)
    angles = torch.empty((many, 64), dtype=torch.float32, device="meta")
    refused(kvp.kvp_rope_append, row, row, row, row, pool, pool, angles, one, one)
    angles = torch.empty((9, 64), dtype=torch.float32, device="meta")
    refused(kvp.kvp_rope_append, row, row, row, row, pool, pool, angles, i32(2, 1), one,
            sections=(2 ** 32 + 16, 16))
    refused(kvp.kvp_rope_append, row, row, row, row, torch.empty((many, 1, 16, 64), **f16), pool,
            angles, one, one)
