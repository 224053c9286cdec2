"""The Python binding and its build, without a GPU."""
import torch

import pagedattention_decode_kvp_gb300 as kvp


class Recorder:
    """A library whose calls are recorded and succeed."""

    def __init__(self):
        self.calls = []

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
