"""What a caller sees of errors of the norms, quantisers and products, by a library that makes
them (no GPU needed)."""
import ctypes

import pytest
import torch

import pagedattention_decode_kvp_gb300 as kvp

U8 = torch.uint8


class Stream:
    device_index = 0
    cuda_stream = 7


class Library:
    """Calls return `status`; a product leaves `word` in the status word that it is given, as a
    kernel whose wait gave up does."""

    def __init__(self, status=0, word=0):
        self.status, self.word = status, word

    def kvp_status_string(self, status):
        return b"KVP_ERR_CUDA" if status == kvp.KVP_ERR_CUDA else b"status"

    def kvp_matmul_fp8(self, *args):
        if args[-2] is not None and self.word:
            ctypes.c_int32.from_address(args[-2]).value = self.word
        return self.status

    def kvp_read_status(self, at, stream):
        return ctypes.c_int32.from_address(at).value

    def __getattr__(self, name):
        return lambda *args: self.status


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(kvp, "load_library", lambda: lib)
    monkeypatch.setattr(kvp, "_on_one_device", lambda stream, *ts: 7)
    return lib


def calls():
    """Every entry point on tensors in order, and its arguments by name."""
    x, w = torch.zeros((3, 256), dtype=torch.float16), torch.zeros(256, dtype=torch.float16)
    codes, scales = torch.zeros((3, 256), dtype=U8), torch.zeros((3, 2))
    s = dict(stream=Stream)
    return {"kvp_rms_norm": lambda: kvp.kvp_rms_norm(x, x, w, 1e-5, **s),
            "kvp_rms_norm_fp8": lambda: kvp.kvp_rms_norm_fp8(codes, scales, x, w, 1e-5, **s),
            "kvp_quantise_fp8": lambda: kvp.kvp_quantise_fp8(codes, scales, x, **s),
            "kvp_matmul_fp8": lambda: kvp.kvp_matmul_fp8(
                torch.zeros((3, 3)), codes, scales, codes, torch.zeros((1, 2)), **s)}


@pytest.mark.parametrize("name", sorted(calls()))
def test_a_failed_launch_is_an_error(library, name):
    calls()[name]()
    library.status = kvp.KVP_ERR_CUDA
    with pytest.raises(kvp.KvpError, match=name) as e:
        calls()[name]()
    assert e.value.status == kvp.KVP_ERR_CUDA


def test_a_wait_that_gave_up_is_in_the_status_word(library):
    """The call itself returns: what happened on the GPU is read from the word."""
    library.word = kvp.KVP_ERR_TIMEOUT
    codes, scales = torch.zeros((3, 256), dtype=U8), torch.zeros((3, 2))
    status = torch.zeros(1, dtype=torch.int32)
    args = (torch.zeros((3, 3)), codes, scales, codes, torch.zeros((1, 2)))
    kvp.kvp_matmul_fp8(*args, stream=Stream)
    assert kvp.kvp_read_status(status, Stream) == kvp.KVP_OK
    kvp.kvp_matmul_fp8(*args, status=status, stream=Stream)
    assert kvp.kvp_read_status(status, Stream) == kvp.KVP_ERR_TIMEOUT
