"""Calls over the 8-bit cache and of the log probabilities that have to be refused, and what the binding
asks of its tensors (no GPU needed: every case ends before any device work)."""
import ctypes

import pytest

import verify_step_b200 as sd
from verify_step_b200 import build as B

A = 4096  # an aligned non-null address that is never read
BAD, UNSUP = sd.SD_ERR_INVALID_ARG, sd.SD_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    B.build()
    return sd.lib()


@pytest.mark.parametrize("cache", [sd.SD_E4M3, sd.SD_BF16])
def test_queries_turned_in_place_need_one_row_stride(L, cache):
    """Rows of one stride would be written over rows of the other that are still to be read."""
    d = sd.AppendDesc(batch=2, n_new=3, n_rows=6, h_q=8, h_kv=2, head_dim=128, block_size=16,
                      max_blocks_per_seq=4, num_blocks=8, ld_k=256, ld_v=256, ld_q=1024,
                      ld_q_out=2048, dtype=sd.SD_BF16, cache_dtype=cache)
    r = sd.Rotary(A, 128, sd.SD_ROPE_HALF, 1.0)
    call = lambda: L.sd_append_kv(ctypes.byref(d), ctypes.byref(r), A, A, A, A, A, A, A, A, A, None, A,
                                  None)
    assert call() == BAD
    d.ld_q, d.ld_q_out = 2048, 1024
    assert call() == BAD


def test_blocks_whose_elements_do_not_fit_32_bits_are_refused(L):
    d = sd.AppendDesc(batch=1, n_new=1, n_rows=1, h_kv=1, head_dim=64, block_size=1 << 25,
                      max_blocks_per_seq=1, num_blocks=1, ld_k=64, ld_v=64, dtype=sd.SD_BF16,
                      cache_dtype=sd.SD_E4M3)
    call = lambda: L.sd_append_kv(ctypes.byref(d), None, A, A, None, A, A, A, A, A, A, None, None, None)
    assert call() == UNSUP
    d.head_dim, d.ld_k, d.ld_v, d.block_size = 512, 512, 512, 1 << 22
    assert call() == UNSUP
    d.n_rows = d.n_new = 0
    d.block_size = 1 << 21
    assert call() == sd.SD_OK


class OnDevice:
    """A contiguous CUDA tensor as far as the binding looks."""
    is_cuda = True

    def __init__(self, device):
        self.device, self.asked = device, False

    def get_device(self):
        self.asked = True
        return self.device

    def is_contiguous(self):
        return True

    def numel(self):
        return 1 << 30

    def data_ptr(self):
        return A

    def element_size(self):
        return 1


CALLS = {  # a call of n tensors, whose empty descriptor is refused by the library
    "sd_rope_freqs": (lambda t: sd.sd_rope_freqs(sd.RopeFreqDesc(), t[0]), 1),
    "sd_rope": (lambda t: sd.sd_rope(sd.RopeDesc(), turns(t[0]), *t[1:]), 5),
    "sd_append_kv": (lambda t: sd.sd_append_kv(sd.AppendDesc(), turns(t[0]), *t[1:]), 12),
    "sd_verify_attn_q8": (lambda t: sd.sd_verify_attn_q8(sd.AttnDesc(), *t), 9),
    "sd_draft_xattn_q8": (lambda t: sd.sd_draft_xattn_q8(sd.AttnDesc(), *t), 10),
    "sd_logprobs": (lambda t: sd.sd_logprobs(sd.LogprobsDesc(), *t), 7)}


def turns(table):
    r = sd.Rotary(A, 64, sd.SD_ROPE_HALF, 1.0)
    r.table = table
    return r


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_of_another_device_is_refused(L, monkeypatch, name):
    """Whichever argument it is, the rotation's table and the workspace among them: the kernels of a
    call run on the current device."""
    monkeypatch.setattr(sd, "_current_device", lambda: 0)
    monkeypatch.setattr(sd, "_stream", lambda s: 0)
    monkeypatch.setattr(sd, "_nbytes", lambda t: 0)
    call, n = CALLS[name]
    good = [OnDevice(0) for _ in range(n)]
    with pytest.raises(sd.SdError):  # the empty descriptor is refused, after the tensors
        call(good)
    assert all(t.asked for t in good)
    for i in range(n):
        t = [OnDevice(0) for _ in range(n)]
        t[i] = OnDevice(1)
        with pytest.raises(ValueError, match="current device"):
            call(t)


def test_the_current_stream_without_torch_s_inner_calls(monkeypatch):
    """Where a torch has no raw calls for the current device and stream, the public ones serve."""
    import torch
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)

    class Stream:
        def __init__(self, device):
            self.cuda_stream = 1000 + device

    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(sd, "_cuda", None)
    assert sd._current_device() == 3 and sd._stream(None) == 1003


def test_row_counts_at_the_integer_limit_are_refused(L):
    """Rows are counted up to whole CTAs in 32 bits."""
    r = sd.Rotary(A, 2, sd.SD_ROPE_HALF, 1.0)
    n = (1 << 31) - 1
    d = sd.RopeDesc(rows=n, heads=1, head_dim=2, ld_x=2, ld_out=2, dtype=sd.SD_BF16, rows_per_seq=1)
    assert L.sd_rope(ctypes.byref(d), ctypes.byref(r), A, A, None, 2 * A, None) == UNSUP
    e = sd.AppendDesc(batch=1, n_new=n, n_rows=n, h_kv=1, head_dim=2, block_size=16,
                      max_blocks_per_seq=4, num_blocks=8, ld_k=2, ld_v=2, dtype=sd.SD_BF16,
                      cache_dtype=sd.SD_BF16)
    assert L.sd_append_kv(ctypes.byref(e), None, A, A, None, A, A, None, None, A, A, None, None,
                          None) == UNSUP
