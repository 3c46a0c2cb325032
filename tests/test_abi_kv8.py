"""Host-side validation and descriptor layouts of the rotary, append, 8-bit attention and log
probability calls (no GPU needed: every case is refused or empty before any device work)."""
import ctypes
import os
import subprocess

import pytest

import verify_step_b200 as sd
from verify_step_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 4096  # an aligned non-null address that is never read
BAD, UNSUP, WS = sd.SD_ERR_INVALID_ARG, sd.SD_ERR_UNSUPPORTED, sd.SD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    B.build()
    return sd.lib()


def with_(d, **kw):
    e = type(d).from_buffer_copy(d)
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def test_descriptor_layouts_match_the_header(tmp_path):
    structs = {"sd_rope_freq_desc": sd.RopeFreqDesc, "sd_rotary": sd.Rotary,
               "sd_rope_desc": sd.RopeDesc, "sd_append_desc": sd.AppendDesc,
               "sd_logprobs_desc": sd.LogprobsDesc}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "sd_verify.h"',
             'int main(void) {']
    for cname, py in structs.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        for fname, _ in py._fields_:
            lines.append(f'  printf("{cname} {fname} %zu\\n", offsetof({cname}, {fname}));')
    lines += ['  printf("e4m3 v %d\\n", (int)SD_E4M3);', '  return 0;', '}']
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = {}
    for line in subprocess.run([str(exe)], capture_output=True, text=True,
                               check=True).stdout.splitlines():
        cname, fname, v = line.split()
        got[(cname, fname)] = int(v)
    for cname, py in structs.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for fname, _ in py._fields_:
            assert got[(cname, fname)] == getattr(py, fname).offset, (cname, fname)
    assert got[("e4m3", "v")] == sd.SD_E4M3


def test_rope_freqs_refusals(L):
    d = sd.RopeFreqDesc(rot_dim=64, base=10000.0, scaling=sd.SD_ROPE_BY_PARTS, factor=4.0,
                        orig_ctx=4096, beta_fast=32.0, beta_slow=1.0)
    call = lambda e: L.sd_rope_freqs(ctypes.byref(e), A, None, None)
    assert L.sd_rope_freqs(None, A, None, None) == BAD
    assert L.sd_rope_freqs(ctypes.byref(d), None, None, None) == BAD
    for kw in (dict(rot_dim=0), dict(rot_dim=7), dict(base=1.0), dict(base=float("nan")),
               dict(scaling=3), dict(factor=0.5), dict(factor=float("nan")), dict(orig_ctx=0),
               dict(beta_fast=1.0), dict(beta_slow=-1.0)):
        assert call(with_(d, **kw)) == BAD, kw


def test_rope_refusals(L):
    d = sd.RopeDesc(rows=4, heads=2, head_dim=64, ld_x=128, ld_out=128, dtype=sd.SD_BF16,
                    rows_per_seq=1)
    r = sd.Rotary(A, 64, sd.SD_ROPE_HALF, 1.0)

    def call(e=d, rot=r, x=A, pos=A, ctx=None, out=2 * A):
        return L.sd_rope(ctypes.byref(e), ctypes.byref(rot), x, pos, ctx, out, None)
    assert L.sd_rope(None, ctypes.byref(r), A, A, None, A, None) == BAD
    assert L.sd_rope(ctypes.byref(d), None, A, A, None, A, None) == BAD
    for kw in (dict(rows=-1), dict(heads=0), dict(head_dim=0), dict(ld_x=127), dict(ld_out=100),
               dict(dtype=sd.SD_E4M3), dict(dtype=9)):
        assert call(with_(d, **kw)) == BAD, kw
    for kw in (dict(rot_dim=66), dict(rot_dim=0), dict(rot_dim=33), dict(layout=2),
               dict(freqs=None), dict(amplitude=float("nan"))):
        assert call(rot=with_(r, **kw)) == BAD, kw
    assert call(x=None) == BAD and call(out=None) == BAD and call(pos=None) == BAD
    assert call(x=A + 1) == BAD and call(out=A + 1) == BAD
    assert call(with_(d, rows_per_seq=0), pos=None, ctx=A) == BAD
    assert call(with_(d, ld_out=256), x=A, out=A) == BAD  # in place with another stride
    assert call(with_(d, rows=0), x=None, pos=None, out=None) == sd.SD_OK


def test_append_refusals(L):
    d = sd.AppendDesc(batch=2, n_new=3, n_rows=6, h_q=8, h_kv=2, head_dim=128, block_size=16,
                      max_blocks_per_seq=4, num_blocks=8, ld_k=256, ld_v=256, ld_q=1024,
                      ld_q_out=1024, dtype=sd.SD_BF16, cache_dtype=sd.SD_E4M3)
    r = sd.Rotary(A, 128, sd.SD_ROPE_HALF, 1.0)

    def call(e=d, rot=r, k=A, v=A, q=A, kc=A, vc=A, ks=A, vs=A, t=A, ctx=A, cu=None, qo=A):
        return L.sd_append_kv(ctypes.byref(e), ctypes.byref(rot) if rot else None, k, v, q, kc,
                              vc, ks, vs, t, ctx, cu, qo, None)
    assert L.sd_append_kv(None, *([None] * 13)) == BAD
    for kw in (dict(batch=0), dict(n_rows=-1), dict(h_q=-1), dict(h_kv=0), dict(head_dim=0),
               dict(block_size=0), dict(max_blocks_per_seq=0), dict(num_blocks=0),
               dict(n_new=2), dict(n_new=-3), dict(ld_k=255), dict(ld_v=128), dict(ld_q=1000),
               dict(ld_q_out=1000), dict(dtype=sd.SD_E4M3), dict(cache_dtype=sd.SD_F32),
               dict(cache_dtype=7), dict(ld_k=260), dict(ld_q=1028)):
        assert call(with_(d, **kw)) == BAD, kw
    for kw in (dict(block_size=8), dict(num_blocks=1 << 26),
               dict(head_dim=192, ld_k=384, ld_v=384, ld_q=1536, ld_q_out=1536)):
        assert call(with_(d, **kw)) == UNSUP, kw
    assert call(rot=with_(r, rot_dim=120)) == UNSUP
    assert call(rot=with_(r, rot_dim=130)) == BAD
    for kw in ("k", "v", "q", "kc", "vc", "ks", "vs", "t", "ctx", "qo"):
        assert call(**{kw: None}) == BAD, kw
    for kw in ("k", "v", "q", "kc", "vc", "qo"):
        assert call(**{kw: A + 8}) == BAD, kw
    # the rows' own type has no such limits, only element alignment
    e = with_(d, cache_dtype=sd.SD_BF16)
    assert call(e, k=A + 1) == BAD and call(e, kc=A + 1) == BAD
    assert call(with_(d, n_new=0, n_rows=0), k=None, v=None) == sd.SD_OK


def test_attention_q8_refusals(L):
    d = sd.AttnDesc(batch=2, n_q=3, h_q=8, h_kv=2, head_dim=256, block_size=16,
                    max_blocks_per_seq=4, num_blocks=8, window=0, scale=0.1, dtype=sd.SD_BF16)
    big = 1 << 40

    def call(e=d, q=A, kc=A, vc=A, ks=A, vs=A, t=A, ctx=A, out=A, ws=A, n=big):
        return L.sd_verify_attn_q8(ctypes.byref(e), q, kc, vc, ks, vs, t, ctx, out, ws, n, None)

    def draft(e, n=big):
        return L.sd_draft_xattn_q8(ctypes.byref(e), A, A, A, A, A, A, A, None, A, A, n, None)
    assert L.sd_verify_attn_q8(None, *([None] * 9), 0, None) == BAD
    for kw in (dict(batch=0), dict(n_q=0), dict(h_q=7), dict(h_kv=0), dict(block_size=0),
               dict(max_blocks_per_seq=0), dict(num_blocks=0), dict(scale=0.0),
               dict(scale=float("nan")), dict(dtype=sd.SD_F32), dict(dtype=sd.SD_E4M3)):
        assert call(with_(d, **kw)) == BAD, kw
        assert L.sd_verify_attn_q8_workspace_size(ctypes.byref(with_(d, **kw))) == 0
    for kw in (dict(head_dim=96), dict(block_size=24), dict(h_q=64), dict(num_blocks=1 << 27)):
        assert call(with_(d, **kw)) == UNSUP, kw
    assert draft(d) == BAD  # one query a sequence
    for kw in ("q", "kc", "vc", "ks", "vs", "t", "ctx", "out"):
        assert call(**{kw: None}) == BAD, kw
    for kw in ("q", "kc", "vc", "out"):
        assert call(**{kw: A + 8}) == BAD, kw
    assert call(ws=None) == WS and call(n=16) == WS and draft(with_(d, n_q=1), n=16) == WS


def test_logprobs_refusals(L):
    d = sd.LogprobsDesc(rows=4, vocab=100000, ld_logits=0, temperature=1.0, top_n=5)

    def call(e=d, z=A, t=A, lp=A, H=None, ids=A, top=A, ws=None, n=0):
        return L.sd_logprobs(ctypes.byref(e), z, t, lp, H, ids, top, ws, n, None)
    assert L.sd_logprobs(None, *([None] * 7), 0, None) == BAD
    for kw in (dict(rows=-1), dict(vocab=0), dict(ld_logits=99999), dict(temperature=0.0),
               dict(temperature=float("nan")), dict(temperature=float("inf")),
               dict(temperature=-1.0), dict(top_n=-1), dict(vocab=4)):
        assert call(with_(d, **kw)) == BAD, kw
    assert call(with_(d, top_n=33)) == UNSUP
    for kw in ("z", "t", "lp", "ids", "top"):
        assert call(**{kw: None}) == BAD, kw
    assert call(with_(d, rows=0), z=None) == sd.SD_OK


def test_binding_checks_row_tensors():
    import torch
    with pytest.raises(ValueError):
        sd._rows_ptr(torch.zeros(4, 8), 8, 4, 8)  # not on a device
    assert sd._rows_ptr(None, 8, 4, 8) is None and sd._rows_ptr(A, 8, 4, 8) == A


def test_a_temperature_whose_scale_overflows_is_refused(L):
    """log2(e) / T has to be finite: at 3e-39 1 / T still is."""
    d = sd.LogprobsDesc(rows=1, vocab=8, ld_logits=0, temperature=3e-39, top_n=0)
    assert sd.sd_logprobs_workspace_size(d) == 0
    assert L.sd_logprobs(ctypes.byref(d), A, A, A, None, None, None, None, 0, None) == BAD
    d.rows, d.temperature = 0, 5e-39
    assert L.sd_logprobs(ctypes.byref(d), A, A, A, None, None, None, None, 0, None) == sd.SD_OK


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Before anything of the call runs: a call is launched on the current device."""
    class Other:
        is_cuda = True

        def get_device(self):
            return 1

    monkeypatch.setattr(sd, "_current_device", lambda: 0)
    x = Other()
    for call in (lambda: sd.sd_rope(sd.RopeDesc(), None, x, None, None, None),
                 lambda: sd.sd_append_kv(sd.AppendDesc(), None, x, *[None] * 8),
                 lambda: sd.sd_verify_attn_q8(sd.AttnDesc(), x, *[None] * 8),
                 lambda: sd.sd_draft_xattn_q8(sd.AttnDesc(), x, *[None] * 9),
                 lambda: sd.sd_logprobs(sd.LogprobsDesc(), x, None, None)):
        with pytest.raises(ValueError, match="current device"):
            call()
