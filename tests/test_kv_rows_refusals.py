"""What the row-batch operators refuse, on the host before any CUDA call (CPU only)."""
import ctypes as C

import pytest

from transformer_decoder_kv_b200 import binding as b

P = 1 << 20      # a 16-byte aligned address; a refused call never reads it


def _view(**kw):
    a = dict(n_kv_heads=2, page_rows=16, pages_per_slot=4, n_slots=3, n_pages=12, table=None)
    a.update(kw)
    return b.DecKvView(*a.values())


def _rows(**kw):
    a = dict(batch=3, n_rows=10, max_rows=5, row_start=P, slots=None, lens=P)
    a.update(kw)
    return b.DecKvRows(*a.values())


BAD_VIEWS = [dict(n_kv_heads=0), dict(page_rows=0), dict(pages_per_slot=0), dict(n_slots=0), dict(n_pages=0),
             dict(n_pages=11), dict(n_pages=-1), dict(pages_per_slot=1 << 27, table=P),
             dict(n_slots=1 << 20, pages_per_slot=1 << 12, n_pages=5, table=P), dict(page_rows=48, table=P)]
BAD_ROWS = [dict(batch=0), dict(batch=65536), dict(n_rows=0), dict(max_rows=0), dict(max_rows=11), dict(lens=None),
            dict(row_start=None), dict(row_start=None, max_rows=1, n_rows=2)]


def _refused(status, *words):
    assert status == b.DEC_EINVAL
    msg = b.lib().dec_last_error(None).decode()
    for w in words:
        assert w in msg, msg


def _calls(view, rows, kv4_only=False):
    lib, v, r = b.lib(), C.byref(view), C.byref(rows)
    yield "dec_kv4_write", lib.dec_kv4_write(v, r, P, P, 128, P, None)
    yield "dec_kv4_read", lib.dec_kv4_read(v, r, P, P, P, 128, None)
    yield "dec_attention_kv4", lib.dec_attention_kv4(v, r, P, 256, 4, P, 0, 0, P, 256, P, 1 << 40, None)
    if not kv4_only:
        yield "dec_attention_window", lib.dec_attention_window(v, r, P, 256, 4, P, P, 0, 0, P, 256, P, 1 << 40, None)


@pytest.mark.parametrize("bad", BAD_VIEWS, ids=str)
def test_bad_views(bad):
    v = _view(**bad)
    for name, st in _calls(v, _rows()):
        _refused(st, name)
    assert b.lib().dec_kv4_bytes(C.byref(v)) == 0


@pytest.mark.parametrize("bad", BAD_ROWS, ids=str)
def test_bad_rows(bad):
    r = _rows(**bad)
    for name, st in _calls(_view(), r):
        _refused(st, name)
    assert b.lib().dec_attention_rows_workspace_size(C.byref(_view()), C.byref(r), 4) == 0


def test_odd_page_rows_are_for_one_page_f32_slots_only():
    v = _view(page_rows=300, pages_per_slot=1, n_pages=3)
    for name, st in _calls(v, _rows(), kv4_only=True):
        _refused(st, name, "page_rows")
    assert b.lib().dec_attention_rows_workspace_size(C.byref(v), C.byref(_rows()), 4) > 0
    _refused(b.lib().dec_attention_window(C.byref(_view(page_rows=300, pages_per_slot=2, n_pages=6)), C.byref(_rows()),
                                          P, 256, 4, P, P, 0, 0, P, 256, P, 1 << 40, None), "page_rows")


def test_null_structs_and_pointers():
    lib, v, r = b.lib(), C.byref(_view()), C.byref(_rows())
    _refused(lib.dec_kv4_write(None, r, P, P, 128, P, None), "view")
    _refused(lib.dec_kv4_write(v, None, P, P, 128, P, None), "rows")
    for i in range(3):
        p = [P, P, P]
        p[i] = None
        _refused(lib.dec_kv4_write(v, r, p[0], p[1], 128, p[2], None), "null")
        _refused(lib.dec_kv4_read(v, r, p[2], p[0], p[1], 128, None), "null")
    for i in range(4):
        p = [P] * 4
        p[i] = None
        _refused(lib.dec_attention_kv4(v, r, p[0], 256, 4, p[1], 0, 0, p[2], 256, p[3], 1 << 40, None), "null")
        _refused(lib.dec_attention_window(v, r, p[0], 256, 4, p[1], P, 0, 0, p[2], 256, p[3], 1 << 40, None), "null")
    _refused(lib.dec_attention_window(v, r, P, 256, 4, P, None, 0, 0, P, 256, P, 1 << 40, None), "null")


def test_strides_alignment_heads_window_and_workspace():
    lib, v, r = b.lib(), C.byref(_view()), C.byref(_rows())
    for ld in (124, 127, 130, -128):
        _refused(lib.dec_kv4_write(v, r, P, P, ld, P, None), "ld")
    for ptrs in ((P + 4, P, P), (P, P + 8, P), (P, P, P + 1)):
        _refused(lib.dec_kv4_write(v, r, ptrs[0], ptrs[1], 128, ptrs[2], None), "aligned")

    def kv4(q=P, q_ld=256, heads=4, cache=P, window=0, sinks=0, out=P, out_ld=256, ws=P, nb=1 << 40):
        return lib.dec_attention_kv4(v, r, q, q_ld, heads, cache, window, sinks, out, out_ld, ws, nb, None)
    for heads in (0, -2, 3, 65536):
        _refused(kv4(heads=heads, q_ld=1 << 30, out_ld=1 << 30), "n_heads")
        if heads != 65536:
            assert lib.dec_attention_rows_workspace_size(v, r, heads) == 0
    _refused(kv4(window=-1), "window")
    _refused(kv4(sinks=-1), "sinks")
    _refused(kv4(q_ld=252), "q_ld")
    _refused(kv4(out_ld=258), "out_ld")
    for a in (dict(q=P + 4), dict(cache=P + 8), dict(out=P + 4), dict(ws=P + 4)):
        _refused(kv4(**a), "aligned")
    _refused(kv4(nb=lib.dec_attention_rows_workspace_size(v, r, 4) - 1), "workspace")


def test_binding_checks_types_shapes_and_devices():
    import torch
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    with pytest.raises(b.DecError, match="int32"):
        b.KvRows(2, torch.zeros(2))
    with pytest.raises(b.DecError, match="elements"):
        b.KvRows(3, i32(1, 2))
    with pytest.raises(b.DecError, match="CUDA"):
        b.KvRows(2, i32(1, 2))
    with pytest.raises(b.DecError, match="CUDA"):
        b.KvView(1, 16, 2, 1, 2, i32(0, 1))
    with pytest.raises(b.DecError, match="contiguous"):
        b.KvView(1, 16, 2, 1, 2, torch.zeros((2, 2), dtype=torch.int32)[:, 0])
    with pytest.raises(b.DecError, match="float32"):
        b._row_buffer("q", torch.zeros((2, 64), dtype=torch.float16), 2, 64)
    with pytest.raises(b.DecError, match="CUDA"):
        b._row_buffer("q", torch.zeros((2, 64)), 2, 64)
    with pytest.raises(b.DecError, match="device tensor"):
        b.KvRows(2, [1, 2])
    with pytest.raises(b.DecError, match="device tensor"):
        b._row_buffer("q", [[0.0] * 64], 1, 64)
    rows = type("Rows", (), {"device": None})()
    for ws, n, word in ((torch.zeros(4), 17, "needs 17"), (torch.zeros(8)[::2], 16, "contiguous"),
                        (torch.zeros(4), 16, "CUDA"), (object(), 16, "device tensor")):
        with pytest.raises(b.DecError, match=word):
            b._scratch(rows, ws, n)
    with pytest.raises(b.DecError, match="bad view"):
        b.kv4_bytes(b.KvView(1, 48, 2, 1))


def test_pool_bytes():
    assert b.kv4_bytes(b.KvView(2, 16, 4, 3)) == 12 * 2 * 16 * 72
    assert b.kv4_bytes(b.KvView(8, 64, 1024, 4096)) == 4096 * 1024 * 8 * 64 * 72      # beyond 32 bits


def test_places_of_malformed_batches_stay_in_range():
    import os
    import shutil
    import subprocess
    import tempfile
    here = os.path.dirname(os.path.abspath(__file__))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not available")
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "kv_rows_check")
        r = subprocess.run([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_100a,code=sm_100a", "-I",
                            os.path.join(os.path.dirname(here), "transformer_decoder_kv_b200", "csrc"),
                            os.path.join(here, "kv_rows_check.cu"), "-o", exe], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-3000:]
        r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-3000:]
