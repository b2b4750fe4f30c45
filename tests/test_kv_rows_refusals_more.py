"""More of what the row-batch operators refuse, on the host before any CUDA call (CPU only)."""
import ctypes as C

import pytest

from transformer_decoder_kv_b200 import binding as b

P = 1 << 20      # an aligned address; a refused call never reads it


def _calls(table=None, row_start=P, slots=None, lens=P):
    lib = b.lib()
    view, rows = b.DecKvView(2, 16, 4, 3, 12, table), b.DecKvRows(3, 10, 5, row_start, slots, lens)
    v, r = C.byref(view), C.byref(rows)
    yield lib.dec_kv4_write(v, r, P, P, 128, P, None)
    yield lib.dec_kv4_write_scaled(v, r, P, P, 128, P, 1, None)
    yield lib.dec_kv4_read(v, r, P, P, P, 128, None)
    yield lib.dec_attention_kv4(v, r, P, 256, 4, P, 0, 0, P, 256, P, 1 << 40, None)
    yield lib.dec_attention_window(v, r, P, 256, 4, P, P, 0, 0, P, 256, P, 1 << 40, None)
    assert lib.dec_attention_rows_workspace_size(v, r, 4) == 0


@pytest.mark.parametrize("name", ["table", "row_start", "slots", "lens"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_index_arrays_off_their_alignment(name, off):
    for st in _calls(**{name: P + off}):
        assert st == b.DEC_EINVAL
        msg = b.lib().dec_last_error(None).decode()
        assert name in msg and "4-byte" in msg


def test_a_workspace_of_negative_size():
    import torch
    rows = type("Rows", (), {"device": None})()
    for n in (-1, -(1 << 40)):
        with pytest.raises(b.DecError, match=f"needs {n}"):
            b._scratch(rows, torch.zeros(4), n)


BIG = [1 << 31, 1 << 32, (1 << 32) + 1, -(1 << 31) - 1]


@pytest.mark.parametrize("n", BIG)
def test_whole_numbers_beyond_32_bits(n):
    for i in range(5):
        a = [2, 16, 4, 3, 12]
        a[i] = n
        with pytest.raises(b.DecError, match="beyond 32 bits"):
            b.KvView(*a)
    for kw in (dict(batch=n), dict(batch=1, n_rows=n), dict(batch=1, max_rows=n)):
        with pytest.raises(b.DecError, match="beyond 32 bits"):
            b.KvRows(lens=None, **kw)
    view = b.KvView(2, 16, 4, 3)
    rows = type("Rows", (), {"torch": None, "ref": None})()
    with pytest.raises(b.DecError, match="beyond 32 bits"):
        b.attention_rows_workspace_size(view, rows, n)
    for kw in (dict(window=n), dict(sinks=n)):
        with pytest.raises(b.DecError, match="beyond 32 bits"):
            b.attention_kv4(view, rows, None, None, 4, None, None, 0, **kw)
        with pytest.raises(b.DecError, match="beyond 32 bits"):
            b.attention_window(view, rows, None, None, None, 4, None, None, 0, **kw)
    with pytest.raises(b.DecError, match="beyond 32 bits"):
        b.attention_kv4(view, rows, None, None, n, None, None, 0)
