"""What dec_kv4_write_scaled refuses, on the host before any CUDA call (CPU only)."""
import ctypes as C

import pytest

from transformer_decoder_kv_b200 import binding as b

P = 1 << 20      # a 16-byte aligned address; a refused call never reads it


@pytest.mark.parametrize("kw,word", [(dict(rule=2), "scale_rule"), (dict(rule=-1), "scale_rule"), (dict(ld=124), "ld"),
                                     (dict(k=None), "null"), (dict(cache=P + 8), "aligned")], ids=str)
def test_refused(kw, word):
    a = dict(k=P, ld=128, cache=P, rule=1)
    a.update(kw)
    view, rows = b.DecKvView(2, 16, 4, 3, 12, None), b.DecKvRows(3, 10, 5, P, None, P)
    st = b.lib().dec_kv4_write_scaled(C.byref(view), C.byref(rows), a["k"], P, a["ld"], a["cache"], a["rule"], None)
    assert st == b.DEC_EINVAL
    msg = b.lib().dec_last_error(None).decode()
    assert "dec_kv4_write_scaled" in msg and word in msg


def test_binding_names_the_rules():
    with pytest.raises(b.DecError, match="product"):
        b.kv4_write(None, None, None, None, None, scale="sevenths")
