"""The row-batch attentions over values of very different size: keys that some or all rows do not see,
keys without weight, tiles that are not finite, lengths past a slot's end.

Tolerance of a row (`_reference`), every term a bound of one step: scores are off by 2^-18 of sum |q k| / 8 at
most (operands carried to 22 bits, 3 2^-22, and 64 terms in three products summed in f32), a key's own and the
maximum's; values by 3 2^-22 (two operands of 22 bits, the product of the low parts left out) and sums over
keys by 2^-23 per step of 16 keys or more, all of them relative to sum p |v|; a weight below f16's range is
off by 2^-37 of the largest.
"""
import numpy as np
import pytest

from tests._kvrows import D, Setup, check, kv4_values

pytestmark = pytest.mark.gpu

# rows of one stream with one head: each of the kernels
KINDS = [(True, 1), (True, 6), (True, 12), (True, 100), (False, 1), (False, 2), (False, 5), (False, 20), (False, 100)]
SHARED = [k for k in KINDS if k[1] > 2]
_id = lambda k: f"{'kv4' if k[0] else 'f32'}-{k[1]}" if isinstance(k, tuple) else None


def _stream(kind, n, page_rows=16, seed=3):
    kv4, r = kind
    s = Setup(1, 1, [n], [r], page_rows, False, seed=seed, spare_slots=0, pad_rows=0)
    s.v[0] *= np.float32(0.5)
    return s


def _reference(s, kv4, window, sinks, pos=None):
    k, v = (kv4_values(x[0]) if kv4 else x[0] for x in (s.k, s.v))
    k, v = np.asarray(k, np.float64)[:, 0], np.asarray(v, np.float64)[:, 0]
    r, j = s.rows[0], np.arange(len(k))
    pos = np.arange(s.lens[0] - r, s.lens[0]) if pos is None else pos
    out, tol = np.zeros((r, D)), np.zeros((r, 1))
    for i, p in enumerate(pos):
        see = (j <= p) & ((j > p - window) | (j < sinks)) if window else j <= p
        kk, vv, q = k[see], v[see], s.q[i, 0].astype(np.float64)
        with np.errstate(all="ignore"):
            x = kk @ q / 8
            w = np.exp(x - x.max()) if len(x) else x
            if not (len(w) and np.isfinite(w.sum()) and w.sum() > 0):
                continue
            w = w / w.sum()
            out[i] = np.where(w[:, None] == 0, 0, w[:, None] * vv).sum(0)
            live = w > 1e-40                        # e^-92: far below the smallest weight that counts
            amp = np.abs(np.where(np.isfinite(kk), kk, 0) * q)[live].sum(1).max() / 8
            mass = np.where(np.isfinite(vv), np.abs(vv), 0)[live]
            tol[i] = ((w[live, None] * mass).sum(0).max() * (2 * 2.0 ** -18 * amp + 3 * 2.0 ** -22 + (len(w) / 16 + 32) * 2.0 ** -23)
                      + mass.max() * 2.0 ** -37 * live.sum())
    return out, tol


def _caches(s, kv4):
    if not kv4:
        return s.f32_pools()
    c = s.new_cache()
    s.write_all(c)
    return c


def _check(s, kv4, window=0, sinks=0, caches=None):
    out = s.attend(kv4, window, sinks, _caches(s, kv4) if caches is None else caches)
    s.torch.cuda.synchronize()
    ref, tol = _reference(s, kv4, window, sinks)
    check(out.cpu().numpy(), ref, tol)


@pytest.mark.parametrize("value", [1e12, -1e30, 3e38])
@pytest.mark.parametrize("kind", KINDS, ids=_id)
def test_large_values_that_no_row_sees(kind, value):
    """Behind the window and past the sinks, the border chunks of both among them."""
    s = _stream(kind, 300)
    s.k[0][4:300 - kind[1] - 40 + 1, 0, ::5] = value
    s.v[0][4:300 - kind[1] - 40 + 1, 0, 3::7] = value
    _check(s, kind[0], 40, 4)


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("rows", [1, 4, 8, 16, 100])
def test_rows_never_written_hold_anything(rows, seed):
    """Every bit pattern of codes and scales outside the rows that are seen."""
    s = _stream((True, rows), 300, seed=seed)
    t = s.torch
    g = t.Generator(device="cuda").manual_seed(seed)
    cache = t.randint(0, 256, (s.pkg.kv4_bytes(s.view),), dtype=t.uint8, device="cuda", generator=g)
    lo, sinks = 300 - rows - 40 + 1, 4
    one = lambda a, n: s.f32(a[0][a_lo:a_lo + n].reshape(n, D))
    for a_lo, n in ((0, sinks), (lo, 300 - lo)):
        s.pkg.kv4_write(s.view, s.make_rows([a_lo + n], [n]), one(s.k, n), one(s.v, n), cache)
    _check(s, True, 40, sinks, cache)


@pytest.mark.parametrize("window", [0, 30])
@pytest.mark.parametrize("page_rows", [37, 100, 129])
@pytest.mark.parametrize("kind", [k for k in KINDS if not k[0] and k[1] < 37], ids=_id)
def test_queries_past_the_end_of_a_slot_of_any_size(kind, page_rows, window):
    s = _stream(kind, page_rows, page_rows)
    caches = s.f32_pools()
    for past in (1, 8, 20):
        s.batch = s.make_rows([page_rows + past], s.rows)
        out = s.attend(False, window, 0, caches)
        s.torch.cuda.synchronize()
        ref, tol = _reference(s, False, window, 0, np.arange(page_rows + past - kind[1], page_rows + past))
        check(out.cpu().numpy(), ref, tol, past)


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("value", [np.float32(63.99), np.float32(65535) / 1024])
@pytest.mark.parametrize("rows", [20, 100])
def test_values_just_below_a_power_of_two(rows, value, what):
    """Tiles of values below 2, and one of a later tile whose size in f16 would round up to infinity."""
    s = _stream((False, rows), 900)
    for x in (s.k, s.v):
        np.clip(x[0], -1.9, 1.9, out=x[0])
        x[0][:, 0, 0] = 1.5
    for at in (200, 330, 600):
        (s.k if what == "k" else s.v)[0][at, 0, 9] = value
    s.q[:, 0, 9] *= np.float32(0.05)
    _check(s, False)


@pytest.mark.parametrize("flat", [False, True], ids=["scaled", "flat"])
@pytest.mark.parametrize("kind", SHARED, ids=_id)
def test_a_first_tile_that_is_not_finite(kind, flat):
    """NaN in the last row's own key: the rows before it, with values of 1000 or weights all alike, do not see it."""
    kv4, r = kind
    for n in (r + 3, r + 60):
        s = _stream(kind, n)
        if flat:
            s.q[:] = 0
            s.v[0][:] = 1
        else:
            s.v[0] *= np.float32(1000)
        s.v[0][n - 1, 0, 3] = np.nan
        s.k[0][n - 2, 0, 5] = np.inf
        if flat:
            s.k[0][n - 2, 0, 5] = 1.0
        _check(s, kv4)


@pytest.mark.parametrize("value", [1e5, 1e9, 1e12, 1e30, 3e38])
@pytest.mark.parametrize("what", ["k", "v", "kv"])
@pytest.mark.parametrize("kind", SHARED, ids=_id)
def test_large_values_that_only_some_rows_see(kind, what, value):
    kv4, r = kind
    for n, window, at in ((r + 2, 0, -1), (400, 0, -1), (400, 100, 400 - r - 99)):
        s = _stream(kind, n)
        if "k" in what:
            s.k[0][at, 0, 2] = value
        if "v" in what:
            s.v[0][at, 0, 2] = value
        sees = np.arange(n - r, n) >= n - 1 if at < 0 else np.arange(n - r, n) - window < at
        out = s.attend(kv4, window, 0, _caches(s, kv4))
        s.torch.cuda.synchronize()
        ref, tol = _reference(s, kv4, window, 0)
        assert 0 < sees.sum() < r
        check(out.cpu().numpy()[~sees], ref[~sees], tol[~sees], (n, window))
        if "k" not in what:
            check(out.cpu().numpy()[sees], ref[sees], tol[sees], (n, window))


@pytest.mark.parametrize("value", [1e5, 1e9, 1e12, 1e30, 1e38])
@pytest.mark.parametrize("kind", KINDS, ids=_id)
def test_large_values_without_weight(kind, value):
    """A key far below the others' scores holds a large V: the outputs are the others'. The same for a large K."""
    kv4, r = kind
    for n, at in ((r + 30, 5), (700, 340)):
        for large_k in (False, True):
            s = _stream(kind, n)
            s.q = (s.q[:1] * np.ones((r, 1, 1)) + 0.1 * s.q).astype(np.float32)
            low = -s.q[0, 0] * np.float32(200)
            s.k[0][at, 0] = np.where(np.abs(low) > 20, low, 0)
            if large_k:
                i = int(np.argmax(np.abs(s.q[0, 0])))
                s.k[0][at, 0, i] = -np.sign(s.q[0, 0, i]) * value
            else:
                s.v[0][at, 0, 7] = value
            _check(s, kv4)


@pytest.mark.parametrize("value", [1e30, 1e36, 3e-30])
@pytest.mark.parametrize("n", [300, 4000])
@pytest.mark.parametrize("kind", KINDS, ids=_id)
def test_values_near_the_ends_of_the_range(kind, n, value):
    """Sums over many keys of about equal weight: every one of them is a number in f32."""
    s = _stream(kind, n)
    s.q *= np.float32(0.01)
    s.v[0] *= np.float32(value)
    _check(s, kind[0])


@pytest.mark.parametrize("kind", KINDS, ids=_id)
def test_the_low_halves_of_operands_count(kind):
    """Three keys with scores of 1 and -1, one operand 2^-12 off its nearest f16 in every element. Left at 11
    bits it takes a score 2^-12 off and the output 2^-14 (weights 0.79 and 0.21), or a value 2^-12 off; the
    tolerance is 2^-16 and less. (Equal scores: the weights' own bits.)"""
    kv4, r = kind
    off = np.float32(1 + 2.0 ** -11 + 2.0 ** -12)         # f16 has 1 and 1 + 2^-10
    sign = np.where(np.arange(D) % 2, 1, -1).astype(np.float32)
    for q, k, v in ((off, 1, 1), (1, off, 1), (0.01, 1, off), (0.01, 1, 1)):
        s = _stream(kind, max(3, r), page_rows=64)
        s.q[:, 0] = sign * np.float32(0.25) * np.float32(q)
        s.k[0][:, 0] = sign * np.float32(0.5)
        s.k[0][::2, 0] *= -np.float32(k)
        s.v[0][:, 0] = np.float32(v)
        s.v[0][::2, 0] = np.float32(-1 - 2.0 ** -5)
        _check(s, kv4)
