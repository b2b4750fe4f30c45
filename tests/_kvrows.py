"""64-bit reference of the row-batch cache operators, and the set-up of their tests.

The 4-bit code (per row, head and group of 32 dims): s = bf16(f32(max |x| / 7)), 0 below 2^-126;
c = x / s to the nearest integer, ties to even; value c s; NaN for a group that is not finite.
"""
import numpy as np

D = 64


def bf16_round(a):
    """f32 -> bf16 (nearest, ties to even), as f32."""
    u = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7fff + ((u >> 16) & 1)) >> 16) << 16
    return r.astype(np.uint32).view(np.float32)


def kv4_values(x):
    """What a 4-bit cache stands for, of f32 rows [..., 64]."""
    x = np.asarray(x, np.float32)
    g = x.reshape(-1, 32)
    finite = np.isfinite(g).all(axis=1)
    gf = np.where(np.isfinite(g), g, np.float32(0))
    a = np.abs(gf).max(axis=1)
    s = bf16_round(a / np.float32(7))
    s = np.where(s < np.float32(2.0 ** -126), np.float32(0), s)
    s64 = s.astype(np.float64)[:, None]
    c = np.rint(np.divide(gf.astype(np.float64), s64, out=np.zeros(g.shape), where=s64 > 0))
    assert np.abs(c).max(initial=0) <= 7
    v = c * s64
    v[~finite] = np.nan
    return v.reshape(x.shape)


def attention(q, k, v, pos, window, sinks, hidden=None):
    """One stream: q [n, H, 64] at positions pos[n], k and v [m, HK, 64] -> [n, H, 64] in f64, and the
    error the tests allow per row. `hidden` [m]: keys on bad pages."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    n, H, _ = q.shape
    m, HK, _ = k.shape
    out, tol = np.zeros((n, H, D)), np.zeros((n, H, 1))
    j = np.arange(m)
    for i in range(n):
        see = j <= pos[i]
        if window:
            see &= (j > pos[i] - window) | (j < sinks)
        if hidden is not None:
            see &= ~hidden
        idx = np.nonzero(see)[0]
        if len(idx) == 0:
            continue
        for h in range(H):
            kk, vv = k[idx, h // (H // HK)], v[idx, h // (H // HK)]
            with np.errstate(all="ignore"):
                s = kk @ q[i, h] / 8
                p = np.exp(s - s.max())
                l = p.sum()
                if not (np.isfinite(l) and l > 0):
                    continue
                w = p / l
                out[i, h] = np.where((w == 0)[:, None], 0, w[:, None] * vv).sum(axis=0)
                amp = np.abs(np.where(np.isfinite(kk), kk, 0) * q[i, h]).sum(axis=1).max() / 8
                big = np.abs(vv[np.isfinite(vv)]).max(initial=0)
            # scores: f32 operands carried to 22 bits or more and 64 terms summed in f32, 2^-18 of
            # sum |q k| / 8 at most, twice (a key's own and the maximum's); exp and the sums over
            # keys: each step of 16 keys or more rounds its partial sum by 2^-23 at most
            tol[i, h] = big * (2.0 ** -17 * amp + (len(idx) / 16 + 32) * 2.0 ** -23)
    return out, tol


def check(got, ref, tol, what=""):
    got = np.asarray(got, np.float64)
    bad_kind = (np.isnan(got) != np.isnan(ref))
    assert not bad_kind.any(), (what, "NaN in other places", np.argwhere(bad_kind)[:4].tolist())
    with np.errstate(invalid="ignore"):
        ok = np.isnan(ref) | (got == ref) | (np.abs(got - ref) <= tol)
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.size} outside; first at {i}: got {got[i]!r} ref {ref[i]!r} "
                             f"tol {np.broadcast_to(tol, ok.shape)[i]!r}")


class Setup:
    """Streams with lens[b] cached positions, rows[b] of them in this batch, over a dense or paged
    cache of either kind. Everything a query must not see is NaN."""

    def __init__(self, heads, kv_heads, lens, rows, page_rows, paged, seed=0, spare_slots=1, pad_rows=2, dev="cuda"):
        import torch
        import transformer_decoder_kv_b200 as pkg
        self.torch, self.pkg, self.dev = torch, pkg, dev
        self.rng = rng = np.random.default_rng(seed)
        self.H, self.HK, self.pr = heads, kv_heads, page_rows
        self.lens, self.rows = list(lens), list(rows)
        B = self.B = len(lens)
        self.pps = max(1, -(-max(max(lens), 1) // page_rows))
        self.n_slots = B + spare_slots
        self.slots = rng.permutation(self.n_slots)[:B].astype(np.int32)
        self.n_pages = self.n_slots * self.pps + (3 if paged else 0)
        self.table = None
        if paged:
            self.table = rng.permutation(self.n_pages)[:self.n_slots * self.pps].astype(np.int32).reshape(-1, self.pps)
        self.start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.n_buf = int(self.start[-1]) + pad_rows
        self.view = pkg.KvView(kv_heads, page_rows, self.pps, self.n_slots, self.n_pages, self.i32(self.table))
        self.batch = self.make_rows(self.lens, self.rows, pad_rows)
        self.k = [rng.standard_normal((n, kv_heads, D)).astype(np.float32) * np.float32(1.5) for n in lens]
        self.v = [rng.standard_normal((n, kv_heads, D)).astype(np.float32) for n in lens]
        self.q = rng.standard_normal((self.n_buf, heads, D)).astype(np.float32)

    def i32(self, a):
        return None if a is None else self.torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(self.dev)

    def f32(self, a):
        return self.torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(self.dev)

    def make_rows(self, lens, rows, pad=0):
        start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        return self.pkg.KvRows(len(lens), self.i32(np.array(lens)), self.i32(self.slots), self.i32(start),
                               int(start[-1]) + pad, max(max(rows), 1))

    def new_cache(self):
        """A 4-bit pool whose every scale is NaN and every code 15."""
        return self.torch.full((self.pkg.kv4_bytes(self.view),), 255, dtype=self.torch.uint8, device=self.dev)

    def write_all(self, cache, upto=None, stream=0):
        """Store positions 0 .. upto[b] - 1 (default: all) of every stream."""
        upto = self.lens if upto is None else upto
        if sum(upto) == 0:
            return
        r = self.make_rows(upto, upto)
        cat = lambda xs: self.f32(np.concatenate([x[:n].reshape(n, self.HK * D) for x, n in zip(xs, upto)]))
        self.pkg.kv4_write(self.view, r, cat(self.k), cat(self.v), cache, stream=stream)

    def f32_pools(self):
        out = []
        for x in (self.k, self.v):
            pool = np.full((self.n_pages, self.HK, self.pr, D), np.nan, np.float32)
            for b in range(self.B):
                for t in range(self.lens[b]):
                    lp = t // self.pr
                    page = self.table[self.slots[b], lp] if self.table is not None else self.slots[b] * self.pps + lp
                    if 0 <= page < self.n_pages:
                        pool[page, :, t % self.pr] = x[b][t]
            out.append(self.f32(pool))
        return out

    def attend(self, kv4, window, sinks, caches, out=None, ws=None, stream=0):
        t = self.torch
        nb = self.pkg.attention_rows_workspace_size(self.view, self.batch, self.H)
        ws = t.randint(0, 255, (nb,), dtype=t.uint8, device=self.dev) if ws is None else ws
        out = t.full((self.n_buf, self.H * D), 7.5, device=self.dev) if out is None else out
        q = self.f32(self.q.reshape(self.n_buf, -1)) if not hasattr(self, "qd") else self.qd
        if kv4:
            self.pkg.attention_kv4(self.view, self.batch, q, caches, self.H, out, ws, nb, window, sinks, stream)
        else:
            self.pkg.attention_window(self.view, self.batch, q, *caches, self.H, out, ws, nb, window, sinks, stream)
        return out

    def reference(self, kv4, window, sinks, hidden=None):
        out = np.full((self.n_buf, self.H, D), 7.5)
        tol = np.zeros((self.n_buf, self.H, 1))
        for b in range(self.B):
            r0, r1 = self.start[b], self.start[b + 1]
            k, v = (kv4_values(self.k[b]), kv4_values(self.v[b])) if kv4 else (self.k[b], self.v[b])
            pos = np.arange(self.lens[b] - self.rows[b], self.lens[b])
            out[r0:r1], tol[r0:r1] = attention(self.q[r0:r1], k, v, pos, window, sinks,
                                               None if hidden is None else hidden[b])
        return out, tol

    def check(self, kv4, window, sinks, hidden=None, what=""):
        if kv4:
            caches = self.new_cache()
            self.write_all(caches)
        else:
            caches = self.f32_pools()
        out = self.attend(kv4, window, sinks, caches)
        self.torch.cuda.synchronize()
        ref, tol = self.reference(kv4, window, sinks, hidden)
        check(out.cpu().numpy().reshape(ref.shape), ref, tol, what)
        return out
