"""The 4-bit cache (dec_kv4_write, dec_kv4_read) and the windowed attentions over 4-bit and f32
caches (dec_attention_kv4, dec_attention_window) against 64-bit references."""
import numpy as np
import pytest

from tests._kvrows import D, Setup, attention, check, kv4_values

pytestmark = pytest.mark.gpu

# heads, kv heads, lens, rows, page_rows, paged
SHAPES = {
    "one_row_one_key": (1, 1, [1], [1], 64, False),
    "short": (6, 6, [1, 2, 15, 16, 17, 63, 64, 65], [1] * 8, 16, True),
    "gqa7": (14, 2, [130, 1, 257, 1000], [1] * 4, 64, True),
    "gqa16": (16, 1, [200, 999], [1, 1], 32, True),
    "wide_group": (40, 1, [70, 333], [1, 1], 32, False),
    "long": (4, 2, [4129, 3, 2048], [1] * 3, 32, True),
    "empty_streams": (2, 2, [0, 40, 0, 5], [0, 1, 0, 1], 16, False),
    "few_rows": (14, 2, [300, 70, 5], [3, 2, 5], 64, True),
    "ragged": (4, 4, [37, 300, 129, 64], [37, 1, 128, 64], 16, True),
    "ragged_gqa": (12, 4, [450, 129, 700], [200, 129, 17], 32, True),
    "prompt": (2, 1, [520], [520], 64, False),
}


def setup(name, **kw):
    h, hk, lens, rows, pr, paged = SHAPES[name]
    return Setup(h, hk, lens, rows, pr, paged, seed=len(name), **kw)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (17, 1), (64, 4), (100, 70), (5000, 3)])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_attention_matches_reference(kv4, shape, window, sinks):
    setup(shape).check(kv4, window, sinks, what=f"{shape} {window} {sinks}")


@pytest.mark.parametrize("shape", SHAPES)
def test_write_then_read_is_the_code_bit_for_bit(shape):
    s = setup(shape)
    cache = s.new_cache()
    s.write_all(cache)
    t = s.torch
    ko, vo = (t.full((s.n_buf, s.HK * D), 7.5, device="cuda") for _ in range(2))
    s.pkg.kv4_read(s.view, s.batch, cache, ko, vo)
    t.cuda.synchronize()
    for got, x in ((ko, s.k), (vo, s.v)):
        got = got.cpu().numpy().reshape(s.n_buf, s.HK, D)
        assert (got[s.start[-1]:] == 7.5).all()          # rows of no stream
        for b in range(s.B):
            want = kv4_values(x[b])[s.lens[b] - s.rows[b]:]
            assert np.array_equal(got[s.start[b]:s.start[b + 1]].astype(np.float64), want)


def _round_trip(rows):
    """rows [n, 64] as the K of one stream (V their negative)."""
    import torch
    import transformer_decoder_kv_b200 as pkg
    n = len(rows)
    view = pkg.KvView(1, 16, -(-n // 16), 1)
    batch = pkg.KvRows(1, torch.tensor([n], dtype=torch.int32, device="cuda"), None,
                       torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, n)
    cache = torch.full((pkg.kv4_bytes(view),), 255, dtype=torch.uint8, device="cuda")
    k = torch.from_numpy(rows).cuda()
    pkg.kv4_write(view, batch, k, -k, cache)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    pkg.kv4_read(view, batch, cache, ko, vo)
    torch.cuda.synchronize()
    return ko.cpu().numpy(), vo.cpu().numpy()


def test_codes_at_borders_ties_and_extremes():
    rng = np.random.default_rng(3)
    rows = []
    for e in (-126, -125, -100, -3, 0, 7, 90, 125):
        for _ in range(40):                          # values on and next to (c + 1/2) s, scale from the maximum
            s = np.float32((1 + rng.integers(0, 128) / 128) * 2.0 ** min(e, 124))
            c = rng.integers(-7, 7, 64) + 0.5
            x = (c * np.float64(s)).astype(np.float32)
            x[::3] = np.nextafter(x[::3], np.float32(np.inf))
            x[1::3] = np.nextafter(x[1::3], np.float32(-np.inf))
            x[5], x[40] = 7 * s, -7 * s
            rows.append(x)
    rows += [np.zeros(64), np.full(64, 1e-45), np.full(64, 2e-38), np.full(64, 3.4e38),
             np.linspace(-1e-37, 1e-37, 64), np.linspace(-3.4e38, 3.4e38, 64)]
    rows = np.stack(rows).astype(np.float32)
    k, v = _round_trip(rows)
    want = kv4_values(rows)
    assert np.array_equal(k.astype(np.float64), want)
    assert np.array_equal(v.astype(np.float64), -want)
    # half a step at most: |x - c s| <= s / 2 <= max |x| / 14 (1 + 2^-8); below 7 2^-126 everything is 0
    amax = np.abs(rows.reshape(-1, 2, 32).astype(np.float64)).max(axis=2, keepdims=True)
    err = np.abs(want - rows).reshape(-1, 2, 32)
    assert (err <= np.maximum(amax / 14 * (1 + 2.0 ** -8), 7.1 * 2.0 ** -126)).all()


def test_groups_that_are_not_finite_read_back_as_nan():
    rows = np.ones((4, 64), np.float32)
    rows[0, 3], rows[1, 40], rows[2, 31] = np.nan, np.inf, -np.inf
    k, _ = _round_trip(rows)
    want = kv4_values(rows)
    assert np.array_equal(np.isnan(k), np.isnan(want)) and np.isnan(k).sum() == 3 * 32
    assert np.array_equal(k[~np.isnan(want)], want[~np.isnan(want)].astype(np.float32))


def test_rows_inside_a_fused_buffer_and_strided_queries():
    s = setup("ragged_gqa")
    t = s.torch
    cache, plain = s.new_cache(), s.new_cache()
    s.write_all(plain)
    n, w = sum(s.lens), s.HK * D
    fused = t.full((n, 3 * w + 4), float("nan"), device="cuda")
    fused[:, w:2 * w] = s.f32(np.concatenate(s.k).reshape(n, -1))
    fused[:, 2 * w:3 * w] = s.f32(np.concatenate(s.v).reshape(n, -1))
    s.pkg.kv4_write(s.view, s.make_rows(s.lens, s.lens), fused[:, w:2 * w], fused[:, 2 * w:3 * w], cache)
    assert t.equal(cache, plain)
    qbuf = t.full((s.n_buf, s.H * D + 8), float("nan"), device="cuda")
    qbuf[:, 4:-4] = s.f32(s.q.reshape(s.n_buf, -1))
    s.qd = qbuf[:, 4:-4]
    obuf = t.full((s.n_buf, s.H * D + 4), 7.5, device="cuda")
    s.attend(True, 100, 4, cache, out=obuf[:, 4:])
    t.cuda.synchronize()
    ref, tol = s.reference(True, 100, 4)
    assert (obuf[:, :4] == 7.5).all()
    check(obuf[:, 4:].cpu().numpy().reshape(ref.shape), ref, tol)


@pytest.mark.parametrize("shape", ["few_rows", "ragged_gqa", "gqa7"])
@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_values_a_query_does_not_see_do_not_reach_it(kv4, shape):
    """NaN and infinities in rows behind the window and in rows only later queries of the same
    stream see; those later queries get what the definition gives."""
    s = setup(shape)
    window, sinks = 64, 2
    for b in range(s.B):
        n, r = s.lens[b], s.rows[b]
        dead = np.arange(n) <= n - r - window
        dead[:sinks] = False
        s.k[b][dead], s.v[b][dead] = np.nan, np.inf
        if r > 2:                       # positions of the batch's own rows: visible to later ones only
            s.v[b][n - 2, :, 7] = np.inf
            s.v[b][n - r // 2, :, 40] = np.nan
            s.k[b][n - 1, :, 3] = np.nan
    s.check(kv4, window, sinks, what=shape)


@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_bad_pages_slots_and_lengths_are_left_out(kv4):
    s = Setup(4, 2, [200, 150, 90, 64], [3, 70, 1, 1], 16, True, seed=9)
    hidden = [np.zeros(n, bool) for n in s.lens]
    for b, lp, bad in ((0, 2, -1), (0, 12, 1 << 30), (1, 5, s.n_pages), (2, 0, -(1 << 31))):
        s.table[s.slots[b], lp] = bad
        hidden[b][lp * 16:(lp + 1) * 16] = True
    s.view = s.pkg.KvView(2, 16, s.pps, s.n_slots, s.n_pages, s.i32(s.table))
    s.check(kv4, 0, 0, hidden)
    caches = None if kv4 else s.f32_pools()
    # slots out of range
    s.slots[0], s.slots[2] = s.n_slots, -1
    s.batch = s.make_rows(s.lens, s.rows, 2)
    if kv4:
        caches = s.new_cache()
        s.write_all(caches)
        ko, vo = (s.torch.full((s.n_buf, s.HK * D), 7.5, device="cuda") for _ in range(2))
        s.pkg.kv4_read(s.view, s.batch, caches, ko, vo)
        assert (ko[:3] == 0).all() and (vo[:3] == 0).all() and (ko[-2:] == 7.5).all()
    out = s.attend(kv4, 0, 0, caches)
    assert (out[:3] == 0).all() and (out[73] == 0).all() and (out[74] != 0).any()


@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_lengths_outside_the_slot_and_row_starts_out_of_range(kv4):
    import torch
    s = Setup(2, 2, [32, 32, 32], [2, 2, 2], 16, False, seed=4, spare_slots=0)
    caches = s.new_cache() if kv4 else s.f32_pools()
    if kv4:
        s.write_all(caches)
    lens = torch.tensor([-5, 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    s.batch = s.pkg.KvRows(3, lens, s.i32(s.slots), s.i32([0, 2, 4, 6]), s.n_buf, 2)
    out = s.attend(kv4, 0, 0, caches)
    torch.cuda.synchronize()
    assert (out[:3] == 0).all()                    # below position 0
    ref, tol = attention(s.q[3:4], *(kv4_values(x[1]) if kv4 else x[1] for x in (s.k, s.v)), [0], 0, 0)
    check(out[3:4].cpu().numpy().reshape(ref.shape), ref, tol)
    ref, tol = attention(s.q[4:6], *(kv4_values(x[2]) if kv4 else x[2] for x in (s.k, s.v)), [40, 41], 0, 0)
    check(out[4:6].cpu().numpy().reshape(ref.shape), ref, tol)
    s.batch = s.pkg.KvRows(3, s.i32([32, 32, 32]), s.i32(s.slots), s.i32([-7, 2, 1, 1 << 30]), s.n_buf, 2)
    out = s.attend(kv4, 0, 0, caches)              # stream 1 is empty, the others are clipped
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and (out[4:] == 7.5).all() if s.n_buf > 4 else True


@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_extreme_scores_and_sums(kv4):
    """Scores far apart, large and tiny rows, a zero query, infinite queries (zeros, as in dec_attention)."""
    s = setup("few_rows")
    s.q[0] *= 1e4
    s.q[1] *= 1e-30
    s.q[2] = 0
    s.q[3, 0, 5] = np.inf
    s.q[4, 1, 9] = np.nan
    s.k[0][10:20] *= 1e4
    s.v[0][30:40] *= 1e-20
    s.v[0][50] *= 1e18
    s.k[1][:] = 0
    ref, _ = s.reference(kv4, 0, 0)
    assert (ref[3, 0] == 0).all() and (ref[4, 1] == 0).all()
    s.check(kv4, 0, 0)


def test_chunked_prompt_then_tokens_write_read_and_attend_together():
    """A prompt in chunks and then single tokens, as a serving loop stores and attends them, with
    some streams a step behind: every step's outputs are the reference's, and the cache ends as
    one call over everything would have left it."""
    s = setup("ragged_gqa")
    t = s.torch
    cache, whole = s.new_cache(), s.new_cache()
    s.write_all(whole)
    done = [0] * s.B
    steps = [[100, 0, 33], [100, 128, 600], [1, 0, 1], [1, 1, 1]]
    final = s.lens
    for step in steps:
        step = [min(x, final[b] - done[b]) for b, x in enumerate(step)]
        done = [d + x for d, x in zip(done, step)]
        s.rows, s.lens = step, done
        s.start = np.concatenate([[0], np.cumsum(step)]).astype(np.int32)
        s.n_buf = max(int(s.start[-1]), 1)
        s.batch = s.make_rows(done, step, 0 if sum(step) else 1)
        cat = lambda xs: s.f32(np.concatenate([x[d - n:d].reshape(n, s.HK * D) for x, d, n in zip(xs, done, step)]))
        s.pkg.kv4_write(s.view, s.batch, cat(s.k), cat(s.v), cache)
        s.q = s.rng.standard_normal((s.n_buf, s.H, D)).astype(np.float32)
        out = s.attend(True, 150, 4, cache)
        ref, tol = [], []
        for b in range(s.B):
            o, e = attention(s.q[s.start[b]:s.start[b + 1]], kv4_values(s.k[b][:done[b]]), kv4_values(s.v[b][:done[b]]),
                             np.arange(done[b] - step[b], done[b]), 150, 4)
            ref.append(o), tol.append(e)
        check(out.cpu().numpy().reshape(s.n_buf, s.H, D), np.concatenate(ref), np.concatenate(tol), f"step {step}")
    s.lens = done
    ko, vo, kw, vw = (t.zeros((sum(done), s.HK * D), device="cuda") for _ in range(4))
    every = s.make_rows(done, done)
    s.pkg.kv4_read(s.view, every, cache, ko, vo)
    s.pkg.kv4_read(s.view, every, whole, kw, vw)
    assert t.equal(ko, kw) and t.equal(vo, vw)


@pytest.mark.parametrize("shape", ["gqa7", "long", "ragged_gqa"])
@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_repeated_calls_streams_and_graph_replays_give_the_same_bits(kv4, shape):
    s = setup(shape)
    t = s.torch
    caches = s.new_cache() if kv4 else s.f32_pools()
    if kv4:
        s.write_all(caches)
    s.qd = s.f32(s.q.reshape(s.n_buf, -1))
    first = s.attend(kv4, 100, 2, caches)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    nb = s.pkg.attention_rows_workspace_size(s.view, s.batch, s.H)
    ws = t.full((nb,), 255, dtype=t.uint8, device="cuda")
    out = t.full_like(first, 7.5)
    t.cuda.synchronize()
    with t.cuda.stream(side):
        s.attend(kv4, 100, 2, caches, out=out, ws=ws, stream=side.cuda_stream)
    side.synchronize()
    assert t.equal(out, first)
    # two captured graphs that share the workspace, replayed one after the other
    graphs, outs = [], []
    for window in (100, 30):
        g, o = t.cuda.CUDAGraph(), t.full_like(first, 7.5)
        t.cuda.synchronize()
        with t.cuda.graph(g, stream=side):
            s.attend(kv4, window, 2, caches, out=o, ws=ws, stream=t.cuda.current_stream().cuda_stream)
        graphs.append(g), outs.append(o)
    other = s.attend(kv4, 30, 2, caches)
    for _ in range(2):
        for g in graphs:
            g.replay()
    t.cuda.synchronize()
    assert t.equal(outs[0], first) and t.equal(outs[1], other)


@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_replay_follows_rewritten_lengths(kv4):
    s = setup("gqa7")
    t = s.torch
    caches = s.new_cache() if kv4 else s.f32_pools()
    if kv4:
        s.write_all(caches)
    s.qd = s.f32(s.q.reshape(s.n_buf, -1))
    nb = s.pkg.attention_rows_workspace_size(s.view, s.batch, s.H)
    ws = t.empty((nb,), dtype=t.uint8, device="cuda")
    out = t.full((s.n_buf, s.H * D), 7.5, device="cuda")
    g, side = t.cuda.CUDAGraph(), t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.graph(g, stream=side):
        s.attend(kv4, 0, 0, caches, out=out, ws=ws, stream=t.cuda.current_stream().cuda_stream)
    s.lens = [n // 2 + 1 if n > 1 else 1 for n in s.lens]
    s.batch.keep[0].copy_(s.i32(s.lens))
    s.k, s.v = [x[:n] for x, n in zip(s.k, s.lens)], [x[:n] for x, n in zip(s.v, s.lens)]
    g.replay()
    t.cuda.synchronize()
    ref, tol = s.reference(kv4, 0, 0)
    check(out.cpu().numpy().reshape(ref.shape), ref, tol)


def test_window_zero_sinks_zero_equals_dec_attention_within_rounding():
    import torch
    from transformer_decoder_kv_b200 import attention as dec_attention, attention_workspace_size
    B, H, ld = 3, 4, 300
    lens = [1, 200, 300]
    s = Setup(H, H, lens, [1] * B, ld, False, seed=2, spare_slots=0, pad_rows=0)
    s.slots = np.arange(B, dtype=np.int32)
    s.batch = s.make_rows(lens, [1] * B)
    k, v = s.f32_pools()
    out = s.attend(False, 0, 0, (k, v))
    nb = attention_workspace_size(B, H, ld)
    ws = torch.zeros(nb // 4 + 1, dtype=torch.int32, device="cuda")
    want = torch.empty((B, H, D), device="cuda")
    dec_attention(s.f32(s.q), k, v, s.i32(lens), B, H, ld, want, ws, nb)
    torch.cuda.synchronize()
    _, tol = s.reference(False, 0, 0)
    check(out.cpu().numpy().reshape(B, H, D), want.cpu().numpy().astype(np.float64), 2 * tol)


@pytest.mark.parametrize("rows", [1, 40, 130])
@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_pools_beyond_32_bit_offsets(kv4, rows):
    """The same pages at the bottom of a small pool and at the top of one whose offsets pass 32 bits."""
    import torch
    import transformer_decoder_kv_b200 as pkg
    HK, H, pr, n_len = 8, 16, 64, 300
    far = 125_000 if kv4 else 70_000             # 36,864 bytes (kv4), 32,768 floats (f32) a page
    assert far * (36_864 if kv4 else 32_768) > 1 << (32 if kv4 else 31)
    g = torch.Generator(device="cuda").manual_seed(5)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = (torch.randn((n_len, HK * D), device="cuda", generator=g) for _ in range(2))
    q = torch.randn((rows, H * D), device="cuda", generator=g)
    outs = []
    for n_pages in (5, far):
        table = i32([[n_pages - 1 - i for i in range(5)]])
        view = pkg.KvView(HK, pr, 5, 1, n_pages, table)
        batch = pkg.KvRows(1, i32([n_len]), None, i32([0, rows]), rows, rows)
        every = pkg.KvRows(1, i32([n_len]), None, i32([0, n_len]), n_len, n_len)
        nb = pkg.attention_rows_workspace_size(view, batch, H)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        if kv4:
            cache = torch.empty(pkg.kv4_bytes(view), dtype=torch.uint8, device="cuda")
            pkg.kv4_write(view, every, k, v, cache)
            ko, vo = torch.empty_like(k), torch.empty_like(v)
            pkg.kv4_read(view, every, cache, ko, vo)
            assert np.array_equal(ko.cpu().numpy().reshape(-1, D), kv4_values(k.cpu().numpy().reshape(-1, D)))
            pkg.attention_kv4(view, batch, q, cache, H, out, ws, nb, 100, 3)
        else:
            pools = []
            for x in (k, v):
                pool = torch.empty((n_pages, HK, pr, D), device="cuda")
                for lp in range(5):
                    part = x[lp * pr:(lp + 1) * pr].view(-1, HK, D)
                    pool[n_pages - 1 - lp, :, :len(part)] = part.transpose(0, 1)
                pools.append(pool)
            pkg.attention_window(view, batch, q, *pools, H, out, ws, nb, 100, 3)
        outs.append(out)
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("shape", ["gqa7", "ragged_gqa"])
@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_calls_that_overlap_on_two_streams(kv4, shape):
    s = setup(shape)
    t = s.torch
    caches = s.new_cache() if kv4 else s.f32_pools()
    if kv4:
        s.write_all(caches)
    s.qd = s.f32(s.q.reshape(s.n_buf, -1))
    want = [s.attend(kv4, w, 2, caches) for w in (0, 70)]
    streams = [t.cuda.Stream() for _ in range(2)]
    nb = s.pkg.attention_rows_workspace_size(s.view, s.batch, s.H)
    ws = [t.empty(nb, dtype=t.uint8, device="cuda") for _ in range(2)]
    outs = [t.full_like(want[0], 7.5) for _ in range(2)]
    t.cuda.synchronize()
    for _ in range(20):
        for i, w in enumerate((0, 70)):
            s.attend(kv4, w, 2, caches, out=outs[i], ws=ws[i], stream=streams[i].cuda_stream)
    t.cuda.synchronize()
    assert t.equal(outs[0], want[0]) and t.equal(outs[1], want[1])


@pytest.mark.parametrize("kv4", [True, False], ids=["kv4", "f32"])
def test_shared_slots_shared_pages_and_a_row_limit(kv4):
    """One slot in two streams, two slots with the same first pages, and a stream with more rows than
    max_rows: its first ones are processed, the others left."""
    import torch
    s = Setup(4, 2, [100, 100], [2, 2], 16, True, seed=1, pad_rows=0)
    caches = s.new_cache() if kv4 else s.f32_pools()
    if kv4:
        s.write_all(caches)
    s.q[2:4] = s.q[:2]
    table = s.table.copy()
    table[s.slots[1], :] = table[s.slots[0], :]
    for view, slots in ((s.view, [s.slots[0]] * 2), (s.pkg.KvView(2, 16, s.pps, s.n_slots, s.n_pages, s.i32(table)), s.slots)):
        s.view = view
        s.batch = s.pkg.KvRows(2, s.i32([100, 100]), s.i32(slots), s.i32([0, 2, 4]), 4, 2)
        out = s.attend(kv4, 0, 0, caches)
        assert torch.equal(out[:2], out[2:]) and torch.isfinite(out).all()
    s.batch = s.pkg.KvRows(2, s.i32([100, 100]), s.i32(slots), s.i32([0, 2, 4]), 4, 1)
    out = s.attend(kv4, 0, 0, caches)
    assert (out[1] == 7.5).all() and (out[3] == 7.5).all()
    ref, tol = attention(s.q[:1], *(kv4_values(x[0]) if kv4 else x[0] for x in (s.k, s.v)), [98], 0, 0)
    check(out[:1].cpu().numpy().reshape(ref.shape), ref, tol)


def test_largest_batch():
    import torch
    import transformer_decoder_kv_b200 as pkg
    B = 65535
    view = pkg.KvView(1, 16, 1, 1)
    lens = torch.arange(B, dtype=torch.int32, device="cuda") % 17
    slots = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache = torch.empty(pkg.kv4_bytes(view), dtype=torch.uint8, device="cuda")
    kv = torch.randn((16, D), device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pkg.kv4_write(view, pkg.KvRows(1, i32([16]), None, i32([0, 16]), 16, 16), kv, kv, cache)
    batch = pkg.KvRows(B, lens, slots)
    q = torch.randn((1, D), device="cuda").expand(B, D).contiguous()
    out = torch.full((B, D), 7.5, device="cuda")
    nb = pkg.attention_rows_workspace_size(view, batch, 1)
    pkg.attention_kv4(view, batch, q, cache, 1, out, torch.empty(nb, dtype=torch.uint8, device="cuda"), nb)
    assert (out[lens == 0] == 0).all()
    for n in (1, 16):
        rows = out[lens == n]
        assert (rows == rows[0]).all()
    values = kv4_values(kv.cpu().numpy())
    assert np.allclose(out[1].cpu().numpy(), values[0], rtol=1e-5)
