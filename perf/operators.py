"""Measured workloads of the row-batch cache operators: kv4_write, kv4_read, attention_kv4 and
attention_window.

Each case is one pass of one operator as a serving program calls it. `run` computes it either
in its plain form (elementary torch operations) or, with `own` set, through the package's
entry points; `exact` gives the same outputs from the definitions in 64 bits.

The operators share one description of a batch: stream b owns rows[b] consecutive rows of the
row buffers, which sit at positions lens[b] - rows[b] .. lens[b] - 1 of cache slot slots[b].

  kv4 code   per (row, K/V head, group of 32 dims): a = max |x|, s = bf16(a / 7) (0 below the
             smallest normal number), c = x / s rounded to the nearest integer, ties to even;
             the cache stands for c s
  attention  query row at position p, head h: s_j = (q . k_j) / 8 over the keys j <= p with
             j > p - window (window 0: all) or j < sinks, softmax, sum_j p_j v_j
"""
import math

import torch

own = False

D = 64          # head dim
GROUP = 32      # dims per scale
DEV = "cuda"


# ---- the cases ------------------------------------------------------------------------------

def _case(name, op, batch, heads, kv_heads, len_min, len_max, rows_min=1, rows_max=1, page_rows=64, paged=False,
          window=0, sinks=0, pad_rows=0):
    c = dict(op=op, batch=batch, heads=heads, kv_heads=kv_heads, len_min=len_min, len_max=len_max, rows_min=rows_min,
             rows_max=rows_max, page_rows=page_rows, paged=paged, window=window, sinks=sinks, pad_rows=pad_rows)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step's new rows of 64 streams, 16 K/V heads, stored and handed back (latency)
        _case("kv4_write_step", "kv4_write", 64, 16, 16, 17, 4129, page_rows=16, paged=True),
        # ragged prompts of an admission burst, up to 2000 rows each, with padding rows behind
        _case("kv4_write_prompts", "kv4_write", 8, 16, 16, 37, 2000, 37, 2000, pad_rows=3),
        # the tail of one stream's cache, two K/V heads (latency)
        _case("kv4_read_tail", "kv4_read", 1, 14, 2, 333, 333, 301, 301),
        # whole streams read back into f32 rows, e.g. to move them to an unquantised cache
        _case("kv4_read_streams", "kv4_read", 16, 14, 2, 1000, 4129, 1000, 4129, page_rows=32, paged=True),
        # the first steps of one short stream: launch latency is all there is
        _case("attn_kv4_first", "attention_kv4", 1, 14, 2, 17, 17),
        # the default serving step's caches: 64 streams of about 4096 rows, one K/V head per query head
        _case("attn_kv4_step", "attention_kv4", 64, 16, 16, 4000, 4129, page_rows=64, paged=True),
        # a few long streams over grouped heads, everything visible
        _case("attn_kv4_long", "attention_kv4", 16, 14, 2, 30001, 32768, page_rows=32, paged=True),
        # many long streams with a sliding window and four sinks
        _case("attn_kv4_window", "attention_kv4", 128, 14, 2, 700, 32768, page_rows=16, paged=True, window=1024,
              sinks=4),
        # prompt chunks of up to 128 rows next to short ones, over grown caches
        _case("attn_kv4_chunks", "attention_kv4", 16, 14, 2, 513, 4129, 5, 128, page_rows=64, paged=True, pad_rows=7),
        # one short unquantised stream, small window (latency)
        _case("attn_window_first", "attention_window", 1, 6, 6, 448, 448, page_rows=448, window=64, sinks=1),
        # an unquantised 448-row cache per stream, batch 32 of 20 heads, half of it in the window
        _case("attn_window_step", "attention_window", 32, 20, 20, 100, 448, page_rows=448, window=224, sinks=4),
        # one whole prompt over the unquantised paged cache
        _case("attn_window_prompt", "attention_window", 1, 16, 16, 2040, 2040, 2040, 2040, page_rows=64, paged=True,
              window=512, sinks=4),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["kv4_write", "kv4_read", "attention_kv4", "attention_kv4", "attention_window",
                     "attention_window"])
    heads, kv_heads = rng.choice([(16, 16), (14, 2), (14, 2), (20, 20), (8, 8), (6, 6), (12, 4), (16, 2), (4, 1)])
    paged = rng.random() < 0.6
    page_rows = rng.choice([16, 32, 64])
    long_rows = rng.random() < 0.45
    if op in ("kv4_write", "kv4_read"):
        budget = 120000                    # head rows
        rows_max = _logint(rng, 2, 4000) if long_rows else 1
        batch = _logint(rng, 1, max(1, min(128, budget // (rows_max * kv_heads))))
        len_max = rows_max + _logint(rng, 1, 2000)
        window, sinks = 0, 0
    elif long_rows:
        window = rng.choice([0, _logint(rng, 1, 1024)])
        sinks = rng.choice([0, 1, 4, 64])
        rows_max = _logint(rng, 2, 1024)
        len_max = rows_max + _logint(rng, 1, 2048)
        cost = rows_max * heads * min(len_max, window or len_max)     # query-key pairs of a stream
        limit = 24_000_000 if op == "attention_kv4" else 12_000_000
        batch = max(1, min(16, int(limit // cost)))
        if cost > limit:
            rows_max = max(2, int(rows_max * limit / cost))
    else:
        window = rng.choice([0, _logint(rng, 1, 2048)])
        sinks = rng.choice([0, 1, 4, 64])
        rows_max = 1
        len_max = _logint(rng, 1, 32768 if op == "attention_kv4" else 4129)
        budget = 4_000_000 if op == "attention_kv4" else 600_000       # cached head rows
        batch = _logint(rng, 1, max(1, min(128, budget // (len_max * kv_heads))))
    if op == "attention_window" and not paged:
        page_rows = len_max + rng.choice([0, 1, 37])
    rows_min = max(1, int(rows_max * rng.uniform(0.05, 1.0)))
    len_min = min(len_max, rows_max + int((len_max - rows_max) * rng.random()))
    return _case("", op, batch, heads, kv_heads, max(1, len_min), len_max, rows_min, rows_max, page_rows, paged, window,
                 sinks, rng.choice([0, 0, 3]) if rows_max > 1 else 0)


def _spread(lo, hi, n, salt):
    """n integers in [lo, hi], spread over it, both ends among them where n allows."""
    out = [lo + int((hi - lo + 1) * ((0.6180339887498949 * (i + 1) + salt) % 1.0)) for i in range(n)]
    out[0] = hi
    if n > 1:
        out[n // 2] = lo
    return out


def _geometry(case):
    lens = _spread(case["len_min"], case["len_max"], case["batch"], 0.0)
    rows = [min(r, n) for r, n in zip(_spread(case["rows_min"], case["rows_max"], case["batch"], 0.31), lens)]
    ragged = case["rows_max"] > 1
    cap_pages = -(-case["len_max"] // case["page_rows"])
    return lens, rows, ragged, cap_pages


def _visible(pos, window, sinks):
    """Keys a query at position pos attends."""
    if pos < 0:
        return 0
    lo = max(0, pos - window + 1) if window else 0
    return (pos - lo + 1) + min(sinks, lo)


def work(case):
    lens, rows, _, _ = _geometry(case)
    H, HK, n = case["heads"], case["kv_heads"], sum(rows)
    if case["op"] == "kv4_write":      # rows in, codes and scales stored, rows handed back
        return {"bytes": n * HK * 2 * (256 + 36 + 256), "flops": n * HK * 2 * D * 6}
    if case["op"] == "kv4_read":
        return {"bytes": n * HK * 2 * (36 + 256), "flops": n * HK * 2 * D}
    per_key = 72 if case["op"] == "attention_kv4" else 512
    w, s = case["window"], case["sinks"]
    keys = pairs = 0
    for ln, r in zip(lens, rows):
        lo = max(0, ln - r - w + 1) if w else 0
        keys += ln - lo + min(s, lo)
        pairs += sum(_visible(p, w, s) for p in range(ln - r, ln))
    return {"bytes": keys * HK * per_key + 2 * n * H * D * 4, "flops": pairs * H * 4 * D}


# ---- inputs ---------------------------------------------------------------------------------

def _inputs(case, seed):
    """Everything drawn from the seed: slot order, page table, rows and queries."""
    lens, rows, ragged, cap_pages = _geometry(case)
    B, HK = case["batch"], case["kv_heads"]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    i = {"slots": torch.randperm(B, generator=g, device=DEV, dtype=torch.int64).to(torch.int32)}
    n_pages = B * cap_pages
    i["table"] = None
    if case["paged"]:
        i["table"] = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).view(B, cap_pages)
    i["n_pages"] = n_pages
    # per-channel magnitudes: a few channels of K stand out, as they do behind rotary positions
    mag = torch.exp(0.5 * torch.randn((HK, D), generator=g, device=DEV))
    n = sum(rows)

    def rows_of(count, scale):
        return (torch.randn((count, HK, D), generator=g, device=DEV) * scale).view(count, HK * D)

    if case["op"] == "kv4_write":
        i["k"], i["v"] = rows_of(n + case["pad_rows"], mag), rows_of(n + case["pad_rows"], 1.0)
    else:
        total = sum(lens)
        i["k"], i["v"] = rows_of(total, mag), rows_of(total, 1.0)
        if case["op"] != "kv4_read":
            i["q"] = torch.randn((n + case["pad_rows"], case["heads"] * D), generator=g, device=DEV)
    return i


def _starts(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


def _pages(case, i, b_slot, cap_pages):
    """Physical pages of one slot, in order."""
    if i["table"] is None:
        return torch.arange(cap_pages, device=DEV) + b_slot * cap_pages
    return i["table"][b_slot].long()


def _quantise(x):
    """Codes and scales of f32 rows [n, HK, 64], the quotient in 64 bits (values next to a border)."""
    g = x.view(x.shape[0], x.shape[1], D // GROUP, GROUP)
    s = (g.abs().amax(-1) / 7.0).to(torch.bfloat16).float()
    s = torch.where(s < 2.0 ** -126, torch.zeros_like(s), s)
    q = torch.round(g.double() / torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1))
    q = torch.where(s.unsqueeze(-1) > 0, q, torch.zeros_like(q)).clamp(-7, 7)
    return q.to(torch.int8).view_as(x), s


def _dequantise(c, s):
    return (c.view(*c.shape[:-1], D // GROUP, GROUP).float() * s.unsqueeze(-1)).view(c.shape)


def _where(case, i, b_slot, positions, cap_pages):
    """Page and row within it of each position of a slot."""
    pages = _pages(case, i, b_slot, cap_pages)
    return pages[positions // case["page_rows"]], positions % case["page_rows"]


def prepare(case, seed):
    lens, rows, ragged, cap_pages = _geometry(case)
    i = _inputs(case, seed)
    B, HK, H, pr = case["batch"], case["kv_heads"], case["heads"], case["page_rows"]
    n_buf = sum(rows) + case["pad_rows"]
    st = {"case": case, "i": i, "lens": lens, "rows": rows, "cap_pages": cap_pages, "slots": i["slots"].tolist()}
    quantised = case["op"] != "attention_window"
    if own:
        import transformer_decoder_kv_b200 as pkg
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        st["pkg"] = pkg
        st["view"] = pkg.KvView(HK, pr, cap_pages, B, i["n_pages"], i["table"])
        st["batch"] = pkg.KvRows(B, dev(lens), i["slots"], dev(_starts(rows)) if ragged else None, n_buf,
                                 case["rows_max"])
        if quantised:
            st["cache"] = torch.zeros(pkg.kv4_bytes(st["view"]), dtype=torch.uint8, device=DEV)
        if case["op"] in ("kv4_read", "attention_kv4"):
            every = pkg.KvRows(B, dev(lens), i["slots"], dev(_starts(lens)), sum(lens), max(lens))
            pkg.kv4_write(st["view"], every, i["k"], i["v"], st["cache"], scale="product")
        if case["op"] in ("attention_kv4", "attention_window"):
            nb = pkg.attention_rows_workspace_size(st["view"], st["batch"], H)
            st["ws"] = torch.zeros((nb + 3) // 4, dtype=torch.int32, device=DEV)
            st["out"] = torch.zeros((n_buf, H * D), device=DEV)
        else:
            st["ko"] = torch.zeros((n_buf, HK * D), device=DEV)
            st["vo"] = torch.zeros((n_buf, HK * D), device=DEV)
    if quantised and not own:
        for x in "kv":
            st[x + "c"] = torch.zeros((i["n_pages"], HK, pr, D), dtype=torch.int8, device=DEV)
            st[x + "s"] = torch.zeros((i["n_pages"], HK, pr, D // GROUP), device=DEV)
    if case["op"] == "attention_window":
        for x in "kv":
            st[x] = torch.zeros((i["n_pages"], HK, pr, D), device=DEV)
    if not (own and quantised) and case["op"] != "kv4_write":
        first = _starts(lens)
        for b in range(B):
            pos = torch.arange(lens[b], device=DEV)
            page, r = _where(case, i, st["slots"][b], pos, cap_pages)
            for x in "kv":
                src = i[x][first[b]:first[b + 1]].view(-1, HK, D)
                if quantised:
                    c, s = _quantise(src)
                    st[x + "c"][page, :, r] = c
                    st[x + "s"][page, :, r] = s
                else:
                    st[x][page, :, r] = src
    if case["op"] != "kv4_write":     # the program keeps the cache, not the rows it came from
        del i["k"], i["v"]
    return st


# ---- one pass -------------------------------------------------------------------------------

def _run_own(st):
    case, pkg, i = st["case"], st["pkg"], st["i"]
    if case["op"] == "kv4_write":
        pkg.kv4_write(st["view"], st["batch"], i["k"], i["v"], st["cache"], scale="product")
        pkg.kv4_read(st["view"], st["batch"], st["cache"], st["ko"], st["vo"])
        return st["ko"], st["vo"]
    if case["op"] == "kv4_read":
        pkg.kv4_read(st["view"], st["batch"], st["cache"], st["ko"], st["vo"])
        return st["ko"], st["vo"]
    if case["op"] == "attention_kv4":
        pkg.attention_kv4(st["view"], st["batch"], i["q"], st["cache"], case["heads"], st["out"], st["ws"],
                          st["ws"].numel() * 4, window=case["window"], sinks=case["sinks"])
    else:
        pkg.attention_window(st["view"], st["batch"], i["q"], st["k"], st["v"], case["heads"], st["out"], st["ws"],
                             st["ws"].numel() * 4, window=case["window"], sinks=case["sinks"])
    return st["out"]


def _run_plain(st):
    case, i = st["case"], st["i"]
    lens, rows, cap_pages = st["lens"], st["rows"], st["cap_pages"]
    HK, H, n_buf = case["kv_heads"], case["heads"], sum(rows) + case["pad_rows"]
    first = _starts(rows)
    if case["op"] in ("kv4_write", "kv4_read"):
        outs = []
        for x in "kv":
            o = torch.zeros((n_buf, HK * D), device=DEV)
            for b in range(case["batch"]):
                pos = torch.arange(lens[b] - rows[b], lens[b], device=DEV)
                page, r = _where(case, i, st["slots"][b], pos, cap_pages)
                if case["op"] == "kv4_write":
                    c, s = _quantise(i[x][first[b]:first[b + 1]].view(-1, HK, D))
                    st[x + "c"][page, :, r] = c
                    st[x + "s"][page, :, r] = s
                o[first[b]:first[b + 1]] = _dequantise(st[x + "c"][page, :, r], st[x + "s"][page, :, r]).view(-1, HK * D)
            outs.append(o)
        return tuple(outs)
    out = torch.zeros((n_buf, H * D), device=DEV)
    w, sinks = case["window"], case["sinks"]
    for b in range(case["batch"]):
        if rows[b] == 0:
            continue
        pos = torch.arange(lens[b], device=DEV)
        lo = max(0, lens[b] - rows[b] - w + 1) if w else 0
        if lo > sinks:                    # keys no row of the stream can see are not read
            pos = torch.cat([pos[:sinks], pos[lo:]])
        page, r = _where(case, i, st["slots"][b], pos, cap_pages)
        if case["op"] == "attention_kv4":
            k = _dequantise(st["kc"][page, :, r], st["ks"][page, :, r])
            v = _dequantise(st["vc"][page, :, r], st["vs"][page, :, r])
        else:
            k, v = st["k"][page, :, r], st["v"][page, :, r]
        q = i["q"][first[b]:first[b + 1]].view(rows[b], HK, H // HK, D)
        p0 = torch.arange(lens[b] - rows[b], lens[b], device=DEV)
        keep = pos[None, :] <= p0[:, None]
        if w:
            keep &= (pos[None, :] > p0[:, None] - w) | (pos[None, :] < sinks)
        s = torch.einsum("rhgd,nhd->hgrn", q, k) * 0.125
        s = s.masked_fill(~keep, float("-inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        out[first[b]:first[b + 1]] = torch.einsum("hgrn,nhd->rhgd", p, v).reshape(rows[b], H * D)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits ----------------------------------------------------------------

def _exact_values(x, heads):
    """What the 4-bit cache stands for, of f32 rows [n, heads * 64]."""
    y = x.to(torch.float64).reshape(-1, heads, 2, 32)
    a = y.abs().max(dim=3, keepdim=True).values
    s = (a / 7.0).to(torch.float32).to(torch.bfloat16).to(torch.float64)
    live = s >= 2.0 ** -126
    codes = torch.where(live, (y / torch.where(live, s, torch.ones_like(s))).round(), torch.zeros_like(y))
    return (codes * torch.where(live, s, torch.zeros_like(s))).reshape(-1, heads, 64)


def exact(case, seed):
    lens, rows, _, _ = _geometry(case)
    x = _inputs(case, seed)
    hk, h, total = case["kv_heads"], case["heads"], sum(rows)
    ends, key_ends = _starts(rows), _starts(lens)
    if case["op"] == "kv4_write":
        res = []
        for name in ("k", "v"):
            o = torch.zeros((total + case["pad_rows"], hk * 64), dtype=torch.float64, device=DEV)
            o[:total] = _exact_values(x[name][:total], hk).reshape(total, hk * 64)
            res.append(o)
        return tuple(res)
    if case["op"] == "kv4_read":
        res = []
        for name in ("k", "v"):
            o = torch.zeros((total + case["pad_rows"], hk * 64), dtype=torch.float64, device=DEV)
            for b in range(case["batch"]):
                tail = x[name][key_ends[b + 1] - rows[b]:key_ends[b + 1]]
                o[ends[b]:ends[b + 1]] = _exact_values(tail, hk).reshape(rows[b], hk * 64)
            res.append(o)
        return tuple(res)
    o = torch.zeros((total + case["pad_rows"], h, 64), dtype=torch.float64, device=DEV)
    for b in range(case["batch"]):
        ks, vs = x["k"][key_ends[b]:key_ends[b + 1]], x["v"][key_ends[b]:key_ends[b + 1]]
        if case["op"] == "attention_kv4":
            ks, vs = _exact_values(ks, hk), _exact_values(vs, hk)
        else:
            ks, vs = ks.double().reshape(-1, hk, 64), vs.double().reshape(-1, hk, 64)
        q = x["q"][ends[b]:ends[b + 1]].double().reshape(rows[b], h, 64)
        j = torch.arange(lens[b], device=DEV).unsqueeze(0)
        p = torch.arange(lens[b] - rows[b], lens[b], device=DEV).unsqueeze(1)
        hidden = j > p
        if case["window"]:
            hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
        for head in range(h):
            kv = head // (h // hk)
            score = (q[:, head] @ ks[:, kv].T / 8.0).masked_fill(hidden, -math.inf)
            o[ends[b]:ends[b + 1], head] = torch.softmax(score, dim=1) @ vs[:, kv]
    return o.reshape(-1, h * 64)
