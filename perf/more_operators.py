"""The softmax layer's paged cache of keys and values, as calls that can be
measured one at a time.

A cache holds pages [pages, H, page_rows, 64]; row j of sequence s stands in
page table[s, j // page_rows].  Pages are bf16, or e4m3 with a power of two for
every row and head.  The packed rows row_cu[s] .. row_cu[s+1] of a call are the
last ones of the sequence's seq_len[s].

Three operators:

* ``write``: new rows of k and v into their pages, quantised on the way;
* ``read``: rows of the cache back into packed k and v;
* ``attend``: softmax attention of each sequence's last rows (one token, some
  drafted ones, a chunk of a prompt) over its cached rows up to each of them.

``run`` computes them in plain torch operations, or, where ``own`` is set, by
this package's calls.
"""
import math

import numpy as np
import torch

own = False
D = 64


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The newest token of eight sequences goes into the cache: latency counts.
        dict(name="write 8 tokens", op="write", rows="bf16", cache="e4m3", Hk=16, page=64, seqs=8, len_lo=500, len_hi=18000,
             row_lo=1, row_hi=1, long=0, layout=0),
        # Four prompts of a pass, in fp32, into a quantised cache.
        dict(name="write four prompts", op="write", rows="f32", cache="e4m3", Hk=16, page=64, seqs=4, len_lo=3000,
             len_hi=18000, row_lo=0, row_hi=0, long=4, layout=0),
        # One kept view of 7,400 rows read back for the branches that are scored over it.
        dict(name="read one view", op="read", rows="bf16", cache="e4m3", Hk=16, page=64, seqs=1, len_lo=7400, len_hi=7400,
             row_lo=0, row_hi=0, long=1, layout=0),
        # Sixteen kept views out of small pages.
        dict(name="read sixteen views", op="read", rows="bf16", cache="bf16", Hk=16, page=16, seqs=16, len_lo=500,
             len_hi=18000, row_lo=0, row_hi=0, long=16, layout=0),
        # One sequence's next token behind a prompt of 7,400: latency counts.
        dict(name="attend one token", op="attend", rows="bf16", cache="bf16", Hk=16, group=1, page=64, seqs=1, len_lo=7401,
             len_hi=7401, row_lo=1, row_hi=1, long=0, layout=0),
        # One token behind a very long context, few key heads, quantised: the work of one row over the whole card.
        dict(name="attend one token, 131,072", op="attend", rows="bf16", cache="e4m3", Hk=2, group=8, page=128, seqs=1,
             len_lo=131072, len_hi=131072, row_lo=1, row_hi=1, long=0, layout=0),
        # A ragged decode batch over a quantised cache.
        dict(name="attend 61 tokens", op="attend", rows="bf16", cache="e4m3", Hk=16, group=1, page=64, seqs=61, len_lo=500,
             len_hi=18000, row_lo=1, row_hi=1, long=0, layout=0),
        # A large decode batch with four query heads to a key head, in small pages.
        dict(name="attend 128 tokens, grouped", op="attend", rows="bf16", cache="bf16", Hk=8, group=4, page=16, seqs=128,
             len_lo=500, len_hi=18000, row_lo=1, row_hi=1, long=0, layout=0),
        # Four drafted tokens of each of 24 sequences checked in one call.
        dict(name="attend 24 x 4 drafted", op="attend", rows="bf16", cache="bf16", Hk=4, group=4, page=32, seqs=24,
             len_lo=500, len_hi=18000, row_lo=4, row_hi=4, long=0, layout=0),
        # A chunk of 512 new rows behind a view of 7,400.
        dict(name="attend chunk of 512", op="attend", rows="bf16", cache="bf16", Hk=16, group=1, page=64, seqs=1, len_lo=7912,
             len_hi=7912, row_lo=512, row_hi=512, long=1, layout=0),
        # A large chunk far into a long prompt, grouped heads, quantised cache.
        dict(name="attend chunk of 2,048", op="attend", rows="bf16", cache="e4m3", Hk=4, group=4, page=64, seqs=1,
             len_lo=20048, len_hi=20048, row_lo=2048, row_hi=2048, long=1, layout=0),
        # A serving step that mixes two chunks of prompts with single tokens of 30 others.
        dict(name="attend mixed step", op="attend", rows="bf16", cache="bf16", Hk=16, group=1, page=64, seqs=32, len_lo=900,
             len_hi=8000, row_lo=300, row_hi=800, long=2, layout=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend"])
    c = dict(op=op, rows=rng.choice(["bf16", "bf16", "f32"]) if op != "attend" else "bf16",
             cache=rng.choice(["bf16", "e4m3"]), Hk=rng.choice([1, 2, 3, 4, 5, 8, 16]), page=rng.choice([16, 32, 64, 128]))
    if op == "attend":
        c["group"] = rng.choice([1, 1, 2, 3, 4, 6, 8])
    seqs = _log_int(rng, 1, 100)
    hi = _log_int(rng, 1, 18000)
    hi = max(1, min(hi, 3000000 // (seqs * c["Hk"])))
    lo = max(1, hi // rng.choice([1, 8, 36]))
    kind = rng.choice(["one", "few", "chunk", "mixed"])
    long = {"one": 0, "few": 0, "chunk": seqs, "mixed": min(2, seqs)}[kind]
    row_hi = {"one": 1, "few": rng.randrange(2, 9), "chunk": _log_int(rng, 1, 1024), "mixed": _log_int(rng, 2, 1024)}[kind]
    row_hi = min(row_hi, hi) if op != "attend" else min(row_hi, hi, max(1, 60000000 // (hi * seqs * c["Hk"] * c["group"])))
    c.update(seqs=seqs, len_lo=lo, len_hi=hi, row_lo=row_hi if kind in ("one", "few") else max(1, row_hi // 4), row_hi=row_hi,
             long=long, layout=rng.randrange(1 << 30))
    return c


def _lens(case):
    """Rows in the cache after the call, and rows of the call, of each sequence.  row_hi = 0: all of them."""
    rng = np.random.default_rng([case["layout"], 0])
    n = case["seqs"]
    total = np.exp(rng.uniform(math.log(case["len_lo"]), math.log(case["len_hi"]), n)).round().astype(np.int64)
    total = np.clip(total, case["len_lo"], case["len_hi"])
    if case["row_hi"] == 0:
        return total, total
    if case["long"] == 0:
        rows = np.full(n, case["row_hi"], dtype=np.int64)
    else:
        rows = np.ones(n, dtype=np.int64)
        which = rng.permutation(n)[:case["long"]]
        rows[which] = rng.integers(case["row_lo"], case["row_hi"] + 1, case["long"])
    return total, np.minimum(rows, total)


# ------------------------------------------------------------------ states
def _dequantised(x, scale):
    """What e4m3 values and their powers of two [..., 1 per row] stand for, in fp32."""
    return x.float() * torch.exp2(scale.float() - 127.0)[..., None]


def _quantised(x):
    """(e4m3 values, powers of two as their exponent + 127) of fp32 rows [..., 64]: the least power of two at which a
    row's largest magnitude is at most 448."""
    mantissa, exponent = torch.frexp(x.abs().amax(-1))
    e = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp(min=-126)
    return torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    randn = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    total, rows = _lens(case)
    Hk, R, S = case["Hk"], case["page"], case["seqs"]
    used = -(-total // R)
    width, pool = int(used.max()), int(used.sum()) + 3
    rng = np.random.default_rng([case["layout"], 1])
    order = rng.permutation(pool)                                      # pages in no order, three of them unused
    table = np.zeros((S, width), dtype=np.int32)
    for s, at in enumerate(np.concatenate([[0], np.cumsum(used)[:-1]])):
        table[s, :used[s]] = order[at:at + used[s]]
    quant = case["cache"] == "e4m3"
    cu = np.concatenate([[0], np.cumsum(rows)])
    T = int(cu[-1])
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    st = dict(case=case, table=put(table), seq_len=put(total), row_cu=put(cu), T=T, max_rows=int(rows.max()), k_scale=None,
              v_scale=None)
    single = bool((rows == 1).all())
    st["own_cu"] = None if single else st["row_cu"]                    # a program with one row a sequence names none
    if case["op"] == "write":
        # Keys and values as a layer makes them: heads of different sizes.
        size = torch.exp2(torch.arange(Hk, device=dev, dtype=torch.float32) % 5 - 2)[:, None]
        dt = torch.bfloat16 if case["rows"] == "bf16" else torch.float32
        st.update(k=(randn(T, Hk, D) * size).to(dt), v=(randn(T, Hk, D) / size).to(dt))
        for x in ("k", "v"):
            if quant:
                st[x + "_pages"] = torch.zeros(pool, Hk, R, D, device=dev, dtype=torch.uint8).view(torch.float8_e4m3fn)
                st[x + "_scale"] = torch.full((pool, Hk, R), 127, device=dev, dtype=torch.uint8)
            else:
                st[x + "_pages"] = torch.zeros(pool, Hk, R, D, device=dev, dtype=torch.bfloat16)
        return st
    for x in ("k", "v"):
        if quant:
            st[x + "_pages"], st[x + "_scale"] = _quantised(randn(pool, Hk, R, D))
        else:
            st[x + "_pages"] = randn(pool, Hk, R, D).to(torch.bfloat16)
    if case["op"] == "attend":
        st["q"] = randn(T, Hk * case["group"], D).to(torch.bfloat16)
    return st


# ------------------------------------------------------------------ plain forms
def _places(s):
    """Page and row in it of every packed row."""
    R = s["case"]["page"]
    t = torch.arange(s["T"], device=s["table"].device)
    seq = torch.searchsorted(s["row_cu"][1:].long(), t, right=True)
    pos = (s["seq_len"][seq] - (s["row_cu"][seq + 1] - t)).long()
    return s["table"][seq, pos // R].long(), pos % R


def _plain_write(s):
    page, off = _places(s)
    for x in ("k", "v"):
        if s["k_scale"] is None:
            s[x + "_pages"][page, :, off] = s[x].to(torch.bfloat16)
        else:
            val, scale = _quantised(s[x].float())
            s[x + "_pages"].view(torch.uint8)[page, :, off] = val.view(torch.uint8)
            s[x + "_scale"][page, :, off] = scale
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _plain_read(s):
    page, off = _places(s)
    dt = torch.bfloat16 if s["case"]["rows"] == "bf16" else torch.float32

    def one(x):
        if s["k_scale"] is None:
            return s[x + "_pages"][page, :, off].to(dt)
        val = s[x + "_pages"].view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn)
        return _dequantised(val, s[x + "_scale"][page, :, off]).to(dt)

    return one("k"), one("v")


def _plain_attend(s):
    case = s["case"]
    Hk, G, R, n = case["Hk"], case["group"], case["page"], s["max_rows"]
    S, width = s["table"].shape
    at = s["table"].long()

    def rows_of(x):                                                    # [S, Hk, width * R, 64] in fp32
        if s["k_scale"] is None:
            p = s[x + "_pages"][at].float()
        else:
            p = _dequantised(s[x + "_pages"].view(torch.uint8)[at].view(torch.float8_e4m3fn), s[x + "_scale"][at])
        return p.permute(0, 2, 1, 3, 4).reshape(S, Hk, width * R, D)

    K, V = rows_of("k"), rows_of("v")
    i = torch.arange(n, device=at.device)
    count = s["row_cu"][1:] - s["row_cu"][:-1]
    real = i[None] < count[:, None]                                    # [S, n]
    rows = torch.where(real, s["row_cu"][:-1, None] + i[None], 0).long()
    Q = s["q"][rows].float().view(S, n, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hk, n * G, D)
    X = Q @ K.transpose(-1, -2) * (1.0 / math.sqrt(D))                 # [S, Hk, n * G, width * R]
    last = s["seq_len"][:, None] - count[:, None] + i[None]            # the last row that a row sees
    seen = torch.arange(width * R, device=at.device)[None, None] <= last[..., None]       # [S, n, width * R]
    seen = seen[:, None, :, None].expand(S, 1, n, G, width * R).reshape(S, 1, n * G, width * R)
    X = torch.where(seen, X, -torch.inf)
    m = X.amax(-1, keepdim=True)
    P = torch.exp(X - m)
    total = P.sum(-1, keepdim=True)
    O = (P @ V) / total
    lse = (m + torch.log(total))[..., 0]
    out = torch.empty_like(s["q"])
    log = torch.empty(s["T"], Hk * G, device=at.device, dtype=torch.float32)
    out[rows[real]] = O.view(S, Hk, n, G, D).permute(0, 2, 1, 3, 4).reshape(S, n, Hk * G, D)[real].to(out.dtype)
    log[rows[real]] = lse.view(S, Hk, n, G).permute(0, 2, 1, 3).reshape(S, n, Hk * G)[real]
    return out, log


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import hybrid_linear_attention_packed_gb300 as spanla
        if op == "write":
            spanla.span_la_kv_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["seq_len"], s["own_cu"],
                                    s["k_scale"], s["v_scale"])
            return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
        if op == "read":
            dt = torch.bfloat16 if s["case"]["rows"] == "bf16" else torch.float32
            return spanla.span_la_kv_read(s["k_pages"], s["v_pages"], s["table"], s["seq_len"], s["row_cu"], s["T"],
                                          s["k_scale"], s["v_scale"], dtype=dt)
        lse = torch.empty(s["q"].shape[:2], device=s["q"].device, dtype=torch.float32)
        out = spanla.span_la_softmax_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_len"], s["own_cu"],
                                           s["k_scale"], s["v_scale"], max_rows=s["max_rows"], lse=lse)
        return out, lse
    return _plain_write(s) if op == "write" else _plain_read(s) if op == "read" else _plain_attend(s)


def work(case):
    total, rows = _lens(case)
    Hk, T = case["Hk"], int(rows.sum())
    cached = 2 * (D * 2 if case["cache"] == "bf16" else D + 1)         # bytes of k and v of a row and head in the cache
    packed = 2 * D * (2 if case["rows"] == "bf16" else 4)
    if case["op"] != "attend":
        # (quantising: a magnitude, a maximum, a product and a rounding an element)
        return {"bytes": T * Hk * (cached + packed), "flops": T * Hk * 2 * D * (4 if case["cache"] == "e4m3" else 1)}
    H = Hk * case["group"]
    pairs = int((rows * total - rows * (rows - 1) // 2).sum())         # (row, cached row) pairs that see each other
    return {"bytes": int(total.sum()) * Hk * cached + T * H * (2 * D * 2 + 4), "flops": pairs * H * 4 * D}


# ------------------------------------------------------------------ 64 bits
def _exact_quantised(x):
    """As _quantised, from the grids' definitions: e4m3 has steps of 2^(floor(log2 |y|) - 3), of 2^-9 below 2^-6."""
    x = x.double()
    top = x.abs().amax(-1)
    e = torch.ceil(torch.log2(torch.where(top > 0, top, 1e-300) / 448.0))
    e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)             # (log2 rounds)
    e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
    y = x / torch.exp2(e)[..., None]
    size = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    size = torch.where(y.abs().clamp(min=2.0 ** -6) < torch.exp2(size), size - 1, size)
    step = torch.exp2(size - 3)
    return torch.round(y / step) * step, (e + 127).to(torch.uint8)     # (round: halves to even)


def exact(case, seed):
    s = prepare(case, seed)
    total, rows = _lens(case)
    table, R = s["table"].cpu().numpy().astype(np.int64), case["page"]
    quant = case["cache"] == "e4m3"

    def cached(x, seq, lo, hi):
        """Rows lo .. hi of a sequence, [hi - lo, Hk, 64] in 64 bits, page by page."""
        pages = table[seq, lo // R:-(-hi // R)]
        at = torch.from_numpy(pages).to(s["table"].device)
        raw = s[x + "_pages"].view(torch.uint8)[at].view(s[x + "_pages"].dtype) if quant else s[x + "_pages"][at]
        y = raw.to(torch.float64)
        if quant:
            y = y * 2.0 ** (s[x + "_scale"][at].double() - 127)[..., None]
        return y.transpose(1, 2).reshape(-1, case["Hk"], D)[lo % R:lo % R + hi - lo]

    first = np.concatenate([[0], np.cumsum(rows)])
    if case["op"] == "write":
        res = []
        for x in ("k", "v"):
            pages = s[x + "_pages"].to(torch.float64)
            scale = s[x + "_scale"]
            for q in range(case["seqs"]):
                lo, hi = int(total[q] - rows[q]), int(total[q])
                pos = np.arange(lo, hi)
                page, off = (torch.from_numpy(a).to(pages.device) for a in (table[q, pos // R], pos % R))
                new = s[x][first[q]:first[q + 1]]
                if quant:
                    new, e = _exact_quantised(new)
                    scale[page, :, off] = e
                pages[page, :, off] = new.double()
            res += [(pages, scale)]
        return res[0][0], res[1][0], res[0][1], res[1][1]
    if case["op"] == "read":
        both = []
        for x in ("k", "v"):
            both.append(torch.cat([cached(x, q, int(total[q] - rows[q]), int(total[q])) for q in range(case["seqs"])]))
        return tuple(both)
    H = case["Hk"] * case["group"]
    out = torch.empty(s["T"], H, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["T"], H, dtype=torch.float64, device=s["q"].device)
    for q in range(case["seqs"]):
        n, m = int(total[q]), int(rows[q])
        K, V = cached("k", q, 0, n), cached("v", q, 0, n)
        for r in range(0, m, 256):                                     # some rows at a time
            e = min(r + 256, m)
            hidden = torch.arange(n, device=out.device)[None] > torch.arange(n - m + r, n - m + e, device=out.device)[:, None]
            for h in range(H):
                x = s["q"][first[q] + r:first[q] + e, h].double() @ K[:, h // case["group"]].T / 8.0
                x = x.masked_fill(hidden, -torch.inf)
                z = torch.logsumexp(x, -1)
                lse[first[q] + r:first[q] + e, h] = z
                out[first[q] + r:first[q] + e, h] = torch.exp(x - z[:, None]) @ V[:, h // case["group"]]
    return out, lse
