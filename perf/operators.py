"""The hybrid model's decayed linear layer and the preparation of its queries
and keys, as calls that can be measured one at a time.

Three operators:

* ``pass`` / ``fork``: linear attention with a decay for each head over a packed
  pass, S_t = a S_{t-1} + k_t v_t^T and o_t = S_t^T q_t per head with
  a = exp(log_decay[h]).  Views start from zero, branches from their parent
  view's final state (``pass``) or from a kept one (``fork``).
* ``step``: the same recurrence for single tokens, states updated in place.
* ``rope``: RMS norm of every head's query and key followed by the position
  rotation of its first ``rotary`` dimensions.

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
        # The smallest pass of the tests: one fp32 head, two views, three short branches each.
        dict(name="pass tiny fp32", op="pass", dtype="f32", H=1, views=2, view_lo=77, view_hi=130, br_lo=3, br_hi=3,
             len_lo=9, len_hi=20, decay="slopes", layout=0),
        # One scoring request: a 7,400-token view with 8 behaviours to score.
        dict(name="pass one request", op="pass", dtype="bf16", H=16, views=1, view_lo=7400, view_hi=7400, br_lo=8, br_hi=8,
             len_lo=32, len_hi=96, decay="slopes", layout=0),
        # The same request in fp32 (a check of a model against its training numerics).
        dict(name="pass one request fp32", op="pass", dtype="f32", H=16, views=1, view_lo=7400, view_hi=7400, br_lo=8,
             br_hi=8, len_lo=32, len_hi=96, decay="slopes", layout=0),
        # Four requests packed into one pass.
        dict(name="pass four requests", op="pass", dtype="bf16", H=16, views=4, view_lo=500, view_hi=18000, br_lo=8, br_hi=8,
             len_lo=32, len_hi=96, decay="mixed", layout=0),
        # A throughput pass: sixteen requests, up to a few hundred branches each.
        dict(name="pass sixteen requests", op="pass", dtype="bf16", H=16, views=16, view_lo=500, view_hi=18000, br_lo=1,
             br_hi=300, len_lo=16, len_hi=128, decay="slopes", layout=0),
        # A shard of a long request: 64 branches forked from one view's kept state.
        dict(name="fork shard of 64", op="fork", dtype="bf16", H=16, views=1, view_lo=0, view_hi=0, br_lo=64, br_hi=64,
             len_lo=24, len_hi=128, decay="slopes", layout=0),
        # One sequence's next token: latency counts.
        dict(name="step one token", op="step", dtype="bf16", H=16, n=1, pool=1, decay="slopes", layout=0),
        # A ragged decode batch out of a larger pool of states, fp32 rows.
        dict(name="step 61 of 80 fp32", op="step", dtype="f32", H=16, n=61, pool=80, decay="mixed", layout=0),
        # The largest decode batch: a thousand sequences' states, 268 MB.
        dict(name="step 1024", op="step", dtype="bf16", H=16, n=1024, pool=1024, decay="slopes", layout=0),
        # Queries and keys of a small decode batch, far into their sequences.
        dict(name="rope 8 tokens", op="rope", dtype="bf16", T=8, Hq=16, Hk=16, rotary=64, interleaved=False, base=1e6,
             start=900000, fused=False, layout=0),
        # Queries and keys of one request out of a fused projection's rows.
        dict(name="rope one request", op="rope", dtype="bf16", T=7829, Hq=16, Hk=16, rotary=64, interleaved=False,
             base=10000.0, start=0, fused=True, layout=0),
        # A four-request pass in fp32, half of each head rotated, neighbouring dimensions paired.
        dict(name="rope four requests fp32", op="rope", dtype="f32", T=43758, Hq=16, Hk=16, rotary=32, interleaved=True,
             base=10000.0, start=0, fused=False, layout=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pass", "pass", "fork", "step", "rope"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    layout = rng.randrange(1 << 30)
    if op == "rope":
        T = _log_int(rng, 1, 40000)
        return dict(op=op, dtype=dtype, T=T, Hq=rng.choice([1, 3, 8, 16]), Hk=rng.choice([1, 3, 8, 16]),
                    rotary=rng.choice([64, 64, 32, 16]), interleaved=rng.random() < 0.5, base=rng.choice([10000.0, 1e6]),
                    start=rng.choice([0, 0, rng.randrange(1 << 20)]), fused=rng.random() < 0.5, layout=layout)
    H = rng.choice([1, 2, 5, 8, 16, 16, 24])
    decay = rng.choice(["slopes", "mixed"])
    if op == "step":
        n = _log_int(rng, 1, 600)
        return dict(op=op, dtype=dtype, H=H, n=n, pool=n + rng.randrange(0, 30), decay=decay, layout=layout)
    views = _log_int(rng, 1, 12)
    hi = _log_int(rng, 1, 18000 if dtype == "bf16" else 6000)
    br = _log_int(rng, 1, 40)
    ln = _log_int(rng, 1, 400)
    return dict(op=op, dtype=dtype, H=min(H, 16), views=views, view_lo=max(1, hi // 8), view_hi=hi, br_lo=max(0, br // 4),
                br_hi=br, len_lo=max(1, ln // 4), len_hi=ln, decay=decay, layout=layout)


def _lens(case):
    """View lengths, branch lengths and branch parents of a case."""
    rng = np.random.default_rng([case["layout"], 0])
    log_u = lambda lo, hi, n: np.clip(np.round(np.exp(rng.uniform(  # noqa: E731
        math.log(max(lo, 1)), math.log(max(hi, 1)), n))), lo, hi).astype(np.int64)
    views = rng.integers(case["view_lo"], case["view_hi"] + 1, case["views"]).astype(np.int64)
    counts = log_u(case["br_lo"], case["br_hi"], case["views"])
    branches = rng.integers(case["len_lo"], case["len_hi"] + 1, int(counts.sum())).astype(np.int64)
    return views, branches, np.repeat(np.arange(case["views"]), counts)


def _log_decay(case):
    """Slopes 2^(-8 (h+1) / H), or with heads among them that forget nothing and that forget at once."""
    H = case["H"]
    ld = [-(2.0 ** (-8.0 * (h + 1) / H)) for h in range(H)]
    if case["decay"] == "mixed":
        for h in range(0, H, 5):
            ld[h] = 0.0
        for h in range(3, H, 5):
            ld[h] = -6.0
    return ld


# ------------------------------------------------------------------ states
def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    randn = lambda *s: torch.randn(s, generator=g, device=dev, dtype=torch.float32)  # noqa: E731
    if case["op"] == "rope":
        T, Hq, Hk = case["T"], case["Hq"], case["Hk"]
        if case["fused"]:   # q and k are parts of a fused projection's rows
            rows = randn(T, (Hq + 2 * Hk) * D).to(dt)
            q = rows[:, :Hq * D].view(T, Hq, D)
            k = rows[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        else:
            q, k = randn(T, Hq, D).to(dt), randn(T, Hk, D).to(dt)
        half = case["rotary"] // 2
        freq = np.asarray([case["base"] ** (-2.0 * i / case["rotary"]) for i in range(half)], dtype=np.float64)
        pos = (case["start"] + torch.arange(T, device=dev)).to(torch.int32)
        return dict(case=case, q=q, k=k, q_weight=(1.0 + 0.2 * randn(D)).to(dt), k_weight=(1.0 + 0.2 * randn(D)).to(dt),
                    positions=pos, inv_freq=freq, inv_freq_dev=torch.from_numpy(freq).to(dev), eps=1e-6)
    H = case["H"]
    ld = torch.tensor(_log_decay(case), dtype=torch.float32, device=dev)
    if case["op"] == "step":
        n, pool = case["n"], case["pool"]
        index = np.random.default_rng([case["layout"], 1]).permutation(pool)[:n].astype(np.int32)
        return dict(case=case, q=(randn(n, H, D) / 8).to(dt), k=(randn(n, H, D) / 8).to(dt), v=randn(n, H, D).to(dt),
                    states=randn(pool, H, D, D), log_decay=ld, index=index,
                    index_dev=torch.from_numpy(index.astype(np.int64)).to(dev))
    views, branches, parent = _lens(case)
    fork = case["op"] == "fork"
    vcu = np.concatenate([[0], np.cumsum(views)]).astype(np.int32)
    first = 0 if fork else int(vcu[-1])
    bcu = (first + np.concatenate([[0], np.cumsum(branches)])).astype(np.int32)
    T = int(bcu[-1])
    s = dict(case=case, q=(randn(T, H, D) / 8).to(dt), k=(randn(T, H, D) / 8).to(dt), v=randn(T, H, D).to(dt), log_decay=ld,
             view_cu=vcu, branch_cu=bcu, parent=parent.astype(np.int32))
    if fork:
        s["kept"] = randn(case["views"], H, D, D)
    put = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int64)).to(dev)  # noqa: E731
    s.update(view_cu_dev=put(vcu), branch_cu_dev=put(bcu), parent_dev=put(parent), longest_view=int(views.max()),
             longest_branch=int(branches.max()) if len(branches) else 0)
    return s


# ------------------------------------------------------------------ plain forms
def _segments(q, k, v, ld, cu, longest, start, out, want_final):
    """The segments cu[s] .. cu[s+1] (device int64), chunk by chunk in fp32: rows of `out` are written, the final states
    returned.  `start`: the states they start from, [n, H, 64, 64], or None."""
    C = 64
    n, H = cu.numel() - 1, q.shape[1]
    nc = max(1, -(-longest // C))
    at = torch.arange(nc * C, device=q.device)
    length = (cu[1:] - cu[:-1])
    real = at[None] < length[:, None]                                  # [n, nc*C]
    rows = torch.where(real, cu[:-1, None] + at[None], 0)
    pick = lambda x: (x[rows].float() * real[..., None, None]).view(n, nc, C, H, D).permute(0, 3, 1, 2, 4)  # noqa: E731
    Q, K, V = pick(q), pick(k), pick(v)                                # [n, H, nc, C, 64]
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    L = ld.float()
    gap = i[:, None] - i[None]
    inside = torch.where(gap >= 0, torch.exp(L[:, None, None] * gap.clamp(min=0)), 0.0)          # [H, C, C]
    O = ((Q @ K.transpose(-1, -2)) * inside[None, :, None]) @ V
    KV = (K * torch.exp(L[:, None] * (C - 1 - i))[None, :, None, :, None]).transpose(-1, -2) @ V  # [n, H, nc, 64, 64]
    c = torch.arange(nc, device=q.device, dtype=torch.float32)
    far = c[:, None] - c[None] - 1
    between = torch.where(far >= 0, torch.exp(L[:, None, None] * C * far.clamp(min=0)), 0.0)      # [H, nc, nc]
    S = (between[None] @ KV.reshape(n, H, nc, D * D)).view(n, H, nc, D, D)
    if start is not None:
        S = S + torch.exp(L[:, None] * C * c)[None, :, :, None, None] * start[:, :, None]
    O = O + torch.exp(L[:, None] * (i + 1))[None, :, None, :, None] * (Q @ S)
    out[rows[real]] = O.permute(0, 2, 3, 1, 4).reshape(n, nc * C, H, D)[real].to(out.dtype)
    if not want_final:
        return None
    left = (length[:, None] - 1 - at[None]).clamp(min=0).float()       # [n, nc*C]
    w = torch.exp(L[None, :, None] * left[:, None])                    # [n, H, nc*C]
    K2, V2 = K.reshape(n, H, nc * C, D), V.reshape(n, H, nc * C, D)
    return (K2 * w[..., None]).transpose(-1, -2) @ V2


def _plain_pass(s):
    q, k, v, ld = s["q"], s["k"], s["v"], s["log_decay"]
    out = torch.empty_like(q)
    if "kept" in s:
        final = s["kept"]
    else:
        final = _segments(q, k, v, ld, s["view_cu_dev"], s["longest_view"], None, out, True)
    if s["longest_branch"]:
        _segments(q, k, v, ld, s["branch_cu_dev"], s["longest_branch"], final[s["parent_dev"]], out, False)
    return out if "kept" in s else (out, final)


def _plain_step(s):
    at = s["index_dev"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    S = torch.exp(s["log_decay"])[None, :, None, None] * s["states"][at] + k[..., :, None] * v[..., None, :]
    s["states"][at] = S
    return (q[..., :, None] * S).sum(-2).to(s["q"].dtype), s["states"]


def _plain_rope(s):
    case = s["case"]
    r = case["rotary"]
    turn = s["positions"].double()[:, None] * s["inv_freq_dev"][None]   # far positions: 64 bits
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]

    def one(x, w):
        x = x.float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * w.float()
        z = y.clone()
        if case["interleaved"]:
            a, b = y[..., 0:r:2], y[..., 1:r:2]
            z[..., 0:r:2], z[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = y[..., :r // 2], y[..., r // 2:r]
            z[..., :r // 2], z[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
        return z

    return one(s["q"], s["q_weight"]).to(s["q"].dtype), one(s["k"], s["k_weight"]).to(s["k"].dtype)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import hybrid_linear_attention_packed_gb300 as spanla
        if op == "rope":
            return spanla.span_la_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                                               eps=s["eps"], interleaved=s["case"]["interleaved"])
        if op == "step":
            out = spanla.span_la_decay_step(s["q"], s["k"], s["v"], s["states"], s["log_decay"], state_index=s["index"])
            return out, s["states"]
        if op == "fork":
            return spanla.span_la_decay_branches_from_state(s["kept"], s["q"], s["k"], s["v"], s["log_decay"],
                                                            s["branch_cu"], s["parent"])
        return spanla.span_la_decay_pass(s["q"], s["k"], s["v"], s["log_decay"], s["view_cu"], s["branch_cu"], s["parent"])
    return _plain_rope(s) if op == "rope" else _plain_step(s) if op == "step" else _plain_pass(s)


def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        vectors = case["T"] * (case["Hq"] + case["Hk"])
        return {"bytes": vectors * 2 * D * esz + 4 * case["T"], "flops": vectors * D * 7}
    H = case["H"]
    if case["op"] == "step":
        return {"bytes": case["n"] * H * (2 * D * D * 4 + 4 * D * esz), "flops": case["n"] * H * 5 * D * D}
    views, branches, parent = _lens(case)
    fork = case["op"] == "fork"
    rows = int(branches.sum()) + (0 if fork else int(views.sum()))
    states = len(set(parent.tolist())) if fork else len(views)   # kept states read, or final states written
    # by the recurrence: decay, update and output of a 64 x 64 state for every row and head
    return {"bytes": rows * H * 4 * D * esz + states * H * D * D * 4, "flops": rows * H * 5 * D * D}


# ------------------------------------------------------------------ 64 bits
def _exact_segment(q, k, v, a, S):
    """One segment's rows [n, H, 64] in fp64 from state S [H, 64, 64] by blocks of its rows; a: log decay [H]."""
    outs = []
    for r in range(0, q.shape[0], 256):
        x, y, z = (t[r:r + 256].double().transpose(0, 1) for t in (q, k, v))   # [H, m, 64]
        m = x.shape[1]
        t = torch.arange(m, device=q.device, dtype=torch.float64)
        weight = torch.tril(torch.exp(a[:, None, None] * (t[:, None] - t[None]).clamp(min=0)))
        o = (torch.bmm(x, y.transpose(1, 2)) * weight) @ z
        o = o + torch.exp(a[:, None] * (t + 1))[..., None] * (x @ S)
        S = torch.exp(a * m)[:, None, None] * S + (y * torch.exp(a[:, None] * (m - 1 - t))[..., None]).transpose(1, 2) @ z
        outs.append(o.transpose(0, 1))
    return (torch.cat(outs) if outs else q.double()), S


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        r, pos = case["rotary"], s["positions"].cpu().numpy().astype(np.float64)
        ang = torch.from_numpy(pos[:, None] * s["inv_freq"][None]).to(s["q"].device)
        rot = torch.polar(torch.ones_like(ang), ang)[:, None]                   # [T, 1, r/2], complex128
        res = []
        for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
            x = x.double()
            y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + s["eps"]) * w.double()
            first = (torch.arange(r // 2, device=x.device) * 2) if case["interleaved"] else torch.arange(r // 2, device=x.device)
            second = first + (1 if case["interleaved"] else r // 2)
            z = torch.complex(y[..., first], y[..., second]) * rot
            y[..., first], y[..., second] = z.real, z.imag
            res.append(y)
        return tuple(res)
    a = s["log_decay"].double()
    if op == "step":
        S = s["states"].double()
        outs = []
        for t, slot in enumerate(s["index"].tolist()):
            new = torch.exp(a)[:, None, None] * S[slot] + torch.einsum("hi,hj->hij", s["k"][t].double(), s["v"][t].double())
            S[slot] = new
            outs.append(torch.einsum("hi,hij->hj", s["q"][t].double(), new))
        return torch.stack(outs), S
    q, k, v = s["q"], s["k"], s["v"]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    zero = torch.zeros(case["H"], D, D, dtype=torch.float64, device=q.device)
    finals = [x.double() for x in s["kept"]] if op == "fork" else []
    for i in range(0 if op == "fork" else case["views"]):
        lo, hi = int(s["view_cu"][i]), int(s["view_cu"][i + 1])
        out[lo:hi], S = _exact_segment(q[lo:hi], k[lo:hi], v[lo:hi], a, zero)
        finals.append(S)
    for b, p in enumerate(s["parent"].tolist()):
        lo, hi = int(s["branch_cu"][b]), int(s["branch_cu"][b + 1])
        out[lo:hi], _ = _exact_segment(q[lo:hi], k[lo:hi], v[lo:hi], a, finals[p])
    return out if op == "fork" else (out, torch.stack(finals))
