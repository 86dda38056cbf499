"""The operators that take prompts through a softmax-attention layer, measured: causal attention of
packed prompts over a paged cache, the norm of every head with its rotary position (and with the
append to that cache), and that norm's gradient.

``run`` computes an operator in its plain form, elementary torch operations in 32 bits, or, where
``own`` is true, by the framework's calls.  ``exact`` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one short question to an idle server: the latency of the smallest prompt
        dict(name="prompt one short", op="prompt", B=1, T=61, HQ=16, HKV=2, D=256, P=16, context=0, rows="even",
             dtype="bf16"),
        # prompts of different lengths that arrived together, packed one behind another
        dict(name="prompt packed", op="prompt", B=8, T=4096, HQ=32, HKV=8, D=128, P=64, context=0, rows="ragged",
             dtype="bf16"),
        # a long document, heads of 256
        dict(name="prompt long", op="prompt", B=2, T=16384, HQ=16, HKV=2, D=256, P=128, context=0, rows="ragged",
             dtype="bf16"),
        # the next chunk of four long prompts, most of which lies in the cache
        dict(name="prompt chunk behind context", op="prompt", B=4, T=1024, HQ=64, HKV=8, D=128, P=64, context=30000,
             rows="ragged", dtype="bf16"),
        # a serving step: prompt chunks beside rows that decode one token
        dict(name="prompt mixed with decode", op="prompt", B=96, T=1500, HQ=16, HKV=2, D=256, P=64, context=3000,
             rows="mixed", dtype="bf16"),
        # 32-bit inputs, three query heads a group, odd counts, an empty row, a padding row, a row without context
        dict(name="prompt odd fp32", op="prompt", B=7, T=523, HQ=6, HKV=2, D=64, P=16, context=777, rows="odd",
             dtype="fp32"),
        # decode: one new token for each of eight requests, a quarter of the head rotated, weights around zero
        dict(name="norm append one token", op="append", B=8, T=1, HQ=16, HKV=2, D=256, rot=64, P=16, context=900,
             rows="even", dtype="bf16", layout="half", scaling="none", offset=1.0),
        # the prompts of a serving step, packed
        dict(name="norm append packed prompts", op="append", B=8, T=6000, HQ=32, HKV=8, D=128, rot=128, P=64,
             context=100000, rows="ragged", dtype="bf16", layout="half", scaling="yarn", offset=0.0),
        # queries on the way forward in training
        dict(name="norm rotate", op="rotate", N=16384, heads=16, D=128, rot=128, dtype="bf16", layout="half",
             scaling="none", offset=0.0),
        # few tokens, heads of 96 dims, 32 bits
        dict(name="norm rotate odd fp32", op="rotate", N=977, heads=5, D=96, rot=48, dtype="fp32",
             layout="interleaved", scaling="bands", offset=1.0),
        # the way back: gradients of the queries and of the weights that all heads share
        dict(name="norm gradient", op="gradient", N=16384, heads=16, D=128, rot=128, dtype="bf16", layout="half",
             scaling="none", offset=0.0),
        # the same in 32 bits at an odd size
        dict(name="norm gradient odd fp32", op="gradient", N=3001, heads=6, D=256, rot=64, dtype="fp32",
             layout="interleaved", scaling="linear", offset=1.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prompt", "prompt", "append", "rotate", "gradient"])
    if kind == "prompt":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        D, HKV, G = rng.choice([64, 96, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8])
        B, rows = _log_int(rng, 1, 128), rng.choice(["even", "ragged", "mixed", "odd"])
        # at most 2.5e12 operations, 4 D HQ for each pair of a query and a key, and 3e8 values of keys
        pairs = (2.5e12 if dtype == "bf16" else 3.0e10) / (4.0 * D * HKV * G)
        T = _log_int(rng, 1, 16384)
        full = max(1, -(-B // 16)) if rows == "mixed" else B
        T = max(1, min(T, int(math.sqrt(pairs / full)), int(1.0e8 / (B * HKV * D))))
        most = min(pairs / (full * T + B), 2.0e8 / (B * HKV * D))
        context = 0 if rng.random() < 0.3 else _log_int(rng, 1, max(2, min(65536, int(most))))
        return dict(op="prompt", B=B, T=T, HQ=HKV * G, HKV=HKV, D=D, P=rng.choice([16, 32, 64, 128]), context=context,
                    rows=rows, dtype=dtype)
    D = rng.choice([64, 96, 128, 256])
    case = dict(op=kind, D=D, rot=D // rng.choice([1, 2, 4]), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                layout=rng.choice(["half", "interleaved"]), offset=rng.choice([0.0, 1.0]),
                scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]))
    if kind == "append":
        B, HKV = _log_int(rng, 1, 256), rng.choice([1, 2, 4, 8])
        HQ = HKV * rng.choice([1, 3, 4, 8])
        token = (HQ + 2 * HKV) * D * (4 if case["dtype"] == "bf16" else 8)
        return dict(case, B=B, T=_log_int(rng, 1, max(2, min(6000, int(6.0e8 / (B * token))))), HQ=HQ, HKV=HKV,
                    P=rng.choice([16, 32, 64, 128]), context=_log_int(rng, 10, 200000),
                    rows=rng.choice(["even", "ragged", "mixed"]))
    return dict(case, N=_log_int(rng, 1, 16384), heads=rng.choice([1, 3, 5, 8, 16]))


# ------------------------------------------------------------------ what a case fixes

def _part(n):
    return (np.arange(n) * 0.6180339887498949) % 1.0


def _counts(case):
    """New tokens of each row."""
    B, T, kind = case["B"], case["T"], case["rows"]
    if kind == "even":
        return np.full(B, T, np.int64)
    if kind == "mixed":                                    # every sixteenth row brings a prompt, the others decode
        return np.where(np.arange(B) % 16 == 0, T, 1).astype(np.int64)
    n = np.maximum(1, np.round(T * (1 - 0.6 * _part(B)))).astype(np.int64)
    if kind == "odd" and B >= 2:
        n[1] = 0
    return n


def _lengths(case):
    """Committed tokens of each row."""
    B, n = case["B"], case["context"]
    ln = np.round(n * (1 - 0.4 * _part(B))).astype(np.int64)
    if case["rows"] == "odd" and B >= 4:
        ln[3] = 0
    return ln


def _slots(case):
    s = np.arange(case["B"])
    if case["rows"] == "odd" and case["B"] >= 3:
        s[2] = -1                                          # a padding row: its tokens are there, its outputs are zeros
    return s


def _starts(case):
    return np.concatenate([[0], np.cumsum(_counts(case))])


ROPE = {"none": dict(base=1.0e6), "linear": dict(base=1.0e4, factor=4.0),
        "ntk": dict(base=1.0e4, factor=8.0),
        "yarn": dict(base=1.0e4, factor=32.0, original=4096.0, fast=32.0, slow=1.0),
        "bands": dict(base=5.0e5, factor=8.0, original=8192.0, low=1.0, high=4.0)}
EPS = 1.0e-6


def _frequencies(case):
    """(radians a position for each pair in 64 bits, the factor on cos and sin)."""
    kind, p, rot = case["scaling"], ROPE[case["scaling"]], case["rot"]
    i = np.arange(rot // 2, dtype=np.float64)
    base = p["base"]
    if kind == "ntk":
        base *= p["factor"] ** (rot / (rot - 2.0))
    f = base ** (-2.0 * i / rot)
    if kind == "linear":
        return f / p["factor"], 1.0
    if kind == "yarn":
        def turn(n):
            return rot * math.log(p["original"] / (n * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(turn(p["fast"])), 0), min(math.ceil(turn(p["slow"])), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / p["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(p["factor"]) + 1.0
    if kind == "bands":
        wave = 2 * math.pi / f
        mix = np.clip((p["original"] / wave - p["low"]) / (p["high"] - p["low"]), 0.0, 1.0)
        return (1 - mix) * f / p["factor"] + mix * f, 1.0
    return f, 1.0


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype):
    """Standard normal values, made a slice at a time so that no large 32-bit copy is kept."""
    out = torch.empty(shape, dtype=TYPES[dtype], device=DEV)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        part = flat[a:a + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV))
    return out


def _int32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _cache(case, g, lens, tokens, fill, r):
    """The tensors of a cache of one layer whose slots hold `tokens` tokens, `lens` of them committed;
    pages in random order."""
    B, P = case["B"], case["P"]
    need = -(-tokens // P)
    num_pages, max_pages = int(need.sum()) + 1, max(int(need.max()), 1)
    table, order, at = np.full((B, max_pages), -1, np.int64), r.permutation(num_pages), 0
    for s in range(B):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    shape = (1, num_pages, case["HKV"], P, case["D"])
    make = (lambda: _normal(g, shape, case["dtype"])) if fill else (
        lambda: torch.zeros(shape, dtype=TYPES[case["dtype"]], device=DEV))
    return dict(dims=dict(n_layers=1, num_pages=num_pages, HKV=case["HKV"], P=P, D=case["D"], num_slots=B,
                          max_pages=max_pages),
                dtype=case["dtype"], k=make(), v=make(), page_table=_int32(table), n_pages=_int32(need),
                length=_int32(lens), handle=None)


def _handle(c):
    """The framework's cache over the tensors of `c`, made once and kept, as a program keeps it."""
    if c["handle"] is None:
        from gated_delta_rule_spec_gb300 import binding
        c["handle"] = binding.KvCache(**c["dims"], io_dtype=c["dtype"], tensors={
            n: c[n] for n in ("k", "v", "page_table", "n_pages", "length")})
    return c["handle"]


def _plan(state):
    """The framework's rotary plan, made once and kept."""
    if state["plan"] is None:
        from gated_delta_rule_spec_gb300 import binding
        case = state["case"]
        state["plan"] = binding.RopePlan(case["D"], case["rot"], layout=case["layout"], scaling=case["scaling"],
                                         **ROPE[case["scaling"]])
    return state["plan"]


def _norms(state):
    """The framework's norms over the weights, made once and kept."""
    if state["norms"] is None:
        from gated_delta_rule_spec_gb300 import binding
        state["norms"] = [binding.HeadNorm(w, eps=EPS, offset=state["case"]["offset"]) for w in state["weights"]]
    return state["norms"]


# ------------------------------------------------------------------ prepare

def prepare(case, seed):
    g, r = _generator(seed), np.random.default_rng(int(seed))
    return {"prompt": _prepare_prompt, "append": _prepare_append, "rotate": _prepare_rotate,
            "gradient": _prepare_rotate}[case["op"]](case, g, r)


def _prepare_prompt(case, g, r):
    ln, ct = _lengths(case), _counts(case)
    c = _cache(case, g, ln, ln + ct, True, r)
    n = int(ct.sum())
    return dict(case=case, cache=c, q=_normal(g, (n, case["HQ"], case["D"]), case["dtype"]), slots=_int32(_slots(case)),
                starts=_int32(_starts(case)), scale=case["D"] ** -0.5, work=None)


def _weights(case, g, n):
    """Weights of trained norms: around one, kept as they are or as what is added to one."""
    w = 1.0 - case["offset"] + 0.2 * torch.randn(n, case["D"], generator=g, device=DEV)
    return [w[i].clone() for i in range(n)]


def _table(first, rows, f, m):
    """cos and sin of the positions in use, in 32 bits, as a program keeps them."""
    a = torch.arange(first, first + rows, dtype=torch.float64, device=DEV)[:, None] * torch.as_tensor(f, device=DEV)
    return torch.stack([torch.cos(a) * m, torch.sin(a) * m]).float()


def _prepare_append(case, g, r):
    P, ct = case["P"], _counts(case)
    pos = np.concatenate([a + np.arange(n) for a, n in zip(_lengths(case), ct)])
    ln = _lengths(case) % (4 * P)                          # where in its pages a row ends; its positions run on
    c = _cache(case, g, ln, ln + ct, False, r)
    heads = case["HQ"] + 2 * case["HKV"]
    qkv = _normal(g, (int(ct.sum()), heads, case["D"]), case["dtype"])   # one projection's output, q, k and v side by side
    f, m = _frequencies(case)
    first = int(pos.min())
    return dict(case=case, cache=c, qkv=qkv, slots=_int32(np.arange(case["B"])), starts=_int32(_starts(case)),
                pos=_int32(pos), weights=_weights(case, g, 2), norms=None, plan=None,
                table=_table(first, int(pos.max()) - first + 1, f, m), first=first)


def _prepare_rotate(case, g, r):
    shape = (case["N"], case["heads"], case["D"])
    f, m = _frequencies(case)
    return dict(case=case, x=_normal(g, shape, case["dtype"]),
                dy=_normal(g, shape, case["dtype"]) if case["op"] == "gradient" else None,
                weights=_weights(case, g, 1), norms=None, pos=_int32(np.arange(case["N"])), plan=None,
                table=_table(0, case["N"], f, m), first=0, work=None)


# ------------------------------------------------------------------ run

def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "append": _own_append, "rotate": _own_rotate, "gradient": _own_gradient}[op](state)
    return {"prompt": _plain_prompt, "append": _plain_append, "rotate": _plain_rotate,
            "gradient": _plain_gradient}[op](state)


def _own_prompt(s):
    from gated_delta_rule_spec_gb300 import binding
    case, c = s["case"], _handle(s["cache"])
    if s["work"] is None:
        s["work"] = torch.empty(binding.prompt_attn_workspace(c, case["B"], s["q"].shape[0], case["HQ"]),
                                dtype=torch.uint8, device=DEV)
    return binding.prompt_attn(c, 0, s["slots"], s["starts"], s["q"], scale=s["scale"], workspace=s["work"])


def _own_append(s):
    from gated_delta_rule_spec_gb300 import binding
    case, c = s["case"], _handle(s["cache"])
    hq, hk = case["HQ"], case["HKV"]
    q_norm, k_norm = _norms(s)
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:]
    out = binding.norm_rope_append(_plan(s), c, 0, s["slots"], s["starts"], q, k, v, q_norm=q_norm, k_norm=k_norm,
                                   pos=s["pos"])
    return out, c.k, c.v


def _own_rotate(s):
    from gated_delta_rule_spec_gb300 import binding
    return binding.norm_rope(_plan(s), _norms(s)[0], s["pos"], s["x"])


def _own_gradient(s):
    from gated_delta_rule_spec_gb300 import binding
    case = s["case"]
    if s["work"] is None:
        s["work"] = torch.empty(max(16, binding.norm_rope_grad_workspace(case["N"], case["heads"], case["D"])),
                                dtype=torch.uint8, device=DEV)
    return binding.norm_rope_grad(_plan(s), _norms(s)[0], s["pos"], s["x"], s["dy"], workspace=s["work"])


def _groups(case):
    """Rows that the plain form takes together, padded to the longest: those of up to eight tokens, and
    every other row by itself in pieces of 1024 tokens: (rows, first token, tokens)."""
    ct = _counts(case)
    small = np.nonzero((ct > 0) & (ct <= 8))[0]
    out = [(small, 0, int(ct[small].max()))] if len(small) else []
    for b in np.nonzero(ct > 8)[0]:
        for t in range(0, int(ct[b]), 1024):
            out.append((np.array([b]), t, min(1024, int(ct[b]) - t)))
    return out


def _plain_prompt(s):
    case, c = s["case"], s["cache"]
    HQ, HKV, D, P = case["HQ"], case["HKV"], case["D"], case["P"]
    G, ln, ct, slots, starts = HQ // HKV, _lengths(case), _counts(case), _slots(case), _starts(case)
    out = torch.zeros_like(s["q"])
    for rows, t0, T in _groups(case):
        rows = rows[slots[rows] >= 0]
        if not len(rows):
            continue
        R, S = len(rows), int((ln[rows] + np.minimum(ct[rows], t0 + T)).max())
        table = c["page_table"][_int32(rows).long()][:, :-(-S // P)].long().clamp(min=0)
        k = c["k"][0][table].permute(0, 2, 1, 3, 4).reshape(R, HKV, -1, D)[:, :, :S].float()
        t = torch.arange(t0, t0 + T, device=DEV)
        live = t[None] < _int32(ct[rows]).long()[:, None]
        token = torch.where(live, _int32(starts[rows]).long()[:, None] + t[None], 0)
        q = s["q"][token].float().view(R, T, HKV, G, D).permute(0, 2, 1, 3, 4).reshape(R, HKV, T * G, D)
        x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(R, HKV, T, G, S)
        del k
        far = torch.arange(S, device=DEV)[None, None] > (_int32(ln[rows]).long()[:, None] + t[None])[:, :, None]
        x = x.masked_fill_(far[:, None, :, None], -math.inf)
        x = x.sub_(x.amax(-1, keepdim=True)).exp_()
        total = x.sum(-1, keepdim=True)
        v = c["v"][0][table].permute(0, 2, 1, 3, 4).reshape(R, HKV, -1, D)[:, :, :S].float()
        o = (x.view(R, HKV, T * G, S) @ v).view(R, HKV, T, G, D) / total
        o = o.permute(0, 2, 1, 3, 4).reshape(R, T, HQ, D).to(TYPES[case["dtype"]])
        out[token[live]] = o[live]
    return out


def _turned(x, cos, sin, case):
    """x [.., heads, D] in 32 bits turned by cos, sin [.., 1, rot / 2]."""
    rot = case["rot"]
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _normed(x, w, case):
    """x [.., D] in 32 bits over its root mean square, times the weights."""
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w + case["offset"])


def _angles(s):
    row = s["pos"].long() - s["first"]
    return s["table"][0][row][:, None], s["table"][1][row][:, None]


def _plain_append(s):
    case, c = s["case"], s["cache"]
    P, hq, hk = case["P"], case["HQ"], case["HKV"]
    cos, sin = _angles(s)
    q = _turned(_normed(s["qkv"][:, :hq].float(), s["weights"][0], case), cos, sin, case).to(TYPES[case["dtype"]])
    k = _turned(_normed(s["qkv"][:, hq:hq + hk].float(), s["weights"][1], case), cos, sin, case)
    token = torch.arange(s["qkv"].shape[0], device=DEV)
    b = (s["starts"].long()[None, 1:] <= token[:, None]).sum(1)
    at = c["length"].long()[b] + token - s["starts"].long()[b]
    page, off = c["page_table"].long()[b, at // P], at % P
    c["k"][0][page, :, off] = k.to(TYPES[case["dtype"]])
    c["v"][0][page, :, off] = s["qkv"][:, hq + hk:]
    return q, c["k"], c["v"]


def _plain_rotate(s):
    case = s["case"]
    cos, sin = _angles(s)
    return _turned(_normed(s["x"].float(), s["weights"][0], case), cos, sin, case).to(TYPES[case["dtype"]])


def _plain_gradient(s):
    case = s["case"]
    cos, sin = _angles(s)
    x = s["x"].float()
    g = _turned(s["dy"].float(), cos, -sin, case)          # the transposed turn
    inv = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    unit = x * inv
    dw = (g * unit).sum((0, 1))
    g = g * (s["weights"][0] + case["offset"])
    return (inv * (g - unit * (g * unit).mean(-1, keepdim=True))).to(TYPES[case["dtype"]]), dw


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        return _exact_prompt(s)
    if case["op"] == "append":
        return _exact_append(s)
    angle = s["pos"].double()[:, None, None]
    if case["op"] == "rotate":
        return _exact_turn(_exact_norm(s["x"].double(), s["weights"][0], case), angle, case, 1.0)
    # the gradient: dx_i = r (w_i g_i) - r^3 x_i / D sum_j w_j g_j x_j, with g the transposed turn of dy
    x, w = s["x"].double(), s["weights"][0].double() + case["offset"]
    g = _exact_turn(s["dy"].double(), angle, case, -1.0)
    r = 1.0 / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / case["D"] + EPS)
    inner = (w * g * x).sum(-1, keepdim=True)
    return r * w * g - r ** 3 / case["D"] * x * inner, (g * x * r).sum(1).sum(0)


def _exact_prompt(s):
    case, c = s["case"], s["cache"]
    HQ, HKV, D, P = (case[n] for n in ("HQ", "HKV", "D", "P"))
    G, ln, ct, slots, starts = HQ // HKV, _lengths(case), _counts(case), _slots(case), _starts(case)
    if float(((ln + 0.5 * ct) * ct).sum()) * 4 * D * HQ > 8.0e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        if slots[b] < 0 or not ct[b]:
            continue
        pages = c["page_table"][int(slots[b])][:-(-int(ln[b] + ct[b]) // P)].long()
        for h in range(HKV):
            k, v = (c[x][0][pages, h].reshape(-1, D).double() for x in ("k", "v"))
            for t in range(0, int(ct[b]), 512):
                e = min(t + 512, int(ct[b]))
                n, first = int(ln[b]) + e, int(starts[b])
                q = s["q"][first + t:first + e, h * G:(h + 1) * G].double().transpose(0, 1)
                x = torch.einsum("gtd,sd->gts", q, k[:n]) * s["scale"]
                ahead = torch.ones(e - t, n, dtype=torch.bool, device=DEV).triu(int(ln[b]) + t + 1)
                x = torch.softmax(x.masked_fill_(ahead, -math.inf), -1)
                out[first + t:first + e, h * G:(h + 1) * G] = torch.einsum("gts,sd->tgd", x, v[:n])
    return out


def _exact_turn(x, pos, case, sign):
    f, m = _frequencies(case)
    half = case["rot"] // 2
    first = np.arange(half) if case["layout"] == "half" else 2 * np.arange(half)
    other = first + (half if case["layout"] == "half" else 1)
    first, other = torch.as_tensor(first, device=DEV), torch.as_tensor(other, device=DEV)
    angle = pos * torch.as_tensor(f, dtype=torch.float64, device=DEV) * sign
    y = x.clone()
    y[..., first] = m * (x[..., first] * torch.cos(angle) - x[..., other] * torch.sin(angle))
    y[..., other] = m * (x[..., other] * torch.cos(angle) + x[..., first] * torch.sin(angle))
    return y


def _exact_norm(x, w, case):
    return x / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / case["D"] + EPS) * (w.double() + case["offset"])


def _exact_append(s):
    case, c = s["case"], s["cache"]
    hq, hk, P = case["HQ"], case["HKV"], case["P"]
    k, v, starts, ct = c["k"].double(), c["v"].double(), _starts(case), _counts(case)
    angle = s["pos"].double()[:, None, None]
    x = s["qkv"].double()
    q = _exact_turn(_exact_norm(x[:, :hq], s["weights"][0], case), angle, case, 1.0)
    x[:, hq:hq + hk] = _exact_turn(_exact_norm(x[:, hq:hq + hk], s["weights"][1], case), angle, case, 1.0)
    for b in range(case["B"]):
        where = int(c["length"][b]) + torch.arange(int(ct[b]), device=DEV)
        page = c["page_table"][b].long()[where // P]
        row = x[int(starts[b]):int(starts[b + 1])]
        k[0, page, :, where % P] = row[:, hq:hq + hk]
        v[0, page, :, where % P] = row[:, hq + hk:]
    return q, k, v


# ------------------------------------------------------------------ work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "prompt":
        ln, ct, on = _lengths(case), _counts(case), _slots(case) >= 0
        read = int(((ln + ct) * on * (ct > 0)).sum()) * case["HKV"] * case["D"] * 2 * es
        rows = int((ct * on).sum()) * case["HQ"] * case["D"] * es
        pad = int((ct * ~on).sum()) * case["HQ"] * case["D"] * es      # zeros that are written
        pairs = int((on * (ln * ct + ct * (ct + 1) // 2)).sum())
        return {"bytes": read + 2 * rows + pad, "flops": 4 * case["D"] * case["HQ"] * pairs}
    if case["op"] == "append":
        n = int(_counts(case).sum())
        turned = n * (case["HQ"] + case["HKV"])
        return {"bytes": 2 * n * (case["HQ"] + 2 * case["HKV"]) * case["D"] * es,
                "flops": turned * (4 * case["D"] + 3 * case["rot"])}
    n = case["N"] * case["heads"]
    if case["op"] == "rotate":
        return {"bytes": 2 * n * case["D"] * es, "flops": n * (4 * case["D"] + 3 * case["rot"])}
    return {"bytes": 3 * n * case["D"] * es + 4 * case["D"], "flops": n * (12 * case["D"] + 3 * case["rot"])}
