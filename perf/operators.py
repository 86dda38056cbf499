"""The operators of a softmax-attention layer's speculative step, measured: attention of drafted
tokens (a tree) over a paged cache, rotary positions with and without the append to that cache, and
the cache's pages (reserve, fork, commit, free).

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
        # one request, one token, a short context: the latency of a single decode step
        dict(name="attend one token", op="attend", B=1, T=1, HQ=16, HKV=2, D=256, P=16, length=700,
             spread=0, dtype="bf16", tree="chain", ragged=False),
        # plain decode over long contexts, few rows
        dict(name="attend long context", op="attend", B=4, T=1, HQ=32, HKV=8, D=128, P=64,
             length=131072, spread=50, dtype="bf16", tree="chain", ragged=False),
        # a serving batch, trees of eight drafts
        dict(name="attend batch of trees", op="attend", B=128, T=8, HQ=16, HKV=2, D=256, P=64,
             length=4096, spread=70, dtype="bf16", tree="tree", ragged=False),
        # wide trees over grouped heads: 512 query rows for each key/value head, bound by the products
        dict(name="attend wide trees", op="attend", B=32, T=64, HQ=64, HKV=8, D=128, P=128,
             length=8192, spread=40, dtype="bf16", tree="tree", ragged=True),
        # 32-bit inputs, three query heads a group, odd lengths, a padding row and an empty context
        dict(name="attend odd fp32", op="attend", B=7, T=5, HQ=6, HKV=2, D=64, P=16, length=2037,
             spread=90, dtype="fp32", tree="tree", ragged=True),
        # decode: one new token for each of eight requests
        dict(name="append one token", op="append", B=8, T=1, HQ=16, HKV=2, D=256, rot=64, P=16,
             length=900, dtype="bf16", layout="half", scaling="none", ragged=False),
        # the drafted window of a serving batch, a quarter of the head rotated
        dict(name="append windows", op="append", B=128, T=8, HQ=16, HKV=2, D=256, rot=64, P=64,
             length=4096, dtype="bf16", layout="half", scaling="none", ragged=True),
        # a prompt chunk of eight requests at long positions, scaled frequencies
        dict(name="append prompt chunk", op="append", B=8, T=4096, HQ=32, HKV=8, D=128, rot=128, P=64,
             length=100000, dtype="bf16", layout="interleaved", scaling="yarn", ragged=False),
        # the gradient of rotated queries in training, 32 bits
        dict(name="rotate gradient fp32", op="rotate", N=8191, heads=16, D=128, rot=128, dtype="fp32",
             layout="half", scaling="bands", transpose=True),
        # four continuations of one prompt: the bookkeeping's latency
        dict(name="pages four rows", op="pages", B=4, T=4, HKV=2, D=256, P=16, layers=4, length=500,
             parents=1, dtype="bf16"),
        # a serving batch after a step of eight drafts
        dict(name="pages serving batch", op="pages", B=128, T=8, HKV=2, D=256, P=64, layers=12,
             length=4096, parents=32, dtype="bf16"),
        # wide trees, long tables, much to copy
        dict(name="pages wide trees", op="pages", B=256, T=64, HKV=8, D=128, P=128, layers=8,
             length=16000, parents=8, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "append", "rotate", "pages"])
    if kind == "attend":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
        D = rng.choice([64, 128, 256])
        HKV = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 6, 8])
        T = rng.choice([1, 1, 2, 4, 5, 7, 8, 16, 33, 64])
        if dtype == "fp32":
            T = min(T, 8)
            G = min(G, 4)
        B = _log_int(rng, 1, 256)
        # at most 0.35 G values of keys in the cache and 1e11 products
        most = min(3.5e8 / (B * HKV * D), 1.0e11 / (B * T * HKV * G * D))
        if dtype == "fp32":
            most /= 16
        length = _log_int(rng, 33, max(64, min(131072, int(most))))
        return dict(op="attend", B=B, T=T, HQ=HKV * G, HKV=HKV, D=D, P=rng.choice([16, 32, 64, 128]),
                    length=length, spread=rng.choice([0, 30, 60, 90]), dtype=dtype,
                    tree="chain" if T == 1 else rng.choice(["chain", "tree"]),
                    ragged=T > 1 and rng.random() < 0.5)
    if kind == "append":
        D = rng.choice([64, 128, 256])
        HKV = rng.choice([1, 2, 4, 8])
        B = _log_int(rng, 1, 256)
        HQ, dtype = HKV * rng.choice([1, 3, 4, 8]), rng.choice(["bf16", "bf16", "fp32"])
        token = (HQ + 2 * HKV) * D * (4 if dtype == "bf16" else 8)
        T = _log_int(rng, 1, max(2, min(4096, int(8.0e8 / (B * token)))))
        return dict(op="append", B=B, T=T, HQ=HQ, HKV=HKV, D=D,
                    rot=D // rng.choice([1, 2, 4]), P=rng.choice([16, 32, 64, 128]),
                    length=_log_int(rng, 10, 200000), dtype=dtype,
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    ragged=T > 1 and rng.random() < 0.5)
    if kind == "rotate":
        D = rng.choice([64, 96, 128, 256])
        return dict(op="rotate", N=_log_int(rng, 1, 8191), heads=rng.choice([1, 3, 8, 16]), D=D,
                    rot=D // rng.choice([1, 2]), dtype=rng.choice(["bf16", "fp32"]),
                    layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    transpose=rng.random() < 0.5)
    B = _log_int(rng, 1, 256)
    case = dict(op="pages", B=B, T=rng.choice([1, 3, 4, 8, 16, 64]), HKV=rng.choice([1, 2, 8]),
                D=rng.choice([64, 128]), P=rng.choice([16, 32, 64, 128]), layers=1,
                length=_log_int(rng, 20, 16000), parents=rng.randint(1, min(B, 16)),
                dtype=rng.choice(["bf16", "fp32"]))
    tokens = case["parents"] * case["length"] + B * (case["T"] + 3 * case["P"])
    layer = tokens * case["HKV"] * case["D"] * (4 if case["dtype"] == "bf16" else 8)
    return dict(case, layers=rng.randint(1, max(1, min(16, int(6.0e9 / layer)))))


# ------------------------------------------------------------------ what a case fixes

def _lengths(case, rows):
    """Committed tokens of each row: `length` less a part of up to `spread` per cent."""
    n, cut = case["length"], case.get("spread", 40)
    frac = (np.arange(rows) * 0.6180339887498949) % 1.0
    return np.maximum(1, np.round(n * (1 - frac * cut / 100.0))).astype(np.int64)


def _counts(case):
    """Tokens of each row's window."""
    B, T = case["B"], case["T"]
    if not case.get("ragged"):
        return np.full(B, T, np.int64)
    return np.maximum(1, T - (np.arange(B) * 5) % (T // 2 + 1)).astype(np.int64)


def _attend_rows(case):
    """(lengths, counts, slots): an odd case has a padding row and a row without context too."""
    ln, ct = _lengths(case, case["B"]), _counts(case)
    slots = np.arange(case["B"])
    if case["dtype"] == "fp32" and case["B"] >= 3:
        ln[1] = 0
        slots[2] = -1
    return ln, ct, slots


ROPE = {"none": dict(base=1.0e6), "linear": dict(base=1.0e4, factor=4.0),
        "ntk": dict(base=1.0e4, factor=8.0),
        "yarn": dict(base=1.0e4, factor=32.0, original=4096.0, fast=32.0, slow=1.0),
        "bands": dict(base=5.0e5, factor=8.0, original=8192.0, low=1.0, high=4.0)}


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


def _trees(case, counts, r):
    """A random tree for each row (a parent comes before its children): ancestor masks, a path from
    a root to a node, and the path's length."""
    B, T = case["B"], case["T"]
    mask, path, acc = np.zeros((B, T), np.uint64), np.zeros((B, T), np.int64), np.zeros(B, np.int64)
    for b in range(B):
        parent = [-1] * T
        for j in range(int(counts[b])):
            parent[j] = j - 1 if case.get("tree") == "chain" else int(r.integers(max(-1, j - 6), j))
            up = mask[b, parent[j]] if parent[j] >= 0 else np.uint64(0)
            mask[b, j] = up | np.uint64(1 << j)
        node, nodes = int(counts[b]) - 1 - int(r.integers(0, max(1, int(counts[b]) // 2))), []
        while node >= 0:
            nodes.append(node)
            node = parent[node]
        acc[b] = len(nodes)
        path[b, :len(nodes)] = nodes[::-1]
    return mask, path, acc


def _page_table(need, num_slots, max_pages, num_pages, r):
    """Pages handed out in random order, -1 where a slot has none."""
    table = np.full((num_slots, max_pages), -1, np.int64)
    order, at = r.permutation(num_pages), 0
    for s in range(len(need)):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
    return table


def _cache(case, g, layers, num_pages, num_slots, max_pages, fill=True):
    """The framework's cache where it has one; else the same tensors."""
    dims = dict(n_layers=layers, num_pages=num_pages, HKV=case["HKV"], P=case["P"], D=case["D"],
                num_slots=num_slots, max_pages=max_pages)
    shape = (layers, num_pages, case["HKV"], case["P"], case["D"])
    make = (lambda: _normal(g, shape, case["dtype"])) if fill else (
        lambda: torch.zeros(shape, dtype=TYPES[case["dtype"]], device=DEV))
    zeros = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    words = (num_pages + 31) // 32
    return dict(dims=dims, dtype=case["dtype"], k=make(), v=make(),
                page_table=torch.full((num_slots, max_pages), -1, dtype=torch.int32, device=DEV),
                n_pages=zeros(num_slots), length=zeros(num_slots), ref=zeros(num_pages),
                free_bits=zeros(words), status=zeros(4), handle=None)


def _handle(c):
    """The framework's cache over the tensors of `c`, made once and kept, as a program keeps it."""
    if c["handle"] is None:
        from gated_delta_rule_spec_gb300 import binding
        c["handle"] = binding.KvCache(**c["dims"], io_dtype=c["dtype"], tensors={
            n: c[n] for n in ("k", "v", "page_table", "n_pages", "length", "ref", "free_bits", "status")})
    return c["handle"]


def _plan(state):
    """The framework's rotary plan, made once and kept."""
    if state["plan"] is None:
        from gated_delta_rule_spec_gb300 import binding
        case = state["case"]
        p = dict(ROPE[case["scaling"]])
        state["plan"] = binding.RopePlan(case["D"], case["rot"], layout=case["layout"],
                                         scaling=case["scaling"], **p)
    return state["plan"]


def _pack_bits(free):
    """Words of 32 truth values, the first in the lowest bit, as int32."""
    n = free.numel()
    pad = torch.nn.functional.pad(free.to(torch.int64), (0, -n % 32)).view(-1, 32)
    word = (pad << torch.arange(32, device=free.device)).sum(1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


# ------------------------------------------------------------------ prepare

def prepare(case, seed):
    g, r = _generator(seed), np.random.default_rng(int(seed))
    return {"attend": _prepare_attend, "append": _prepare_append, "rotate": _prepare_rotate,
            "pages": _prepare_pages}[case["op"]](case, g, r)


def _prepare_attend(case, g, r):
    B, T, P, D = case["B"], case["T"], case["P"], case["D"]
    ln, ct, slots = _attend_rows(case)
    mask, _, _ = _trees(case, ct, r)
    need = -(-(ln + T) // P)
    num_pages, max_pages = int(need.sum()) + 3, int(need.max())
    c = _cache(case, g, 1, num_pages, B, max_pages)
    c["page_table"].copy_(_int32(_page_table(need, B, max_pages, num_pages, r)))
    c["n_pages"].copy_(_int32(need))
    c["length"].copy_(_int32(ln))
    q = _normal(g, (B, T, case["HQ"], D), case["dtype"])
    return dict(case=case, cache=c, q=q, slots=_int32(slots), counts=_int32(ct),
                mask=torch.as_tensor(mask.view(np.int64), device=DEV), scale=D ** -0.5, work=None)


def _prepare_append(case, g, r):
    B, T, P, D = case["B"], case["T"], case["P"], case["D"]
    ln, ct = _lengths(case, B) % (4 * P), _counts(case)   # where in its pages a row ends; its positions run on
    need = -(-(ln + T) // P)
    num_pages, max_pages = int(need.sum()) + 1, int(need.max())
    c = _cache(case, g, 1, num_pages, B, max_pages, fill=False)
    c["page_table"].copy_(_int32(_page_table(need, B, max_pages, num_pages, r)))
    c["n_pages"].copy_(_int32(need))
    c["length"].copy_(_int32(ln))
    heads = case["HQ"] + 2 * case["HKV"]
    qkv = _normal(g, (B, T, heads, D), case["dtype"])     # one projection's output, q, k and v side by side
    pos = _lengths(case, B)[:, None] + np.arange(T)[None]
    f, m = _frequencies(case)
    first, rows = int(pos.min()), int(pos.max()) - int(pos.min()) + 1
    return dict(case=case, cache=c, qkv=qkv, slots=_int32(np.arange(B)), counts=_int32(ct), pos=_int32(pos),
                plan=None, table=_table(first, rows, f, m), first=first)


def _table(first, rows, f, m):
    """cos and sin of the positions in use, in 32 bits, as a program keeps them."""
    a = torch.arange(first, first + rows, dtype=torch.float64, device=DEV)[:, None] * torch.as_tensor(f, device=DEV)
    return torch.stack([torch.cos(a) * m, torch.sin(a) * m]).float()


def _prepare_rotate(case, g, r):
    x = _normal(g, (case["N"], case["heads"], case["D"]), case["dtype"])
    f, m = _frequencies(case)
    return dict(case=case, x=x, pos=_int32(np.arange(case["N"])), plan=None, table=_table(0, case["N"], f, m),
                first=0)


def _prepare_pages(case, g, r):
    B, T, P, par = case["B"], case["T"], case["P"], case["parents"]
    ln = np.maximum(_lengths(case, par), 1)
    need = -(-ln // P)
    src = np.arange(B) % par
    each = 1 + -(-T // P) + 1                              # a copied page and those of the drafts
    num_pages = int(need.sum()) + B * each
    max_pages = int(need.max()) + each
    num_slots = par + B
    c = _cache(case, g, case["layers"], num_pages, num_slots, max_pages)
    table = _page_table(need, num_slots, max_pages, num_pages, r)
    c["page_table"].copy_(_int32(table))
    c["n_pages"][:par] = _int32(need)
    c["length"][:par] = _int32(ln)
    held = torch.as_tensor(table[table >= 0], device=DEV)
    c["ref"][held] = 1
    c["free_bits"].copy_(_pack_bits(c["ref"] == 0))
    _, path, acc = _trees(case, np.full(B, T), r)
    return dict(case=case, cache=c, src=_int32(src), dst=_int32(par + np.arange(B)), path=_int32(path),
                acc=_int32(acc), done=torch.zeros(2, B, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------------ run

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "append": _own_append, "rotate": _own_rotate, "pages": _own_pages}[op](state)
    return {"attend": _plain_attend, "append": _plain_append, "rotate": _plain_rotate, "pages": _plain_pages}[op](state)


def _own_attend(s):
    from gated_delta_rule_spec_gb300 import binding
    case, c = s["case"], _handle(s["cache"])
    if s["work"] is None:
        s["work"] = torch.empty(binding.tree_attn_workspace(c, case["B"], case["T"], case["HQ"]),
                                dtype=torch.uint8, device=DEV)
    return binding.tree_attn(c, 0, s["slots"], s["q"], s["mask"] if case["tree"] == "tree" else None,
                             s["counts"] if case["ragged"] else None, scale=s["scale"], workspace=s["work"])


def _own_append(s):
    from gated_delta_rule_spec_gb300 import binding
    case, c = s["case"], _handle(s["cache"])
    hq, hk = case["HQ"], case["HKV"]
    q, k, v = s["qkv"][:, :, :hq], s["qkv"][:, :, hq:hq + hk], s["qkv"][:, :, hq + hk:]
    out = binding.rope_append(_plan(s), c, 0, s["slots"], q, k, v, pos=s["pos"],
                              n_tokens=s["counts"] if case["ragged"] else None)
    return out, c.k, c.v


def _own_rotate(s):
    from gated_delta_rule_spec_gb300 import binding
    return binding.rope(_plan(s), s["pos"], s["x"], transpose=s["case"]["transpose"])


def _own_pages(s):
    from gated_delta_rule_spec_gb300 import binding
    c, T = _handle(s["cache"]), s["case"]["T"]
    binding.kv_free(c, s["dst"])
    binding.kv_fork(c, s["src"], s["dst"], done=s["done"][0])
    binding.kv_reserve(c, s["dst"], T, done=s["done"][1])
    binding.kv_commit(c, s["dst"], s["acc"], T, path=s["path"])
    return c.page_table, c.n_pages, c.length, c.ref, c.free_bits, s["done"], c.k, c.v


def _visible(s, S):
    """[B, T, S]: what each drafted token attends to."""
    case, c = s["case"], s["cache"]
    T = case["T"]
    on = s["slots"] >= 0
    ln = torch.where(on, c["length"][s["slots"].long().clamp(min=0)], 0).long()
    at = torch.arange(S, device=DEV)
    node = at[None] - ln[:, None]                                        # which drafted token a position is
    bit = (s["mask"][:, :, None] >> node.clamp(0, 63)[:, None]) & 1
    inside = (node >= 0) & (node < s["counts"][:, None])
    seen = (at[None] < ln[:, None])[:, None] | (inside[:, None] & (bit != 0))
    row = (torch.arange(T, device=DEV)[None] < s["counts"][:, None]) & on[:, None]
    return seen & row[:, :, None]


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    B, T, HQ, HKV, D = case["B"], case["T"], case["HQ"], case["HKV"], case["D"]
    table = c["page_table"][s["slots"].long().clamp(min=0)].long().clamp(min=0)
    S = table.shape[1] * case["P"]
    k = c["k"][0][table].permute(0, 2, 1, 3, 4).reshape(B, HKV, S, D).float()
    q = s["q"].float().view(B, T, HKV, HQ // HKV, D).permute(0, 2, 1, 3, 4).reshape(B, HKV, -1, D)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, HKV, T, HQ // HKV, S)
    del k
    x = x.masked_fill_(~_visible(s, S)[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_(min=-3.0e38)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    v = c["v"][0][table].permute(0, 2, 1, 3, 4).reshape(B, HKV, S, D).float()
    o = x.view(B, HKV, -1, S) @ v
    o = o.view(B, HKV, T, HQ // HKV, D) / torch.where(total > 0, total, 1.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, HQ, D).to(TYPES[case["dtype"]])


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


def _plain_append(s):
    case, c = s["case"], s["cache"]
    B, T, P, hq, hk = case["B"], case["T"], case["P"], case["HQ"], case["HKV"]
    row = s["pos"].long() - s["first"]
    cos, sin = s["table"][0][row][:, :, None], s["table"][1][row][:, :, None]
    x = _turned(s["qkv"][:, :, :hq + hk].float(), cos, sin, case).to(TYPES[case["dtype"]])
    t = torch.arange(T, device=DEV)
    live = t[None] < s["counts"][:, None]
    q = torch.where(live[:, :, None, None], x[:, :, :hq], 0)
    # a token past the row's count writes nothing: it goes where its row's last one goes, with that value
    t = torch.minimum(t[None], s["counts"][:, None].long() - 1)
    at = c["length"][:, None].long() + t
    page, off = c["page_table"].long().gather(1, at // P), at % P
    b = torch.arange(B, device=DEV)[:, None]
    c["k"][0][page, :, off] = x[:, :, hq:][b, t]
    c["v"][0][page, :, off] = s["qkv"][:, :, hq + hk:][b, t]
    return q, c["k"], c["v"]


def _plain_rotate(s):
    case = s["case"]
    row = s["pos"].long() - s["first"]
    cos, sin = s["table"][0][row][:, None], s["table"][1][row][:, None]
    return _turned(s["x"].float(), cos, -sin if case["transpose"] else sin, case).to(TYPES[case["dtype"]])


def _plain_pages(s):
    case, c = s["case"], s["cache"]
    B, T, P = case["B"], case["T"], case["P"]
    src, dst = s["src"].long(), s["dst"].long()
    k, v, ref, length, table = c["k"], c["v"], c["ref"], c["length"], c["page_table"]
    M = table.shape[1]
    col = torch.arange(M, device=DEV)[None]
    # free: the slots' pages lose a holder
    held = col < c["n_pages"][dst][:, None]
    ref.index_add_(0, table[dst].clamp(min=0).long().flatten(), -held.flatten().to(torch.int32))
    # fork: full pages are shared, a part of a page is copied to a free one (the lowest first)
    ln = length[src].long()
    full, part = ln // P, ln % P
    need = (part > 0).long()
    free = torch.argsort((ref != 0).to(torch.int8), stable=True)
    page = free[(need.cumsum(0) - need)]
    t = torch.where(col < full[:, None], table[src], -1)
    t = torch.where((col == full[:, None]) & (need[:, None] > 0), page[:, None].to(torch.int32), t)
    table[dst] = t
    ref.index_add_(0, t.clamp(min=0).long().flatten(), (t >= 0).flatten().to(torch.int32))
    old = table[src].long().gather(1, (full[:, None]).clamp(max=M - 1))[:, 0].clamp(min=0)
    old = torch.where(need > 0, old, table[src][:, 0].long())
    new = torch.where(need > 0, page, old)                               # no copy: a page onto itself
    some = (torch.arange(P, device=DEV)[None] < part[:, None])[None, :, None, :, None]
    k[:, new] = torch.where(some, k[:, old], k[:, new])
    v[:, new] = torch.where(some, v[:, old], v[:, new])
    length[dst] = ln.to(torch.int32)
    # reserve: pages for T more tokens
    have = full + need
    want = -(-(ln + T) // P) - have
    free = torch.argsort((ref != 0).to(torch.int8), stable=True)
    rank = (want.cumsum(0) - want)[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + want)[:, None])
    t = torch.where(fresh, free[rank.clamp(0, free.numel() - 1)].to(torch.int32), t)
    table[dst] = t
    ref.index_add_(0, t.clamp(min=0).long().flatten(), fresh.flatten().to(torch.int32))
    c["n_pages"][dst] = (have + want).to(torch.int32)
    # commit: the accepted drafts move together, in place
    i = torch.arange(T, device=DEV)[None]
    keep = i < s["acc"][:, None]
    to = ln[:, None] + i
    frm = torch.where(keep, ln[:, None] + s["path"], to)
    tl = t.long()
    pf, pt, of, ot = tl.gather(1, frm // P), tl.gather(1, to // P), frm % P, to % P
    k[:, pt, :, ot] = k[:, pf, :, of]
    v[:, pt, :, ot] = v[:, pf, :, of]
    length[dst] = (ln + s["acc"]).to(torch.int32)
    c["free_bits"].copy_(_pack_bits(ref == 0))
    s["done"].fill_(1)
    return table, c["n_pages"], length, ref, c["free_bits"], s["done"], k, v


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "rotate":
        f, m = _frequencies(case)
        return _exact_turn(s["x"].double(), s["pos"].double()[:, None, None], f, m, case,
                           -1.0 if case["transpose"] else 1.0)
    return None


def _exact_attend(s):
    case, c = s["case"], s["cache"]
    B, T, HQ, HKV, D, P = (case[n] for n in ("B", "T", "HQ", "HKV", "D", "P"))
    G = HQ // HKV
    ln, ct, slots = _attend_rows(case)
    if sum(int(x) for x in ln) * T * HQ * D > 4.0e12:
        return None
    out = torch.zeros(B, T, HQ, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        if slots[b] < 0:
            continue
        n = int(ln[b] + ct[b])
        pages = c["page_table"][int(slots[b])][:-(-n // P)].long()
        see = torch.ones(int(ct[b]), n, dtype=torch.bool, device=DEV)
        for t in range(int(ct[b])):
            word = int(s["mask"][b, t].item()) & (2 ** 64 - 1)
            see[t, int(ln[b]):] = torch.tensor([bool(word >> j & 1) for j in range(int(ct[b]))], device=DEV)
        for h in range(HKV):
            k = c["k"][0][pages, h].reshape(-1, D)[:n].double()
            v = c["v"][0][pages, h].reshape(-1, D)[:n].double()
            q = s["q"][b, :int(ct[b]), h * G:(h + 1) * G].double().reshape(-1, D)
            x = (q @ k.T) * s["scale"]
            x = x.view(-1, G, n).masked_fill(~see[:, None], -math.inf).view(-1, n)
            out[b, :int(ct[b]), h * G:(h + 1) * G] = (torch.softmax(x, -1) @ v).view(-1, G, D)
    return out


def _exact_turn(x, pos, f, m, case, sign):
    half = case["rot"] // 2
    first = np.arange(half) if case["layout"] == "half" else 2 * np.arange(half)
    other = first + (half if case["layout"] == "half" else 1)
    first, other = torch.as_tensor(first, device=DEV), torch.as_tensor(other, device=DEV)
    angle = pos * torch.as_tensor(f, dtype=torch.float64, device=DEV) * sign
    y = x.clone()
    y[..., first] = m * (x[..., first] * torch.cos(angle) - x[..., other] * torch.sin(angle))
    y[..., other] = m * (x[..., other] * torch.cos(angle) + x[..., first] * torch.sin(angle))
    return y


def _exact_append(s):
    case, c = s["case"], s["cache"]
    hq, hk, P = case["HQ"], case["HKV"], case["P"]
    f, m = _frequencies(case)
    k, v = c["k"].double(), c["v"].double()
    q = torch.zeros(case["B"], case["T"], hq, case["D"], dtype=torch.float64, device=DEV)
    for b in range(case["B"]):
        n, at = int(s["counts"][b]), int(c["length"][b])
        x = s["qkv"][b, :n].double()
        x[:, :hq + hk] = _exact_turn(x[:, :hq + hk], s["pos"][b, :n].double()[:, None, None], f, m, case, 1.0)
        q[b, :n] = x[:, :hq]
        where = at + torch.arange(n, device=DEV)
        page = c["page_table"][b].long()[where // P]
        k[0, page, :, where % P] = x[:, hq:hq + hk]
        v[0, page, :, where % P] = x[:, hq + hk:]
    return q, k, v


# ------------------------------------------------------------------ work

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "attend":
        ln, ct, slots = _attend_rows(case)
        on = slots >= 0
        read = int(((ln + ct) * on).sum()) * case["HKV"] * case["D"] * 2 * es
        rows = case["B"] * case["T"] * case["HQ"] * case["D"] * es
        return {"bytes": read + 2 * rows, "flops": 4 * case["D"] * case["HQ"] * int(((ln + 1) * ct * on).sum())}
    if case["op"] == "append":
        live = int(_counts(case).sum())
        heads = case["HQ"] + 2 * case["HKV"]
        dead = case["B"] * case["T"] - live
        return {"bytes": (2 * live * heads + dead * case["HQ"]) * case["D"] * es,
                "flops": 3 * live * (case["HQ"] + case["HKV"]) * case["rot"]}
    if case["op"] == "rotate":
        n = case["N"] * case["heads"]
        return {"bytes": 2 * n * case["D"] * es, "flops": 3 * n * case["rot"]}
    # the copied parts of pages, the moved drafts (about half of a path moves), the tables
    ln = np.maximum(_lengths(case, case["parents"]), 1)
    src = np.arange(case["B"]) % case["parents"]
    token = case["layers"] * case["HKV"] * case["D"] * 2 * es
    part = int((ln[src] % case["P"]).sum())
    pages = int((-(-ln // case["P"]))[src].sum()) + 2 * case["B"]
    return {"bytes": 2 * part * token + case["B"] * token + 16 * pages, "flops": pages}
