"""More operators of a decode or prompt step, as they are measured: products
with 4-bit weights and group scales, the norm and rotary positions of query and
key heads, and attention over a paged 8-bit cache of which a batch shares a
prefix.

``run`` computes a case with the library's entry points where ``own`` is
true, else in plain torch operations in fp32.  ``exact`` computes it in 64
bits from the definitions.

Definitions.  A 4-bit weight is (q - zero)·scale with q from 0 to 15, two to a
byte, the even column in the low half, and one scale and zero (8, where there
is none) for each row and group of columns.  A head is divided by the root of
its mean square and weighted, then its first columns are rotated in pairs by
position·frequency.  A cache block holds 16 tokens of one head in int8 or e4m3
with one fp32 scale each for K and V.  K is stored (pages, heads, page_size,
dim), V (pages, heads, page_size / 16, dim, 16).
"""

import math
import random

import torch

own = False

DEVICE = "cuda"
TOKENS = 16          # tokens of a cache block
EPS = 1e-6           # of the norm
FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one decoded token through an output projection: latency counts
        dict(name="product 1 token", op="product", tokens=1, rows=4096, cols=4096, group=128, zero=False, dtype="f16",
             out="f32", bias=False),
        # one token through a projection with long rows, straight from fp32 activations
        dict(name="product 1 token long rows", op="product", tokens=1, rows=4096, cols=11008, group=32, zero=True,
             dtype="f32", out="f32", bias=True),
        # the gate projection of 16 sequences that each decode one token
        dict(name="product 16 tokens gate", op="product", tokens=16, rows=14336, cols=4096, group=128, zero=True,
             dtype="bf16", out="bf16", bias=False),
        # a prompt through the gate projection
        dict(name="product 2000 tokens gate", op="product", tokens=2000, rows=14336, cols=4096, group=64, zero=True,
             dtype="bf16", out="bf16", bias=False),
        # one decoded token's heads, without norms: a launch's latency
        dict(name="rotary 1 token", op="rotary", batch=1, longest=4000, new=1, q_heads=32, heads=8, dim=128, rotated=128,
             interleaved=False, norm=False, dtype="bf16", q_out="bf16", k_out="bf16", magnitude=1.0),
        # 64 sequences' heads straight from fp32 products; keys stay fp32 for the append
        dict(name="rotary 64 tokens fp32", op="rotary", batch=64, longest=8192, new=1, q_heads=32, heads=8, dim=128,
             rotated=128, interleaved=False, norm=True, dtype="f32", q_out="bf16", k_out="f32", magnitude=1.0),
        # prompts of a batch with normed heads
        dict(name="rotary prompts", op="rotary", batch=5, longest=4096, new=3000, q_heads=32, heads=8, dim=128,
             rotated=128, interleaved=False, norm=True, dtype="bf16", q_out="bf16", k_out="bf16", magnitude=1.0),
        # the end of a very long context, a quarter of each wide head rotated in neighbouring pairs, scaled
        dict(name="rotary far positions", op="rotary", batch=3, longest=131071, new=1999, q_heads=16, heads=16, dim=256,
             rotated=64, interleaved=True, norm=False, dtype="f16", q_out="f16", k_out="f16", magnitude=1.2079),
        # four answers to one question: latency counts
        dict(name="attend 4 shared 2000", op="attend", batch=4, shared=2000, tail=100, new=1, q_heads=32, heads=8,
             dim=128, page=64, format="int8", dtype="f16", window=0, sinks=0),
        # a serving batch behind one long instruction
        dict(name="attend 64 shared 8192", op="attend", batch=64, shared=8192, tail=1000, new=1, q_heads=32, heads=8,
             dim=128, page=64, format="e4m3", dtype="bf16", window=0, sinks=0),
        # 16 questions about one very long document
        dict(name="attend 16 shared 65536", op="attend", batch=16, shared=65536, tail=500, new=1, q_heads=32, heads=8,
             dim=128, page=128, format="int8", dtype="bf16", window=0, sinks=0),
        # short prompts behind one cached prefix
        dict(name="attend prompts shared 4000", op="attend", batch=12, shared=4000, tail=300, new=150, q_heads=32,
             heads=8, dim=128, page=16, format="e4m3", dtype="bf16", window=0, sinks=0),
    ]


def _between(rng, low, high):
    """Whole number between low and high, spread over the logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def _aligned(rng, n):
    """n itself (odd as it may be), or the multiple of 16 or 128 above it, as most models have."""
    step = rng.choice((1, 16, 128))
    return -(-n // step) * step


def draw(rng):
    op = rng.choice(("product", "rotary", "attend"))
    if op == "product":
        while True:
            dtype = rng.choice(("f32", "f16", "bf16"))
            c = dict(op=op, tokens=rng.choice((1, _between(rng, 1, 64), _between(rng, 1, 4096))),
                     rows=_aligned(rng, _between(rng, 64, 16384)), cols=_aligned(rng, _between(rng, 64, 16384)),
                     group=rng.choice((32, 64, 128, 128)), zero=rng.random() < 0.6, dtype=dtype,
                     out=rng.choice(("f32", dtype)), bias=rng.random() < 0.4)
            # (fp32 vectors go to the matrix cores in three parts)
            if c["tokens"] * c["rows"] * c["cols"] * (4 if dtype == "f32" else 1) <= 2000 * 14336 * 4096:
                return c
    if op == "rotary":
        while True:
            dim = rng.choice((64, 80, 96, 128, 128, 256, 2 * rng.randint(8, 128)))
            heads = rng.choice((1, 2, 4, 8, 16))
            dtype = rng.choice(("f32", "f16", "bf16"))
            longest = _between(rng, 16, 131072)
            half = rng.choice((dtype, "bf16") if dtype == "f32" else (dtype,))
            c = dict(op=op, batch=_between(rng, 1, 64), longest=longest,
                     new=rng.choice((1, _between(rng, 2, min(longest, 4096)))), q_heads=heads * rng.choice((1, 2, 4, 5, 8)),
                     heads=heads, dim=dim, rotated=rng.choice((dim, dim, dim // 4 * 2, 2 * rng.randint(1, dim // 2))),
                     interleaved=rng.random() < 0.4, norm=rng.random() < 0.5, dtype=dtype, q_out=half,
                     k_out=rng.choice((dtype, half)), magnitude=rng.choice((1.0, 1.0, 1.2079)))
            if c["batch"] * c["new"] * (c["q_heads"] + heads) * dim * SIZE[dtype] <= 5 * 3000 * 40 * 128 * 2:
                return c
    while True:
        heads = rng.choice((1, 2, 4, 8, 16))
        shared, tail = _between(rng, 16, 65536), _between(rng, 1, 2000)
        c = dict(op=op, batch=_between(rng, 2, 96), shared=shared, tail=tail,
                 new=rng.choice((1, 1, _between(rng, 1, min(tail, 200)))), q_heads=heads * rng.choice((1, 2, 4, 5, 8)),
                 heads=heads, dim=rng.choice((64, 128, 128, 256)), page=rng.choice((16, 32, 64, 128)),
                 format=rng.choice(("int8", "e4m3")), dtype=rng.choice(("f16", "bf16")),
                 window=rng.choice((0, 0, 0, _between(rng, 16, shared + tail))), sinks=rng.choice((0, 4, 70)))
        if (c["batch"] * c["new"] * (shared + tail) * c["q_heads"] * c["dim"] <= 12 * 150 * 4300 * 32 * 128
                and c["batch"] * c["new"] * (shared + tail) * c["q_heads"] <= 16 * 66036 * 32 * 4
                and (shared + c["batch"] * tail) * heads * c["dim"] <= 73728 * 8 * 128):
            return c


# ---------------------------------------------------------------------------
# a batch's lengths, by the case alone
# ---------------------------------------------------------------------------

def _lengths(case):
    """(length after the call, new tokens) of each sequence."""
    before, longest = case.get("shared", 0), case["tail"] if "tail" in case else case["longest"]
    r = random.Random(case["batch"] * 1000003 + longest * 31 + case["new"])
    lens, new = [], []
    for b in range(case["batch"]):
        n = case["new"] if b == 0 or case["new"] == 1 else r.randint(1, case["new"])
        lens.append(before + (longest if b == 0 else r.randint(n, longest)))
        new.append(n)
    return lens, new


def _visible(case):
    """(query-token pairs, tokens that any query sees, the shared ones once) over the whole batch."""
    pairs = tokens = 0
    w, s, shared = case["window"], case["sinks"], case["shared"]
    lens, new = _lengths(case)
    least = shared
    for n, m in zip(lens, new):
        first = n - m
        for p in range(first, n):
            low = max(0, p - w + 1) if w else 0
            pairs += p + 1 - low + min(low, s)
        low = max(0, first - w + 1) if w else 0
        least = min(least, low)
        tokens += n - max(low, shared) + max(0, min(low, s) - shared)
    return pairs, tokens + shared - least + min(least, s)


def work(case):
    op = case["op"]
    if op == "product":
        t, m, k = case["tokens"], case["rows"], case["cols"]
        size, groups = SIZE[case["dtype"]], -(-k // case["group"])
        return {"bytes": m * -(-k // 2) + m * groups * (size + case["zero"]) + t * k * size + t * m * SIZE[case["out"]]
                + 4 * m * case["bias"], "flops": 2 * t * m * k}
    lens, new = _lengths(case)
    total, d = sum(new), case["dim"]
    if op == "rotary":
        q, k = total * case["q_heads"] * d, total * case["heads"] * d
        size = SIZE[case["dtype"]]
        return {"bytes": q * (size + SIZE[case["q_out"]]) + k * (size + SIZE[case["k_out"]]) + 2 * case["rotated"],
                "flops": (q + k) * (3 + 4 * case["norm"])}
    pairs, tokens = _visible(case)
    h = case["heads"]
    q = total * case["q_heads"] * d * SIZE[case["dtype"]]
    return {"bytes": 2 * tokens * h * d + 8 * h * -(-tokens // TOKENS) + 2 * q, "flops": 4 * pairs * case["q_heads"] * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _activations(g, rows, cols):
    """Hidden states: normal, with a few channels far larger than the others, as trained models have them."""
    x = torch.randn(rows, cols, device=DEVICE, generator=g)
    loud = torch.rand(cols, device=DEVICE, generator=g) < 0.005
    return x * torch.where(loud, 20.0, 1.0)


def _weights(case, g):
    """Normal weights held in 4 bits: (packed codes, scales, zeros or None)."""
    m, k, group = case["rows"], case["cols"], case["group"]
    w = torch.randn(m, k, device=DEVICE, generator=g) * 0.02
    w = torch.nn.functional.pad(w, (0, -k % group)).view(m, -1, group)
    if case["zero"]:
        low = torch.clamp(w.amin(dim=2), max=0.0)
        scale = ((torch.clamp(w.amax(dim=2), min=0.0) - low) / 15.0 + 1e-8).to(FLOAT[case["dtype"]])
        zero = torch.clamp(torch.round(-low / scale.float()), 0, 15)
    else:
        scale = (w.abs().amax(dim=2) / 7.5 + 1e-8).to(FLOAT[case["dtype"]])
        zero = torch.full_like(w[:, :, 0], 8.0)
    q = torch.clamp(torch.round(w / scale.float()[:, :, None]) + zero[:, :, None], 0, 15).to(torch.uint8)
    q = torch.nn.functional.pad(q.view(m, -1)[:, :k], (0, k % 2))
    return (q[:, ::2] | q[:, 1::2] << 4).contiguous(), scale, zero.to(torch.uint8) if case["zero"] else None


def _tables(case, g):
    """The pages: whole shared ones named by every sequence, own ones behind them, -1 in the unused entries.
    (number of pages, table, the column of the first own pages)"""
    lens, _ = _lengths(case)
    page = case["page"]
    both = case["shared"] // page
    need = [-(-n // page) - both for n in lens]
    order = torch.randperm(both + sum(need), device=DEVICE, generator=g).to(torch.int32) + 1
    table = torch.full((case["batch"], both + max(need)), -1, dtype=torch.int32, device=DEVICE)
    table[:, :both] = order[:both]
    held = torch.arange(max(need), device=DEVICE)[None, :] < torch.tensor(need, device=DEVICE)[:, None]
    table[:, both:][held] = order[both:]
    return both + sum(need) + 1, table, both


def _fill(case, g, pages, table, both):
    """A cache as many appends leave it: values over the whole 8-bit range, scales that are powers of two.
    A page that is shared in part is a copy of the first sequence's."""
    h, d, page, per = case["heads"], case["dim"], case["page"], case["page"] // TOKENS
    out = {}
    for name, shape in (("k", (pages, h, page, d)), ("v", (pages, h, per, d, TOKENS))):
        x = torch.empty(shape, device=DEVICE).normal_(generator=g)
        x = torch.clamp(x * 38.0, -127.0, 127.0).round_().to(torch.int8) if case["format"] == "int8" else \
            torch.clamp(x * 130.0, -448.0, 448.0).to(torch.float8_e4m3fn)
        out[name] = x
        up = torch.randint(0, 3, (pages, h, per), device=DEVICE, generator=g).float()
        out[name + "_scale"] = torch.exp2(up - 6.0 if case["format"] == "int8" else up - 8.0)
    if case["shared"] % page:
        into = table[:, both].long()
        for x in out.values():
            x = x.view(torch.uint8) if x.element_size() == 1 else x
            x[into] = x[into[:1]].clone()
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 7919 + 13)
    op = case["op"]
    s = {"case": case}
    if op == "product":
        s["q"], s["scale"], s["zero"] = _weights(case, g)
        s["x"] = _activations(g, case["tokens"], case["cols"]).to(FLOAT[case["dtype"]])
        s["bias"] = torch.randn(case["rows"], device=DEVICE, generator=g) if case["bias"] else None
        return s
    lens, new = _lengths(case)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    total, d = starts[-1], case["dim"]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEVICE)
    s["starts"] = None if case["new"] == 1 else torch.tensor(starts, dtype=torch.int32, device=DEVICE)
    if op == "rotary":
        # queries, keys and values side by side, as one product gives them
        qh, h, pairs = case["q_heads"], case["heads"], case["rotated"] // 2
        both = torch.randn(total, (qh + 2 * h) * d, device=DEVICE, generator=g).to(FLOAT[case["dtype"]]).view(total, -1, d)
        s["xq"], s["xk"] = both[:, :qh], both[:, qh:qh + h]
        s["freq"] = torch.exp(torch.arange(pairs, device=DEVICE).double() * (-math.log(500000.0) / pairs)).float()
        for name in ("q_weight", "k_weight"):
            s[name] = 1.0 + 0.2 * torch.randn(d, device=DEVICE, generator=g) if case["norm"] else None
        return s
    pages, s["table"], both = _tables(case, g)
    s["cache"] = _fill(case, g, pages, s["table"], both)
    s["query"] = torch.randn(total, case["q_heads"], d, device=DEVICE, generator=g).to(FLOAT[case["dtype"]])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "product":
        return _product(case, state)
    if case["op"] == "rotary":
        return _rotary(case, state)
    return _attend(case, state)


def _run_own(case, state):
    import memory_bound_gemv_f32_amd as lg
    if case["op"] == "product":
        return lg.gemv_q4(state["q"], state["scale"], state["x"], state["bias"], zero=state["zero"],
                          group=case["group"], out_dtype=FLOAT[case["out"]])
    if case["op"] == "rotary":
        return lg.gemv_rotary(state["xq"], state["xk"], state["freq"], state["lens"], state["starts"],
                              q_weight=state["q_weight"], k_weight=state["k_weight"], eps=EPS,
                              interleaved=case["interleaved"], magnitude=case["magnitude"],
                              q_dtype=FLOAT[case["q_out"]], k_dtype=FLOAT[case["k_out"]])
    c = state["cache"]
    cache = lg.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    return lg.gemv_kv_attend(state["query"], cache, state["table"], state["lens"], state["starts"],
                             window=case["window"], sinks=case["sinks"], shared=case["shared"])


def _product(case, state):
    m, k = case["rows"], case["cols"]
    q = torch.stack((state["q"] & 15, state["q"] >> 4), dim=2).view(m, -1)
    w = torch.nn.functional.pad(q, (0, max(0, -(-k // case["group"]) * case["group"] - q.shape[1]))).float()
    w = w.view(m, -1, case["group"])
    w = (w - (8.0 if state["zero"] is None else state["zero"].float()[:, :, None])) * state["scale"].float()[:, :, None]
    y = state["x"].float() @ w.view(m, -1)[:, :k].t()
    if state["bias"] is not None:
        y += state["bias"]
    return y.to(FLOAT[case["out"]])


def _sequences(state, total):
    """Of each row its sequence and its position, and the first rows of the sequences."""
    lens = state["lens"].long()
    starts = torch.arange(len(lens) + 1, device=DEVICE) if state["starts"] is None else state["starts"].long()
    row = torch.arange(total, device=DEVICE)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return starts, seq, lens[seq] - starts[seq + 1] + row


def _rotary(case, state):
    _, _, pos = _sequences(state, state["xq"].shape[0])
    angle = pos[:, None, None].double() * state["freq"].double()
    cos, sin = (angle.cos() * case["magnitude"]).float(), (angle.sin() * case["magnitude"]).float()

    def turned(x, weight, out):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(dim=2, keepdim=True) + EPS) * weight
        r = case["rotated"]
        if case["interleaved"]:
            a, b = x[..., 0:r:2], x[..., 1:r:2]
            pairs = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=3).flatten(2)
        else:
            a, b = x[..., :r // 2], x[..., r // 2:r]
            pairs = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=2)
        return torch.cat((pairs, x[..., r:]), dim=2).to(FLOAT[out])

    return (turned(state["xq"], state["q_weight"], case["q_out"]),
            turned(state["xk"], state["k_weight"], case["k_out"]))


def _attend(case, state):
    cache, q = state["cache"], state["query"]
    h, d, page, group = case["heads"], case["dim"], case["page"], case["q_heads"] // case["heads"]
    batch, both = case["batch"], case["shared"] // page
    total, most = q.shape[0], case["new"]
    starts, seq, pos = _sequences(state, total)
    table = torch.clamp(state["table"].long(), min=0)

    def gather(pages):
        """Keys and values of (n, pages) pages as (n, heads, tokens, dim)."""
        n = pages.shape[0]
        k = cache["k"][pages].float().view(n, -1, h, page // TOKENS, TOKENS, d) * cache["k_scale"][pages][..., None, None]
        v = cache["v"][pages].float() * cache["v_scale"][pages][..., None, None]
        return (k.transpose(1, 2).reshape(n, h, -1, d),
                v.transpose(1, 2).transpose(4, 5).reshape(n, h, -1, d))

    k0, v0 = gather(table[:1, :both])
    k1, v1 = gather(table[:, both:])
    # the queries padded to the longest sequence's
    at = torch.arange(total, device=DEVICE) - starts[seq]
    rows = torch.zeros(batch, most, h, group, d, device=DEVICE)
    rows[seq, at] = q.float().view(total, h, group, d) * (1.0 / math.sqrt(d))
    where = torch.full((batch, most), -1, dtype=torch.long, device=DEVICE)
    where[seq, at] = pos
    rows = rows.permute(0, 2, 1, 3, 4).reshape(batch, h, most * group, d)
    # every row with the shared tokens, then each sequence with its own
    once = rows.transpose(0, 1).reshape(h, batch * most * group, d)
    s0 = (once @ k0[0].transpose(1, 2).contiguous()).view(h, batch, most * group, -1).transpose(0, 1)
    s = torch.cat((s0, rows @ k1.transpose(2, 3).contiguous()), dim=3)
    j = torch.arange(s.shape[3], device=DEVICE)
    sees = j <= where[:, :, None]
    if case["window"]:
        sees &= (where[:, :, None] - j < case["window"]) | (j < case["sinks"])
    s = s.view(batch, h, most, group, -1).masked_fill_(~sees[:, None, :, None], -math.inf)
    p = torch.exp(s - torch.clamp(s.amax(dim=-1, keepdim=True), min=-1e30))
    l = torch.clamp(p.sum(dim=-1, keepdim=True), min=1e-30)
    p = p.view(batch, h, most * group, -1)
    p0 = p[..., :both * page].transpose(0, 1).reshape(h, batch * most * group, both * page)
    o = (p0 @ v0[0]).view(h, batch, most * group, d).transpose(0, 1) + p[..., both * page:].contiguous() @ v1
    o = o.reshape(batch, h, most, group, d) / l
    return o.permute(0, 2, 1, 3, 4)[seq, at].reshape(total, case["q_heads"], d).to(q.dtype)


# ---------------------------------------------------------------------------
# in 64 bits, from the definitions
# ---------------------------------------------------------------------------

def _e4m3_grid():
    """The values of the bytes 0 to 255."""
    grid = []
    for byte in range(256):
        e, m = byte >> 3 & 15, byte & 7
        x = math.nan if (byte & 127) == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        grid.append(-x if byte & 128 else x)
    return torch.tensor(grid, dtype=torch.float64, device=DEVICE)


def _to_64(q):
    return q.double() if q.dtype == torch.int8 else _e4m3_grid()[q.view(torch.uint8).long()]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        m, k, group = case["rows"], case["cols"], case["group"]
        w = torch.empty(m, k, dtype=torch.float64, device=DEVICE)
        w[:, 0::2] = (s["q"] % 16)[:, :-(-k // 2)].double()
        w[:, 1::2] = (s["q"] // 16)[:, :k // 2].double()
        for j in range(-(-k // group)):
            part = w[:, j * group:(j + 1) * group]
            part -= 8.0 if s["zero"] is None else s["zero"][:, j:j + 1].double()
            part *= s["scale"][:, j:j + 1].double()
        y = torch.mm(s["x"].double(), w.t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()
    lens, new = _lengths(case)
    if op == "rotary":
        out = []
        for x, weight in ((s["xq"], s["q_weight"]), (s["xk"], s["k_weight"])):
            x, row = x.double().clone(), 0
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(dim=2, keepdim=True) / case["dim"] + EPS) * weight.double()
            y = x.clone()
            half = case["rotated"] // 2
            step, far = (2, 1) if case["interleaved"] else (1, half)
            for n, m in zip(lens, new):
                at = torch.arange(n - m, n, dtype=torch.float64, device=DEVICE)
                for i in range(half):
                    turn = at * float(s["freq"][i].double())
                    c, d = torch.cos(turn)[:, None], torch.sin(turn)[:, None]
                    a, b = x[row:row + m, :, step * i], x[row:row + m, :, step * i + far]
                    y[row:row + m, :, step * i] = case["magnitude"] * (a * c - b * d)
                    y[row:row + m, :, step * i + far] = case["magnitude"] * (a * d + b * c)
                row += m
            out.append(y)
        return tuple(out)
    cache, page, row = s["cache"], case["page"], 0
    group, d = case["q_heads"] // case["heads"], case["dim"]
    o = torch.zeros(s["query"].shape, dtype=torch.float64, device=DEVICE)
    for b, (n, m) in enumerate(zip(lens, new)):
        pages = s["table"][b, :-(-n // page)].long()
        pos = torch.arange(n - m, n, device=DEVICE)[:, None]
        j = torch.arange(n, device=DEVICE)[None, :]
        hidden = j > pos
        if case["window"]:
            hidden |= (pos - j >= case["window"]) & (j >= case["sinks"])
        for h in range(case["heads"]):
            k = _to_64(cache["k"][pages, h]).view(-1, TOKENS, d) * cache["k_scale"][pages, h].double().view(-1, 1, 1)
            v = _to_64(cache["v"][pages, h]).view(-1, d, TOKENS) * cache["v_scale"][pages, h].double().view(-1, 1, 1)
            k, v = k.reshape(-1, d)[:n], v.transpose(1, 2).reshape(-1, d)[:n]
            for i in range(h * group, (h + 1) * group):
                a = torch.softmax((s["query"][row:row + m, i].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf), dim=1)
                o[row:row + m, i] = a @ v
        row += m
    return o
