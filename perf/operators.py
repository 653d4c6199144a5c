"""The 8-bit operators of a decode or prompt step, as they are measured: the
block-scaled e4m3 quantiser and matrix product, the append to a paged 8-bit
cache and the attention over it.

``run`` computes a case with the library's entry points where ``own`` is
true, else in plain torch operations in fp32.  ``exact`` computes it in 64
bits from the definitions.

Definitions.  A quantised block of 1 or 128 rows by 128 columns holds e4m3
values with one fp32 scale, max(amax / 448, 2^-126).  A cache block holds 16
tokens of one head in int8 or e4m3 with one fp32 scale each for K and V, a
power of two when the append chose it.  K is stored (pages, heads, page_size,
dim), V (pages, heads, page_size / 16, dim, 16).
"""

import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 128          # columns (and weight rows) that share a scale
TOKENS = 16          # tokens of a cache block
TINY = 2.0 ** -126   # the smallest scale
FLOAT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
STORE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
QMAX = {"int8": 127.0, "e4m3": 448.0}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token's key or value projection: 1024 rows of 4096, launch-bound
        dict(name="product 1 token k/v", op="product", tokens=1, rows=1024, cols=4096, out="f32", bias=False),
        # the gate projection of 16 sequences that each decode one token
        dict(name="product 16 tokens gate", op="product", tokens=16, rows=14336, cols=4096, out="bf16", bias=False),
        # the ragged end of a prompt through a projection with long rows
        dict(name="product 250 tokens long rows", op="product", tokens=250, rows=4096, cols=11008, out="f16", bias=True),
        # a prompt of 4096 tokens through the gate projection
        dict(name="product 4096 tokens gate", op="product", tokens=4096, rows=14336, cols=4096, out="bf16", bias=False),
        # 16 decoded tokens' hidden states on their way into a product, fp32 as the matrix-vector products give them
        dict(name="quantise 16 tokens", op="quantise", rows=16, cols=4096, dtype="f32", block_rows=1),
        # a prompt's hidden states in front of the down projection
        dict(name="quantise 4096 tokens", op="quantise", rows=4096, cols=14336, dtype="bf16", block_rows=1),
        # one new token for each of 64 running sequences, straight from fp32 projections
        dict(name="append 64 tokens", op="append", batch=64, longest=2000, new=1, heads=8, dim=128, page=64,
             format="int8", dtype="f32"),
        # prompts of very different lengths, some of them behind a cached prefix
        dict(name="append prompts", op="append", batch=5, longest=4096, new=3000, heads=8, dim=128, page=16,
             format="e4m3", dtype="bf16"),
        # four conversations under a sliding window with 4 first tokens that stay visible: latency counts
        dict(name="attend 4 windowed", op="attend", batch=4, longest=2000, new=1, q_heads=32, heads=8, dim=128, page=64,
             format="int8", dtype="f16", window=512, sinks=4),
        # one sequence with a very long context: the split over the tokens does the work
        dict(name="attend 1 long", op="attend", batch=1, longest=131071, new=1, q_heads=32, heads=8, dim=128, page=128,
             format="int8", dtype="bf16", window=0, sinks=0),
        # a full serving batch of unequal lengths
        dict(name="attend 64 ragged", op="attend", batch=64, longest=8192, new=1, q_heads=32, heads=8, dim=128, page=64,
             format="e4m3", dtype="bf16", window=0, sinks=0),
        # prompt chunks over cached prefixes
        dict(name="attend prompts", op="attend", batch=4, longest=4096, new=1024, q_heads=32, heads=8, dim=128, page=16,
             format="e4m3", dtype="bf16", window=0, sinks=0),
    ]


def _between(rng, low, high):
    """Whole number between low and high, spread over the logarithm."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def _aligned(rng, n):
    """n itself (odd as it may be), or the multiple of 16 or 128 above it, as most models have."""
    step = rng.choice((1, 16, 128))
    return -(-n // step) * step


def draw(rng):
    op = rng.choice(("product", "quantise", "append", "attend"))
    if op == "product":
        while True:
            c = dict(op=op, tokens=_between(rng, 1, 4096), rows=_aligned(rng, _between(rng, 64, 16384)),
                     cols=_aligned(rng, _between(rng, 64, 16384)), out=rng.choice(("f32", "f16", "bf16")),
                     bias=rng.random() < 0.5)
            if c["tokens"] * c["rows"] * c["cols"] <= 4096 * 14336 * 4096:
                return c
    if op == "quantise":
        while True:
            c = dict(op=op, rows=_between(rng, 1, 8192), cols=_aligned(rng, _between(rng, 16, 16384)),
                     dtype=rng.choice(("f32", "f16", "bf16")), block_rows=rng.choice((1, 1, 128)))
            if c["rows"] * c["cols"] * SIZE[c["dtype"]] <= 4096 * 14336 * 2:
                return c
    shape = dict(dim=rng.choice((64, 128, 128, 256)), page=rng.choice((16, 32, 64, 128)),
                 format=rng.choice(("int8", "e4m3")))
    if op == "append":
        while True:
            longest = _between(rng, 16, 8192)
            c = dict(op=op, batch=_between(rng, 1, 128), longest=longest, new=rng.choice((1, _between(rng, 2, longest))),
                     heads=rng.choice((1, 2, 4, 8, 16, 32)), **shape, dtype=rng.choice(("f32", "f16", "bf16")))
            if (c["batch"] * c["new"] * c["heads"] * c["dim"] <= 5 * 3000 * 8 * 128
                    and c["batch"] * c["longest"] * c["heads"] * c["dim"] <= 64 * 8192 * 8 * 128):
                return c
    while True:
        longest = _between(rng, 16, 131072)
        heads = rng.choice((1, 2, 4, 8, 16))
        c = dict(op=op, batch=_between(rng, 1, 64), longest=longest, new=rng.choice((1, 1, _between(rng, 2, min(longest, 1024)))),
                 q_heads=heads * rng.choice((1, 2, 4, 5, 8)), heads=heads, **shape, dtype=rng.choice(("f16", "bf16")),
                 window=rng.choice((0, 0, _between(rng, 16, longest))), sinks=rng.choice((0, 1, 4, 70)))
        if (c["batch"] * c["longest"] * c["heads"] * c["dim"] <= 64 * 8192 * 8 * 128
                and c["batch"] * c["new"] * c["longest"] * c["q_heads"] * c["dim"] <= 4 * 1024 * 4096 * 32 * 128):
            return c


# ---------------------------------------------------------------------------
# a batch's lengths, by the case alone
# ---------------------------------------------------------------------------

def _lengths(case):
    """(length after the call, new tokens) of each sequence."""
    r = random.Random(case["batch"] * 1000003 + case["longest"] * 31 + case["new"])
    lens, new = [], []
    for b in range(case["batch"]):
        n = case["new"] if b == 0 or case["new"] == 1 else r.randint(1, case["new"])
        lens.append(case["longest"] if b == 0 else r.randint(n, case["longest"]))
        new.append(n)
    return lens, new


def _visible(case):
    """(query-token pairs, tokens that any query sees) over the whole batch."""
    pairs = tokens = 0
    for n, new in zip(*_lengths(case)):
        first = n - new
        if not case["window"]:
            tokens += n
            pairs += new * first + new * (new + 1) // 2
            continue
        w, s = case["window"], case["sinks"]
        low = max(0, first - w + 1)
        tokens += n - low + min(low, s)
        for p in range(first, n):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(low, s)
    return pairs, tokens


def work(case):
    op = case["op"]
    if op == "product":
        t, m, k = case["tokens"], case["rows"], case["cols"]
        nb = -(-k // BLOCK)
        return {"bytes": m * k + t * k + 4 * nb * (t + -(-m // BLOCK)) + t * m * SIZE[case["out"]] + (4 * m if case["bias"] else 0),
                "flops": 2 * t * m * k}
    if op == "quantise":
        n = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // BLOCK)
        return {"bytes": n * (SIZE[case["dtype"]] + 1) + 4 * scales, "flops": 3 * n}
    lens, new = _lengths(case)
    h, d = case["heads"], case["dim"]
    if op == "append":
        # each new value read and held in 8 bits; of a block that has tokens already, its scales
        blocks = sum(-(-n // TOKENS) - (n - m) // TOKENS for n, m in zip(lens, new))
        stays = sum(1 for n, m in zip(lens, new) if (n - m) % TOKENS)
        values = 2 * sum(new) * h * d
        return {"bytes": values * (SIZE[case["dtype"]] + 1) + 8 * h * (blocks + stays), "flops": 3 * values}
    pairs, tokens = _visible(case)
    q = sum(new) * case["q_heads"] * d * SIZE[case["dtype"]]
    return {"bytes": 2 * tokens * h * d + 8 * h * -(-tokens // TOKENS) + 2 * q, "flops": 4 * pairs * case["q_heads"] * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _blocks(x, rows):
    """x in fp32 as (row blocks, rows, column blocks, 128), zeros behind its ends."""
    r, k = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -k % BLOCK, 0, -r % rows))
    return x.view(-1, rows, x.shape[1] // BLOCK, BLOCK)


def _quantise(x, rows):
    """The quantiser in plain operations: (e4m3 values, fp32 scales)."""
    r, k = x.shape
    b = _blocks(x, rows)
    scale = torch.clamp(b.abs().amax(dim=(1, 3)) / torch.full((), 448.0, device=x.device), min=TINY)
    q = b * (torch.ones((), device=x.device) / scale)[:, None, :, None]
    q = q.to(torch.float8_e4m3fn).view(torch.uint8).view(b.shape[0] * rows, -1)[:r, :k]
    return q.contiguous().view(torch.float8_e4m3fn), scale


def _activations(g, rows, cols):
    """Hidden states: normal, with a few channels far larger than the others, as trained models have them."""
    x = torch.randn(rows, cols, device=DEVICE, generator=g)
    loud = torch.rand(cols, device=DEVICE, generator=g) < 0.005
    return x * torch.where(loud, 20.0, 1.0)


def _tables(case, g):
    """Shuffled pages (page 0 is nobody's), -1 in the unused entries, the lengths and the first row of each sequence."""
    lens, new = _lengths(case)
    page = case["page"]
    need = [-(-n // page) for n in lens]
    order = torch.randperm(sum(need), device=DEVICE, generator=g).to(torch.int32) + 1
    table = torch.full((case["batch"], max(need)), -1, dtype=torch.int32, device=DEVICE)
    held = torch.arange(max(need), device=DEVICE)[None, :] < torch.tensor(need, device=DEVICE)[:, None]
    table[held] = order
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    return (sum(need) + 1, table, torch.tensor(lens, dtype=torch.int32, device=DEVICE),
            None if case["new"] == 1 else torch.tensor(starts, dtype=torch.int32, device=DEVICE))


def _fill(case, g, pages):
    """A cache as many appends leave it: values over the whole 8-bit range, scales that are powers of two."""
    h, d, page, per = case["heads"], case["dim"], case["page"], case["page"] // TOKENS
    out = {}
    for name, shape in (("k", (pages, h, page, d)), ("v", (pages, h, per, d, TOKENS))):
        x = torch.empty(shape, device=DEVICE).normal_(generator=g)
        x = torch.clamp(x * 38.0, -127.0, 127.0).round_().to(torch.int8) if case["format"] == "int8" else \
            torch.clamp(x * 130.0, -448.0, 448.0).to(torch.float8_e4m3fn)
        out[name] = x
        up = torch.randint(0, 3, (pages, h, per), device=DEVICE, generator=g).float()
        out[name + "_scale"] = torch.exp2(up - 6.0 if case["format"] == "int8" else up - 8.0)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed * 7919 + 11)
    op = case["op"]
    s = {"case": case}
    if op == "product":
        w = torch.randn(case["rows"], case["cols"], device=DEVICE, generator=g) * 0.02
        s["w"], s["w_scale"] = _quantise(w, BLOCK)
        s["x"], s["x_scale"] = _quantise(_activations(g, case["tokens"], case["cols"]), 1)
        s["bias"] = torch.randn(case["rows"], device=DEVICE, generator=g) if case["bias"] else None
    elif op == "quantise":
        s["x"] = _activations(g, case["rows"], case["cols"]).to(FLOAT[case["dtype"]])
    else:
        pages, s["table"], s["lens"], s["starts"] = _tables(case, g)
        s["cache"] = _fill(case, g, pages)
        total = sum(_lengths(case)[1])
        if op == "append":
            for name in ("k", "v"):
                s[name] = _activations(g, total, case["heads"] * case["dim"]).to(FLOAT[case["dtype"]]) \
                    .view(total, case["heads"], case["dim"])
        else:
            s["q"] = torch.randn(total, case["q_heads"], case["dim"], device=DEVICE, generator=g).to(FLOAT[case["dtype"]])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(op, case, state)
    if op == "product":
        y = _values(state["x"], state["x_scale"], 1) @ _values(state["w"], state["w_scale"], BLOCK).t()
        if state["bias"] is not None:
            y += state["bias"]
        return y.to(FLOAT[case["out"]])
    if op == "quantise":
        return _quantise(state["x"], case["block_rows"])
    if op == "append":
        return _append(case, state)
    return _attend(case, state)


def _run_own(op, case, state):
    import memory_bound_gemv_f32_amd as lg
    if op == "product":
        return lg.gemv_fp8(state["w"], state["w_scale"], state["x"], state["x_scale"], state["bias"],
                           out_dtype=FLOAT[case["out"]])
    if op == "quantise":
        return lg.gemv_fp8_quantise(state["x"], block_rows=case["block_rows"])
    c = state["cache"]
    cache = lg.KVCache(c["k"], c["v"], c["k_scale"], c["v_scale"])
    if op == "append":
        lg.gemv_kv_append(cache, state["k"], state["v"], state["table"], state["lens"], state["starts"])
        return {name: c[name] for name in ("k", "v", "k_scale", "v_scale")}
    return lg.gemv_kv_attend(state["q"], cache, state["table"], state["lens"], state["starts"],
                             window=case["window"], sinks=case["sinks"])


def _values(q, scale, rows):
    """The fp32 values that a quantised matrix stands for."""
    r, k = q.shape
    b = _blocks(q, rows) * scale[:, None, :, None]
    return b.view(b.shape[0] * rows, -1)[:r, :k].contiguous()


def _sequences(state, total):
    """Of each row its sequence and its position, and of each sequence its first row and new tokens."""
    lens = state["lens"].long()
    starts = torch.arange(len(lens) + 1, device=DEVICE) if state["starts"] is None else state["starts"].long()
    new = starts[1:] - starts[:-1]
    row = torch.arange(total, device=DEVICE)
    seq = torch.searchsorted(starts, row, right=True) - 1
    return lens, starts, new, seq, lens[seq] - new[seq] + row - starts[seq]


def _round(x, form):
    """Values over their scale, held in 8 bits."""
    x = torch.clamp(x, -QMAX[form], QMAX[form])
    return x.round().to(torch.int8) if form == "int8" else x.to(torch.float8_e4m3fn)


def _append(case, state):
    form, per = case["format"], case["page"] // TOKENS
    cache, table = state["cache"], state["table"].long()
    total, h, d = state["k"].shape
    lens, starts, new, _, _ = _sequences(state, total)
    # room for every block that a sequence can touch; the spare places write
    # back what block 0 of the unused page 0 holds
    room = starts // TOKENS + 2 * torch.arange(len(starts), device=DEVICE)
    item = torch.arange(total // TOKENS + 2 * len(lens), device=DEVICE)
    seq = torch.clamp(torch.searchsorted(room, item, right=True) - 1, max=len(lens) - 1)
    first = lens[seq] - new[seq]
    block = first // TOKENS + item - room[seq]
    used = block * TOKENS < lens[seq]
    page = torch.where(used, table[seq, torch.clamp(block // per, max=table.shape[1] - 1)], 0)
    sub = torch.where(used, block % per, 0)
    pos = block[:, None] * TOKENS + torch.arange(TOKENS, device=DEVICE)
    fresh = used[:, None] & (pos >= first[:, None]) & (pos < lens[seq][:, None])      # (items, 16)
    stays = used[:, None] & (pos < first[:, None])
    row = torch.where(fresh, starts[seq][:, None] + pos - first[:, None], 0)
    for name in ("k", "v"):
        held = cache[name].view(torch.uint8)
        if name == "k":
            held = held.view(-1, h, per, TOKENS, d)[page, :, sub]                       # (items, h, 16, d)
        else:
            held = held[page, :, sub].transpose(2, 3)
        held = held.contiguous().view(STORE[form])
        x = torch.where(fresh[:, :, None, None], state[name].float()[row], 0.0).transpose(1, 2)
        mantissa, power = torch.frexp(x.abs().amax(dim=(2, 3)))
        power = power - (7 if form == "int8" else 9) + (mantissa > (127.0 / 128.0 if form == "int8" else 0.875))
        scale = torch.exp2(torch.clamp(torch.where(mantissa > 0, power, -126), min=-126).double()).float()
        old = cache[name + "_scale"][page, :, sub]
        scale = torch.where(stays[:, :1], torch.maximum(scale, old), scale)
        again = _round(held.float() * (old / scale)[:, :, None, None], form).view(torch.uint8)
        put = _round(x * (torch.ones((), device=DEVICE) / scale)[:, :, None, None], form).view(torch.uint8)
        put = torch.where(fresh[:, None, :, None], put, torch.where(stays[:, None, :, None], again, held.view(torch.uint8)))
        if name == "k":
            cache[name].view(torch.uint8).view(-1, h, per, TOKENS, d)[page, :, sub] = put
        else:
            cache[name].view(torch.uint8)[page, :, sub] = put.transpose(2, 3)
        cache[name + "_scale"][page, :, sub] = torch.where(used[:, None], scale, old)
    return {name: cache[name] for name in ("k", "v", "k_scale", "v_scale")}


def _attend(case, state):
    cache, q = state["cache"], state["q"]
    h, d, group = case["heads"], case["dim"], case["q_heads"] // case["heads"]
    batch, span = state["table"].shape[0], state["table"].shape[1] * case["page"]
    total = q.shape[0]
    lens, starts, new, seq, pos = _sequences(state, total)
    table = torch.clamp(state["table"].long(), min=0)
    # every sequence's tokens as (batch, heads, span, dim)
    k = cache["k"][table].float().view(batch, -1, h, case["page"] // TOKENS, TOKENS, d) \
        * cache["k_scale"][table][..., None, None]
    k = k.transpose(1, 2).reshape(batch, h, span, d)
    v = cache["v"][table].float() * cache["v_scale"][table][..., None, None]
    v = v.transpose(1, 2).transpose(4, 5).reshape(batch, h, span, d)
    # the queries padded to the longest sequence's
    most = case["new"]
    at = row_in = torch.arange(total, device=DEVICE) - starts[seq]
    rows = torch.zeros(batch, most, h, group, d, device=DEVICE)
    rows[seq, at] = q.float().view(total, h, group, d)
    where = torch.full((batch, most), -1, dtype=torch.long, device=DEVICE)
    where[seq, row_in] = pos
    rows = rows.permute(0, 2, 1, 3, 4).reshape(batch, h, most * group, d)
    s = (rows * (1.0 / math.sqrt(d))) @ k.transpose(2, 3).contiguous()
    j = torch.arange(span, device=DEVICE)
    sees = j <= where[:, :, None]
    if case["window"]:
        sees &= (where[:, :, None] - j < case["window"]) | (j < case["sinks"])
    s = s.view(batch, h, most, group, span).masked_fill_(~sees[:, None, :, None], -math.inf)
    p = torch.exp(s - torch.clamp(s.amax(dim=-1, keepdim=True), min=-1e30))
    o = (p.view(batch, h, most * group, span) @ v).view(batch, h, most, group, d)
    o = o / torch.clamp(p.sum(dim=-1, keepdim=True), min=1e-30)
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


def _rounded_64(x, form):
    """64-bit values rounded to the nearest that the 8 bits hold, ties to even."""
    if form == "int8":
        return torch.clamp(torch.round(x), -127, 127)
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(x.abs(), min=2.0 ** -30))), min=-6) - 3)
    return torch.clamp(torch.round(x / step) * step, -448, 448)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        def full(q, scale, rows):
            r, k = q.shape
            by = scale.double().repeat_interleave(rows, 0)[:r].repeat_interleave(BLOCK, 1)[:, :k]
            return _to_64(q) * by
        w, x = full(s["w"], s["w_scale"], BLOCK), full(s["x"], s["x_scale"], 1)
        y = torch.mm(x, w.t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "quantise":
        x, r = s["x"].double(), case["block_rows"]
        scales = torch.empty(-(-x.shape[0] // r), -(-x.shape[1] // BLOCK), dtype=torch.float64, device=DEVICE)
        q = torch.empty_like(x)
        for j in range(scales.shape[1]):
            part = x[:, j * BLOCK:(j + 1) * BLOCK]
            top = part.abs().amax(dim=1)
            if r > 1:
                top = torch.stack([piece.amax() for piece in top.split(r)])
            scales[:, j] = torch.clamp(top / 448, min=TINY)
            q[:, j * BLOCK:(j + 1) * BLOCK] = _rounded_64(part / scales[:, j].repeat_interleave(r)[:len(x), None], "e4m3")
        return q, scales
    lens, new = _lengths(case)
    cache, table, page, per = s["cache"], s["table"].cpu(), case["page"], case["page"] // TOKENS
    row = 0
    if op == "append":
        out = {name: _to_64(cache[name]) for name in ("k", "v")}
        out.update({name: cache[name].double() for name in ("k_scale", "v_scale")})
        limit = QMAX[case["format"]]
        for b, (n, m) in enumerate(zip(lens, new)):
            p = n - m
            while p < n:
                at, off = int(table[b, p // page]), p % TOKENS
                take, sub = min(TOKENS - off, n - p), p % page // TOKENS
                for name in ("k", "v"):
                    x = s[name][row:row + take].double().transpose(0, 1)             # (heads, take, dim)
                    need = torch.exp2(torch.ceil(torch.log2(torch.clamp(x.abs().amax(dim=(1, 2)) / limit, min=TINY))))
                    scale = out[name + "_scale"][at, :, sub]
                    now = torch.maximum(scale, need) if off else need
                    block = out[name][at, :, sub * TOKENS:(sub + 1) * TOKENS] if name == "k" else \
                        out[name][at, :, sub].transpose(1, 2)
                    block[:, :off] = _rounded_64(block[:, :off] * (scale / now)[:, None, None], case["format"])
                    block[:, off:off + take] = _rounded_64(x / now[:, None, None], case["format"])
                    scale.copy_(now)
                p, row = p + take, row + take
        return {name: out[name] if name.endswith("scale") or case["format"] == "e4m3" else out[name].to(torch.int8)
                for name in ("k", "v", "k_scale", "v_scale")}
    group, d = case["q_heads"] // case["heads"], case["dim"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
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
                a = torch.softmax((s["q"][row:row + m, i].double() @ k.t() / math.sqrt(d)).masked_fill(hidden, -math.inf), dim=1)
                o[row:row + m, i] = a @ v
        row += m
    return o
