"""Cases of the operators around the attention path: batch tables, FP8 block quantisation and the
FP8 matrix product with a scale for each block of 128.

`run` computes a case in its plain form (elementary torch operations in 32 bits), or, with `own`
set, through the library's calls.
"""
import math

import torch

own = False

BLOCK = 128            # elements that share an activation scale; a weight scale covers 128 x 128
FP8_MAX = 448.0        # the largest E4M3 value
PAGE = 64              # cache entries per page
WINDOW = 128           # sliding window in tokens
# the cache groups of a layer stack: name, tokens per entry, window (0: every entry is kept)
GROUPS = (("swa", 1, WINDOW), ("c4", 4, 0), ("c128", 128, 0))
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def listed():
    return [
        # the quantiser between the two output projections of a decode step, one row per sequence
        {"name": "quant decode 32 rows", "op": "quant", "rows": 32, "cols": 8192, "type": "bf16", "block_rows": 1},
        # the same in a prefill chunk of 8192 tokens
        {"name": "quant prefill 8192 rows", "op": "quant", "rows": 8192, "cols": 8192, "type": "bf16", "block_rows": 1},
        # a weight matrix quantised at load time, ragged in both directions
        {"name": "quant weights 4000x8176", "op": "quant", "rows": 4000, "cols": 8176, "type": "fp32", "block_rows": 128},
        # the grouped output projection (64 heads of 512 in 8 groups) of one sequence's decode step,
        # its result quantised for the projection that follows: latency and reading the weights
        {"name": "product decode 1 token", "op": "matmul", "tokens": 1, "groups": 8, "n": 1024, "k": 4096, "type": "e4m3"},
        # the same at the headline decode batch
        {"name": "product decode 32 tokens", "op": "matmul", "tokens": 32, "groups": 8, "n": 1024, "k": 4096, "type": "e4m3"},
        # the projection that follows it, batch 64
        {"name": "product decode 64 tokens", "op": "matmul", "tokens": 64, "groups": 1, "n": 4096, "k": 8192, "type": "bf16"},
        # a short ragged chunk with odd sizes everywhere: last blocks of n and k partly filled
        {"name": "product ragged 333 tokens", "op": "matmul", "tokens": 333, "groups": 3, "n": 1000, "k": 1392, "type": "fp32"},
        # prefill chunks: the grouped projection and the one that follows, at the tensor rate
        {"name": "product prefill 4096 grouped", "op": "matmul", "tokens": 4096, "groups": 8, "n": 1024, "k": 4096, "type": "bf16"},
        {"name": "product prefill 8192", "op": "matmul", "tokens": 8192, "groups": 1, "n": 4096, "k": 8192, "type": "bf16"},
        # one decode step of the headline batch: tables and slot maps of all three cache groups
        {"name": "tables decode 32 seqs", "op": "tables", "seqs": 32, "max_ctx": 32768, "max_tokens": 32, "mixed": False},
        # continuous batching: decodes, prefill chunks, idle and finished sequences side by side
        {"name": "tables mixed 200 seqs", "op": "tables", "seqs": 200, "max_ctx": 65536, "max_tokens": 8192, "mixed": True},
        # a large service: thousands of sequences with contexts up to 128K
        {"name": "tables mixed 2048 seqs", "op": "tables", "seqs": 2048, "max_ctx": 131072, "max_tokens": 32768, "mixed": True},
    ]


def _spread(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("quant", "matmul", "matmul", "matmul", "tables"))
    if op == "quant":
        block_rows = rng.choice((1, 1, BLOCK))
        rows, cols = _spread(rng, 1, 8192), _spread(rng, 64, 8192)
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(("bf16", "fp16", "fp32")), "block_rows": block_rows}
    if op == "matmul":
        while True:
            case = {"op": op, "tokens": _spread(rng, 1, 8192), "groups": rng.choice((1, 1, 2, 3, 4, 8, 16)), "n": _spread(rng, 64, 8192),
                    "k": 16 * _spread(rng, 8, 512), "type": rng.choice(("bf16", "fp16", "fp32", "e4m3"))}
            if case["tokens"] * case["groups"] * case["n"] * case["k"] <= 8192 * 4096 * 8192 and case["groups"] * case["n"] * case["k"] <= 1 << 28:
                return case
    mixed = rng.random() < 0.7
    seqs = _spread(rng, 1, 2048)
    tokens = seqs if not mixed else max(seqs, _spread(rng, 16, 32768))
    return {"op": op, "seqs": seqs, "max_ctx": _spread(rng, 512, 131072), "max_tokens": tokens, "mixed": mixed}


# ---- inputs ---------------------------------------------------------------------------------------


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(shape, g):
    """Rows as a projection leaves them: normal values, each row of its own size, a few large channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(torch.randn(shape[:-1], generator=g, device="cuda"))[..., None]
    big = torch.rand(shape[-1], generator=g, device="cuda") < 0.01
    return x * torch.where(big, 16.0, 1.0)


def _pages(tokens, ratio):
    """Pages that hold the entries of so many tokens."""
    return (tokens // ratio + (PAGE - 1)) // PAGE


def _first_live(tokens, window):
    """The first page that a query at position `tokens` still reads."""
    return torch.clamp(tokens - (window - 1), min=0) // PAGE if window else torch.zeros_like(tokens)


def _stride(case, ratio):
    return _pages(case["max_ctx"] + case["max_tokens"], ratio) or 1


def _tables_state(case, g):
    s, top, most = case["seqs"], case["max_ctx"], case["max_tokens"]
    u = torch.rand(s, generator=g, device="cuda", dtype=torch.float64)
    v = torch.rand(s, generator=g, device="cuda", dtype=torch.float64)
    kind = torch.rand(s, generator=g, device="cuda", dtype=torch.float64)
    computed = ((0.5 + 0.5 * u) * (top - 1)).long()
    new = torch.ones_like(computed)
    if case["mixed"]:
        prompt = kind < 0.25          # a chunk of a prompt, half of them its first
        chunk = torch.exp(v * math.log(max(2.0, most / 4))).long()
        computed = torch.where(prompt, torch.where(kind < 0.125, 0, (u * top).long()), computed)
        new = torch.where(prompt, chunk, new)
        fits = torch.cumsum(new, 0) <= most
        new = torch.where(fits, new, 0)
        new = torch.where((kind > 0.85) & (kind < 0.95), 0, new)      # idle
        new = torch.where(kind >= 0.95, -1, new)                      # finished: its pages go back
    state = {"case": case, "computed": computed.int(), "new": new.int(), "groups": []}
    for name, ratio, window in GROUPS:
        stride = _stride(case, ratio)
        lo, hi = _first_live(computed, window), _pages(computed, ratio)
        held = hi - lo
        used = int(held.sum())
        # a pool that holds every sequence at its longest, and the step's new pages
        held_most = (WINDOW // PAGE + 1) if window else _pages(top, ratio)
        pages = s * (held_most + 1) + _pages(most, ratio) + PAGE
        order = torch.randperm(pages, generator=g, device="cuda").int()
        col = torch.arange(stride, device="cuda")[None]
        at = (torch.cumsum(held, 0) - held)[:, None] + col - lo[:, None]
        live = (col >= lo[:, None]) & (col < hi[:, None])
        owned = torch.where(live, order[at.clamp(0, pages - 1)], -1).int().contiguous()
        head = int(torch.randint(0, 4 * pages, (1,), generator=g, device="cuda"))
        ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        ring[(head + torch.arange(pages - used, device="cuda")) % pages] = order[used:]
        pool = torch.tensor([head, head + pages - used], dtype=torch.int64, device="cuda")
        state["groups"].append({"ratio": ratio, "window": window, "owned": owned, "ring": ring, "pool": pool, "num_pages": pages})
    return state


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "quant":
        x = _activations((case["rows"], case["cols"]), g).to(TYPES[case["type"]])
        state = {"case": case, "x": x}
    elif case["op"] == "matmul":
        t, gr, n, k = case["tokens"], case["groups"], case["n"], case["k"]
        x, xs = _quantise(_activations((t * gr, k), g), 1)
        w, ws = zip(*[_quantise(torch.randn((n, k), generator=g, device="cuda") / math.sqrt(k), BLOCK) for _ in range(gr)])
        state = {"case": case, "x": x.view(t, gr, k), "xs": xs.view(t, gr, -1), "w": torch.stack(w), "ws": torch.stack(ws)}
    else:
        state = _tables_state(case, g)
    return _with_buffers(state) if own else state


def _with_buffers(state):
    """The output buffers and handles that a program keeps next to its inputs."""
    from deepseek_v4_compressed_gb300 import binding as B
    case, dev = state["case"], "cuda"
    if case["op"] == "quant":
        blocks = -(-case["cols"] // BLOCK)
        state["codes"] = torch.empty((case["rows"], case["cols"]), dtype=torch.float8_e4m3fn, device=dev)
        state["scales"] = torch.empty((-(-case["rows"] // case["block_rows"]), blocks), device=dev)
    elif case["op"] == "matmul":
        t, gr, n = case["tokens"], case["groups"], case["n"]
        state["weights"] = B.Fp8Weights(state["w"], state["ws"])
        state["out"] = torch.empty((t, gr, n), dtype=TYPES[case["type"]], device=dev)
        state["out_scales"] = torch.empty((t, gr, -(-n // BLOCK)), device=dev) if case["type"] == "e4m3" else None
    else:
        s, most = case["seqs"], case["max_tokens"]
        i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=dev)  # noqa: E731
        for gr in state["groups"]:
            gr["table"] = i32(*gr["owned"].shape)
            gr["pool_out"] = torch.empty(2, dtype=torch.int64, device=dev)
            gr["slots"] = torch.empty(most, dtype=torch.int64, device=dev)
        state["out"] = {"offsets": i32(s + 1), "ctx_len": i32(s), "positions": i32(most), "seqs": i32(most), "row_ctx": i32(most)}
        state["tables"] = B.BatchTables(
            groups=[B.TableGroup(ratio=gr["ratio"], window=gr["window"], num_pages=gr["num_pages"], owned=gr["owned"], table=gr["table"], ring=gr["ring"],
                                 pool_in=gr["pool"], pool_out=gr["pool_out"], slots=gr["slots"]) for gr in state["groups"]],
            **state["out"])
    return state


# ---- one pass -------------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "quant":
        return _quantise(state["x"], state["case"]["block_rows"])
    if op == "matmul":
        return _plain_product(state)
    return _plain_tables(state)


def _run_own(state, op):
    from deepseek_v4_compressed_gb300 import binding as B
    if op == "quant":
        B.fp8_block_quant(state["x"], state["codes"], state["scales"], block_rows=state["case"]["block_rows"])
        return state["codes"], state["scales"]
    if op == "matmul":
        B.fp8_block_matmul(state["x"], state["xs"], state["weights"], state["out"], state["out_scales"])
        return state["out"] if state["out_scales"] is None else (state["out"], state["out_scales"])
    state["tables"].build(state["computed"], state["new"])
    keys = ("owned", "table", "ring", "pool_out", "slots")
    return dict(state["out"], groups=[[g[k] for k in keys] for g in state["groups"]])


def _quantise(x, block_rows):
    """E4M3 codes and one fp32 scale, amax / 448, for each block of block_rows x 128; a scale of 0 becomes 1."""
    rows, cols = x.shape
    up = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK, 0, -rows % block_rows))
    tiles = up.view(up.shape[0] // block_rows, block_rows, up.shape[1] // BLOCK, BLOCK)
    scale = tiles.abs().amax(dim=(1, 3)) / torch.full((), FP8_MAX, device=x.device)   # by a tensor: a true division
    scale = torch.where(scale > 0, scale, 1.0)
    codes = (tiles / scale[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return codes.view(up.shape)[:rows, :cols].contiguous(), scale


def _plain_product(state):
    case = state["case"]
    t, gr, n, k = case["tokens"], case["groups"], case["n"], case["k"]
    x = state["x"].float() * state["xs"].repeat_interleave(BLOCK, -1)[..., :k]
    w = state["w"].float() * state["ws"].repeat_interleave(BLOCK, -1)[..., :k].repeat_interleave(BLOCK, 1)[:, :n]
    y = torch.matmul(x.transpose(0, 1), w.transpose(1, 2)).transpose(0, 1)
    if case["type"] != "e4m3":
        return y.to(TYPES[case["type"]])
    codes, scale = _quantise(y.reshape(t * gr, n), 1)
    return codes.view(t, gr, n), scale.view(t, gr, -1)


def _plain_tables(state):
    case = state["case"]
    computed, asked = state["computed"].long(), state["new"].long()
    new, done = asked.clamp(min=0), asked < 0
    ends = torch.cumsum(new, 0)
    offsets = torch.cat((torch.zeros_like(ends[:1]), ends))
    at = torch.arange(case["max_tokens"], device=ends.device)
    seq = torch.searchsorted(ends, at, right=True).clamp(max=case["seqs"] - 1)
    real = at < ends[-1]
    pos = computed[seq] + at - offsets[seq]
    out = {"offsets": offsets.int(), "ctx_len": torch.where(done, 0, computed + new).int(), "positions": torch.where(real, pos, -1).int(),
           "seqs": torch.where(real, seq, -1).int(), "row_ctx": torch.where(real, pos + 1, 0).int()}
    out["groups"] = [_plain_group(g, computed, new, done, pos, seq, real) for g in state["groups"]]
    return out


def _plain_group(g, computed, new, done, pos, seq, real):
    ratio, window, ring = g["ratio"], g["window"], g["ring"]
    cap, head, tail = ring.numel(), g["pool"][0], g["pool"][1]
    lo, before, after = _first_live(computed, window), _pages(computed, ratio), _pages(computed + new, ratio)
    gone = torch.where(done, before, _first_live(computed + new, window))       # pages lo .. gone go back
    taken, freed = after - before, gone - lo
    first_taken, first_freed = torch.cumsum(taken, 0) - taken, torch.cumsum(freed, 0) - freed
    col = torch.arange(g["owned"].shape[1], device=ring.device)[None]
    fresh = (col >= before[:, None]) & (col < after[:, None])
    owned = torch.where(fresh, ring[(head + first_taken[:, None] + col - before[:, None]) % cap], g["owned"])
    live = (col >= lo[:, None]) & (col < after[:, None]) & ~done[:, None]
    table = torch.where(live, owned, -1)
    back = (col >= lo[:, None]) & (col < gone[:, None])
    to = torch.where(back, (tail + first_freed[:, None] + col - lo[:, None]) % cap, cap)
    ring_out = torch.cat((ring, ring[:1])).scatter(0, to.flatten(), owned.flatten())[:cap]
    pool_out = torch.stack((head + taken.sum(), tail + freed.sum()))
    entry = pos // ratio
    page = owned[seq, (entry // PAGE).clamp(0, owned.shape[1] - 1)].long()
    slots = torch.where(real & ((pos + 1) % ratio == 0), page * PAGE + entry % PAGE, -1)
    return [owned, table, ring_out, pool_out, slots]


# ---- what a pass cannot do without ------------------------------------------------------------------


def work(case):
    if case["op"] == "quant":
        cells = case["rows"] * case["cols"]
        scales = -(-case["rows"] // case["block_rows"]) * -(-case["cols"] // BLOCK)
        return {"bytes": cells * (SIZE[case["type"]] + 1) + 4 * scales, "flops": 3 * cells}
    if case["op"] == "matmul":
        t, gr, n, k = case["tokens"], case["groups"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        out = t * gr * (n * SIZE[case["type"]] + (4 * nb if case["type"] == "e4m3" else 0))
        return {"bytes": gr * (t * (k + 4 * kb) + n * k + 4 * nb * kb) + out, "flops": 2 * t * gr * n * k}
    # lengths in, tables out, per-token arrays out, and the live old entries read (three quarters of the
    # longest context on average)
    s, most = case["seqs"], case["max_tokens"]
    held = sum((WINDOW // PAGE + 1) if w else int(_pages(0.75 * case["max_ctx"], r)) for _, r, w in GROUPS)
    tables = sum(_stride(case, r) for _, r, _ in GROUPS)
    return {"bytes": s * (8 + 8 + 4 * held + 4 * tables) + most * (12 + 8 * len(GROUPS)), "flops": 0}


# ---- the definition in 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "tables":
        return None                                   # whole numbers only: they have to be equal
    state = prepare(case, seed)
    if case["op"] == "quant":
        return _exact_codes(state["x"].double(), case["block_rows"])
    t, gr, n, k = case["tokens"], case["groups"], case["n"], case["k"]
    y = torch.zeros((t, gr, n), dtype=torch.float64, device="cuda")
    row_block = torch.arange(n, device="cuda") // BLOCK
    for g in range(gr):
        for b in range(-(-k // BLOCK)):
            cut = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
            part = state["x"][:, g, cut].double() @ state["w"][g, :, cut].double().T
            y[:, g] += part * state["xs"][:, g, b].double()[:, None] * state["ws"][g, row_block, b].double()[None]
    if case["type"] != "e4m3":
        return y
    codes, scales = _exact_codes(y.reshape(t * gr, n), 1)
    return codes.view(t, gr, n), scales.view(t, gr, -1)


def _exact_codes(x, block_rows):
    """Codes as values and their scales, block by block of columns."""
    rows, cols = x.shape
    codes, scales = torch.empty_like(x), []
    group = torch.arange(rows, device=x.device) // block_rows
    for c in range(0, cols, BLOCK):
        part = x[:, c:c + BLOCK]
        top = torch.zeros(int(group[-1]) + 1, dtype=x.dtype, device=x.device).scatter_reduce(0, group, part.abs().amax(1), "amax")
        scale = torch.where(top > 0, top / FP8_MAX, 1.0)
        scales.append(scale)
        value = part / scale[group][:, None]
        # E4M3: 3 bits behind the leading one, the smallest exponent -6; half steps go to the even code
        step = torch.exp2(torch.floor(torch.log2(value.abs().clamp(min=2.0 ** -6))) - 3)
        codes[:, c:c + BLOCK] = (torch.round(value / step) * step).clamp(-FP8_MAX, FP8_MAX)
    return codes, torch.stack(scales, 1)
