"""Cases of a prompt chunk's path: 8-bit quantisation and products, rotary positions with several axes, and attention of the chunk over a paged cache.

Hidden rows are normed or quantised to e4m3 with a power-of-two scale for each 128 values, multiplied with 8-bit weights that
have one scale for each 128 x 128 block, rotated by positions on one or more axes, written to the cache, and attend to it.

A case's "op" is one of
  quant    bf16 values -> e4m3 codes and power-of-two scales, the smallest at or above amax / 448 (1 for zeros), of 128
           values of a row ("square": false: activations) or of 128 x 128 values ("square": true: weights)
  product  out[n][outs] = (codes * scales)[n][ins] times the transposed (codes * scales)[outs][ins] of a weight
  rotate   a chunk's queries rotated into their places beside the latent part, and its rows written to the cache: rotary
           pairs that turn by the position on one of `axes` axes each (time, height, width)
  chunk    absorbed attention of ragged requests' newest tokens over 4-bit cache rows behind a page table: causal over
           every cached token, or over a list of k tokens for each query token
"""
import math
import random

import torch

own = False   # set by the caller: true runs the framework's operators

LATENT, ROPE, ROW = 512, 64, 576
ROW_BYTES = {"bf16": 1152, "compact": 656, "q4": 400}
EPS = 1e-6
SM_SCALE = 1.0 / math.sqrt(ROW)
PAGE = 64


def listed():
    return [
        # attention outputs of a prompt's chunk, on their way to the output projection
        {"name": "quant_rows_prompt", "op": "quant", "n": 16384, "dim": 4096, "square": False},
        # a weight as it is loaded
        {"name": "quant_weight", "op": "quant", "n": 1600, "dim": 4096, "square": True},
        # the projection to a query latent and a cache row, for a decode step of four requests
        {"name": "product_few", "op": "product", "n": 4, "ins": 4096, "outs": 1600, "out": "bf16"},
        # the queries of 128 heads for a decode step of 32 requests
        {"name": "product_step", "op": "product", "n": 32, "ins": 1024, "outs": 24576, "out": "bf16"},
        # a ragged chunk, odd in every size, with 32-bit results
        {"name": "product_ragged", "op": "product", "n": 333, "ins": 4112, "outs": 1601, "out": "fp32"},
        # a prompt's chunk
        {"name": "product_prompt", "op": "product", "n": 8192, "ins": 4096, "outs": 8192, "out": "bf16"},
        # one decode step of eight requests, text only
        {"name": "rotate_step", "op": "rotate", "n": 8, "heads": 128, "axes": 1, "format": "bf16", "pairs": "adjacent"},
        # a chunk of a prompt with images, whose tokens have a time, a height and a width
        {"name": "rotate_prompt", "op": "rotate", "n": 8191, "heads": 128, "axes": 3, "format": "compact", "pairs": "halves"},
        # a short follow-up of one request, few heads
        {"name": "chunk_one", "op": "chunk", "batch": 1, "new": 16, "T": 4096, "heads": 16, "k": 0, "edge": False},
        # a batch of ragged chunks, with a request that has none, a first token and a prompt without a prefix
        {"name": "chunk_ragged", "op": "chunk", "batch": 7, "new": 200, "T": 8192, "heads": 128, "k": 0, "edge": True},
        # a chunk of a long prompt
        {"name": "chunk_long", "op": "chunk", "batch": 1, "new": 512, "T": 32768, "heads": 128, "k": 0, "edge": False},
        # a chunk whose queries read the 2048 tokens that an indexer selected for each
        {"name": "chunk_listed", "op": "chunk", "batch": 2, "new": 160, "T": 32768, "heads": 128, "k": 2048, "edge": False},
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "product", "product", "product", "rotate", "chunk", "chunk", "chunk"])
    if op == "quant":
        dim = 8 * _between(rng, 8, 2048) if rng.random() < 0.5 else 128 * rng.randint(1, 128)
        return {"op": op, "n": max(1, min(65536, _between(rng, 1, 1 << 26) // dim)), "dim": dim, "square": rng.random() < 0.5}
    if op == "product":
        ins = 16 * _between(rng, 4, 1024) if rng.random() < 0.4 else 128 * _between(rng, 1, 128)
        outs = _between(rng, 64, 24576) if rng.random() < 0.4 else 64 * _between(rng, 2, 384)
        n = _between(rng, 1, max(1, min(16384, (1 << 38) // (ins * outs))))
        return {"op": op, "n": n, "ins": ins, "outs": outs, "out": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "rotate":
        heads = rng.choice([1, 8, 16, 20, 64, 96, 128])
        return {"op": op, "n": _between(rng, 1, min(65536, 8192 * 128 // heads)), "heads": heads, "axes": rng.choice([1, 2, 3, 3, 4]),
                "format": rng.choice(list(ROW_BYTES)), "pairs": rng.choice(["adjacent", "halves"])}
    batch, heads = rng.choice([1, 1, 2, 3, 4, 8]), rng.choice([8, 16, 20, 32, 64, 96, 128, 128])
    new = _between(rng, 1, 1024)
    T = max(1, min(_between(rng, 1, 131072), (1 << 30) // (batch * new * heads)))
    new = min(new, T)
    k = rng.choice([0, 0, 0, 256, 512, 2048])
    if k:
        new = max(1, min(new, 320 // batch))
    return {"op": op, "batch": batch, "new": new, "T": T, "heads": heads, "k": k, "edge": batch >= 4 and rng.random() < 0.6}


def _requests(case):
    """(new tokens, tokens) of each request: the first has `new` and T, the others 10 to 100 % and 30 to 100 % of them;
    `edge`: of the last three one is a prompt without a prefix, one a first token, and one has no query."""
    rng = random.Random(case["batch"] * 1000003 + case["T"] * 31 + case["new"])
    got = [(case["new"], case["T"])]
    for _ in range(case["batch"] - 1):
        T = max(1, int(case["T"] * rng.uniform(0.3, 1.0)))
        got.append((max(1, min(T, int(case["new"] * rng.uniform(0.1, 1.0)))), T))
    if case["edge"]:
        got[-3:] = [(case["new"], case["new"]), (1, 1), (0, got[-1][1])]
    return got


def work(case):
    op = case["op"]
    if op == "quant":
        n, dim = case["n"], case["dim"]
        groups = -(-n // 128) if case["square"] else n
        return {"bytes": n * dim * 3 + groups * -(-dim // 128) * 4, "flops": n * dim * 2}
    if op == "product":
        n, ins, outs = case["n"], case["ins"], case["outs"]
        groups = -(-ins // 128)
        return {"bytes": (n + outs) * ins + n * groups * 4 + -(-outs // 128) * groups * 4 + n * outs * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * n * ins * outs}
    if op == "rotate":
        n, heads = case["n"], case["heads"]
        return {"bytes": n * (heads * ROPE * 2 * 2 + ROW * 2 + 8 + 4 * case["axes"] + ROW_BYTES[case["format"]]) + LATENT * 2,
                "flops": n * (heads * ROPE * 3 + ROW * 6)}
    heads, rows, scored, new = case["heads"], 0, 0, 0
    for n, T in _requests(case):
        new += n
        seen = [T - n + i + 1 for i in range(n)]
        if case["k"]:
            scored += sum(min(case["k"], s) for s in seen)
            rows += min(T, sum(min(case["k"], s) for s in seen))   # each row of the cache once
        else:
            scored += sum(seen)
            rows += T if n else 0
    return {"bytes": rows * 400 + new * heads * (ROW * 2 + LATENT * 2 + 4) + new * 4 * case["k"],
            "flops": scored * heads * 2 * (ROW + LATENT)}


# ------------------------------------------------------------------ inputs

def _power_of_two_at_least(x):
    """The smallest power of two at or above x > 0, as its exponent; 0 where x is 0."""
    m, e = torch.frexp(x)
    return torch.where(x > 0, e.to(torch.int32) - (m == 0.5).to(torch.int32), torch.zeros_like(e, dtype=torch.int32))


def _quant(x, square):
    """float32 [n][dim] -> (e4m3 codes [n][dim], float32 scales of 128 values of a row or of 128 x 128)."""
    n, dim = x.shape
    high = 128 if square else 1
    t = torch.nn.functional.pad(x, (0, -dim % 128, 0, -n % high))
    t = t.view(t.shape[0] // high, high, -1, 128)
    scale = torch.ldexp(torch.ones((), device=x.device), _power_of_two_at_least(t.abs().amax((1, 3)) / 448.0).clamp(min=-126))
    codes = (t / scale[:, None, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes.view(-1, t.shape[2] * 128)[:n, :dim].contiguous(), scale


def _encode(y, rope, fmt):
    """float32 [n, 512] and bf16 [n, 64] -> rows, uint8 [n, row bytes]."""
    n = y.shape[0]
    tail = rope.contiguous().view(torch.uint8)
    if fmt == "bf16":
        return torch.cat([y.to(torch.bfloat16).view(torch.uint8), tail], 1)
    if fmt == "compact":
        codes, scale = _quant(y, False)
        return torch.cat([codes.view(torch.uint8), scale.view(torch.uint8), tail], 1)
    t = y.view(n, 16, 32)
    e = _power_of_two_at_least(t.abs().amax(2) / 6.0).clamp(-23, 13)
    t = t / torch.ldexp(torch.ones((), device=y.device), e)[:, :, None]
    a = t.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(t).to(torch.uint8)).view(n, 256, 2)
    return torch.cat([code[:, :, 0] + 16 * code[:, :, 1], (e + 127).to(torch.uint8), tail], 1)


def _activations(n, dim, g):
    """Unit rows of uneven size with a few dims several times larger than the rest, as hidden rows have."""
    x = torch.randn(n, dim, generator=g, device="cuda") * (0.25 + 2.0 * torch.rand(n, 1, generator=g, device="cuda"))
    x[:, ::97] *= 8.0
    return x


def _axis_of_pair(axes):
    """The axis of each of the 32 pairs: the first half of them on the first (time), the rest in equal sections."""
    if axes == 1:
        return [0] * 32
    first = 16
    return [0] * first + [1 + i * (axes - 1) // (32 - first) for i in range(32 - first)]


def _freqs():
    return [10000.0 ** (-i / 32.0) for i in range(32)]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = dict(case)
    op = case["op"]
    if op == "quant":
        s["x"] = _activations(case["n"], case["dim"], g).to(torch.bfloat16)
    elif op == "product":
        s["codes"], s["scales"] = _quant(_activations(case["n"], case["ins"], g), False)
        w = torch.randn(case["outs"], case["ins"], generator=g, device="cuda") / math.sqrt(case["ins"])
        w *= torch.exp2(torch.randint(-3, 4, (case["outs"], 1), generator=g, device="cuda").float() / 2.0)
        s["w_codes"], s["w_scales"] = _quant(w, True)
        if own:
            from host_latent_cache_gb300.products import Weight8
            s["weight"] = Weight8(s["w_codes"], s["w_scales"])
    elif op == "rotate":
        n, heads, axes = case["n"], case["heads"], case["axes"]
        n_pages = -(-n // PAGE) + 3
        order = (torch.randperm(n_pages, generator=g, device="cuda")[:, None] * PAGE + torch.arange(PAGE, device="cuda")).view(-1)
        s["slots"] = order[:n].contiguous()
        s["kv"] = torch.randn(n, ROW, generator=g, device="cuda").to(torch.bfloat16)
        s["gamma"] = (0.5 + torch.rand(LATENT, generator=g, device="cuda")).to(torch.bfloat16)
        s["rows"] = torch.zeros(n_pages * PAGE, ROW_BYTES[case["format"]], dtype=torch.uint8, device="cuda")
        # the projection's queries hold 128 values without a position, then the 64 that turn
        s["q"] = torch.randn(n, heads, 192, generator=g, device="cuda").to(torch.bfloat16)
        s["absorbed"] = torch.zeros(n, heads, ROW, dtype=torch.bfloat16, device="cuda")
        t = torch.arange(n, device="cuda") + int(seed) % 100000
        side = 24   # images of 24 x 24 tokens: height and width within them, the time from image to image
        places = [t, t // side % side, t % side, t // (side * side)]
        s["pos"] = torch.stack(places[:axes]).to(torch.int32) if axes > 1 else t.to(torch.int32)
        s["freq"], s["axis"] = _freqs(), _axis_of_pair(axes) if axes > 1 else None
        if own:
            from host_latent_cache_gb300.rows import RowCache
            s["cache"] = RowCache(s["rows"], case["format"], page=PAGE)
    else:
        batch, heads = case["batch"], case["heads"]
        requests = _requests(case)
        total = sum(n for n, _ in requests)
        per = -(-case["T"] // PAGE)
        s["table"] = torch.randperm(batch * per, generator=g, device="cuda").view(batch, per).to(torch.int32)
        s["T_dev"] = torch.tensor([T for _, T in requests], dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor([sum(n for n, _ in requests[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")
        weight = 0.5 + torch.rand(LATENT, generator=g, device="cuda")
        weight[::61] *= 6.0
        rope = torch.randn(batch * per * PAGE, ROPE, generator=g, device="cuda").to(torch.bfloat16)
        s["rows"] = _encode(torch.randn(batch * per * PAGE, LATENT, generator=g, device="cuda") * weight, rope, "q4")
        s["queries"] = (0.5 * torch.randn(total, heads, ROW, generator=g, device="cuda")).to(torch.bfloat16)
        s["most"] = max(n for n, _ in requests)   # a host's bound for the plain form's padding
        s["list"] = None
        if case["k"]:   # distinct tokens that each query may see, in ascending order, as a selection emits them
            b = torch.repeat_interleave(torch.arange(batch, device="cuda"), s["cu"].diff().long(), output_size=total)
            seen = s["T_dev"][b] - (s["cu"][b + 1] - torch.arange(total, device="cuda")) + 1
            pick = torch.rand(total, case["T"], generator=g, device="cuda")
            pick.masked_fill_(torch.arange(case["T"], device="cuda") >= seen[:, None], -1.0)
            idx = pick.topk(min(case["k"], case["T"]), dim=1).indices
            far = torch.where(torch.gather(pick, 1, idx) < 0, torch.full_like(idx, 1 << 30), idx).sort(1).values
            s["list"] = torch.full((total, case["k"]), -1, dtype=torch.int32, device="cuda")
            s["list"][:, :far.shape[1]] = torch.where(far >= case["T"], torch.full_like(far, -1), far).to(torch.int32)
        if own:
            from host_latent_cache_gb300.rows import RowCache
            s["cache"] = RowCache(s["rows"], "q4", page=PAGE)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _run_own(s)
    return {"quant": _run_quant, "product": _run_product, "rotate": _run_rotate, "chunk": _run_chunk}[s["op"]](s)


def _run_own(s):
    op = s["op"]
    if op == "quant":
        from host_latent_cache_gb300.products import quant_q8
        codes, scales = quant_q8(s["x"], square=s["square"])
        return {"codes": codes, "scales": scales}
    if op == "product":
        return {"out": s["weight"].product(s["codes"], s["scales"], dtype=torch.bfloat16 if s["out"] == "bf16" else torch.float32)}
    if op == "rotate":
        from host_latent_cache_gb300.rows import rotate
        s["cache"].write(s["kv"], s["slots"], gamma=s["gamma"], eps=EPS, pos=s["pos"], inv_freq=s["freq"], pairs=s["pairs"], axes=s["axis"])
        q = rotate(s["q"][:, :, 128:], s["pos"], s["freq"], pairs=s["pairs"], axes=s["axis"], out=s["absorbed"][:, :, LATENT:])
        return {"q": q, **({"rows": s["cache"].read(s["slots"])} if s["format"] == "q4" else _parts(s["rows"], s["format"]))}
    out, lse = s["cache"].attend_chunk(s["queries"], s["cu"], s["table"], s["T_dev"], SM_SCALE, tokens=s["list"])
    return {"out": out, "lse": lse}


def _run_quant(s):
    codes, scales = _quant(s["x"].float(), s["square"])
    return {"codes": codes, "scales": scales}


def _run_product(s):
    x = s["codes"].float() * s["scales"].repeat_interleave(128, 1)[:, :s["ins"]]
    w = s["w_codes"].float() * s["w_scales"].repeat_interleave(128, 0)[:s["outs"]].repeat_interleave(128, 1)[:, :s["ins"]]
    y = x @ w.T
    return {"out": y.to(torch.bfloat16) if s["out"] == "bf16" else y}


def _parts(rows, fmt):
    """The whole cache as views of what it holds."""
    if fmt == "bf16":
        return {"rows": rows.view(torch.bfloat16)}
    return {"codes": rows[:, :512].view(torch.float8_e4m3fn), "scales": rows[:, 512:528].view(torch.float32),
            "rope": rows[:, 528:].view(torch.bfloat16)}


def _decode_q4(rows):
    """uint8 [..., 400] -> float32 [..., 576]."""
    lead = rows.shape[:-1]
    packed = rows[..., :256].int()
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=rows.device)
    level = torch.cat([level, -level])
    y = level[torch.stack([packed & 15, packed >> 4], -1)].view(*lead, 16, 32)
    y = torch.ldexp(y, rows[..., 256:272].int()[..., None] - 127)
    rope = rows[..., 272:].contiguous().view(torch.bfloat16).float()
    return torch.cat([y.view(*lead, 512), rope], -1)


def _turned(k, pos, freq, axis, pairs):
    """k float32 [n][..., 64] turned by the angles of its rows."""
    f = torch.tensor(freq, dtype=torch.float64, device="cuda")
    p = pos[None] if pos.dim() == 1 else pos
    angle = p.double()[torch.tensor(axis or [0] * 32, device="cuda")].T * f     # [n][32]
    angle = angle.view(k.shape[0], *[1] * (k.dim() - 2), 32)
    cos, sin = angle.cos().float(), angle.sin().float()
    if pairs == "adjacent":
        a, b = k[..., 0::2], k[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).view(k.shape)
    a, b = k[..., :32], k[..., 32:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _run_rotate(s):
    x = s["kv"].float()
    c = x[:, :LATENT]
    # the mean of squares in 64 bits: the codes of values next to a border hang on its last bits
    r = (1.0 / (c.double().square().mean(1, keepdim=True) + EPS).sqrt()).float()
    rope = _turned(x[:, LATENT:], s["pos"], s["freq"], s["axis"], s["pairs"]).to(torch.bfloat16)
    s["rows"][s["slots"]] = _encode(c * r * s["gamma"].float(), rope, s["format"])
    s["absorbed"][:, :, LATENT:] = _turned(s["q"][:, :, 128:].float(), s["pos"], s["freq"], s["axis"], s["pairs"]).to(torch.bfloat16)
    q = s["absorbed"][:, :, LATENT:]
    if s["format"] == "q4":   # packed codes are read back, as the values that they stand for
        return {"q": q, "rows": _decode_q4(s["rows"][s["slots"]]).to(torch.bfloat16)}
    return {"q": q, **_parts(s["rows"], s["format"])}


def _softmax_values(score, live, values):
    """(weighted values, logarithm of the sum) of the live scores; zeros and -infinity where none is."""
    score = torch.where(live, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = (p @ values) / torch.where(total > 0, total, torch.ones_like(total))
    return out, torch.where(total > 0, top + torch.log(total), torch.full_like(top, -math.inf))[..., 0]


def _run_chunk(s):
    q, T, cu, table = s["queries"].float(), s["T_dev"].long(), s["cu"].long(), s["table"].long()
    total, heads, _ = q.shape
    batch = s["batch"]
    b = torch.searchsorted(cu, torch.arange(total, device="cuda"), right=True) - 1
    i = torch.arange(total, device="cuda") - cu[b]
    if s["list"] is not None:
        t = s["list"].long()
        live = (t >= 0)[:, None]
        t = t.clamp(min=0)
        k = _decode_q4(s["rows"][torch.gather(table[b], 1, t // PAGE) * PAGE + t % PAGE])   # [total][k][576]
        out, lse = _softmax_values((q @ k.transpose(1, 2)) * SM_SCALE, live, k[..., :LATENT])
        return {"out": out.to(torch.bfloat16), "lse": lse}
    most = s["most"]
    padded = torch.zeros(batch, most, heads, ROW, device="cuda")
    padded[b, i] = q
    t = torch.arange(s["T"], device="cuda")
    k = _decode_q4(s["rows"][table[:, t // PAGE] * PAGE + t % PAGE])                        # [batch][T][576]
    seen = (T - cu.diff())[:, None] + torch.arange(most, device="cuda") + 1                 # tokens that a query sees
    live = (t < seen[:, :, None])[:, :, None].expand(-1, -1, heads, -1).reshape(batch, most * heads, -1)
    out, lse = _softmax_values((padded.view(batch, most * heads, ROW) @ k.transpose(1, 2)) * SM_SCALE, live, k[..., :LATENT])
    return {"out": out.view(batch, most, heads, LATENT)[b, i].to(torch.bfloat16), "lse": lse.view(batch, most, heads)[b, i].contiguous()}


# ------------------------------------------------------------------ 64 bits, from the definitions

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _e4m3_levels():
    return [m / 8.0 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8.0) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(a, levels):
    """The index of the nearest level of each magnitude (the even one of two as near, the largest above all)."""
    lv = torch.tensor(levels, dtype=torch.float64, device=a.device)
    i = torch.searchsorted(lv, a.contiguous()).clamp(1, len(levels) - 1)
    down, up = a - lv[i - 1], lv[i] - a
    return torch.where((down < up) | ((down == up) & (i % 2 == 1)), i - 1, i)


def _steps(amax, most):
    """2^e, the smallest at or above amax / most in 32 bits; 1 for 0."""
    x = (amax.float() / most).double()
    e = torch.ceil(torch.log2(torch.where(x > 0, x, torch.ones_like(x))))
    e = torch.where(torch.exp2(e - 1) >= x, e - 1, e)
    e = torch.where(torch.exp2(e) < x, e + 1, e)
    return torch.where(x > 0, torch.exp2(e), torch.ones_like(x))


def _on_levels(y, high, wide, levels, lo, hi):
    """(values on the levels, steps) of blocks of high x wide values, the last ones filled up with zeros."""
    n, dim = y.shape
    whole = torch.zeros(-(-n // high) * high, -(-dim // wide) * wide, dtype=torch.float64, device=y.device)
    whole[:n, :dim] = y
    blocks = whole.unflatten(0, (-1, high)).unflatten(2, (-1, wide))
    step = _steps(blocks.abs().amax((1, 3)), levels[-1]).clamp(2.0 ** lo, 2.0 ** hi)
    unit = blocks / step[:, None, :, None]
    value = torch.tensor(levels, dtype=torch.float64, device=y.device)[_nearest(unit.abs(), levels)] * torch.sign(unit)
    return value.flatten(2).flatten(0, 1)[:n, :dim], step


def _values_of_codes(codes):
    raw = codes.view(torch.uint8).long()
    lv = torch.tensor(_e4m3_levels() + [math.nan], dtype=torch.float64, device=codes.device)
    return lv[raw % 128] * (1.0 - 2.0 * (raw // 128).double())


def _q4_values(rows):
    lv = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device=rows.device)
    y = torch.empty(rows.shape[0], LATENT, dtype=torch.float64, device=rows.device)
    y[:, 0::2], y[:, 1::2] = lv[(rows[:, :256] % 16).long()], lv[(rows[:, :256] // 16).long()]
    y *= torch.exp2(rows[:, 256:272].double() - 127.0).repeat_interleave(32, 1)
    return torch.cat([y, rows[:, 272:].contiguous().view(torch.bfloat16).double()], 1)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"quant": _exact_quant, "product": _exact_product, "rotate": _exact_rotate, "chunk": _exact_chunk}[case["op"]](s)


def _exact_quant(s):
    codes, step = _on_levels(s["x"].double(), 128 if s["square"] else 1, 128, _e4m3_levels(), -126, 127)
    return {"codes": codes, "scales": step}


def _exact_product(s):
    x, w = _values_of_codes(s["codes"]), _values_of_codes(s["w_codes"])
    out = torch.zeros(s["n"], s["outs"], dtype=torch.float64, device="cuda")
    for j in range(s["scales"].shape[1]):   # one group of 128 at a time
        at = slice(128 * j, min(128 * j + 128, s["ins"]))
        out += (x[:, at] * s["scales"][:, j:j + 1].double()) @ (w[:, at] * s["w_scales"][torch.arange(s["outs"], device="cuda") // 128, j, None].double()).T
    return {"out": out}


def _exact_turn(k, s):
    """k [n][..., 64] as 32 complex numbers, times a unit one each."""
    k = k.double()
    z = torch.complex(k[..., 0::2].contiguous(), k[..., 1::2].contiguous()) if s["pairs"] == "adjacent" else torch.complex(k[..., :32].contiguous(), k[..., 32:].contiguous())
    axis = s["axis"] or [0] * 32
    pos = s["pos"].view(-1, s["n"])
    angle = torch.stack([pos[axis[i]].double() * s["freq"][i] for i in range(32)], 1)
    z = z * torch.polar(torch.ones_like(angle), angle).view(s["n"], *[1] * (k.dim() - 2), 32)
    return torch.view_as_real(z).flatten(-2) if s["pairs"] == "adjacent" else torch.cat([z.real, z.imag], -1)


def _exact_rotate(s):
    c = s["kv"][:, :LATENT].double()
    y = c / torch.sqrt((c * c).sum(1, keepdim=True) / LATENT + EPS) * s["gamma"].double()
    rope, size = _exact_turn(s["kv"][:, LATENT:], s), s["rows"].shape[0]

    def whole(v):
        full = torch.zeros(size, v.shape[1], dtype=torch.float64, device="cuda")
        full[s["slots"]] = v.double()
        return full

    q = _exact_turn(s["q"][:, :, 128:], s)
    if s["format"] == "bf16":
        return {"q": q, "rows": whole(torch.cat([y, rope], 1))}
    if s["format"] == "compact":
        codes, step = _on_levels(y, 1, 128, _e4m3_levels(), -126, 127)
        return {"q": q, "codes": whole(codes), "scales": whole(step), "rope": whole(rope)}
    codes, step = _on_levels(y, 1, 32, _E2M1, -23, 13)
    return {"q": q, "rows": torch.cat([codes * step.repeat_interleave(32, 1), rope], 1)}


def _exact_chunk(s):
    requests = _requests(s)
    total, heads, _ = s["queries"].shape
    out = torch.zeros(total, heads, LATENT, dtype=torch.float64, device="cuda")
    lse = torch.full((total, heads), -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, T) in enumerate(requests):
        t = torch.arange(T, device="cuda")
        rows = _q4_values(s["rows"][s["table"][b, t // PAGE].long() * PAGE + t % PAGE])
        some = 1 if s["list"] is not None else max(1, (1 << 24) // (heads * T))   # query tokens at a time
        for i in range(0, n, some):
            to = slice(at + i, at + min(n, i + some))
            if s["list"] is not None:
                pick = s["list"][at + i]
                k = rows[pick[pick >= 0].long()]
                hide = None
            else:
                k = rows[:T - n + min(n, i + some)]
                hide = torch.arange(k.shape[0], device="cuda") > (T - n + torch.arange(i, min(n, i + some), device="cuda"))[:, None, None]
            z = s["queries"][to].double() @ k.T / math.sqrt(ROW)
            if hide is not None:
                z = z.masked_fill(hide, -math.inf)
            lse[to] = torch.logsumexp(z, -1)
            out[to] = torch.exp(z - lse[to][..., None]) @ k[:, :LATENT]
        at += n
    return {"out": out, "lse": lse}
