"""The attention operators' workloads: a transformer block's rotary positions
and attention over packed sequences, forward and backward, for prompts and for
single tokens over a cache.

``listed()`` gives the fixed cases, ``draw(rng)`` one more of the same ranges.
``prepare(case, seed)`` makes a case's device tensors, ``run(state)`` is one
pass: the framework's calls where the module's ``own`` is true, and the plain
form otherwise (elementary torch operations in FP32, angles in FP64, rounded
once at the end).  ``exact(case, seed)`` evaluates the definitions in FP64,
written apart from the plain form.  ``work(case)`` counts the bytes and
operations that a pass cannot do without.

Layouts: tokens are rows; a token's heads follow one another, ``dim`` values
each.  Sequence s owns q_len[s] rows of Q and k_len[s] rows of K and V.

  rotary           (a, b) -> amplitude (a cos p - b sin p, a sin p + b cos p),
                   p = position * frequency, on the first ``rot`` values of a head
  rotary_backward  the transpose of that map on the gradients
  attention        O = softmax(scale Q K^T) V over the keys that a row sees,
                   LSE = log sum exp(scale Q K^T); causal: key j of row i with
                   j <= i + k_len - q_len; a row without keys gives zeros
  attention_backward  P = exp(scale Q K^T - LSE), dS = P (dO V^T - sum(dO O)),
                   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO, the heads
                   of a group summed in dK and dV
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases


def _ragged(total, count, seed):
    """`count` lengths of sum `total`, uneven, from the seed alone."""
    x, parts = seed * 2654435761 % 4294967291 + 1, []
    for _ in range(count):
        x = x * 48271 % 2147483647
        parts.append(1.0 + (x % 1000) ** 2 / 2e4)
    cuts, at = [0], 0.0
    for p in parts:
        at += p
        cuts.append(int(round(at / sum(parts) * total)))
    cuts[-1] = total
    return [b - a for a, b in zip(cuts, cuts[1:])]


def lengths(case):
    """(rows of Q, keys) of each sequence.  `kind`: "self" (a packed batch whose
    sequences attend themselves), "chunk" (new rows behind what a cache keeps)
    and "cross" (Q and K of unrelated lengths).  `even`: as many rows of Q each."""
    n, t = case["seqs"], case["tokens"]
    q = [t // n] * n if case["even"] else _ragged(t, n, case["shape_seed"])
    if case["kind"] == "self":
        return q, list(q)
    k = _ragged(case["keys"], n, case["shape_seed"] + 1)
    if case["kind"] == "chunk":
        k = [a + b for a, b in zip(q, k)]
    return q, k


def _capacity(case):
    """Cache rows kept for each sequence (0: packed keys)."""
    return max(lengths(case)[1]) + case["room"] if case["kind"] == "chunk" else 0


def _attention(name, op, dtype, kind, seqs, tokens, heads, kv, dim, keys=0, even=False, causal=True,
               shape_seed=1, room=0):
    return {"name": name, "op": op, "dtype": dtype, "kind": kind, "seqs": seqs, "tokens": tokens,
            "keys": keys, "even": even, "shape_seed": shape_seed, "heads": heads, "kv": kv,
            "dim": dim, "causal": causal, "room": room}


def _rotary(name, op, dtype, tokens, heads, dim, rot, layout, scaling, pad, far):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "heads": heads, "dim": dim,
            "rot": rot, "layout": layout, "scaling": scaling, "pad": pad, "far": far}


def listed():
    return [
        # A decoding step's Q and K heads of eight sequences at far positions,
        # with the frequencies of a long context: the smallest call.
        _rotary("rotary_tokens", "rotary", "bf16", 8, 40, 128, 128, "halves", "bands", 0, 131072),
        # A long prompt's Q and K heads inside the packed QKV rows.
        _rotary("rotary_prompt_8192", "rotary", "bf16", 8192, 40, 128, 128, "halves", "linear", 1024,
                0),
        # A training step's gradients, a third of each head turned, pairs.
        _rotary("rotary_backward_part", "rotary_backward", "fp16", 4099, 20, 96, 32, "pairs", "none",
                0, 0),
        # Decoding: one new token of each of 32 sequences over a cache of uneven
        # fill (354 to 11799 keys), as many rows kept for each.
        _attention("attention_tokens", "attention", "bf16", "chunk", 32, 32, 32, 8, 128, keys=131072,
                   even=True, shape_seed=3, room=64),
        # Decoding one sequence with a very long context: few rows, a long axis.
        _attention("attention_long_token", "attention", "bf16", "chunk", 1, 1, 32, 8, 128,
                   keys=131071, even=True),
        # A whole prompt.
        _attention("attention_prompt_8192", "attention", "bf16", "self", 1, 8192, 32, 8, 128),
        # A packed batch of uneven prompts, every head with its own keys.
        _attention("attention_packed", "attention", "fp16", "self", 13, 8191, 16, 16, 64,
                   shape_seed=5),
        # The next chunk of a long prompt behind what the cache holds already.
        _attention("attention_chunk", "attention", "bf16", "chunk", 1, 500, 32, 8, 128, keys=16000,
                   room=140),
        # Short texts of an encoder: no mask, a head size between two tiles.
        _attention("attention_short", "attention", "fp16", "self", 16, 333, 12, 12, 80, causal=False,
                   shape_seed=7),
        # A training step on one long sequence: the largest case.
        _attention("attention_backward_8192", "attention_backward", "bf16", "self", 1, 8192, 32, 8,
                   128),
        # A training step on a packed batch.
        _attention("attention_backward_packed", "attention_backward", "fp16", "self", 13, 4099, 16,
                   4, 64, shape_seed=5),
        # Rows and keys of unrelated lengths, odd head size; under the causal
        # rule some rows see no key.
        _attention("attention_backward_cross", "attention_backward", "bf16", "cross", 5, 901, 6, 2,
                   72, keys=777, shape_seed=9),
    ]


# The largest listed case's operations (one long sequence, backward).
MOST_FLOPS = 10.0 * 128 * 32 * 8192 * 8193 / 2


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_backward", "attention", "attention", "attention",
                     "attention_backward", "attention_backward"])
    if op.startswith("rotary"):
        dim = rng.choice([64, 128, 128, 80, 96, 72, 256])
        rot = rng.choice([dim, dim, dim // 2 // 2 * 2, dim // 4 // 2 * 2])
        return _rotary("", op, rng.choice(["bf16", "fp16", "f32"]), _spread(rng, 1, 8192),
                       _spread(rng, 1, 40), dim, rot, rng.choice(["halves", "pairs"]),
                       rng.choice(["none", "linear", "base", "bands"]), rng.choice([0, 0, 8, 3]),
                       rng.choice([0, 0, 131072, 1000000]))
    while True:
        kv = rng.choice([1, 2, 4, 8, 8, 16])
        heads = kv * rng.choice([1, 1, 2, 4, 4, 8, 3, 7])
        kind = rng.choice(["self", "self", "cross"] if op == "attention_backward"
                          else ["self", "self", "chunk", "chunk", "cross"])
        seqs = _spread(rng, 1, 64)
        if kind == "chunk" and rng.random() < 0.6:
            tokens = seqs * rng.choice([1, 1, 1, 2, 4])  # decoding
            even, keys = rng.random() < 0.8, _spread(rng, seqs, 262144)
        else:
            tokens = max(seqs, _spread(rng, 1, 8192))
            even, keys = rng.random() < 0.2, max(seqs, _spread(rng, 16, 32768))
        case = _attention("", op, rng.choice(["bf16", "fp16"]), kind, seqs, tokens, heads, kv,
                          rng.choice([64, 64, 128, 128, 128, 80, 96, 72, 40, 32]),
                          keys=0 if kind == "self" else keys, even=even,
                          causal=rng.random() < 0.75, shape_seed=rng.randrange(1, 1000))
        if even:
            case["tokens"] = tokens // seqs * seqs
        case["room"] = rng.choice([0, 5, 64])
        q, k = lengths(case)
        if heads <= 64 and work(case)["flops"] <= MOST_FLOPS and work(case)["bytes"] < 2e9 and \
                sum(k) * case["kv"] * case["dim"] < 3e8 and \
                seqs * _capacity(case) * case["kv"] * case["dim"] < 1e9 and \
                max(a * b for a, b in zip(q, k)) * heads <= 2.2e9:
            return case


def _pairs(case):
    """(row, key) pairs that are seen, over one head."""
    n = 0
    for a, b in zip(*lengths(case)):
        if not case["causal"]:
            n += a * b
        else:
            rows, lead = min(a, b), max(b - a, 0)  # rows with a key; keys that all of them see
            n += rows * lead + rows * (rows + 1) // 2
    return n


def work(case):
    if case["op"].startswith("rotary"):
        e = 4 if case["dtype"] == "f32" else 2
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * e + 8 * case["tokens"] + 4 * case["rot"],
                "flops": 3 * n * case["rot"]}
    h, kv, d = case["heads"], case["kv"], case["dim"]
    tq, tk = (sum(x) for x in lengths(case))
    pairs = _pairs(case)
    if case["op"] == "attention":
        return {"bytes": 2 * d * (2 * tq * h + 2 * tk * kv) + 4 * tq * h, "flops": 4 * d * h * pairs}
    return {"bytes": 2 * d * (4 * tq * h + 4 * tk * kv) + 4 * tq * h, "flops": 10 * d * h * pairs}


# ------------------------------------------------------------------ frequencies

BASE = 500000.0
FACTOR, LOW, HIGH, ORIGINAL = 8.0, 1.0, 4.0, 8192.0


def _frequencies(case):
    """Radians a position, FP64."""
    r = case["rot"]
    i = torch.arange(0, r, 2, dtype=torch.float64)
    base = BASE
    if case["scaling"] == "base":
        base = BASE * FACTOR ** (r / (r - 2)) if r > 2 else BASE
    f = torch.pow(torch.tensor(base, dtype=torch.float64), -i / r)
    if case["scaling"] == "linear":
        f = f / FACTOR
    if case["scaling"] == "bands":
        turns = ORIGINAL * f / (2 * math.pi)
        g = torch.clamp((turns - LOW) / (HIGH - LOW), 0.0, 1.0)
        f = g * f + (1 - g) * f / FACTOR
    return f


AMPLITUDE = {"none": 1.0, "linear": 1.0, "base": 1.0, "bands": 1.125}


# ------------------------------------------------------------------ inputs


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rotary_inputs(case, seed):
    g = _gen(seed)
    t, h, d = case["tokens"], case["heads"], case["dim"]
    buf = torch.full((t, h * d + case["pad"]), float("nan"), dtype=TYPES[case["dtype"]], device="cuda")
    x = buf[:, : h * d].unflatten(1, (h, d))
    x.copy_(torch.randn(t, h, d, generator=g, device="cuda"))
    if case["far"]:
        pos = torch.randint(0, case["far"], (t,), generator=g, device="cuda")
    else:
        pos = torch.arange(t, device="cuda")
    return {"X": x, "positions": pos}


def _starts(sizes):
    s = [0]
    for n in sizes:
        s.append(s[-1] + n)
    return s


def _attention_inputs(case, seed):
    """Q, K, V (and dO, O, LSE), the sequences' starts on the host."""
    g = _gen(seed)
    t, h, kv, d = TYPES[case["dtype"]], case["heads"], case["kv"], case["dim"]
    q_len, k_len = lengths(case)
    tq = sum(q_len)
    if case["kind"] == "self":  # views of one QKV projection's rows
        qkv = torch.randn(tq, h + 2 * kv, d, generator=g, device="cuda").to(t)
        s = {"Q": qkv[:, :h], "K": qkv[:, h: h + kv], "V": qkv[:, h + kv:]}
        k_at = _starts(q_len)
    else:
        cap = _capacity(case)
        rows = cap * case["seqs"] if cap else sum(k_len)
        s = {"Q": torch.randn(tq, h, d, generator=g, device="cuda").to(t)}
        for name in "KV":
            s[name] = torch.randn(rows, kv, d, generator=g, device="cuda").to(t)
        k_at = [i * cap for i in range(case["seqs"] + 1)] if cap else _starts(k_len)
    s["q_at"], s["k_at"], s["q_len"], s["k_len"] = _starts(q_len), k_at, q_len, k_len
    if case["op"] == "attention_backward":
        s["dO"] = torch.randn(tq, h, d, generator=g, device="cuda").to(t)
        o = _plain_attention(case, s)
        s["O"], s["LSE"] = o["O"], o["LSE"]
    return s


def prepare(case, seed):
    """The inputs, the buffers that the outputs go to, and the frequencies or
    the sequences' starts on the device, which a program makes once a batch."""
    t = TYPES[case["dtype"]]
    if case["op"].startswith("rotary"):
        s = {"case": case, "in": _rotary_inputs(case, seed), "freq": _frequencies(case).cuda()}
        s["out"] = {"Y": torch.empty(case["tokens"], case["heads"], case["dim"], dtype=t, device="cuda")}
        if own:
            import dense_gemm_epilogue_gb300 as tg

            steps = tg.tg_rotary_steps(case["rot"], BASE, case["scaling"], FACTOR, LOW, HIGH, ORIGINAL)
            s["steps"] = torch.tensor(steps, dtype=torch.int64, device="cuda")
        return s
    i = _attention_inputs(case, seed)
    s = {"case": case, "in": i, "out": {}}
    s["device"] = {name: torch.tensor(i[name], dtype=torch.int64, device="cuda")
                   for name in ("q_at", "k_at", "k_len")}
    if case["op"] == "attention":
        s["out"]["O"] = torch.empty(i["Q"].shape, dtype=t, device="cuda")
        s["out"]["LSE"] = torch.empty(case["heads"], i["Q"].shape[0], device="cuda")
    else:
        for name in "QKV":
            s["out"]["d" + name] = torch.empty(i[name].shape, dtype=t, device="cuda")
    return s


# ------------------------------------------------------------------ the plain form


def _plain_rotary(case, i, freq):
    t, r = TYPES[case["dtype"]], case["rot"]
    angle = i["positions"].double()[:, None] * freq
    c = (torch.cos(angle) * AMPLITUDE[case["scaling"]]).float()[:, None]
    s = (torch.sin(angle) * AMPLITUDE[case["scaling"]]).float()[:, None]
    if case["op"] == "rotary_backward":
        s = -s
    x = i["X"].float()
    y = x.clone()
    if case["layout"] == "halves":
        a, b = slice(0, r // 2), slice(r // 2, r)
    else:
        a, b = slice(0, r, 2), slice(1, r, 2)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return {"Y": y.to(t)}


def _sequences(case, i):
    """(rows, keys, q_len, k_len) of each sequence that has rows."""
    for n in range(case["seqs"]):
        a, b = i["q_len"][n], i["k_len"][n]
        if a:
            yield (slice(i["q_at"][n], i["q_at"][n] + a), slice(i["k_at"][n], i["k_at"][n] + b), a, b)


def _hidden(case, a, b):
    """True where row i of a does not see key j of b, or None."""
    if not case["causal"] or a == 1:
        return None
    i = torch.arange(a, device="cuda")[:, None]
    return torch.arange(b, device="cuda") > i + (b - a)


def _groups(case, a, b):
    """Slices of K's heads, as many at a time as keep the scores at 1 GB."""
    g = case["heads"] // case["kv"]
    n = max(1, (1 << 28) // (g * a * b))
    return [slice(j, min(j + n, case["kv"])) for j in range(0, case["kv"], n)]


def _by_group(x, n, g):
    """(rows, heads, dim) of the query side to (groups, heads of one, rows, dim), FP32."""
    return x[:, n.start * g: n.stop * g].float().unflatten(1, (n.stop - n.start, g)).permute(1, 2, 0, 3)


def _scores(case, q, k, hidden):
    """scale Q K^T: (groups, heads of one, rows, keys), FP32."""
    s = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(case["dim"]))
    return s if hidden is None else s.masked_fill_(hidden, -math.inf)


def _plain_attention(case, i):
    t, g = TYPES[case["dtype"]], case["heads"] // case["kv"]
    tq = i["Q"].shape[0]
    o = torch.zeros(tq, case["heads"], case["dim"], dtype=t, device="cuda")
    lse = torch.full((case["heads"], tq), -math.inf, device="cuda")
    for rows, keys, a, b in _sequences(case, i):
        if b == 0:
            continue
        hidden = _hidden(case, a, b)
        for n in _groups(case, a, b):
            hs = slice(n.start * g, n.stop * g)
            q = _by_group(i["Q"][rows], n, g)
            k, v = (i[x][keys, n].float().transpose(0, 1)[:, None] for x in "KV")
            s = _scores(case, q, k, hidden)
            m = s.amax(-1, keepdim=True).clamp_(min=-3e38)
            p = s.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            lse[hs, rows] = (m + l.log())[..., 0].flatten(0, 1)
            y = (p @ v).div_(l.clamp(min=1e-30))
            o[rows, hs] = y.permute(2, 0, 1, 3).flatten(1, 2).to(t)
    return {"O": o, "LSE": lse}


def _plain_backward(case, i):
    t, g = TYPES[case["dtype"]], case["heads"] // case["kv"]
    scale = 1.0 / math.sqrt(case["dim"])
    out = {"d" + name: torch.zeros(i[name].shape, dtype=t, device="cuda") for name in "QKV"}
    for rows, keys, a, b in _sequences(case, i):
        if b == 0:
            continue
        hidden = _hidden(case, a, b)
        for n in _groups(case, a, b):
            hs = slice(n.start * g, n.stop * g)
            q, do, o = (_by_group(i[x][rows], n, g) for x in ("Q", "dO", "O"))
            k, v = (i[x][keys, n].float().transpose(0, 1)[:, None] for x in "KV")
            lse = i["LSE"][hs, rows].unflatten(0, (n.stop - n.start, g))[..., None]
            p = _scores(case, q, k, hidden).sub_(lse).exp_()
            if b < a:
                p = torch.where(lse == -math.inf, torch.zeros_like(p), p)
            delta = (do * o).sum(-1, keepdim=True)
            out["dV"][keys, n] = (p.transpose(-1, -2) @ do).sum(1).transpose(0, 1).to(t)
            ds = (do @ v.transpose(-1, -2)).sub_(delta).mul_(p).mul_(scale)
            del p
            out["dQ"][rows, hs] = (ds @ k).permute(2, 0, 1, 3).flatten(1, 2).to(t)
            out["dK"][keys, n] = (ds.transpose(-1, -2) @ q).sum(1).transpose(0, 1).to(t)
    return out


# ------------------------------------------------------------------ the framework's calls


def _space(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def _lay(x):
    """A tensor with its token and head strides."""
    return x, x.stride(0), x.stride(1)


def _framework_rotary(state):
    import dense_gemm_epilogue_gb300 as tg

    case, i, y = state["case"], state["in"], state["out"]["Y"]
    st = torch.cuda.current_stream()
    if case["op"] == "rotary":
        tg.check(tg.tg_rotary(case["tokens"], case["heads"], case["dim"], case["rot"], *_lay(i["X"]),
                              *_lay(y), 0, i["positions"], None, state["steps"], case["layout"],
                              AMPLITUDE[case["scaling"]], case["dtype"], st))
    else:
        tg.check(tg.tg_rotary_backward(case["tokens"], case["heads"], case["dim"], case["rot"],
                                       *_lay(i["X"]), *_lay(y), i["positions"], state["steps"],
                                       case["layout"], AMPLITUDE[case["scaling"]], case["dtype"], st))
    return state["out"]


def _framework_attention(state):
    import dense_gemm_epilogue_gb300 as tg

    case, i, o, at = state["case"], state["in"], state["out"], state["device"]
    st = torch.cuda.current_stream()
    scale = 1.0 / math.sqrt(case["dim"])
    size = (case["seqs"], i["Q"].shape[0], i["K"].shape[0], case["heads"], case["kv"], case["dim"])
    top = (max(i["q_len"]), max(i["k_len"]))
    k_len = at["k_len"] if case["kind"] == "chunk" else None
    if case["op"] == "attention":
        ws = _space(tg.tg_attention_workspace_bytes(*size, *top, case["dtype"]))
        tg.check(tg.tg_attention(*size, *_lay(i["Q"]), *_lay(i["K"]), *_lay(i["V"]), at["q_at"], None,
                                 at["k_at"], k_len, *top, case["causal"], scale, *_lay(o["O"]),
                                 o["LSE"], case["dtype"], ws, st))
    else:
        ws = _space(tg.tg_attention_backward_workspace_bytes(*size, *top, case["dtype"]))
        tg.check(tg.tg_attention_backward(*size, *_lay(i["Q"]), *_lay(i["K"]), *_lay(i["V"]),
                                          *_lay(i["O"]), *_lay(i["dO"]), i["LSE"], at["q_at"], None,
                                          at["k_at"], k_len, *top, case["causal"], scale,
                                          *_lay(o["dQ"]), *_lay(o["dK"]), *_lay(o["dV"]),
                                          case["dtype"], ws, st))
    return o


def run(state):
    case = state["case"]
    if case["op"].startswith("rotary"):
        if own:
            return _framework_rotary(state)
        return _plain_rotary(case, state["in"], state["freq"])
    if own:
        return _framework_attention(state)
    return (_plain_attention if case["op"] == "attention" else _plain_backward)(case, state["in"])


# ------------------------------------------------------------------ the definitions in 64 bits


def _exact_rotary(case, i):
    """As a product of complex numbers."""
    z = torch.polar(torch.tensor(AMPLITUDE[case["scaling"]], dtype=torch.float64, device="cuda"),
                    torch.einsum("t,i->ti", i["positions"].double(), _frequencies(case).cuda()))
    if case["op"] == "rotary_backward":
        z = z.conj()
    r, x = case["rot"], i["X"].double()
    if case["layout"] == "halves":
        w = torch.complex(x[..., : r // 2], x[..., r // 2: r]) * z[:, None]
        y = torch.cat([w.real, w.imag, x[..., r:]], -1)
    else:
        w = torch.complex(x[..., 0:r:2], x[..., 1:r:2]) * z[:, None]
        y = torch.cat([torch.view_as_real(w).flatten(-2), x[..., r:]], -1)
    return {"Y": y}


def _exact_head(case, i, n, h):
    """Sequence n, head h, in blocks of rows: (rows, visible keys, S) in FP64."""
    a, b, q0, k0 = i["q_len"][n], i["k_len"][n], i["q_at"][n], i["k_at"][n]
    k = i["K"][k0: k0 + b, h // (case["heads"] // case["kv"])].double()
    for r in range(0, a, 2048):
        e = min(r + 2048, a)
        seen = b if not case["causal"] else min(b, max(0, e + b - a))
        if seen == 0:
            continue
        q = i["Q"][q0 + r: q0 + e, h].double()
        s = torch.einsum("id,jd->ij", q, k[:seen]) / math.sqrt(case["dim"])
        if case["causal"]:
            keep = torch.ones(e - r, seen, dtype=torch.bool, device="cuda").tril(r + b - a)
            s = torch.where(keep, s, torch.full_like(s, -math.inf))
        yield slice(q0 + r, q0 + e), slice(k0, k0 + seen), s


def _exact_attention(case, i):
    o = torch.zeros(i["Q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["heads"], i["Q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for n in range(case["seqs"]):
        for h in range(case["heads"]):
            for rows, keys, s in _exact_head(case, i, n, h):
                z = torch.logsumexp(s, 1)
                p = torch.where(z[:, None] == -math.inf, 0.0, torch.exp(s - z[:, None]))
                v = i["V"][keys, h // (case["heads"] // case["kv"])].double()
                lse[h, rows] = z
                o[rows, h] = torch.einsum("ij,jd->id", p, v)
    return {"O": o, "LSE": lse}


def _exact_backward(case, i):
    out = {"d" + name: torch.zeros(i[name].shape, dtype=torch.float64, device="cuda") for name in "QKV"}
    g = case["heads"] // case["kv"]
    for n in range(case["seqs"]):
        for h in range(case["heads"]):
            for rows, keys, s in _exact_head(case, i, n, h):
                z = i["LSE"][h, rows].double()[:, None]
                p = torch.where(z == -math.inf, 0.0, torch.exp(s - z))
                do, o = i["dO"][rows, h].double(), i["O"][rows, h].double()
                k, v = i["K"][keys, h // g].double(), i["V"][keys, h // g].double()
                delta = torch.einsum("id,id->i", do, o)[:, None]
                ds = p * (torch.einsum("id,jd->ij", do, v) - delta) / math.sqrt(case["dim"])
                out["dV"][keys, h // g] += torch.einsum("ij,id->jd", p, do)
                out["dK"][keys, h // g] += torch.einsum("ij,id->jd", ds, i["Q"][rows, h].double())
                out["dQ"][rows, h] = torch.einsum("ij,jd->id", ds, k)
    return out


def exact(case, seed):
    if case["op"].startswith("rotary"):
        return _exact_rotary(case, _rotary_inputs(case, seed))
    if case["seqs"] * case["heads"] * 8 > 40000:  # (one small step for each sequence and head)
        return None
    i = _attention_inputs(case, seed)
    return (_exact_attention if case["op"] == "attention" else _exact_backward)(case, i)
