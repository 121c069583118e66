"""Performance cases of the operators around verification: the token history
of every request, the rules applied to the logits (penalties for repeated
tokens, biases, grammar masks), and the output head with 4-bit weights.

    listed()           the named cases
    draw(rng)          one more case of the same ranges
    prepare(case, s)   the inputs of one case on the GPU, from the seed s
    run(state)         one pass; `own` selects the library's kernels (true)
                       or the plain torch form (false)
    work(case)         bytes and operations that one pass cannot do without
    exact(case, s)     the result in 64 bits
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# Cases.
# ---------------------------------------------------------------------------
def _history(name, kind, B, S, V):
    return dict(name=name, op="history", kind=kind, B=B, S=S, V=V)


def _process(name, B, K, V, dtype, in_place, ragged, prompt, output, bias, grammar):
    """K drafts and the position after them; `grammar`: percent of the rows
    whose positions carry a mask."""
    return dict(name=name, op="process", B=B, K=K, V=V, dtype=dtype, in_place=in_place,
                ragged=ragged, prompt=prompt, output=output, bias=bias, grammar=grammar)


def _head(name, B, P, H, V, group, zero, out, scale, ragged):
    return dict(name=name, op="head", B=B, P=P, H=H, V=V, group=group, zero=zero, out=out,
                scale=scale, ragged=ragged)


def listed():
    return [
        # The emitted tokens of one verification step of four short requests.
        _history("commit_small", "output", 4, 5, 1000),
        # The same for a full serving batch: up to nine tokens a row.
        _history("commit", "output", 256, 9, 129280),
        # Prompts of a new batch of requests, ragged, up to 4096 tokens.
        _history("prompt", "prompt", 64, 4096, 129280),
        # Every rule on a toy batch, in place: launch latency counts.
        _process("rules_small", 4, 4, 1000, "f32", True, False, 40, 20, 4, 50),
        # The target logits of a serving batch before verification, in place:
        # scheduled lengths, long histories, a quarter of the rows under a grammar.
        _process("rules_batch", 256, 8, 129280, "bf16", True, True, 2000, 800, 16, 25),
        # Plain decoding (no drafts) under grammars, a vocabulary that is no
        # multiple of anything, so that no two vectors are aligned alike.
        _process("rules_decode", 33, 0, 50001, "bf16", True, False, 500, 300, 0, 100),
        # Raw logits kept for reporting: the processed ones go to a second buffer.
        _process("rules_copy", 64, 4, 129280, "bf16", False, False, 1000, 500, 8, 25),
        # Long draft blocks in fp32, kept raw, with long answers behind them.
        _process("rules_wide", 128, 16, 129280, "f32", False, True, 4000, 4000, 32, 10),
        # One token of one request: the head is a matrix-vector product.
        _head("head_single", 1, 1, 4096, 129280, 128, False, "bf16", "bf16", False),
        # One request's block of eight drafts and the position after them.
        _head("head_block", 1, 9, 4096, 129280, 64, True, "f32", "bf16", False),
        # A serving batch, positions past the scheduled length pruned.
        _head("head_batch", 64, 5, 4096, 129280, 128, False, "bf16", "bf16", True),
        # A small drafter's head, odd everywhere.
        _head("head_odd", 3, 5, 1120, 10007, 32, True, "f32", "f32", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    # the plain forms pass over [B, P, V] or [V, H] whatever the rules leave out
    dense = (case["B"] * (case["K"] + 1) * case["V"] if case["op"] == "process" else
             case["V"] * case["H"] if case["op"] == "head" else case["B"] * case["V"])
    return w["bytes"], w["flops"], dense


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = tuple(max(a, b) for a, b in zip(top.get(c["op"], (0, 0, 0)), _cost(c)))
    while True:
        op = rng.choice(["history", "process", "process", "head", "head"])
        V = _log(rng, 1000, 160000)
        if op == "history":
            if rng.random() < 0.5:
                c = _history("", "output", _log(rng, 1, 300), rng.randint(1, 17), V)
            else:
                c = _history("", "prompt", _log(rng, 1, 64), _log(rng, 16, 4096), V)
        elif op == "process":
            c = _process("", _log(rng, 1, 256), rng.choice([0, 1, 2, 3, 4, 5, 8, 11, 16]), V,
                         rng.choice(["f32", "bf16"]), rng.random() < 0.5, rng.random() < 0.5,
                         _log(rng, 10, 4000), _log(rng, 10, 4000), rng.choice([0, 1, 7, 32]),
                         rng.choice([0, 10, 25, 50, 100]))
        else:
            group = rng.choice([32, 64, 128])
            c = _head("", _log(rng, 1, 64), rng.randint(1, 9), group * _log(rng, 4, 64), V, group,
                      rng.random() < 0.5, rng.choice(["f32", "bf16"]),
                      rng.choice(["f32", "bf16"]), rng.random() < 0.5)
        del c["name"]
        if all(a <= b for a, b in zip(_cost(c), top[op])):
            return c


# ---------------------------------------------------------------------------
# Inputs.
# ---------------------------------------------------------------------------
def _tokens(g, shape, V):
    """Token ids with the head-heavy frequencies of text: P(id < n) ~ log n."""
    u = torch.rand(shape, generator=g, device=DEV, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1)) - 1).long().clamp_(0, V - 1).int()


def _pack(flags):
    """[..., V] truth values as [..., ceil(V / 32)] words, bit v % 32 of word v // 32."""
    V = flags.shape[-1]
    flags = torch.nn.functional.pad(flags, (0, -V % 32)).unflatten(-1, (-1, 32))
    weight = 1 << torch.arange(32, device=flags.device)
    words = (flags * weight).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).int()


def _unpack(words, V):
    bits = words.unsqueeze(-1) >> torch.arange(32, device=words.device, dtype=torch.int32) & 1
    return bits.flatten(-2)[..., :V].bool()


def _lengths(g, B, K, ragged):
    if ragged:
        return torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    return torch.full((B,), K, device=DEV, dtype=torch.int32)


def _request_state(g, B, V, prompt, output):
    """The history of B requests after `prompt` and `output` tokens."""
    p, o = _tokens(g, (B, prompt), V).long(), _tokens(g, (B, output), V).long()
    seen = torch.zeros(B, V, dtype=torch.bool, device=DEV).scatter_(1, p, True)
    counts = torch.zeros(B, V, dtype=torch.int32, device=DEV)
    counts.scatter_add_(1, o, torch.ones_like(o, dtype=torch.int32))
    return dict(prompt_bits=_pack(seen), output_bits=_pack(counts > 0), output_counts=counts)


def _prepare_history(c, g):
    B, S, V = c["B"], c["S"], c["V"]
    s = _request_state(g, B, V, 200, 100)
    tokens = _tokens(g, (B, S), V)
    if c["kind"] == "output":       # what verification returns: -1 behind the emitted tokens
        n = torch.randint(-1, S, (B,), generator=g, device=DEV, dtype=torch.int32)
        at = torch.arange(S, device=DEV)
        s["tokens"] = torch.where(at <= n[:, None], tokens, -1)
        s["lens"] = n
    else:
        s["tokens"] = tokens
        s["lens"] = torch.randint(max(1, S // 4), S + 1, (B,), generator=g, device=DEV,
                                  dtype=torch.int32)
    return s


def _prepare_process(c, g):
    B, K, V, P = c["B"], c["K"], c["V"], c["K"] + 1
    dt = DTYPES[c["dtype"]]
    s = _request_state(g, B, V, c["prompt"], c["output"])
    s["logits"] = torch.empty(B, P, V, dtype=dt, device=DEV).normal_(0.0, 3.0, generator=g)
    s["out"] = s["logits"] if c["in_place"] else torch.zeros_like(s["logits"])
    s["drafts"] = _tokens(g, (B, K), V) if K else None
    s["lengths"] = _lengths(g, B, K, c["ragged"])
    u = torch.rand(3, B, generator=g, device=DEV)
    s["repetition"], s["frequency"], s["presence"] = 1.0 + 0.3 * u[0], 0.5 * u[1], 0.5 * u[2]
    s["bias_begin"] = s["bias_tokens"] = s["bias_values"] = None
    if c["bias"]:
        n = c["bias"]
        first = torch.randint(0, V, (B, 1), generator=g, device=DEV)
        step = max(1, V // n)
        s["bias_tokens"] = ((first + step * torch.arange(n, device=DEV)) % V).int().flatten()
        s["bias_values"] = 4.0 * torch.randn(B * n, generator=g, device=DEV)
        s["bias_begin"] = torch.arange(0, B * n + 1, n, device=DEV, dtype=torch.int32)
    s["mask"] = s["mask_index"] = None
    rows = B * c["grammar"] // 100
    if rows:
        # inside a text field nearly every token is allowed, at a structural place a few
        share = torch.where(torch.rand(rows * P, 1, generator=g, device=DEV) < 0.5, 0.95, 0.002)
        allowed = torch.rand(rows * P, V, generator=g, device=DEV) < share
        allowed.scatter_(1, torch.randint(0, V, (rows * P, 4), generator=g, device=DEV), True)
        s["mask"] = _pack(allowed)
        s["mask_index"] = torch.full((B, P), -1, device=DEV, dtype=torch.int32)
        which = torch.randperm(B, generator=g, device=DEV)[:rows]
        s["mask_index"][which] = torch.arange(rows * P, device=DEV, dtype=torch.int32).view(rows, P)
    return s


def _prepare_head(c, g):
    B, P, H, V, G = c["B"], c["P"], c["H"], c["V"], c["H"] // c["group"]
    s = {}
    s["x"] = torch.empty(B, P, H, dtype=torch.bfloat16, device=DEV).normal_(0.0, 1.0, generator=g)
    s["codes"] = torch.randint(0, 256, (V, H // 2), generator=g, device=DEV, dtype=torch.uint8)
    s["scale"] = (torch.rand(V, G, generator=g, device=DEV).add_(0.5).mul_(0.2 / math.sqrt(H))
                  .to(DTYPES[c["scale"]]))
    s["zero"] = (torch.randint(5, 11, (V, G), generator=g, device=DEV, dtype=torch.uint8)
                 if c["zero"] else None)
    s["lengths"] = _lengths(g, B, P - 1, c["ragged"])
    s["out"] = torch.zeros(B, P, V, dtype=DTYPES[c["out"]], device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    make = {"history": _prepare_history, "process": _prepare_process, "head": _prepare_head}
    s = make[case["op"]](case, g)
    s["case"] = case
    if own:      # the descriptors that a serving loop keeps beside its buffers
        import speculative_decoding_verification_93_b200 as sv
        s["sv"] = sv
        if case["op"] != "head":
            s["history"] = sv.TokenHistory(case["V"], s["prompt_bits"], s["output_bits"],
                                           s["output_counts"])
        if case["op"] == "process":
            s["rules"] = sv.LogitRules(
                history=s["history"], repetition=s["repetition"], frequency=s["frequency"],
                presence=s["presence"], bias_begin=s["bias_begin"], bias_tokens=s["bias_tokens"],
                bias_values=s["bias_values"], mask=s["mask"], mask_index=s["mask_index"])
        if case["op"] == "head":
            s["weight"] = sv.W4Weight(s["codes"], s["scale"], s["zero"])
            n = sv.sv_head_w4_workspace_bytes(s["weight"], case["B"], case["P"])
            s["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# One pass.
# ---------------------------------------------------------------------------
def _plain_history(s, c):
    V, output = c["V"], c["kind"] == "output"
    lens = s["lens"] + 1 if output else s["lens"]
    valid = torch.arange(c["S"], device=DEV) < lens[:, None]
    token = torch.where(valid, s["tokens"], 0).long()
    if not output:
        seen = _unpack(s["prompt_bits"], V).int().scatter_add_(1, token, valid.int())
        s["prompt_bits"].copy_(_pack(seen > 0))
        return s["prompt_bits"]
    s["output_counts"].scatter_add_(1, token, valid.int())
    s["output_bits"].copy_(_pack(s["output_counts"] > 0))
    return s["output_bits"], s["output_counts"]


def _plain_process(s, c):
    B, K, V, P = c["B"], c["K"], c["V"], c["K"] + 1
    z = s["logits"].float()
    count = torch.zeros(B, P, V, dtype=torch.int32, device=DEV)
    if K:            # drafts 0 .. i-1 stand before position i
        at = s["drafts"].long().unsqueeze(-1)
        count[:, 1:].scatter_(2, at, 1)
        count = count.cumsum(1, dtype=torch.int32)
    count += s["output_counts"][:, None]
    seen = (count > 0) | _unpack(s["prompt_bits"], V)[:, None]
    by_row = lambda t: t.view(B, 1, 1)  # noqa: E731
    rep = by_row(s["repetition"])
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - by_row(s["frequency"]) * count - by_row(s["presence"]) * (count > 0)
    if c["bias"]:
        bias = torch.zeros(B, V, device=DEV)
        bias.scatter_(1, s["bias_tokens"].view(B, -1).long(), s["bias_values"].view(B, -1))
        z = z + bias[:, None]
    if s["mask"] is not None:
        index = s["mask_index"].flatten().long()
        free = (index < 0)[:, None]
        allowed = _unpack(s["mask"], V)[index.clamp(min=0)] | free
        z = torch.where(allowed.view(B, P, V), z, -math.inf)
    live = torch.arange(P, device=DEV) <= s["lengths"][:, None]
    s["out"].copy_(torch.where(live.unsqueeze(-1), z.to(s["out"].dtype), s["out"]))
    return s["out"]


def _plain_head(s, c):
    B, P, H, V, group = c["B"], c["P"], c["H"], c["V"], c["group"]
    code = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(V, H // group, group).float()
    zero = s["zero"].float().unsqueeze(-1) if s["zero"] is not None else 8.0
    w = ((code - zero) * s["scale"].float().unsqueeze(-1)).view(V, H)
    z = (s["x"].float().view(B * P, H) @ w.t()).view(B, P, V).to(s["out"].dtype)
    live = torch.arange(P, device=DEV) <= s["lengths"][:, None]
    s["out"].copy_(torch.where(live.unsqueeze(-1), z, s["out"]))
    return s["out"]


def run(state):
    s, c = state, state["case"]
    if not own:
        form = {"history": _plain_history, "process": _plain_process, "head": _plain_head}
        return form[c["op"]](s, c)
    sv = s["sv"]
    if c["op"] == "history":
        if c["kind"] == "prompt":
            sv.sv_history_add(s["history"], s["tokens"], s["lens"], sv.SV_HISTORY_PROMPT)
            return s["prompt_bits"]
        sv.sv_history_add(s["history"], s["tokens"], s["lens"], sv.SV_HISTORY_OUTPUT, extra=1)
        return s["output_bits"], s["output_counts"]
    if c["op"] == "process":
        sv.sv_logits_process(s["logits"], s["out"], s["rules"], draft_tokens=s["drafts"],
                             lengths=s["lengths"], extra=1)
        return s["out"]
    sv.sv_head_w4(s["weight"], s["x"], s["out"], s["workspace"], lengths=s["lengths"], extra=1)
    return s["out"]


# ---------------------------------------------------------------------------
# What a pass cannot do without.
# ---------------------------------------------------------------------------
def _distinct(n, V):
    """Expected distinct ids among n of _tokens(): sum over v of 1 - (1 - p_v)^n."""
    L = math.log(V + 1)
    return sum(-math.expm1(-n * math.log((v + 2) / (v + 1)) / L) *
               (1 if v < 64 else max(1, v // 32)) for v in _grid(V))


def _grid(V):
    """0 .. 63, then every (v // 32)-th id: the terms change slowly there."""
    v, out = 0, []
    while v < V:
        out.append(v)
        v += 1 if v < 64 else max(1, v // 32)
    return out


def work(case):
    c, B, V = case, case["B"], case["V"]
    W = -(-V // 32)
    if c["op"] == "history":
        n = B * c["S"] * (0.625 if c["kind"] == "prompt" else 0.5)
        d = min(n, B * _distinct(n / B, V))
        # the tokens, and a read and a write of each word they touch
        return {"bytes": 4 * n + 4 * B + d * (8 if c["kind"] == "prompt" else 16), "flops": n}
    if c["op"] == "process":
        K, P, e = c["K"], c["K"] + 1, 4 if c["dtype"] == "f32" else 2
        pos = B * (K / 2 + 1 if c["ragged"] else P)
        rows = B * c["grammar"] // 100
        masked = pos * rows / B
        seen = min(V, _distinct(c["prompt"] + c["output"], V) + c["bias"])
        bits = B * 2 * W * 4 + masked * W * 4 + B * (_distinct(c["output"], V) * 4 + c["bias"] * 8)
        touched = pos * seen
        if c["in_place"]:      # the touched logits read and written, the forbidden ones written
            logits = 2 * touched * e + masked * V * (0.5 * 0.05 + 0.5 * 0.998) * e
        else:
            logits = 2 * pos * V * e
        return {"bytes": bits + logits, "flops": 6 * touched}
    H, G, e = c["H"], c["H"] // c["group"], 4 if c["out"] == "f32" else 2
    pos = c["B"] * ((c["P"] + 1) / 2 if c["ragged"] else c["P"])
    weight = V * (H / 2 + G * ((4 if c["scale"] == "f32" else 2) + (1 if c["zero"] else 0)))
    return {"bytes": weight + pos * (2 * H + V * e), "flops": 2 * pos * V * H}


# ---------------------------------------------------------------------------
# The result in 64 bits, row by row from the definitions.
# ---------------------------------------------------------------------------
def _allowed(words, V):
    v = torch.arange(V, device=DEV)
    return (words[v // 32].long() >> (v % 32)) % 2 != 0


def _exact_process(c, s):
    out = s["out"].double()
    for b in range(c["B"]):
        said = s["output_counts"][b].double()
        before = _allowed(s["prompt_bits"][b], c["V"])
        rep, freq, pres = (s[k][b].double() for k in ("repetition", "frequency", "presence"))
        bias = torch.zeros(c["V"], dtype=torch.float64, device=DEV)
        if c["bias"]:
            lo, hi = s["bias_begin"][b:b + 2].tolist()
            bias.index_put_((s["bias_tokens"][lo:hi].long(),), s["bias_values"][lo:hi].double())
        index = [-1] * (c["K"] + 1) if s["mask"] is None else s["mask_index"][b].tolist()
        for i in range(int(s["lengths"][b]) + 1):
            if i:
                said[s["drafts"][b, i - 1].long()] += 1.0
            z = s["logits"][b, i].double()
            factor = torch.where(z > 0, 1.0 / rep, rep)
            z = z * torch.where(before | (said > 0), factor, 1.0)
            z = z - (freq * said + pres * (said > 0)) + bias
            if index[i] >= 0:
                z[~_allowed(s["mask"][index[i]], c["V"])] = -math.inf
            out[b, i] = z
    return out


def _exact_head(c, s):
    B, P, H, V, n = c["B"], c["P"], c["H"], c["V"], c["group"]
    x = s["x"].double().view(B * P, H)
    total = torch.zeros(B * P, V, dtype=torch.float64, device=DEV)
    for j in range(H // n):          # scale * (sum of x * code - zero * sum of x), by group
        part = s["codes"][:, j * n // 2:(j + 1) * n // 2].double()
        high = torch.floor(part / 16)
        even, odd = x[:, j * n:(j + 1) * n:2], x[:, j * n + 1:(j + 1) * n:2]
        dot = even @ (part - 16 * high).t() + odd @ high.t()
        zero = s["zero"][:, j].double() if s["zero"] is not None else 8.0
        total += s["scale"][:, j].double() * (dot - zero * (even + odd).sum(1, keepdim=True))
    out = s["out"].double()
    for b in range(B):
        n = int(s["lengths"][b]) + 1
        out[b, :n] = total.view(B, P, V)[b, :n]
    return out


def exact(case, seed):
    if case["op"] == "history":
        return None
    s = prepare(case, seed)
    return _exact_process(case, s) if case["op"] == "process" else _exact_head(case, s)
