"""Measured cases of the operators between and behind the layers of a serving step: the
root-mean-square norm (with the residual's addition or a gate, into 16 or 8 bits), products with
4-bit weights, token probabilities and the verification of drafted tokens.

`run` makes one pass: with `own` false in elementary torch operations (the plain form), with `own`
true through the package's entry points. `exact` computes the same outputs in 64 bits, written apart
from the plain form.
"""
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1}


# ---------------------------------------------------------------------------
# cases

def listed():
    return [
        # One token of one request between two layers: the residual stream takes a layer's output
        # in and is normed for the next. Latency alone.
        dict(name="norm_token_one", op="norm", rows=1, hidden=2560, groups=1, mode="add",
             dtype="bf16", residual="bf16", out="bf16", weight=True),
        # A layer prompt's rows, the residual stream in 32 bits.
        dict(name="norm_prompt_layer", op="norm", rows=4096, hidden=2560, groups=1, mode="add",
             dtype="bf16", residual="f32", out="bf16", weight=True),
        # The gated norm behind the scan of a verify step: 128 requests of 3 tokens, 8 groups, the
        # gate a slice of the input projection's rows.
        dict(name="norm_gated_verify", op="norm", rows=384, hidden=8192, groups=8, mode="gate",
             dtype="bf16", residual="bf16", out="bf16", weight=True),
        # One token through a Mamba2 layer's input projection (80 heads of 64, one group of 128).
        dict(name="linear_token_one", op="linear", tokens=1, k=2560, n=10576, x="bf16",
             out="bf16", bias=False),
        # A small ragged batch: odd sizes, 8-bit rows in, 32 bits out, a bias.
        dict(name="linear_few_ragged", op="linear", tokens=77, k=1056, n=1111, x="e4m3",
             out="f32", bias=True),
        # The layer prompt's input projection in bf16.
        dict(name="linear_prompt_layer", op="linear", tokens=4096, k=2560, n=10576, x="bf16",
             out="bf16", bias=False),
        # The layer prompt's output projection, 8-bit rows.
        dict(name="linear_prompt_8bit", op="linear", tokens=4096, k=5120, n=2560, x="e4m3",
             out="bf16", bias=False),
        # A verify step's way into a layer: add, norm into 8 bits, input projection (128 heads of
        # 64, 8 groups of 128).
        dict(name="norm_linear_verify", op="chain", rows=384, hidden=4096, n=18560, dtype="bf16",
             residual="bf16", out="bf16"),
        # One request's next token: one row of logits in 32 bits.
        dict(name="probs_token_one", op="probs", reqs=1, tokens=1, vocab=50257, dtype="f32"),
        # The verify step's logits, a temperature a request, some of them greedy.
        dict(name="probs_verify", op="probs", reqs=128, tokens=3, vocab=131072, dtype="bf16"),
        # One request whose drafts were copied from its prompt: no draft probabilities.
        dict(name="verify_one", op="verify", reqs=1, tokens=6, vocab=50257, draft_probs=False,
             ragged=False),
        # The verify step of 128 requests with two drafts each, some requests with fewer.
        dict(name="verify_batch", op="verify", reqs=128, tokens=3, vocab=131072,
             draft_probs=True, ragged=True),
    ]


def spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "chain", "probs", "verify",
                     "verify"])
    if op == "norm":
        rows = spread(rng, 1, 8192)
        hidden = spread(rng, 16, min(16384, (1 << 24) // rows))
        groups = rng.choice([1, 1, 2, 4, 8])
        return dict(op=op, rows=rows, hidden=max(1, hidden // groups) * groups, groups=groups,
                    mode=rng.choice(["add", "add", "gate", "plain"]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    weight=rng.random() < 0.8)
    if op == "linear":
        tokens = spread(rng, 1, 4096)
        k = 32 * spread(rng, 1, 256)
        most = min(4096 * 2560 * 10576 // (tokens * k), (80 << 20) // k, (40 << 20) // tokens)
        return dict(op=op, tokens=tokens, k=k, n=spread(rng, 1, min(20000, most)),
                    x=rng.choice(["bf16", "e4m3"]), out=rng.choice(["bf16", "bf16", "f32"]),
                    bias=rng.random() < 0.3)
    if op == "chain":
        rows, hidden = spread(rng, 1, 1024), 32 * spread(rng, 4, 160)
        return dict(op=op, rows=rows, hidden=hidden, n=spread(rng, 16, 18560), dtype="bf16",
                    residual=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
    tokens, reqs = rng.randint(1, 8), spread(rng, 1, 128)
    vocab = spread(rng, 100, min(160000, (36 << 20) // (reqs * tokens)))
    if op == "probs":
        return dict(op=op, reqs=reqs, tokens=tokens, vocab=vocab,
                    dtype=rng.choice(["bf16", "f32"]))
    return dict(op=op, reqs=reqs, tokens=tokens, vocab=vocab, draft_probs=rng.random() < 0.6,
                ragged=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# what a user's program has in hand before the call

def prepare(case, seed):
    return globals()["_prepare_" + case["op"]](case, torch.Generator(DEV).manual_seed(seed))


def _normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _stream_rows(g, rows, hidden, dtype):
    """Rows of a residual stream: a few channels far larger than the others."""
    wide = torch.exp(_normal(g, hidden, scale=0.5))
    wide[torch.rand(hidden, generator=g, device=DEV) < 0.01] *= 20
    return (_normal(g, rows, hidden) * wide).to(dtype)


def _prepare_norm(c, g):
    ti, rows, h = TYPES[c["dtype"]], c["rows"], c["hidden"]
    s = dict(case=c, residual=None, residual_out=None, gate=None, weight=None)
    s["x"] = _normal(g, rows, h, dtype=ti)
    if c["mode"] == "add":
        s["residual"] = _stream_rows(g, rows, h, TYPES[c["residual"]])
        s["residual_out"] = torch.empty_like(s["residual"])
    elif c["mode"] == "gate":
        # the gate is the first part of the input projection's rows, the scan's inputs follow
        s["gate"] = _normal(g, rows, 2 * h, dtype=ti)[:, :h]
    if c["weight"]:
        s["weight"] = 1 + _normal(g, h, scale=0.1)
    s["out"] = torch.empty(rows, h, dtype=TYPES[c["out"]], device=DEV)
    if own:
        import state_space_model_varlen_amd as ssd
        s["p"] = ssd.make_norm_problem(rows, h, ti, TYPES[c["out"]], groups=c["groups"],
                                       residual_dtype=TYPES[c["residual"]], eps=1e-5)
    return s


def _weights(g, n, k):
    """4-bit weights as a checkpoint holds them: random codes of a normal distribution's shape, an
    exponent byte for 32 of them."""
    w = torch.randn(n, k, generator=g, device=DEV, dtype=torch.bfloat16)
    code = torch.zeros(n, k, dtype=torch.uint8, device=DEV)
    for edge in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):        # between neighbours of 0 .. 6
        code += (w.abs() * 2 > edge)
    code += 8 * (w < 0)
    packed = code[:, 0::2] | (code[:, 1::2] << 4)               # even index in the low half
    e = 127 - round(0.5 * torch.log2(torch.tensor(float(k))).item())
    scale = torch.randint(e - 2, e + 1, (n, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    return packed, scale


def _prepare_linear(c, g):
    t, k, n = c["tokens"], c["k"], c["n"]
    s = dict(case=c, x_scale=None, bias=None)
    s["x"] = _normal(g, t, k, dtype=torch.bfloat16)
    if c["x"] == "e4m3":
        s["x"], s["x_scale"] = _encode(s["x"])
    s["weight"], s["weight_scale"] = _weights(g, n, k)
    if c["bias"]:
        s["bias"] = _normal(g, n, scale=0.1)
    s["out"] = torch.empty(t, n, dtype=TYPES[c["out"]], device=DEV)
    if own:
        import state_space_model_varlen_amd as ssd
        s["p"] = ssd.make_linear_problem(t, k, n, TYPES[c["x"]], TYPES[c["out"]])
        s["workspace"] = ssd.alloc_linear_workspace(s["p"], DEV)
    return s


def _prepare_chain(c, g):
    rows, h, n = c["rows"], c["hidden"], c["n"]
    s = dict(case=c, x=_normal(g, rows, h, dtype=torch.bfloat16),
             residual=_stream_rows(g, rows, h, TYPES[c["residual"]]),
             weight=1 + _normal(g, h, scale=0.1))
    s["residual_out"] = torch.empty_like(s["residual"])
    s["w"], s["w_scale"] = _weights(g, n, h)
    s["out"] = torch.empty(rows, n, dtype=TYPES[c["out"]], device=DEV)
    if own:
        import state_space_model_varlen_amd as ssd
        s["normed"] = torch.empty(rows, h, dtype=torch.float8_e4m3fn, device=DEV)
        s["normed_scale"] = torch.empty(rows, h // 32, dtype=torch.uint8, device=DEV)
        s["p"] = ssd.make_norm_problem(rows, h, torch.bfloat16, torch.float8_e4m3fn,
                                       residual_dtype=TYPES[c["residual"]], eps=1e-5)
        s["lp"] = ssd.make_linear_problem(rows, h, n, torch.float8_e4m3fn, TYPES[c["out"]])
        s["workspace"] = ssd.alloc_linear_workspace(s["lp"], DEV)
    return s


def _logits(g, rows, vocab):
    """Logits as a trained head gives them: most far below the few that matter."""
    x = _normal(g, rows, vocab, scale=2.0)
    top = torch.randint(0, vocab, (rows, 8), generator=g, device=DEV)
    return x.scatter_add_(1, top, 8 + _normal(g, rows, 8, scale=2.0))


def _prepare_probs(c, g):
    r, t, v = c["reqs"], c["tokens"], c["vocab"]
    s = dict(case=c, logits=_logits(g, r * t, v).to(TYPES[c["dtype"]]).view(r, t, v))
    temp = torch.tensor([1.0, 0.7, 0.0, 1.3], device=DEV)
    pick = torch.randint(0, 4, (r,), generator=g, device=DEV)
    s["temperature"] = temp[pick if r > 1 else pick % 2]
    s["probs"] = torch.empty(r, t, v, dtype=torch.float32, device=DEV)
    if own:
        import state_space_model_varlen_amd as ssd
        s["p"] = ssd.make_probs_problem(r, t, v, TYPES[c["dtype"]])
        s["workspace"] = ssd.alloc_probs_workspace(s["p"], DEV)
    return s


def _prepare_verify(c, g):
    r, t, v = c["reqs"], c["tokens"], c["vocab"]
    logits = _logits(g, r * t, v)
    s = dict(case=c, draft_probs=None, num_drafts=None)
    s["target"] = torch.softmax(logits, 1).view(r, t, v)
    # the draft model is a rougher version of the target; its tokens come from its probabilities
    logits += _normal(g, r * t, v, scale=0.7)
    q = torch.softmax(logits, 1).view(r, t, v)[:, :t - 1].contiguous()
    drafts = q if t > 1 else s["target"][:, :0]
    pick = torch.rand(r, t - 1, 1, generator=g, device=DEV, dtype=torch.float64)
    drafts = torch.searchsorted(drafts.double().cumsum(-1), pick)[..., 0].clamp(max=v - 1)
    s["drafts"] = drafts.to(torch.int32).contiguous()
    if c["draft_probs"]:
        s["draft_probs"] = q
    if c["ragged"]:
        s["num_drafts"] = torch.randint(0, t, (r,), generator=g, device=DEV, dtype=torch.int32)
    s["uniform"] = torch.rand(r, t, generator=g, device=DEV)
    s["accepted"] = torch.empty(r, dtype=torch.int32, device=DEV)
    s["tokens"] = torch.empty(r, t, dtype=torch.int32, device=DEV)
    if own:
        import state_space_model_varlen_amd as ssd
        s["p"] = ssd.make_verify_problem(r, t, v)
        s["workspace"] = ssd.alloc_verify_workspace(s["p"], DEV)
    return s


# ---------------------------------------------------------------------------
# one pass

def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_norm(s):
    import state_space_model_varlen_amd as ssd
    ssd.rms_norm(s["p"], s["x"], s["weight"], s["out"], residual=s["residual"],
                 residual_out=s["residual_out"], gate=s["gate"])
    return _norm_result(s)


def _norm_result(s):
    if s["residual"] is None:
        return {"out": s["out"]}
    return {"out": s["out"], "residual": s["residual_out"]}


def _own_linear(s):
    import state_space_model_varlen_amd as ssd
    ssd.linear_w4(s["p"], s["x"], s["weight"], s["weight_scale"], s["out"], x_scale=s["x_scale"],
                  bias=s["bias"], workspace=s["workspace"])
    return {"out": s["out"]}


def _own_chain(s):
    import state_space_model_varlen_amd as ssd
    ssd.rms_norm(s["p"], s["x"], s["weight"], s["normed"], residual=s["residual"],
                 residual_out=s["residual_out"], out_scale=s["normed_scale"])
    ssd.linear_w4(s["lp"], s["normed"], s["w"], s["w_scale"], s["out"],
                  x_scale=s["normed_scale"], workspace=s["workspace"])
    return {"out": s["out"], "residual": s["residual_out"]}


def _own_probs(s):
    import state_space_model_varlen_amd as ssd
    ssd.token_probs(s["p"], s["logits"], s["temperature"], s["probs"], workspace=s["workspace"])
    return {"probs": s["probs"]}


def _own_verify(s):
    import state_space_model_varlen_amd as ssd
    ssd.verify_drafts(s["p"], s["target"], s["draft_probs"], s["drafts"], s["num_drafts"],
                      s["uniform"], s["accepted"], s["tokens"], workspace=s["workspace"])
    return {"accepted": s["accepted"], "tokens": s["tokens"]}


def _plain_normed(x, gate, residual, residual_out, weight, groups):
    v = x.float()
    if gate is not None:
        z = gate.float()
        v = v * (z * torch.sigmoid(z))
    if residual is not None:
        v = v + residual.float()
        residual_out.copy_(v)
    v = v.unflatten(1, (groups, -1))
    v = (v * torch.rsqrt(v.square().mean(-1, keepdim=True) + 1e-5)).flatten(1)
    return v if weight is None else v * weight


def _plain_norm(s):
    s["out"].copy_(_plain_normed(s["x"], s["gate"], s["residual"], s["residual_out"], s["weight"],
                                 s["case"]["groups"]))
    return _norm_result(s)


def _power(e):
    """2 ** e of whole e in [-126, 127], from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x):
    """Rows in 8 bits: codes, and for 32 of them the exponent byte of the least power of two of
    which none is more than 448 times."""
    x = x.float().unflatten(1, (-1, 32))
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -126).clamp(-126, 127)
    return ((x * _power(-e)[..., None]).to(torch.float8_e4m3fn).flatten(1),
            (e + 127).to(torch.uint8))


def _decoded(x, scale):
    if scale is None:
        return x.float()
    return (x.float().unflatten(1, (-1, 32)) * _power(scale.int() - 127)[..., None]).flatten(1)


def _plain_product(x, packed, scale):
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    value = torch.cat([value, -value])
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(1)
    w = (value[codes.int()].unflatten(1, (-1, 32)) * _power(scale.int() - 127)[..., None]).flatten(1)
    return torch.matmul(x, w.t())


def _plain_linear(s):
    y = _plain_product(_decoded(s["x"], s["x_scale"]), s["weight"], s["weight_scale"])
    s["out"].copy_(y if s["bias"] is None else y + s["bias"])
    return {"out": s["out"]}


def _plain_chain(s):
    v = _plain_normed(s["x"], None, s["residual"], s["residual_out"], s["weight"], 1)
    s["out"].copy_(_plain_product(_decoded(*_encode(v)), s["w"], s["w_scale"]))
    return {"out": s["out"], "residual": s["residual_out"]}


def _plain_probs(s):
    x, t = s["logits"].float(), s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    e = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    e = e / e.sum(-1, keepdim=True)
    # temperature 0: all of it on the first of the largest
    place = torch.arange(x.shape[-1], device=DEV)
    first = torch.where(x == top, place, x.shape[-1]).amin(-1, keepdim=True)
    torch.where(t > 0, e, (place == first).float(), out=s["probs"])
    return {"probs": s["probs"]}


def _plain_verify(s):
    c, p, q, d = s["case"], s["target"], s["draft_probs"], s["drafts"].long()
    r, t, v = c["reqs"], c["tokens"], c["vocab"]
    u = s["uniform"].double()
    count = (torch.full((r,), t - 1, device=DEV) if s["num_drafts"] is None
             else s["num_drafts"].long())
    pd = p[:, :t - 1].gather(2, d[..., None])[..., 0].double()
    qd = torch.ones_like(pd) if q is None else q.gather(2, d[..., None])[..., 0].double()
    place = torch.arange(t - 1, device=DEV)
    ok = (u[:, :t - 1] * qd < pd) & (place < count[:, None])
    acc = ok.long().cumprod(1).sum(1)                                   # [r]
    row = torch.arange(r, device=DEV)
    w = p[row, acc].double()
    cut = torch.nonzero(acc < count)[:, 0]                              # a draft was turned down
    if t > 1:
        if q is None:
            w[cut, d[cut, acc[cut]]] = 0
        else:
            w[cut] = (w[cut] - q[cut, acc[cut]].double()).clamp(min=0)
    left = w.sum(1, keepdim=True) > 0                                   # nothing left: p itself
    w = torch.where(left, w, p[row, acc].double())
    cdf = w.cumsum(1)
    new = (cdf <= u[:, t - 1:] * cdf[:, -1:]).sum(1).clamp(max=v - 1)
    place = torch.arange(t, device=DEV)
    tokens = torch.cat([d, new[:, None]], 1)
    tokens = torch.where(place == acc[:, None], new[:, None], tokens)
    s["tokens"].copy_(torch.where(place > acc[:, None], -1, tokens))
    s["accepted"].copy_(acc)
    return {"accepted": s["accepted"], "tokens": s["tokens"]}


# ---------------------------------------------------------------------------
# bytes and operations that a pass cannot do without

def work(case):
    c, op = case, case["op"]
    if op == "norm":
        e, h = BYTES[c["dtype"]], c["hidden"]
        per = e + BYTES[c["out"]]
        per += {"add": 2 * BYTES[c["residual"]], "gate": e, "plain": 0}[c["mode"]]
        return {"bytes": c["rows"] * h * per + (4 * h if c["weight"] else 0),
                "flops": c["rows"] * h * (8 if c["mode"] == "gate" else 5)}
    if op in ("linear", "chain"):
        t, k = (c["tokens"], c["k"]) if op == "linear" else (c["rows"], c["hidden"])
        n = c["n"]
        b, f = n * k // 2 + n * k // 32 + t * n * BYTES[c["out"]], 2 * t * k * n
        if op == "linear":
            b += t * k * BYTES[c["x"]] + (t * k // 32 if c["x"] == "e4m3" else 0)
            return {"bytes": b + (4 * n if c["bias"] else 0), "flops": f}
        # the normed rows stay inside the pass
        return {"bytes": b + t * k * (2 + 2 * BYTES[c["residual"]]) + 4 * k, "flops": f + 6 * t * k}
    rows, v = c["reqs"] * c["tokens"], c["vocab"]
    if op == "probs":
        return {"bytes": rows * v * (BYTES[c["dtype"]] + 4), "flops": 4 * rows * v}
    # one row of each request is summed up (two, where drafts have probabilities)
    return {"bytes": c["reqs"] * v * 4 * (2 if c["draft_probs"] and c["tokens"] > 1 else 1),
            "flops": 3 * c["reqs"] * v}


# ---------------------------------------------------------------------------
# the same outputs in 64 bits

def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))


def _exact_rows(s, groups):
    v = s["x"].double()
    if s.get("gate") is not None:
        v = v * s["gate"].double() / (1 + torch.exp(-s["gate"].double()))
    if s["residual"] is not None:
        v = v + s["residual"].double()
    total, out = v.clone(), torch.empty_like(v)
    per = v.shape[1] // groups
    for i in range(groups):
        part = v[:, i * per:(i + 1) * per]
        out[:, i * per:(i + 1) * per] = part / torch.sqrt((part ** 2).sum(1, keepdim=True) / per
                                                          + 1e-5)
    if s["weight"] is not None:
        out *= s["weight"].double()
    return out, total


def _exact_norm(s):
    out, total = _exact_rows(s, s["case"]["groups"])
    return {"out": out} if s["residual"] is None else {"out": out, "residual": total}


def _exact_product(x, packed, scale):
    """x [t, k] in 64 bits; two magnitude bits above a half: 0, 1/2, then 1 + m/2 times 2^(e-1)."""
    out = torch.empty(x.shape[0], packed.shape[0], dtype=torch.float64, device=DEV)
    for a in range(0, packed.shape[0], 4096):
        pk = packed[a:a + 4096].int()
        w = torch.empty(pk.shape[0], 2 * pk.shape[1], dtype=torch.float64, device=DEV)
        for half in (0, 1):
            code = (pk >> (4 * half)) & 15
            e, m = (code >> 1) & 3, (code & 1).double()
            size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
            w[:, half::2] = torch.where(code >= 8, -size, size)
        w *= torch.exp2(scale[a:a + 4096].double() - 127).repeat_interleave(32, 1)
        out[:, a:a + 4096] = x @ w.t()
    return out


def _exact_linear(s):
    x = s["x"].double()
    if s["x_scale"] is not None:
        x = x * torch.exp2(s["x_scale"].double() - 127).repeat_interleave(32, 1)
    y = _exact_product(x, s["weight"], s["weight_scale"])
    return {"out": y if s["bias"] is None else y + s["bias"].double()}


def _exact_chain(s):
    v, total = _exact_rows(s, 1)
    # least power of two whose 448-fold reaches the 32 values; then 3 bits after the leading one
    b = v.unflatten(1, (-1, 32))
    unit = torch.exp2(torch.ceil(torch.log2(b.abs().amax(-1, keepdim=True) / 448)))
    lead = torch.floor(torch.log2((b / unit).abs())).clamp(min=-6)
    b = torch.round(b / unit / torch.exp2(lead - 3)) * torch.exp2(lead - 3) * unit
    return {"out": _exact_product(b.flatten(1), s["w"], s["w_scale"]), "residual": total}


def _exact_probs(s):
    out = torch.empty(s["probs"].shape, dtype=torch.float64, device=DEV)
    for i, t in enumerate(s["temperature"].double().tolist()):
        x = s["logits"][i].double()
        if t > 0:
            out[i] = torch.softmax(x / t, -1)
        else:
            out[i] = 0
            for j, row in enumerate(x):
                out[i, j, torch.nonzero(row == row.max())[0, 0]] = 1
    return {"probs": out}


def _exact_verify(s):
    c, u = s["case"], s["uniform"].double().tolist()
    accepted, tokens = [], []
    for i in range(c["reqs"]):
        count = c["tokens"] - 1 if s["num_drafts"] is None else int(s["num_drafts"][i])
        drafts, got = s["drafts"][i].tolist(), []
        weights = None
        for j in range(count):
            p = s["target"][i, j].double()
            if s["draft_probs"] is None:
                q = torch.zeros_like(p)
                q[drafts[j]] = 1
            else:
                q = s["draft_probs"][i, j].double()
            if u[i][j] * float(q[drafts[j]]) < float(p[drafts[j]]):
                got.append(drafts[j])
                continue
            weights = torch.where(p > q, p - q, 0.0)
            if not bool((weights > 0).any()):
                weights = p
            break
        accepted.append(len(got))
        if weights is None:
            weights = s["target"][i, count].double()
        line = torch.cumsum(weights, 0)
        at = torch.searchsorted(line, line[-1:] * u[i][-1], right=True)
        got.append(min(int(at), c["vocab"] - 1))
        tokens.append(got + [-1] * (c["tokens"] - len(got)))
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device=DEV),
            "tokens": torch.tensor(tokens, dtype=torch.int32, device=DEV)}
