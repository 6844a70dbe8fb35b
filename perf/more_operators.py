"""The operators around a selective state space mixer and a model's input, as they are measured.

Three operators: the selective state space scan ("ssm"), the short causal convolution
in front of it ("conv") and the embedding lookup ("embed").  Each is here in its plain form
(elementary torch operations in 32 bits), as a user calls it from the package (`own`), and
in 64 bits from its definition (`exact`).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- the cases ---
def ssm_case(mode, batch, length, d, n, groups, dtype, gate, packed, ragged):
    """mode: train, prompt (forward with the final state) or step (one token on a state).  packed: several sequences in a row,
    marked by their starts; ragged: rows of different lengths."""
    return dict(op="ssm", mode=mode, batch=batch, length=length, d=d, n=n, groups=groups, dtype=dtype, gate=gate, packed=packed, ragged=ragged)


def conv_case(mode, batch, length, d, width, dtype, silu, packed, state):
    """state: inputs from before the first token are given, and their gradient asked for in training."""
    return dict(op="conv", mode=mode, batch=batch, length=length, d=d, width=width, dtype=dtype, silu=silu, packed=packed, state=state)


def embed_case(tokens, d, vocab, weight, out, zipf, train):
    """zipf: the frequencies of a text's tokens, else all alike."""
    return dict(op="embed", tokens=tokens, d=d, vocab=vocab, weight=weight, out=out, zipf=zipf, train=train)


def listed():
    return [
        # one decoding step of 16 sequences: launch latency
        dict(ssm_case("step", 16, 1, 2048, 16, 1, "bf16", True, False, False), name="ssm_token"),
        # prompts of 4 requests of different lengths, padded to 1024 tokens
        dict(ssm_case("prompt", 4, 1024, 2048, 16, 1, "bf16", True, False, True), name="ssm_prompt"),
        # odd sizes in 32 bits, packed sequences, no gate
        dict(ssm_case("train", 3, 777, 1537, 13, 1, "f32", False, True, False), name="ssm_odd"),
        # two training sequences of 2048 tokens
        dict(ssm_case("train", 2, 2048, 2048, 16, 1, "bf16", True, False, False), name="ssm_train"),
        # one row of 32768 tokens, packed
        dict(ssm_case("train", 1, 32768, 2048, 16, 1, "bf16", True, True, False), name="ssm_long"),
        # one decoding step of 16 sequences: launch latency
        dict(conv_case("step", 16, 1, 2048, 4, "bf16", True, False, True), name="conv_token"),
        # two training sequences of 2048 tokens
        dict(conv_case("train", 2, 2048, 2048, 4, "bf16", True, False, False), name="conv_train"),
        # an odd width in 32 bits, packed sequences that go on from a state
        dict(conv_case("train", 3, 777, 1537, 3, "f32", False, True, True), name="conv_odd"),
        # one row of 32768 tokens at width 2560, packed
        dict(conv_case("train", 1, 32768, 2560, 4, "bf16", True, True, False), name="conv_long"),
        # the input of one decoding step of 16 sequences: launch latency
        dict(embed_case(16, 2048, 32000, "bf16", "bf16", False, False), name="embed_token"),
        # odd token count and vocabulary, the residual stream in 32 bits
        dict(embed_case(1000, 1536, 50257, "bf16", "f32", True, True), name="embed_odd"),
        # 4 rows of 8192 tokens, a large vocabulary
        dict(embed_case(32768, 2048, 128000, "bf16", "bf16", True, True), name="embed_large"),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def width(rng, lo, hi):
    """Mostly a multiple of 64, else any."""
    d = spread(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.6 else d


def draw(rng):
    op = rng.choice(["ssm", "ssm", "conv", "embed"])
    if op == "ssm":
        mode = rng.choice(["train", "train", "prompt", "step"])
        n = rng.choice([16, 16, 16, 8, 4, 32, 64, rng.randrange(1, 33)])
        d, groups = width(rng, 64, 4096), rng.choice([1, 1, 1, 2, 4])
        d = max(groups, d // groups * groups)
        kind = rng.choice(["bf16", "bf16", "f32"])
        if mode == "step":
            return ssm_case(mode, spread(rng, 1, 512), 1, d, n, groups, kind, rng.random() < 0.7, False, False)
        batch = spread(rng, 1, 16)
        length = min(spread(rng, 1, 32768), max(1, 32768 * 2048 * 16 // (batch * d * n)))
        return ssm_case(mode, batch, length, d, n, groups, kind, rng.random() < 0.7, rng.random() < 0.3, rng.random() < 0.3)
    if op == "conv":
        mode, d, w = rng.choice(["train", "train", "prompt", "step"]), width(rng, 64, 8192), rng.choice([4, 4, 3, 2])
        kind, silu = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.7
        if mode == "step":
            return conv_case(mode, spread(rng, 1, 512), 1, d, w, kind, silu, False, True)
        batch = spread(rng, 1, 16)
        length = min(spread(rng, 1, 32768), max(1, 32768 * 2560 // (batch * d * BYTES[kind] // 2)))
        return conv_case(mode, batch, length, d, w, kind, silu, rng.random() < 0.3, rng.random() < 0.3)
    tokens, d = spread(rng, 1, 32768), width(rng, 64, 4096)
    vocab = min(spread(rng, 1000, 128000), 128000 * 2048 // d)
    return embed_case(min(tokens, 32768 * 2048 // d), d, vocab, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"]),
                      rng.random() < 0.6, rng.random() < 0.7)


# ------------------------------------------------------------------- inputs ---
def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)

    def uniform(shape):
        return torch.rand(shape, generator=gen, device=DEV)

    s = dict(case=case)
    if case["op"] == "embed":
        n, v, d = case["tokens"], case["vocab"], case["d"]
        if case["zipf"]:                                                     # rank r with a frequency near 1 / r
            tok = torch.exp(uniform(n) * math.log(v)).long().sub(1).clamp(0, v - 1)
        else:
            tok = torch.randint(0, v, (n,), generator=gen, device=DEV)
        s["tokens"] = torch.where(uniform(n) < 0.03, torch.full_like(tok, -1), tok)    # the others are padding
        s["w"], s["scale"] = normal((v, d), DTYPES[case["weight"]], d ** -0.5), math.sqrt(d)
        if case["train"]:
            s["dout"] = normal((n, d), DTYPES[case["out"]], 1e-3)
        return s
    kind, b, l, d, step = DTYPES[case["dtype"]], case["batch"], case["length"], case["d"], case["mode"] == "step"
    lead = (b,) if step else (b, l)
    s["reset"] = s["lengths"] = None
    if case["packed"]:
        s["reset"] = (uniform((b, l)) < 4.0 / l).to(torch.uint8)
        s["reset"][:, 0] = 1
        if case["op"] == "conv":
            s["reset"][:, 0] = 0                                             # the first sequence goes on from the state
    if case["op"] == "conv":
        w = case["width"]
        s["x"] = normal((*lead, 2 * d), kind)[..., :d]                       # half of the projection before it
        s["w"], s["bias"] = normal((d, w), std=w ** -0.5), normal(d, std=0.1)
        s["state"] = normal((b, w - 1, d), kind) if case["state"] else None
        if case["mode"] == "train":
            s["dy"] = normal((*lead, d), kind)
        return s
    n, g = case["n"], case["groups"]
    if case["ragged"]:
        s["lengths"] = torch.randint(max(1, l // 4), l + 1, (b,), generator=gen, device=DEV, dtype=torch.int32)
    s["u"] = normal((*lead, d), kind)
    s["dt"] = normal((*lead, d), kind, 0.5)
    step_size = torch.exp(uniform(d) * math.log(100.0) + math.log(1e-3))     # softplus(dt_bias), from 0.001 to 0.1
    s["dt_bias"] = step_size + torch.log(-torch.expm1(-step_size))
    s["a"] = -torch.arange(1, n + 1, device=DEV) * torch.exp(normal((d, n), std=0.1))
    both = normal((*lead, d // 16 + 2 * g * n), kind)                        # a projection's: what dt is formed from, then b and c
    s["b"], s["c"] = [both[..., d // 16 + k * g * n:d // 16 + (k + 1) * g * n].unflatten(-1, (g, n)) for k in (0, 1)]
    s["d"] = normal(d, std=0.1, mean=1.0)
    s["z"] = normal((*lead, 2 * d), kind)[..., d:] if case["gate"] else None
    if step:
        s["h"] = normal((b, d, n), std=0.3)
    if case["mode"] == "train":
        s["dy"] = normal((*lead, d), kind)
    return s


# -------------------------------------------------------------- one pass each ---
def run(s):
    return {"ssm": run_ssm, "conv": run_conv, "embed": run_embed}[s["case"]["op"]](s)


def sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(x.clamp_max(20.0))))


def scan(decay, drive):
    """h_t = decay_t h_{t-1} + drive_t along dimension 1, from zero, by doubling (both arguments are used up)."""
    k, length = 1, drive.shape[1]
    while k < length:
        drive = torch.cat([drive[:, :k], drive[:, k:] + decay[:, k:] * drive[:, :-k]], 1)
        if 2 * k < length:
            decay = torch.cat([decay[:, :k], decay[:, k:] * decay[:, :-k]], 1)
        k *= 2
    return drive


def run_ssm(s):
    c = s["case"]
    if own:
        from linear_recurrence_sequence_amd import ssm
        args = [s[k] for k in ("u", "dt", "a", "b", "c", "d", "z", "dt_bias")]
        if c["mode"] == "step":
            return dict(y=ssm.ssm_scan_step(s["h"], *args), h=s["h"])
        y, h, saved = ssm.ssm_scan_fwd(*args, reset=s["reset"], lengths=s["lengths"], want_saved=c["mode"] == "train")
        out = dict(y=y, h=h)
        if c["mode"] == "train":
            out.update(ssm.ssm_scan_bwd(*args, saved, s["dy"], reset=s["reset"], lengths=s["lengths"]))
        return out
    n, kind, per = c["n"], DTYPES[c["dtype"]], c["d"] // c["groups"]
    u, a = s["u"].float(), s["a"]
    raw = s["dt"].float() + s["dt_bias"]
    dt = softplus(raw)
    b, q = [s[k].float().repeat_interleave(per, -2) for k in ("b", "c")]     # [..., d, n]
    z = s["z"].float() if c["gate"] else None
    sg = sigmoid(z) if c["gate"] else 1.0
    gate = z * sg if c["gate"] else 1.0
    if c["mode"] == "step":
        h = s["h"]
        h.mul_(torch.exp(dt[..., None] * a)).add_((dt * u)[..., None] * b)
        return dict(y=(((h * q).sum(-1) + s["d"] * u) * gate).to(kind), h=h)
    on = torch.ones_like(dt[..., :1], dtype=torch.bool)
    if c["ragged"]:
        on = (torch.arange(c["length"], device=u.device) < s["lengths"][:, None])[..., None]
        u, dt = u * on, dt * on
    decay = torch.exp(dt[..., None] * a)
    if c["packed"]:
        decay = decay * (s["reset"] == 0)[..., None, None]
    h = scan(decay, (dt * u)[..., None] * b)
    yp = (h * q).sum(-1) + s["d"] * u
    out = dict(y=(yp * gate * on).to(kind), h=h[:, -1].contiguous())
    if c["mode"] != "train":
        return out
    dy = s["dy"].float() * on
    dyp = dy * gate
    # cotangents of the states, from the last token to the first
    nxt = torch.cat([decay[:, 1:], torch.zeros_like(decay[:, :1])], 1)
    g = scan(nxt.flip(1), (dyp[..., None] * q).flip(1)).flip(1)
    del nxt, q
    sb = (g * b).sum(-1)
    del b
    heads = (*dyp.shape[:2], c["groups"], per)
    out["dc"] = (dyp[..., None] * h).unflatten(2, heads[2:]).sum(3).to(kind)
    out["db"] = ((dt * u)[..., None] * g).unflatten(2, heads[2:]).sum(3).to(kind)
    h = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    g = g * decay * h
    del h, decay
    out["du"] = (dt * sb + s["d"] * dyp).to(kind)
    ddt = (u * sb + (g * a).sum(-1)) * sigmoid(raw) * on
    out["ddt"] = ddt.to(kind)
    out["da"] = (g * dt[..., None]).sum((0, 1))
    out["dd"], out["ddt_bias"] = (dyp * u).sum((0, 1)), ddt.sum((0, 1))
    if c["gate"]:
        out["dz"] = (dy * yp * (sg + gate * (1.0 - sg))).to(kind)
    return out


def taps(x, state, width):
    """x with the inputs from before its first token in front."""
    if state is None:
        state = torch.zeros_like(x[:, :1]).expand(-1, width - 1, -1)
    return torch.cat([state, x], 1)


def run_conv(s):
    c = s["case"]
    if own:
        from linear_recurrence_sequence_amd import ssm
        act = "silu" if c["silu"] else "none"
        if c["mode"] == "step":
            return dict(y=ssm.causal_conv_step(s["x"], s["w"], s["bias"], s["state"], act=act), state=s["state"])
        y, last = ssm.causal_conv_fwd(s["x"], s["w"], s["bias"], act=act, state=s["state"], reset=s["reset"])
        out = dict(y=y, last=last)
        if c["mode"] == "train":
            out.update(ssm.causal_conv_bwd(s["x"], s["w"], s["bias"], s["dy"], act=act, state=s["state"], reset=s["reset"]))
        return out
    w, l, kind, train = c["width"], c["length"], DTYPES[c["dtype"]], c["mode"] == "train"
    if c["mode"] == "step":
        every = torch.cat([s["state"], s["x"][:, None]], 1).float()
        pre = s["bias"] + (every * s["w"].t()).sum(1)
        s["state"].copy_(every[:, 1:])
        return dict(y=(pre * sigmoid(pre) if c["silu"] else pre).to(kind), state=s["state"])
    leaf = {k: s[k].float().requires_grad_(train) for k in ("x", "w", "bias", "state") if s[k] is not None}
    every = taps(leaf["x"], leaf.get("state"), w)
    seg = torch.zeros((c["batch"], l + w - 1), dtype=torch.int32, device=every.device)      # the sequence that an input belongs to
    if c["packed"]:
        seg[:, w - 1:] = s["reset"].cumsum(1)
    pre = leaf["bias"]
    for k in range(w):
        pre = pre + leaf["w"][:, k] * every[:, k:k + l] * (seg[:, k:k + l] == seg[:, w - 1:])[..., None]
    y = pre * sigmoid(pre) if c["silu"] else pre
    last = every[:, l:].detach() * (seg[:, l:] == seg[:, -1:])[..., None]
    out = dict(y=y.detach().to(kind), last=last.to(kind))
    if train:
        g = torch.autograd.grad(y, list(leaf.values()), s["dy"].float())
        out.update({"d" + k: v.to(kind) if k in ("x", "state") else v for k, v in zip(leaf, g)})
    return out


def run_embed(s):
    c = s["case"]
    if own:
        from linear_recurrence_sequence_amd import lm
        out = dict(out=lm.embed_fwd(s["tokens"], s["w"], scale=s["scale"], out_dtype=DTYPES[c["out"]]))
        if c["train"]:
            out["dw"] = lm.embed_bwd(s["tokens"], s["dout"], c["vocab"], scale=s["scale"], grad_dtype=DTYPES[c["weight"]])
        return out
    on, t = (s["tokens"] >= 0)[:, None], s["tokens"].clamp_min(0)
    out = dict(out=(s["w"][t].float() * s["scale"] * on).to(DTYPES[c["out"]]))
    if c["train"]:
        dw = torch.zeros((c["vocab"], c["d"]), device=s["w"].device)
        out["dw"] = dw.index_add_(0, t, s["dout"].float() * on).mul_(s["scale"]).to(DTYPES[c["weight"]])
    return out


# ------------------------------------------------------------ from 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    return {"ssm": exact_ssm, "conv": exact_conv, "embed": exact_embed}[case["op"]](case, s)


def exact_ssm(case, s):
    step, n, per = case["mode"] == "step", case["n"], case["d"] // case["groups"]
    if step:
        s = dict(s, **{k: s[k][:, None] for k in ("u", "dt", "b", "c")}, z=s["z"][:, None] if case["gate"] else None)
    u, raw, a, dd = s["u"].double(), s["dt"].double() + s["dt_bias"].double(), s["a"].double(), s["d"].double()
    batch, length, d = u.shape
    dt = torch.nn.functional.softplus(raw, threshold=50.0)
    on = torch.ones((batch, length, 1), dtype=torch.float64, device=u.device)
    if case["ragged"]:
        for i, k in enumerate(s["lengths"].tolist()):
            on[i, k:] = 0.0
    keep = (1.0 - s["reset"].double()) if case["packed"] else torch.ones((batch, length), dtype=torch.float64, device=u.device)
    grouped = (batch, case["groups"], per, n)

    def outer(x, y):                                                         # [batch, d] and [batch, groups, n] to [batch, d, n]
        return (x.reshape(*grouped[:3], 1) * y[:, :, None]).reshape(batch, d, n)

    h = s["h"].double() if step else torch.zeros((batch, d, n), dtype=torch.float64, device=u.device)
    yp, states = torch.empty_like(u), [h]
    b, c = s["b"].double(), s["c"].double()
    for t in range(length):
        x = on[:, t] * dt[:, t]
        h = torch.exp(x[..., None] * a) * keep[:, t, None, None] * h + outer(x * u[:, t], b[:, t])
        if case["mode"] == "train":
            states.append(h)
        yp[:, t] = (h.reshape(grouped) * c[:, t, :, None]).sum(-1).reshape(batch, d) + dd * u[:, t]
    gate, slope = torch.ones_like(u), torch.zeros_like(u)
    if case["gate"]:
        z = s["z"].double()
        gate, slope = z * torch.sigmoid(z), torch.sigmoid(z) * (1 + z * (1 - torch.sigmoid(z)))
    y = yp * gate * on
    if step:
        return dict(y=y[:, 0], h=h)
    out = dict(y=y, h=h)
    if case["mode"] != "train":
        return out
    dy = s["dy"].double() * on
    dyp = dy * gate
    du, ddt, db, dc = torch.empty_like(u), torch.empty_like(u), torch.empty_like(b), torch.empty_like(c)
    da, g = torch.zeros_like(a), torch.zeros_like(h)
    for t in reversed(range(length)):
        x = on[:, t] * dt[:, t]
        dc[:, t] = (dyp[:, t].reshape(*grouped[:3], 1) * states.pop().reshape(grouped)).sum(2)
        g = g + outer(dyp[:, t], c[:, t])
        sb = (g.reshape(grouped) * b[:, t, :, None]).sum(-1).reshape(batch, d)
        db[:, t] = ((x * u[:, t]).reshape(*grouped[:3], 1) * g.reshape(grouped)).sum(2)
        g = g * torch.exp(x[..., None] * a) * keep[:, t, None, None]
        q = g * states[-1]
        da += (q * x[..., None]).sum(0)
        du[:, t] = x * sb + dd * dyp[:, t]
        ddt[:, t] = (u[:, t] * sb + (q * a).sum(-1)) * torch.sigmoid(raw[:, t]) * on[:, t]
    out.update(du=du, ddt=ddt, db=db, dc=dc, da=da, dd=(dyp * u).sum((0, 1)), ddt_bias=ddt.sum((0, 1)))
    if case["gate"]:
        out["dz"] = dy * yp * slope
    return out


def exact_conv(case, s):
    w, weight, bias = case["width"], s["w"].double(), s["bias"].double()
    x = s["x"].double()
    if case["mode"] == "step":
        x = x[:, None]
    batch, length, d = x.shape
    before = s["state"].double() if case["state"] else torch.zeros((batch, w - 1, d), dtype=torch.float64, device=x.device)
    every = torch.cat([before, x], 1)
    ends = torch.full((batch, length + w - 1), 0, dtype=torch.int64, device=x.device)     # where an input's sequence began
    if case["packed"]:
        at = torch.arange(w - 1, length + w - 1, device=x.device)
        ends[:, w - 1:] = torch.where(s["reset"] != 0, at, torch.zeros_like(at)).cummax(1).values
    now = torch.arange(w - 1, length + w - 1, device=x.device)
    pre = bias.expand(batch, length, d).clone()
    seen = [(now - j >= ends[:, w - 1:])[..., None].double() for j in range(w)]             # input j tokens back is of the same sequence
    for j in range(w):
        pre += weight[:, w - 1 - j] * every[:, w - 1 - j:w - 1 - j + length] * seen[j]
    sg = torch.sigmoid(pre)
    y = pre * sg if case["silu"] else pre
    last = every[:, length:] * (torch.arange(length, length + w - 1, device=x.device) >= ends[:, -1:])[..., None]
    if case["mode"] == "step":
        return dict(y=y[:, 0], state=last)
    out = dict(y=y, last=last)
    if case["mode"] == "train":
        g = s["dy"].double() * (sg * (1 + pre * (1 - sg)) if case["silu"] else 1.0)
        dx, dw = torch.zeros_like(every), torch.zeros_like(weight)
        for j in range(w):
            k = slice(w - 1 - j, w - 1 - j + length)
            dx[:, k] += weight[:, w - 1 - j] * g * seen[j]
            dw[:, w - 1 - j] = (g * every[:, k] * seen[j]).sum((0, 1))
        out.update(dx=dx[:, w - 1:], dw=dw, dbias=g.sum((0, 1)))
        if case["state"]:
            out["dstate"] = dx[:, :w - 1]
    return out


def exact_embed(case, s):
    on = s["tokens"] >= 0
    table = torch.cat([s["w"].double() * s["scale"], torch.zeros((1, case["d"]), dtype=torch.float64, device=DEV)])
    out = dict(out=table[torch.where(on, s["tokens"], torch.full_like(s["tokens"], case["vocab"]))])
    if case["train"]:
        order = torch.argsort(s["tokens"])[int((~on).sum()):]
        rows, counts = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        dw = torch.zeros((case["vocab"], case["d"]), dtype=torch.float64, device=DEV)
        of = torch.repeat_interleave(torch.arange(len(rows), device=DEV), counts)
        sums = torch.zeros((len(rows), case["d"]), dtype=torch.float64, device=DEV)
        sums.index_put_((of,), s["dout"][order].double(), accumulate=True)
        dw[rows] = sums * s["scale"]
        out["dw"] = dw
    return out


# -------------------------------------------------------------------- floors ---
def work(case):
    if case["op"] == "embed":
        n, d, wb, ob = case["tokens"], case["d"], BYTES[case["weight"]], BYTES[case["out"]]
        rows = min(n, case["vocab"])
        out = {"bytes": n * 8 + rows * d * wb + n * d * ob, "flops": n * d}
        if case["train"]:
            out["bytes"] += n * d * ob + case["vocab"] * d * wb
            out["flops"] += 2 * n * d
        return out
    rows, d, size, train = case["batch"] * case["length"], case["d"], BYTES[case["dtype"]], case["mode"] == "train"
    if case["op"] == "conv":
        w, step = case["width"], case["mode"] == "step"
        state = (2 if step or train else 1) * case["batch"] * (w - 1) * d * size if case["state"] else 0
        return {"bytes": rows * d * size * (4 if train else 2) + state + d * (w + 1) * 4 * (2 if train else 1),
                "flops": rows * d * ((6 if train else 2) * w + (10 if case["silu"] else 0))}
    n, g = case["n"], case["groups"]
    streams, states = (3 + case["gate"]) * (2 if train else 1), {"step": 2, "prompt": 1, "train": 1}[case["mode"]]
    # a state's update is exp(dt a) h + dt u b and its use c h; the backward forms it again, then the cotangents
    return {"bytes": rows * size * (streams * d + 2 * g * n * (2 if train else 1)) + case["batch"] * d * n * 4 * states
            + (n + 2) * d * 4 * (2 if train else 1),
            "flops": rows * d * n * (30 if train else 7)}
