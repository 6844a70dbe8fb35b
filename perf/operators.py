"""The operators of a language model around the recurrent mixers, as they are measured.

Three operators: the norms around a block with its gate and residual scale
("norm"), the softmax cross entropy of a linear head ("ce") and the AdamW step
over many tensors ("adamw").  Each is here in its plain form (elementary torch
operations in 32 bits), as a user calls it from the package (`own`), and in 64
bits from its definition (`exact`).
"""
import math

import torch

own = False

EPS = 1e-6                                  # norms
LR, BETA1, BETA2, ADAM_EPS = 1e-3, 0.9, 0.95, 1e-8
BLOCK, TOP, LEAST, FLOOR = 256, 448.0, 2.0 ** -9, 2.0 ** -96    # 8-bit states: block, e4m3's largest and least value, least scale
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
DEV = "cuda" if torch.cuda.is_available() else "cpu"


# ---------------------------------------------------------------- the cases ---
def norm_case(rows, d, stream, branch, gate, full, train):
    """full: norm after the block with its weight and a residual scale; else the plain residual sum before the next norm."""
    return dict(op="norm", rows=rows, d=d, stream=stream, branch=branch, gate=gate, full=full, train=train)


def ce_case(tokens, d, vocab, cap, zloss, train):
    return dict(op="ce", tokens=tokens, d=d, vocab=vocab, cap=cap, zloss=zloss, train=train)


def adamw_case(layers, d, vocab, ragged, param, grad, master, bits):
    """layers of width d and an embedding (ragged = 0), or that many tensors of odd sizes up to d * vocab."""
    return dict(op="adamw", layers=layers, d=d, vocab=vocab, ragged=ragged, param=param, grad=grad, master=master, bits=bits)


def listed():
    return [
        # one decoding step of 16 sequences: launch latency
        dict(norm_case(16, 2048, "bf16", "bf16", "silu", True, False), name="norm_token"),
        # one training sequence of 2048 tokens at width 1024
        dict(norm_case(2048, 1024, "bf16", "bf16", "silu", True, True), name="norm_train"),
        # an odd width in 32 bits, residual sum and next norm only
        dict(norm_case(777, 1537, "f32", "f32", "none", False, True), name="norm_odd"),
        # 4 packed rows of 8192 tokens at width 2560, the residual stream kept in 32 bits
        dict(norm_case(32768, 2560, "f32", "bf16", "sigmoid", True, True), name="norm_wide"),
        # log-likelihood of a few tokens: the head's weights are read once
        dict(ce_case(16, 1024, 32000, 0.0, False, False), name="ce_score"),
        # one training sequence of 2048 tokens, a small vocabulary
        dict(ce_case(2048, 1024, 32000, 0.0, False, True), name="ce_train"),
        # odd token count and vocabulary, logits capped, a penalty on the log-sum
        dict(ce_case(1000, 1536, 50257, 30.0, True, True), name="ce_odd"),
        # 8192 tokens against a large vocabulary
        dict(ce_case(8192, 2048, 128000, 0.0, False, True), name="ce_large"),
        # a small model in 32 bits: launch latency over many small tensors
        dict(adamw_case(2, 256, 1000, 0, "f32", "f32", False, 32), name="adamw_small"),
        # tensors of odd sizes, 8-bit states
        dict(adamw_case(0, 1000, 1000, 24, "f32", "bf16", False, 8), name="adamw_ragged_8bit"),
        # a model of width 1024, bf16 weights with a 32-bit copy
        dict(adamw_case(8, 1024, 32000, 0, "bf16", "bf16", True, 32), name="adamw_32bit"),
        # a model of width 2048 and a large vocabulary, the same with 8-bit states
        dict(adamw_case(12, 2048, 128000, 0, "bf16", "bf16", True, 8), name="adamw_8bit"),
    ]


def spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "ce", "adamw"])
    if op == "norm":
        rows = spread(rng, 1, 32768)
        d = min(spread(rng, 64, 8192), 32768 * 2560 // rows)
        if rng.random() < 0.6:
            d = max(8, d // 8 * 8)
        return norm_case(rows, d, rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.choice(["none", "sigmoid", "silu"]),
                         rng.random() < 0.7, rng.random() < 0.7)
    if op == "ce":
        tokens, d = spread(rng, 1, 8192), 8 * spread(rng, 32, 320)
        vocab = min(spread(rng, 1000, 128000), 8192 * 2048 * 128000 // (tokens * d))
        return ce_case(tokens, d, vocab, rng.choice([0.0, 0.0, 30.0]), rng.random() < 0.3, rng.random() < 0.7)
    kind = rng.choice([("bf16", "bf16", True), ("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", False)])
    if rng.random() < 0.4:
        return adamw_case(0, rng.randrange(100, 2000), rng.randrange(100, 2000), rng.randrange(1, 64), *kind, rng.choice([8, 32]))
    return adamw_case(rng.randrange(1, 9), 16 * spread(rng, 8, 128), spread(rng, 500, 64000), 0, *kind, rng.choice([8, 32]))


# ------------------------------------------------------------------- inputs ---
def sizes(case):
    """Element counts of the tensors that one optimizer step updates."""
    if case["ragged"]:
        top, n = case["d"] * case["vocab"], case["ragged"]
        return [max(1, int(top ** ((i + 1) / n)) - i % 3) for i in range(n)]
    d = case["d"]
    one = [2 * d * d, d * d] + [d * d // 16] * 2 + [d] * 6   # in, out, two gate projections; their biases, retention, norms, scale
    return [case["vocab"] * d] + one * case["layers"] + [d]


def decays(case):
    """Matrices decay, vectors do not (of the ragged tensors, every second one)."""
    if case["ragged"]:
        return [0.1 * (i % 2) for i in range(case["ragged"])]
    return [0.1] + ([0.1] * 4 + [0.0] * 6) * case["layers"] + [0.0]


def encode(x, least=False):
    """Blocks of 256 values as e4m3 codes and a scale each; `least`: a positive value takes at least the least code."""
    b = x.reshape(-1, BLOCK)
    s = (b.abs().amax(1, keepdim=True) / TOP).clamp_min(FLOOR)
    q = b * (1.0 / s)
    if least:
        q = torch.where(b > 0, q.clamp_min(LEAST), q)
    return q.to(torch.float8_e4m3fn).reshape(-1), s.reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std + mean).to(dtype)

    s = dict(case=case)
    if case["op"] == "norm":
        rows, d, st, br = case["rows"], case["d"], DTYPES[case["stream"]], DTYPES[case["branch"]]
        s["x"], s["y"] = normal((rows, d), st, 2.0), normal((rows, d), br, 1.5)
        s["gate"] = None if case["gate"] == "none" else normal((rows, d), br)
        s["w_post"] = normal(d, std=0.1, mean=1.0) if case["full"] else None
        s["scale"] = normal(d, std=0.1, mean=0.5) if case["full"] else None
        s["w_pre"] = normal(d, std=0.1, mean=1.0)
        if case["train"]:
            s["dr"], s["dn"] = normal((rows, d), st), normal((rows, d), br)
        return s
    if case["op"] == "ce":
        n, d, v = case["tokens"], case["d"], case["vocab"]
        w = normal((v, d), std=2.0 / math.sqrt(d))
        t = torch.randint(0, v, (n,), generator=gen, device=DEV)
        sure = 3.0 * torch.rand((n, 1), generator=gen, device=DEV)          # how sure the model is of a token
        s["h"], s["w"] = (normal((n, d)) + sure * w[t]).bfloat16(), w.bfloat16()
        counts = torch.rand(n, generator=gen, device=DEV) >= 0.05            # the others are prompt or padding
        counts[0] = True
        s["target"] = torch.where(counts, t, torch.full_like(t, -100))
        s["dloss"] = torch.full((n,), 1.0, device=DEV) / counts.sum()
        s["dlse"] = 1e-3 * torch.rand(n, generator=gen, device=DEV) / n if case["zloss"] else None
        return s
    sz = sizes(case)
    at, total = [], 0
    for k in sz:                                                             # every tensor starts on a block
        at.append(total)
        total += -(-k // BLOCK) * BLOCK
    inside = torch.zeros(total, device=DEV)
    for o, k in zip(at, sz):
        inside[o:o + k] = 1.0

    def views(flat, per=1):
        return [flat[o // per:o // per + -(-k // per)] for o, k in zip(at, sz)]

    flat = {"p": normal(total, std=0.02) * inside}
    flat["g"] = (normal(total, std=1e-3) * inside).to(DTYPES[case["grad"]])
    if case["master"]:
        flat["master"] = flat["p"]
    flat["p"] = flat["p"].to(DTYPES[case["param"]])
    m, root = normal(total, std=3e-4) * inside, (normal(total, std=1e-3).abs() + 1e-5) * inside
    if case["bits"] == 8:
        flat["m"], flat["m_scale"] = encode(m)
        flat["v"], flat["v_scale"] = encode(root, True)
    else:
        flat["m"], flat["v"] = m, root * root
    s["flat"] = flat
    s["lists"] = {k: views(t, BLOCK if k.endswith("_scale") else 1) for k, t in flat.items()}
    s["decay"] = decays(case)
    blocks = torch.tensor([-(-k // BLOCK) for k in sz], device=DEV)
    s["decay_of_block"] = torch.repeat_interleave(torch.tensor(s["decay"], device=DEV), blocks)
    s["step"] = 1000
    return s


# -------------------------------------------------------------- one pass each ---
def run(s):
    return {"norm": run_norm, "ce": run_ce, "adamw": run_adamw}[s["case"]["op"]](s)


def run_norm(s):
    c = s["case"]
    if own:
        from linear_recurrence_sequence_amd import lm
        r, n, stats = lm.block_norm_fwd(s["x"], s["y"], s["gate"], s["w_post"], s["scale"], s["w_pre"], eps=EPS, gate_act=c["gate"])
        out = dict(r=r, n=n)
        if c["train"]:
            out.update(lm.block_norm_bwd(s["x"], s["y"], s["gate"], s["w_post"], s["scale"], s["w_pre"], stats, s["dr"], s["dn"],
                                         eps=EPS, gate_act=c["gate"]))
        return out
    leaf = {k: s[k].float().requires_grad_(c["train"]) for k in ("x", "y", "gate", "w_post", "scale", "w_pre") if s[k] is not None}

    def norm(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w

    u = norm(leaf["y"], leaf["w_post"]) if c["full"] else leaf["y"]
    if c["gate"] != "none":
        a = 1.0 / (1.0 + torch.exp(-leaf["gate"]))
        u = u * (a * leaf["gate"] if c["gate"] == "silu" else a)
    if c["full"]:
        u = u * leaf["scale"]
    r = leaf["x"] + u
    n = norm(r, leaf["w_pre"])
    st, br = s["x"].dtype, s["y"].dtype
    out = dict(r=r.detach().to(st), n=n.detach().to(br))
    if c["train"]:
        g = torch.autograd.grad([r, n], list(leaf.values()), [s["dr"].float(), s["dn"].float()])
        kept = {"x": st, "y": br, "gate": br}
        out.update({"d" + k: v.to(kept.get(k, torch.float32)) for k, v in zip(leaf, g)})
    return out


def run_ce(s):
    c = s["case"]
    if own:
        from linear_recurrence_sequence_amd import lm
        loss, lse = lm.linear_ce_fwd(s["h"], s["w"], s["target"], softcap=c["cap"])
        out = dict(loss=loss, lse=lse)
        if c["train"]:
            out.update(lm.linear_ce_bwd(s["h"], s["w"], s["target"], lse, s["dloss"], s["dlse"], softcap=c["cap"]))
        return out
    h, w = s["h"].float().requires_grad_(c["train"]), s["w"].float().requires_grad_(c["train"])
    z = h @ w.t()
    if c["cap"]:
        z = c["cap"] * torch.tanh(z / c["cap"])
    top = z.detach().amax(1, keepdim=True)
    lse = (torch.log(torch.exp(z - top).sum(1, keepdim=True)) + top)[:, 0]
    counts = s["target"] >= 0
    picked = z.gather(1, s["target"].clamp_min(0)[:, None])[:, 0]
    loss = torch.where(counts, lse - picked, torch.zeros_like(lse))
    out = dict(loss=loss.detach(), lse=lse.detach())
    if c["train"]:
        dh, dw = torch.autograd.grad([loss, lse], [h, w], [s["dloss"], torch.zeros_like(s["dloss"]) if s["dlse"] is None else s["dlse"]])
        out.update(dh=dh.bfloat16(), dw=dw.bfloat16())
    return out


def run_adamw(s):
    c, f = s["case"], s["flat"]
    new = {k: t for k, t in f.items() if k != "g"}
    if own:
        from linear_recurrence_sequence_amd import lm
        v = s["lists"]
        lm.adamw_step(v["p"], v["g"], v["m"], v["v"], step=s["step"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS, weight_decay=s["decay"],
                      masters=v.get("master"), m_scales=v.get("m_scale"), v_scales=v.get("v_scale"))
        return new
    g = f["g"].float()
    m, v = f["m"].float(), f["v"].float()
    if c["bits"] == 8:
        m = (m.reshape(-1, BLOCK) * f["m_scale"][:, None]).reshape(-1)
        v = (v.reshape(-1, BLOCK) * f["v_scale"][:, None]).reshape(-1)
        v = v * v
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    root = torch.sqrt(v)
    update = m / (root * (1 / math.sqrt(1 - BETA2 ** s["step"])) + ADAM_EPS)
    p = (f["master"] if c["master"] else f["p"].float()).reshape(-1, BLOCK)
    p = (p * (1 - LR * s["decay_of_block"])[:, None]).reshape(-1) - (LR / (1 - BETA1 ** s["step"])) * update
    if c["master"]:
        f["master"].copy_(p)
    f["p"].copy_(p)
    if c["bits"] == 8:
        for k, x in (("m", m), ("v", root)):
            q, scale = encode(x, k == "v")
            f[k].copy_(q)
            f[k + "_scale"].copy_(scale)
    else:
        f["m"].copy_(m)
        f["v"].copy_(v)
    return new


# ------------------------------------------------------------ from 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "ce": exact_ce, "adamw": exact_adamw}[case["op"]](case, s)


def exact_norm(case, s):
    x, y, w2 = s["x"].double(), s["y"].double(), s["w_pre"].double()
    d = case["d"]
    one = torch.ones(d, dtype=torch.float64, device=DEV)
    w1, sc = (s["w_post"].double(), s["scale"].double()) if case["full"] else (one, one)
    rs1 = 1.0 / torch.sqrt(y.pow(2).sum(1, keepdim=True) / d + EPS) if case["full"] else torch.ones_like(y[:, :1])
    yh = y * rs1
    a, da = torch.ones_like(y), torch.zeros_like(y)
    if case["gate"] != "none":
        g = s["gate"].double()
        a = torch.sigmoid(g)
        da = a * (1 - a)
        if case["gate"] == "silu":
            a, da = a * g, a + g * da
    r = x + sc * a * yh * w1
    rs2 = 1.0 / torch.sqrt(r.pow(2).sum(1, keepdim=True) / d + EPS)
    out = dict(r=r, n=r * rs2 * w2)
    if not case["train"]:
        return out
    dr, dn = s["dr"].double(), s["dn"].double()
    rh, t = r * rs2, dn * w2
    v = dr + rs2 * (t - rh * (t * rh).sum(1, keepdim=True) / d)
    t = v * sc * a * w1
    out.update(dx=v, dw_pre=(dn * rh).sum(0),
               dy=rs1 * (t - yh * (t * yh).sum(1, keepdim=True) / d) if case["full"] else t)
    if case["full"]:
        out.update(dw_post=(v * sc * a * yh).sum(0), dscale=(v * a * yh * w1).sum(0))
    if case["gate"] != "none":
        out["dgate"] = v * sc * yh * w1 * da
    return out


def exact_ce(case, s):
    w, parts = s["w"].double(), []
    dw = torch.zeros_like(w) if case["train"] else None
    for n0 in range(0, case["tokens"], 2048):                                # some tokens at a time: the logits in 64 bits are large
        k = slice(n0, min(n0 + 2048, case["tokens"]))
        h, t = s["h"][k].double(), s["target"][k]
        z = h @ w.t()
        slope = None
        if case["cap"]:
            slope = torch.tanh(z / case["cap"])
            z = case["cap"] * slope
            slope = 1 - slope * slope
        lse = torch.logsumexp(z, 1)
        on, row = t >= 0, torch.arange(len(t), device=DEV)
        part = dict(loss=(lse - z[row, t.clamp_min(0)]) * on, lse=lse)
        if case["train"]:
            dl = s["dloss"][k].double() * on
            dz = torch.exp(z - lse[:, None]) * (dl if s["dlse"] is None else dl + s["dlse"][k].double())[:, None]
            dz[row, t.clamp_min(0)] -= dl
            if slope is not None:
                dz *= slope
            part["dh"] = dz @ w
            dw += dz.t() @ h
        parts.append(part)
    out = {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
    if case["train"]:
        out["dw"] = dw
    return out


def exact_adamw(case, s):
    f, out = {k: t.double() for k, t in s["flat"].items()}, {}
    rows = {k: t.reshape(-1, BLOCK) for k, t in f.items() if not k.endswith("_scale")}
    m, v = rows["m"], rows["v"]
    if case["bits"] == 8:
        m, v = m * f["m_scale"][:, None], (v * f["v_scale"][:, None]) ** 2
    m = BETA1 * m + (1 - BETA1) * rows["g"]
    v = BETA2 * v + (1 - BETA2) * rows["g"] ** 2
    t = s["step"]
    p = rows["master" if case["master"] else "p"]
    p = p - LR * s["decay_of_block"].double()[:, None] * p
    p = p - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + ADAM_EPS)
    for k, x in (("m", m), ("v", torch.sqrt(v))):
        if case["bits"] == 8:
            scale = torch.clamp(x.abs().max(1).values / TOP, min=FLOOR)
            q = x / scale[:, None]
            if k == "v":
                q = torch.where(x > 0, torch.clamp(q, min=LEAST), q)
            out[k], out[k + "_scale"] = q.float().to(torch.float8_e4m3fn).double().reshape(-1), scale
        else:
            out[k] = (x * x if k == "v" else x).reshape(-1)
    out["p"] = p.reshape(-1)
    if case["master"]:
        out["master"] = out["p"]
    return out


# -------------------------------------------------------------------- floors ---
def work(case):
    if case["op"] == "norm":
        st, br = BYTES[case["stream"]], BYTES[case["branch"]]
        gates, vectors = case["gate"] != "none", 3 if case["full"] else 1
        per, flops = 2 * st + (2 + gates) * br, 20                          # x, r; y, n, gate
        if case["train"]:
            per, flops = per + 2 * st + (2 + gates) * br, 60                # dr, dx; dn, dy, dgate
        return {"bytes": case["rows"] * case["d"] * per + vectors * case["d"] * 4 * (2 if case["train"] else 1),
                "flops": flops * case["rows"] * case["d"]}
    if case["op"] == "ce":
        n, d, v = case["tokens"], case["d"], case["vocab"]
        if case["train"]:   # logits, and the two products of the gradient; the logits are not kept, so they are formed again
            return {"bytes": 4 * (n + v) * d + n * 24, "flops": 8 * n * d * v}
        return {"bytes": 2 * (n + v) * d + n * 16, "flops": 2 * n * d * v}
    n, state = sum(sizes(case)), 1 if case["bits"] == 8 else 4
    per = BYTES[case["grad"]] + 4 * state + (8 + BYTES[case["param"]] if case["master"] else 2 * BYTES[case["param"]])
    return {"bytes": n * (per + (16 / BLOCK if case["bits"] == 8 else 0)), "flops": 20 * n}
