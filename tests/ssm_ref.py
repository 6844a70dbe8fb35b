"""The selective scan, the causal convolution and the embedding from their
definitions, in 64 bits, and how far a computation in 32 bits may be off.

With absolute=True every term counts by its size: the result bounds, for each
output, the sum of the sizes of all that was added up for it, which is what roundings
are relative to.
"""
import torch

U = 2.0 ** -24                       # half a step of FP32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def on_mask(batch, length, lengths, device):
    on = torch.ones((batch, length), dtype=torch.float64, device=device)
    if lengths is not None:
        for i, k in enumerate(lengths.tolist()):
            on[i, max(0, k):] = 0.0
    return on


def clean(t, on):
    """t [batch, length, ...] in 64 bits with zeros for padding, whatever it holds there."""
    if t is None:
        return None
    keep = (on != 0).reshape(*on.shape, *[1] * (t.dim() - 2))
    return torch.where(keep, t.double(), torch.zeros_like(t, dtype=torch.float64))


def scan_ref(u, dt, a, b, c, d=None, z=None, dt_bias=None, h0=None, *, softplus=True, reset=None, lengths=None, dy=None, dh_final=None,
             absolute=False):
    """dict(y, h[, du, ddt, da, db, dc, dd, dz, ddt_bias, dh0]) in 64 bits."""
    batch, length, width = u.shape
    groups, n = b.shape[-2:]
    per, dev = width // groups, u.device
    size = torch.abs if absolute else (lambda t: t)
    on = on_mask(batch, length, lengths, dev)
    u, b, c = size(clean(u, on)), size(clean(b, on)), size(clean(c, on))
    a = a.double()
    skip = torch.zeros(width, dtype=torch.float64, device=dev) if d is None else size(d.double())
    raw = clean(dt, on) + (0.0 if dt_bias is None else dt_bias.double())
    s = (torch.nn.functional.softplus(raw, threshold=60.0) if softplus else raw) * on[..., None]
    slope = torch.sigmoid(raw) if softplus else torch.ones_like(raw)
    if z is None:
        gate, gate_slope = torch.ones_like(u), torch.zeros_like(u)
    else:
        z = clean(z, on)
        sg = torch.sigmoid(z)
        # the slope is a sum of two terms that cancel near z = -1.28, where its roundings are those of 1 and z (1 - sg)
        gate, gate_slope = size(z * sg), sg * (1 + size(z) * (1 - sg)) if absolute else sg * (1 + z * (1 - sg))
    keep = torch.ones((batch, length), dtype=torch.bool, device=dev)
    if reset is not None:
        keep = reset == 0                                        # in the padding too

    def spread(x):                                              # [batch, groups, n] to [batch, width, n]
        return x.repeat_interleave(per, 1)

    def before(h, t):
        return torch.where(keep[:, t, None, None], h, torch.zeros_like(h))

    h = torch.zeros((batch, width, n), dtype=torch.float64, device=dev) if h0 is None else size(h0.double())
    sized = torch.abs(s) if absolute else s
    states, yp = [h], torch.zeros_like(u)
    for t in range(length):
        h = torch.exp(s[:, t, :, None] * a) * before(h, t) + (sized[:, t] * u[:, t])[..., None] * spread(b[:, t])
        states.append(h)
        yp[:, t] = (h * spread(c[:, t])).sum(-1) + skip * u[:, t]
    out = dict(y=yp * gate * on[..., None], h=h)
    if dy is None:
        return out
    dy = size(clean(dy, on))
    e = dy * gate
    g = torch.zeros_like(h) if dh_final is None else size(dh_final.double())
    du, ds, db, dc = torch.zeros_like(u), torch.zeros_like(u), torch.zeros_like(b), torch.zeros_like(c)
    da, rate = torch.zeros_like(a), size(a)
    for t in reversed(range(length)):
        live = on[:, t, None]
        g = g + e[:, t, :, None] * spread(c[:, t])
        dc[:, t] = (e[:, t, :, None] * states[t + 1]).unflatten(1, (groups, per)).sum(2)
        db[:, t] = ((sized[:, t] * u[:, t])[..., None] * g).unflatten(1, (groups, per)).sum(2)
        gb = (g * spread(b[:, t])).sum(-1)
        g = before(torch.exp(s[:, t, :, None] * a) * g, t)
        r = g * before(states[t], t)
        du[:, t] = sized[:, t] * gb + skip * e[:, t]
        ds[:, t] = (u[:, t] * gb + (r * rate).sum(-1)) * live
        da += (r * sized[:, t, :, None]).sum(0)
    ddt = ds * slope
    out.update(du=du * on[..., None], ddt=ddt, db=db, dc=dc, da=da, dd=(e * u).sum((0, 1)), ddt_bias=ddt.sum((0, 1)), dh0=g,
               dz=dy * yp * gate_slope)
    return out


def scan_tolerance(sizes, ref, length, dtype, wide=("h", "da", "dd", "ddt_bias", "dh0")):
    """A token's step rounds: s (the exponential, the logarithm, two quotients and their products: 10), its product with a
    and the exponential of it (an argument x is off by 3 halves of a step of itself, which moves e^-x by at most 3 x e^-x, 1.2, and two
    for the exponential: 4), s u b (3), the multiply-add (1): fewer than 20 halves of a step, each relative to the
    sizes that were added up.  A state carries those of all tokens before it, a cotangent those behind it; what meets both adds them up;
    the sums over states, channels and tokens, the gate (6), the slope (4) and the skip take fewer than 100 more (a sum of k values in
    FP32 in parts of 8, 4 and the workgroups' takes fewer than 50).  With 20 (2 length + 6) halves of a step all of it is covered; a result of
    `dtype` is rounded once more."""
    out = {}
    for k, m in sizes.items():
        t = 20 * (2 * length + 6) * U * m
        out[k] = t + (0.0 if k in wide else half_step(dtype)) * ref[k].abs() + 1e-37
    return out


def conv_ref(x, w, bias=None, *, silu=True, state=None, reset=None, lengths=None, dy=None, dstate_out=None, absolute=False):
    """dict(y, last[, dx, dw, dbias, dstate]) in 64 bits."""
    batch, length, d = x.shape
    width, dev = w.shape[1], x.device
    size = torch.abs if absolute else (lambda t: t)
    on = on_mask(batch, length, lengths, dev)
    n = on.sum(1).long()
    front = torch.zeros((batch, width - 1, d), dtype=torch.float64, device=dev) if state is None else state.double()
    raw = torch.cat([front, clean(x, on)], 1)                   # token t at t + width - 1
    every = size(raw)
    w64, b64 = w.double(), torch.zeros(d, dtype=torch.float64, device=dev) if bias is None else bias.double()
    seg = torch.zeros((batch, length + width - 1), dtype=torch.int64, device=dev)
    if reset is not None:
        seg[:, width - 1:] = ((reset != 0) & (on != 0)).long().cumsum(1)
    p, sizes = b64.expand(batch, length, d).clone(), b64.abs().expand(batch, length, d).clone()
    same = []
    for j in range(width):
        k = slice(width - 1 - j, width - 1 - j + length)
        m = (seg[:, k] == seg[:, width - 1:])[..., None]
        same.append(m)
        p += torch.where(m, raw[:, k], torch.zeros_like(raw[:, k])) * w64[:, width - 1 - j]
        sizes += torch.where(m, raw[:, k].abs(), torch.zeros_like(raw[:, k])) * w64[:, width - 1 - j].abs()
    sg = torch.sigmoid(p) if silu else torch.ones_like(p)
    slope = sg * (1 + p * (1 - sg)) if silu else torch.ones_like(p)
    y = (sizes if absolute else p) * sg
    if absolute and silu:
        # p's error reaches the slope through its own derivative, which is below 0.6, and 1 + p (1 - s) cancels
        slope = slope.abs() + 0.6 * sizes + sg * (1 + p.abs() * (1 - sg))
    last = torch.zeros((batch, width - 1, d), dtype=torch.float64, device=dev)
    for i in range(batch):
        k = int(n[i])
        last[i] = torch.where((seg[i, k:k + width - 1] == seg[i, k + width - 2])[:, None], every[i, k:k + width - 1], last[i])
    out = dict(y=y * on[..., None], last=last)
    if dy is None:
        return out
    g = size(clean(dy, on)) * slope * on[..., None]
    w64 = size(w64)
    dx, dw = torch.zeros_like(every), torch.zeros_like(w64)
    for j in range(width):
        k = slice(width - 1 - j, width - 1 - j + length)
        m = same[j]
        dx[:, k] += torch.where(m, g, torch.zeros_like(g)) * w64[:, width - 1 - j]
        dw[:, width - 1 - j] = torch.where(m, g * every[:, k], torch.zeros_like(g)).sum((0, 1))
    if dstate_out is not None:
        o = size(dstate_out.double())
        for i in range(batch):
            k = int(n[i])
            dx[i, k:k + width - 1] += torch.where((seg[i, k:k + width - 1] == seg[i, k + width - 2])[:, None], o[i], torch.zeros_like(o[i]))
    out.update(dx=dx[:, width - 1:], dw=dw, dbias=g.sum((0, 1)), dstate=dx[:, :width - 1])
    return out


def embed_ref(tokens, dout, v, scale, absolute=False):
    """The embedding's gradient in 64 bits."""
    dw = torch.zeros((v, dout.shape[-1]), dtype=torch.float64, device=dout.device)
    on = (tokens >= 0) & (tokens < v)
    g = dout.double()
    dw.index_add_(0, tokens[on], (g.abs() if absolute else g)[on])
    return dw * (abs(scale) if absolute else scale)
