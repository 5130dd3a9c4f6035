"""Plain 64-bit references of the layer operators (numpy, on the CPU), with
the sums of magnitudes their error bounds are stated in.  Written from the
operators' definitions position by position and group by group; no code is
shared with the library or with its binding."""
import numpy as np

BLOCK = 128


def bf16(x):
    """x rounded to bf16 (nearest, ties to even), as float64 values."""
    f = np.asarray(x, np.float64).astype(np.float32)
    b = f.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(f), np.nan, r).astype(np.float64)


def f64(t):
    """A torch tensor's values as float64."""
    return t.detach().float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------- residual norm --
def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def spread(gate, channels):
    """A gate per group (or channel) as one per channel."""
    if gate is None:
        return 1.0
    return np.repeat(gate, channels // gate.shape[1], axis=1)


def _groups(x, groups):
    return x.reshape(x.shape[0], groups, -1)


def rms(x, groups, eps):
    """1 / root mean square of each group [rows, groups]."""
    return 1.0 / np.sqrt((_groups(x, groups) ** 2).mean(-1) + eps)


def per_channel(s, channels):
    return np.repeat(s, channels // s.shape[1], axis=1)


def norm_out(r, y, gate, w, s, groups, eps, alpha):
    """(out before rounding, u, magnitude of out's terms)."""
    c = r.shape[1]
    u = rms(y, groups, eps)
    a = spread(None if gate is None else sigmoid(gate), c)
    branch = s * a * w * y * per_channel(u, c)
    return alpha * r + branch, u, np.abs(alpha * r) + np.abs(branch)


def norm_next(out, wn, groups, eps):
    """(next before rounding, v) of the rounded out."""
    v = rms(out, groups, eps)
    return out * per_channel(v, out.shape[1]) * wn, v


def norm_grads(d_out, d_next, out, v, y, u, gate, w, s, wn, groups, alpha):
    """Gradients (float64) and, for each, the magnitude its rounding errors scale with."""
    rows, c = (d_out if d_out is not None else out).shape
    n = c // groups

    def mean(x):
        return np.repeat(_groups(x, groups).mean(-1), n, axis=1)

    grads, mags = {}, {}
    dR, mR = np.zeros((rows, c)), np.zeros((rows, c))
    if d_out is not None:
        dR, mR = dR + d_out, mR + np.abs(d_out)
    if wn is not None:
        vv = per_channel(v, c)
        gx, xh = d_next * wn, out * vv
        dR = dR + vv * (gx - xh * mean(gx * xh))
        mR = mR + vv * (np.abs(gx) + np.abs(xh) * mean(np.abs(gx * xh)))
        grads["w_next"], mags["w_next"] = (d_next * xh).sum(0), np.abs(d_next * xh).sum(0)
    grads["residual"], mags["residual"] = alpha * dR, np.abs(alpha) * mR
    if y is None:
        return grads, mags
    uu = per_channel(u, c)
    yh = y * uu
    a = spread(None if gate is None else sigmoid(gate), c)
    q, mq = dR * a * s * w, mR * a * np.abs(s * w)
    grads["y"] = uu * (q - yh * mean(q * yh))
    mags["y"] = uu * (mq + np.abs(yh) * mean(mq * np.abs(yh)))
    d, md = (dR * a * yh).sum(0), (mR * a * np.abs(yh)).sum(0)
    grads["w_post"], mags["w_post"] = s * d, np.abs(s) * md
    grads["scale"], mags["scale"] = w * d, np.abs(w) * md
    if gate is not None:
        na = spread(sigmoid(-gate), c)
        dz, mz = na * q * yh, na * mq * np.abs(yh)
        if gate.shape[1] == groups and gate.shape[1] != c:
            dz, mz = _groups(dz, groups).sum(-1), _groups(mz, groups).sum(-1)
        grads["gate"], mags["gate"] = dz, mz
    return grads, mags


# --------------------------------------------------------- 8-bit checkpoints --
def encode(x):
    """(codes int8, scales float32 [rows, blocks]) of float32 values x [rows, channels]."""
    x = np.asarray(x, np.float32)
    rows, c = x.shape
    blocks = -(-c // BLOCK)
    codes, scales = np.zeros((rows, c), np.int8), np.zeros((rows, blocks), np.float32)
    for b in range(blocks):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        finite = np.isfinite(part).all(1)
        m = np.where(finite, np.abs(np.where(np.isfinite(part), part, 0)).max(1), 0).astype(
            np.float32)
        on = finite & (m >= np.float32(2.0) ** -120)
        safe = np.where(on, m, 1).astype(np.float32)
        scale = np.where(on, safe / np.float32(127), 0).astype(np.float32)
        inv = np.float32(127) / safe
        with np.errstate(invalid="ignore", over="ignore"):
            q = np.rint(part * inv[:, None])
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.where(on[:, None], q, 0).astype(np.int8)
        scales[:, b] = np.where(finite, scale, np.float32("nan"))
    return codes, scales


def decode(codes, scales):
    """float32 values of codes [rows, channels] (rows of one scale a BLOCK channels)."""
    s = np.repeat(scales, BLOCK, axis=1)[:, :codes.shape[1]]
    return (codes.astype(np.float32) * s).astype(np.float32)


# --------------------------------------------------------------- convolution --
def conv_pairs(length, halo_len, dilation, taps, seg):
    """For one row: the pairs (p, t, j) of positions counted from the halo's start where output
    t = p + j * dilation reads p: t in the sequence, no segment beginning in (p, t]."""
    begins = np.zeros(length, np.int64)
    if seg is not None:
        begins[1:] = seg[1:] != seg[:-1]
    run = np.cumsum(begins)
    for j in range(taps):
        for p in range(length):
            t = p + j * dilation
            if halo_len <= t < length and run[t] == run[p]:
                yield p, t, j


def conv_forward(x, w, dilation, bias=None, seg=None, halo=None):
    batch, seq, c = x.shape
    h = 0 if halo is None else halo.shape[1]
    out = np.zeros((batch, seq, c))
    if bias is not None:
        out += bias
    for b in range(batch):
        xx = x[b] if h == 0 else np.concatenate([halo[b], x[b]])
        for p, t, j in conv_pairs(h + seq, h, dilation, w.shape[1],
                                  None if seg is None else seg[b]):
            out[b, t - h] += w[:, w.shape[1] - 1 - j] * xx[p]
    return out


def conv_grads(g, x, w, dilation, seg=None, halo=None):
    """Gradients and their magnitudes: x, halo, weight, bias."""
    batch, seq, c = g.shape
    h, K = 0 if halo is None else halo.shape[1], w.shape[1]
    dx, mx = np.zeros((batch, h + seq, c)), np.zeros((batch, h + seq, c))
    dw, mw = np.zeros((c, K)), np.zeros((c, K))
    for b in range(batch):
        xx = x[b] if h == 0 else np.concatenate([halo[b], x[b]])
        for p, t, j in conv_pairs(h + seq, h, dilation, K, None if seg is None else seg[b]):
            k = K - 1 - j
            dx[b, p] += w[:, k] * g[b, t - h]
            mx[b, p] += np.abs(w[:, k] * g[b, t - h])
            dw[:, k] += g[b, t - h] * xx[p]
            mw[:, k] += np.abs(g[b, t - h] * xx[p])
    grads = dict(x=dx[:, h:], halo=dx[:, :h], weight=dw, bias=g.sum((0, 1)))
    mags = dict(x=mx[:, h:], halo=mx[:, :h], weight=mw, bias=np.abs(g).sum((0, 1)))
    return grads, mags


# ----------------------------------------------------------------- embedding --
def embed_grad(tokens, grads, table_rows, scale):
    """float64 sums scaled and rounded once to float32."""
    out = np.zeros((table_rows, grads.shape[1]))
    ok = (tokens >= 0) & (tokens < table_rows)
    np.add.at(out, tokens[ok], grads[ok])
    return (out * float(np.float32(scale))).astype(np.float32)


# -------------------------------------------------------------------- bounds --
def within(got, want, mag, steps, rounding=0.0):
    """|got - want| <= rounding * |want| + steps * 2^-24 * mag, element by element (steps: the
    fp32 roundings on the longest path to a value; rounding: the last one, of the output's
    type), non-finite values alike.  Returns what of the bound the worst element took."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(fine, np.isfinite(got)), "non-finite values at other places"
    bound = rounding * np.abs(want) + steps * 2.0 ** -24 * np.broadcast_to(mag, want.shape)
    err = np.abs(got - want)
    tiny = 2.0 ** -126  # where bf16 and fp32 stop being exact to a part
    over = np.where(fine, err - bound - tiny, 0.0)
    worst = float((err[fine] / (bound[fine] + tiny)).max()) if fine.any() else 0.0
    assert not (over > 0).any(), f"worst element at {worst:.3g} of its bound"
    return worst


BF16_ROUNDING = 2.0 ** -8  # half a step either side of a rounding boundary
