"""Plain implementations, in 64 bits, of the operators at the vocabulary's end (include/
engram_vocab.h), and the tolerances their kernels are held to.  torch, on any device; loops over
rows and beams."""
import math

import torch

LEAST_REST = 2.0 ** -20

# What a sum of fp32 exponentials may be off by, relative to itself: v_exp_f32's 1 ulp (2^-23);
# the roundings of a term's exponent x (a subtraction, a product, an fma: 3 * 2^-24 * x * ln 2),
# whose mean over the terms is at most the distribution's entropy, 18 bits for 2^18 values; the
# additions of one lane, one a chunk of at most 2^18 values / 256 lanes / 8 = 128, one for a value
# before the first whole cache line, and 3 within a chunk, 2^-24 each.
SUM = (2 + 3 * 18 * math.log(2) + 132) * 2.0 ** -24
# A gradient's share q: that, a term's own roundings (x up to 200 among those that are not lost:
# 2^-23 + 200 * 3 * 2^-24 * ln 2), and twice the fp32 rounding of an lse up to 64 (2^-19 each).
SHARE = SUM + 2.0 ** -23 + 600 * math.log(2) * 2.0 ** -24 + 2.0 ** -18


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def target(ids, teacher, vocab, temperature, teacher_lse, rest):
    """(P [vocab], named [vocab], m, r, none) of one row."""
    dev = teacher.device
    y = teacher.double() / temperature
    used = (ids >= 0) & (ids < vocab)
    P = torch.zeros(vocab, dtype=torch.float64, device=dev)
    named = torch.zeros(vocab, dtype=torch.bool, device=dev)
    ids, y = ids[used], y[used]
    named[ids] = True
    none = ids.numel() == 0
    if none:
        return P, named, 0.0, 0.0, True
    if teacher_lse is None:
        if bool((y == -math.inf).all()):
            return P, named, 0.0, 0.0, True
        p = torch.softmax(y, 0)
    else:
        p = (y - teacher_lse.double()).exp()
    P.index_add_(0, ids, p)
    m, r = float(p.sum()), 0.0
    if teacher_lse is None:
        m = m if math.isnan(m) else 1.0
    elif rest:
        r = 1.0 - m
        r = r if r >= LEAST_REST else 0.0
    return P, named, m, r, none


def distill(logits, ids, teacher, teacher_lse=None, rest=False, temperature=1.0, grad_loss=None):
    """dict(loss, lse, lse_rest, grad, slack) of [rows, vocab] logits: the definition, row by row.
    slack: what a gradient is a difference of, which its error goes by."""
    rows, vocab = logits.shape
    dev, f = logits.device, torch.float64
    out = {k: torch.zeros(rows, dtype=f, device=dev)
           for k in ("loss", "lse", "lse_rest", "scale")}
    out["grad"], out["slack"] = (torch.zeros((rows, vocab), dtype=f, device=dev) for _ in range(2))
    for t in range(rows):
        z = logits[t].double() / temperature
        P, named, m, r, none = target(ids[t], teacher[t], vocab, temperature,
                                      None if teacher_lse is None else teacher_lse[t], rest)
        bad = bool(torch.isnan(z).any() | (z == math.inf).any())
        empty = bool((z == -math.inf).all())
        lse = math.nan if bad else -math.inf if empty else float(torch.logsumexp(z, 0))
        # (of differences to the largest: z - lse loses log(vocab) beside a mask's lowest value)
        logq = torch.full_like(z, -math.inf) if empty else torch.log_softmax(z, 0)
        q = logq.exp()
        outside = z.masked_fill(named, -math.inf)
        lse_rest = math.nan if bool(torch.isnan(outside).any() | (outside == math.inf).any()) \
            else float(torch.logsumexp(outside, 0))
        log_s = -math.inf if lse_rest == -math.inf else lse_rest - lse
        out["lse"][t], out["lse_rest"][t] = lse, lse_rest
        if none:
            continue
        on = P != 0
        loss = float((P[on] * (P[on].log() - logq[on])).sum())
        if r != 0:
            loss += r * (math.log(r) - log_s)
        out["loss"][t] = math.nan if bad else loss
        if grad_loss is None or float(grad_loss[t]) == 0.0:
            continue
        g = float(grad_loss[t]) / temperature
        out["scale"][t] = abs(g)
        share = torch.zeros_like(z)  # of an unnamed value in its own sum
        if lse_rest != -math.inf:
            share = torch.where(named, 0.0, torch.softmax(outside, 0))
        out["grad"][t] = math.nan if bad else g * (q * (m + r) - P - r * share)
        out["slack"][t] = abs(g) * (q * (m + r) + r * share) if not bad else 0.0
    return out


def check_distill(got, want, kept=None):
    """Loss, statistics and gradient against distill()'s.  kept: the statistics were read in fp32
    (SHARE allows for it)."""
    def close(a, b, tol, what):
        a = a.double().reshape(b.shape)
        same = (a == b) | (a.isnan() & b.isnan())
        off = torch.where(same, torch.zeros_like(b), (a - b).abs())
        ok = (off <= tol) & (same | (torch.isfinite(a) & torch.isfinite(b)))
        assert bool(ok.all()), (what, float(off[~ok].max()), int((~ok).sum()),
                                (~ok).nonzero()[0].tolist())

    finite = torch.nan_to_num(want["lse"], 0.0, 0.0, 0.0).abs()
    if got.get("lse") is not None:
        close(got["lse"], want["lse"], SUM + half_step(torch.float32) * finite, "lse")
    if got.get("lse_rest") is not None:
        size = torch.nan_to_num(want["lse_rest"], 0.0, 0.0, 0.0).abs()
        close(got["lse_rest"], want["lse_rest"], SUM + half_step(torch.float32) * size, "lse_rest")
    if got.get("loss") is not None:
        # (m + r is 1 or less, and both logarithms are off by SUM; the rest is in 64 bits)
        size = torch.nan_to_num(want["loss"], 0.0, 0.0, 0.0).abs()
        close(got["loss"], want["loss"], 2 * SUM + half_step(torch.float32) * size, "loss")
    if got.get("grad") is not None:
        g = got["grad"]
        size = torch.nan_to_num(want["grad"]).abs()
        # A term exp((z - max) / T) below fp32's normal numbers, 2^-126, is lost before it is
        # multiplied by at most |g| / T * (m + r) <= |g| / T; a product below them is too.
        least = 2.0 ** -126 * (1 + want["scale"].reshape(-1, *[1] * (want["grad"].dim() - 1)))
        close(g, want["grad"], half_step(g.dtype) * size * 1.01 + SHARE * want["slack"] + least,
              "grad")


def beam_values(logits, scores, finished=None, eos=-1):
    """Every candidate's value, [beams, vocab] for each sequence of [batch, beams, vocab]."""
    batch, beams, vocab = logits.shape
    for b in range(batch):
        z = logits[b].double()
        every = torch.full((beams, vocab), -math.inf, dtype=torch.float64, device=z.device)
        for w in range(beams):
            s = float(scores[b, w])
            if not math.isfinite(s):
                continue
            if finished is not None and bool(finished[b, w]):
                every[w, eos] = s
                continue
            if bool(torch.isnan(z[w]).any()):
                continue
            lse = float(torch.logsumexp(z[w], 0))
            if math.isfinite(lse):
                every[w] = s + (z[w] - lse)
        yield every


def beam_select(logits, scores, count, finished=None, eos=-1):
    """(scores, parents, tokens, finished) of [batch, beams, vocab] logits."""
    vocab = logits.shape[2]
    out = []
    for b, every in enumerate(beam_values(logits, scores, finished, eos)):
        flat = every.flatten()
        n = min(count, flat.numel())
        value, at = torch.sort(flat, descending=True, stable=True)
        value, at = value[:n], at[:n]
        there = value > -math.inf
        parent = torch.where(there, at // vocab, -1)
        token = torch.where(there, at % vocab, -1)
        ended = there & (token == eos)
        if finished is not None:
            ended |= there & finished[b][parent.clamp(min=0)]
        pad = count - n
        out.append((torch.nn.functional.pad(value, (0, pad), value=-math.inf),
                    torch.nn.functional.pad(parent, (0, pad), value=-1),
                    torch.nn.functional.pad(token, (0, pad), value=-1),
                    torch.nn.functional.pad(ended, (0, pad), value=False)))
    return tuple(torch.stack(x) for x in zip(*out))


def beam_fork(parents, slots, slot_count):
    """(new slots, {slot: the slot it is copied from}, invalid entries) of lists of lists."""
    new, copies, bad = [], {}, 0
    for chosen, have in zip(parents, slots):
        beams = len(have)
        valid = [p if 0 <= p < beams else None for p in chosen]
        bad += sum(p is None and q != -1 for p, q in zip(valid, chosen))
        bad += sum(s != -1 and not 0 <= s < slot_count for s in have)
        free = [have[w] for w in range(beams) if w not in valid]
        seen, row = set(), []
        for p in valid:
            if p is not None and p not in seen:
                seen.add(p)
                row.append(have[p])
                continue
            to = free.pop(0)
            row.append(to)
            if p is not None and 0 <= to < slot_count and 0 <= have[p] < slot_count:
                copies[to] = have[p]
        new.append(row)
    return new, copies, bad
