"""The operators at the vocabulary's end of the layer, measured: distillation from a teacher's
top logits (loss, gradient, both in one call), the selection of a beam search over beams and
vocabulary, and the reordering of the decoding states (rings in slots, token histories) after it.

``own`` false: plain torch.  ``own`` true: the framework's calls.
"""
import math

import torch

own = False

VOCAB = 151936
LEAST_REST = 2.0 ** -20  # a smaller remainder of the teacher's mass is the rounding of its lse

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}
_LARGEST = 4096 * VOCAB * 2  # bytes of the largest listed logits


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the loss of a short validation sequence over a small float vocabulary
        dict(name="distill_small", op="distill", rows=9, vocab=1003, top=5, type="f32",
             teacher="f32", target="kept", temperature=1.0),
        # the loss of a validation batch over a vocabulary of odd length, the teacher's true
        # probabilities and one class for the rest
        dict(name="distill_eval", op="distill", rows=1031, vocab=50257, top=20, type="bf16",
             teacher="f32", target="rest", temperature=1.0),
        # the gradient from what a forward pass kept, float logits
        dict(name="distill_backward", op="distill_backward", rows=2049, vocab=32000, top=64,
             type="f32", teacher="bf16", target="kept", temperature=1.5),
        # a small training step over the whole vocabulary
        dict(name="distill_train_few", op="distill_train", rows=64, vocab=VOCAB, top=32,
             type="bf16", teacher="bf16", target="part", temperature=1.0),
        # a training step of 4096 tokens: loss and gradient of 1.2 GB of logits
        dict(name="distill_train", op="distill_train", rows=4096, vocab=VOCAB, top=128,
             type="bf16", teacher="bf16", target="rest", temperature=2.0),
        # one sequence with four beams: a decoding step where latency counts
        dict(name="select_few", op="select", batch=1, beams=4, vocab=VOCAB, count=4,
             type="bf16", finished=0.0, allowed=0),
        # a serving batch, twice as many candidates as beams
        dict(name="select_batch", op="select", batch=64, beams=8, vocab=VOCAB, count=16,
             type="bf16", finished=0.0, allowed=0),
        # float logits of an odd vocabulary under a grammar's mask, some beams finished
        dict(name="select_masked", op="select", batch=13, beams=5, vocab=50257, count=10,
             type="f32", finished=0.2, allowed=400),
        # four beams' rings after a step
        dict(name="fork_few", op="fork", batch=1, beams=4, rows=9, channels=1024, history=3),
        # a serving batch's rings
        dict(name="fork_many", op="fork", batch=64, beams=8, rows=12, channels=8192, history=4),
        # selection, then the states: what a decoding loop calls in turn
        dict(name="beam_step", op="step", batch=16, beams=8, vocab=VOCAB, count=8, type="bf16",
             finished=0.05, allowed=0, rows=12, channels=2048, history=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["distill", "distill_backward", "distill_train", "select", "select", "fork",
                     "step"])
    kind = rng.choice(["bf16", "f32"])
    vocab = _log(rng, 100, VOCAB)
    if op.startswith("distill"):
        top = min(_log(rng, 1, 256), vocab)
        most = min(16384, _LARGEST // (vocab * _BYTES[kind]), (1 << 27) // (top * top))
        return dict(op=op, rows=_log(rng, 1, most), vocab=vocab, top=top, type=kind,
                    teacher=rng.choice(["bf16", "f32"]),
                    target=rng.choice(["kept", "part", "rest"]),
                    temperature=rng.choice([0.7, 1.0, 1.0, 2.0, 4.0]))
    beams = rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
    case = dict(op=op, batch=_log(rng, 1, 512 // beams), beams=beams)
    if op != "fork":
        count = beams if op == "step" else min(rng.choice([beams, 2 * beams, 32]), vocab)
        case |= dict(vocab=vocab, count=count, type=kind, finished=rng.choice([0.0, 0.1, 0.3]),
                     allowed=rng.choice([0, 0, min(50, vocab)]))
    if op != "select":
        case |= dict(rows=rng.randint(1, 16), channels=8 * _log(rng, 8, 768),
                     history=rng.randint(1, 8))
    return case


# ------------------------------------------------------------------ inputs --
def _normal(g, shape, std=1.0, dtype=torch.float32):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
    return t.to(dtype)


def _prepare_distill(s, g):
    R, V, K, T = s["rows"], s["vocab"], s["top"], s["temperature"]
    s["logits"] = _normal(g, (R, V), 4.0, _TYPES[s["type"]])
    teacher = s["logits"].float().mul_(0.8).add_(_normal(g, (R, V), 1.5))
    top = torch.topk(teacher, K, dim=1)
    s["ids"], s["top_logits"] = top.indices, top.values.to(_TYPES[s["teacher"]])
    # rows with fewer entries, some with none
    used = torch.randint(0, 2 * K + 1, (R, 1), generator=g, device="cuda").clamp_(max=K)
    s["ids"] = torch.where(torch.arange(K, device="cuda") < used, s["ids"], -1).contiguous()
    s["teacher_lse"] = None
    if s["target"] != "kept":
        s["teacher_lse"] = torch.logsumexp(teacher.div_(T).double(), 1).float()
    # the mean over the answer's tokens; the prompt's have no weight
    on = torch.rand((R,), generator=g, device="cuda") < 0.9
    s["weight"] = on.float() * (T * T / R)
    if s["op"] == "distill_backward":  # what a forward pass kept
        z = s["logits"].double() / T
        s["lse"] = torch.logsumexp(z, 1).float()
        s["lse_rest"] = None
        if s["target"] == "rest":
            s["lse_rest"] = torch.logsumexp(_without(z, s["ids"]), 1).float()
    else:
        s["lse"] = s["lse_rest"] = None


def _without(z, ids):
    """z with the columns `ids` of each row at minus infinity."""
    more = torch.nn.functional.pad(z, (0, 1))  # a column for the unused entries
    at = torch.where(ids >= 0, ids, z.shape[1])
    return more.scatter_(1, at, -math.inf)[:, :-1]


def _prepare_select(s, g):
    B, W, V = s["batch"], s["beams"], s["vocab"]
    z = _normal(g, (B * W, V), 4.0, _TYPES[s["type"]])
    if s["allowed"]:
        keep = torch.rand((B * W, V), generator=g, device="cuda") < s["allowed"] / V
        z = torch.where(keep, z, torch.full_like(z, -math.inf))
    s["logits"] = z
    s["scores"] = -torch.rand((B, W), generator=g, device="cuda") * 3.0 - 20.0
    s["finished"], s["eos"] = None, -1
    if s["finished_share"]:
        s["finished"] = torch.rand((B, W), generator=g, device="cuda") < s["finished_share"]
        s["eos"] = V - 1


def _prepare_fork(s, g):
    B, W = s["batch"], s["beams"]
    n = B * W
    s["pool"] = _normal(g, (n + 3, s["rows"], s["channels"]), dtype=torch.bfloat16)
    s["slots"] = torch.randperm(n + 3, generator=g, device="cuda")[:n].view(B, W).contiguous()
    s["history_ids"] = torch.randint(0, VOCAB, (B, W, s["history"]), generator=g, device="cuda")
    if s["op"] == "fork":
        s["tokens"] = torch.randint(0, VOCAB, (B, W), generator=g, device="cuda")
        parents = torch.randint(0, W, (B, W), generator=g, device="cuda")
        unused = torch.rand((B, W), generator=g, device="cuda") < 0.02
        s["parents"] = torch.where(unused, -1, parents)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    s = dict(case)
    if s["op"].startswith("distill"):
        _prepare_distill(s, g)
        return s
    if s["op"] != "fork":
        s["finished_share"] = s["finished"]
        _prepare_select(s, g)
    if s["op"] != "select":
        _prepare_fork(s, g)
    return s


# ------------------------------------------------------------- plain forms --
def _target(s):
    """(p of every entry, the mass of each entry's id, sum of p, mass of the rest), few values and
    in 64 bits: a loss near zero is a difference of these."""
    ids, used = s["ids"], s["ids"] >= 0
    y = torch.where(used, s["top_logits"].double() / s["temperature"], -math.inf)
    if s["teacher_lse"] is None:
        e = torch.exp(y - y.amax(1, keepdim=True).clamp(min=-1e300))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
        rest = torch.zeros_like(p[:, 0])
    else:
        p = torch.exp(y - s["teacher_lse"].double()[:, None])
        rest = torch.zeros_like(p[:, 0])
        if s["target"] == "rest":
            left = 1.0 - p.sum(1)
            rest = torch.where((left >= LEAST_REST) & used.any(1), left, 0.0)
    whole = ((ids[:, :, None] == ids[:, None, :]) * p[:, None, :]).sum(2)
    return p, whole, p.sum(1), rest


def _lse(z):
    m = z.amax(1)
    return m.double() + torch.log(torch.exp(z - m[:, None]).sum(1, dtype=torch.float64))


def _distill(s):
    """(loss, lse, lse of the rest or None) of every row."""
    z = s["logits"].float() / s["temperature"]
    p, whole, _, rest = _target(s)
    lse = _lse(z)
    at = s["logits"].gather(1, s["ids"].clamp(min=0)).double() / s["temperature"]
    far = torch.log(whole) - (at - lse[:, None])
    loss = torch.where(p > 0, p * far, 0.0).sum(1)
    if s["target"] != "rest":
        return loss.float(), lse.float(), None
    lse_rest = _lse(_without(z, s["ids"]))
    loss += torch.where(rest > 0, rest * (torch.log(rest) - (lse_rest - lse)), 0.0)
    return loss.float(), lse.float(), lse_rest.float()


def _distill_grad(s, lse, lse_rest):
    z = s["logits"].float() / s["temperature"]
    p, _, m, rest = (x.float() for x in _target(s))
    grad = torch.exp(z - lse[:, None]) * (m + rest)[:, None]
    if lse_rest is not None:
        grad -= rest[:, None] * torch.exp(_without(z, s["ids"]) - lse_rest[:, None])
    grad.scatter_add_(1, s["ids"].clamp(min=0), -torch.where(s["ids"] >= 0, p, 0.0))
    grad *= (s["weight"] / s["temperature"])[:, None]
    return grad.to(s["logits"].dtype)


def _select(s):
    B, W, V, K = s["batch"], s["beams"], s["vocab"], s["count"]
    z = s["logits"].float() + 0.0  # minus zero is zero
    # sums in 64 bits: candidates of two beams may lie next to each other
    m = z.amax(1, keepdim=True).double()
    lse = m + torch.log(torch.exp(z - m).sum(1, keepdim=True))
    # each row's first K by (logit, lowest id), as whole numbers that differ
    bits = z.view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) << 32
    key = key + (V - 1 - torch.arange(V, device="cuda"))
    k = min(K, V)
    first = (V - 1) - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
    value = s["scores"].view(-1, 1).double() + (z.gather(1, first).double() - lse)
    done = torch.zeros((B, W), dtype=torch.bool, device="cuda")
    if s["finished"] is not None:
        done = s["finished"]
        only = torch.full_like(value, -math.inf)
        only[:, 0] = s["scores"].view(-1)
        value = torch.where(done.view(-1, 1), only, value)
        first = torch.where(done.view(-1, 1), s["eos"], first)
    value = torch.where(value.isnan(), -math.inf, value).view(B, W * k)
    best = torch.sort(value, dim=1, descending=True, stable=True)
    at = best.indices[:, :K]
    scores = best.values[:, :K].float()
    there = scores > -math.inf
    parents = torch.where(there, at // k, -1)
    tokens = torch.where(there, first.view(B, W * k).gather(1, at), -1)
    ended = there & (done.gather(1, parents.clamp(min=0)) | (tokens == s["eos"]))
    return scores, parents, tokens, ended


def _fork(s, parents, tokens):
    """(the new slots, the pool, the new histories)."""
    W = s["beams"]
    beam = torch.arange(W, device="cuda")
    there = parents >= 0
    same = (parents[:, :, None] == parents[:, None, :]) & (beam[None, :] < beam[:, None])
    keeps = there & ~same.any(2)  # the first child of its parent
    bare = ~(parents[:, :, None] == beam).any(1)  # no child
    old = torch.where(there, parents, beam)
    takes = torch.argsort(keeps.int(), dim=1, stable=True)
    free = torch.argsort(1 - bare.int(), dim=1, stable=True)
    given = torch.empty_like(free).scatter_(1, takes, free)
    slots = s["slots"].gather(1, torch.where(keeps, old, given))
    source = torch.where(there, s["slots"].gather(1, old), slots)
    s["pool"][slots.view(-1)] = s["pool"][source.view(-1)]
    history = s["history_ids"].gather(1, old[:, :, None].expand_as(s["history_ids"]))
    return slots, s["pool"], torch.cat([history[:, :, 1:], tokens[:, :, None]], 2)


def _plain(s):
    op = s["op"]
    if op == "distill":
        return [x for x in _distill(s) if x is not None]
    if op == "distill_backward":
        return _distill_grad(s, s["lse"], s["lse_rest"])
    if op == "distill_train":
        loss, lse, lse_rest = _distill(s)
        return [loss, _distill_grad(s, lse, lse_rest)]
    if op == "select":
        return list(_select(s))
    if op == "fork":
        return list(_fork(s, s["parents"], s["tokens"]))
    chosen = _select(s)
    return [*chosen, *_fork(s, chosen[1], chosen[2])]


# ---------------------------------------------------------------- the pass --
def _own(s):
    from gram_hashed_embedding_amd import vocab as V

    op = s["op"]
    if op.startswith("distill"):
        shared = dict(teacher_lse=s["teacher_lse"], temperature=s["temperature"])
        if op == "distill_backward":
            return V.engram_distill_backward(s["weight"], s["logits"], s["ids"], s["top_logits"],
                                             s["lse"], lse_rest=s["lse_rest"], **shared)
        d = V.engram_distill(s["logits"], s["ids"], s["top_logits"], rest=s["target"] == "rest",
                             grad_loss=s["weight"] if op == "distill_train" else None, **shared)
        if op == "distill_train":
            return [d.loss, d.grad]
        return [x for x in (d.loss, d.lse, d.lse_rest) if x is not None]
    out, parents, tokens = [], None, None
    if op != "fork":
        b = V.engram_beam_select(s["logits"], s["scores"], s["count"], finished=s["finished"],
                                 eos=s["eos"])
        out, parents, tokens = [b.scores, b.parents, b.tokens, b.finished], b.parents, b.tokens
    if op == "select":
        return out
    if op == "fork":
        parents, tokens = s["parents"], s["tokens"]
    f = V.engram_beam_fork(parents, [s["pool"]], slots=s["slots"], tokens=tokens,
                           history=s["history_ids"])
    return [*out, f.slots, s["pool"], f.history]


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work --
def work(case):
    op, n, flops = case["op"], 0, 0
    if op.startswith("distill"):
        R, V, K = case["rows"], case["vocab"], case["top"]
        row = V * _BYTES[case["type"]]
        small = K * (8 + _BYTES[case["teacher"]]) + (8 if case["target"] == "kept" else 12)
        passes = 1 if op == "distill" else 2  # the logits read, the gradient written
        return {"bytes": R * (passes * row + small),
                "flops": R * V * {"distill": 4, "distill_backward": 4, "distill_train": 8}[op]}
    beams = case["batch"] * case["beams"]
    if op != "fork":
        live = beams * (1.0 - case["finished"])  # a finished beam's logits are not needed
        n += live * case["vocab"] * _BYTES[case["type"]] + case["batch"] * case["count"] * 21
        flops += 4 * live * case["vocab"]
    if op != "select":
        W = case["beams"]
        copies = beams * (1.0 - 1.0 / W) ** W  # beams without a child, were parents uniform
        n += copies * 2 * (2 * case["rows"] * case["channels"])
        n += beams * (8 * 2 * case["history"] + 32)
    return {"bytes": n, "flops": flops}


# ------------------------------------------------------------- in 64 bits --
def _exact_distill(s):
    """Row by row from the definition: the two distributions over all classes written out."""
    f, T, V = torch.float64, s["temperature"], s["vocab"]
    R, rest_class = s["rows"], s["target"] == "rest"
    loss, lse = (torch.zeros((R,), dtype=f, device="cuda") for _ in range(2))
    lse_rest = torch.zeros((R,), dtype=f, device="cuda")
    grad = torch.zeros((R, V), dtype=f, device="cuda") if s["op"] != "distill" else None
    step = max(1, min(R, (1 << 27) // V))
    for a in range(0, R, step):
        c = slice(a, min(R, a + step))
        z, ids = s["logits"][c].to(f) / T, s["ids"][c]
        on, n = ids >= 0, ids.shape[0]
        y = torch.where(on, s["top_logits"][c].to(f) / T, torch.full((), -math.inf, dtype=f,
                                                                     device="cuda"))
        if s["teacher_lse"] is None:
            p = torch.softmax(y, 1)
        else:
            p = (y - s["teacher_lse"][c, None].to(f)).exp()
        p = torch.where(on, p, torch.zeros_like(p))
        P = torch.zeros((n, V + 1), dtype=f, device="cuda")
        P.scatter_add_(1, torch.where(on, ids, V), p)
        inside = torch.zeros((n, V + 1), dtype=torch.bool, device="cuda")
        inside.scatter_(1, torch.where(on, ids, V), True)
        P, inside = P[:, :V], inside[:, :V]
        total = torch.logsumexp(z, 1)
        outside = torch.logsumexp(z.masked_fill(inside, -math.inf), 1)
        if s["lse"] is not None:
            total = s["lse"][c].to(f)
            outside = s["lse_rest"][c].to(f) if rest_class else outside
        left = torch.zeros((n,), dtype=f, device="cuda")
        if rest_class:
            left = 1 - p.sum(1)
            left = torch.where((left >= LEAST_REST) & on.any(1), left, torch.zeros_like(left))
        lse[c], lse_rest[c] = total, outside
        loss[c] = (torch.xlogy(P, P) - P * (z - total[:, None])).sum(1)
        loss[c] += torch.xlogy(left, left) - left * (outside - total)
        if grad is not None:
            q = (z - total[:, None]).exp()
            d = q * (p.sum(1) + left)[:, None] - P
            d -= torch.where(inside, torch.zeros_like(z),
                             left[:, None] * (z - outside[:, None]).exp())
            grad[c] = d * (s["weight"][c, None].to(f) / T)
    if s["op"] == "distill":
        return [loss, lse, lse_rest] if rest_class else [loss, lse]
    return grad if s["op"] == "distill_backward" else [loss, grad]


def _exact_select(s):
    """Sequence by sequence: every candidate's score, sorted."""
    W, V, K, f = s["beams"], s["vocab"], s["count"], torch.float64
    scores, parents, tokens = [], [], []
    for b in range(s["batch"]):
        z = s["logits"][b * W:(b + 1) * W].to(f)
        every = s["scores"][b].to(f)[:, None] + torch.log_softmax(z, 1)
        if s["finished"] is not None:
            for w in s["finished"][b].nonzero().flatten().tolist():
                every[w] = -math.inf
                every[w, s["eos"]] = s["scores"][b, w].to(f)
        best = torch.sort(torch.nan_to_num(every, nan=-math.inf).flatten(), descending=True,
                          stable=True)
        value, at = best.values[:K], best.indices[:K]
        some = value > -math.inf
        scores.append(value)
        parents.append(torch.where(some, at // V, -1))
        tokens.append(torch.where(some, at % V, -1))
    return torch.stack(scores), torch.stack(parents), torch.stack(tokens)


def _exact_pool(s, parents):
    """The pool after the reordering, beam by beam."""
    old = s["pool"].to(torch.float64)
    new = old.clone()
    for slots, chosen in zip(s["slots"].tolist(), parents.tolist()):
        free = [slots[w] for w in range(s["beams"]) if w not in chosen]
        seen = set()
        for p in chosen:
            if p >= 0 and p not in seen:
                seen.add(p)  # keeps its slot
                continue
            to = free.pop(0)
            if p >= 0:
                new[to] = old[slots[p]]
    return new


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("distill"):
        return _exact_distill(s)
    if op == "fork":
        return [None, _exact_pool(s, s["parents"]), None]
    scores, parents, _ = _exact_select(s)
    if op == "select":
        return [scores, None, None, None]
    return [scores, None, None, None, None, _exact_pool(s, parents), None]
