"""Cases of the training operators at the two ends of a rank's model, next to
its sharded optimizer step.

Four operators:
  embed        y[i] = scale * table[token[i]], then dropout; the table is a
               tensor of the rank's flat 16-bit or fp32 parameter buffer
  embed_grad   its gradient, summed over equal tokens in position order, into
               the rank's flat gradient buffer or into the slice that one owner
               receives
  dropout      y = residual + keep * x / (1 - p), the mask from a counter and
               never stored; with no residual it is also its own backward pass
  preference   from logits to the paired preference loss
               mean_i [-(1-e) log s(h_i) - e log s(-h_i)],
               h_i = beta (sum_chosen (lp - ref) - sum_rejected (lp - ref)),
               lp the log-softmax at the label; a training pass also returns
               the gradient of the logits

Where ``own`` is false the operators are elementary torch operations in 32 bits
(64 where a long sum needs it), rounded once; where it is true they are the
library's calls.

Dropout's mask: element e of a tensor takes the 16 bits at position e mod 4 of
mix64(key + (e div 4 + 1) * GAMMA) (SplitMix64); it is kept where they are at
least round(65536 p), and divided by the share that is kept then.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"f32": 0, "f16": 1, "bf16": 2}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
MASK64 = (1 << 64) - 1
GAMMA, MIX1, MIX2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB
SITE, STEP = 7, 12            # which dropout of the model, which training step
ALIGN = 64                    # shard alignment of the flat buffers, elements


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _embed(n, vocab, hidden, dt, p, before=0):
    return {"op": "embed", "tokens": n, "vocab": vocab, "hidden": hidden, "dtype": dt, "p": p, "before": before}


def _grad(n, vocab, hidden, dt, p, ranks=1, rank=-1, before=0):
    return {"op": "embed_grad", "tokens": n, "vocab": vocab, "hidden": hidden, "dtype": dt, "p": p,
            "ranks": ranks, "rank": rank, "before": before}


def _drop(n, dt, p, residual, first=0):
    return {"op": "dropout", "n": n, "dtype": dt, "p": p, "residual": residual, "first": first}


def _pref(pairs, length, vocab, dt, train):
    return {"op": "preference", "pairs": pairs, "length": length, "vocab": vocab, "dtype": dt, "train": train}


def listed():
    cases = {
        # One row of the GPT-2-small table: nothing but latency.
        "embed one token": _embed(1, 50257, 768, "bf16", 0.0),
        # A long-context batch through a wide table, with embedding dropout.
        "embed wide": _embed(65536, 50257, 8192, "f16", 0.1),
        # A short odd batch into a small odd table behind an odd-sized tensor.
        "embed_grad small odd": _grad(37, 1009, 65, "f16", 0.0, before=33),
        # GPT-2-small: 8 sequences of 1024 tokens, the whole gradient buffer.
        "embed_grad gpt2": _grad(8192, 50257, 768, "bf16", 0.1),
        # One owner's slice of eight from a bigger batch (Stage 2).
        "embed_grad owner slice": _grad(65536, 50257, 2048, "bf16", 0.0, ranks=8, rank=0),
        # The wide table: as many bytes of activations as of gradient.
        "embed_grad wide": _grad(65536, 50257, 8192, "bf16", 0.1),
        # One token's hidden vector.
        "dropout one row": _drop(768, "bf16", 0.1, False),
        # The residual branch of a wide layer, 8192 tokens.
        "dropout residual": _drop(8192 * 8192, "bf16", 0.1, True),
        # One short pair and a small odd vocabulary.
        "preference one pair": _pref(1, 24, 1009, "f16", True),
        # Scoring with the reference model: the forward half, odd rows.
        "preference score": _pref(8, 512, 50257, "bf16", False),
        # A training batch over the GPT-2 vocabulary, fp16 logits.
        "preference train": _pref(4, 512, 50257, "f16", True),
        # A training batch over a large vocabulary: 4.3 GB of logits.
        "preference train wide": _pref(8, 1024, 131072, "bf16", True),
    }
    return [{"name": k, **v} for k, v in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "embed_grad", "dropout", "preference", "preference"])
    dt = rng.choice(["bf16", "f16", "bf16", "f16", "f32"])
    p = rng.choice([0.0, 0.1, 0.1, 0.25, rng.uniform(0.01, 0.6)])
    if op in ("embed", "embed_grad"):
        n, vocab, hidden = _log(rng, 1, 65536), _log(rng, 128, 131072), _log(rng, 32, 8192)
        if rng.random() < 0.5:
            hidden = max(64, hidden // 64 * 64)
        while n * hidden > 1 << 28 or vocab * hidden > 1 << 28:
            n, vocab = max(1, n // 2), max(128, vocab // 2)
        before = rng.choice([0, 0, 64, rng.randrange(1, 5000)])
        if op == "embed":
            return _embed(n, vocab, hidden, dt, p, before)
        ranks = rng.choice([1, 1, 4, 8])
        return _grad(n, vocab, hidden, dt, p, ranks, -1 if ranks == 1 else rng.randrange(ranks), before)
    if op == "dropout":
        return _drop(_log(rng, 1, 1 << 25), dt, p, rng.random() < 0.5, rng.choice([0, rng.randrange(1 << 34)]))
    pairs, length, vocab = rng.randrange(1, 9), _log(rng, 8, 1024), _log(rng, 200, 131072)
    while pairs * length * vocab > 1 << 28:
        length = max(8, length // 2)
        vocab = vocab // 2 + rng.randrange(2)
    return _pref(pairs, length, vocab, dt, rng.random() < 0.7)


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------

def _slice(case):
    """(elements of the flat buffer, first, last + 1) of the part returned."""
    size = case["before"] + case["vocab"] * case["hidden"]
    unit = case.get("ranks", 1) * ALIGN
    padded = -(-size // unit) * unit
    if case.get("rank", -1) < 0:
        return padded, 0, padded
    share = padded // case["ranks"]
    return padded, case["rank"] * share, (case["rank"] + 1) * share


def _tokens(case, g):
    """Token ids with the skew of text (the k-th most frequent at 1/(k + 2.7)),
    about one in a hundred a padding id."""
    n, vocab = case["tokens"], case["vocab"]
    weight = 1.0 / (torch.arange(vocab, device="cuda", dtype=torch.float64) + 2.7)
    edge = torch.cumsum(weight, 0)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * edge[-1]
    rank = torch.searchsorted(edge, u).clamp_(max=vocab - 1)
    ids = torch.randperm(vocab, generator=g, device="cuda")[rank]
    if n > 1:
        ids[torch.rand(n, generator=g, device="cuda") < 0.01] = -1
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case, seed=seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] in ("embed", "embed_grad"):
        n, vocab, hidden = case["tokens"], case["vocab"], case["hidden"]
        padded, lo, hi = _slice(case)
        s["ids"] = _tokens(case, g)
        s["scale"] = math.sqrt(hidden) if case["op"] == "embed" else 1.0 / max(1, n)
        if case["op"] == "embed":
            s["params"] = torch.empty(padded, device="cuda", dtype=dt).normal_(0, 0.02, generator=g)
            s["out"] = torch.empty((n, hidden), device="cuda", dtype=dt)
        else:
            s["dy"] = torch.empty((n, hidden), device="cuda", dtype=dt).normal_(0, 1.0, generator=g)
            s["grad"] = torch.zeros(hi - lo, device="cuda", dtype=dt)
    elif case["op"] == "dropout":
        s["x"] = torch.empty(case["n"], device="cuda", dtype=dt).normal_(0, 1.0, generator=g)
        s["res"] = torch.empty_like(s["x"]).normal_(0, 1.0, generator=g) if case["residual"] else None
        s["out"] = torch.empty_like(s["x"])
    else:
        pairs, length, vocab = case["pairs"], case["length"], case["vocab"]
        rows = 2 * pairs * length
        shift = torch.randint(-(length // 4), length // 4 + 1, (pairs,), generator=g, device="cuda")
        lens = torch.cat([length + shift, length - shift])
        s["offsets"] = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
        s["labels"] = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
        s["logits"] = torch.empty((rows, vocab), device="cuda", dtype=dt)
        ref = torch.empty(rows, device="cuda")
        for a in range(0, rows, 1024):     # the reference model's values lie near the policy's
            part = s["logits"][a:a + 1024].normal_(0, 2.0, generator=g)
            lab = s["labels"][a:a + 1024, None]
            part.scatter_(1, lab, part.gather(1, lab) + 6)
            part = part.float()
            ref[a:a + 1024] = part.gather(1, lab)[:, 0] - torch.logsumexp(part, 1)
        # a few tenths apart, and drifted by some thirty nats over a sequence.
        drift = 30.0 * torch.randn(2 * pairs, generator=g, device="cuda") / lens
        s["ref"] = ref + 0.3 * torch.randn(rows, generator=g, device="cuda") - drift.repeat_interleave(lens)
        # The prompt, a quarter of a sequence, is not scored.
        for first in s["offsets"][:-1].tolist():
            s["labels"][first:first + length // 4] = -100
        s["ref"][s["labels"] < 0] = 0
        s["beta"], s["smoothing"], s["grad_scale"] = 0.1, 0.05, 1024.0
        for name, n in (("logp", rows), ("stats", 2 * rows), ("coef", rows), ("loss", 1), ("pair_loss", pairs),
                        ("rewards", 2 * pairs)):
            s[name] = torch.empty(n, device="cuda")
        s["dlogits"] = torch.empty_like(s["logits"]) if case["train"] else None
    if own:
        _handles(s)
    return s


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "embed":
        n = case["tokens"] * case["hidden"]
        rows = min(case["tokens"], case["vocab"])          # distinct rows at most
        return {"bytes": rows * case["hidden"] * b + n * b + 8 * case["tokens"], "flops": 2 * n}
    if case["op"] == "embed_grad":
        _, lo, hi = _slice(case)
        first, last = max(lo, case["before"]), min(hi, case["before"] + case["vocab"] * case["hidden"])
        share = max(0, last - first) / (case["vocab"] * case["hidden"])
        n = case["tokens"] * case["hidden"] * share        # the activations of that share of the ids
        return {"bytes": n * b + max(0, last - first) * b + 8 * case["tokens"], "flops": 2 * n}
    if case["op"] == "dropout":
        return {"bytes": case["n"] * b * (3 if case["residual"] else 2), "flops": 3 * case["n"]}
    rows = 2 * case["pairs"] * case["length"]
    scored = rows - 2 * case["pairs"] * (case["length"] // 4)
    read, written = scored * case["vocab"] * b, rows * case["vocab"] * b if case["train"] else 0
    return {"bytes": read + written + 20 * rows, "flops": scored * case["vocab"] * (7 if case["train"] else 4)}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _handles(s):
    import zero_sharded_mixed_02_amd as Z
    code = CODES[s["dtype"]]
    s["drop"] = Z.Drop(s["p"], s["seed"], site=SITE, step=STEP, first=s.get("first", 0)) if s.get("p") else None
    if s["op"] in ("embed", "embed_grad"):
        sizes = [s["before"], s["vocab"] * s["hidden"]]
        s["plan"] = Z.zero_plan(sum(sizes), s.get("ranks", 1), sizes, 0, ALIGN)
    if s["op"] == "embed_grad":
        n = s["tokens"]
        s["sorted"], s["order"] = (torch.empty(n, device="cuda", dtype=torch.int32) for _ in range(2))
        need = max(Z.zero_token_order_workspace_bytes(n, s["vocab"]), Z.zero_embed_grad_workspace_bytes(n, s["hidden"]))
        s["ws"] = torch.empty(max(1, need), device="cuda", dtype=torch.uint8)
    if s["op"] == "preference":
        need = Z.zero_token_logp_workspace_bytes(s["logits"].shape[0], s["vocab"])
        s["ws"] = torch.empty(max(1, need), device="cuda", dtype=torch.uint8)
    s["Z"], s["code"] = Z, code


def _run_own(s):
    Z, code = s["Z"], s["code"]
    if s["op"] == "embed":
        Z.zero_embed(s["plan"], 1, s["hidden"], s["params"], code, s["ids"], s["scale"], s["out"], code, drop=s["drop"])
        return s["out"]
    if s["op"] == "embed_grad":
        Z.zero_token_order(s["ids"], s["vocab"], s["sorted"], s["order"], s["ws"])
        Z.zero_embed_grad(s["plan"], 1, s["hidden"], s["sorted"], s["order"], s["dy"], code, s["scale"], s["grad"],
                          code, drop=s["drop"], rank=s["rank"], workspace=s["ws"])
        return s["grad"]
    if s["op"] == "dropout":
        drop = s["drop"] or Z.Drop(0.0, s["seed"], site=SITE, step=STEP, first=s["first"])
        Z.zero_dropout(s["x"], s["res"], s["out"], code, drop)
        return s["out"]
    Z.zero_token_logp(s["logits"], code, s["labels"], s["logp"], s["stats"], s["ws"])
    Z.zero_preference_loss(s["offsets"], s["labels"], s["vocab"], s["logp"], s["ref"], s["beta"], s["smoothing"],
                           s["grad_scale"], s["loss"], s["pair_loss"], s["rewards"], s["coef"])
    got = {"loss": s["loss"], "rewards": s["rewards"], "logp": s["logp"]}
    if s["train"]:
        Z.zero_token_logp_grad(s["logits"], code, s["labels"], s["stats"], s["coef"], s["dlogits"])
        got["dlogits"] = s["dlogits"]
    return got


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _signed(v):
    return v - (1 << 64) if v >> 63 else v


def _mix64_int(z):
    z = ((z ^ (z >> 30)) * MIX1) & MASK64
    z = ((z ^ (z >> 27)) * MIX2) & MASK64
    return z ^ (z >> 31)


def _key(seed):
    k = seed & MASK64
    for field in (SITE, STEP):
        k = _mix64_int(((k ^ field) + GAMMA) & MASK64)
    return k


def _cut(p):
    return int(round(p * 65536))


def _keep(seed, p, first, n):
    """Dropout's mask of elements [first, first + n)."""
    a, b = first // 4, (first + n + 3) // 4
    z = torch.arange(a + 1, b + 1, device="cuda") * _signed(GAMMA) + _signed(_key(seed))
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _signed(MIX1)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _signed(MIX2)
    z = z ^ ((z >> 31) & ((1 << 33) - 1))
    bits = z.view(torch.int16)[first - 4 * a:first - 4 * a + n]
    return (bits.int() & 0xFFFF) >= _cut(p)


def _dropped(x, seed, p, first=0):
    if not p:
        return x
    keep = _keep(seed, p, first, x.numel()).view(x.shape)
    return torch.where(keep, x * (65536.0 / (65536 - _cut(p))), torch.zeros_like(x))


def _run_plain(s):
    dt = DTYPES[s["dtype"]]
    if s["op"] == "embed":
        table = s["params"][s["before"]:s["before"] + s["vocab"] * s["hidden"]].view(s["vocab"], s["hidden"])
        y = table[s["ids"].clamp(min=0)].float() * s["scale"]
        y = torch.where((s["ids"] >= 0)[:, None], y, torch.zeros_like(y))
        return _dropped(y, s["seed"], s["p"]).to(dt)
    if s["op"] == "embed_grad":
        _, lo, hi = _slice(s)
        dy = _dropped(s["dy"].float(), s["seed"], s["p"])
        grad = torch.zeros((s["vocab"] + 1, s["hidden"]), device="cuda")     # the last row takes the padding ids
        grad.index_add_(0, torch.where(s["ids"] < 0, s["vocab"], s["ids"]), dy)
        flat = (grad[:s["vocab"]] * s["scale"]).to(dt).view(-1)
        out = torch.zeros(hi - lo, device="cuda", dtype=dt)
        first, last = max(lo, s["before"]), min(hi, s["before"] + flat.numel())
        if first < last:
            out[first - lo:last - lo] = flat[first - s["before"]:last - s["before"]]
        return out
    if s["op"] == "dropout":
        y = _dropped(s["x"].float(), s["seed"], s["p"], s["first"])
        return (y if s["res"] is None else y + s["res"].float()).to(dt)
    x, labels = s["logits"].float(), s["labels"]
    valid = labels >= 0
    at = labels.clamp(min=0)[:, None]
    top = x.max(1, keepdim=True).values
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    logp = (x.gather(1, at) - top - torch.log(total))[:, 0]
    logp = torch.where(valid, logp, torch.zeros_like(logp))
    seq = torch.bucketize(torch.arange(x.shape[0], device="cuda"), s["offsets"][1:], right=True)
    sums = torch.zeros(2 * s["pairs"], device="cuda", dtype=torch.float64)
    sums.index_add_(0, seq, torch.where(valid, logp.double() - s["ref"].double(), 0.0))
    rewards = s["beta"] * sums
    h = rewards[:s["pairs"]] - rewards[s["pairs"]:]
    down = torch.log1p(torch.exp(-h.abs()))
    loss = ((1 - s["smoothing"]) * (down + (-h).clamp(min=0)) + s["smoothing"] * (down + h.clamp(min=0))).mean()
    got = {"loss": loss.float().view(1), "rewards": rewards.float(), "logp": logp}
    if s["train"]:
        up = 1 / (1 + torch.exp(-h))
        slope = s["beta"] * s["grad_scale"] / s["pairs"] * (s["smoothing"] * up - (1 - s["smoothing"]) * (1 - up))
        coef = torch.where(valid, torch.cat([slope, -slope])[seq], 0.0).float()[:, None]
        d = e.mul_(-coef / total)
        d.scatter_add_(1, at, coef)
        got["dlogits"] = d.to(dt)
    return got


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------------------------
# In 64 bits
# ---------------------------------------------------------------------------

def _mul64(lo, hi, c):
    """Low 64 bits of (hi 2^32 + lo) * c, as two halves held in int64."""
    c0, c1 = c & 0xFFFFFFFF, c >> 32
    a0, a1 = lo & 0xFFFF, lo >> 16
    low, mid = a0 * c0, a1 * c0                       # both below 2^48
    part = (low >> 16) + (mid & 0xFFFFFFFFFFFF)       # lo * c0, in units of 2^16
    new_lo = ((part & 0xFFFF) << 16) | (low & 0xFFFF)
    carry = part >> 16
    b0, b1 = lo & 0xFFFF, lo >> 16
    cross = (b0 * c1 + ((b1 * c1 & 0xFFFF) << 16)) & 0xFFFFFFFF
    d0, d1 = hi & 0xFFFF, hi >> 16
    cross2 = (d0 * c0 + ((d1 * c0 & 0xFFFF) << 16)) & 0xFFFFFFFF
    return new_lo, (carry + cross + cross2) & 0xFFFFFFFF


def _xorshift(lo, hi, k):
    """z ^ (z >> k) for k < 32."""
    return lo ^ (((lo >> k) | (hi << (32 - k))) & 0xFFFFFFFF), hi ^ (hi >> k)


def _factor64(seed, p, first, n):
    """keep / (share kept) of elements [first, first + n), by the definition, the 64-bit words in halves."""
    if not p:
        return torch.ones(n, device="cuda", dtype=torch.float64)
    key = _key(seed)
    e = torch.arange(first, first + n, device="cuda")
    word = torch.div(e, 4, rounding_mode="floor") + 1
    lo, hi = _mul64(word & 0xFFFFFFFF, word >> 32, GAMMA)
    lo = lo + (key & 0xFFFFFFFF)
    hi = (hi + (key >> 32) + (lo >> 32)) & 0xFFFFFFFF
    lo = lo & 0xFFFFFFFF
    lo, hi = _mul64(*_xorshift(lo, hi, 30), MIX1)
    lo, hi = _mul64(*_xorshift(lo, hi, 27), MIX2)
    lo, hi = _xorshift(lo, hi, 31)
    quarter = e % 4
    sixteen = torch.where(quarter >= 2, hi, lo) >> (16 * (quarter % 2)) & 0xFFFF
    cut = int(np.rint(p * 65536))
    return (sixteen >= cut).double() * (65536.0 / (65536 - cut))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        out = torch.empty(case["n"], device="cuda", dtype=torch.float64)
        for a in range(0, case["n"], 1 << 24):
            x = s["x"][a:a + (1 << 24)].double()
            x = x * _factor64(seed, case["p"], case["first"] + a, x.numel())
            out[a:a + (1 << 24)] = x if s["res"] is None else x + s["res"][a:a + (1 << 24)].double()
        return out
    if case["op"] == "embed":
        n, hidden = case["tokens"], case["hidden"]
        out = torch.zeros((n, hidden), device="cuda", dtype=torch.float64)
        step = max(1, (1 << 24) // hidden)
        for a in range(0, n, step):
            ids = s["ids"][a:a + step]
            at = case["before"] + ids[:, None] * hidden + torch.arange(hidden, device="cuda")
            rows = s["params"][at.clamp(min=0)].double() * (ids >= 0).double()[:, None]
            mask = _factor64(seed, case["p"], a * hidden, rows.numel()).view(rows.shape)
            out[a:a + step] = rows * (math.sqrt(hidden) * mask)
        return out
    if case["op"] == "embed_grad":
        n, vocab, hidden = case["tokens"], case["vocab"], case["hidden"]
        padded, lo, hi = _slice(case)
        flat = torch.zeros(padded, device="cuda", dtype=torch.float64)
        table = flat[case["before"]:case["before"] + vocab * hidden].view(vocab, hidden)
        step = max(1, (1 << 24) // hidden)
        for a in range(0, n, step):
            ids = s["ids"][a:a + step]
            dy = s["dy"][a:a + step].double()
            dy = dy * _factor64(seed, case["p"], a * hidden, dy.numel()).view(dy.shape)
            good = ids >= 0
            table.index_add_(0, ids[good], dy[good] / max(1, n))
        return flat[lo:hi]
    pairs, rows = case["pairs"], s["logits"].shape[0]
    logp = torch.zeros(rows, device="cuda", dtype=torch.float64)
    lse = torch.zeros_like(logp)
    scored = s["labels"] >= 0
    for a in range(0, rows, 256):
        part = s["logits"][a:a + 256].double()
        lse[a:a + 256] = torch.logsumexp(part, 1)
        logp[a:a + 256] = part.gather(1, s["labels"][a:a + 256, None].clamp(min=0))[:, 0] - lse[a:a + 256]
    logp *= scored
    ratio = (logp - s["ref"].double()) * scored
    bounds = s["offsets"].tolist()
    rewards = torch.stack([ratio[a:b].sum() for a, b in zip(bounds, bounds[1:])]) * s["beta"]
    margin = rewards[:pairs] - rewards[pairs:]
    eps = s["smoothing"]
    up, down = torch.sigmoid(margin), torch.sigmoid(-margin)
    loss = -((1 - eps) * torch.nn.functional.logsigmoid(margin) + eps * torch.nn.functional.logsigmoid(-margin))
    got = {"loss": loss.mean().view(1), "rewards": rewards, "logp": logp}
    if case["train"]:
        slope = (eps * up - (1 - eps) * down) * s["beta"] * s["grad_scale"] / pairs
        d = torch.empty(s["logits"].shape, device="cuda", dtype=torch.float64)
        signed = torch.cat([slope, -slope])
        lengths = s["offsets"][1:] - s["offsets"][:-1]
        coef = torch.repeat_interleave(signed, lengths) * scored
        for a in range(0, rows, 256):
            part = torch.exp(s["logits"][a:a + 256].double() - lse[a:a + 256, None])
            at = s["labels"][a:a + 256, None].clamp(min=0)
            hot = torch.zeros_like(part).scatter_(1, at, 1.0)
            d[a:a + 256] = coef[a:a + 256, None] * (hot - part)
        got["dlogits"] = d
    return got
