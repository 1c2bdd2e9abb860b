"""Plain numpy forms, in 64 bits, of the operators at the model's two ends,
and the error bounds of their fp32 kernels.

Rounding: u = 2^-24 is half a step of fp32; a result in type t is off by
another eps(t) / 2 of itself, or half a step of the smallest subnormal."""
import math

import numpy as np

U = 2.0 ** -24
M64 = (1 << 64) - 1
GAMMA, MIX1, MIX2 = 0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB
F32, F16, BF16 = 0, 1, 2
NAMES = {F32: "float32", F16: "float16", BF16: "bfloat16"}


def torch_type(dt):
    import torch
    return getattr(torch, NAMES[dt])


def to64(t):
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(want, dt):
    """Half a step of type dt at each value of want."""
    import torch
    f = torch.finfo(torch_type(dt))
    return np.maximum(np.abs(want) * f.eps / 2, f.tiny * f.eps / 2)


def check(got, want, tol, what=""):
    """NaN where NaN is wanted, equal infinities, and within tol elsewhere."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN", np.argwhere(np.isnan(got) != np.isnan(want))[:4])
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), (what, "inf")
    fine = np.isfinite(want)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want) - np.broadcast_to(tol, want.shape)
    bad = fine & ~(off <= 0)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4],
                           np.broadcast_to(tol, want.shape)[bad][:4])


def mix64(z):
    z = ((z ^ (z >> 30)) * MIX1) & M64
    z = ((z ^ (z >> 27)) * MIX2) & M64
    return z ^ (z >> 31)


def drop_key(seed, site, step):
    k = seed & M64
    for f in (site, step):
        k = mix64(((k ^ (f & M64)) + GAMMA) & M64)
    return k


def cut_of(p):
    return round(p * 65536)


def keep_mask(seed, site, step, p, positions):
    """Which of the elements at these mask positions are kept (plain integers)."""
    key, cut, words, out = drop_key(seed, site, step), cut_of(p), {}, []
    for e in positions:
        g = int(e) // 4
        if g not in words:
            words[g] = mix64((key + (g + 1) * GAMMA) & M64)
        out.append((words[g] >> (16 * (int(e) % 4)) & 0xFFFF) >= cut)
    return np.array(out, bool)


def mask_block(seed, site, step, p, first, n):
    """The same for [first, first + n), vectorised."""
    a, b = first // 4, (first + n + 3) // 4
    with np.errstate(over="ignore"):
        z = np.arange(a + 1, b + 1, dtype=np.uint64) * np.uint64(GAMMA) + np.uint64(drop_key(seed, site, step))
        z = (z ^ (z >> np.uint64(30))) * np.uint64(MIX1)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(MIX2)
        z = z ^ (z >> np.uint64(31))
    return z.view(np.uint16)[first - 4 * a:first - 4 * a + n].astype(np.int64) >= cut_of(p)


def mask_at(seed, site, step, p, positions):
    """The same at an array of positions."""
    e = np.asarray(positions, np.int64)
    with np.errstate(over="ignore"):
        z = (e // 4 + 1).astype(np.uint64) * np.uint64(GAMMA) + np.uint64(drop_key(seed, site, step))
        z = (z ^ (z >> np.uint64(30))) * np.uint64(MIX1)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(MIX2)
        z = z ^ (z >> np.uint64(31))
    return (z >> (16 * (e % 4)).astype(np.uint64) & np.uint64(0xFFFF)).astype(np.int64) >= cut_of(p)


def keep_factor(p):
    cut = cut_of(p)
    return 65536.0 / (65536 - cut) if cut < 65536 else 0.0


def embed(table, ids, scale, drop):
    rows, hidden = table.shape
    good = (ids >= 0) & (ids < rows)
    out = np.zeros((len(ids), hidden))
    out[good] = table[ids[good]] * scale
    if drop is not None:
        seed, site, step, p, first = drop
        keep = mask_block(seed, site, step, p, first, out.size).reshape(out.shape)
        out = np.where(keep, out * keep_factor(p), 0.0)
    return out


def embed_grad(ids, dy, rows, scale, drop):
    """(gradient, error bound of its fp32 sums and factor)."""
    n, hidden = dy.shape
    f = scale
    if drop is not None:
        seed, site, step, p, first = drop
        keep = mask_block(seed, site, step, p, first, dy.size).reshape(dy.shape)
        dy, f = np.where(keep, dy, 0.0), f * keep_factor(p)
    good = (ids >= 0) & (ids < rows)
    g, mag, count = np.zeros((rows, hidden)), np.zeros((rows, hidden)), np.zeros(rows)
    np.add.at(g, ids[good], dy[good])
    np.add.at(mag, ids[good], np.abs(dy[good]))
    np.add.at(count, ids[good], 1)
    # k terms: at most k - 1 roundings of partial sums that the sum of the
    # absolute values bounds, in whatever grouping (n u / (1 - n u) form), then
    # the factor's own rounding and the product's.
    k = count[:, None] * U
    return g * f, abs(f) * mag * (k / (1 - k) + 3 * U)


def softmax_rows(x, labels):
    """(max, log of the sum, logp) of scored rows, 0 elsewhere."""
    n, v = x.shape
    top, ls, lp = np.zeros(n), np.zeros(n), np.zeros(n)
    for t in range(n):
        if not 0 <= labels[t] < v:
            continue
        with np.errstate(all="ignore"):
            top[t] = -np.inf if np.isnan(x[t]).all() else np.nanmax(x[t])
            s = np.exp(x[t] - top[t]).sum() if top[t] > -np.inf or np.isnan(x[t]).any() else 0.0
            ls[t] = np.log(s)
            lp[t] = (x[t, labels[t]] - top[t]) - ls[t]
    return top, ls, lp


def logsum_bound(v):
    """Error of log(sum): a term is off by 2 u (the exponential) and by u |t|
    for its argument t = z log2 e, whose mean over the distribution is at most
    log2 v; the sum takes v / 4096 + 32 additions in a thread (of 512 threads
    with 8 elements each, in groups of 32 at most), 6 across a wave and 8
    across the waves, and each change of the maximum scales it once more, at
    most as often as a group is taken; splits add at most 16."""
    groups = v / 4096 + 4
    terms = 2 + 2 * math.log2(v + 1) + (v / 512 + 33) + 14 + 16 + groups * (3 + math.log2(v + 1))
    return terms * U


def preference(offsets, counted, logp, ref, beta, eps, grad_scale):
    """(loss, pair losses, rewards, coef)."""
    pairs = (len(offsets) - 1) // 2
    ratio = np.where(counted, logp - (0.0 if ref is None else ref), 0.0)
    off = np.clip(offsets, 0, len(logp))
    rewards = np.array([beta * math.fsum(ratio[a:b]) for a, b in zip(off, off[1:])])
    h = rewards[:pairs] - rewards[pairs:]
    soft = lambda z: np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z)))  # noqa: E731
    sig = lambda z: np.exp(-soft(-z))                                 # noqa: E731
    pair = (1 - eps) * soft(-h) + eps * soft(h)
    slope = beta * grad_scale / max(1, pairs) * (eps * sig(h) - (1 - eps) * sig(-h))
    coef = np.zeros(len(logp))
    for i in range(pairs):
        coef[off[i]:off[i + 1]] = slope[i]
        coef[off[pairs + i]:off[pairs + i + 1]] = -slope[i]
    return pair.mean() if pairs else 0.0, pair, rewards, np.where(counted, coef, 0.0)
