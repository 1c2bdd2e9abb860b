"""The operators at the model's two ends on the GPU, against their plain forms
in 64 bits (tests/ops_reference.py), at the sizes, types and ids where they can
go wrong.  Every output lies between guard elements that have to stay as they
were.  Tolerances are the error bounds of ops_reference, one rounding counted
as half a step."""
import numpy as np
import pytest

from tests import ops_reference as R
from tests.ops_reference import BF16, F16, F32, U

pytestmark = pytest.mark.gpu
GUARD = 37


def say(msg):
    print(msg, flush=True)


class Guarded:
    """n elements of a type inside a larger buffer, at an odd offset, with a
    pattern around them."""

    def __init__(self, torch, dev, n, dtype, shift=1):
        self.torch, self.n, self.at = torch, n, GUARD + shift
        self.buf = torch.full((n + 2 * GUARD + shift,), 77, dtype=dtype, device=dev)
        self.t = self.buf[self.at:self.at + n]

    def check(self):
        assert bool((self.buf[:self.at] == 77).all()) and bool((self.buf[self.at + self.n:] == 77).all()), "guard"


def randn(torch, dev, rng, shape, dt, sigma=1.0):
    x = torch.from_numpy((rng.standard_normal(shape) * sigma).astype(np.float32))
    return x.to(R.torch_type(dt)).to(dev)


def make_ids(rng, n, rows, kind):
    if rows == 0:
        ids = rng.integers(-3, 5, n)
    elif kind == "uniform":
        ids = rng.integers(0, rows, n)
    elif kind == "skew":
        ids = np.minimum((rng.pareto(0.4, n) * 2).astype(np.int64), rows - 1)
    elif kind == "one":
        ids = np.full(n, rows // 2)
    elif kind == "padding":
        ids = np.full(n, -1)
    else:                       # wild: every kind of id outside the table too
        ids = rng.integers(0, rows, n)
        pick = rng.random(n)
        ids = np.where(pick < 0.1, -1, ids)
        ids = np.where((pick >= 0.1) & (pick < 0.15), rows, ids)
        ids = np.where((pick >= 0.15) & (pick < 0.2), np.iinfo(np.int32).max, ids)
        ids = np.where((pick >= 0.2) & (pick < 0.25), np.iinfo(np.int32).min, ids)
    return ids.astype(np.int64)


def as_ids(torch, dev, ids, wide, extra=True):
    """On the GPU as int64 or int32; int64 ids also hold values past 32 bits."""
    if wide and extra and len(ids) > 3:
        ids = ids.copy()
        ids[1], ids[2] = (1 << 40) + 1, -(1 << 40)
    t = torch.from_numpy(ids if wide else ids.astype(np.int32)).to(dev)
    return t, ids


def make_drop(Z, p, first=0, seed=(1 << 63) + 12345, site=3, step=9):
    return (None, None) if p is None else (Z.Drop(p, seed, site, step, first), (seed, site, step, p, first))


# ---------------------------------------------------------------------------
# Embedding lookup
# ---------------------------------------------------------------------------

EMBED = [
    # n, rows, hidden, table, out, p, before, gap, kind, wide
    (1, 5, 1, F32, F32, None, 0, 0, "uniform", True),
    (1, 50257, 768, BF16, BF16, None, 0, 0, "uniform", True),
    (0, 9, 8, BF16, BF16, 0.1, 0, 0, "uniform", True),
    (33, 0, 8, F16, F16, None, 3, 0, "wild", True),
    (257, 100, 3, F16, F16, 0.25, 1, 0, "wild", False),
    (130, 40, 7, BF16, BF16, 0.5, 5, 2, "wild", True),
    (130, 40, 8, BF16, BF16, 0.5, 5, 1, "skew", False),
    (99, 77, 9, F16, F16, None, 7, 0, "wild", True),
    (515, 1009, 65, F16, F16, 0.1, 33, 0, "wild", True),
    (300, 64, 768, BF16, BF16, 0.1, 0, 0, "wild", True),
    (70, 30, 1000, F32, F32, 0.3, 9, 24, "wild", False),
    (70, 30, 1001, F32, BF16, 0.3, 9, 0, "wild", True),
    (70, 30, 514, F16, F32, 0.3, 2, 5, "wild", True),
    (65, 30, 4096, BF16, F16, 0.1, 64, 0, "one", True),
    (40, 12, 2, BF16, F32, 1.0, 0, 0, "uniform", True),
    (9, 12, 66000, BF16, BF16, 0.0, 3, 0, "padding", True),
]


@pytest.mark.parametrize("case", EMBED, ids=lambda c: "-".join(map(str, c)))
def test_embed(gpu, zero_lib, case):
    import torch
    Z = zero_lib
    n, rows, hidden, tdt, odt, p, before, gap, kind, wide = case
    say(f"[embed] {case}")
    rng = np.random.default_rng(abs(hash(case[:3])) % 2 ** 31)
    plan = Z.zero_plan(before + rows * hidden + 11, 3, [before, rows * hidden, 11], 0, 1)
    params = randn(torch, gpu, rng, plan.psi_pad, tdt)
    ids_t, ids = as_ids(torch, gpu, make_ids(rng, n, rows, kind), wide)
    drop, spec = make_drop(Z, p, first=int(rng.integers(0, 9)) + (hidden % 2 << 40))
    stride = hidden + gap
    g = Guarded(torch, gpu, max(0, n * stride), R.torch_type(odt))
    out = g.t.view(n, stride)[:, :hidden]
    Z.zero_embed(plan, 1, hidden, params, tdt, ids_t, 1.7, out, odt, drop=drop)
    torch.cuda.synchronize()
    g.check()
    if gap and n:
        assert bool((g.t.view(n, stride)[:, hidden:] == 77).all())
    table = R.to64(params[before:before + rows * hidden]).reshape(rows, hidden)
    want = R.embed(table, ids, 1.7, spec)
    # the factor and the product round in fp32, then the result to its type
    R.check(R.to64(out), want, np.abs(want) * 3 * U + R.half_step(want * (1 + 3 * U), odt) + 2.0 ** -149, "embed")
    dropped = want == 0
    assert bool((R.to64(out)[dropped] == 0).all())


# ---------------------------------------------------------------------------
# Token order
# ---------------------------------------------------------------------------

ORDER = [(0, 10, "uniform"), (1, 1, "uniform"), (2, 3, "wild"), (31, 0, "wild"), (33, 1009, "wild"),
         (1000, 50257, "skew"), (8191, 50257, "wild"), (8192, 50257, "uniform"), (8193, 50257, "wild"),
         (5000, (1 << 19) - 1, "wild"), (5000, (1 << 19) - 2, "uniform"), (12289, 1, "wild"), (20000, 300000, "skew"),
         (70000, 511, "one"), (70000, 512, "skew"), (70001, (1 << 31) - 2, "wild"), (200003, 131072, "wild"),
         (1 << 20, 50257, "skew"), ((1 << 20) + 4097, 50257, "wild")]


@pytest.mark.parametrize("n,rows,kind", ORDER)
def test_token_order(gpu, zero_lib, n, rows, kind):
    import torch
    Z = zero_lib
    say(f"[order] n={n} rows={rows} {kind}")
    rng = np.random.default_rng(n + rows % 1000)
    ids_t, ids = as_ids(torch, gpu, make_ids(rng, n, rows, kind), n % 2 == 0 or kind != "wild" or rows > 1 << 30,
                        extra=kind == "wild")
    s, o = (Guarded(torch, gpu, n, torch.int32) for _ in range(2))
    need = Z.zero_token_order_workspace_bytes(n, rows)
    w = Guarded(torch, gpu, (need + 15) // 16 * 16, torch.uint8, shift=11)      # 48 bytes in: 16-byte aligned
    Z.zero_token_order(ids_t, rows, s.t, o.t, w.t)
    torch.cuda.synchronize()
    for g in (s, o, w):
        g.check()
    key = np.where((ids >= 0) & (ids < rows), ids, rows)
    want = np.argsort(key, kind="stable")
    assert np.array_equal(o.t.cpu().numpy(), want)
    assert np.array_equal(s.t.cpu().numpy(), key[want])


# ---------------------------------------------------------------------------
# Gradient of the table
# ---------------------------------------------------------------------------

def order_of(torch, Z, ids_t, rows):
    n = ids_t.numel()
    s, o = (torch.empty(n, dtype=torch.int32, device=ids_t.device) for _ in range(2))
    ws = torch.empty(max(1, Z.zero_token_order_workspace_bytes(n, rows)), dtype=torch.uint8, device=ids_t.device)
    Z.zero_token_order(ids_t, rows, s, o, ws)
    return s, o


GRAD = [
    # n, rows, hidden, dy, dst, p, before, gap, kind, n_d
    (0, 20, 8, BF16, BF16, None, 3, 0, "uniform", 2),
    (1, 5, 1, F32, F32, None, 0, 0, "uniform", 1),
    (37, 1009, 65, F16, F16, None, 33, 0, "wild", 2),
    (100, 20, 3, F16, F16, 0.5, 1, 1, "wild", 3),
    (100, 20, 4, BF16, F16, None, 2, 0, "skew", 3),
    (100, 20, 7, BF16, BF16, 0.5, 1, 1, "wild", 3),
    (64, 20, 8, BF16, BF16, 0.25, 1, 0, "one", 3),
    (65, 20, 9, F16, F32, 0.25, 1, 0, "one", 3),
    (8, 20, 16, F32, BF16, None, 0, 0, "one", 1),
    (9, 20, 16, F32, BF16, None, 0, 0, "one", 1),
    (50, 20, 16, F32, F32, 0.1, 5, 3, "padding", 2),
    (1000, 300, 256, BF16, BF16, 0.1, 0, 0, "wild", 4),
    (1000, 50, 768, BF16, BF16, 0.1, 0, 0, "skew", 4),
    (700, 50, 513, BF16, BF16, None, 7, 0, "skew", 4),
    (700, 50, 512, F16, F16, None, 7, 8, "wild", 5),
    (2000, 30, 1100, F16, F16, 0.3, 64, 0, "skew", 8),
    (9000, 2000, 40, BF16, F32, None, 64, 0, "wild", 8),
    (20000, 50, 96, BF16, BF16, 0.1, 0, 0, "one", 3),
    (3000, 4, 2050, F32, F32, None, 1, 0, "skew", 2),
]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("case", GRAD, ids=lambda c: "-".join(map(str, c)))
def test_embed_grad(gpu, zero_lib, case, accumulate):
    """The full buffer, then every owner's slice of it."""
    import torch
    Z = zero_lib
    n, rows, hidden, ydt, gdt, p, before, gap, kind, n_d = case
    say(f"[grad] {case} accumulate={accumulate}")
    rng = np.random.default_rng(n * 7 + hidden)
    plan = Z.zero_plan(before + rows * hidden + 11, n_d, [before, rows * hidden, 11], 0, 1 if hidden % 2 else 8)
    ids_t, ids = as_ids(torch, gpu, make_ids(rng, n, rows, kind), n % 3 != 0)
    wide = randn(torch, gpu, rng, (n, hidden + gap), ydt)
    dy = wide[:, :hidden]
    drop, spec = make_drop(Z, p, first=int(rng.integers(0, 9)) + (hidden % 2 << 40))
    s, o = order_of(torch, Z, ids_t, rows)
    ws = torch.empty(max(1, Z.zero_embed_grad_workspace_bytes(n, hidden)), dtype=torch.uint8, device=gpu)
    scale = 0.37
    want, bound = R.embed_grad(ids, R.to64(dy), rows, scale, spec)
    want, bound = want.ravel(), bound.ravel()
    present = np.repeat(np.isin(np.arange(rows), ids), hidden)
    (flat_off, numel, padded, share, _), = plan.buckets()
    for rank in [-1] + list(range(n_d)):
        size = plan.psi_pad if rank < 0 else plan.shard_total
        at = flat_off if rank < 0 else flat_off + rank * share          # flat position of dst[0]
        g = Guarded(torch, gpu, size, R.torch_type(gdt), shift=rank % 3 + 1)
        old = randn(torch, gpu, rng, size, gdt)
        g.t.copy_(old)
        Z.zero_embed_grad(plan, 1, hidden, s, o, dy, ydt, scale, g.t, gdt, drop=drop, rank=rank,
                          accumulate=accumulate, workspace=ws)
        torch.cuda.synchronize()
        g.check()
        got, old = R.to64(g.t), R.to64(old)
        lo, hi = max(at, before), min(at + size, before + rows * hidden)
        lo, hi = lo - at, max(lo, hi) - at
        assert np.array_equal(got[:lo], old[:lo]) and np.array_equal(got[hi:], old[hi:]), "outside the tensor"
        if hi <= lo:
            continue
        w, b, here = (v[lo + at - before:hi + at - before] for v in (want, bound, present))
        if accumulate:
            base = old[lo:hi]
            # the sum with the old value rounds once more in fp32
            tol = b + (np.abs(base) + np.abs(w) + b) * U + R.half_step(np.abs(base + w) + b, gdt)
            R.check(got[lo:hi], np.where(here, base + w, base), np.where(here, tol, 0.0), f"rank {rank}")
        else:
            R.check(got[lo:hi], w, np.where(here, b + R.half_step(np.abs(w) + b, gdt) + 2.0 ** -149, 0.0), f"rank {rank}")


@pytest.mark.parametrize("first", [0, 1, 4])
@pytest.mark.parametrize("hidden", [64, 66, 520])
def test_embed_and_grad_in_a_later_bucket(gpu, zero_lib, hidden, first):
    """A table whose bucket is not the plan's first, so that an owner's slice
    holds it behind other buckets' parts; masks that start a word and that do
    not."""
    import torch
    Z = zero_lib
    n, rows, n_d = 900, 60, 3
    rng = np.random.default_rng(hidden + first)
    sizes = [500, 33, rows * hidden, 77]
    plan = Z.zero_plan(sum(sizes), n_d, sizes, 540, 4)
    assert plan.tensor(2)[0] == 1 and plan.n_buckets == 3
    ids_t, ids = as_ids(torch, gpu, make_ids(rng, n, rows, "wild"), True)
    drop, spec = make_drop(Z, 0.3, first=first)
    params = randn(torch, gpu, rng, plan.psi_pad, BF16)
    off = plan.tensor(2)[1]
    y = torch.empty((n, hidden), dtype=torch.bfloat16, device=gpu)
    Z.zero_embed(plan, 2, hidden, params, BF16, ids_t, 0.5, y, BF16, drop=drop)
    want = R.embed(R.to64(params[off:off + rows * hidden]).reshape(rows, hidden), ids, 0.5, spec)
    R.check(R.to64(y), want, np.abs(want) * 3 * U + R.half_step(want * (1 + 3 * U), BF16), "embed")
    dy = randn(torch, gpu, rng, (n, hidden), F16)
    s, o = order_of(torch, Z, ids_t, rows)
    ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    want, bound = (v.ravel() for v in R.embed_grad(ids, R.to64(dy), rows, 0.5, spec))
    tol = bound + R.half_step(np.abs(want) + bound, F16)
    _, _, _, share, shard_off = plan.bucket(1)
    flat_off = plan.bucket(1)[0]
    for rank in range(n_d):
        dst = torch.full((plan.shard_total,), 5, dtype=torch.float16, device=gpu)
        Z.zero_embed_grad(plan, 2, hidden, s, o, dy, F16, 0.5, dst, F16, drop=drop, rank=rank, workspace=ws)
        got = R.to64(dst)
        at = flat_off + rank * share - off              # tensor element of the slice's part of this bucket
        lo, hi = max(0, at), min(rows * hidden, at + share)
        a, b = shard_off + lo - at, shard_off + hi - at
        R.check(got[a:b], want[lo:hi], tol[lo:hi], f"rank {rank}")
        assert (got[:a] == 5).all() and (got[b:] == 5).all()


def test_embed_grad_repeats_bit_for_bit(gpu, zero_lib):
    """The same inputs twice, the second time in a workspace full of other
    values and with NaN in the rows of padding ids."""
    import torch
    Z = zero_lib
    n, rows, hidden = 6000, 700, 384
    rng = np.random.default_rng(5)
    ids = make_ids(rng, n, rows, "skew")
    ids[::10] = -1
    ids_t, _ = as_ids(torch, gpu, ids, True, extra=False)
    plan = Z.zero_plan(rows * hidden, 2, [rows * hidden], 0, 8)
    dy = randn(torch, gpu, rng, (n, hidden), BF16)
    s, o = order_of(torch, Z, ids_t, rows)
    ws = torch.zeros(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    a = torch.zeros(plan.psi_pad, dtype=torch.bfloat16, device=gpu)
    Z.zero_embed_grad(plan, 0, hidden, s, o, dy, BF16, 1.0, a, BF16, workspace=ws)
    b = torch.full_like(a, 3)
    ws.fill_(255)
    dy[::10] = float("nan")
    Z.zero_embed_grad(plan, 0, hidden, s, o, dy, BF16, 1.0, b, BF16, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a[:rows * hidden].view(torch.int16), b[:rows * hidden].view(torch.int16))


SLICES = [
    # n, rows, hidden, dy, p, before, kind, n_d
    (8192, 5000, 768, F32, None, 0, "skew", 8),
    (8192, 300, 768, BF16, 0.1, 33, "uniform", 8),
    (16384, 3000, 2048, F32, 0.1, 7, "skew", 8),
    (65536, 5000, 512, F32, None, 0, "skew", 16),
    (20000, 40, 1601, F32, 0.3, 1, "skew", 3),
    (30001, 60000, 640, F32, None, 0, "wild", 64),
    (65536, 700, 2048, BF16, None, 64, "skew", 4),
    (40000, 900, 768, F32, 0.25, 0, "one", 2),
    (36000, 2000, 700, F32, None, 5, "skew", 64),             # chunks of 28, shared by three waves
    ((1 << 21) - 77, 5000, 8, F32, None, 1, "uniform", 128),     # chunks of 64, shared by four
]


@pytest.mark.parametrize("case", SLICES, ids=lambda c: "-".join(map(str, c)))
def test_embed_grad_slices_hold_the_bits_of_the_whole(gpu, zero_lib, case):
    """What each owner's slice receives is what the full buffer holds there,
    bit for bit in fp32, whether the waves share chunks or not; and the full
    buffer is right."""
    import torch
    Z = zero_lib
    n, rows, hidden, ydt, p, before, kind, n_d = case
    say(f"[slices] {case}")
    rng = np.random.default_rng(n + hidden)
    plan = Z.zero_plan(before + rows * hidden, n_d, [before, rows * hidden], 0, 1)
    ids = make_ids(rng, n, rows, kind)
    if kind == "skew":                       # a third of them over the whole table, in every owner's slice
        ids[::3] = rng.integers(0, rows, len(ids[::3]))
    ids_t, _ = as_ids(torch, gpu, ids, True, extra=False)
    dy = randn(torch, gpu, rng, (n, hidden), ydt)
    drop, spec = make_drop(Z, p, first=5)
    s, o = order_of(torch, Z, ids_t, rows)
    ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    full = torch.zeros(plan.psi_pad, device=gpu)
    Z.zero_embed_grad(plan, 1, hidden, s, o, dy, ydt, 0.7, full, F32, drop=drop, workspace=ws)
    S = plan.shard_total
    for rank in range(n_d):
        part = torch.zeros(S, device=gpu)
        Z.zero_embed_grad(plan, 1, hidden, s, o, dy, ydt, 0.7, part, F32, drop=drop, rank=rank, workspace=ws)
        assert torch.equal(part.view(torch.int32), full[rank * S:(rank + 1) * S].view(torch.int32)), rank
    sums = torch.arange(plan.psi_pad, device=gpu).remainder(97).float()          # added to a tied table's gradient
    old = sums.clone()
    Z.zero_embed_grad(plan, 1, hidden, s, o, dy, ydt, 0.7, sums, F32, drop=drop, accumulate=True, workspace=ws)
    for rank in range(n_d):
        part = old[rank * S:(rank + 1) * S].clone()
        Z.zero_embed_grad(plan, 1, hidden, s, o, dy, ydt, 0.7, part, F32, drop=drop, rank=rank, accumulate=True, workspace=ws)
        assert torch.equal(part.view(torch.int32), sums[rank * S:(rank + 1) * S].view(torch.int32)), rank
    cols = sorted({0, hidden // 2, hidden - 1})
    dyn = np.zeros((n, len(cols)))
    for k, c in enumerate(cols):             # columns of the definition: the mask's positions are of whole rows
        dyn[:, k] = R.to64(dy[:, c])
        if spec is not None:
            keep = np.concatenate([R.mask_block(*spec[:4], spec[4] + i * hidden + c, 1) for i in range(n)])
            dyn[:, k] = np.where(keep, dyn[:, k], 0.0)
    f = 0.7 * (R.keep_factor(p) if p else 1.0)
    want, bound = R.embed_grad(ids, dyn, rows, f, None)
    got = R.to64(full[before:before + rows * hidden].view(rows, hidden)[:, cols])
    R.check(got, want, bound + np.abs(want) * U + 2.0 ** -149, "columns")
    base = R.to64(old[before:before + rows * hidden].view(rows, hidden)[:, cols])
    got = R.to64(sums[before:before + rows * hidden].view(rows, hidden)[:, cols])
    R.check(got, base + want, bound + (2 * np.abs(want) + np.abs(base)) * 2 * U, "columns of the sum")


def test_embed_grad_against_differences(gpu, zero_lib):
    """The lookup is linear in the table: <dy, embed(T + D) - embed(T)> equals
    <grad, D> up to rounding, with the same dropout in both."""
    import torch
    Z = zero_lib
    n, rows, hidden = 500, 90, 70
    rng = np.random.default_rng(11)
    plan = Z.zero_plan(rows * hidden, 1, [rows * hidden], 0, 1)
    ids_t, ids = as_ids(torch, gpu, make_ids(rng, n, rows, "wild"), True)
    T, D = (rng.standard_normal(rows * hidden) for _ in range(2))
    T, D = np.round(T * 256) / 256, np.round(D * 256) / 256         # T + D is exact in fp32
    drop, _ = make_drop(Z, 0.2)
    y = [torch.empty((n, hidden), device=gpu) for _ in range(2)]
    for out, table in zip(y, (T, T + D)):
        Z.zero_embed(plan, 0, hidden, torch.from_numpy(table.astype(np.float32)).to(gpu), F32, ids_t, 2.5, out, F32,
                     drop=drop)
    dy = randn(torch, gpu, rng, (n, hidden), F32)
    s, o = order_of(torch, Z, ids_t, rows)
    ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    g = torch.empty(rows * hidden, device=gpu)
    Z.zero_embed_grad(plan, 0, hidden, s, o, dy, F32, 2.5, g, F32, drop=drop, workspace=ws)
    y0, y1, dyn, gn = R.to64(y[0]), R.to64(y[1]), R.to64(dy), R.to64(g)
    left, right = float((dyn * (y1 - y0)).sum()), float((gn * D).sum())
    # each lookup is off by 2 u of its value, each gradient by its bound
    _, bound = R.embed_grad(ids, dyn, rows, 2.5, (drop.c.seed, 3, 9, 0.2, 0))
    tol = float((np.abs(dyn) * 3 * U * (np.abs(y0) + np.abs(y1))).sum() + ((bound.ravel() + np.abs(gn) * U) * np.abs(D)).sum())
    assert abs(left - right) <= tol, (left, right, tol)


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------

DROPOUT = [(1, F32, 0.5, False, 0), (3, F16, 0.5, True, 3), (8, BF16, 0.1, True, 1), (9, BF16, 0.1, False, 2),
           (768, BF16, 0.1, False, 0), (2047, F16, 0.3, True, 5), (8192 * 3, BF16, 0.1, True, 0),
           (100003, F32, 0.25, True, (1 << 34) + 1), (100003, F16, 0.25, False, 4), (65537, BF16, 0.0, True, 2),
           (65537, BF16, 1.0, True, 2), (4099, F32, 1e-6, False, 2), (0, F32, 0.1, True, 0)]


@pytest.mark.parametrize("inplace", ["", "x", "residual"])
@pytest.mark.parametrize("n,dt,p,residual,first", DROPOUT)
def test_dropout(gpu, zero_lib, n, dt, p, residual, first, inplace):
    import torch
    Z = zero_lib
    if inplace == "residual" and not residual:
        residual = True
    say(f"[dropout] n={n} dt={dt} p={p} residual={residual} first={first} inplace={inplace}")
    rng = np.random.default_rng(n)
    bufs = [Guarded(torch, gpu, n, R.torch_type(dt), shift=k) for k in range(3)]
    x, r, out = (b.t for b in bufs)
    x.copy_(randn(torch, gpu, rng, n, dt))
    r.copy_(randn(torch, gpu, rng, n, dt))
    keep = R.mask_block(77, 1, 2, p, first, n)
    if n > 100 and p < 1:                       # what is dropped may hold anything
        bad = torch.from_numpy(np.flatnonzero(~keep)[:5]).to(gpu)
        x[bad] = float("nan")
    x64, r64 = R.to64(x), R.to64(r)
    dst = {"": out, "x": x, "residual": r}[inplace]
    Z.zero_dropout(x, r if residual else None, dst, dt, Z.Drop(p, 77, 1, 2, first))
    torch.cuda.synchronize()
    for b in bufs:
        b.check()
    y = np.where(keep, np.nan_to_num(x64) * R.keep_factor(p), 0.0)
    want = y + (r64 if residual else 0.0)
    tol = np.abs(y) * 3 * U + (np.abs(y) + np.abs(want)) * U * residual
    R.check(R.to64(dst), want, tol + R.half_step(np.abs(want) + tol, dt) + 2.0 ** -149, "dropout")
    if not residual:
        assert bool((R.to64(dst)[~keep] == 0).all())


def test_dropout_pieces_make_the_whole(gpu, zero_lib):
    """Three pieces of a tensor, each at its own position, give what one call
    gives, bit for bit; another step gives another mask."""
    import torch
    Z = zero_lib
    rng = np.random.default_rng(3)
    x = randn(torch, gpu, rng, 10007, F16)
    whole, parts, other = (torch.empty_like(x) for _ in range(3))
    Z.zero_dropout(x, None, whole, F16, Z.Drop(0.3, 1, 2, 3))
    for a, b in ((0, 1001), (1001, 1006), (1006, 10007)):
        Z.zero_dropout(x[a:b], None, parts[a:b], F16, Z.Drop(0.3, 1, 2, 3, first=a))
    Z.zero_dropout(x, None, other, F16, Z.Drop(0.3, 1, 2, 4))
    assert torch.equal(whole, parts) and not torch.equal(whole, other)


# ---------------------------------------------------------------------------
# Token log-probabilities and the gradient of the logits
# ---------------------------------------------------------------------------

LOGP = [
    # n, vocab, dtype, gap, wide labels
    (1, 1, F32, 0, True), (5, 2, BF16, 0, True), (7, 7, F16, 0, False), (7, 8, F16, 1, True), (3, 9, BF16, 0, True),
    (40, 1009, F16, 0, True), (40, 1009, F32, 3, False), (33, 5000, BF16, 24, True), (17, 16384, BF16, 0, True),
    (9, 16391, F32, 0, True), (6, 50257, F16, 0, True), (2, 131072, BF16, 0, True), (1, 131071, F32, 1, True),
    (1030, 300, BF16, 0, True), (1024, 8200, BF16, 0, False),
]


def make_logits(torch, dev, rng, n, vocab, dt, gap, wide):
    """Rows behind each other `gap` apart, one element into the buffer; labels
    of which about a fifth are not scored, the logits there NaN; some rows hold
    -inf and the type's lowest value."""
    stride = vocab + gap
    g = Guarded(torch, dev, n * stride, R.torch_type(dt))
    x = g.t.view(n, stride)[:, :vocab]
    x.copy_(randn(torch, dev, rng, (n, vocab), dt, 3.0))
    labels = rng.integers(0, vocab, n)
    for t in range(n):
        if n > 3 and t % 5 == 1:
            labels[t] = (-100, vocab, -1)[t % 3]
            x[t] = float("nan")
        elif t % 7 == 2 and vocab > 2:
            x[t, ::2] = float("-inf")
        elif t % 7 == 3 and vocab > 2:
            x[t, 1::2] = torch.finfo(R.torch_type(dt)).min
        elif t % 7 == 4:
            x[t, int(labels[t])] = 30.0
    labels = labels.astype(np.int64)
    return g, x, torch.from_numpy(labels if wide else labels.astype(np.int32)).to(dev), labels


@pytest.mark.parametrize("case", LOGP, ids=lambda c: "-".join(map(str, c)))
def test_token_logp_and_grad(gpu, zero_lib, case):
    import torch
    Z = zero_lib
    n, vocab, dt, gap, wide = case
    say(f"[logp] {case}")
    rng = np.random.default_rng(n + vocab)
    gx, x, lab_t, labels = make_logits(torch, gpu, rng, n, vocab, dt, gap, wide)
    lp, st = Guarded(torch, gpu, n, torch.float32), Guarded(torch, gpu, 2 * n, torch.float32)
    ws = torch.full((max(1, Z.zero_token_logp_workspace_bytes(n, vocab)),), 255, dtype=torch.uint8, device=gpu)
    Z.zero_token_logp(x, dt, lab_t, lp.t, st.t, ws)
    torch.cuda.synchronize()
    for g in (gx, lp, st):
        g.check()
    x64 = R.to64(x)
    top, ls, want = R.softmax_rows(x64, labels)
    e = R.logsum_bound(vocab)
    got_st = R.to64(st.t).reshape(n, 2)
    R.check(got_st[:, 0], top, 0.0, "max")
    R.check(got_st[:, 1], ls, e + np.abs(ls) * U, "log of the sum")
    # taken in fp64 from the fp32 sum, rounded once
    R.check(R.to64(lp.t), want, e + np.where(np.isfinite(want), np.abs(want), 0) * U * 2, "logp")

    # Gradient, into a buffer of its own (rows at another distance) and in place.
    scored = (labels >= 0) & (labels < vocab)
    coef = rng.standard_normal(n).astype(np.float32) * 5
    coef[::6] = 0
    co = torch.from_numpy(coef).to(gpu)
    p = np.zeros((n, vocab))
    rel = np.zeros((n, vocab))
    for t in np.flatnonzero(scored & (coef != 0)):
        with np.errstate(all="ignore"):
            z = x64[t] - top[t]
            p[t] = np.exp(z - ls[t])
            # x - max rounds (u |z|), minus the log sum again (u |z - ls|, and the
            # log sum's own error), the exponential 2 u and u for its argument
            a = np.where(np.isfinite(z), np.abs(z), 0) + np.abs(ls[t])
            rel[t] = (3 * a + 2 * a + 4) * U + e
    hot = np.zeros((n, vocab))
    hot[np.flatnonzero(scored), labels[scored]] = 1
    live = (scored & (coef != 0))[:, None]
    dwant = np.where(live, coef[:, None].astype(np.float64) * (hot - p), 0.0)
    tol = np.abs(coef)[:, None] * (p * np.minimum(rel, 1) + (hot + p) * 2 * U) * live
    # 2^-126: the exponential gives 0 below fp32's normal range
    tol = tol + live * (R.half_step(np.abs(dwant) + tol, dt) + np.abs(coef)[:, None] * 2.0 ** -126)
    gd = Guarded(torch, gpu, n * (vocab + 3), R.torch_type(dt), shift=2)
    d = gd.t.view(n, vocab + 3)[:, :vocab]
    Z.zero_token_logp_grad(x, dt, lab_t, st.t, co, d)
    torch.cuda.synchronize()
    gd.check()
    gx.check()
    assert bool((gd.t.view(n, vocab + 3)[:, vocab:] == 77).all())
    R.check(R.to64(d), dwant, tol, "dlogits")
    want_bits = d.clone()
    Z.zero_token_logp_grad(x, dt, lab_t, st.t, co, x)
    torch.cuda.synchronize()
    gx.check()
    assert torch.equal(x.contiguous().view(torch.uint8), want_bits.view(torch.uint8))


def test_token_logp_without_a_distribution(gpu, zero_lib):
    """A row of -inf alone, a row with NaN and one with +inf have no log
    probabilities (NaN); a row of the type's lowest value alone is uniform; the
    rows beside them are untouched by it."""
    import torch
    Z = zero_lib
    for dt in (F32, F16, BF16):
        for vocab in (5, 9000, 70000):
            say(f"[logp] special rows dt={dt} vocab={vocab}")
            x = torch.zeros((5, vocab), dtype=R.torch_type(dt), device=gpu)
            x[0] = float("-inf")
            x[1, vocab // 2] = float("nan")
            x[2, vocab - 1] = float("inf")
            x[3] = torch.finfo(R.torch_type(dt)).min
            labels = torch.full((5,), 1, dtype=torch.int64, device=gpu)
            lp, st = torch.empty(5, device=gpu), torch.empty(10, device=gpu)
            ws = torch.empty(max(1, Z.zero_token_logp_workspace_bytes(5, vocab)), dtype=torch.uint8, device=gpu)
            Z.zero_token_logp(x, dt, labels, lp, st, ws)
            d = torch.empty_like(x)
            Z.zero_token_logp_grad(x, dt, labels, st, torch.full((5,), 2.0, device=gpu), d)
            got = R.to64(lp)
            assert np.isnan(got[:3]).all(), got
            tol = R.logsum_bound(vocab) + np.log(vocab) * 2 * U
            assert np.all(np.abs(got[3:] + np.log(vocab)) <= tol), got
            d = R.to64(d)
            p = 1 / vocab
            for t in (3, 4):
                want = np.full(vocab, -2 * p)
                want[1] += 2
                R.check(d[t], want, np.abs(want) * 2 * (tol + 20 * U) + R.half_step(np.abs(want) * (1 + tol), dt), f"row {t}")


SURE = [(7, 9, 1), (12, 1009, 0), (9, 1009, 2), (7, 8200, 1), (6, 50257, 0), (5, 50257, 2), (3, 131071, 0), (4, 131072, 2),
        (1030, 300, 0)]


@pytest.mark.parametrize("n,vocab,dt", SURE)
def test_labels_that_are_almost_certain(gpu, zero_lib, n, vocab, dt):
    """Labels whose logit stands up to 90 above the others', at the row's ends
    and inside: the log-probability, the log of the sum and the label's
    gradient keep their relative accuracy, however close the probability is to
    1, and a row's gradient sums to zero."""
    import torch
    Z = zero_lib
    say(f"[sure] {n} x {vocab} dt={dt}")
    rng = np.random.default_rng(vocab + n)
    g = Guarded(torch, gpu, n * vocab, R.torch_type(dt))
    x = g.t.view(n, vocab)
    x.copy_(randn(torch, gpu, rng, (n, vocab), dt))
    labels = rng.integers(0, vocab, n)
    labels[:2] = 0, vocab - 1
    x[torch.arange(n), torch.from_numpy(labels).to(gpu)] = torch.tensor([6.0, 10, 14, 18, 22, 28, 40, 90])[np.arange(n) % 8].to(x.dtype).to(gpu)
    lab_t = torch.from_numpy(labels).to(gpu)
    lp, st, d = torch.empty(n, device=gpu), torch.empty(2 * n, device=gpu), torch.empty((n, vocab), dtype=x.dtype, device=gpu)
    ws = torch.empty(max(1, Z.zero_token_logp_workspace_bytes(n, vocab)), dtype=torch.uint8, device=gpu)
    coef = rng.standard_normal(n).astype(np.float32)
    Z.zero_token_logp(x, dt, lab_t, lp, st, ws)
    Z.zero_token_logp_grad(x, dt, lab_t, st, torch.from_numpy(coef).to(gpu), d)
    torch.cuda.synchronize()
    g.check()
    x64, coef = R.to64(x), coef.astype(np.float64)
    y = x64[np.arange(n), labels]
    others = x64.copy()
    others[np.arange(n), labels] = -np.inf
    with np.errstate(under="ignore"):
        rest = np.exp(others - y[:, None]).sum(1)
    top = np.maximum(y, others.max(1))
    ls = np.where(y == top, np.log1p(rest), np.log1p(rest) + (y - top))
    # the sum over the others is off by e of itself, and log1p and expm1 of it by
    # no more; each result rounds once, and 2^-149 is fp32's smallest step
    e = R.logsum_bound(vocab)
    R.check(R.to64(st).reshape(n, 2)[:, 1], ls, np.where(y == top, ls, 1 + np.abs(ls)) * (e + 2 * U) + 2.0 ** -149, "log of the sum")
    R.check(R.to64(lp), -np.log1p(rest), np.log1p(rest) * (e + 2 * U) * np.where(y == top, 1, 4) + 2.0 ** -149, "logp")
    want = coef * (rest / (1 + rest))
    # where the label is not the maximum, (x - max) - ls is rounded twice more
    rel = e + (8 + np.where(y == top, 0, 4 * (np.abs(y - top) + 1))) * U
    got = R.to64(d)
    R.check(got[np.arange(n), labels], want, np.abs(want) * rel + R.half_step(want * (1 + rel), dt) + 2.0 ** -126, "label")
    if dt == F32:
        off = got.sum(1)                      # in 64 bits, of entries that are off by their own rounding
        with np.errstate(under="ignore"):
            z = np.where(np.isfinite(others), np.abs(others - top[:, None]), 0)
            span = (np.exp(others - y[:, None]) / (1 + rest[:, None]) * z).sum(1)      # the exponents' roundings
        R.check(off, np.zeros(n), np.abs(coef) * (2 * rest / (1 + rest) * (rel + e + 16 * U) + 6 * U * span) + vocab * 2.0 ** -126, "row sum")


def test_labels_on_special_logits(gpu, zero_lib):
    """Labels whose own logit is NaN or +inf (no log-probability), -inf beside
    finite ones, and finite beside nothing but -inf (probability 1)."""
    import torch
    Z = zero_lib
    for dt in (F32, F16, BF16):
        for vocab in (1, 2, 5, 1001, 9000, 70001):
            say(f"[logp] special labels dt={dt} vocab={vocab}")
            at = vocab // 2
            x = torch.zeros((5, vocab), dtype=R.torch_type(dt), device=gpu)
            x[0, at] = float("nan")
            x[1, at] = float("inf")
            x[2, at] = float("-inf")
            x[3] = float("-inf")
            x[3, at] = -3.0
            x[4, at] = torch.finfo(R.torch_type(dt)).min
            labels = torch.full((5,), at, dtype=torch.int64, device=gpu)
            lp, st, d = torch.empty(5, device=gpu), torch.empty(10, device=gpu), torch.empty_like(x)
            ws = torch.empty(max(1, Z.zero_token_logp_workspace_bytes(5, vocab)), dtype=torch.uint8, device=gpu)
            Z.zero_token_logp(x, dt, labels, lp, st, ws)
            Z.zero_token_logp_grad(x, dt, labels, st, torch.full((5,), 2.0, device=gpu), d)
            got, d = R.to64(lp), R.to64(d)
            assert np.isnan(got[:2]).all() and np.isnan(d[0]).all() and np.isnan(d[1, at]), got
            assert got[3] == 0 and not d[3].any()
            if vocab == 1:                       # nothing but -inf, and one finite logit
                assert np.isnan(got[2]) and got[4] == 0 and d[4, 0] == 0
                continue
            want = R.to64(x[4, at]).item() - np.log(vocab - 1)
            assert got[2] == -np.inf and abs(got[4] - want) <= abs(want) * 2 * U + R.logsum_bound(vocab), got
            p = np.full(vocab, -2 / (vocab - 1))
            p[at] = 2
            for t in (2, 4):                     # exp of fp16's lowest value is 0 in fp32
                tol = np.abs(p) * (R.logsum_bound(vocab) + 24 * U)
                R.check(d[t], p, tol + R.half_step(np.abs(p) + tol, dt), f"row {t}")


# ---------------------------------------------------------------------------
# Preference loss
# ---------------------------------------------------------------------------

PREF = [
    # lengths (chosen, then rejected), rows before, rows behind, beta, smoothing, grad scale, ref, labels, wide
    ([3], [2], 0, 0, 0.1, 0.0, 1.0, True, True, True),
    ([0], [5], 0, 0, 0.5, 0.1, 2.0, True, True, False),
    ([0, 0], [0, 0], 3, 4, 0.5, 0.1, 2.0, True, True, True),
    ([], [], 0, 6, 0.5, 0.1, 2.0, True, True, True),
    ([1, 700, 63], [64, 1030, 5], 2, 9, 0.1, 0.05, 1024.0, True, True, True),
    ([40] * 20, [37] * 20, 0, 1, 0.3, 0.5, 1.0, False, True, False),
    ([40, 2], [37, 1], 0, 1, 30.0, 0.0, 1.0, True, False, True),
    ([400], [370], 0, 0, 3.0, 1.0, -4.0, True, False, True),
    ([2500], [1025], 5, 0, 0.0, 0.2, 1.0, True, True, True),
]


@pytest.mark.parametrize("case", PREF, ids=lambda c: str(len(c[0])) + "-" + "-".join(map(str, c[2:])))
def test_preference_loss(gpu, zero_lib, case):
    import torch
    Z = zero_lib
    chosen, rejected, before, behind, beta, eps, gs, with_ref, with_labels, wide = case
    say(f"[preference] {case}")
    rng = np.random.default_rng(len(chosen) + behind)
    pairs, vocab = len(chosen), 10
    offsets = np.cumsum([before] + list(chosen) + list(rejected)) if pairs else np.array([before])
    n = int(offsets[-1]) + behind
    labels = rng.integers(0, vocab, n)
    labels[rng.random(n) < 0.3] = -100
    logp, ref = (-rng.random(n).astype(np.float32) * 9 for _ in range(2))
    counted = labels >= 0 if with_labels else np.ones(n, bool)
    logp_in, ref_in = logp.copy(), ref.copy()
    logp_in[~counted] = np.nan                       # what does not count may hold anything
    ref_in[~counted] = np.inf
    it = torch.int64 if wide else torch.int32
    outs = [Guarded(torch, gpu, k, torch.float32) for k in (1, pairs, 2 * pairs, n)]
    loss, pair, rewards, coef = (g.t for g in outs)
    Z.zero_preference_loss(torch.from_numpy(offsets).to(it).to(gpu),
                           torch.from_numpy(labels).to(it).to(gpu) if with_labels else None, vocab,
                           torch.from_numpy(logp_in).to(gpu), torch.from_numpy(ref_in).to(gpu) if with_ref else None,
                           beta, eps, gs, loss, pair, rewards, coef)
    torch.cuda.synchronize()
    for g in outs:
        g.check()
    w_loss, w_pair, w_rew, w_coef = R.preference(offsets, counted, logp.astype(np.float64),
                                                 ref.astype(np.float64) if with_ref else None, beta, eps, gs)
    # fp64 inside (2^-40 of the summed magnitudes is far above its error and
    # far below fp32), rounded once; the mean takes the rounded pair losses
    slack = 2.0 ** -40 * (1 + abs(beta)) * (18.0 * max(chosen + rejected + [1]))
    R.check(R.to64(rewards), w_rew, np.abs(w_rew) * U + slack, "rewards")
    R.check(R.to64(pair), w_pair, np.abs(w_pair) * U + slack + 2.0 ** -149, "pair losses")
    R.check(R.to64(loss), np.array([w_loss]), abs(w_loss) * 2 * U + slack + 2.0 ** -149, "loss")
    R.check(R.to64(coef), w_coef, np.abs(w_coef) * (U + slack) + 2.0 ** -149, "coef")


def test_preference_offsets_are_held_to_the_rows(gpu, zero_lib):
    """Offsets outside [0, n], or descending, neither read nor write outside."""
    import torch
    Z = zero_lib
    n = 50
    logp = torch.full((n,), -1.0, device=gpu)
    for offs in ([-5, 20, 10 ** 12], [30, 10, 60], [60, 70, 80], [-9, -8, -7]):
        outs = [Guarded(torch, gpu, k, torch.float32) for k in (1, 1, 2, n)]
        Z.zero_preference_loss(torch.tensor(offs, device=gpu), None, 1, logp, None, 0.1, 0.0, 1.0, *(g.t for g in outs))
        torch.cuda.synchronize()
        for g in outs:
            g.check()
        if offs == [-5, 20, 10 ** 12]:
            r = R.to64(outs[2].t)
            assert np.allclose(r, [-2.0, -3.0], atol=1e-6)


def loss_of(torch, Z, x, dt, labels, offsets, ref, beta, eps):
    n, vocab = x.shape
    dev = x.device
    lp, st, co = (torch.empty(k, device=dev) for k in (n, 2 * n, n))
    loss, pair, rew = (torch.empty(k, device=dev) for k in (1, len(offsets) // 2, len(offsets) - 1))
    ws = torch.empty(max(1, Z.zero_token_logp_workspace_bytes(n, vocab)), dtype=torch.uint8, device=dev)
    Z.zero_token_logp(x, dt, labels, lp, st, ws)
    Z.zero_preference_loss(offsets, labels, vocab, lp, ref, beta, eps, 1.0, loss, pair, rew, co)
    return loss, lp, st, co


def test_preference_gradient_against_differences(gpu, zero_lib):
    """The loss along a direction, by central differences of the kernels' own
    losses, against the kernels' gradient; the truncation of the difference is
    taken from the same difference in 64 bits."""
    import torch
    Z = zero_lib
    rng = np.random.default_rng(8)
    lens, vocab, beta, eps = [6, 4, 5, 7], 40, 0.7, 0.1
    offsets = np.cumsum([0] + lens)
    n = int(offsets[-1])
    labels = rng.integers(0, vocab, n)
    labels[[2, 9]] = -1
    x0 = np.round(rng.standard_normal((n, vocab)) * 64) / 64
    ref = (-np.log(vocab) + 0.2 * rng.standard_normal(n)).astype(np.float32)
    off_t, lab_t = torch.from_numpy(offsets).to(gpu), torch.from_numpy(labels).to(gpu)
    ref_t = torch.from_numpy(ref).to(gpu)

    def kernel(x):
        return loss_of(torch, Z, torch.from_numpy(x.astype(np.float32)).to(gpu), F32, lab_t, off_t, ref_t, beta, eps)

    def plain(x):
        _, _, lp = R.softmax_rows(x, labels)
        return R.preference(offsets, labels >= 0, lp, ref.astype(np.float64), beta, eps, 1.0)[0]

    loss, lp, st, co = kernel(x0)
    d = torch.empty((n, vocab), device=gpu)
    Z.zero_token_logp_grad(torch.from_numpy(x0.astype(np.float32)).to(gpu), F32, lab_t, st, co, d)
    d = R.to64(d)
    # 64-bit gradient of the same formula, for the truncation alone
    top, ls, _ = R.softmax_rows(x0, labels)
    h = 2.0 ** -4
    for k in range(4):
        v = np.round(rng.standard_normal((n, vocab)) * 8) / 8
        v[labels < 0] = 0
        num = float(R.to64(kernel(x0 + h * v)[0])[0] - R.to64(kernel(x0 - h * v)[0])[0]) / (2 * h)
        num64 = (plain(x0 + h * v) - plain(x0 - h * v)) / (2 * h)
        fine = (plain(x0 + 2.0 ** -14 * v) - plain(x0 - 2.0 ** -14 * v)) / 2.0 ** -13
        trunc = num64 - fine                           # fine's own truncation is 2^-20 of it
        # a loss is off by 2 u of itself and by beta / pairs times the rows' errors
        noise = 2 * (2 * U * 2.0 + beta / 2 * n * (R.logsum_bound(vocab) + 8 * U)) / (2 * h)
        own = float((d * v).sum())
        slack = float((np.abs(v) * (np.abs(d) * 64 * U)).sum()) + abs(trunc) * 2.0 ** -18 + 1e-9
        assert abs(num - (own + trunc)) <= noise + slack, (k, num, own, trunc, noise)


# ---------------------------------------------------------------------------
# Graphs, streams, and the operators together
# ---------------------------------------------------------------------------

def test_graph_replays(gpu, zero_lib):
    """All operators captured once: each replay, with eager work in between and
    the step number changed on the device, gives what the eager calls give."""
    import torch
    Z = zero_lib
    rng = np.random.default_rng(21)
    n, rows, hidden, vocab = 9000, 300, 96, 1500
    plan = Z.zero_plan(rows * hidden, 2, [rows * hidden], 0, 8)
    params = randn(torch, gpu, rng, plan.psi_pad, BF16)
    ids_t, _ = as_ids(torch, gpu, make_ids(rng, n, rows, "skew"), True)
    step = torch.zeros(1, dtype=torch.int64, device=gpu)
    drop = Z.Drop(0.2, 5, 6, step_dev=step)
    logits = randn(torch, gpu, rng, (60, vocab), F16, 2.0)
    labels = torch.from_numpy(rng.integers(-1, vocab, 60)).to(gpu)
    offsets = torch.tensor([0, 10, 30, 45, 58], device=gpu)
    need = max(Z.zero_token_order_workspace_bytes(n, rows), Z.zero_embed_grad_workspace_bytes(n, hidden),
               Z.zero_token_logp_workspace_bytes(60, vocab), 1)

    def buffers():
        e = lambda *s, dt=torch.float32: torch.zeros(s, dtype=dt, device=gpu)  # noqa: E731
        return dict(y=e(n, hidden, dt=torch.bfloat16), z=e(n, hidden, dt=torch.bfloat16), s=e(n, dt=torch.int32),
                    o=e(n, dt=torch.int32), g=e(plan.psi_pad, dt=torch.bfloat16), lp=e(60), st=e(120), loss=e(1),
                    pl=e(2), rw=e(4), co=e(60), d=e(60, vocab, dt=torch.float16), ws=e(need, dt=torch.uint8))

    def go(b):
        Z.zero_embed(plan, 0, hidden, params, BF16, ids_t, 2.0, b["y"], BF16, drop=drop)
        Z.zero_dropout(b["y"], b["y"], b["z"], BF16, drop)
        Z.zero_token_order(ids_t, rows, b["s"], b["o"], b["ws"])
        Z.zero_embed_grad(plan, 0, hidden, b["s"], b["o"], b["z"], BF16, 2.0, b["g"], BF16, drop=drop, workspace=b["ws"])
        Z.zero_token_logp(logits, F16, labels, b["lp"], b["st"], b["ws"])
        Z.zero_preference_loss(offsets, labels, vocab, b["lp"], None, 0.1, 0.1, 8.0, b["loss"], b["pl"], b["rw"], b["co"])
        Z.zero_token_logp_grad(logits, F16, labels, b["st"], b["co"], b["d"])

    eager, graphed = buffers(), buffers()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(graphed)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(graphed)
    seen = []
    for rep in range(4):
        step.fill_(rep // 2)
        graph.replay()
        go(eager)
        torch.cuda.synchronize()
        for k in eager:
            if k != "ws":
                assert torch.equal(eager[k].view(torch.uint8), graphed[k].view(torch.uint8)), (rep, k)
        seen.append(eager["y"].clone())
        graphed["g"].fill_(1)
        logits.add_(0.125)
    assert torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_an_error_left_by_another_call_is_not_reported(gpu, zero_lib):
    """A runtime error that some other part of the program left pending (here a
    device number that does not exist) is neither returned nor cleared."""
    import ctypes
    import torch
    Z = zero_lib
    hip = ctypes.CDLL(next(line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line))
    x = torch.ones(1000, device=gpu)
    out, lp, st, co = torch.empty(1000, device=gpu), torch.empty(2, device=gpu), torch.empty(4, device=gpu), torch.empty(2, device=gpu)
    ids, lab = torch.zeros(10, dtype=torch.int64, device=gpu), torch.zeros(2, dtype=torch.int64, device=gpu)
    s, o = torch.empty(10, dtype=torch.int32, device=gpu), torch.empty(10, dtype=torch.int32, device=gpu)
    plan = Z.zero_plan(1000, 1, [1000], 0, 1)
    ws = torch.empty(4096, dtype=torch.uint8, device=gpu)
    y = torch.empty((10, 10), device=gpu)
    off = torch.tensor([0, 1, 2], device=gpu)
    one, pl, two = (torch.empty(k, device=gpu) for k in (1, 1, 2))
    torch.cuda.synchronize()
    stream = int(torch.cuda.current_stream().cuda_stream)
    assert hip.hipSetDevice(12345) != 0
    try:
        Z.zero_dropout(x, None, out, F32, Z.Drop(0.5, 1), stream=stream)
        Z.zero_embed(plan, 0, 10, x, F32, ids, 2.0, y, F32, stream=stream)
        Z.zero_token_order(ids, 100, s, o, stream=stream)
        Z.zero_embed_grad(plan, 0, 10, s, o, y, F32, 1.0, out, F32, workspace=ws, stream=stream)
        Z.zero_token_logp(x.view(2, 500), F32, lab, lp, st, stream=stream)
        Z.zero_preference_loss(off, lab, 500, lp, None, 0.1, 0.0, 1.0, one, pl, two, co, stream=stream)
        Z.zero_token_logp_grad(x.view(2, 500), F32, lab, st, co, out.view(2, 500), stream=stream)
    finally:
        pending = hip.hipGetLastError()
        torch.cuda.synchronize()
    assert pending != 0
    assert bool((y == 2).all())


def test_two_streams(gpu, zero_lib):
    """Two gradients at once, each on its own stream with its own workspace."""
    import torch
    Z = zero_lib
    rng = np.random.default_rng(22)
    n, rows, hidden = 5000, 100, 512
    plan = Z.zero_plan(rows * hidden, 1, [rows * hidden], 0, 8)
    ids_t, _ = as_ids(torch, gpu, make_ids(rng, n, rows, "skew"), True)
    ys = [randn(torch, gpu, rng, (n, hidden), BF16) for _ in range(2)]
    need = max(Z.zero_token_order_workspace_bytes(n, rows), Z.zero_embed_grad_workspace_bytes(n, hidden))

    def go(y, ws, s, o, g, stream):
        Z.zero_token_order(ids_t, rows, s, o, ws, stream=stream)
        Z.zero_embed_grad(plan, 0, hidden, s, o, y, BF16, 1.0, g, BF16, workspace=ws, stream=stream)

    def bufs():
        return (torch.empty(need, dtype=torch.uint8, device=gpu), torch.empty(n, dtype=torch.int32, device=gpu),
                torch.empty(n, dtype=torch.int32, device=gpu), torch.zeros(plan.psi_pad, dtype=torch.bfloat16, device=gpu))
    alone = []
    for y in ys:
        b = bufs()
        go(y, *b, None)
        alone.append(b[3])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [bufs() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for y, b, s in zip(ys, sets, streams):
            go(y, *b, s)
    torch.cuda.synchronize()
    for a, b in zip(alone, sets):
        assert torch.equal(a, b[3])


def test_a_training_step_from_tokens_to_parameters(gpu, zero_lib):
    """The operators as one step uses them, with a table that is also the
    output matrix: lookup and dropout, logits against the table, the
    preference loss, its gradient back through both uses of the table into
    each rank's flat gradient buffer, and the owner's Adam step on the sum.
    Against the same step in 64 bits."""
    import torch
    Z = zero_lib
    rng = np.random.default_rng(31)
    n_d, rows, hidden, other = 2, 90, 32, 13
    sizes = [rows * hidden, other]
    plan = Z.zero_plan(sum(sizes), n_d, sizes, 0, 8)
    lens, beta, eps, gs = [9, 12, 8, 11], 0.5, 0.05, 64.0
    offsets = np.cumsum([0] + lens)
    n = int(offsets[-1])
    w = np.zeros(plan.psi_pad, np.float32)
    w[:sum(sizes)] = (rng.standard_normal(sum(sizes)) * 0.3).astype(np.float32)
    params = torch.from_numpy(w).to(gpu)                       # an fp32 copy of the parameters
    table64 = w[:rows * hidden].astype(np.float64).reshape(rows, hidden)
    off_t = torch.from_numpy(offsets).to(gpu)
    contributions, total64 = [], np.zeros((rows, hidden))
    for rank in range(n_d):
        ids = make_ids(rng, n, rows, "uniform")
        ids[3] = -1
        labels = rng.integers(0, rows, n)
        labels[[0, 10]] = -100
        ids_t, lab_t = torch.from_numpy(ids).to(gpu), torch.from_numpy(labels).to(gpu)
        drop = Z.Drop(0.2, 100 + rank, 1, 1)
        f32 = lambda *s: torch.empty(s, device=gpu)  # noqa: E731
        h = f32(n, hidden)
        Z.zero_embed(plan, 0, hidden, params, F32, ids_t, 4.0, h, F32, drop=drop)
        table = params[:rows * hidden].view(rows, hidden)
        x = h @ table.t()
        lp, st, co, loss, pl, rw = f32(n), f32(2 * n), f32(n), f32(1), f32(2), f32(4)
        ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
        Z.zero_token_logp(x, F32, lab_t, lp, st)
        Z.zero_preference_loss(off_t, lab_t, rows, lp, None, beta, eps, gs, loss, pl, rw, co)
        Z.zero_token_logp_grad(x, F32, lab_t, st, co, x)       # in place
        dh = x @ table
        flat = torch.zeros(plan.psi_pad, device=gpu)
        flat[:rows * hidden] = (x.t() @ h).reshape(-1)
        s, o = order_of(torch, Z, ids_t, rows)
        Z.zero_embed_grad(plan, 0, hidden, s, o, dh, F32, 4.0, flat, F32, drop=drop, accumulate=True, workspace=ws)
        contributions.append(flat.to(torch.bfloat16))
        # the same in 64 bits
        spec = (100 + rank, 1, 1, 0.2, 0)
        h64 = R.embed(table64, ids, 4.0, spec)
        x64 = h64 @ table64.T
        top, ls, lp64 = R.softmax_rows(x64, labels)
        good = labels >= 0
        l64, _, _, c64 = R.preference(offsets, good, lp64, None, beta, eps, gs)
        hot = np.zeros((n, rows))
        hot[np.flatnonzero(good), labels[good]] = 1
        d64 = c64[:, None] * (hot - np.exp(x64 - top[:, None] - ls[:, None]) * good[:, None])
        g64, _ = R.embed_grad(ids, d64 @ table64, rows, 4.0, spec)
        g64 = g64 + d64.T @ h64
        assert abs(float(loss) - l64) < 1e-5 * max(1, abs(l64))
        got = R.to64(flat[:rows * hidden]).reshape(rows, hidden)
        # fp32 throughout: logits of 32 products of size up to ~20 are off by
        # 32 * 20 u, which the softmax carries on relatively; sums of n terms
        assert np.linalg.norm(got - g64) <= 2000 * U * np.linalg.norm(g64)
        total64 += g64
    owner = 0
    S = plan.shard_total
    master = params[:S].clone()
    m, v = torch.zeros(S, device=gpu), torch.zeros(S, device=gpu)
    full = torch.zeros(plan.psi_pad, dtype=torch.float16, device=gpu)
    src = Z.GradSrc(BF16, contributions, [1, 1])
    Z.zero_adam_step(plan, owner, 1e-2, 0.9, 0.999, 1e-8, 1.0 / (n_d * gs), 1, src, None, master, m, v, full, F16, True)
    torch.cuda.synchronize()
    mean = (R.to64(contributions[0]) + R.to64(contributions[1]))[:S] / (n_d * gs)
    R.check(R.to64(m), 0.1 * mean, np.abs(mean) * 0.1 * 8 * U + np.max(np.abs(mean)) * 4 * U, "momentum")
    want = total64.ravel()[:S] / (n_d * gs)
    # each contribution was rounded to bf16 once
    assert np.linalg.norm(R.to64(m) / 0.1 - want) <= (2.0 ** -8 + 2000 * U) * np.linalg.norm(want) * 2
    moved = R.to64(master) - w[:S]
    big = np.abs(want) > 1e-3 * np.abs(want).max()
    assert np.all(np.sign(moved[big]) == -np.sign(want[big]))


# ---------------------------------------------------------------------------
# Offsets past 32 bits
# ---------------------------------------------------------------------------

@pytest.mark.big
def test_embed_and_grad_past_32_bits(gpu, zero_lib):
    """A table of 2.4e9 elements behind an odd-sized tensor: the rows that are
    named, the last ones among them, and zeros everywhere else."""
    import torch
    Z = zero_lib
    rows, hidden, before, n = 300_001, 8192, 5, 211
    say("[big] embed and its gradient")
    plan = Z.zero_plan(before + rows * hidden, 1, [before, rows * hidden], 0, 1)
    g = torch.Generator(device=gpu).manual_seed(1)
    buf = torch.empty(plan.psi_pad, dtype=torch.bfloat16, device=gpu).normal_(generator=g)
    ids = torch.randint(0, rows, (n,), generator=g, device=gpu)
    ids[:4] = torch.tensor([rows - 1, rows - 2, 0, rows], device=gpu)
    ids[100:130] = rows - 1
    good = ids < rows
    table = buf[before:].view(rows, hidden)
    out = torch.empty((n, hidden), dtype=torch.bfloat16, device=gpu)
    Z.zero_embed(plan, 1, hidden, buf, BF16, ids, 3.0, out, BF16)
    want = torch.where(good[:, None], table[ids.clamp(max=rows - 1)].float() * 3.0, 0.0).bfloat16()
    assert torch.equal(out, want)             # one product, one rounding: the same bits
    del table
    dy = torch.empty((n, hidden), dtype=torch.bfloat16, device=gpu).normal_(generator=g)
    buf.fill_(7)
    s, o = order_of(torch, Z, ids, rows)
    ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    Z.zero_embed_grad(plan, 1, hidden, s, o, dy, BF16, 1.0, buf, BF16, workspace=ws)
    torch.cuda.synchronize()
    assert bool((buf[:before] == 7).all())
    grad = buf[before:].view(rows, hidden)
    named = torch.unique(ids[good])
    idn = ids.cpu().numpy()
    for r in named.tolist():
        rows_of = R.to64(dy[torch.from_numpy(np.flatnonzero(idn == r)).to(gpu)])
        w, mag = rows_of.sum(0), np.abs(rows_of).sum(0)
        tol = mag * (len(rows_of) * 1.01 + 3) * U
        R.check(R.to64(grad[r]), w, tol + R.half_step(np.abs(w) + tol, BF16), f"row {r}")
    grad[named] = 0
    assert not bool(torch.any(grad.view(torch.int16)))


@pytest.mark.big
def test_embed_grad_of_many_activations(gpu, zero_lib):
    """dy of 2.4e9 elements, a third of it one token: some columns at both ends
    against 64 bits."""
    import torch
    Z = zero_lib
    n, rows, hidden = 300_001, 1000, 8192
    say("[big] gradient of many activations")
    g = torch.Generator(device=gpu).manual_seed(2)
    dy = torch.empty((n, hidden), dtype=torch.bfloat16, device=gpu).normal_(generator=g)
    ids = torch.randint(-1, rows, (n,), generator=g, device=gpu)
    ids[::3] = 17
    plan = Z.zero_plan(rows * hidden, 1, [rows * hidden], 0, 1)
    s, o = order_of(torch, Z, ids, rows)
    ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    grad = torch.empty(plan.psi_pad, dtype=torch.float32, device=gpu)
    Z.zero_embed_grad(plan, 0, hidden, s, o, dy, BF16, 1.0, grad, F32, workspace=ws)
    cols = torch.tensor([0, 1, 255, 256, 4095, hidden - 9, hidden - 2, hidden - 1], device=gpu)
    want, bound = R.embed_grad(ids.cpu().numpy(), R.to64(dy[:, cols]), rows, 1.0, None)
    R.check(R.to64(grad[:rows * hidden].view(rows, hidden)[:, cols]), want, bound, "columns")


@pytest.mark.big
@pytest.mark.parametrize("hidden,dt,gdt,first,n_d", [(1024, BF16, BF16, 0, 1), (1024, F16, F16, 3, 1), (1536, BF16, F16, 4, 8),
                                                     (1030, BF16, BF16, 1, 1), (512, F32, BF16, 4, 1), (1024, BF16, BF16, None, 4)])
def test_embed_grad_past_the_caches(gpu, zero_lib, hidden, dt, gdt, first, n_d):
    """dy larger than the 256 MiB cache, which is read past it, into 16-bit
    gradients: masks that start a word and that do not, and none; some columns
    against 64 bits, of the full buffer and of an owner's slice."""
    import torch
    Z = zero_lib
    rows, before = 3000, 64
    n = (260 << 20) // (hidden * (4 if dt == F32 else 2)) + 77
    say(f"[big] gradient past the caches {n} x {hidden} dt={dt}")
    g = torch.Generator(device=gpu).manual_seed(5)
    dy = torch.empty((n, hidden), dtype=R.torch_type(dt), device=gpu).normal_(generator=g)
    ids = torch.randint(-1, rows, (n,), generator=g, device=gpu)
    ids[::4] = 17                            # one token in many chunks
    idn = ids.cpu().numpy()
    plan = Z.zero_plan(before + rows * hidden, n_d, [before, rows * hidden], 0, 8)
    drop, spec = (None, None) if first is None else make_drop(Z, 0.1, first=first)
    s, o = order_of(torch, Z, ids, rows)
    ws = torch.empty(Z.zero_embed_grad_workspace_bytes(n, hidden), dtype=torch.uint8, device=gpu)
    full = torch.empty(plan.psi_pad, dtype=R.torch_type(gdt), device=gpu)
    Z.zero_embed_grad(plan, 1, hidden, s, o, dy, dt, 0.03, full, gdt, drop=drop, workspace=ws)
    cols = [0, 1, 7, 255, 256, 511, hidden // 2 + 3, hidden - 9, hidden - 2, hidden - 1]
    part = R.to64(dy[:, torch.tensor(cols, device=gpu)])
    f = 0.03
    if spec is not None:
        at = spec[4] + np.arange(n)[:, None] * hidden + np.array(cols)[None]
        part, f = np.where(R.mask_at(*spec[:4], at), part, 0.0), f * R.keep_factor(0.1)
    want, bound = R.embed_grad(idn, part, rows, f, None)
    got = full[before:before + rows * hidden].view(rows, hidden)[:, torch.tensor(cols, device=gpu)]
    tol = bound + np.abs(want) * U
    R.check(R.to64(got), want, tol + R.half_step(np.abs(want) + tol, gdt), "columns")
    if n_d > 1:
        S = plan.shard_total
        for rank in (0, n_d - 1):
            mine = torch.zeros(S, dtype=full.dtype, device=gpu)
            Z.zero_embed_grad(plan, 1, hidden, s, o, dy, dt, 0.03, mine, gdt, drop=drop, rank=rank, workspace=ws)
            lo, hi = max(0, before - rank * S), min(S, before + rows * hidden - rank * S)
            assert torch.equal(mine[lo:hi], full[rank * S + lo:rank * S + hi]), rank


@pytest.mark.big
@pytest.mark.parametrize("n,vocab,dt", [(4100, 9001, BF16), (4096, 32767, F16), (4097, 8192, F32), (4095, 9001, BF16)])
def test_logp_of_many_middling_rows(gpu, zero_lib, n, vocab, dt):
    """Rows that one wave reads where there are 4096 of them (and a whole
    workgroup where there is one less), some against 64 bits."""
    import torch
    Z = zero_lib
    say(f"[big] logp {n} x {vocab} dt={dt}")
    g = torch.Generator(device=gpu).manual_seed(n)
    x = torch.empty((n, vocab), dtype=R.torch_type(dt), device=gpu).normal_(0, 2, generator=g)
    labels = torch.randint(0, vocab, (n,), generator=g, device=gpu)
    labels[5::9] = -100
    lp, st = torch.full((n,), 7.0, device=gpu), torch.full((2 * n,), 7.0, device=gpu)
    Z.zero_token_logp(x, dt, labels, lp, st)
    pick = sorted({0, 1, 2, 5, 63, 64, n // 2, n - 2, n - 1})
    lab = labels[pick].cpu().numpy()
    top, ls, want = R.softmax_rows(R.to64(x[pick]), lab)
    # one wave's threads see eight times as many groups as logsum_bound counts,
    # each a sum of 16 terms (or 8) and a change of the maximum at worst
    e = R.logsum_bound(vocab) + (vocab / 512 + 4) * (4 + np.log2(vocab + 1)) * U
    R.check(R.to64(st).reshape(n, 2)[pick, 0], top, 0.0, "max")
    R.check(R.to64(lp[pick]), want, e + np.abs(want) * 2 * U, "logp")
    whole = torch.where(labels >= 0, torch.log_softmax(x.float(), 1).gather(1, labels.clamp(min=0)[:, None])[:, 0], 0.0)
    assert float((lp - whole).abs().max()) <= 2 * (e + 32 * 2 * U)       # torch's fp32 form is off as much at most, by its own sums


@pytest.mark.big
def test_logits_past_32_bits(gpu, zero_lib):
    """2.6e9 logits: the first and the last rows, forward and in place backward."""
    import torch
    Z = zero_lib
    n, vocab = 20_003, 131_071
    say("[big] logits")
    g = torch.Generator(device=gpu).manual_seed(3)
    x = torch.empty((n, vocab), dtype=torch.bfloat16, device=gpu).normal_(0, 2, generator=g)
    labels = torch.randint(0, vocab, (n,), generator=g, device=gpu)
    lp, st = torch.empty(n, device=gpu), torch.empty(2 * n, device=gpu)
    Z.zero_token_logp(x, BF16, labels, lp, st)
    pick = [0, 1, 2, 16_383, 16_384, 16_385, n - 2, n - 1]       # 2^31 elements lie before row 16384
    x64, lab = R.to64(x[pick]), labels[pick].cpu().numpy()
    top, ls, want = R.softmax_rows(x64, lab)
    e = R.logsum_bound(vocab)
    R.check(R.to64(lp[pick]), want, e + np.abs(want) * 2 * U, "logp")
    Z.zero_token_logp_grad(x, BF16, labels, st, torch.ones(n, device=gpu), x)
    z = x64 - top[:, None]
    p = np.exp(z - ls[:, None])
    hot = np.zeros_like(p)
    hot[np.arange(len(pick)), lab] = 1
    d = hot - p
    tol = p * ((5 * (np.abs(z) + ls[:, None]) + 4) * U + e) + 2 * U * (hot + p)
    R.check(R.to64(x[pick]), d, tol + R.half_step(np.abs(d) + tol, BF16) + 2.0 ** -126, "dlogits")


@pytest.mark.big
def test_dropout_past_32_bits(gpu, zero_lib):
    import torch
    Z = zero_lib
    n = (1 << 31) + 1001
    say("[big] dropout")
    x = torch.ones(n, dtype=torch.bfloat16, device=gpu)
    Z.zero_dropout(x, None, x, BF16, Z.Drop(0.25, 9, 8, 7, first=3))
    torch.cuda.synchronize()
    for a in (0, (1 << 31) - 500, n - 1000):
        keep = R.mask_block(9, 8, 7, 0.25, 3 + a, 1000)
        want = torch.where(torch.from_numpy(keep), torch.tensor(4 / 3, dtype=torch.float32).bfloat16(), torch.zeros((), dtype=torch.bfloat16))
        assert torch.equal(x[a:a + 1000].cpu(), want)


# ---------------------------------------------------------------------------
# More work than one launch takes (2^32 work items)
# ---------------------------------------------------------------------------

@pytest.mark.big
def test_dropout_of_two_launches(gpu, zero_lib):
    """2^35 elements and some in place: around the place where the second
    launch begins, and at both ends."""
    import torch
    Z = zero_lib
    n = (1 << 35) + 1001
    say("[big] dropout of two launches")
    x = torch.ones(n, dtype=torch.bfloat16, device=gpu)
    Z.zero_dropout(x, None, x, BF16, Z.Drop(0.25, 9, 8, 7, first=3))
    torch.cuda.synchronize()
    for a in (0, (1 << 35) - 4096 - 500, n - 1000):
        keep = R.mask_block(9, 8, 7, 0.25, 3 + a, 1000)
        want = torch.where(torch.from_numpy(keep), torch.tensor(4 / 3, dtype=torch.float32).bfloat16(), torch.zeros((), dtype=torch.bfloat16))
        assert torch.equal(x[a:a + 1000].cpu(), want)


@pytest.mark.big
def test_embed_of_two_launches(gpu, zero_lib):
    """Rows of seven elements, each taken singly: 2^34 of them and more."""
    import torch
    Z = zero_lib
    rows, hidden = 5, 7
    n = ((1 << 34) + 5000) // hidden
    say("[big] embed of two launches")
    plan = Z.zero_plan(rows * hidden, 1, [rows * hidden], 0, 1)
    params = torch.arange(1, rows * hidden + 1, device=gpu).to(torch.bfloat16)
    ids = torch.randint(-1, rows, (n,), generator=torch.Generator(device=gpu).manual_seed(4), device=gpu, dtype=torch.int32)
    out = torch.empty((n, hidden), dtype=torch.bfloat16, device=gpu)
    Z.zero_embed(plan, 0, hidden, params, BF16, ids, 1.0, out, BF16, drop=Z.Drop(0.5, 9, 8, 7, first=2))
    torch.cuda.synchronize()
    for a in (0, n // 2 - 400, n // 2, n - 800):        # the launches take equal parts
        got, i = R.to64(out[a:a + 800]), ids[a:a + 800].cpu().numpy()
        table = np.arange(1, rows * hidden + 1, dtype=np.float64).reshape(rows, hidden)
        want = R.embed(table, i, 1.0, (9, 8, 7, 0.5, 2 + a * hidden))       # whole numbers up to 70: exact
        assert np.array_equal(got, want), a


@pytest.mark.big
def test_logits_of_two_launches(gpu, zero_lib):
    """2^26 rows of two logits and some more (2^26 is one launch of the forward
    pass and two of the gradient), all rows against 64 bits."""
    import torch
    Z = zero_lib
    n, vocab = (1 << 26) + 999, 2
    say("[big] logits of two launches")
    g = torch.Generator(device=gpu).manual_seed(6)
    x = torch.empty((n, vocab), dtype=torch.bfloat16, device=gpu).normal_(0, 2, generator=g)
    labels = torch.randint(-1, vocab, (n,), generator=g, device=gpu, dtype=torch.int32)
    coef = torch.empty(n, device=gpu).normal_(generator=g)
    lp, st = torch.full((n,), 7.0, device=gpu), torch.full((2 * n,), 7.0, device=gpu)
    keep = x.clone()
    Z.zero_token_logp(x, BF16, labels, lp, st)
    Z.zero_token_logp_grad(x, BF16, labels, st, coef, x)
    e = R.logsum_bound(vocab)
    for a in range(0, n, 1 << 24):
        z, lab, c = keep[a:a + (1 << 24)].double(), labels[a:a + (1 << 24)].long(), coef[a:a + (1 << 24)].double()
        good = lab >= 0
        at = lab.clamp(min=0)[:, None]
        logp = torch.log_softmax(z, 1)
        want = torch.where(good, logp.gather(1, at)[:, 0], 0.0)
        assert bool(((lp[a:a + (1 << 24)].double() - want).abs() <= e + want.abs() * 2 * U).all())
        hot = torch.zeros_like(z).scatter_(1, at, 1.0)
        p, span = logp.exp(), (z[:, :1] - z[:, 1:]).abs()
        want = torch.where(good[:, None], c[:, None] * (hot - p), 0.0)
        tol = c.abs()[:, None] * (p * ((5 * (span + 1) + 4) * U + e) + 2 * U * (hot + p))
        tol = tol + (want.abs() + tol) * 2.0 ** -8 + 2.0 ** -126        # one rounding to bf16
        assert bool(((x[a:a + (1 << 24)].double() - want).abs() <= tol * good[:, None]).all())


@pytest.mark.big
def test_preference_of_two_launches(gpu, zero_lib):
    """2^22 pairs and some of one or two rows each, all against 64 bits."""
    import torch
    Z = zero_lib
    pairs, beta, eps, gs = (1 << 22) + 77, 0.5, 0.1, 64.0
    say("[big] preference of two launches")
    g = torch.Generator(device=gpu).manual_seed(7)
    lens = torch.randint(1, 3, (2 * pairs,), generator=g, device=gpu)
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)]) + 3
    n = int(offsets[-1]) + 5
    logp = -torch.rand(n, generator=g, device=gpu) * 4
    loss, pl, rw, co = (torch.full((k,), 7.0, device=gpu) for k in (1, pairs, 2 * pairs, n))
    Z.zero_preference_loss(offsets, None, 1, logp, None, beta, eps, gs, loss, pl, rw, co)
    total = torch.cat([logp.new_zeros(1).double(), logp.double().cumsum(0)])
    reward = beta * (total[offsets[1:]] - total[offsets[:-1]])
    # the running total of 1.3e7 rows of up to 4 is off by its own roundings in 64 bits
    slack = 5e7 * 2.0 ** -50
    assert bool(((rw.double() - reward).abs() <= reward.abs() * U + slack).all())
    h = reward[:pairs] - reward[pairs:]
    want = -(1 - eps) * torch.nn.functional.logsigmoid(h) - eps * torch.nn.functional.logsigmoid(-h)
    assert bool(((pl.double() - want).abs() <= want * U + 2 * slack).all())
    assert abs(float(loss) - float(want.mean())) <= float(want.mean()) * 2 * U + 2 * slack
    slope = beta * gs / pairs * (eps * torch.sigmoid(h) - (1 - eps) * torch.sigmoid(-h))
    rows = torch.repeat_interleave(torch.cat([slope, -slope]), lens)
    assert bool(((co[3:-5].double() - rows).abs() <= rows.abs() * (U + 4 * slack) + 2.0 ** -126 + beta * gs / pairs * 2 * slack).all())
    assert not bool(co[:3].any()) and not bool(co[-5:].any())


# ---------------------------------------------------------------------------
# Seeded random sizes, types, ids and owners
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(8))
def test_random_cases(gpu, zero_lib, seed):
    """The tests above at drawn sizes, spread over their logarithm."""
    import math
    import random
    r = random.Random(1000 + seed)
    size = lambda hi: int(round(math.exp(r.uniform(0, math.log(hi)))))  # noqa: E731
    for _ in range(12):
        n, rows, hidden = size(6000), size(3000), size(1500)
        if r.random() < 0.4:
            hidden = max(8, hidden // 8 * 8)
        n, rows = min(n, max(1, 1500000 // hidden)), min(rows, max(1, 1500000 // hidden))
        kind = r.choice(["uniform", "skew", "one", "wild", "wild", "padding"])
        case = (n, rows, hidden, r.randrange(3), r.randrange(3), r.choice([None, None, 0.1, 0.5, 1.0]),
                r.choice([0, r.randrange(100)]), r.choice([0, 0, 3, 8]), kind)
        test_embed_grad(gpu, zero_lib, case + (r.randint(1, 5),), r.random() < 0.5)
        test_embed(gpu, zero_lib, case + (r.random() < 0.5,))
        test_token_order(gpu, zero_lib, size(60000), r.choice([size(100000), size(2 ** 31 - 2)]), kind)
        test_token_logp_and_grad(gpu, zero_lib, (size(60), size(9000), r.randrange(3), r.choice([0, 1, 5]), r.random() < 0.5))
        test_dropout(gpu, zero_lib, size(200000), r.randrange(3), r.choice([0.0, 0.1, 0.7]), r.random() < 0.5,
                     r.randrange(1 << 36), r.choice(["", "x", "residual"]))
        pairs = r.randint(1, 30)
        test_preference_loss(gpu, zero_lib, ([r.randrange(60) for _ in range(pairs)], [r.randrange(60) for _ in range(pairs)],
                                             r.randrange(4), r.randrange(4), 2 * r.random(), r.random(), r.uniform(-9, 9),
                                             r.random() < 0.5, r.random() < 0.5, r.random() < 0.5))
