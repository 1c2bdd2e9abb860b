"""The operators on the hidden matrices on the GPU, against their formulas in 64
bits, at the sizes, types, strides and values where they can go wrong.  Outputs
lie between guard elements that have to stay as they were.

Tolerances, with u = 2^-24 and h(t) half a step of the output type:
  a product of k terms     2 k u sum |x| |w|   (sums in fp32, in any order)
  an activation            1e-5 of its value (exp2's argument of up to 128 is
                           rounded to 2^-17, erfcx is within 1.2e-6), its slope
                           2e-5, and 1.2 times the error of its argument (no
                           activation or slope is steeper than 1.2)
  then h of the finished value
The orthogonalisation's are at its tests."""
import math

import numpy as np
import pytest

from tests import ops_reference as R
from tests.ops_reference import BF16, F16, F32, U

pytestmark = pytest.mark.gpu
GUARD = 24
NONE, RELU, GELU, GELU_TANH, SILU = range(5)


@pytest.fixture(scope="module")
def T(gpu):
    import torch
    return torch


@pytest.fixture()
def Z(zero_lib):
    return zero_lib


class Rows:
    """n rows of `width` elements, `stride` apart, `shift` elements into a
    buffer filled with 77."""

    def __init__(self, T, n, width, stride, dt, shift, values=None):
        self.n, self.width, self.stride, self.at = n, width, stride, GUARD + shift
        self.buf = T.full((self.at + max(1, n) * stride + GUARD,), 77, dtype=R.torch_type(dt), device="cuda")
        self.t = self.buf[self.at:].as_strided((n, width), (stride, 1))
        if values is not None:
            self.t.copy_(values)

    def check(self):
        copy = self.buf.clone()
        copy[self.at:].as_strided((self.n, self.width), (self.stride, 1)).fill_(77)
        assert bool((copy == 77).all()), "written outside the rows"


def randn(T, shape, dt, seed, sigma=1.0):
    g = T.Generator(device="cuda").manual_seed(seed)
    return T.empty(shape, dtype=R.torch_type(dt), device="cuda").normal_(0, sigma, generator=g)


def act64(T, kind, z):
    if kind == RELU:
        return T.where(z > 0, z, 0.0 * z)
    if kind == GELU:
        return z * 0.5 * T.special.erfc(-z * math.sqrt(0.5))       # 1 + erf would cancel in the tail
    if kind == GELU_TANH:
        return z * T.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == SILU:
        return z * T.sigmoid(z)
    return z


def slope64(T, kind, z):
    if kind == RELU:
        return (z > 0).double()
    z = z.detach().clone().requires_grad_(True)
    return T.autograd.grad(act64(T, kind, z).sum(), z)[0]


def ws_of(T, n):
    return T.full((max(1, n),), 0x7f, dtype=T.uint8, device="cuda")      # what an earlier call left: NaN


def h(T, want, dt):
    f = T.finfo(R.torch_type(dt))
    return T.clamp(want.abs() * (f.eps / 2), min=f.tiny * f.eps / 2)


def close(T, got, want, tol, what):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4].tolist(), want[bad][:4].tolist(),
                                 tol[bad][:4].tolist() if tol.shape == want.shape else tol)


# rows, in, out, before, dtype, act, bias, residual, pre, gap: the distance of rows beyond their width
LINEAR = [
    (1, 1, 1, 0, BF16, NONE, False, False, False, 0),
    (1, 768, 768, 0, BF16, NONE, True, True, False, 0),
    (3, 5, 7, 3, F16, GELU, True, True, True, 1),
    (17, 64, 64, 0, F16, RELU, True, False, True, 0),
    (33, 65, 129, 1, BF16, GELU_TANH, True, True, False, 3),
    (64, 128, 64, 0, F16, SILU, False, True, True, 8),
    (65, 72, 200, 8, BF16, GELU, True, True, True, 8),
    (127, 1000, 333, 5, F16, SILU, True, True, True, 0),
    (200, 264, 136, 0, BF16, NONE, False, False, True, 0),
    (2, 65536, 40, 0, BF16, GELU, True, True, True, 0),           # pieces of k
    (5, 20001, 33, 1, F16, GELU_TANH, True, True, True, 2),        # odd pieces of k
    (1000, 520, 1030, 2, BF16, GELU, True, True, True, 0),
    (2048, 768, 768, 0, F16, NONE, True, False, False, 0),
    (1025, 328, 50257, 0, BF16, NONE, False, False, False, 0),     # a tied table's logits, odd rows
    (2049, 2048, 2056, 0, BF16, SILU, True, True, False, 16),      # the largest tiles, ragged
    (100, 130, 134, 2, BF16, NONE, True, False, False, 2),         # rows 4-byte aligned, k inside a unit
    (600, 30, 1030, 0, F16, GELU, True, True, True, 0),            # k shorter than a stage
    (2050, 1090, 1042, 4, BF16, RELU, True, False, False, 6),
    (1500, 1201, 1301, 3, F16, NONE, True, False, False, 0),       # odd rows in the larger tiles
    (9, 3, 2, 0, BF16, NONE, False, False, False, 0),              # rows shorter than a unit
    (3001, 1201, 1301, 3, BF16, GELU, True, True, True, 0),        # odd rows, copied first
    (3001, 1200, 1301, 3, F16, NONE, False, False, False, 0),      # a weight behind an odd tensor
    (3001, 1201, 1301, 0, BF16, NONE, True, False, False, 4),      # the same, odd strides
]


@pytest.mark.parametrize("case", LINEAR, ids=str)
def test_linear(T, Z, case):
    n, inner, outer, before, dt, act, bias, residual, pre, gap = case
    sizes = [before, inner * outer, outer]
    plan = Z.zero_plan(sum(sizes), 1, sizes, 0, 1)
    params = randn(T, (plan.psi_pad,), dt, 1, 0.05)
    w = params[before:before + inner * outer].view(outer, inner).double()
    b = params[before + inner * outer:].double() if bias else T.zeros(outer, dtype=T.float64, device="cuda")
    x = Rows(T, n, inner, inner + gap, dt, gap % 5, randn(T, (n, inner), dt, 2))
    r = Rows(T, n, outer, outer + gap, dt, gap % 3, randn(T, (n, outer), dt, 3)) if residual else None
    y, p = Rows(T, n, outer, outer + gap, dt, 1), Rows(T, n, outer, outer + 2 * gap, dt, 0)
    ws = ws_of(T, Z.zero_linear_workspace_bytes(plan, 1, inner, n))

    def run():
        Z.zero_linear(plan, 1, inner, params, dt, x.t, y.t, bias=2 if bias else -1, act=act, residual=r.t if r else None,
                      pre=p.t if pre else None, workspace=ws)

    run()
    z = x.t.double() @ w.t() + b
    off = 2 * (inner + 1) * U * (x.t.double().abs() @ w.abs().t() + b.abs())
    a = act64(T, act, z)
    if pre:
        close(T, p.t, z, off + h(T, z, dt), "pre")
        p.check()
    want = a + (r.t.double() if r else 0.0)
    off = 1.2 * off + 1e-5 * a.abs() + 2 * U * want.abs() + 1e-37
    close(T, y.t, want, off + h(T, want.abs() + off, dt), "y")
    y.check()
    first = y.t.clone()
    run()
    assert T.equal(first, y.t), "the same call gives other bits"
    if r:       # in place of the residual
        Z.zero_linear(plan, 1, inner, params, dt, x.t, r.t, bias=2 if bias else -1, act=act, residual=r.t, workspace=ws)
        assert T.equal(first, r.t)
        r.check()


GRAD = [
    # rows, in, out, before, dtype, act, addend, gap
    (1, 1, 1, 0, BF16, NONE, False, 0),
    (1, 768, 768, 0, BF16, GELU, True, 0),
    (7, 5, 3, 1, F16, SILU, True, 1),
    (33, 65, 129, 1, BF16, GELU_TANH, True, 3),
    (64, 64, 128, 0, F16, RELU, False, 0),
    (127, 333, 1000, 5, F16, GELU, True, 0),
    (130, 136, 264, 0, BF16, NONE, True, 8),
    (3, 40, 65536, 0, BF16, GELU, True, 0),
    (5, 33, 20001, 1, F16, GELU_TANH, True, 2),
    (129, 328, 50257, 0, BF16, NONE, False, 0),       # back from a tied table's logits
    (2049, 2056, 2048, 0, BF16, SILU, True, 16),
    (100, 134, 130, 2, BF16, NONE, False, 2),
    (600, 1030, 30, 0, F16, GELU, True, 0),
    (1500, 1301, 1201, 3, F16, NONE, True, 0),
    (2050, 1042, 1090, 4, BF16, RELU, True, 6),
    (3001, 1201, 1301, 3, BF16, GELU, True, 0),
    (3001, 1200, 1301, 3, F16, NONE, False, 0),
    (3001, 1201, 1301, 0, BF16, SILU, True, 4),
    (9001, 33, 6001, 0, BF16, NONE, False, 0),
]


@pytest.mark.parametrize("case", GRAD, ids=str)
def test_input_grad(T, Z, case):
    n, inner, outer, before, dt, act, addend, gap = case
    sizes = [before, inner * outer]
    plan = Z.zero_plan(sum(sizes), 1, sizes, 0, 1)
    params = randn(T, (plan.psi_pad,), dt, 1, 0.05)
    w = params[before:].view(outer, inner).double()
    dz = Rows(T, n, outer, outer + gap, dt, gap % 5, randn(T, (n, outer), dt, 2))
    pre = Rows(T, n, inner, inner + gap, dt, 1, randn(T, (n, inner), dt, 3, 2.0)) if act else None
    add = Rows(T, n, inner, inner + 2 * gap, dt, 0, randn(T, (n, inner), dt, 4)) if addend else None
    dx = Rows(T, n, inner, inner + gap, dt, 1)
    ws = ws_of(T, Z.zero_linear_input_grad_workspace_bytes(plan, 1, inner, n))

    def run(out, a):
        Z.zero_linear_input_grad(plan, 1, inner, params, dt, dz.t, out, act=act, pre=pre.t if act else None, addend=a, workspace=ws)

    run(dx.t, add.t if addend else None)
    v = dz.t.double() @ w
    s = slope64(T, act, pre.t.double()) if act else T.ones_like(v)
    want = v * s + (add.t.double() if addend else 0.0)
    off = 1.2 * 2 * outer * U * (dz.t.double().abs() @ w.abs()) + (2e-5 if act else 0.0) * v.abs() + 2 * U * want.abs() + 1e-37
    close(T, dx.t, want, off + h(T, want.abs() + off, dt), "dx")
    dx.check()
    if addend:
        run(add.t, add.t)
        assert T.equal(add.t, dx.t)
        add.check()


WEIGHT = [
    # rows, in, out, before, dtype, dst, ranks, gap
    (0, 5, 3, 1, BF16, BF16, 2, 0),
    (1, 1, 1, 0, BF16, BF16, 1, 0),
    (1, 65, 33, 3, F16, F32, 4, 1),
    (7, 5, 3, 1, F16, F16, 3, 1),
    (37, 65, 129, 1, BF16, F32, 8, 3),
    (64, 64, 128, 0, F16, F16, 2, 0),
    (333, 127, 1000, 5, F16, BF16, 4, 0),
    (1000, 136, 264, 8, BF16, BF16, 8, 8),
    (8191, 96, 96, 0, BF16, F32, 8, 0),
    (4099, 65, 33, 1, F16, F16, 2, 5),
    (2048, 768, 768, 64, BF16, BF16, 8, 0),
    (520, 1032, 2056, 0, F16, F16, 4, 16),
    (257, 328, 50257, 0, BF16, BF16, 8, 0),
    (330, 130, 134, 2, BF16, BF16, 4, 2),
    (1201, 1301, 1499, 3, F16, F16, 2, 0),
    (1202, 1302, 1498, 4, F16, F32, 8, 6),
    (70, 3, 5, 0, BF16, F32, 2, 0),
    (90, 75, 131, 1, F16, F32, 2, 1),                  # odd rows an even distance apart
    (65, 131, 67, 0, BF16, BF16, 3, 5),
    (3001, 1201, 1301, 3, BF16, BF16, 3, 0),
    (9001, 33, 6001, 0, F16, F32, 2, 0),
    (9001, 6001, 33, 0, BF16, BF16, 4, 2),
]


@pytest.mark.parametrize("case", WEIGHT, ids=str)
def test_weight_grad(T, Z, case):
    n, inner, outer, before, dt, ddt, ranks, gap = case
    sizes = [before, inner * outer, outer]
    plan = Z.zero_plan(sum(sizes), ranks, sizes, 0, 8)
    dz = Rows(T, n, outer, outer + gap, dt, gap % 5, randn(T, (n, outer), dt, 2))
    x = Rows(T, n, inner, inner + gap, dt, gap % 3, randn(T, (n, inner), dt, 3))
    scale = 0.75 / max(1, n)
    old = randn(T, (plan.psi_pad,), ddt, 4)
    full = old.clone()
    ws = ws_of(T, Z.zero_linear_weight_grad_workspace_bytes(plan, 1, inner, n))

    def run(dst, rank=-1, accumulate=False, bias=2):
        Z.zero_linear_weight_grad(plan, 1, inner, dz.t, x.t, dt, scale, dst, ddt, bias=bias, rank=rank, accumulate=accumulate,
                                  workspace=ws)

    run(full)
    lo, mid = before, before + inner * outer
    dw = scale * (dz.t.double().t() @ x.t.double())
    db = scale * dz.t.double().sum(0)
    off_w = 2 * (n + 2) * U * scale * (dz.t.double().abs().t() @ x.t.double().abs())
    off_b = 2 * (n + 2) * U * scale * dz.t.double().abs().sum(0)
    close(T, full[lo:mid].view(outer, inner), dw, off_w + h(T, dw.abs() + off_w, ddt), "dW")
    close(T, full[mid:mid + outer], db, off_b + h(T, db.abs() + off_b, ddt), "db")
    assert T.equal(full[:lo], old[:lo]) and T.equal(full[mid + outer:], old[mid + outer:]), "outside the tensors"
    # Every owner's slice holds the bits of the full buffer, and nothing else is written.
    flat_off, _, padded, share, _ = plan.bucket(0)
    for rank in range(ranks):
        mine = slice(rank * share, (rank + 1) * share)
        got = old[mine].clone()
        run(got, rank)
        assert T.equal(got, full[mine]), f"slice of rank {rank}"
    # The weight alone, and added to what is there.
    alone = old.clone()
    run(alone, bias=-1)
    assert T.equal(alone[lo:mid], full[lo:mid]) and T.equal(alone[mid:], old[mid:])
    more = old.clone()
    run(more, accumulate=True)
    for a, b, want, off in ((lo, mid, dw.reshape(-1), off_w.reshape(-1)), (mid, mid + outer, db, off_b)):
        want = want + old[a:b].double()
        off = off + 2 * U * want.abs()
        close(T, more[a:b], want, off + h(T, want.abs() + off, ddt), "accumulated")
    for rank in range(ranks):
        got = old[rank * share:(rank + 1) * share].clone()
        run(got, rank, accumulate=True)
        assert T.equal(got, more[rank * share:(rank + 1) * share])


@pytest.mark.parametrize("act", [NONE, RELU, GELU, GELU_TANH, SILU])
@pytest.mark.parametrize("dt", [F16, BF16])
def test_activation_every_value(T, Z, act, dt):
    """Every 16-bit value through an activation and its slope; infinities, NaN
    and both zeros among them."""
    bits = T.arange(-32768, 32768, dtype=T.int32, device="cuda").to(T.int16)
    z = bits.view(R.torch_type(dt))
    plan = Z.zero_plan(1, 1, [1], 0, 1)
    one = T.ones(1, dtype=R.torch_type(dt), device="cuda")
    y = T.empty_like(z)
    Z.zero_linear(plan, 0, 1, one, dt, z.view(-1, 1), y.view(-1, 1), act=act)       # x * 1
    z64 = z.double()
    nan, big = z64.isnan(), z64.abs() > 1e4
    safe = T.where(nan | big, T.zeros_like(z64), z64)
    want = act64(T, act, safe)
    ends = {NONE: z64, RELU: T.clamp(z64, min=0)}.get(act, T.where(z64 > 0, z64, T.zeros_like(z64)))
    want = T.where(big, ends, want)
    assert bool((y.isnan() == nan).all())
    inf = want.isinf()
    assert T.equal(y[inf].double(), want[inf])
    ok = ~nan & ~inf
    # A sigmoid or distribution function below the smallest normal number, 2^-126, may come out as 0.
    tol = 1e-5 * want.abs() + T.clamp(z64.abs(), max=128.0) * 2.0 ** -126
    close(T, y[ok], want[ok], (tol + h(T, want.abs() + tol, dt))[ok], "act")
    dy = T.full_like(z, 0.5)
    dz = T.empty_like(z)
    Z.zero_activation_grad(dy, z, dz, dt, act)
    s = T.where(big, {NONE: T.ones_like(z64)}.get(act, (z64 > 0).double()), slope64(T, act, safe))
    want = 0.5 * s
    tol = T.full_like(want, 1e-5 if act > RELU else 0.0)
    if act == NONE:
        assert bool((dz == 0.5).all())
    else:
        assert bool((dz.isnan() == nan).all())
        close(T, dz[~nan], want[~nan], (tol + h(T, want.abs() + tol, dt))[~nan], "slope")
    Z.zero_activation_grad(dy, z, dy, dt, act)                                       # in place
    assert T.equal(dy.view(T.int16)[~nan], dz.view(T.int16)[~nan])


def test_activation_grad_sizes(T, Z):
    for n in (0, 1, 7, 8, 9, 2047, 100003):
        buf = T.full((3, n + 3), 77, dtype=T.float16, device="cuda")
        dy, pre = randn(T, (n,), F16, 1), randn(T, (n,), F16, 2, 2.0)
        out = buf.view(-1)[n + 4:2 * n + 4]
        Z.zero_activation_grad(dy, pre, out, F16, SILU)
        want = dy.double() * slope64(T, SILU, pre.double()) if n else T.zeros(0, dtype=T.float64, device="cuda")
        tol = 2e-5 * dy.double().abs()
        close(T, out, want, tol + h(T, want.abs() + tol, F16), "dz")
        assert bool((buf.view(-1)[:n + 4] == 77).all()) and bool((buf.view(-1)[2 * n + 4:] == 77).all())


def test_linear_special_values(T, Z):
    """A row with NaN or an infinity stays its own affair, in whole and ragged
    tiles and behind the last element of k."""
    for n, inner, outer in ((70, 100, 90), (300, 264, 136), (3, 33000, 20)):
        plan = Z.zero_plan(inner * outer, 1, [inner * outer], 0, 1)
        params = randn(T, (plan.psi_pad,), BF16, 1)
        x = randn(T, (n, inner), BF16, 2)
        y, clean = (T.empty((n, outer), dtype=T.bfloat16, device="cuda") for _ in range(2))
        ws = ws_of(T, Z.zero_linear_workspace_bytes(plan, 0, inner, n))
        Z.zero_linear(plan, 0, inner, params, BF16, x, clean, workspace=ws)
        x[1, inner - 1] = math.nan
        x[2, 0] = math.inf
        Z.zero_linear(plan, 0, inner, params, BF16, x, y, workspace=ws)
        assert bool(y[1].isnan().all())
        w = params.view(outer, inner)
        assert T.equal(y[2] > 0, w[:, 0] > 0) and bool((y[2].isinf() | (w[:, 0] == 0)).all())
        rest = [i for i in range(n) if i not in (1, 2)]
        assert T.equal(y[rest], clean[rest])


# ---------------------------------------------------------------------------
# Orthogonalisation
# ---------------------------------------------------------------------------

def ortho64(T, g, scale, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7):
    x = g.double()
    x = x / (x.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for _ in range(steps):
        m = x @ x.t()
        x = a * x + (b * m + c * m @ m) @ x
    return scale * (x.t() if tall else x)


def matrix(T, rows, cols, dt, seed, kind):
    g = randn(T, (rows, cols), F32, seed)
    k = min(rows, cols)
    if kind == "low rank" and k > 1:       # a few strong directions over little noise
        u, v = randn(T, (rows, min(8, k)), F32, seed + 1), randn(T, (min(8, k), cols), F32, seed + 2)
        g = 1e-3 * g + (u / T.arange(1, u.shape[1] + 1, device="cuda") ** 2) @ v
    return (g * 1e-3).to(R.torch_type(dt))


# Each product rounds its operands to fp16, half a step of 2^-11 each, at random
# and independently: an error of about 2^-11 / sqrt(3) in norm for each of X, A and
# B, times their weight in the step (a few) and the growth of later steps (at most
# 1.6 each on converged directions), some 2e-3 at most; a mistake in a product or
# coefficient is off by tenths.  Then the rounding of the result.
ORTHO_TOL = 4e-3


def ortho_close(T, got, want, dt, what):
    norm = float(want.norm())
    off = float((got.double() - want).norm())
    assert off <= (ORTHO_TOL + T.finfo(R.torch_type(dt)).eps / 2) * norm, (what, off / max(norm, 1e-300))


ORTHO = [
    # shapes (rows, cols, how many), src, dst, before
    ([(1, 1, 1)], BF16, BF16, 0),
    ([(1, 100, 1), (100, 1, 2)], F16, F16, 1),
    ([(7, 9, 1), (9, 7, 1)], BF16, BF16, 3),
    ([(33, 65, 2), (65, 33, 3), (64, 64, 1)], BF16, F16, 5),
    ([(128, 128, 4)], F16, BF16, 0),
    ([(64, 4096, 1), (4096, 64, 1)], BF16, BF16, 0),        # pieces of k
    ([(129, 1000, 3), (1000, 129, 1)], F16, F16, 7),
    ([(260, 300, 40)], BF16, BF16, 0),
    ([(8, 8, 300)], BF16, BF16, 0),                          # more than one launch's table
    ([(768, 768, 5), (768, 2304, 2), (2304, 768, 2)], BF16, BF16, 64),
    ([(1100, 1030, 1)], BF16, BF16, 0),
    ([(32, 512, 2), (512, 32, 1), (31, 511, 1), (127, 128, 3), (96, 160, 2), (160, 96, 1)], BF16, BF16, 1),   # the largest of one workgroup
    ([(33, 512, 1), (129, 128, 1), (140, 130, 2), (200, 8, 1), (8, 300, 2)], F16, BF16, 0),                  # and the next
    ([(4097, 200, 1), (200, 4097, 2)], BF16, BF16, 0),
    ([(130, 136, 131)], BF16, BF16, 3),                      # two batches, the last of which is shorter
    ([(2050, 2300, 1)], F16, BF16, 0),
    # short sides: pieces of A, P X, tall and wide, odd, more than one batch
    ([(8, 3000, 2), (3000, 8, 1), (17, 5001, 3), (5001, 17, 1), (57, 1000, 1)], BF16, BF16, 3),
    ([(64, 300, 140), (300, 64, 2), (49, 33333, 1), (33333, 40, 2)], F16, BF16, 0),
    ([(1, 70000, 1), (70000, 1, 1), (64, 257, 3), (257, 63, 1)], BF16, F16, 1),
    ([(65, 300, 3), (300, 65, 1), (72, 1000, 2)], BF16, BF16, 0),            # the next longer
]


@pytest.mark.parametrize("kind", ["normal", "low rank"])
@pytest.mark.parametrize("case", ORTHO, ids=str)
def test_orthogonalize(T, Z, case, kind):
    shapes, sdt, ddt, before = case
    sizes, entries, mats = [before], [], []
    for i, (r, c, count) in enumerate(shapes):
        for k in range(count):
            if k % 2:                       # a tensor of its own, or one more in the last
                sizes[-1] += r * c
            else:
                sizes.append(r * c)
                entries.append((len(sizes) - 1, r, c, 0.5 + 0.25 * len(entries)))
            mats.append((len(sizes) - 1, r, c, entries[-1][3], matrix(T, r, c, sdt, 100 * i + k, kind)))
    sizes.append(11)                        # a tensor that is not listed
    plan = Z.zero_plan(sum(sizes), 2, sizes, 0, 8)
    src = T.full((plan.psi_pad,), 77, dtype=R.torch_type(sdt), device="cuda")
    places, at = [], {}
    for t, r, c, s, g in mats:
        lo = plan.tensor(t)[1] + at.get(t, 0)
        at[t] = at.get(t, 0) + r * c
        src[lo:lo + r * c] = g.reshape(-1)
        places.append(lo)
    dst = T.full((plan.psi_pad,), 55, dtype=R.torch_type(ddt), device="cuda")
    m = Z.Matrices(entries[::-1])
    ws = ws_of(T, Z.zero_orthogonalize_workspace_bytes(plan, m))
    kept = src.clone()
    Z.zero_orthogonalize(plan, m, src, sdt, dst, ddt, workspace=ws)
    assert T.equal(src, kept)
    rest = T.ones(plan.psi_pad, dtype=T.bool, device="cuda")
    for (t, r, c, s, g), lo in zip(mats, places):
        ortho_close(T, dst[lo:lo + r * c].view(r, c), ortho64(T, g, s), ddt, (r, c, t))
        rest[lo:lo + r * c] = False
    assert bool((dst[rest] == 55).all())
    again = T.full_like(dst, 55)
    Z.zero_orthogonalize(plan, m, src, sdt, again, ddt, workspace=ws)
    assert T.equal(dst, again)
    if sdt == ddt:
        Z.zero_orthogonalize(plan, m, src, sdt, src, sdt, workspace=ws)
        assert T.equal(src[~rest], dst[~rest]) and T.equal(src[rest], kept[rest])


@pytest.mark.parametrize("n,k", [(40, 40), (150, 150), (40, 700), (700, 40)])
def test_orthogonalize_values(T, Z, n, k):
    """Zeros, tiny and huge entries, NaN and infinities, each matrix on its own."""
    plan = Z.zero_plan(7 * n * k, 1, [n * k] * 7, 0, 1)
    src = randn(T, (plan.psi_pad,), BF16, 1)
    g = src.view(7, n, k)
    g[1] = 0
    g[2, 3, 4] = math.nan
    g[3, 0, 0] = -math.inf
    g[4] *= 1e-25
    g[5] *= 1e35
    g[6] = 0
    g[6, n - 1, k - 1] = 3.0
    m = Z.Matrices([(t, n, k, 1.0) for t in range(7)])
    ws = ws_of(T, Z.zero_orthogonalize_workspace_bytes(plan, m))
    dst = T.empty_like(src)
    Z.zero_orthogonalize(plan, m, src, BF16, dst, BF16, workspace=ws)
    out = dst.view(7, n, k)
    for t in (0, 4, 5, 6):
        ortho_close(T, out[t], ortho64(T, g[t], 1.0), BF16, t)
    assert bool((out[1] == 0).all())
    assert bool(out[2].isnan().all()) and bool(out[3].isnan().all())


@pytest.mark.parametrize("shape", [(96, 200), (64, 100), (100, 64), (40, 900), (900, 40)], ids=str)
@pytest.mark.parametrize("poly", [(1, 3.4445, -4.7750, 2.0315, 1e-7), (7, 3.4445, -4.7750, 2.0315, 1e-7),
                                  (12, 1.875, -1.25, 0.375, 1e-12), (3, 2.0, 0.0, 0.0, 1e-7), (4, 1.5, -0.5, 0.0, 1.0)], ids=str)
def test_orthogonalize_polynomials(T, Z, poly, shape):
    r, c = shape
    plan = Z.zero_plan(r * c, 1, [r * c], 0, 1)
    g = matrix(T, r, c, BF16, 3, "normal") * 1000
    dst = T.empty(plan.psi_pad, dtype=T.bfloat16, device="cuda")
    m = Z.Matrices([(0, r, c, 2.0)])
    ws = ws_of(T, Z.zero_orthogonalize_workspace_bytes(plan, m))
    Z.zero_orthogonalize(plan, m, g.reshape(-1), BF16, dst, BF16, poly=Z.NewtonSchulz(*poly), workspace=ws)
    ortho_close(T, dst.view(r, c), ortho64(T, g, 2.0, *poly), BF16, poly)


@pytest.mark.parametrize("shape", [(24, 30), (40, 900), (900, 40), (64, 2000), (150, 200)], ids=str)
@pytest.mark.parametrize("steps", [5, 10, 11, 14, 15, 16, 30])
def test_orthogonalize_lacking_directions(T, Z, steps, shape):
    """Equal, opposite and empty rows and columns: directions that the matrix has
    nothing of, however many the steps."""
    r, c = shape
    g = matrix(T, r, c, BF16, 5, "normal")
    n = min(r, c) // 3
    g[1:1 + n] = g[0]
    g[n:n + 4] *= -1
    g[n + 5:n + 8] = 0
    g[:, 2:2 + n] = g[:, :1]
    g[:, n + 2:n + 5] = 0
    plan = Z.zero_plan(r * c, 1, [r * c], 0, 1)
    m = Z.Matrices([(0, r, c, 1.0)])
    poly = (steps, 1.875, -1.25, 0.375, 1e-7)
    dst = T.empty(plan.psi_pad, dtype=T.bfloat16, device="cuda")

    def run():
        Z.zero_orthogonalize(plan, m, g.reshape(-1).contiguous(), BF16, dst, BF16, poly=Z.NewtonSchulz(*poly),
                             workspace=ws_of(T, Z.zero_orthogonalize_workspace_bytes(plan, m)))

    if 1.875 ** steps > 10000:
        with pytest.raises(Z.ZeroError):
            run()
        return
    run()
    ortho_close(T, dst.view(r, c), ortho64(T, g, 1.0, *poly), BF16, poly)


# ---------------------------------------------------------------------------
# The two halves of the step
# ---------------------------------------------------------------------------

def f32(T, x):
    return T.tensor(float(np.float32(x)), dtype=T.float32)


@pytest.mark.parametrize("sizes,ranks,align,cap", [([1], 1, 1, 0), ([1003], 2, 1, 0), ([4097, 33, 700], 3, 8, 1000), ([70001], 4, 64, 0),
                                                   ([300000, 5], 8, 64, 0), ([9001], 16, 1, 0), ([12345], 70, 1, 0)], ids=str)
@pytest.mark.parametrize("gdt,udt,nesterov,full,shift", [(BF16, BF16, True, True, 0), (F16, BF16, False, False, 1), (BF16, F16, True, False, 0),
                                                         (F16, F16, True, True, 1)], ids=str)
def test_muon_momentum(T, Z, sizes, ranks, align, cap, gdt, udt, nesterov, full, shift):
    """Bit for bit: one fp32 operation after another."""
    plan = Z.zero_plan(sum(sizes), ranks, sizes, cap, align)
    S, P = plan.shard_total, plan.psi_pad
    rank = ranks - 1
    hyper = Z.MuonHyper(lr=0.02, momentum=0.95, grad_scale=1.0 / ranks, nesterov=nesterov)
    # Rank 0's contribution is a whole gradient buffer, the others are slices.
    whole = randn(T, (P + shift,), gdt, 1, 1e-2)[shift:]
    slices = [whole] + [randn(T, (S + shift,), gdt, 2 + q, 1e-2)[shift:] for q in range(1, ranks)]
    own = T.cat([T.arange(f + rank * s, f + (rank + 1) * s) for f, _, _, s, _ in plan.buckets()])
    parts = [whole.cpu()[own]] + [x.cpu() for x in slices[1:]]
    m0 = randn(T, (S,), F32, 99)
    g = parts[0].float()
    for x in parts[1:]:
        g = g + x.float()
    g = g * f32(T, 1.0 / ranks)
    mu = f32(T, 0.95)
    m = mu * m0.cpu() + g
    u = (g + mu * m if nesterov else m).to(R.torch_type(udt))
    got_m, got_u = m0.clone(), T.full((P if full else S,), 77, dtype=R.torch_type(udt), device="cuda")
    src = Z.GradSrc(gdt, slices, [1] + [0] * (ranks - 1))
    Z.zero_muon_momentum(plan, rank, hyper, src, None, got_m, got_u, udt, full)
    assert T.equal(got_m.cpu(), m)
    want = T.full((P,), 77, dtype=R.torch_type(udt))
    want[own] = u
    assert T.equal(got_u.cpu(), want if full else u)
    # From the reduced gradient: the same bits.
    red = T.empty(S, device="cuda")
    Z.zero_shard_reduce(plan, rank, src, 1.0 / ranks, red)
    again_m, again_u = m0.clone(), T.full_like(got_u, 77)
    Z.zero_muon_momentum(plan, rank, hyper, None, red, again_m, again_u, udt, full)
    assert T.equal(again_m, got_m) and T.equal(again_u, got_u)


@pytest.mark.parametrize("sizes,ranks,align,cap", [([1], 1, 1, 0), ([1003], 2, 1, 0), ([4097, 33, 700], 3, 8, 1000), ([70001], 4, 64, 0),
                                                   ([300000, 5], 8, 64, 0)], ids=str)
@pytest.mark.parametrize("odt,pdt,ofull,full,shift", [(BF16, BF16, True, True, 0), (F16, BF16, False, False, 1), (BF16, F16, True, False, 0),
                                                      (F16, F16, False, True, 0)], ids=str)
def test_muon_apply(T, Z, sizes, ranks, align, cap, odt, pdt, ofull, full, shift):
    plan = Z.zero_plan(sum(sizes), ranks, sizes, cap, align)
    S, P = plan.shard_total, plan.psi_pad
    rank = ranks // 2
    hyper = Z.MuonHyper(lr=0.02, weight_decay=0.1)
    own = T.cat([T.arange(f + rank * s, f + (rank + 1) * s) for f, _, _, s, _ in plan.buckets()])
    o = randn(T, ((P if ofull else S) + shift,), odt, 1, 0.2)[shift:]
    w0 = randn(T, (S,), F32, 2, 0.02)
    w = f32(T, 1 - 0.02 * 0.1) * w0.cpu() - f32(T, 0.02) * (o.cpu()[own] if ofull else o.cpu()).float()
    got_w, got_p = w0.clone(), T.full((P if full else S,), 77, dtype=R.torch_type(pdt), device="cuda")
    Z.zero_muon_apply(plan, rank, hyper, o, odt, ofull, got_w, got_p, pdt, full)
    assert T.equal(got_w.cpu(), w)
    want = T.full((P,), 77, dtype=R.torch_type(pdt))
    want[own] = w.to(R.torch_type(pdt))
    assert T.equal(got_p.cpu(), want if full else want[own])


# ---------------------------------------------------------------------------
# Together, captured, and on streams
# ---------------------------------------------------------------------------

class Block:
    """Two linear layers with a residual around them, trained by Muon on one
    GPU that holds both of two ranks' shares: h = x + gelu(x W1^T + b1) W2^T + b2,
    loss = sum(h target).  Biases take no part in the step."""

    def __init__(self, T, Z, n=96, wide=48, inner=80, seed=0):
        self.T, self.Z, self.n, self.wide, self.inner = T, Z, n, wide, inner
        sizes = [inner * wide, inner, wide * inner, wide]
        self.plan = Z.zero_plan(sum(sizes), 2, sizes, 0, 8)
        P, S = self.plan.psi_pad, self.plan.shard_total
        self.params = randn(T, (P,), BF16, seed + 1, 0.1)
        self.params[sum(sizes):] = 0
        self.x = [randn(T, (n, wide), BF16, seed + 2 + r) for r in range(2)]
        self.target = [randn(T, (n, wide), BF16, seed + 4 + r) for r in range(2)]
        self.master = [self.params[r * S:(r + 1) * S].float() for r in range(2)]
        self.mom = [T.zeros(S, device="cuda") for _ in range(2)]
        self.pre, self.act, self.dact = (T.empty((n, inner), dtype=T.bfloat16, device="cuda") for _ in range(3))
        self.out, self.dx = (T.empty((n, wide), dtype=T.bfloat16, device="cuda") for _ in range(2))
        self.grad = [T.zeros(P, dtype=T.bfloat16, device="cuda") for _ in range(2)]
        self.update = T.zeros(P, dtype=T.bfloat16, device="cuda")
        self.matrices = Z.Matrices([(0, inner, wide, 1.0), (2, wide, inner, 1.0)])
        self.hyper = Z.MuonHyper(lr=0.05, momentum=0.9, weight_decay=0.01, grad_scale=0.5)
        need = [Z.zero_orthogonalize_workspace_bytes(self.plan, self.matrices)]
        for t, i in ((0, wide), (2, inner)):
            need += [Z.zero_linear_workspace_bytes(self.plan, t, i, n), Z.zero_linear_input_grad_workspace_bytes(self.plan, t, i, n),
                     Z.zero_linear_weight_grad_workspace_bytes(self.plan, t, i, n)]
        self.ws = ws_of(T, max(need))

    def step(self):
        Z, p, ws = self.Z, self.plan, self.ws
        for r in range(2):
            Z.zero_linear(p, 0, self.wide, self.params, BF16, self.x[r], self.act, bias=1, act=GELU, pre=self.pre, workspace=ws)
            Z.zero_linear(p, 2, self.inner, self.params, BF16, self.act, self.out, bias=3, residual=self.x[r], workspace=ws)
            dh = self.target[r]
            Z.zero_linear_weight_grad(p, 2, self.inner, dh, self.act, BF16, 1.0, self.grad[r], BF16, bias=3, workspace=ws)
            Z.zero_linear_input_grad(p, 2, self.inner, self.params, BF16, dh, self.dact, act=GELU, pre=self.pre, workspace=ws)
            Z.zero_linear_weight_grad(p, 0, self.wide, self.dact, self.x[r], BF16, 1.0, self.grad[r], BF16, bias=1, workspace=ws)
            Z.zero_linear_input_grad(p, 0, self.wide, self.params, BF16, self.dact, self.dx, addend=dh, workspace=ws)
        src = Z.GradSrc(BF16, self.grad, [1, 1])
        for r in range(2):
            Z.zero_muon_momentum(p, r, self.hyper, src, None, self.mom[r], self.update, BF16, True)
        Z.zero_orthogonalize(p, self.matrices, self.update, BF16, self.update, BF16, workspace=ws)
        for r in range(2):
            Z.zero_muon_apply(p, r, self.hyper, self.update, BF16, True, self.master[r], self.params, BF16, True)

    def state(self):
        return [t.clone() for t in (self.out, self.dx, *self.grad, *self.mom, self.update, *self.master, self.params)]


def test_block_step(T, Z):
    """The operators one after another, against autograd in 64 bits."""
    b = Block(T, Z)
    wide, inner, plan = b.wide, b.inner, b.plan
    off = [plan.tensor(t)[1] for t in range(4)]
    start = b.params.double()
    leaves = [start[o:o + k].clone().requires_grad_(True) for o, k in zip(off, plan.tensor_numel)]
    w1, b1, w2, b2 = leaves[0].view(inner, wide), leaves[1], leaves[2].view(wide, inner), leaves[3]
    grads = []
    for r in range(2):
        x = b.x[r].double().requires_grad_(True)
        hh = x + act64(T, GELU, x @ w1.t() + b1) @ w2.t() + b2
        grads.append(T.autograd.grad((hh * b.target[r].double()).sum(), leaves + [x]))
    b.step()
    near = lambda got, want, tol, what: close_norm(got, want, tol, what)   # noqa: E731

    def close_norm(got, want, tol, what):
        off = float((got.double() - want).norm() / want.norm())
        assert off <= tol, (what, off)

    # bf16 steps of 2^-8 at most: the activation and its gradient are rounded on the way.
    near(b.out, hh.detach(), 2 * 2.0 ** -8, "out")
    near(b.dx, grads[1][4], 3 * 2.0 ** -8, "dx")
    for r in range(2):
        for t in range(4):
            near(b.grad[r][off[t]:off[t] + plan.tensor_numel[t]], grads[r][t].reshape(-1), 3 * 2.0 ** -8, (r, t))
    # The step, from the gradients that the GPU holds.
    total = 0.5 * (b.grad[0].double() + b.grad[1].double())
    mom = T.cat(b.mom).double()
    near(mom, total, 1e-6, "momentum")
    u = (total + 0.9 * total).to(T.bfloat16)
    want = start * (1 - 0.05 * 0.01)
    for t, (r, c) in ((0, (inner, wide)), (2, (wide, inner))):
        s = slice(off[t], off[t] + r * c)
        o = ortho64(T, u[s].view(r, c), 1.0)
        ortho_close(T, b.update[s].view(r, c), o, BF16, t)
        want[s] -= 0.05 * o.reshape(-1)
    for t in (1, 3):
        s = slice(off[t], off[t] + plan.tensor_numel[t])
        want[s] -= 0.05 * u[s].double()
    near(T.cat(b.master), want, 2.0 ** -8, "master")
    assert T.equal(T.cat(b.master).to(T.bfloat16), b.params)


def test_captured(T, Z):
    """The whole step captured and replayed, with eager work between the
    replays, against an eager twin."""
    eager, graphed = Block(T, Z), Block(T, Z)
    warm = Block(T, Z, seed=50)
    side = T.cuda.Stream()
    with T.cuda.stream(side):
        warm.step()
    T.cuda.synchronize()
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        graphed.step()
    for i in range(4):
        eager.step()
        g.replay()
        if i % 2:
            warm.step()
        T.cuda.synchronize()
        for a, b in zip(eager.state(), graphed.state()):
            assert T.equal(a.view(T.int16) if a.dtype == T.bfloat16 else a, b.view(T.int16) if b.dtype == T.bfloat16 else b), i


def test_captured_large(T, Z):
    """Products of large tiles, with pieces of k and copied operands, and matrices
    that take every launch of an orthogonalisation, captured and replayed."""
    n, i, o = 2100, 1031, 770
    plan = Z.zero_plan(o * i + o, 2, [o * i, o], 0, 8)
    mats = Z.zero_plan(1100 * 1030, 1, [1100 * 1030], 0, 8)
    m = Z.Matrices([(0, 1100, 1030, 0.5)])
    params, x, dz = (randn(T, shape, BF16, k) for k, shape in enumerate([(plan.psi_pad,), (n, i), (n, o)]))
    update = randn(T, (mats.psi_pad,), BF16, 4)
    ws = ws_of(T, max(Z.zero_linear_workspace_bytes(plan, 0, i, n), Z.zero_linear_input_grad_workspace_bytes(plan, 0, i, n),
                      Z.zero_linear_weight_grad_workspace_bytes(plan, 0, i, n, 1), Z.zero_orthogonalize_workspace_bytes(mats, m)))

    def run(y, dx, grad, out):
        Z.zero_linear(plan, 0, i, params, BF16, x, y, bias=1, act=Z.ZERO_ACT_GELU, workspace=ws)
        Z.zero_linear_input_grad(plan, 0, i, params, BF16, dz, dx, workspace=ws)
        Z.zero_linear_weight_grad(plan, 0, i, dz, x, BF16, 1.0, grad, BF16, bias=1, rank=1, workspace=ws)
        Z.zero_orthogonalize(mats, m, update, BF16, out, BF16, workspace=ws)

    def buffers():
        return [T.zeros(s, dtype=T.bfloat16, device="cuda") for s in [(n, o), (n, i), (plan.shard_total,), (mats.psi_pad,)]]

    got = buffers()
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        run(*got)
    for k in range(3):
        x.mul_(0.5)
        update.add_(x.view(-1)[:update.numel()])
        want = buffers()
        run(*want)
        T.cuda.synchronize()
        g.replay()
        T.cuda.synchronize()
        for a, b in zip(want, got):
            assert T.equal(a, b), k


def test_two_streams(T, Z):
    """Two steps at once on two streams, each with its own workspace."""
    twins = [Block(T, Z, seed=s) for s in (0, 30)]
    alone = [Block(T, Z, seed=s) for s in (0, 30)]
    for b in alone:
        b.step()
        b.step()
    streams = [T.cuda.Stream() for _ in twins]
    T.cuda.synchronize()
    for _ in range(2):
        for b, s in zip(twins, streams):
            with T.cuda.stream(s):
                b.step()
    T.cuda.synchronize()
    for a, b in zip(alone, twins):
        for x, y in zip(a.state(), b.state()):
            assert T.equal(x, y)


def test_gradient_against_differences(T, Z):
    """dx, dW and db against central differences of the layer itself, in fp16."""
    n, inner, outer = 9, 24, 17
    sizes = [inner * outer, outer]
    plan = Z.zero_plan(sum(sizes), 1, sizes, 0, 1)
    # Multiples of 2^-6 and steps of 2^-3: exact in fp16, before and behind a step.
    grid = lambda shape, seed: (randn(T, shape, F32, seed) * 16).round().clamp(-48, 48).div(64).half()   # noqa: E731
    params, x, weight_of_loss = grid((plan.psi_pad,), 1), grid((n, inner), 2), grid((n, outer), 3)
    y, pre = (T.empty((n, outer), dtype=T.float16, device="cuda") for _ in range(2))

    def loss(p, v):
        Z.zero_linear(plan, 0, inner, p, F16, v, y, bias=1, act=SILU, pre=pre)
        return float((y.double() * weight_of_loss.double()).sum())

    loss(params, x)
    dz, dx = T.empty_like(y), T.empty_like(x)
    Z.zero_activation_grad(weight_of_loss, pre, dz, F16, SILU)
    Z.zero_linear_input_grad(plan, 0, inner, params, F16, dz, dx)
    grad = T.zeros(plan.psi_pad, device="cuda")
    ws = ws_of(T, Z.zero_linear_weight_grad_workspace_bytes(plan, 0, inner, n))
    Z.zero_linear_weight_grad(plan, 0, inner, dz, x, F16, 1.0, grad, F32, bias=1, workspace=ws)
    step = 2.0 ** -3
    # y of size about 3 is rounded to 2^-10 on each side of the difference, at most
    # sum |weight| of it; the third derivative of silu is below 0.5, its cube of the
    # step times |x| or |w| below 1; dz is rounded to 2^-11 of itself.
    tol = 2 * 17 * 0.75 * 2.0 ** -10 / (2 * step) + 9 * 17 * 0.75 * 0.5 * step ** 2 / 6 * 0.1 + 0.02
    for buf, got, at in ((x, dx, [(0, 0), (3, 7), (8, 23)]), (params, grad, [(0,), (100,), (inner * outer - 1,), (inner * outer + 5,)])):
        for i in at:
            ends = []
            for sign in (1, -1):
                moved = buf.clone()
                moved[i] += sign * step
                ends.append(loss(moved, x) if buf is params else loss(params, moved))
            assert abs((ends[0] - ends[1]) / (2 * step) - float(got[i])) <= tol, (i, ends, float(got[i]))
