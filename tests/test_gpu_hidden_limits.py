"""The operators on the hidden matrices on the GPU: what the header promises at
its limits, held to its own figures."""
import math

import pytest

from tests import ops_reference as R
from tests.ops_reference import BF16, F16, F32

pytestmark = pytest.mark.gpu
GELU, GELU_TANH, SILU = 2, 3, 4


@pytest.fixture(scope="module")
def T(gpu):
    import torch
    return torch


@pytest.fixture()
def Z(zero_lib):
    return zero_lib


def randn(T, shape, dt, seed, sigma=1.0):
    g = T.Generator(device="cuda").manual_seed(seed)
    return T.empty(shape, dtype=R.torch_type(dt), device="cuda").normal_(0, sigma, generator=g)


# ---------------------------------------------------------------------------
# Orthogonalisation
# ---------------------------------------------------------------------------

DEFAULT = (5, 3.4445, -4.7750, 2.0315, 1e-7)


def ortho64(T, g, steps=5, a=3.4445, b=-4.7750, c=2.0315, eps=1e-7):
    """A stack of matrices by the formula, in 64 bits."""
    x = g.double()
    x = x / (T.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + eps)
    tall = x.shape[1] > x.shape[2]
    x = x.mT.contiguous() if tall else x
    for _ in range(steps):
        m = T.bmm(x, x.mT.contiguous())
        x = a * x + T.bmm(b * m + c * T.bmm(m, m), x)
    return x.mT if tall else x


def orthogonalized(T, Z, g, poly=DEFAULT):
    """The stack through the operator, from bf16 into fp16, whose rounding (2^-11 of
    a value) leaves the operator's own error to be seen."""
    n, r, c = g.shape
    plan = Z.zero_plan(n * r * c, 1, [n * r * c], 0, 1)
    m = Z.Matrices([(0, r, c, 1.0)])
    ws = T.full((max(1, Z.zero_orthogonalize_workspace_bytes(plan, m)),), 0x7f, dtype=T.uint8, device="cuda")
    dst = T.empty(n * r * c, dtype=T.float16, device="cuda")
    Z.zero_orthogonalize(plan, m, g.reshape(-1), BF16, dst, F16, poly=Z.NewtonSchulz(*poly), workspace=ws)
    return dst.view(n, r, c)


def off(T, got, want):
    """Distance over the matrix, relative, of each."""
    return T.linalg.vector_norm(got.double() - want, dim=(1, 2)) / T.linalg.vector_norm(want, dim=(1, 2))


HALF = 2.0 ** -11        # fp16's rounding of a result


@pytest.mark.parametrize("eps", [1e-7, 1e-20, 1e-30, 1e-45, 1e-300])
@pytest.mark.parametrize("r,c", [(5, 7), (40, 40), (40, 700), (700, 40), (150, 150)])
def test_zeros_any_eps(T, Z, r, c, eps):
    """A matrix of zeros gives zeros however small eps is, and its neighbours are
    what they would be."""
    g = randn(T, (3, r, c), BF16, 1)
    g[1] = 0
    poly = DEFAULT[:4] + (eps,)
    out = orthogonalized(T, Z, g, poly)
    assert bool((out[1] == 0).all())
    assert float(off(T, out[::2], ortho64(T, g[::2], *poly)).max()) <= 0.02 + HALF


def kinds(T, kind, n, r, c, seed):
    k = min(r, c)
    g = randn(T, (n, r, c), F32, seed)
    if kind == "low rank":
        q = min(8, k)
        fade = T.arange(1, q + 1, device="cuda") ** 2.0
        g = 1e-3 * g + T.bmm(randn(T, (n, r, q), F32, seed + 1) / fade, randn(T, (n, q, c), F32, seed + 2))
    elif kind == "lower rank":
        q = min(3, k)
        g = 1e-5 * g + T.bmm(randn(T, (n, r, q), F32, seed + 1), randn(T, (n, q, c), F32, seed + 2))
    elif kind == "diagonal":
        d = T.exp(randn(T, (n, k), F32, seed))
        g = T.zeros_like(g)
        T.diagonal(g, dim1=1, dim2=2).copy_(d)
    return g.to(T.bfloat16)


SHORT = [(1, 1), (1, 5), (2, 2), (2, 3), (3, 2), (2, 16), (4, 4), (9, 4), (8, 8), (8, 64), (3, 512), (512, 3), (16, 16), (16, 17), (17, 16),
         (15, 500), (500, 15), (16, 512)]


@pytest.mark.parametrize("kind", ["normal", "low rank", "lower rank", "diagonal"])
@pytest.mark.parametrize("r,c", SHORT)
def test_short_sides(T, Z, r, c, kind):
    """Sides of up to 16: within 0.001 for the default polynomial."""
    g = kinds(T, kind, 300, r, c, 7)
    got = orthogonalized(T, Z, g)
    e = off(T, got, ortho64(T, g))
    assert float(e.max()) <= 0.001 + HALF, (float(e.median()), float(e.max()))
    assert T.equal(got, orthogonalized(T, Z, g))


@pytest.mark.parametrize("kind", ["normal", "low rank", "lower rank", "diagonal"])
@pytest.mark.parametrize("r,c", [(17, 17), (65, 33), (20, 500), (64, 64), (128, 128), (96, 160), (200, 260), (17, 5000), (64, 300)])
def test_longer_sides(T, Z, r, c, kind):
    """Longer ones: within 0.004 where many entries count, 0.02 where few do."""
    g = kinds(T, kind, 60, r, c, 9)
    e = off(T, orthogonalized(T, Z, g), ortho64(T, g))
    assert float(e.max()) <= (0.02 if kind == "diagonal" else 0.004) + HALF, (float(e.median()), float(e.max()))


@pytest.mark.parametrize("kind", ["normal", "low rank", "lower rank"])
@pytest.mark.parametrize("r,c", [(9, 12), (24, 30), (150, 200), (256, 256), (40, 900), (900, 40)])
@pytest.mark.parametrize("poly", [(7, 3.4445, -4.7750, 2.0315, 1e-7), (8, 1.875, -1.25, 0.375, 1e-7), (10, 1.875, -1.25, 0.375, 1e-7),
                                  (12, 1.875, -1.25, 0.375, 1e-7), (14, 1.875, -1.25, 0.375, 1e-7), (22, 1.5, -0.5, 0.0, 1e-7)], ids=str)
def test_other_polynomials(T, Z, poly, r, c, kind):
    """Weak directions that the steps bring up: within 0.005 up to |a|^steps of 500, 0.02 up to 10000."""
    g = kinds(T, kind, 10, r, c, 11)
    e = off(T, orthogonalized(T, Z, g, poly), ortho64(T, g, *poly))
    assert float(e.max()) <= (0.005 if poly[1] ** poly[0] <= 500 else 0.02) + HALF, (float(e.median()), float(e.max()))


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

def test_longest_side(T, Z):
    """2^30 rows of one element, and one row into 2^30 outputs."""
    n = 1 << 30
    plan, long = Z.zero_plan(2, 1, [1, 1], 0, 1), Z.zero_plan(n, 1, [n], 0, 1)
    params = T.tensor([1.5, 0.25], dtype=T.bfloat16, device="cuda")
    x = randn(T, (n, 1), BF16, 1)
    y = T.empty_like(x)
    ws = T.empty(max(Z.zero_linear_workspace_bytes(plan, 0, 1, n), Z.zero_linear_input_grad_workspace_bytes(plan, 0, 1, n),
                     Z.zero_linear_weight_grad_workspace_bytes(plan, 0, 1, n), Z.zero_linear_workspace_bytes(long, 0, 1, 1)), dtype=T.uint8, device="cuda")
    Z.zero_linear(plan, 0, 1, params, BF16, x, y, bias=1, workspace=ws)
    same = lambda got, form: all(T.equal(a, form(b.float()).bfloat16()) for a, b in zip(got.view(-1).split(n // 8), x.view(-1).split(n // 8)))  # noqa: E731
    assert same(y, lambda v: 1.5 * v + 0.25)
    Z.zero_linear_input_grad(plan, 0, 1, params, BF16, x, y, workspace=ws)
    assert same(y, lambda v: 1.5 * v)
    # Whole numbers at places all over the rows: sums without rounding.
    at = T.arange(64, device="cuda") * ((n - 1) // 63)
    x.zero_()
    y.zero_()
    x.view(-1)[at] = T.arange(64, device="cuda").bfloat16()
    y.view(-1)[at] = 2
    grad = T.empty(2, device="cuda")
    Z.zero_linear_weight_grad(plan, 0, 1, y, x, BF16, 1.0, grad, Z.ZERO_F32, bias=1, workspace=ws)
    assert grad.tolist() == [2 * 63 * 64 / 2, 128]
    x.normal_()
    Z.zero_linear(long, 0, 1, x.view(-1), BF16, params[:1].view(1, 1), y.view(1, n), workspace=ws)
    assert same(y, lambda v: 1.5 * v)


def test_no_outputs(T, Z):
    """Back from a layer without outputs: the addend alone, whatever the sizes."""
    for n, inner in ((5, 3), (1 << 20, 33)):
        plan = Z.zero_plan(1, 1, [1, 0], 0, 1)
        params = T.ones(1, dtype=T.bfloat16, device="cuda")
        add, dx = randn(T, (n, inner), BF16, 1), T.empty((n, inner), dtype=T.bfloat16, device="cuda")
        ws = T.empty(max(1, Z.zero_linear_input_grad_workspace_bytes(plan, 1, inner, n)), dtype=T.uint8, device="cuda")
        Z.zero_linear_input_grad(plan, 1, inner, params, BF16, T.empty((n, 0), dtype=T.bfloat16, device="cuda"), dx, addend=add, workspace=ws)
        assert T.equal(dx, add)


# ---------------------------------------------------------------------------
# Activations
# ---------------------------------------------------------------------------

def act64(T, kind, z):
    if kind == GELU:
        return z * 0.5 * T.special.erfc(-z * math.sqrt(0.5))
    if kind == GELU_TANH:
        return z * T.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z * T.sigmoid(z)


def slope64(T, kind, z):
    z = z.detach().clone().requires_grad_(True)
    return T.autograd.grad(act64(T, kind, z).sum(), z)[0]


# exp2's argument t is rounded relative to itself, which exp2 makes an error of ln 2 |t| times
# that; |t| is at most 126 where the value is not below the smallest normal number.  Roundings of
# 2^-24 = 6e-8 and constants off by up to 3e-8, in all: silu 1 and one constant (7.3e-8), gelu 2 and
# one (1.32e-7) beside erfcx's 1.2e-6, gelu_tanh 5 and two (3.5e-7); a few roundings of the rest.
FAR = {GELU: 1.5e-5, GELU_TANH: 3.5e-5, SILU: 1e-5}
NEAR = 5e-6           # from z = -4 on, where |t| is below 16 (gelu_tanh: 16 ln 2 3.5e-7 = 3.9e-6)


@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU])
def test_activation_accuracy(T, Z, act):
    """An activation of sums that are no 16-bit numbers, seen to more bits than bf16
    has: the first result comes back as the residual of a second call, which leaves
    what it had rounded off."""
    plan = Z.zero_plan(3, 1, [3], 0, 1)
    w = T.tensor([1.0, 2.0 ** -8, 2.0 ** -15], dtype=T.bfloat16, device="cuda")
    g = T.Generator(device="cuda").manual_seed(4)
    x = T.randint(-127, 128, (1 << 21, 3), device="cuda", generator=g).bfloat16()      # sums of 22 bits: exact in fp32
    x[:, 0].uniform_(-100 if act == SILU else -14, 14, generator=g)
    x[:, 0].mul_(128).round_().div_(128)
    y, r = (T.empty((x.shape[0], 1), dtype=T.bfloat16, device="cuda") for _ in range(2))
    ws = T.empty(Z.zero_linear_workspace_bytes(plan, 0, 3, x.shape[0]), dtype=T.uint8, device="cuda")
    Z.zero_linear(plan, 0, 3, w, BF16, x, y, act=act, workspace=ws)
    Z.zero_linear(plan, 0, 3, w, BF16, x, r, act=act, residual=-y, workspace=ws)
    z = x.double() @ w.double()
    assert bool((z == z.float().double()).all())
    want = act64(T, act, z)
    err = (y[:, 0].double() + r[:, 0].double() - want).abs()
    room = 2.0 ** -8 * r[:, 0].double().abs() + 2.0 ** -119      # r's own rounding, half a step of bf16
    bound = T.where(z > -4, NEAR, FAR[act])
    assert bool((err <= room + bound * want.abs()).all()), float(((err - room) / want.abs()).max())


@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU])
def test_slope_accuracy(T, Z, act):
    """The same of the slopes, at every bf16 number, through the gradient's addend."""
    bits = T.arange(-32768, 32768, dtype=T.int32, device="cuda").to(T.int16).view(T.bfloat16)
    z = bits[bits.double().abs() < 128].view(-1, 1)
    plan = Z.zero_plan(1, 1, [1], 0, 1)
    one = T.ones(1, dtype=T.bfloat16, device="cuda")
    dz = T.ones_like(z)
    y, r = T.empty_like(z), T.empty_like(z)
    Z.zero_linear_input_grad(plan, 0, 1, one, BF16, dz, y, act=act, pre=z)
    Z.zero_linear_input_grad(plan, 0, 1, one, BF16, dz, r, act=act, pre=z, addend=-y)
    want = slope64(T, act, z.double())
    err = (y.double() + r.double() - want).abs()
    room = 2.0 ** -8 * r.double().abs() + 2.0 ** -119 + T.where(z.abs() <= 3, 1e-6, 0.0)
    assert bool((err <= room + FAR[act] * want.abs()).all()), float(((err - room) / want.abs()).max())


# ---------------------------------------------------------------------------
# Gradients against differences
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act", [GELU, GELU_TANH, SILU])
def test_gradients_against_differences(T, Z, act):
    """Every entry of dx, dW and db against central differences of the layer itself,
    in fp16, to a bound that half a gradient, or one and a half, could not meet."""
    n, inner, outer = 9, 24, 17
    sizes = [inner * outer, outer]
    plan = Z.zero_plan(sum(sizes), 1, sizes, 0, 1)
    # Multiples of 2^-6 and steps of 2^-3: exact in fp16, before and behind a step.
    grid = lambda shape, seed, top: (randn(T, shape, F32, seed) * 32).round().clamp(-64 * top, 64 * top).div(64).half()   # noqa: E731
    params, x, weight = grid((plan.psi_pad,), 1, 0.5), grid((n, inner), 2, 1), grid((n, outer), 3, 2) * 4
    y, pre = (T.empty((n, outer), dtype=T.float16, device="cuda") for _ in range(2))

    def layer(p, v):
        Z.zero_linear(plan, 0, inner, p, F16, v, y, bias=1, act=act, pre=pre)
        return y.double()

    y0 = layer(params, x).clone()
    farthest = float(pre.double().abs().max())
    dz, dx = T.empty_like(y), T.empty_like(x)
    Z.zero_activation_grad(weight, pre, dz, F16, act)
    Z.zero_linear_input_grad(plan, 0, inner, params, F16, dz, dx)
    grad = T.zeros(plan.psi_pad, device="cuda")
    ws = T.empty(Z.zero_linear_weight_grad_workspace_bytes(plan, 0, inner, n), dtype=T.uint8, device="cuda")
    Z.zero_linear_weight_grad(plan, 0, inner, dz, x, F16, 1.0, grad, F32, bias=1, workspace=ws)
    step = 2.0 ** -3
    c = weight.double()
    t = T.linspace(-20, 20, 40001, dtype=T.float64, device="cuda")
    z = t.clone().requires_grad_(True)
    d = act64(T, act, z)
    for _ in range(3):
        d = T.autograd.grad(d.sum(), z, create_graph=True)[0]
    third = float(d.detach().abs().max())
    for buf, got in ((x, dx), (params, grad)):
        want, bound = [], []
        for i in range(buf.numel()):
            ends = []
            for sign in (1, -1):
                moved = buf.clone()
                moved.view(-1)[i] += sign * step
                ends.append((layer(params, moved) if buf is x else layer(moved, x)).clone())
            want.append(float(((ends[0] - ends[1]) * c).sum()) / (2 * step))
            # The outputs that the entry reaches, and how fast they move with it.
            if buf is x:
                rate = T.zeros(n, outer, dtype=T.float64, device="cuda")
                rate[i // inner] = params[:sizes[0]].view(outer, inner)[:, i % inner].double().abs()
            else:
                o = i // inner if i < sizes[0] else i - sizes[0]
                rate = T.zeros(n, outer, dtype=T.float64, device="cuda")
                rate[:, o] = x[:, i % inner].double().abs() if i < sizes[0] else 1.0
            # y rounded to 2^-11 of itself at both ends, which may lie 1.2 step rate farther out; a third
            # derivative; dz rounded to 2^-11 of at most 1.2 |c| from a z that is rounded to 2^-11 of itself
            # (a slope changes by at most 0.8 of that); fp32's and dx's own rounding.
            size = y0.abs() + 1.2 * step * rate
            e = (c.abs() * (2.0 ** -11 * size / step + step ** 2 / 6 * third * rate ** 3)) * (rate > 0)
            e = e + c.abs() * rate * (2.0 ** -11 * 1.2 + 2.0 ** -11 * farthest * 0.8)
            bound.append(float(e.sum()) + 2.0 ** -11 * abs(float(got.view(-1)[i])) + 1e-6)
        want, bound, got = T.tensor(want), T.tensor(bound), got.view(-1).double().cpu()
        assert bool(((want - got).abs() <= bound).all())
        assert float(bound.norm()) <= 0.25 * float(got.norm())
        for factor in (0.0, 0.5, 1.5, 2.0):
            assert not bool(((want - factor * got).abs() <= bound).all())
