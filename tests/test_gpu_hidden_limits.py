"""The operators on the hidden matrices on the GPU: what the header promises at
its limits, held to its own figures."""
import pytest

from tests import ops_reference as R
from tests.ops_reference import BF16, F16

pytestmark = pytest.mark.gpu


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
