"""The 8-bit layer half at the ends of its ranges."""
import pytest
import torch

from activation_sparse_ffn_amd import _abi as A
from gpu_helpers import say
from test_gpu_q8 import DEV, check_norm

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------ norm

NORM_SIZES = [  # largest size of x and of the weights: 127 / max |h w| leaves fp32's normal numbers, scales do too
    (1.0, 1.0), (3e37, 1e3), (3e37, 1e5), (3e38, 1e6), (1e30, 1e13), (3e38, 1e8), (3e38, 3e38), (1e10, 1e-36), (1e10, 1e-43),
    (1e20, 1e-40), (1e-30, 1e38), (1e-40, 1e-3), (1e-44, 1e5)]


def sized_rows(T, d, sizes, seed):
    """Rows of which the first len(sizes) have these sizes, with one strong element in a hundred."""
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(T, d, generator=g, dtype=torch.float64) * 2 - 1
    x *= torch.where(torch.rand(T, d, generator=g) < 0.01, 1.0, 0.05)
    x[:, d // 3] = 1.0
    x[:len(sizes)] *= torch.tensor(sizes, dtype=torch.float64)[:, None]
    return x.float()


@pytest.mark.parametrize("d", [40, 1000, 4096, 9000])
def test_norm_codes_of_any_finite_product(d):
    """Rows up to fp32's largest number with weights of any size: every code is the nearest one, where the
    quotient's factors leave fp32's normal numbers too."""
    say(f"norm sizes {d}")
    for xs, ws in NORM_SIZES:
        x = sized_rows(3, d, [xs, xs / 7, xs / 1000], d)
        w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(1)))
        w = (w.double() / w.abs().max() * ws).float()
        q, s = torch.full((3, d), 99, dtype=torch.int8, device=DEV), torch.full((3,), -1.0, device=DEV)
        r = x.roll(1, 1) / 10
        for res in (None, r):
            ro = None if res is None else res.to(DEV)
            A.sfx_norm_q8(x.to(DEV), q, s, weight=w.to(DEV), residual=ro)
            check_norm((3, d, "f32", None if res is None else "f32", None, True, True), x, res, w, q, s, ro, None)


@pytest.mark.parametrize("d,T", [(333, 160000), (1000, 51000), (2041, 25000), (4096, 12400), (8190, 6300), (16384, 3200)])
def test_norm_codes_of_any_finite_product_many_rows(d, T):
    """The same where rows stay in registers (more than the last-level cache holds)."""
    say(f"norm sizes {T}x{d}")
    for ws in (1e3, 1e6, 1e13, 3e38, 1e-36, 1e-43):
        sizes = [3e38, 3e37, 1e30, 1e20, 1e10, 1.0, 1e-3, 1e-20, 1e-38, 1e-44]
        x = sized_rows(len(sizes), d, sizes, d)
        w = (1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(1)))
        w = (w.double() / w.abs().max() * ws).float()
        big = torch.ones(T, d, device=DEV)
        at = torch.linspace(0, T - 1, len(sizes)).long()
        big[at.to(DEV)] = x.to(DEV)
        q, s = torch.full((T, d), 99, dtype=torch.int8, device=DEV), torch.full((T,), -1.0, device=DEV)
        A.sfx_norm_q8(big, q, s, weight=w.to(DEV))
        check_norm((len(sizes), d, "f32", None, None, True, True), x, None, w, q.cpu()[at], s.cpu()[at], None, None)
