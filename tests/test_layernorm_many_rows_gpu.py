"""dgamma of layer norm where rows are many: wide rows leave their mean and factor
in the workspace, row by row, over several launches and past 2^31 elements, and
another kernel reads them for its sums. Against fp64 sums taken in parts."""

import pytest
import torch

import int4_quantized_gemm_amd as tp
from tests.block_bounds import U
from tests.gpu_util import announce, dev

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _rows(m, k, d, seed):
    """Rows of different means and sizes, so that another row's statistics show."""
    g = torch.Generator(device=d).manual_seed(seed)
    x = torch.empty((m, k), dtype=torch.bfloat16, device=d)
    for r in range(0, m, 8192):
        part = torch.randn((min(8192, m - r), k), generator=g, device=d)
        size = 2.0 ** torch.randint(-3, 4, (len(part), 1), generator=g, device=d).float()
        x[r:r + len(part)] = (part + torch.randn((len(part), 1), generator=g, device=d)) * size
    return x


# rows that keep their sums; wide rows in two launches; past 2^31 elements. few: only
# the last rows and some others have a gradient, so that each of them shows
@pytest.mark.parametrize("m,k", [(2 ** 21 + 77, 1024), (2 ** 21 + 77, 4352), (140001, 16384)])
@pytest.mark.parametrize("few", [False, True])
def test_weight_gradients_of_many_rows(m, k, few):
    d = dev()
    announce("layer norm weight gradients of many rows", m, k, few)
    t, dy = _rows(m, k, d, 1), _rows(m, k, d, 2)
    if few:
        g = torch.Generator(device=d).manual_seed(3)
        rows = torch.cat([torch.randint(0, m, (20,), generator=g, device=d), torch.arange(m - 100, m, device=d)])
        kept = dy[rows].clone()
        dy.zero_()
        dy[rows] = kept
    _, _, dgamma, dbeta = tp.tp_layernorm_rotate_backward(dy, t, eps=EPS, rotate=False)
    zero = lambda: torch.zeros(k, dtype=torch.float64, device=d)  # noqa: E731
    want, size, err, total, mag = zero(), zero(), zero(), zero(), zero()
    for r in range(0, m, 8192):
        g, v = dy[r:r + 8192].double(), t[r:r + 8192].double()
        mean = v.mean(dim=1, keepdim=True)
        v -= mean
        f = torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
        # as tests/branch_bounds.py: two subtractions, the factor's rounding and the
        # product, the mean's two parts
        err += (g.abs() * (4 * U * v.abs() * f + 2.0 ** -47 * mean.abs() * f)).sum(dim=0)
        v *= f * g
        want += v.sum(dim=0)
        size += v.abs().sum(dim=0)
        total += g.sum(dim=0)
        mag += g.abs().sum(dim=0)
    # rows that one thread adds one by one: 512 blocks, or the 16 sets of 512 / groups
    # shares; then its block's 16, and the partial rows (zeros are added exactly)
    groups = k // 256
    adds = 120 if few else (m // 512 if groups <= 16 else m // (16 * -(-512 // groups))) + 1 + 16 + 512
    assert torch.all((dgamma.double() - want).abs() <= 1.01 * (err + adds * U * size)), "dgamma"
    assert torch.all((dbeta.double() - total).abs() <= 1.01 * adds * U * mag), "dbeta"
    if few:  # no room for one row's statistics in another's place
        assert float(((err + adds * U * size) / want.std()).max()) < 1e-3
