"""The weight gradient from an 8-bit checkpoint where a tile's row blocks go
round the ring of stages several times, against 64-bit statements."""
import pytest
import torch

from muon_polar_orthogonalized_b200 import _native as N
from muon_polar_orthogonalized_b200 import api
from tests import operator_refs as R
from tests.test_gpu_operators import dev, rand, wg_checkpoint, whole, ws  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("ddt", [BF16, F32])
@pytest.mark.parametrize("rows,n,k", [(1024, 2048, 1024), (4096, 768, 768), (2048, 1024, 1024), (1500, 1664, 768),
                                      (1987, 500, 777), (5000, 96, 40)])
def test_many_stages_per_tile_on_whole_numbers(dev, ddt, rows, n, k):
    """16 to 79 row blocks a tile (three times as many for fp32 dy).  The sums
    are whole numbers below 2^24: every stage's codes and exponents must meet
    their own rows of dy."""
    ck, values = wg_checkpoint(rows, k, 60, dev, "whole")
    # powers of two that change from row to row and block to block
    g = torch.Generator().manual_seed(61)
    shift = torch.randint(0, 3, ck.exponents.shape, generator=g).to(torch.uint8)
    ck.exponents += shift.to(dev)
    values = R.checkpoint_values(ck.codes, ck.exponents, k)
    dy = whole((rows, n), -4, 4, ddt, 62, dev)
    want, _ = R.weight_grad(dy, values)
    w = ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, ddt), dev)
    for _ in range(3):
        grad = torch.full((n, k), float("nan"), device=dev)
        api.muon_checkpoint_weight_grad(dy, ck, grad, w)
        assert torch.equal(R.f64(grad), want)
        assert api.muon_query_status(w) == N.MUON_OK


@pytest.mark.parametrize("ddt", [BF16, F32])
@pytest.mark.parametrize("rows,n,k", [(777, 1664, 768), (2000, 300, 260), (4096, 512, 512)])
def test_error_of_long_sums(dev, ddt, rows, n, k):
    """The tensor cores add 16 rows at a time and cut what lies below a step of
    the running sum: half a step a time on average, at most u = 2^-24 of it.  The
    terms' signs are random, so that the running sum after j of J groups is
    sqrt(j / J) of the last in root mean square, 2/3 on average over j.  fp32
    dy's lower planes are added to sums 2^-8 of it and less: 2 J u 2^-8.  The
    result is rounded once."""
    ck, values = wg_checkpoint(rows, k, 63, dev, "plain")
    dy = rand((rows, n), 1.0, ddt, 64, dev)
    want, _ = R.weight_grad(dy, values)
    grad = torch.empty(n, k, device=dev)
    api.muon_checkpoint_weight_grad(dy, ck, grad, ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, ddt), dev))
    groups = (rows + 15) // 16
    error = float((R.f64(grad) - want).norm() / want.norm())
    assert error <= (2 / 3 * groups + 2 * groups * 2.0 ** -8 + 1) * R.U32


def test_small_fp32_dy(dev):
    """fp32 dy down to 2^-120: its three bf16 parts keep all that lies at or above
    bf16's smallest number, 2^-133, and drop less than that of each value."""
    rows, n, k = 300, 136, 200
    ck, values = wg_checkpoint(rows, k, 65, dev, "plain")
    g = torch.Generator().manual_seed(66)
    dy = torch.randn(rows, n, generator=g) * torch.pow(2.0, torch.randint(-120, -100, (1, n), generator=g).float())
    dy = dy.to(dev)
    want, mag = R.weight_grad(dy, values)
    dropped = 2.0 ** -133 * values.abs().sum(0)
    grad = torch.empty(n, k, device=dev)
    api.muon_checkpoint_weight_grad(dy, ck, grad, ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, F32), dev))
    bound = dropped + (2 * rows + 8) * R.U32 * mag + R.U32 * want.abs() + 2.0 ** -149 * rows
    assert bool(((R.f64(grad) - want).abs() <= bound).all())


@pytest.mark.parametrize("ddt", [BF16, F32])
def test_subnormal_dy_is_kept(dev, ddt):
    """Whole multiples of bf16's smallest number, 2^-133: the sums are fp32
    subnormals and small normals, all exact."""
    rows, n, k = 200, 72, 130
    ck, values = wg_checkpoint(rows, k, 67, dev, "whole")
    dy = (whole((rows, n), -4, 4, F32, 68, dev).double() * 2.0 ** -133).to(ddt)
    want, _ = R.weight_grad(dy, values)
    assert float(want.abs().max()) > 0
    grad = torch.empty(n, k, device=dev)
    api.muon_checkpoint_weight_grad(dy, ck, grad, ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, ddt), dev))
    assert torch.equal(R.f64(grad), want)
