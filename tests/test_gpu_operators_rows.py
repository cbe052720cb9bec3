"""Layer norm, checkpoints and a training step at batches of many rows: blocks
that hold several rows, several rows per exchange of sums, rings that wrap, and
the last, smaller group.  Tolerances as in test_gpu_operators."""
import pytest
import torch

from muon_polar_orthogonalized_b200 import api
from tests import operator_refs as R
from tests.test_gpu_operators import SUM_TERMS, activations, dev, near, norm_bounds, rand, strided, ws  # noqa: F401
from tests.test_gpu_operators_together import Block

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = R.U32
EPS = float(torch.tensor(1e-5))

MANY = [(1187, 768), (2500, 1664), (3001, 4096), (1500, 40), (9001, 72), (2500, 2049), (1201, 4095), (4000, 13)]
WIDE = [(37, 5120), (1301, 5120), (11, 8192), (700, 8192), (450, 6144), (301, 4104), (500, 8200), (333, 14336), (300, 9001)]


@pytest.mark.parametrize("xdt,ydt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,cols", MANY + WIDE)
def test_layer_norm_forward(dev, xdt, ydt, rows, cols):
    for offset, with_bias in ((0.5, True), (-30.0, False)):
        x = rand((rows, cols), 1.5, xdt, 70, dev, offset)
        gain = rand((cols,), 0.2, F32, 71, dev, 1.0)
        bias = rand((cols,), 0.3, F32, 72, dev) if with_bias else None
        y = torch.full((rows, cols), float("nan"), dtype=ydt, device=dev)
        mean, rstd = torch.full((rows,), float("nan"), device=dev), torch.full((rows,), float("nan"), device=dev)
        api.muon_layer_norm_forward(x, gain, bias, y, mean, rstd, eps=1e-5)
        wy, wm, wr, by, bm, br = norm_bounds(x, gain, bias, EPS, ydt)
        near(mean, wm, bm)
        near(rstd, wr, br)
        near(y, wy, by)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1187, 768), (3001, 4096), (2500, 1664)])
def test_layer_norm_forward_in_place_and_strided(dev, dt, rows, cols):
    """The same bits as into another buffer, from rows further apart, and on top of x."""
    x = rand((rows, cols), 1.5, dt, 73, dev, 0.5)
    gain, bias = rand((cols,), 0.2, F32, 74, dev, 1.0), rand((cols,), 0.3, F32, 75, dev)
    outs = []
    for src, dst in ((x, torch.empty_like(x)), (strided(x, 8)[1], strided(x, 16)[1]), (x, x)):
        mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        api.muon_layer_norm_forward(src, gain, bias, dst, mean, rstd, eps=1e-5)
        outs.append((dst.clone(), mean, rstd))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))


@pytest.mark.parametrize("dt,gdt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", [(1187, 768), (2500, 1664), (9001, 72), (1201, 4095)] + WIDE)
def test_layer_norm_backward(dev, dt, gdt, rows, cols):
    x = rand((rows, cols), 1.5, dt, 76, dev, 0.5)
    dy = rand((rows, cols), 1.0, dt, 77, dev)
    gain = rand((cols,), 0.2, F32, 78, dev, 1.0)
    _, m, r = R.layer_norm(x, gain, None, 1e-5)
    mean, rstd = m.float().to(dev), r.float().to(dev)
    dx64, dg64, db64, mx, mg, mb = R.layer_norm_grad(dy, x, gain, mean, rstd)
    w = ws(api.muon_layer_norm_backward_workspace_size(rows, cols), dev)
    old = rand((2, cols), 1.0, gdt, 79, dev)
    dx = torch.full((rows, cols), float("nan"), dtype=dt, device=dev)
    dg, db = old[0].clone(), old[1].clone()
    api.muon_layer_norm_backward(dy, x, gain, mean, rstd, dx, dg, db, w, accumulate=True)
    near(dx, dx64, (SUM_TERMS + 12) * U * mx + R.HALF[dt] * dx64.abs() * 1.01 + R.TINY[dt])
    for got, want, mag, o in ((dg, dg64, mg, old[0]), (db, db64, mb, old[1])):
        total = want + R.f64(o)
        near(got, total, (rows + 4) * U * (mag + R.f64(o).abs()) + R.HALF[gdt] * total.abs() * 1.01 + R.TINY[gdt])


def encode(x):
    """R.checkpoint_encode for whole matrices: the same search, all blocks at a time."""
    x = R.f64(x)
    rows, cols = x.shape
    nb, pitch = (cols + 127) // 128, (cols + 15) // 16 * 16
    v = torch.zeros(rows, nb * 128, dtype=torch.float64)
    v[:, :cols] = x
    v = v.view(rows, nb, 128)
    big = v.abs().amax(2)
    p = torch.frexp(big)[1].double() - 9     # big = m 2^e, 1/2 <= m < 1: 448 = 7/8 2^9
    p = torch.where(448.0 * 2.0 ** p < big, p + 1, p).clamp(min=-124)
    p = torch.where(big == 0, torch.zeros_like(p), p)
    scaled = (v * 2.0 ** -p[:, :, None])
    mags = R.e4m3_values()[:127]
    j = torch.searchsorted(mags, scaled.abs()).clamp(max=126)
    lo = (j - 1).clamp(min=0)
    dj, dl = (mags[j] - scaled.abs()).abs(), (scaled.abs() - mags[lo]).abs()
    best = torch.where((dl < dj) | ((dl == dj) & (lo % 2 == 0)), lo, j) + 128 * torch.signbit(v)
    return best.to(torch.uint8).view(rows, nb * 128)[:, :pitch].contiguous(), (p + 127).to(torch.uint8)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(3000, 200), (10001, 129), (3001, 264), (20000, 24), (1500, 1025), (300, 9000)])
def test_checkpoint_of_many_rows(dev, dt, rows, cols):
    x = activations(rows, cols, dt, 80, dev)
    wq, we = encode(x)
    few = R.checkpoint_encode(x[:3])
    assert torch.equal(few[0], wq[:3]) and torch.equal(few[1], we[:3])
    ck = api.new_checkpoint(rows, cols, dev)
    ck.codes.fill_(0xEE)
    api.muon_checkpoint_pack(x, ck)
    assert torch.equal(ck.exponents.cpu(), we) and torch.equal(ck.codes.cpu(), wq)
    want = R.checkpoint_values(wq, we, cols)
    for odt in (F32, BF16):
        out = torch.full((rows, cols), float("nan"), dtype=odt, device=dev)
        api.muon_checkpoint_unpack(ck, out)
        assert torch.equal(R.f64(out), want)


@pytest.mark.parametrize("tokens,dim", [(150, 264), (2600, 264), (1300, 777)])
def test_every_stage_of_a_training_step(dev, tokens, dim):
    """What Block.check leaves out: the norm's outputs and dx, on the stage's own inputs."""
    b = Block(dev, dim=dim, tokens=tokens)
    b.forward()
    b.backward()
    b.check()
    wy, wm, wr, by, bm, br = norm_bounds(b.x, b.gain, b.bias, EPS, BF16)
    near(b.mean, wm, bm)
    near(b.rstd, wr, br)
    near(b.y, wy, by)
    dx, _, _, mx, _, _ = R.layer_norm_grad(b.dnorm, b.x, b.gain, b.mean, b.rstd)
    near(b.dx, dx, (SUM_TERMS + 12) * U * mx + R.HALF[BF16] * dx.abs() * 1.01 + R.TINY[BF16])
