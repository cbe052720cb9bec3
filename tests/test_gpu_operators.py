"""The operators that make the optimizer's gradients, on the GPU, against the
64-bit statements in operator_refs.

Tolerances count roundings.  u = 2^-24 is half a step of fp32, h half a step
of the output type.  A sum of m terms added in any order has an error of at
most (m - 1) u times the sum of their magnitudes (to first order), and an
output is rounded once more, by h relative.  Sums of small whole numbers are
exact in fp32 in any order, and are compared for equality.
"""
import pytest
import torch

from muon_polar_orthogonalized_b200 import api
from muon_polar_orthogonalized_b200 import _native as N
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = R.U32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.fail("GPU test selected but no CUDA device is visible")
    return torch.device("cuda:0")


def rand(shape, std, dtype, seed, dev, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + offset).to(dtype).to(dev)


def whole(shape, lo, hi, dtype, seed, dev):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=g).to(dtype).to(dev)


def ws(nbytes, dev, fill=0xFF):
    """A workspace of exactly the needed size, poisoned."""
    return torch.full((max(int(nbytes), 256),), fill, dtype=torch.uint8, device=dev)


def near(got, want, bound):
    got = R.f64(got)
    bad = ~((got - want).abs() <= bound)
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} out of bounds, worst excess " \
                                f"{float(((got - want).abs() - bound).max()):.3e}"


def strided(t, extra):
    """The same values in rows `extra` elements further apart, poisoned between."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), 1e30, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf, buf[:, :t.shape[1]]


def token_ids(n, vocab, kind, seed, dtype=torch.int64):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        ids = torch.full((n,), vocab - 1)
    elif kind == "none":
        ids = torch.full((n,), -1)
    elif kind == "ascending":
        ids = torch.arange(n) % vocab
    elif kind == "zipf":
        w = 1.0 / (torch.arange(vocab, dtype=torch.float64) + 2.7)
        ids = torch.multinomial(w, n, replacement=True, generator=g) if n else torch.zeros(0, dtype=torch.int64)
    else:
        ids = torch.randint(0, vocab, (n,), generator=g)
    if n > 8 and kind != "none":
        ids[torch.randint(0, n, (n // 8,), generator=g)] = -1
        ids[n // 2] = vocab            # just past the table
        ids[n // 3] = 2 ** 31 - 1
    return ids.to(dtype)


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("tdt,odt", [(F32, BF16), (F32, F32), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("vocab,dim,n", [(1, 1, 1), (7, 3, 5), (50, 8, 33), (100, 257, 40), (1000, 768, 129), (33, 1664, 64)])
def test_embedding_forward(dev, tdt, odt, vocab, dim, n):
    table = rand((vocab, dim), 0.02, tdt, 1, dev)
    ids = token_ids(n, vocab, "random", 2)
    scale = 27.75
    want = R.embedding(table, ids, scale)
    for idt in (torch.int64, torch.int32):
        out = torch.full((n, dim), float("nan"), dtype=odt, device=dev)
        api.muon_embedding_forward(table, ids.to(idt).to(dev), out, scale=scale)
        # the fp32 product, then the output type
        near(out, want, want.abs() * (U + R.HALF[odt] * (1 + U)) + R.TINY[odt])


def test_embedding_forward_strided_and_untouched(dev):
    table = rand((64, 40), 1.0, F32, 3, dev)
    ids = token_ids(21, 64, "random", 4).to(dev)
    for extra in (8, 3):
        buf = torch.full((21, 40 + extra), 7.0, dtype=BF16, device=dev)
        api.muon_embedding_forward(table, ids, buf[:, :40])
        assert bool((buf[:, 40:] == 7.0).all())
        near(buf[:, :40], R.embedding(table, ids, 1.0), R.embedding(table, ids, 1.0).abs() * R.HALF[BF16])
    out = torch.empty(0, 40, dtype=BF16, device=dev)
    api.muon_embedding_forward(table, torch.empty(0, dtype=torch.int64, device=dev), out)


@pytest.mark.parametrize("ddt,gdt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("vocab,dim,n,kind", [
    (1, 1, 1, "random"), (3, 5, 2, "none"), (40, 16, 0, "random"), (64, 24, 300, "one"), (10, 257, 129, "random"),
    (500, 264, 4099, "zipf"), (513, 768, 1000, "ascending"), (70000, 8, 20000, "zipf"), (300000, 2, 700, "random"),
])
def test_embedding_grad(dev, ddt, gdt, vocab, dim, n, kind):
    ids = token_ids(n, vocab, kind, 5)
    scale = -1.5
    dout = rand((n, dim), 1.0, ddt, 6, dev)
    want, mag, cnt = R.embedding_grad(dout, ids, vocab, scale)
    old = rand((vocab, dim), 1.0, gdt, 7, dev)
    w = ws(api.muon_embedding_grad_workspace_size(vocab, dim, n), dev)
    for acc in (False, True):
        grad = old.clone()
        api.muon_embedding_grad(dout, ids.to(dev), grad, w, scale=scale, accumulate=acc)
        total = want + (R.f64(old) if acc else 0)
        bound = (cnt[:, None] + 1) * U * (mag + (R.f64(old).abs() if acc else 0)) * 1.01 + \
            R.HALF[gdt] * total.abs() * 1.01 + R.TINY[gdt]
        near(grad, total, bound)
        if acc:
            same = cnt == 0
            assert torch.equal(grad.cpu()[same], old.cpu()[same])


@pytest.mark.parametrize("vocab,dim,n,kind", [(50304, 16, 30011, "zipf"), (5, 72, 70001, "random"), (2, 9, 5000, "one"),
                                              (131073, 8, 65536, "ascending"), (1000, 40, 262147, "zipf")])
def test_embedding_grad_of_whole_numbers_is_exact(dev, vocab, dim, n, kind):
    """Sums of whole numbers below 2^24: every token must land in its row once."""
    ids = token_ids(n, vocab, kind, 8)
    dout = whole((n, dim), -8, 8, BF16, 9, dev)
    want, _, _ = R.embedding_grad(dout, ids, vocab, 2.0)
    w = ws(api.muon_embedding_grad_workspace_size(vocab, dim, n), dev)
    grad = torch.full((vocab, dim), float("nan"), device=dev)
    api.muon_embedding_grad(dout, ids.to(dev), grad, w, scale=2.0)
    assert torch.equal(R.f64(grad), want)
    api.muon_embedding_grad(dout, ids.to(torch.int32).to(dev), grad, w, scale=2.0, accumulate=True)
    assert torch.equal(R.f64(grad), 2 * want)


def test_embedding_grad_repeats_bit_for_bit(dev):
    ids = token_ids(9000, 700, "zipf", 10).to(dev)
    dout = rand((9000, 96), 1.0, F32, 11, dev)
    w = ws(api.muon_embedding_grad_workspace_size(700, 96, 9000), dev)
    outs = []
    for fill in (0xFF, 0x00, 0x5A):
        w.fill_(fill)
        g = torch.empty(700, 96, device=dev)
        api.muon_embedding_grad(dout, ids, g, w)
        outs.append(g)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_embedding_grad_strided_rows(dev):
    ids = token_ids(200, 50, "random", 12)
    dout = whole((200, 24), -4, 4, F32, 13, dev)
    want, _, _ = R.embedding_grad(dout, ids, 50, 1.0)
    for extra in (4, 1):
        _, view = strided(dout, extra)
        g = torch.empty(50, 24, device=dev)
        api.muon_embedding_grad(view, ids.to(dev), g, ws(api.muon_embedding_grad_workspace_size(50, 24, 200), dev))
        assert torch.equal(R.f64(g), want)


# --------------------------------------------------------------- layer norm
# A row's sum: at most 32 terms per thread, then two trees of 5 levels.
SUM_TERMS = 32 + 10


def norm_bounds(x, gain, bias, eps, ydt):
    y, mean, rstd = R.layer_norm(x, gain, bias, eps)
    x64 = R.f64(x)
    e_mean = (SUM_TERMS + 2) * U * x64.abs().mean(1) + U * mean.abs()
    xc = (x64 - mean[:, None]).abs()
    # centred values err by a rounding each and by the mean's error; the
    # variance by its sum's roundings and the square of the mean's error
    e_rstd = (SUM_TERMS + 8) * U + e_mean * rstd * (2 * U + e_mean * rstd)
    y_abs = xc * rstd[:, None] * R.f64(gain).abs()
    by = y_abs * (e_rstd[:, None] + 6 * U) + (e_mean * rstd)[:, None] * R.f64(gain).abs() * 1.01 + \
        (0 if bias is None else R.f64(bias).abs() * 2 * U) + R.HALF[ydt] * y.abs() * 1.01 + R.TINY[ydt]
    return y, mean, rstd, by, e_mean, e_rstd * rstd


NORM_SHAPES = [(1, 1), (3, 2), (5, 7), (9, 64), (17, 257), (33, 768), (4, 1000), (6, 1024), (5, 1032), (7, 1664),
               (3, 2049), (4, 4096), (2, 8191), (2, 14336), (2, 16384)]


@pytest.mark.parametrize("xdt,ydt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES)
def test_layer_norm_forward(dev, xdt, ydt, rows, cols):
    for offset, with_bias in ((0.0, True), (40.0, False)):
        x = rand((rows, cols), 1.5, xdt, 20, dev, offset)
        gain = rand((cols,), 0.2, F32, 21, dev, 1.0)
        bias = rand((cols,), 0.3, F32, 22, dev) if with_bias else None
        y = torch.full((rows, cols), float("nan"), dtype=ydt, device=dev)
        mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        api.muon_layer_norm_forward(x, gain, bias, y, mean, rstd, eps=1e-5)
        wy, wm, wr, by, bm, br = norm_bounds(x, gain, bias, float(torch.tensor(1e-5)), ydt)
        near(mean, wm, bm)
        near(rstd, wr, br)
        near(y, wy, by)


@pytest.mark.parametrize("dt,gdt", [(F32, F32), (BF16, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,cols", NORM_SHAPES + [(2500, 40), (3000, 768), (700, 4096), (400, 13)])
def test_layer_norm_backward(dev, dt, gdt, rows, cols):
    x = rand((rows, cols), 1.5, dt, 23, dev, 0.5)
    dy = rand((rows, cols), 1.0, dt, 24, dev)
    gain = rand((cols,), 0.2, F32, 25, dev, 1.0)
    _, m, r = R.layer_norm(x, gain, None, 1e-5)
    mean, rstd = m.float().to(dev), r.float().to(dev)
    dx64, dg64, db64, mx, mg, mb = R.layer_norm_grad(dy, x, gain, mean, rstd)
    w = ws(api.muon_layer_norm_backward_workspace_size(rows, cols), dev)
    old = rand((2, cols), 1.0, gdt, 26, dev)
    for acc, with_bias in ((False, True), (True, True), (False, False)):
        dx = torch.full((rows, cols), float("nan"), dtype=dt, device=dev)
        dg, db = old[0].clone(), old[1].clone()
        api.muon_layer_norm_backward(dy, x, gain, mean, rstd, dx, dg, db if with_bias else None, w, accumulate=acc)
        near(dx, dx64, (SUM_TERMS + 12) * U * mx + R.HALF[dt] * dx64.abs() * 1.01 + R.TINY[dt])
        for got, want, mag, o in ((dg, dg64, mg, old[0]), (db, db64, mb, old[1])):
            if got is db and not with_bias:
                assert torch.equal(db, old[1])
                continue
            total = want + (R.f64(o) if acc else 0)
            near(got, total, (rows + 4) * U * (mag + (R.f64(o).abs() if acc else 0)) + R.HALF[gdt] * total.abs() * 1.01
                 + R.TINY[gdt])


def test_layer_norm_gradients_agree_with_differences(dev):
    """Central differences of the 64-bit forward pass."""
    rows, cols = 3, 20
    x, dy = rand((rows, cols), 1.0, F32, 27, dev), rand((rows, cols), 1.0, F32, 28, dev)
    gain, bias = rand((cols,), 0.2, F32, 29, dev, 1.0), rand((cols,), 0.2, F32, 30, dev)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    api.muon_layer_norm_forward(x, gain, bias, y, mean, rstd, eps=1e-5)
    dx, dg, db = torch.empty_like(x), torch.empty(cols, device=dev), torch.empty(cols, device=dev)
    api.muon_layer_norm_backward(dy, x, gain, mean, rstd, dx, dg, db,
                                 ws(api.muon_layer_norm_backward_workspace_size(rows, cols), dev))
    leaves = [R.f64(x), R.f64(gain), R.f64(bias)]

    def loss(a):
        return (R.layer_norm(a[0], a[1], a[2], 1e-5)[0] * R.f64(dy)).sum().item()
    h = 1e-5
    for k, got in enumerate((dx, dg, db)):
        flat = leaves[k].reshape(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(leaves)
            flat[i] = keep - h
            down = loss(leaves)
            flat[i] = keep
            # differences err by h^2 times a third derivative of order 10; the gradient by fp32 sums
            assert abs((up - down) / (2 * h) - got.reshape(-1)[i].item()) < 2e-5


def test_layer_norm_in_place_and_strided(dev):
    rows, cols = 37, 1664
    x = rand((rows, cols), 1.0, BF16, 31, dev)
    gain, bias = rand((cols,), 0.2, F32, 32, dev, 1.0), rand((cols,), 0.2, F32, 33, dev)
    dy = rand((rows, cols), 1.0, BF16, 34, dev)
    w = ws(api.muon_layer_norm_backward_workspace_size(rows, cols), dev)

    def run(x, y, dy, dx):
        mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        dg, db = torch.empty(cols, device=dev), torch.empty(cols, device=dev)
        keep = x.clone()
        api.muon_layer_norm_forward(x, gain, bias, y, mean, rstd)
        out = y.clone()
        api.muon_layer_norm_backward(dy, keep, gain, mean, rstd, dx, dg, db, w)
        return out, mean, rstd, dx.clone(), dg, db
    base = run(x, torch.empty_like(x), dy, torch.empty_like(x))
    y = x.clone()
    d = dy.clone()
    for a, b in zip(base, run(y, y, d, d)):
        assert torch.equal(a, b)
    for extra in (8, 1):
        bufs = [strided(t, extra)[1] for t in (x, torch.zeros_like(x), dy, torch.zeros_like(x))]
        for k, (a, b) in enumerate(zip(base, run(*bufs))):
            if extra == 8:
                assert torch.equal(a, b), k
            else:   # another order of the same sums
                assert float((a.float() - b.float()).abs().max()) <= 2e-2 * float(a.float().abs().max()), k
    api.muon_layer_norm_forward(x[:0], gain, bias, y[:0], torch.empty(0, device=dev), torch.empty(0, device=dev))
    dg, db = torch.ones(cols, device=dev), torch.ones(cols, device=dev)
    for acc, val in ((True, 1.0), (False, 0.0)):
        api.muon_layer_norm_backward(dy[:0], x[:0], gain, torch.empty(0, device=dev), torch.empty(0, device=dev),
                                     x[:0], dg, db, w, accumulate=acc)
        assert bool((dg == val).all()) and bool((db == val).all())


def test_layer_norm_of_constant_rows_and_bad_values(dev):
    cols = 768
    x = torch.full((4, cols), 3.0, device=dev)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 9] = float("nan")
    gain, bias = torch.ones(cols, device=dev), torch.full((cols,), 0.5, device=dev)
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device=dev), torch.empty(4, device=dev)
    api.muon_layer_norm_forward(x, gain, bias, y, mean, rstd, eps=1e-5)
    assert bool((y[:2] == 0.5).all()) and bool(torch.isnan(y[2:]).all())
    near(rstd[:2], torch.full((2,), 1e5 ** 0.5, dtype=torch.float64), 1e5 ** 0.5 * 4 * U)


# -------------------------------------------------------------- checkpoints
CKPT_SHAPES = [(1, 1), (3, 7), (2, 16), (5, 127), (4, 128), (3, 129), (7, 1000), (2, 1664), (1, 4100)]


def activations(rows, cols, dtype, seed, dev):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.pow(2.0, torch.randint(-30, 30, (rows, 1), generator=g).float())
    x[torch.rand(rows, cols, generator=g) < 0.05] = 0
    x[torch.rand(rows, cols, generator=g) < 0.05] *= 2.0 ** -12
    return x.to(dtype).to(dev)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,cols", CKPT_SHAPES)
def test_checkpoint_codes_exponents_and_values(dev, dt, rows, cols):
    x = activations(rows, cols, dt, 40, dev)
    wq, we = R.checkpoint_encode(x)
    ck = api.new_checkpoint(rows, cols, dev)
    ck.codes.fill_(0xEE)
    api.muon_checkpoint_pack(x, ck)
    assert torch.equal(ck.exponents.cpu(), we)
    assert torch.equal(ck.codes.cpu(), wq)
    want = R.checkpoint_values(wq, we, cols)
    for odt in (F32, BF16):
        out = torch.full((rows, cols), float("nan"), dtype=odt, device=dev)
        api.muon_checkpoint_unpack(ck, out)
        assert torch.equal(R.f64(out), want)


def test_checkpoint_borders(dev):
    """Magnitudes next to a power-of-two border, ties, the smallest and the
    largest values, blocks of zeros, infinities and NaN."""
    big = torch.finfo(F32).max
    rows = []
    for m in (448.0, 448.00003, 447.99997, 1.75, 1.7500001, 1.0, 2.0 ** -126, 2.0 ** -149, 3e-39, 1e-35, 0.0, 3.2e38):
        r = torch.zeros(128)
        r[0], r[1], r[2], r[3] = m, -m / 2, m / 3, m / 448 * 1.0625
        r[4], r[5], r[6] = m / 448 * 2.0 ** -10, m / 448 * 3 * 2.0 ** -10, -0.0
        rows.append(r)
    x = torch.stack(rows).to(dev)
    wq, we = R.checkpoint_encode(x)
    ck = api.new_checkpoint(x.shape[0], 128, dev)
    api.muon_checkpoint_pack(x, ck)
    assert torch.equal(ck.exponents.cpu(), we) and torch.equal(ck.codes.cpu(), wq)
    out = torch.empty_like(x)
    api.muon_checkpoint_unpack(ck, out)
    assert torch.equal(R.f64(out), R.checkpoint_values(wq, we, 128))
    y = torch.ones(4, 300, device=dev)
    y[0, 5], y[1, 130], y[2, 299], y[3, 0] = float("inf"), float("nan"), float("-inf"), big
    ck = api.new_checkpoint(4, 300, dev)
    api.muon_checkpoint_pack(y, ck)
    out = torch.empty_like(y)
    api.muon_checkpoint_unpack(ck, out)
    nan = torch.isnan(out).cpu()
    assert nan[0, :128].all() and nan[1, 128:256].all() and nan[2, 256:].all() and int(nan.sum()) == 128 + 128 + 44
    assert bool((out[0, 128:] == 1).all()) and bool(torch.isinf(out[3, 0])) and bool((out[3, 1:128] == 0).all())


def test_checkpoint_strided_and_empty(dev):
    x = activations(9, 200, BF16, 41, dev)
    base = api.new_checkpoint(9, 200, dev)
    api.muon_checkpoint_pack(x, base)
    for extra in (8, 3):
        ck = api.new_checkpoint(9, 200, dev)
        api.muon_checkpoint_pack(strided(x, extra)[1], ck)
        assert torch.equal(ck.codes, base.codes) and torch.equal(ck.exponents, base.exponents)
        buf, view = strided(torch.zeros_like(x), extra)
        api.muon_checkpoint_unpack(ck, view)
        assert torch.equal(R.f64(view), R.checkpoint_values(base.codes, base.exponents, 200))
        assert bool((buf[:, 200:] == 1e30).all())
    none = api.new_checkpoint(0, 200, dev)
    api.muon_checkpoint_pack(x[:0], none)
    api.muon_checkpoint_unpack(none, x[:0])


# ----------------------------------------------------------- weight gradient
WG_SHAPES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (17, 64, 128), (64, 128, 128), (65, 130, 129), (129, 256, 257),
             (200, 264, 384), (777, 520, 300), (1000, 33, 1000), (513, 768, 768), (2048, 256, 256), (300, 1001, 130)]


def wg_checkpoint(rows, k, seed, dev, kind):
    if kind == "whole":
        x = whole((rows, k), -8, 8, F32, seed, dev)      # one exact power of two per block
    else:
        x = activations(rows, k, F32, seed, dev) if kind == "wide" else rand((rows, k), 1.0, F32, seed, dev)
    ck = api.new_checkpoint(rows, k, dev)
    api.muon_checkpoint_pack(x, ck)
    return ck, R.checkpoint_values(ck.codes, ck.exponents, k)


@pytest.mark.parametrize("ddt", [BF16, F32])
@pytest.mark.parametrize("rows,n,k", WG_SHAPES + [(4001, 250, 500), (130, 4096, 2560), (200, 5001, 2500), (70, 9472, 1024),
                                                  (321, 8200, 3000)])
def test_weight_grad_of_whole_numbers_is_exact(dev, ddt, rows, n, k):
    ck, values = wg_checkpoint(rows, k, 50, dev, "whole")
    dy = whole((rows, n), -4, 4, ddt, 51, dev)
    want, _ = R.weight_grad(dy, values)
    w = ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, ddt), dev)
    grad = torch.full((n, k), float("nan"), device=dev)
    api.muon_checkpoint_weight_grad(dy, ck, grad, w)
    assert torch.equal(R.f64(grad), want)
    api.muon_checkpoint_weight_grad(dy, ck, grad, w, accumulate=True)
    assert torch.equal(R.f64(grad), 2 * want)
    assert api.muon_query_status(w) == N.MUON_OK


@pytest.mark.parametrize("ddt,gdt", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("rows,n,k", WG_SHAPES)
def test_weight_grad(dev, ddt, gdt, rows, n, k):
    for kind in ("plain", "wide"):
        ck, values = wg_checkpoint(rows, k, 52, dev, kind)
        dy = rand((rows, n), 1.0, ddt, 53, dev)
        want, mag = R.weight_grad(dy, values)
        w = ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, ddt), dev)
        old = rand((n, k), 1.0, gdt, 54, dev)
        for acc in (False, True):
            grad = old.clone()
            api.muon_checkpoint_weight_grad(dy, ck, grad, w, accumulate=acc)
            total = want + (R.f64(old) if acc else 0)
            # an addition may drop the bits below a step: 2 u per term
            near(grad, total, (2 * rows + 8) * U * (mag + (R.f64(old).abs() if acc else 0))
                 + R.HALF[gdt] * total.abs() * 1.01 + R.TINY[gdt])


def test_weight_grad_strided_dy_and_empty(dev):
    rows, n, k = 150, 136, 260
    ck, values = wg_checkpoint(rows, k, 55, dev, "whole")
    dy = whole((rows, n), -4, 4, BF16, 56, dev)
    want, _ = R.weight_grad(dy, values)
    w = ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, BF16, dy_aligned=False), dev)
    for extra in (8, 1):
        grad = torch.empty(n, k, device=dev)
        api.muon_checkpoint_weight_grad(strided(dy, extra)[1], ck, grad, w)
        assert torch.equal(R.f64(grad), want)
    none = api.new_checkpoint(0, k, dev)
    grad = torch.ones(n, k, device=dev)
    api.muon_checkpoint_weight_grad(dy[:0], none, grad, w, accumulate=True)
    assert bool((grad == 1).all())
    api.muon_checkpoint_weight_grad(dy[:0], none, grad, w)
    assert bool((grad == 0).all())


def test_weight_grad_nan_reaches_only_its_block(dev):
    rows, n, k = 40, 32, 300
    x = torch.ones(rows, k, device=dev)
    x[7, 130] = float("inf")
    ck = api.new_checkpoint(rows, k, dev)
    api.muon_checkpoint_pack(x, ck)
    dy = torch.ones(rows, n, dtype=BF16, device=dev)
    grad = torch.empty(n, k, device=dev)
    api.muon_checkpoint_weight_grad(dy, ck, grad, ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, k, BF16), dev))
    nan = torch.isnan(grad)
    assert bool(nan[:, 128:256].all()) and not bool(nan[:, :128].any()) and not bool(nan[:, 256:].any())
    assert bool((grad[:, :128] == rows).all())
