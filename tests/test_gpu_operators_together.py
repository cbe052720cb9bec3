"""The gradient-making operators as a training step uses them: together, with
the optimizer, on other streams, in captured graphs, on large buffers, and
inside guard bands."""
import pytest
import torch

from muon_polar_orthogonalized_b200 import _native as N
from muon_polar_orthogonalized_b200 import api
from muon_polar_orthogonalized_b200.optimizer import MuonAdamW
from tests import operator_refs as R
from tests.test_gpu_operators import dev, near, rand, token_ids, whole, ws  # noqa: F401  (dev: fixture)

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
U = R.U32


class Block:
    """tokens -> embedding -> layer norm -> hidden matrix W, and back.  The
    matrix product itself is torch's; everything else is the library's."""

    def __init__(self, dev, vocab=211, dim=264, hidden=136, tokens=150, seed=1):
        self.vocab, self.dim, self.hidden, self.tokens = vocab, dim, hidden, tokens
        self.scale = 16.25
        self.table = rand((vocab, dim), 0.02, F32, seed, dev)
        self.gain = rand((dim,), 0.1, F32, seed + 1, dev, 1.0)
        self.bias = rand((dim,), 0.1, F32, seed + 2, dev)
        self.weight = rand((hidden, dim), 0.05, F32, seed + 3, dev)
        self.ids = token_ids(tokens, vocab, "zipf", seed + 4).to(dev)
        self.dy = rand((tokens, hidden), 1.0, BF16, seed + 5, dev)   # the loss's gradient
        e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device=dev)
        self.x, self.y = e(tokens, dim, dtype=BF16), e(tokens, dim, dtype=BF16)
        self.mean, self.rstd = e(tokens), e(tokens)
        self.ckpt = api.new_checkpoint(tokens, dim, dev)
        self.dx, self.dnorm = e(tokens, dim, dtype=BF16), e(tokens, dim, dtype=BF16)
        self.dgain, self.dbias, self.dweight, self.dtable = e(dim), e(dim), e(hidden, dim), e(vocab, dim)
        self.ws = ws(max(api.muon_embedding_grad_workspace_size(vocab, dim, tokens),
                         api.muon_layer_norm_backward_workspace_size(tokens, dim),
                         api.muon_checkpoint_weight_grad_workspace_size(tokens, hidden, dim, BF16)), dev)

    def forward(self, stream=None):
        api.muon_embedding_forward(self.table, self.ids, self.x, scale=self.scale, stream=stream)
        api.muon_layer_norm_forward(self.x, self.gain, self.bias, self.y, self.mean, self.rstd, stream=stream)
        api.muon_checkpoint_pack(self.y, self.ckpt, stream=stream)

    def backward_norm(self, stream=None):
        torch.matmul(self.dy, self.weight.to(BF16), out=self.dnorm)
        api.muon_layer_norm_backward(self.dnorm, self.x, self.gain, self.mean, self.rstd, self.dx, self.dgain,
                                     self.dbias, self.ws, stream=stream)

    def backward(self, accumulate=False):
        self.backward_norm()
        api.muon_checkpoint_weight_grad(self.dy, self.ckpt, self.dweight, self.ws, accumulate=accumulate)
        api.muon_embedding_grad(self.dx, self.ids, self.dtable, self.ws, scale=self.scale, accumulate=accumulate)

    def outputs(self):
        return [t.clone() for t in (self.x, self.y, self.mean, self.rstd, self.ckpt.codes, self.ckpt.exponents, self.dx,
                                    self.dgain, self.dbias, self.dweight, self.dtable)]

    def check(self):
        """Each stage against its 64-bit statement on the stage's own inputs."""
        near(self.x, R.embedding(self.table, self.ids, self.scale),
             R.embedding(self.table, self.ids, self.scale).abs() * (U + 2.0 ** -8 * 1.01) + R.TINY[BF16])
        values = R.checkpoint_values(self.ckpt.codes, self.ckpt.exponents, self.dim)
        q, e = R.checkpoint_encode(self.y)
        assert torch.equal(q, self.ckpt.codes.cpu()) and torch.equal(e, self.ckpt.exponents.cpu())
        want, mag = R.weight_grad(self.dy, values)
        near(self.dweight, want, (2 * self.tokens + 8) * U * mag + U * want.abs())
        _, dg, db, _, mg, mb = R.layer_norm_grad(self.dnorm, self.x, self.gain, self.mean, self.rstd)
        near(self.dgain, dg, (self.tokens + 4) * U * mg + U * dg.abs())
        near(self.dbias, db, (self.tokens + 4) * U * mb + U * db.abs())
        want, mag, cnt = R.embedding_grad(self.dx, self.ids, self.vocab, self.scale)
        near(self.dtable, want, (cnt[:, None] + 2) * U * mag)


def test_a_training_step_together(dev):
    b = Block(dev)
    b.forward()
    b.backward()
    b.check()
    # rows of padding: zeros in, a gradient for nothing
    pad = (b.ids < 0) | (b.ids >= b.vocab)
    assert int(pad.sum()) > 5 and bool((b.x[pad] == 0).all())
    assert api.muon_query_status(b.ws) == N.MUON_OK


def test_optimizer_forms_gradients_from_their_factors(dev):
    """MuonAdamW.step on factors does what it does on the gradients written out,
    bit for bit; two micro-batches add up."""
    outs = []
    for by_factors in (False, True):
        b, b2 = Block(dev, seed=1), Block(dev, seed=1)
        b2.ids, b2.dy = token_ids(b2.tokens, b2.vocab, "random", 99).to(dev), rand((b2.tokens, b2.hidden), 1.0, BF16, 98, dev)
        opt = MuonAdamW([b.weight], [dict(params=[b.table, b.gain, b.bias], lr=1e-2)], lr=0.02)
        for blk in (b, b2):
            blk.forward()
            blk.backward_norm()
        b.dgain += b2.dgain
        b.dbias += b2.dbias
        if by_factors:
            opt.step(muon_grads=[[api.LinearGrad(b.dy, b.ckpt), api.LinearGrad(b2.dy, b2.ckpt)]],
                     adamw_grads=[[[api.EmbeddingGrad(b.dx, b.ids, b.scale), api.EmbeddingGrad(b2.dx, b2.ids, b2.scale)],
                                   b.dgain, b.dbias]])
        else:
            for k, blk in enumerate((b, b2)):
                api.muon_checkpoint_weight_grad(blk.dy, blk.ckpt, b.dweight, b.ws, accumulate=k > 0)
                api.muon_embedding_grad(blk.dx, blk.ids, b.dtable, b.ws, scale=b.scale, accumulate=k > 0)
            opt.step(muon_grads=[b.dweight], adamw_grads=[[b.dtable, b.dgain, b.dbias]])
        outs.append([b.weight.clone(), b.table.clone(), b.gain.clone(), b.bias.clone()])
        before = Block(dev, seed=1)
        assert not torch.equal(before.weight, b.weight) and not torch.equal(before.table, b.table)
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_captured_step_on_factors_outlives_a_larger_one(dev):
    """A captured step on factors is replayed after an eager step that needed a
    larger workspace: it forms the same gradients, in memory that nothing else
    was given meanwhile."""
    b, big = Block(dev, seed=1), Block(dev, tokens=6000, seed=7)
    for blk in (b, big):
        blk.forward()
        blk.backward_norm()
    opt = MuonAdamW([b.weight], [dict(params=[b.table], lr=1e-2)], lr=0.02)

    def step(blk, stream=None):
        opt.step(stream=stream, muon_grads=[api.LinearGrad(blk.dy, blk.ckpt)],
                 adamw_grads=[[api.EmbeddingGrad(blk.dx, blk.ids, blk.scale)]])

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step(b, side)
    torch.cuda.synchronize()
    want = [b.weight.grad.clone(), b.table.grad.clone()]
    kept = opt._factor_workspace
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(b, side)
    step(big)
    assert opt._factor_workspace is not kept
    size = kept.numel()
    del kept
    filler = [torch.full((size,), 0xA5, dtype=torch.uint8, device=dev) for _ in range(16)]
    b.weight.grad.zero_()
    b.table.grad.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.weight.grad, want[0]) and torch.equal(b.table.grad, want[1])
    assert all(bool((f == 0xA5).all()) for f in filler)
    del graph


def test_optimizer_refuses_other_factors(dev):
    b = Block(dev)
    opt = MuonAdamW([b.weight], [dict(params=[b.table])])
    with pytest.raises(ValueError, match="gradient is a tensor"):
        opt.step(muon_grads=["dweight"])
    with pytest.raises(ValueError, match="one gradient per parameter"):
        opt.step(muon_grads=[b.dweight], adamw_grads=[[]])


def test_on_another_stream(dev):
    b = Block(dev)
    b.forward()
    b.backward()
    want = b.outputs()
    s = torch.cuda.Stream(dev)
    c = Block(dev)
    s.wait_stream(torch.cuda.current_stream(dev))
    c.forward(stream=s)                      # the stream given
    with torch.cuda.stream(s):               # the stream current
        c.backward()
    torch.cuda.current_stream(dev).wait_stream(s)
    for x, y in zip(want, c.outputs()):
        assert torch.equal(x, y)


def test_two_streams_at_once(dev):
    """Calls on different streams with different workspaces."""
    blocks = [Block(dev, vocab=4000, dim=512, hidden=512, tokens=3000, seed=s) for s in (1, 2)]
    want = []
    for b in blocks:
        b.forward()
        b.backward()
        want.append(b.outputs())
    streams = [torch.cuda.Stream(dev) for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s in zip(blocks, streams):
            with torch.cuda.stream(s):
                b.forward()
                b.backward()
    torch.cuda.synchronize()
    for b, w in zip(blocks, want):
        for x, y in zip(w, b.outputs()):
            assert torch.equal(x, y)


def test_captured_and_replayed_with_new_inputs(dev):
    """One captured step replayed on new inputs; a second captured step shares
    the first's workspace and is replayed after it."""
    b = Block(dev)
    c = Block(dev, seed=20)
    c.ws = b.ws
    for blk in (b, c):
        blk.forward()
        blk.backward()
    torch.cuda.synchronize()
    graphs = []
    for blk in (b, c):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            blk.forward()
            blk.backward()
        graphs.append(g)
    for seed in (50, 60):
        for blk in (b, c):
            blk.ids.copy_(token_ids(blk.tokens, blk.vocab, "random", seed).to(dev))
            blk.dy.copy_(rand((blk.tokens, blk.hidden), 1.0, BF16, seed + 1, dev))
        b.ws.fill_(0xFF)
        for _ in range(2):
            for g in graphs:
                g.replay()
        b.check()
        c.check()
    del graphs


def banded(t):
    """(buffer, view): a copy of t inside canaries."""
    n = t.numel() * t.element_size()
    buf = torch.full((8192 + n,), 0xA5, dtype=torch.uint8, device=t.device)
    view = buf[4096:4096 + n].view(t.dtype).view(t.shape)
    view.copy_(t)
    return buf, view


@pytest.mark.parametrize("dim,hidden,tokens,vocab", [(264, 136, 150, 211), (777, 333, 131, 65), (1032, 2049, 70, 300),
                                                     (64, 4100, 2600, 5000), (4097, 16, 33, 40), (1, 1, 1, 1)])
def test_nothing_is_written_outside_outputs_and_workspace(dev, dim, hidden, tokens, vocab):
    b = Block(dev, vocab=vocab, dim=dim, hidden=hidden, tokens=tokens)
    bands = []
    for name in ("x", "y", "mean", "rstd", "dx", "dgain", "dbias", "dweight", "dtable", "table", "dy"):
        buf, view = banded(getattr(b, name))
        bands.append((name, buf))
        setattr(b, name, view)
    for name in ("codes", "exponents"):
        buf, view = banded(getattr(b.ckpt, name))
        bands.append((name, buf))
        setattr(b.ckpt, name, view)
    b.forward()
    b.backward_norm()
    for size, call in (
            (api.muon_checkpoint_weight_grad_workspace_size(tokens, hidden, dim, BF16),
             lambda w: api.muon_checkpoint_weight_grad(b.dy, b.ckpt, b.dweight, w)),
            (api.muon_embedding_grad_workspace_size(vocab, dim, tokens),
             lambda w: api.muon_embedding_grad(b.dx, b.ids, b.dtable, w, scale=b.scale)),
            (api.muon_layer_norm_backward_workspace_size(tokens, dim),
             lambda w: api.muon_layer_norm_backward(b.dnorm, b.x, b.gain, b.mean, b.rstd, b.dx, b.dgain, b.dbias, w))):
        buf = torch.full((8192 + size,), 0xA5, dtype=torch.uint8, device=dev)
        call(buf[4096:4096 + size])
        bands.append(("workspace", buf))
    torch.cuda.synchronize()
    for name, buf in bands:
        assert bool((buf[:4096] == 0xA5).all()) and bool((buf[-4096:] == 0xA5).all()), name


def test_offsets_beyond_32_bits(dev):
    """Tables, activations and gradients of more than 2^31 elements: the last
    rows come out as the first ones do."""
    vocab, dim = 525000, 4096
    table = torch.empty(vocab, dim, dtype=BF16, device=dev).zero_()
    ids = torch.tensor([vocab - 1, 0, vocab - 1, vocab - 2], device=dev)
    table[vocab - 1], table[0] = 2.0, 1.0
    out = torch.empty(4, dim, dtype=BF16, device=dev)
    api.muon_embedding_forward(table, ids, out, scale=0.5)
    assert out[:, 0].tolist() == [1.0, 0.5, 1.0, 0.0] and bool((out == out[:, :1]).all())
    for n in (4, 5000):   # both sorts
        many = ids.repeat(n // 4)
        dout = torch.ones(n, dim, dtype=BF16, device=dev)
        table.fill_(7.0)
        api.muon_embedding_grad(dout, many, table, ws(api.muon_embedding_grad_workspace_size(vocab, dim, n), dev), scale=0.125)
        got = table[[0, 1, vocab - 3, vocab - 2, vocab - 1], :].float().cpu()
        want = torch.tensor([n // 4 / 8, 0, 0, n // 4 / 8, n // 2 / 8]).to(BF16).float()
        assert torch.equal(got, want[:, None].expand_as(got))
        assert float(table[:, 5].float().sum()) == float(want.sum())
    del table
    rows, cols = 140000, 16384
    x = torch.empty(rows, cols, dtype=BF16, device=dev).zero_()
    x[-1, ::2], x[0, ::2] = 2.0, 2.0
    gain, mean, rstd = torch.ones(cols, device=dev), torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    api.muon_layer_norm_forward(x, gain, None, x, mean, rstd, eps=0.0)
    assert torch.equal(x[-1], x[0]) and x[-1, :2].tolist() == [1.0, -1.0] and mean[-1].item() == 1.0
    ck = api.new_checkpoint(rows, cols, dev)
    x[1:-1] = 0.5
    api.muon_checkpoint_pack(x, ck)
    x.zero_()
    api.muon_checkpoint_unpack(ck, x)
    assert x[-1, :2].tolist() == [1.0, -1.0] and bool((x[rows // 2] == 0.5).all())
    del x
    n = 16
    dy = torch.zeros(rows, n, dtype=BF16, device=dev)
    dy[-1], dy[0] = 1.0, 2.0
    grad = torch.empty(n, cols, device=dev)
    api.muon_checkpoint_weight_grad(dy, ck, grad, ws(api.muon_checkpoint_weight_grad_workspace_size(rows, n, cols, BF16), dev))
    assert bool((grad[:, ::2] == 3.0).all()) and bool((grad[:, 1::2] == -3.0).all())


def test_status_words_are_cleared(dev):
    """Every call with a workspace leaves a status that reads as success."""
    b = Block(dev)
    b.forward()
    b.backward_norm()
    none = torch.empty(0, dtype=torch.int64, device=dev)
    empty = api.new_checkpoint(0, b.dim, dev)
    for call in (lambda w: api.muon_checkpoint_weight_grad(b.dy, b.ckpt, b.dweight, w),
                 lambda w: api.muon_checkpoint_weight_grad(b.dy[:0], empty, b.dweight, w, accumulate=True),
                 lambda w: api.muon_embedding_grad(b.dx, b.ids, b.dtable, w),
                 lambda w: api.muon_embedding_grad(b.dx[:0], none, b.dtable, w, accumulate=True),
                 lambda w: api.muon_embedding_grad(b.dx[:0], none, b.dtable, w),
                 lambda w: api.muon_layer_norm_backward(b.dnorm, b.x, b.gain, b.mean, b.rstd, b.dx, b.dgain, b.dbias, w)):
        b.ws.fill_(0xFF)
        call(b.ws)
        assert api.muon_query_status(b.ws) == N.MUON_OK


def test_profiler_counts_the_operators(dev):
    b = Block(dev)
    api.muon_profiler_reset()
    api.muon_profiler_enable(True)
    try:
        b.forward()
        b.backward()
        kinds = api.muon_profiler_read()
    finally:
        api.muon_profiler_enable(False)
        api.muon_profiler_reset()
    for k in ("embedding", "embedding_sort", "embedding_grad", "layer_norm", "layer_norm_grad", "checkpoint_pack",
              "weight_grad"):
        assert kinds[k][1] >= 1, k
