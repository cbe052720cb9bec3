"""MuonAdamW.step on gradients given by their factors: refusals and failures."""
import pytest
import torch

from muon_polar_orthogonalized_b200 import _native as N
from muon_polar_orthogonalized_b200 import api
from muon_polar_orthogonalized_b200.optimizer import MuonAdamW
from tests.test_gpu_operators import dev, token_ids  # noqa: F401  (dev: fixture)
from tests.test_gpu_operators_together import Block

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def made(dev):
    """A block after its forward pass and the norm's backward, and an optimizer over it."""
    b = Block(dev)
    b.forward()
    b.backward_norm()
    return b, MuonAdamW([b.weight], [dict(params=[b.table, b.gain, b.bias], lr=1e-2)], lr=0.02)


def state(b, opt):
    g = opt.adamw_groups[0]
    return [t.clone() for t in (b.weight, b.table, b.gain, b.bias, *opt.momentum, *g["exp_avg"], *g["exp_avg_sq"])]


def factors(b):
    return dict(muon_grads=[api.LinearGrad(b.dy, b.ckpt)],
                adamw_grads=[[api.EmbeddingGrad(b.dx, b.ids, b.scale), b.dgain, b.dbias]])


def test_a_refused_step_changes_nothing_and_may_be_made_again(dev):
    b, opt = made(dev)
    before = state(b, opt)
    other = api.new_checkpoint(b.tokens - 1, b.dim, dev)
    good = factors(b)
    for bad in (dict(good, adamw_grads=[[api.EmbeddingGrad(b.dx[:-1], b.ids, b.scale), b.dgain, b.dbias]]),
                dict(good, adamw_grads=[[api.EmbeddingGrad(b.dx, b.ids.float(), b.scale), b.dgain, b.dbias]]),
                dict(good, adamw_grads=[[api.EmbeddingGrad(b.dx, b.ids, float("nan")), b.dgain, b.dbias]]),
                dict(good, adamw_grads=[[good["adamw_grads"][0][0], b.dgain[:-1], b.dbias]]),
                dict(good, adamw_grads=[[good["adamw_grads"][0][0], b.dgain]]),
                dict(good, adamw_grads=[[good["adamw_grads"][0][0], b.dgain, good["muon_grads"][0]]]),
                dict(good, muon_grads=[api.LinearGrad(b.dy, other)]),
                dict(good, muon_grads=[api.LinearGrad(b.dy.half(), b.ckpt)]),
                dict(good, muon_grads=[[good["muon_grads"][0], api.LinearGrad(b.dy[:, :-1], b.ckpt)]])):
        with pytest.raises((ValueError, RuntimeError)):
            opt.step(**bad)
        assert opt.step_count == 0
        assert all(torch.equal(x, y) for x, y in zip(before, state(b, opt)))
    opt.step(**good)
    c, fresh = made(dev)
    fresh.step(**factors(c))
    assert opt.step_count == fresh.step_count == 1
    assert all(torch.equal(x, y) for x, y in zip(state(b, opt), state(c, fresh)))


class TimedOut(api.LinearGrad):
    """A factor in whose call a bounded wait runs out (the library's own test of
    its waits, on the call's workspace; the gradient is written as usual)."""

    def write(self, grad, workspace, accumulate=False, stream=None):
        super().write(grad, workspace, accumulate=accumulate, stream=stream)
        s = torch.cuda.current_stream(grad.device) if stream is None else stream
        assert N.lib().muon_selftest_wait_timeout(workspace.data_ptr(), 1000000, s.cuda_stream) == N.MUON_OK


@pytest.mark.parametrize("place", [0, 1, 2])
def test_a_timeout_in_a_factor_is_reported(dev, place):
    b, opt = made(dev)
    assert opt.query_status() == N.MUON_OK
    good = factors(b)
    opt.step(**good)
    assert opt.query_status() == N.MUON_OK
    parts = [api.LinearGrad(b.dy, b.ckpt) for _ in range(3)]
    parts[place] = TimedOut(b.dy, b.ckpt)
    opt.step(**dict(good, muon_grads=[parts]))
    opt.step(**good)
    assert opt.query_status() == N.MUON_ERR_TIMEOUT
    assert opt.query_status() == N.MUON_OK


def test_a_timeout_in_a_replayed_step_is_reported(dev):
    """On a stream of its own, captured, and the workspace outgrown since."""
    b, opt = made(dev)
    big = Block(dev, tokens=6000, seed=7)
    big.forward()
    big.backward_norm()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    opt.step(stream=side, **factors(b))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        opt.step(stream=side, **dict(factors(b), muon_grads=[TimedOut(b.dy, b.ckpt)]))
    assert opt.query_status(side) == N.MUON_OK
    opt.step(stream=side, **factors(big))
    assert opt.query_status(side) == N.MUON_OK
    with torch.cuda.stream(side):
        graph.replay()
    opt.step(stream=side, **factors(big))
    assert opt.query_status(side) == N.MUON_ERR_TIMEOUT
    assert opt.query_status(side) == N.MUON_OK
    del graph
