"""MuonAdamW.step on gradients given by their factors: refusals and failures."""
import pytest
import torch

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
