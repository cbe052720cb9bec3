"""Refusals of the gradient-making operators; no GPU work is launched.

The C ABI rejects a bad call with a status and a reason before any CUDA call;
the Python binding checks the tensors it marshals (CPU tensors stand in here:
every check but the device's comes after it, so those use a fake that says it
is on a GPU)."""
import ctypes

import pytest
import torch

from muon_polar_orthogonalized_b200 import _native as N
from muon_polar_orthogonalized_b200 import api
from muon_polar_orthogonalized_b200.build import build
from tests import operator_refs as R

P = ctypes.c_void_p
BAD, WSP, UNS = N.MUON_ERR_INVALID_ARG, N.MUON_ERR_WORKSPACE, N.MUON_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    build()
    return N.lib()


def call(fn, base, **over):
    """fn(*base) with named arguments replaced."""
    args = dict(base, **over)
    assert set(args) == set(base)
    return fn(*args.values())


EMB = dict(table=P(0x10000), tdt=0, vocab=100, dim=64, ids=P(0x20000), bits=64, n=10, scale=1.0, out=P(0x30000),
           odt=1, pitch=64, stream=None)
EMBG = dict(dout=P(0x10000), ddt=1, pitch=64, ids=P(0x20000), bits=64, n=10, vocab=100, dim=64, scale=1.0,
            grad=P(0x30000), gdt=0, acc=0, ws=P(0x40000), wsb=1 << 40, stream=None)
LN = dict(x=P(0x10000), xdt=1, xp=64, rows=10, cols=64, gain=P(0x20000), bias=P(0x21000), eps=1e-5, y=P(0x30000),
          ydt=1, yp=64, mean=P(0x40000), rstd=P(0x50000), stream=None)
LNB = dict(dy=P(0x10000), dyp=64, x=P(0x20000), dt=1, xp=64, rows=10, cols=64, gain=P(0x30000), mean=P(0x40000),
           rstd=P(0x50000), dx=P(0x60000), dxp=64, dgain=P(0x70000), dbias=P(0x80000), gdt=0, acc=0, ws=P(0x90000),
           wsb=1 << 40, stream=None)
PACK = dict(x=P(0x10000), xdt=1, xp=64, rows=10, cols=64, q=P(0x20000), qp=64, e=P(0x30000), stream=None)
UNPACK = dict(q=P(0x20000), qp=64, e=P(0x30000), rows=10, cols=64, out=P(0x10000), odt=1, op=64, stream=None)
WG = dict(dy=P(0x10000), ddt=1, dyp=32, rows=10, n=32, q=P(0x20000), qp=64, e=P(0x30000), k=64, grad=P(0x40000),
          gdt=0, acc=0, ws=P(0x50000), wsb=1 << 40, stream=None)


@pytest.mark.parametrize("name,base,over,expect", [
    ("muon_embedding_forward", EMB, dict(table=P(0)), BAD),
    ("muon_embedding_forward", EMB, dict(table=P(0x10004)), BAD),
    ("muon_embedding_forward", EMB, dict(tdt=2), BAD),
    ("muon_embedding_forward", EMB, dict(vocab=0), BAD),
    ("muon_embedding_forward", EMB, dict(vocab=1 << 31), BAD),
    ("muon_embedding_forward", EMB, dict(dim=0, pitch=0), BAD),
    ("muon_embedding_forward", EMB, dict(dim=1 << 17, pitch=1 << 17), BAD),
    ("muon_embedding_forward", EMB, dict(vocab=1 << 30, dim=65536, pitch=65536), BAD),
    ("muon_embedding_forward", EMB, dict(ids=P(0)), BAD),
    ("muon_embedding_forward", EMB, dict(ids=P(0x20004)), BAD),
    ("muon_embedding_forward", EMB, dict(bits=16), BAD),
    ("muon_embedding_forward", EMB, dict(n=-1), BAD),
    ("muon_embedding_forward", EMB, dict(scale=float("nan")), BAD),
    ("muon_embedding_forward", EMB, dict(out=P(0)), BAD),
    ("muon_embedding_forward", EMB, dict(out=P(0x30001)), BAD),
    ("muon_embedding_forward", EMB, dict(pitch=63), BAD),
    ("muon_embedding_forward", EMB, dict(pitch=1 << 40), BAD),
    ("muon_embedding_grad", EMBG, dict(grad=P(0)), BAD),
    ("muon_embedding_grad", EMBG, dict(grad=P(0x30008)), BAD),
    ("muon_embedding_grad", EMBG, dict(gdt=-1), BAD),
    ("muon_embedding_grad", EMBG, dict(dout=P(0)), BAD),
    ("muon_embedding_grad", EMBG, dict(ddt=9), BAD),
    ("muon_embedding_grad", EMBG, dict(scale=float("inf")), BAD),
    ("muon_embedding_grad", EMBG, dict(ws=P(0)), WSP),
    ("muon_embedding_grad", EMBG, dict(ws=P(0x40010)), WSP),
    ("muon_embedding_grad", EMBG, dict(wsb=256), WSP),
    ("muon_layer_norm_forward", LN, dict(cols=0, xp=0, yp=0), BAD),
    ("muon_layer_norm_forward", LN, dict(cols=16385, xp=16385, yp=16385), UNS),
    ("muon_layer_norm_forward", LN, dict(rows=-1), BAD),
    ("muon_layer_norm_forward", LN, dict(gain=P(0)), BAD),
    ("muon_layer_norm_forward", LN, dict(gain=P(0x20004)), BAD),
    ("muon_layer_norm_forward", LN, dict(bias=P(0x21008)), BAD),
    ("muon_layer_norm_forward", LN, dict(eps=-1.0), BAD),
    ("muon_layer_norm_forward", LN, dict(eps=float("nan")), BAD),
    ("muon_layer_norm_forward", LN, dict(mean=P(0)), BAD),
    ("muon_layer_norm_forward", LN, dict(x=P(0x10001)), BAD),
    ("muon_layer_norm_forward", LN, dict(yp=32), BAD),
    ("muon_layer_norm_backward", LNB, dict(dgain=P(0)), BAD),
    ("muon_layer_norm_backward", LNB, dict(dbias=P(0x80002)), BAD),
    ("muon_layer_norm_backward", LNB, dict(gdt=5), BAD),
    ("muon_layer_norm_backward", LNB, dict(dt=5), BAD),
    ("muon_layer_norm_backward", LNB, dict(dx=P(0)), BAD),
    ("muon_layer_norm_backward", LNB, dict(ws=P(0)), WSP),
    ("muon_layer_norm_backward", LNB, dict(wsb=300), WSP),
    ("muon_checkpoint_pack", PACK, dict(q=P(0)), BAD),
    ("muon_checkpoint_pack", PACK, dict(q=P(0x20008)), BAD),
    ("muon_checkpoint_pack", PACK, dict(qp=72), BAD),
    ("muon_checkpoint_pack", PACK, dict(qp=48), BAD),
    ("muon_checkpoint_pack", PACK, dict(e=P(0)), BAD),
    ("muon_checkpoint_pack", PACK, dict(x=P(0)), BAD),
    ("muon_checkpoint_pack", PACK, dict(cols=0), BAD),
    ("muon_checkpoint_unpack", UNPACK, dict(out=P(0)), BAD),
    ("muon_checkpoint_unpack", UNPACK, dict(odt=3), BAD),
    ("muon_checkpoint_unpack", UNPACK, dict(rows=(1 << 30) + 1), BAD),
    ("muon_checkpoint_weight_grad", WG, dict(n=0, dyp=0), BAD),
    ("muon_checkpoint_weight_grad", WG, dict(n=1 << 17, dyp=1 << 17), BAD),
    ("muon_checkpoint_weight_grad", WG, dict(dy=P(0x10001)), BAD),
    ("muon_checkpoint_weight_grad", WG, dict(grad=P(0x40004)), BAD),
    ("muon_checkpoint_weight_grad", WG, dict(gdt=2), BAD),
    ("muon_checkpoint_weight_grad", WG, dict(ws=P(0)), WSP),
    ("muon_checkpoint_weight_grad", WG, dict(wsb=255), WSP),
])
def test_entry_points_refuse(L, name, base, over, expect):
    assert call(getattr(L, name), base, **over) == expect
    assert N.last_error() != ""


def test_workspace_sizes_refuse_and_grow(L):
    assert api.muon_embedding_grad_workspace_size(0, 8, 8) == 0
    assert api.muon_embedding_grad_workspace_size(8, 0, 8) == 0
    assert api.muon_embedding_grad_workspace_size(8, 8, -1) == 0
    small, big = (api.muon_embedding_grad_workspace_size(50304, 768, n) for n in (64, 65536))
    # two sort buffers of ids and positions, offsets, the runs, and the pieces' sums
    assert 4 * 50304 < small < big and big >= 20 * 65536 + 65536 // 128 * 768 * 4
    assert api.muon_layer_norm_backward_workspace_size(8, 16385) == 0
    assert api.muon_layer_norm_backward_workspace_size(0, 64) > 0
    assert api.muon_checkpoint_weight_grad_workspace_size(8, 8, 8, torch.float16) == 0
    assert api.muon_checkpoint_weight_grad_workspace_size(8, 8, 8, torch.bfloat16) >= 256


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on a GPU (nothing is launched with it)."""

    def get_device(self):
        return getattr(self, "on", 0)


def fake(*shape, dtype=torch.float32, on=0):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnGpu)
    t.on = on
    return t


def ids(n, dtype=torch.int64):
    return fake(n, dtype=dtype)


@pytest.mark.parametrize("match,call", [
    ("not a CUDA", lambda: api.muon_embedding_forward(torch.zeros(4, 8), ids(3), fake(3, 8))),
    ("another device", lambda: api.muon_embedding_forward(fake(4, 8), ids(3), fake(3, 8, on=1))),
    ("table", lambda: api.muon_embedding_forward(fake(4, 2, 4), ids(3), fake(3, 8))),
    ("table", lambda: api.muon_embedding_forward(fake(4, 16)[:, :8], ids(3), fake(3, 8))),
    ("table must be fp32 or bf16", lambda: api.muon_embedding_forward(fake(4, 8, dtype=torch.float16), ids(3), fake(3, 8))),
    ("ids", lambda: api.muon_embedding_forward(fake(4, 8), ids(3, torch.int16), fake(3, 8))),
    ("ids", lambda: api.muon_embedding_forward(fake(4, 8), ids(6)[::2], fake(3, 8))),
    ("out", lambda: api.muon_embedding_forward(fake(4, 8), ids(3), fake(2, 8))),
    ("out", lambda: api.muon_embedding_forward(fake(4, 8), ids(3), fake(3, 9))),
    ("not adjacent", lambda: api.muon_embedding_forward(fake(4, 8), ids(3), fake(3, 16)[:, ::2])),
    ("constant pitch", lambda: api.muon_embedding_forward(fake(4, 8), ids(6), fake(2, 4, 8)[:, :3])),
    ("overlap", lambda: api.muon_embedding_forward(fake(4, 8), ids(3), fake(1, 8).expand(3, 8))),
    ("dout", lambda: api.muon_embedding_grad(fake(4, 8), ids(3), fake(5, 8), fake(9999))),
    ("grad", lambda: api.muon_embedding_grad(fake(3, 8), ids(3), fake(8, 5).t(), fake(9999))),
    ("workspace", lambda: api.muon_embedding_grad(fake(3, 8), ids(3), fake(5, 8), fake(99, 99)[:, :50])),
    ("gain", lambda: api.muon_layer_norm_forward(fake(3, 8), fake(9), None, fake(3, 8), fake(3), fake(3))),
    ("gain", lambda: api.muon_layer_norm_forward(fake(3, 8), fake(8, dtype=torch.bfloat16), None, fake(3, 8), fake(3), fake(3))),
    ("bias", lambda: api.muon_layer_norm_forward(fake(3, 8), fake(8), fake(7), fake(3, 8), fake(3), fake(3))),
    ("mean", lambda: api.muon_layer_norm_forward(fake(3, 8), fake(8), None, fake(3, 8), fake(4), fake(3))),
    ("y", lambda: api.muon_layer_norm_forward(fake(3, 8), fake(8), None, fake(4, 8), fake(3), fake(3))),
    ("one type", lambda: api.muon_layer_norm_backward(fake(3, 8), fake(3, 8, dtype=torch.bfloat16), fake(8), fake(3),
                                                      fake(3), fake(3, 8), fake(8), None, fake(9999))),
    ("dbias", lambda: api.muon_layer_norm_backward(fake(3, 8), fake(3, 8), fake(8), fake(3), fake(3), fake(3, 8),
                                                   fake(8), fake(8, dtype=torch.bfloat16), fake(9999))),
    ("codes", lambda: api.Checkpoint(torch.zeros(3, 24, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.uint8), 20)),
    ("codes", lambda: api.Checkpoint(torch.zeros(3, 16, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.uint8), 17)),
    ("exponents", lambda: api.Checkpoint(torch.zeros(3, 144, dtype=torch.uint8), torch.zeros(3, 1, dtype=torch.uint8), 129)),
    ("not a CUDA", lambda: api.muon_checkpoint_pack(torch.zeros(3, 20), api.new_checkpoint(3, 20, "cpu"))),
])
def test_binding_refuses(match, call):
    with pytest.raises(ValueError, match=match):
        call()


def test_references_agree_with_each_other():
    """The exhaustive encoder against the code table: every representable
    value maps to itself, and every block's largest code is above 224."""
    v = R.e4m3_values()
    fin = v[~torch.isnan(v)]
    codes, exps = R.checkpoint_encode(fin.reshape(2, 127))
    assert torch.equal(R.checkpoint_values(codes, exps, 127), fin.reshape(2, 127))
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 300, generator=g)
    codes, exps = R.checkpoint_encode(x)
    err = (R.checkpoint_values(codes, exps, 300) - x.double()).abs()
    step = torch.pow(2.0, exps.double() - 127).repeat_interleave(128, 1)[:, :300]
    assert bool((err <= torch.maximum(x.double().abs() * 2.0 ** -4, step * 2.0 ** -10)).all())


def test_formed_gradients_keep_the_workspace_of_a_captured_step(monkeypatch):
    """A captured step writes its workspace at every replay: a later, larger step
    takes another and must not free it.  Steps that were not captured keep none."""
    import types
    from muon_polar_orthogonalized_b200.optimizer import MuonAdamW

    class Factor(api.LinearGrad):
        def __init__(self, need):
            self.need = need

        def workspace_size(self, grad):
            return self.need

        def write(self, grad, workspace, accumulate=False, stream=None):
            assert workspace.numel() >= self.need
            grad.fill_(1.0)

    opt = types.SimpleNamespace(_factor_workspace=None, _captured_workspaces=[])
    param = torch.zeros(4, 4)
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    form = lambda need: MuonAdamW._formed(opt, param, Factor(need), None)
    form(300)
    assert opt._captured_workspaces == []
    capturing[0] = True
    form(300)
    form(200)
    kept = opt._factor_workspace
    assert len(opt._captured_workspaces) == 1 and opt._captured_workspaces[0] is kept
    capturing[0] = False
    form(5000)
    assert opt._factor_workspace is not kept and opt._captured_workspaces[0] is kept
    assert len(opt._captured_workspaces) == 1
