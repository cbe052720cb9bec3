"""The operators of a training step around the optimizer, as measured cases.

Three parameter kinds reach the MuonAdamW step: embedding tables and norm
gains (AdamW) and hidden matrices (Muon).  The cases here run what feeds the
step with their gradients:

  embedding lookup with scaling, and the table's gradient by sorted tokens;
  layer norm's forward and backward pass, with the gain's and bias's gradient;
  activation checkpoints in 8 bits (a block of 128 features shares a power of
  two), stored and restored, and a hidden matrix's gradient from one.

`run` computes a case in plain torch operations in 32 bits, or, with `own`
set, through the library's entry points.  `exact` states the same results in
64 bits from the definitions.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
BLOCK = 128        # features that share one checkpoint exponent
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one short batch looked up in a 1664-wide table; odd token count
        dict(name="embed_short", op="embed", vocab=65536, dim=1664, tokens=777, table="f32", out="bf16"),
        # a training batch on the 128256 x 4096 table
        dict(name="embed_long", op="embed", vocab=128256, dim=4096, tokens=32768, table="f32", out="bf16"),
        # the 768-wide table's gradient from one sequence: latency and the untouched rows' zeros
        dict(name="embed_grad_short", op="embed_grad", vocab=50304, dim=768, tokens=1024, dout="f32", grad="f32"),
        # a training batch's gradient of a 65536 x 1664 table: hot tokens, many single ones
        dict(name="embed_grad_long", op="embed_grad", vocab=65536, dim=1664, tokens=65536, dout="bf16", grad="f32"),
        # norm of a few hundred rows in 32 bits, without bias
        dict(name="norm_short", op="norm", rows=333, cols=768, x="f32", y="f32", bias=False),
        # norm of a training batch, 4096 wide
        dict(name="norm_long", op="norm", rows=32768, cols=4096, x="bf16", y="bf16", bias=True),
        # its backward pass: a small batch in 32 bits, and the training batch
        dict(name="norm_grad_short", op="norm_grad", rows=1000, cols=1664, x="f32", grad="f32", bias=True),
        dict(name="norm_grad_long", op="norm_grad", rows=32768, cols=4096, x="bf16", grad="f32", bias=False),
        # checkpoint and restore: a ragged small one in 32 bits, and the MLP's 14336-wide activations
        dict(name="checkpoint_short", op="checkpoint", rows=257, cols=1000, x="f32"),
        dict(name="checkpoint_long", op="checkpoint", rows=16384, cols=14336, x="bf16"),
        # a hidden matrix's gradient from the checkpoint: one short odd batch, and an MLP matrix of a training batch
        dict(name="weight_grad_short", op="weight_grad", rows=777, n=1664, k=768, dy="bf16", grad="f32"),
        dict(name="weight_grad_long", op="weight_grad", rows=16384, n=14336, k=4096, dy="bf16", grad="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 64, sometimes of 8, sometimes any number."""
    w = _log_int(rng, lo, hi)
    m = rng.choice([64, 64, 8, 1])
    return max(lo, w // m * m)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "checkpoint", "weight_grad"])
    t = lambda: rng.choice(["f32", "bf16"])
    if op in ("embed", "embed_grad"):
        c = dict(op=op, vocab=_log_int(rng, 200, 131072), dim=_width(rng, 16, 4096), tokens=_log_int(rng, 1, 65536))
        while c["vocab"] * c["dim"] > 65536 * 1664:
            c["vocab"] = c["vocab"] // 2 + 1
        while c["tokens"] * c["dim"] > 65536 * 1664:
            c["tokens"] = c["tokens"] // 2 + 1
        c.update(dict(table=t(), out=t()) if op == "embed" else dict(dout=t(), grad=t()))
        return c
    if op in ("norm", "norm_grad"):
        c = dict(op=op, rows=_log_int(rng, 1, 32768), cols=_width(rng, 32, 16384))
        while c["rows"] * c["cols"] > 32768 * 2048:
            c["rows"] = c["rows"] // 2 + 1
        c.update(dict(x=t(), y=t()) if op == "norm" else dict(x=t(), grad=t()))
        c["bias"] = rng.random() < 0.5
        return c
    if op == "checkpoint":
        c = dict(op=op, rows=_log_int(rng, 1, 32768), cols=_width(rng, 16, 16384), x=t())
        while c["rows"] * c["cols"] > 16384 * 7168:
            c["rows"] = c["rows"] // 2 + 1
        return c
    c = dict(op=op, rows=_log_int(rng, 1, 16384), n=_width(rng, 64, 14336), k=_width(rng, 64, 14336),
             dy=rng.choice(["bf16", "bf16", "f32"]), grad=t())
    while c["n"] * c["k"] > 4096 * 14336:
        c["n"], c["k"] = c["n"] // 2 + 1, c["k"] // 2 + 1
    if c["dy"] == "f32":
        c["rows"] = min(c["rows"], 4096)
    return c


# ------------------------------------------------------------------ inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _zipf_cdf(vocab, device):
    """Token frequencies falling with rank, as a tokeniser's ids do."""
    w = 1.0 / (torch.arange(vocab, dtype=torch.float64, device=device) + 2.7)
    return torch.cumsum(w / w.sum(), 0)


def _tokens(g, vocab, n):
    """n token ids; the last sixteenth of a longer batch is padding (-1)."""
    u = torch.rand(n, dtype=torch.float64, device="cuda", generator=g)
    ids = torch.searchsorted(_zipf_cdf(vocab, "cuda"), u).clamp_(max=vocab - 1)
    if n >= 64:
        ids[n - n // 16:] = -1
    return ids


def _activations(g, rows, cols, dtype):
    """Activations of a residual stream: unit scale, a few loud features, an offset."""
    x = torch.empty(rows, cols, dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=g)
    loud = torch.randint(0, cols, (max(1, cols // 256),), device="cuda", generator=g)
    x[:, loud] *= 20.0
    return x.add_(0.25).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case, op=op)
    if op == "embed":
        s["table"] = _normal(g, (case["vocab"], case["dim"]), 0.02, DT[case["table"]])
        s["ids"] = _tokens(g, case["vocab"], case["tokens"])
        s["scale"] = math.sqrt(case["dim"])
        s["result"] = torch.empty(case["tokens"], case["dim"], dtype=DT[case["out"]], device="cuda")
    elif op == "embed_grad":
        s["dout"] = _normal(g, (case["tokens"], case["dim"]), 1e-3, DT[case["dout"]])
        s["ids"] = _tokens(g, case["vocab"], case["tokens"])
        s["scale"] = math.sqrt(case["dim"])
        s["result"] = torch.empty(case["vocab"], case["dim"], dtype=DT[case["grad"]], device="cuda")
    elif op in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(g, rows, cols, DT[case["x"]])
        s["gain"] = _normal(g, (cols,), 0.1, torch.float32) + 1.0
        s["bias"] = _normal(g, (cols,), 0.1, torch.float32) if case["bias"] else None
        if op == "norm":
            s["y"] = torch.empty(rows, cols, dtype=DT[case["y"]], device="cuda")
            s["mean"] = torch.empty(rows, device="cuda")
            s["rstd"] = torch.empty(rows, device="cuda")
        else:
            s["dy"] = _normal(g, (rows, cols), 1e-3, DT[case["x"]])
            xd = s["x"].double()
            s["mean"] = xd.mean(1).float()
            s["rstd"] = torch.rsqrt(xd.var(1, unbiased=False) + EPS).float()
            del xd
            s["dx"] = torch.empty_like(s["x"])
            s["dgain"] = torch.empty(cols, dtype=DT[case["grad"]], device="cuda")
            s["dbias"] = torch.empty(cols, dtype=DT[case["grad"]], device="cuda") if case["bias"] else None
    elif op == "checkpoint":
        s["x"] = _activations(g, case["rows"], case["cols"], DT[case["x"]])
        s["result"] = torch.empty_like(s["x"])
    else:
        rows, n, k = case["rows"], case["n"], case["k"]
        s["q"], s["exps"] = _encode(_activations(g, rows, k, torch.bfloat16))
        s["dy"] = _normal(g, (rows, n), 1e-3, DT[case["dy"]])
        s["result"] = torch.empty(n, k, dtype=DT[case["grad"]], device="cuda")
    if own:
        from muon_polar_orthogonalized_b200 import api
        if op == "embed_grad":
            s["workspace"] = _bytes(api.muon_embedding_grad_workspace_size(case["vocab"], case["dim"], case["tokens"]))
        elif op == "norm_grad":
            s["workspace"] = _bytes(api.muon_layer_norm_backward_workspace_size(case["rows"], case["cols"]))
        elif op == "checkpoint":
            s["ckpt"] = api.new_checkpoint(case["rows"], case["cols"], "cuda")
        elif op == "weight_grad":
            s["ckpt"] = api.Checkpoint(s["q"], s["exps"], case["k"])
            s["workspace"] = _bytes(api.muon_checkpoint_weight_grad_workspace_size(
                case["rows"], case["n"], case["k"], s["dy"].dtype))
    return s


def _bytes(n):
    return torch.empty(max(int(n), 256), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ plain forms
def _encode(x):
    """(codes, exponents) of a checkpoint of x [rows, cols]: 8-bit floats
    (4 exponent, 3 mantissa bits; rows padded to 16 bytes) times 2^(e - 127),
    one e per row and block of 128 features: the smallest power of two that
    brings the block's largest magnitude to at most 448."""
    rows, cols = x.shape
    nb = (cols + BLOCK - 1) // BLOCK
    xf = torch.zeros(rows, nb * BLOCK, dtype=torch.float32, device=x.device)
    xf[:, :cols] = x
    xf = xf.view(rows, nb, BLOCK)
    m, e = torch.frexp(xf.abs().amax(2))
    power = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-124)
    power = torch.where(m == 0, torch.zeros_like(power), power)
    codes = torch.ldexp(xf, -power.unsqueeze(2)).to(torch.float8_e4m3fn)
    pitch = (cols + 15) // 16 * 16
    q = codes.view(torch.uint8).view(rows, nb * BLOCK)[:, :pitch].contiguous()
    return q, (power + 127).to(torch.uint8)


def _decode(q, exps, cols):
    """The values a checkpoint stands for, in 32 bits."""
    rows, nb = exps.shape
    v = q.view(torch.float8_e4m3fn).float()[:, :cols]
    power = (exps.int() - 127).repeat_interleave(BLOCK, 1)[:, :cols]
    return torch.ldexp(v, power)


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "embed":
        ids = s["ids"]
        there = (ids >= 0) & (ids < case["vocab"])
        rows = s["table"][ids.clamp(0, case["vocab"] - 1)].float() * s["scale"]
        return torch.where(there.unsqueeze(1), rows, torch.zeros((), device="cuda")).to(DT[case["out"]])
    if op == "embed_grad":
        ids = s["ids"]
        there = (ids >= 0) & (ids < case["vocab"])
        slot = torch.where(there, ids, torch.full_like(ids, case["vocab"]))
        total = torch.zeros(case["vocab"] + 1, case["dim"], dtype=torch.float32, device="cuda")
        total.index_add_(0, slot, s["dout"].float())
        return (total[:case["vocab"]] * s["scale"]).to(DT[case["grad"]])
    if op == "norm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        centred = x - mean
        rstd = torch.rsqrt((centred * centred).mean(1, keepdim=True) + EPS)
        y = centred * rstd * s["gain"]
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(DT[case["y"]]), mean.squeeze(1), rstd.squeeze(1)
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        xhat = (s["x"].float() - s["mean"].unsqueeze(1)) * rstd
        gy = dy * s["gain"]
        c1 = gy.mean(1, keepdim=True)
        c2 = (gy * xhat).mean(1, keepdim=True)
        dx = (rstd * (gy - c1 - xhat * c2)).to(DT[case["x"]])
        dgain = (dy * xhat).sum(0).to(DT[case["grad"]])
        return (dx, dgain, dy.sum(0).to(DT[case["grad"]])) if case["bias"] else (dx, dgain)
    if op == "checkpoint":
        q, exps = _encode(s["x"])
        return _decode(q, exps, case["cols"]).to(DT[case["x"]])
    x = _decode(s["q"], s["exps"], case["k"])
    return (s["dy"].float().t() @ x).to(DT[case["grad"]])


def _kernels(s):
    from muon_polar_orthogonalized_b200 import api
    op = s["op"]
    if op == "embed":
        api.muon_embedding_forward(s["table"], s["ids"], s["result"], scale=s["scale"])
        return s["result"]
    if op == "embed_grad":
        api.muon_embedding_grad(s["dout"], s["ids"], s["result"], s["workspace"], scale=s["scale"])
        return s["result"]
    if op == "norm":
        api.muon_layer_norm_forward(s["x"], s["gain"], s["bias"], s["y"], s["mean"], s["rstd"], eps=EPS)
        return s["y"], s["mean"], s["rstd"]
    if op == "norm_grad":
        api.muon_layer_norm_backward(s["dy"], s["x"], s["gain"], s["mean"], s["rstd"], s["dx"], s["dgain"],
                                     s["dbias"], s["workspace"])
        return (s["dx"], s["dgain"], s["dbias"]) if s["dbias"] is not None else (s["dx"], s["dgain"])
    if op == "checkpoint":
        api.muon_checkpoint_pack(s["x"], s["ckpt"])
        api.muon_checkpoint_unpack(s["ckpt"], s["result"])
        return s["result"]
    api.muon_checkpoint_weight_grad(s["dy"], s["ckpt"], s["result"], s["workspace"])
    return s["result"]


def run(state):
    return _kernels(state) if own else _plain(state)


# ------------------------------------------------------------------ work
def _distinct(vocab, n):
    """Expected distinct rows among n tokens of the batch's distribution."""
    cdf = _zipf_cdf(vocab, "cpu")
    p = torch.diff(cdf, prepend=torch.zeros(1, dtype=torch.float64))
    n = n - n // 16 if n >= 64 else n
    return float((1.0 - torch.exp(n * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    op = case["op"]
    if op == "embed":
        n, d = case["tokens"], case["dim"]
        rows = _distinct(case["vocab"], n)
        return {"bytes": rows * d * SIZE[case["table"]] + n * 8 + n * d * SIZE[case["out"]], "flops": n * d}
    if op == "embed_grad":
        n, d, v = case["tokens"], case["dim"], case["vocab"]
        there = n - n // 16 if n >= 64 else n
        return {"bytes": there * d * SIZE[case["dout"]] + n * 8 + v * d * SIZE[case["grad"]], "flops": 2 * there * d}
    if op == "norm":
        e = case["rows"] * case["cols"]
        return {"bytes": e * (SIZE[case["x"]] + SIZE[case["y"]]) + case["rows"] * 8
                + case["cols"] * (8 if case["bias"] else 4), "flops": 8 * e}
    if op == "norm_grad":
        e = case["rows"] * case["cols"]
        return {"bytes": 3 * e * SIZE[case["x"]] + case["rows"] * 8
                + case["cols"] * (4 + SIZE[case["grad"]] * (2 if case["bias"] else 1)), "flops": 14 * e}
    if op == "checkpoint":
        e = case["rows"] * case["cols"]
        codes = e + case["rows"] * ((case["cols"] + BLOCK - 1) // BLOCK)
        return {"bytes": 2 * e * SIZE[case["x"]] + 2 * codes, "flops": 4 * e}
    t, n, k = case["rows"], case["n"], case["k"]
    return {"bytes": t * n * SIZE[case["dy"]] + t * k + t * ((k + BLOCK - 1) // BLOCK) + n * k * SIZE[case["grad"]],
            "flops": 2 * t * n * k}


# ------------------------------------------------------------------ 64-bit results
def _code_values(x):
    """What a checkpoint of x stands for, from the format's definition: in each
    block the smallest p >= -124 with max|x| <= 448 * 2^p, and x / 2^p rounded
    to a multiple of 2^(max(floor(log2|.|), -6) - 3), ties to even."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c0 in range(0, x.shape[1], BLOCK):
        b = x[:, c0:c0 + BLOCK].double()
        big = b.abs().amax(1, keepdim=True)
        p = torch.floor(torch.log2(big.clamp(min=1e-300))) - 9
        for _ in range(2):
            p = torch.where(448.0 * torch.exp2(p) < big, p + 1, p)
        p = torch.where(big == 0, torch.zeros_like(p), p.clamp(min=-124))
        v = b * torch.exp2(-p)
        e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
        e = torch.where(v.abs() < torch.exp2(e), e - 1, e)
        e = torch.where(v.abs() >= torch.exp2(e + 1), e + 1, e).clamp(min=-6)
        step = torch.exp2(e - 3)
        out[:, c0:c0 + BLOCK] = torch.round(v / step) * step * torch.exp2(p)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        kept = torch.nonzero(s["ids"] >= 0).squeeze(1)
        out[kept] = s["table"].index_select(0, s["ids"][kept]).double() * s["scale"]
        return out
    if op == "embed_grad":
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        kept = torch.nonzero(s["ids"] >= 0).squeeze(1)
        out.index_put_((s["ids"][kept],), s["dout"][kept].double(), accumulate=True)
        return out.mul_(s["scale"])
    if op == "norm":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = s["gain"].double() * ((x - mean[:, None]) * rstd[:, None])
        return (y if s["bias"] is None else y + s["bias"].double()), mean, rstd
    if op == "norm_grad":
        n = case["cols"]
        r, dy = s["rstd"].double()[:, None], s["dy"].double()
        xh = (s["x"].double() - s["mean"].double()[:, None]) * r
        gy = dy * s["gain"].double()
        dx = (r / n) * (n * gy - gy.sum(1, keepdim=True) - xh * (gy * xh).sum(1, keepdim=True))
        dgain = torch.einsum("tc,tc->c", dy, xh)
        return (dx, dgain, dy.sum(0)) if case["bias"] else (dx, dgain)
    if op == "checkpoint":
        return _code_values(s["x"])
    byte = s["q"][:, :case["k"]].int()
    field, frac = (byte >> 3) & 15, (byte & 7).double()
    mag = torch.where(field == 0, frac * 2.0 ** -9, (1 + frac / 8) * torch.exp2((field - 7).double()))
    x = torch.where(byte >= 128, -mag, mag)
    col = torch.arange(case["k"], device="cuda") // BLOCK
    x = x * torch.exp2(s["exps"].double() - 127)[:, col]
    return torch.matmul(s["dy"].double().transpose(0, 1), x)
