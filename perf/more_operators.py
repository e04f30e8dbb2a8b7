"""More layer operators of the training front end, as measured work.

Calls of ``distributed_bit_matrix_amd.binding`` that a transformer trained with
the optimizer needs beside the layer norm and the embedding: the
root-mean-square norm of the sum of a residual stream and what a layer adds to
it (with an output in 8 bits and scales too), the gated feed-forward block, and
the softmax cross entropy of a linear output layer over the vocabulary, whose
logits are not kept.  Each has its backward pass.

``run`` computes each either in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library.  ``exact`` has the same
results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
IGNORE = -100
BLOCK = 128              # columns that share a scale of the 8-bit output
E4M3_MAX = 448.0
LEAST_SCALE = 2.0 ** -126

# Limits of the drawn cases (the largest listed ones reach them).
MAX_NORM = 1 << 26                       # entries of a norm's input
MAX_BLOCK = 4096 * 4096 * 16384          # rows * width * hidden of a feed-forward block
MAX_LOSS = 12288 * 768 * 50257           # rows * width * vocabulary of a loss


def listed():
    return [
        # one token of a decoder of width 4096, where latency counts
        dict(name="rms one token", op="rms", rows=1, cols=4096, x="bf16", w="bf16", residual=True,
             out="same"),
        # a prompt of a wide model before a product in 8 bits, the largest forward pass
        dict(name="rms wide e4m3", op="rms", rows=16384, cols=4096, x="bf16", w="bf16",
             residual=True, out="e4m3"),
        # a micro-batch of 12 x 1024 tokens at width 768 under float32 master weights
        dict(name="rms grad micro-batch", op="rms_grad", rows=12288, cols=768, x="bf16", w="f32",
             residual=True),
        # the largest backward pass of the norm
        dict(name="rms grad wide", op="rms_grad", rows=16384, cols=4096, x="bf16", w="bf16",
             residual=True),
        # one token of a decoder whose matrices are 4096 x 16384: every weight read once
        dict(name="ffn one token", op="ffn", rows=1, dim=4096, hidden=16384, x="bf16",
             act="silu", keep=False),
        # four sequences of 1024 tokens through the same block in training
        dict(name="ffn wide", op="ffn", rows=4096, dim=4096, hidden=16384, x="bf16", act="silu",
             keep=True),
        # the micro-batch's backward pass at width 768
        dict(name="ffn grad micro-batch", op="ffn_grad", rows=12288, dim=768, hidden=2048,
             x="bf16", act="gelu"),
        # a ragged batch in float32, every size odd
        dict(name="ffn grad ragged", op="ffn_grad", rows=333, dim=1001, hidden=2731, x="f32",
             act="silu"),
        # scoring eight sequences' next tokens against the token table
        dict(name="loss few rows", op="loss", rows=8, dim=768, vocab=50257, x="bf16",
             reduction="none", ignored=0.0),
        # a micro-batch's loss, a tenth of it padding
        dict(name="loss micro-batch", op="loss", rows=12288, dim=768, vocab=50257, x="bf16",
             reduction="mean", ignored=0.1),
        # its gradients of the hidden states and the table: the largest case
        dict(name="loss grad micro-batch", op="loss_grad", rows=12288, dim=768, vocab=50257,
             x="bf16", reduction="mean", ignored=0.1),
        # a ragged batch in float32 over a small vocabulary
        dict(name="loss grad ragged", op="loss_grad", rows=1023, dim=257, vocab=10007, x="f32",
             reduction="sum", ignored=0.3),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform over its logarithm."""
    hi = max(lo, hi)
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rms", "rms_grad", "ffn", "ffn_grad", "loss", "loss_grad"])
    x, w = rng.choice(["f32", "bf16", "bf16"]), rng.choice(["f32", "bf16"])
    if op in ("rms", "rms_grad"):
        cols = _spread(rng, 1, 16384)
        case = dict(op=op, rows=_spread(rng, 1, min(65536, MAX_NORM // cols)), cols=cols, x=x, w=w,
                    residual=rng.random() < 0.7)
        if op == "rms":
            case["out"] = rng.choice(["same", "e4m3"])
        return case
    dim = _spread(rng, 16, 4096)
    if op in ("ffn", "ffn_grad"):
        hidden = _spread(rng, 16, 16384)
        # the backward pass has twice the forward's products
        most = MAX_BLOCK // (2 if op == "ffn_grad" else 1) // (dim * hidden)
        case = dict(op=op, rows=_spread(rng, 1, min(16384, most)), dim=dim, hidden=hidden, x=x,
                    act=rng.choice(["silu", "gelu"]))
        if op == "ffn":
            case["keep"] = rng.random() < 0.5
        return case
    vocab = _spread(rng, 2, 131072)
    return dict(op=op, rows=_spread(rng, 1, min(16384, MAX_LOSS // (dim * vocab))), dim=dim,
                vocab=vocab, x=x, reduction=rng.choice(["mean", "sum", "none"]),
                ignored=rng.choice([0.0, 0.1, 0.5]))


def _ignored(case):
    """How many rows of a loss are padding; one at least is not."""
    return min(case["rows"] - 1, round(case["rows"] * case["ignored"]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype="f32", std=1.0):
        return (std * torch.randn(*shape, device="cuda", generator=gen)).to(DTYPES[dtype])

    x, op, rows = case["x"], case["op"], case["rows"]
    state = dict(case=case)
    if op in ("rms", "rms_grad"):
        cols = case["cols"]
        # a residual stream: some columns far larger than the rest
        stream = torch.randn(rows, cols, device="cuda", generator=gen)
        stream.mul_(1 + 4 * torch.rand(cols, device="cuda", generator=gen) ** 8)
        state["weight"] = (1 + normal(cols, std=0.2)).to(DTYPES[case["w"]])
        if op == "rms":
            state["x"] = normal(rows, cols, dtype=x, std=0.5)
            state["residual"] = stream.to(DTYPES[x]) if case["residual"] else None
            return state
        state["h"] = stream.to(DTYPES[x])
        state["dy"] = normal(rows, cols, dtype=x)
        state["dh"] = normal(rows, cols, dtype=x) if case["residual"] else None
        # what the forward pass saved
        state["rstd"] = torch.rsqrt(state["h"].double().square().mean(1) + EPS).float()
        return state
    dim = case["dim"]
    if op in ("ffn", "ffn_grad"):
        hidden = case["hidden"]
        state["x"] = normal(rows, dim, dtype=x)
        state["w_gate"] = normal(hidden, dim, dtype=x, std=dim ** -0.5)
        state["w_up"] = normal(hidden, dim, dtype=x, std=dim ** -0.5)
        state["w_down"] = normal(dim, hidden, dtype=x, std=hidden ** -0.5)
        if op == "ffn_grad":
            state["dy"] = normal(rows, dim, dtype=x)
            # what the forward pass kept
            state["pre"] = torch.cat([state["x"].float() @ state[k].float().T
                                      for k in ("w_gate", "w_up")], 1)
        return state
    vocab = case["vocab"]
    table = torch.randn(vocab, dim, device="cuda", generator=gen)
    # tokens whose frequencies fall with their rank
    u = torch.rand(rows, device="cuda", generator=gen, dtype=torch.float64)
    targets = (vocab ** u).long().sub_(1).clamp_(0, vocab - 1)
    # hidden states that have learned something: the target's logit stands out
    # by about eight, the other logits have a deviation of one and a half
    hidden = torch.randn(rows, dim, device="cuda", generator=gen)
    hidden.mul_(1.5).add_(table[targets], alpha=8.0 / math.sqrt(dim))
    state["x"] = hidden.to(DTYPES[x])
    state["weight"] = table.mul_(1 / math.sqrt(dim)).to(DTYPES[x])
    padding = torch.randperm(rows, device="cuda", generator=gen)[:_ignored(case)]
    state["targets"] = targets.index_fill_(0, padding, IGNORE)
    if op == "loss_grad":
        shape = (rows,) if case["reduction"] == "none" else ()
        state["dloss"] = 1 + 0.2 * torch.randn(shape, device="cuda", generator=gen)
        # what the forward pass saved
        state["lse"] = torch.cat([torch.logsumexp(part.float() @ state["weight"].float().T, 1)
                                  for part in state["x"].split(2048)])
        state["lse"].masked_fill_(state["targets"] == IGNORE, 0.0)
    return state


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _run_own(case, state)
    if op == "rms":
        return _plain_rms(case, state)
    if op == "rms_grad":
        h, rstd = state["h"].float(), state["rstd"][:, None]
        dy = state["dy"].float()
        xhat = h * rstd
        g = dy * state["weight"].float()
        dx = rstd * (g - xhat * (g * xhat).mean(1, keepdim=True))
        if state["dh"] is not None:
            dx = dx + state["dh"].float()
        return dict(dx=dx.to(state["h"].dtype), dweight=(dy * xhat).sum(0))
    if op == "ffn":
        x = state["x"].float()
        gate, up = x @ state["w_gate"].float().T, x @ state["w_up"].float().T
        y = (_act(case["act"], gate) * up) @ state["w_down"].float().T
        out = dict(y=y.to(state["x"].dtype))
        if case["keep"]:
            out["pre"] = torch.cat([gate, up], 1)
        return out
    if op == "ffn_grad":
        return _plain_ffn_grad(case, state)
    if op == "loss":
        return _plain_loss(case, state)
    return _plain_loss_grad(case, state)


def _plain_rms(case, state):
    # the norm is taken of the sum as it is stored
    h = state["x"]
    if state["residual"] is not None:
        h = (h.float() + state["residual"].float()).to(h.dtype)
    x = h.float()
    rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    y = x * rstd * state["weight"].float()
    out = dict(rstd=rstd[:, 0])
    if state["residual"] is not None:
        out["h"] = h
    if case["out"] == "same":
        return dict(out, y=y.to(h.dtype))
    rows, cols = y.shape
    blocks = -(-cols // BLOCK)
    parts = torch.nn.functional.pad(y, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    scales = (parts.abs().amax(2) / E4M3_MAX).clamp(min=LEAST_SCALE)
    codes = (parts / scales[:, :, None]).to(torch.float8_e4m3fn)
    # the codes' own values; bfloat16 has all of them
    codes = codes.to(torch.bfloat16).view(rows, blocks * BLOCK)[:, :cols]
    return dict(out, codes=codes.contiguous(), scales=scales)


def _act(kind, gate):
    if kind == "silu":
        return gate / (1 + torch.exp(-gate))
    return 0.5 * gate * (1 + torch.erf(gate * math.sqrt(0.5)))


def _act_slope(kind, gate):
    if kind == "silu":
        s = 1 / (1 + torch.exp(-gate))
        return s * (1 + gate * (1 - s))
    bell = torch.exp(-0.5 * gate * gate) / math.sqrt(2 * math.pi)
    return 0.5 * (1 + torch.erf(gate * math.sqrt(0.5))) + gate * bell


def _plain_ffn_grad(case, state):
    dtype = state["x"].dtype
    x, dy = state["x"].float(), state["dy"].float()
    gate, up = state["pre"].chunk(2, 1)
    act = _act(case["act"], gate)
    dw_down = dy.T @ (act * up)
    dh = dy @ state["w_down"].float()
    d_up = dh * act
    d_gate = dh * up * _act_slope(case["act"], gate)
    dx = d_gate @ state["w_gate"].float() + d_up @ state["w_up"].float()
    return dict(dx=dx.to(dtype), dw_gate=(d_gate.T @ x).to(dtype), dw_up=(d_up.T @ x).to(dtype),
                dw_down=dw_down.to(dtype))


def _plain_loss(case, state):
    targets = state["targets"]
    keep = targets != IGNORE
    logits = state["x"].float() @ state["weight"].float().T
    picked = logits.gather(1, targets.clamp(min=0)[:, None])[:, 0]
    most = logits.amax(1)
    lse = most + torch.log(logits.sub_(most[:, None]).exp_().sum(1))
    loss = torch.where(keep, lse - picked, 0.0)
    if case["reduction"] != "none":
        loss = loss.sum()
    if case["reduction"] == "mean":
        loss = loss / keep.sum()
    return dict(loss=loss, lse=torch.where(keep, lse, 0.0))


def _plain_loss_grad(case, state):
    targets = state["targets"]
    keep = targets != IGNORE
    x, weight = state["x"].float(), state["weight"].float()
    g = (x @ weight.T).sub_(state["lse"][:, None]).exp_()
    g.scatter_add_(1, targets.clamp(min=0)[:, None], -torch.ones_like(g[:, :1]))
    scale = torch.where(keep, state["dloss"], 0.0)
    if case["reduction"] == "mean":
        scale = scale / keep.sum()
    g.mul_(scale[:, None])
    g[~keep] = 0.0
    return dict(dx=(g @ weight).to(state["x"].dtype), dweight=(g.T @ x).to(state["x"].dtype))


def _run_own(case, state):
    from distributed_bit_matrix_amd import binding as B

    op = case["op"]
    if op == "rms":
        if case["out"] == "same":
            y, h, rstd = B.rms_norm(state["x"], state["weight"], state["residual"], EPS,
                                    want_stats=True)
            out = dict(y=y, rstd=rstd)
        else:
            codes, scales, h, rstd = B.rms_norm_e4m3(state["x"], state["weight"],
                                                     state["residual"], EPS, block=BLOCK,
                                                     want_stats=True)
            out = dict(codes=codes.to(torch.bfloat16), scales=scales, rstd=rstd)
        if state["residual"] is not None:
            out["h"] = h
        return out
    if op == "rms_grad":
        dx, dweight = B.rms_norm_backward(state["dy"], state["h"], state["weight"], state["rstd"],
                                          dH=state["dh"])
        return dict(dx=dx, dweight=dweight)
    if op == "ffn":
        out = B.gated_mlp(state["x"], state["w_gate"], state["w_up"], state["w_down"],
                          case["act"], want_pre=case["keep"])
        return dict(y=out[0], pre=out[1]) if case["keep"] else dict(y=out)
    if op == "ffn_grad":
        dx, dw_gate, dw_up, dw_down = B.gated_mlp_backward(
            state["dy"], state["x"], state["w_gate"], state["w_up"], state["w_down"],
            state["pre"], case["act"], dtype=state["x"].dtype)
        return dict(dx=dx, dw_gate=dw_gate, dw_up=dw_up, dw_down=dw_down)
    if op == "loss":
        loss, lse = B.linear_cross_entropy(state["x"], state["weight"], state["targets"],
                                           IGNORE, case["reduction"], want_lse=True)
        return dict(loss=loss, lse=lse)
    dx, dweight = B.linear_cross_entropy_backward(
        state["dloss"], state["x"], state["weight"], state["targets"], state["lse"], IGNORE,
        case["reduction"], dtype=state["x"].dtype)
    return dict(dx=dx, dweight=dweight)


def work(case):
    size = {"f32": 4, "bf16": 2}
    op, rows, xs = case["op"], case["rows"], size[case["x"]]
    if op in ("rms", "rms_grad"):
        cols, ws = case["cols"], size[case["w"]]
        n = rows * cols
        if op == "rms":
            out = n * xs if case["out"] == "same" else n + 4 * rows * -(-cols // BLOCK)
            return {"bytes": (3 if case["residual"] else 1) * n * xs + out + cols * ws + 4 * rows,
                    "flops": 6 * n}
        return {"bytes": (4 if case["residual"] else 3) * n * xs + cols * (ws + 4) + 4 * rows,
                "flops": 12 * n}
    dim = case["dim"]
    if op in ("ffn", "ffn_grad"):
        hidden = case["hidden"]
        weights, ends, pre = 3 * dim * hidden * xs, rows * dim * xs, 8 * rows * hidden
        if op == "ffn":
            return {"bytes": weights + 2 * ends + (pre if case["keep"] else 0),
                    "flops": 6 * rows * dim * hidden}
        return {"bytes": 2 * weights + 3 * ends + pre, "flops": 12 * rows * dim * hidden}
    vocab, kept = case["vocab"], rows - _ignored(case)
    read = (kept + vocab) * dim * xs + 8 * rows + 4 * rows
    if op == "loss":
        return {"bytes": read, "flops": 2 * kept * vocab * dim}
    # the logits again, and a product for each of the gradients
    return {"bytes": read + (rows + vocab) * dim * xs, "flops": 6 * kept * vocab * dim}


def _round_e4m3(v):
    """To the nearest value of three fraction bits above 2^-6 and steps of 2^-9
    below it, halves to even; at most 448 comes in."""
    step = torch.exp2(torch.frexp(v).exponent.clamp(min=-5).double() - 4)
    return torch.round(v / step) * step


def exact(case, seed):
    F = torch.nn.functional
    state = prepare(case, seed)
    op = case["op"]
    wide = {k: v.double() for k, v in state.items()
            if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "rms":
        h = wide["x"]
        out = {}
        if state["residual"] is not None:
            out["h"] = h + wide["residual"]
            h = out["h"].to(state["x"].dtype).double()
        var = torch.linalg.vecdot(h, h) / h.shape[1] + EPS
        y = h / torch.sqrt(var)[:, None] * wide["weight"]
        out["rstd"] = 1 / torch.sqrt(var)
        if case["out"] == "same":
            return dict(out, y=y)
        blocks = y.split(BLOCK, 1)
        scales = torch.stack([b.abs().max(1).values for b in blocks], 1) / E4M3_MAX
        scales = torch.maximum(scales, torch.full_like(scales, LEAST_SCALE))
        codes = torch.cat([b / s for b, s in zip(blocks, scales.split(1, 1))], 1)
        return dict(out, codes=_round_e4m3(codes), scales=scales)
    if op == "rms_grad":
        h, dy, r = wide["h"], wide["dy"], wide["rstd"]
        cols = h.shape[1]
        g = wide["weight"] * dy
        dx = g * r[:, None] - h * (torch.linalg.vecdot(g, h) * r ** 3 / cols)[:, None]
        if state["dh"] is not None:
            dx = dx + wide["dh"]
        return dict(dx=dx, dweight=torch.linalg.vecdot(dy, h * r[:, None], dim=0))
    if op in ("ffn", "ffn_grad"):
        act = F.silu if case["act"] == "silu" else F.gelu
        if op == "ffn":
            pre = F.linear(wide["x"], torch.cat([wide["w_gate"], wide["w_up"]]))
            gate, up = pre.tensor_split(2, 1)
            out = dict(y=F.linear(act(gate) * up, wide["w_down"]))
            return dict(out, pre=pre) if case["keep"] else out
        with torch.enable_grad():
            pre, w_down = wide["pre"].requires_grad_(), wide["w_down"].requires_grad_()
            gate, up = pre.tensor_split(2, 1)
            dpre, dw_down = torch.autograd.grad(F.linear(act(gate) * up, w_down), (pre, w_down),
                                                wide["dy"])
        dw = dpre.T.contiguous().mm(wide["x"])
        dw_gate, dw_up = dw.tensor_split(2, 0)
        return dict(dx=dpre.mm(torch.cat([wide["w_gate"], wide["w_up"]])), dw_gate=dw_gate,
                    dw_up=dw_up, dw_down=dw_down)
    targets = state["targets"]
    keep = (targets != IGNORE).nonzero()[:, 0]
    x, weight, at = wide["x"][keep], wide["weight"], targets[keep]
    logits = F.linear(x, weight)
    share = 1.0 / len(keep) if case["reduction"] == "mean" else 1.0
    if op == "loss":
        each = F.cross_entropy(logits, at, reduction="none")
        lse = torch.zeros(len(targets), dtype=torch.float64, device="cuda")
        lse[keep] = each + logits[torch.arange(len(keep), device="cuda"), at]
        if case["reduction"] == "none":
            loss = torch.zeros_like(lse)
            loss[keep] = each
        else:
            loss = each.sum() * share
        return dict(loss=loss, lse=lse)
    g = torch.exp(logits - wide["lse"][keep][:, None])
    del logits
    g[torch.arange(len(keep), device="cuda"), at] -= 1
    g *= (wide["dloss"].expand(len(targets))[keep] * share)[:, None]
    dx = torch.zeros_like(wide["x"])
    dx[keep] = g.mm(weight)
    return dict(dx=dx, dweight=x.T.contiguous().mm(g).T)
