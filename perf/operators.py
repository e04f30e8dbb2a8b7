"""The layer operators of the training front end, as measured work.

Four calls of ``distributed_bit_matrix_amd.binding``: the layer norm's forward
and backward pass and the embedding lookup with its gradient.  They are the
two kinds of layers of a transformer whose parameter gradients are not matrix
products: a gradient of theirs is a reduction over rows, which ends in the
float32 gradient that the optimizer step reads.

``run`` computes each either in its plain form (elementary torch operations in
32 bits) or, with ``own`` set, through the library.  ``exact`` has the same
results from the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5

# Limits of the drawn cases (the largest listed ones reach them).
MAX_NORM = 1 << 26       # entries of a layer norm's input
MAX_GRAD = 1 << 28       # entries of an embedding table
MAX_ROWS = 1 << 27       # entries of the looked-up rows


def listed():
    return [
        # one token of a decoder of width 768, where latency counts
        dict(name="norm one token", op="norm", rows=1, cols=768, x="bf16", w="bf16", bias=True),
        # a micro-batch of 12 x 1024 tokens at width 768
        dict(name="norm micro-batch", op="norm", rows=12288, cols=768, x="bf16", w="bf16",
             bias=True),
        # float32 activations of a wide model, the largest forward pass
        dict(name="norm wide", op="norm", rows=16384, cols=4096, x="f32", w="f32", bias=True),
        # the micro-batch's backward pass: the input's and both weights' gradients
        dict(name="norm grad micro-batch", op="norm_grad", rows=12288, cols=768, x="bf16",
             w="bf16", bias=True),
        # few rows of an odd width without a bias: a ragged batch's tail
        dict(name="norm grad ragged", op="norm_grad", rows=333, cols=1001, x="f32", w="f32",
             bias=False),
        # the largest backward pass, float32 master weights under bfloat16 activations
        dict(name="norm grad wide", op="norm_grad", rows=16384, cols=4096, x="bf16", w="f32",
             bias=True),
        # the lookup for a handful of sequences that each decode one token
        dict(name="embed one step", op="embed", n=8, vocab=50257, dim=768, x="bf16", w="bf16",
             tokens="zipf", scale=1.0),
        # a micro-batch's lookup, scaled by the root of the width
        dict(name="embed micro-batch", op="embed", n=12288, vocab=50257, dim=768, x="bf16",
             w="bf16", tokens="zipf", scale=27.712812921102035),
        # the token table's gradient of a micro-batch, in float32 for the step
        dict(name="embed grad micro-batch", op="embed_grad", n=12288, vocab=50257, dim=768,
             x="bf16", w="f32", tokens="zipf", scale=1.0),
        # the position table's gradient: every row is the sum over the batch
        dict(name="embed grad positions", op="embed_grad", n=65536, vocab=1024, dim=768,
             x="bf16", w="f32", tokens="positions", scale=1.0),
        # a short ragged batch into a small bfloat16 table of odd width
        dict(name="embed grad ragged", op="embed_grad", n=777, vocab=1000, dim=257, x="f32",
             w="bf16", tokens="uniform", scale=0.5),
        # the largest table and batch
        dict(name="embed grad large", op="embed_grad", n=65536, vocab=131072, dim=2048,
             x="bf16", w="f32", tokens="zipf", scale=1.0),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad"])
    x, w = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    if op.startswith("norm"):
        cols = _spread(rng, 1, 16384)
        rows = _spread(rng, 1, min(65536, MAX_NORM // cols))
        return dict(op=op, rows=rows, cols=cols, x=x, w=w, bias=rng.random() < 0.7)
    dim = _spread(rng, 1, 4096)
    return dict(op=op, n=_spread(rng, 1, min(131072, MAX_ROWS // dim)),
                vocab=_spread(rng, 2, min(131072, MAX_GRAD // dim)), dim=dim, x=x, w=w,
                tokens=rng.choice(["zipf", "uniform", "positions", "same"]),
                scale=rng.choice([1.0, 0.5, math.sqrt(dim)]))


def _tokens(kind, n, vocab, gen):
    """Token ids as a batch holds them: frequencies falling with the rank
    ("zipf"), even ones, the positions of equally long sequences, or one id
    repeated (a batch of padding)."""
    if kind == "positions":
        return torch.arange(n, device="cuda") % vocab
    if kind == "same":
        return torch.randint(vocab, (1,), device="cuda", generator=gen).repeat(n)
    if kind == "uniform":
        return torch.randint(vocab, (n,), device="cuda", generator=gen)
    u = torch.rand(n, device="cuda", generator=gen, dtype=torch.float64)
    return (vocab ** u).long().sub_(1).clamp_(0, vocab - 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, dtype="f32", std=1.0):
        return (std * torch.randn(*shape, device="cuda", generator=gen)).to(DTYPES[dtype])

    state = dict(case=case)
    if case["op"].startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        # hidden states: some columns far larger than the rest, a mean that is not zero
        x = torch.randn(rows, cols, device="cuda", generator=gen)
        x.mul_(1 + 4 * torch.rand(cols, device="cuda", generator=gen) ** 8).add_(0.3)
        state["x"] = x.to(DTYPES[case["x"]])
        state["weight"] = (1 + normal(cols, std=0.2)).to(DTYPES[case["w"]])
        state["bias"] = normal(cols, dtype=case["w"], std=0.2) if case["bias"] else None
        if case["op"] == "norm_grad":
            state["dy"] = normal(rows, cols, dtype=case["x"])
            # what the forward pass saved
            x = state["x"].double()
            state["mean"] = x.mean(1).float()
            state["rstd"] = torch.rsqrt(x.var(1, unbiased=False) + EPS).float()
        return state
    n, vocab, dim = case["n"], case["vocab"], case["dim"]
    state["tokens"] = _tokens(case["tokens"], n, vocab, gen)
    if case["op"] == "embed":
        state["weight"] = normal(vocab, dim, dtype=case["w"], std=0.02)
    else:
        state["dy"] = normal(n, dim, dtype=case["x"])
    return state


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "norm":
        x = state["x"].float()
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = torch.rsqrt((xc * xc).mean(1, keepdim=True) + EPS)
        y = xc * rstd * state["weight"].float()
        if state["bias"] is not None:
            y = y + state["bias"].float()
        return dict(y=y.to(state["x"].dtype), mean=mean[:, 0], rstd=rstd[:, 0])
    if case["op"] == "norm_grad":
        dy, rstd = state["dy"].float(), state["rstd"][:, None]
        xhat = (state["x"].float() - state["mean"][:, None]) * rstd
        g = dy * state["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
        out = dict(dx=dx.to(state["x"].dtype), dweight=(dy * xhat).sum(0))
        if state["bias"] is not None:
            out["dbias"] = dy.sum(0)
        return out
    if case["op"] == "embed":
        return (case["scale"] * state["weight"][state["tokens"]].float()).to(DTYPES[case["x"]])
    dw = torch.zeros(case["vocab"], case["dim"], device="cuda")
    dw.index_add_(0, state["tokens"], state["dy"].float())
    return dw.mul_(case["scale"]).to(DTYPES[case["w"]])


def _run_own(case, state):
    from distributed_bit_matrix_amd import binding as B

    if case["op"] == "norm":
        y, mean, rstd = B.layer_norm(state["x"], state["weight"], state["bias"], EPS,
                                     want_stats=True)
        return dict(y=y, mean=mean, rstd=rstd)
    if case["op"] == "norm_grad":
        dx, dweight, dbias = B.layer_norm_backward(
            state["dy"], state["x"], state["weight"], state["mean"], state["rstd"],
            want_bias=state["bias"] is not None)
        out = dict(dx=dx, dweight=dweight)
        if dbias is not None:
            out["dbias"] = dbias
        return out
    if case["op"] == "embed":
        return B.embedding(state["tokens"], state["weight"], case["scale"],
                           out_dtype=DTYPES[case["x"]])
    return B.embedding_backward(state["dy"], state["tokens"], case["vocab"], case["scale"],
                                dtype=DTYPES[case["w"]])


def work(case):
    size = {"f32": 4, "bf16": 2}
    xs, ws = size[case["x"]], size[case["w"]]
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": 2 * rows * cols * xs + (1 + case["bias"]) * cols * ws + 8 * rows,
                "flops": 8 * rows * cols}
    if case["op"] == "norm_grad":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": 3 * rows * cols * xs + cols * ws + (1 + case["bias"]) * cols * 4
                + 8 * rows, "flops": 14 * rows * cols}
    n, vocab, dim = case["n"], case["vocab"], case["dim"]
    if case["op"] == "embed":
        # each distinct row once; a batch has at most as many as the table
        return {"bytes": 8 * n + min(n, vocab) * dim * ws * (case["tokens"] != "same")
                + n * dim * xs, "flops": n * dim}
    return {"bytes": 8 * n + n * dim * xs + vocab * dim * ws, "flops": n * dim}


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"].startswith("norm"):
        x = state["x"].double()
        cols = x.shape[1]
        if case["op"] == "norm":
            mean = x.sum(1) / cols
            var = ((x - mean[:, None]) ** 2).sum(1) / cols
            rstd = 1 / torch.sqrt(var + EPS)
            y = torch.addcmul(state["bias"].double() if state["bias"] is not None
                              else torch.zeros(cols, dtype=torch.float64, device="cuda"),
                              (x - mean[:, None]) / torch.sqrt(var + EPS)[:, None],
                              state["weight"].double())
            return dict(y=y, mean=mean, rstd=rstd)
        dy, mean, rstd = state["dy"].double(), state["mean"].double(), state["rstd"].double()
        xhat = (x - mean[:, None]) * rstd[:, None]
        g = dy * state["weight"].double()
        c1 = g.sum(1) / cols
        c2 = torch.linalg.vecdot(g, xhat) / cols
        out = dict(dx=(g - c1[:, None] - xhat * c2[:, None]) * rstd[:, None],
                   dweight=torch.linalg.vecdot(dy, xhat, dim=0))
        if state["bias"] is not None:
            out["dbias"] = torch.linalg.vecdot(dy, torch.ones_like(dy), dim=0)
        return out
    if case["op"] == "embed":
        return torch.index_select(state["weight"].double(), 0, state["tokens"]) * case["scale"]
    # running sums over the sorted tokens would cancel; every row's own sum instead
    order = torch.argsort(state["tokens"], stable=True)
    found, counts = torch.unique_consecutive(state["tokens"][order], return_counts=True)
    dw = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    dw[found] = torch.segment_reduce(state["dy"][order].double(), "sum", lengths=counts,
                                     axis=0)
    return dw * case["scale"]
