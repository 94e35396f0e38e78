"""Timing cases of the operators that make the optimizer's gradients: the token embedding, the
root-mean-square norm, and 8-bit activation checkpoints with the weight gradient taken from them.

`run` computes a case either with the library's calls (`own` true) or in plain torch operations in
32 bits, on the same inputs; `exact` gives the definition in 64 bits.
"""
import math

import torch

own = False

GPT2_VOCAB, LLAMA_VOCAB = 50257, 128256
BLOCK = 32                      # checkpoint elements under one scale
E4M3_MAX = 448.0
E_LO, E_HI = -117, 119          # range of a scale's exponent
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # decoding: the embedding row of one new token
        dict(name="lookup 1 token", op="embedding", n=1, vocab=LLAMA_VOCAB, dim=4096, table="fp32", out="bf16", ids="int64", scale=1.0),
        # the forward pass of a GPT-2-small batch of 16 sequences
        dict(name="lookup 16384", op="embedding", n=16384, vocab=GPT2_VOCAB, dim=768, table="fp32", out="bf16", ids="int64", scale=math.sqrt(768.0)),
        # a GPT-2-small batch of 12 sequences less their last token, gradients gathered over micro-batches in fp32
        dict(name="embed grad 12276", op="embedding_grad", n=12276, vocab=GPT2_VOCAB, dim=768, dy="bf16", grad="fp32", ids="int64", scale=math.sqrt(768.0), accumulate=True),
        # a Llama-8B batch of two long sequences, the whole gradient for adamw_step
        dict(name="embed grad 16384 wide", op="embedding_grad", n=16384, vocab=LLAMA_VOCAB, dim=4096, dy="bf16", grad="bf16", ids="int32", scale=1.0, accumulate=False),
        # one token through a Llama-8B layer's norm
        dict(name="norm 1 row", op="norm", rows=1, dim=4096, x="bf16", residual=True, y=True, checkpoint=False),
        # a training step's norm: residual stream, input of the next product, and its checkpoint
        dict(name="norm 16384 checkpoint", op="norm", rows=16384, dim=4096, x="bf16", residual=True, y=True, checkpoint=True),
        # its backward pass
        dict(name="norm grad 16384", op="norm_grad", rows=16384, dim=4096, x="bf16", dh=True),
        # fp32 training with odd sizes
        dict(name="norm grad 1021 odd", op="norm_grad", rows=1021, dim=1537, x="fp32", dh=False),
        # a ragged micro-batch of Mamba inner activations stored and restored
        dict(name="checkpoint 1023", op="checkpoint", rows=1023, dim=1536, x="fp32"),
        # the input of a Llama-8B down projection stored for, and restored in, the backward pass
        dict(name="checkpoint 8192 wide", op="checkpoint", rows=8192, dim=14336, x="bf16"),
        # GPT-2-small's QKV weight over a micro-batch, gathered in fp32
        dict(name="weight grad 768x2304", op="weight_grad", rows=8192, n=768, k=2304, dy="bf16", grad="fp32", accumulate=True),
        # a Llama-8B gate projection
        dict(name="weight grad 14336x4096", op="weight_grad", rows=8192, n=14336, k=4096, dy="bf16", grad="bf16", accumulate=False),
    ]


def _size(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm; half of them multiples of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 16 and rng.random() < 0.5:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "norm", "norm_grad", "checkpoint", "weight_grad"])
    t = lambda: rng.choice(["bf16", "bf16", "fp32"])  # noqa: E731
    if op in ("embedding", "embedding_grad"):
        n, vocab, dim = _size(rng, 1, 16384), _size(rng, 1000, LLAMA_VOCAB), _size(rng, 64, 4096)
        case = dict(op=op, n=n, vocab=vocab, dim=dim, ids=rng.choice(["int32", "int64"]), scale=rng.choice([1.0, math.sqrt(dim)]))
        if op == "embedding":
            return dict(case, table=rng.choice(["fp32", "bf16"]), out=t())
        return dict(case, dy=t(), grad=t(), accumulate=rng.random() < 0.4)
    if op in ("norm", "norm_grad"):
        case = dict(op=op, rows=_size(rng, 1, 16384), dim=_size(rng, 64, 8192), x=t())
        while case["rows"] * case["dim"] > 16384 * 4096:
            case["rows"] = _size(rng, 1, 16384)
        if op == "norm":
            y = rng.random() < 0.7
            return dict(case, residual=rng.random() < 0.7, y=y, checkpoint=not y or rng.random() < 0.5)
        return dict(case, dh=rng.random() < 0.6)
    if op == "checkpoint":
        case = dict(op=op, rows=_size(rng, 1, 16384), dim=_size(rng, 64, 14336), x=t())
        while case["rows"] * case["dim"] > 8192 * 14336:
            case["rows"] = _size(rng, 1, 16384)
        return case
    case = dict(op=op, rows=_size(rng, 1, 16384), n=_size(rng, 48, 14336), k=_size(rng, 48, 14336), dy=rng.choice(["bf16", "bf16", "bf16", "fp32"]),
                grad=t(), accumulate=rng.random() < 0.4)
    while case["rows"] * case["n"] * case["k"] > 8192 * 14336 * 4096 / (3 if case["dy"] == "fp32" else 1) or case["n"] * case["k"] > 14336 * 4096:
        case["rows"], case["n"] = _size(rng, 1, 16384), _size(rng, 48, 14336)
    return case


# ---------------------------------------------------------------------------- inputs

def _tokens(case, gen):
    """Token ids whose frequency falls with their rank (id r about as often as 1 / (r + 1)), and a
    few places of padding (-1) at the end of the batch."""
    n, vocab = case["n"], case["vocab"]
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    if n > 64:
        ids[n - n // 64:] = -1
    return ids.to(torch.int32 if case["ids"] == "int32" else torch.int64)


def _normal(shape, gen, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(DTYPES[dtype])


def _columns(shape, gen, std, lo, hi, dtype):
    """Normal values times a scale of each column, spread evenly over the logarithm of [lo, hi]."""
    s = torch.exp(torch.rand(shape[1], generator=gen, device="cuda") * math.log(hi / lo) + math.log(lo))
    return (torch.randn(shape, generator=gen, device="cuda").mul_(std).mul_(s)).to(DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, op = case, case["op"]
    s = dict(case)
    if op == "embedding":
        s["table"] = _normal((c["vocab"], c["dim"]), gen, 0.02, c["table"])
        s["tokens"] = _tokens(c, gen)
    elif op == "embedding_grad":
        s["tokens"] = _tokens(c, gen)
        s["dy"] = _columns((c["n"], c["dim"]), gen, 1e-3, 0.1, 10.0, c["dy"])
        if c["accumulate"]:
            s["buffer"] = _columns((c["vocab"], c["dim"]), gen, 1e-3, 0.1, 10.0, c["grad"])
    elif op == "norm":
        s["x"] = _columns((c["rows"], c["dim"]), gen, 1.0, 0.1, 10.0, c["x"])
        s["r"] = _columns((c["rows"], c["dim"]), gen, 2.0, 0.1, 10.0, c["x"]) if c["residual"] else None
        s["weight"] = 1.0 + 0.1 * torch.randn(c["dim"], generator=gen, device="cuda")
    elif op == "norm_grad":
        s["h"] = _columns((c["rows"], c["dim"]), gen, 2.0, 0.1, 10.0, c["x"])
        s["weight"] = 1.0 + 0.1 * torch.randn(c["dim"], generator=gen, device="cuda")
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + 1e-5).float()
        s["dy"] = _columns((c["rows"], c["dim"]), gen, 1e-3, 0.1, 10.0, c["x"])
        s["dh_in"] = _normal((c["rows"], c["dim"]), gen, 1e-3, c["x"]) if c["dh"] else None
    elif op == "checkpoint":
        s["x"] = _columns((c["rows"], c["dim"]), gen, 1.0, 0.1, 10.0, c["x"])
    else:
        x = _columns((c["rows"], c["k"]), gen, 1.0, 0.1, 10.0, "bf16")
        s["q"], s["scales"] = _quantise(x)
        s["dy"] = _columns((c["rows"], c["n"]), gen, 1e-3, 0.1, 10.0, c["dy"])
        if c["accumulate"]:
            s["buffer"] = _normal((c["n"], c["k"]), gen, 1e-2, c["grad"])
    return s


# ---------------------------------------------------------------------------- the plain forms

def _quantise(x):
    """e4m3 values and power-of-two scales of the blocks of 32 along each row of x: the smallest
    scale whose 448-fold the block does not exceed, within [2^-117, 2^119]."""
    rows, dim = x.shape
    blocks = -(-dim // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, blocks * BLOCK - dim)).view(rows, blocks, BLOCK)
    m, e = torch.frexp(v.abs().amax(2))
    e = (e - 9 + (m > 0.875)).clamp(E_LO, E_HI)
    q = torch.ldexp(v, -e[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).reshape(rows, blocks * BLOCK)[:, :dim]
    return q.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _restore(q, scales):
    rows, dim = q.shape
    return q.float() * scales.float().repeat_interleave(BLOCK, 1)[:, :dim]


def _plain_embedding(s):
    t, vocab = s["tokens"].long(), s["vocab"]
    have = (t >= 0) & (t < vocab)
    rows = s["table"][t.clamp(0, vocab - 1)].float() * s["scale"]
    return torch.where(have[:, None], rows, 0.0).to(DTYPES[s["out"]])


def _plain_embedding_grad(s):
    t, vocab = s["tokens"].long(), s["vocab"]
    have = (t >= 0) & (t < vocab)
    rows = torch.where(have[:, None], s["dy"].float(), 0.0)
    g = torch.zeros((vocab, s["dim"]), device=rows.device).index_add_(0, t.clamp(0, vocab - 1), rows).mul_(s["scale"])
    if not s["accumulate"]:
        return g.to(DTYPES[s["grad"]])
    return s["buffer"].copy_(g.add_(s["buffer"].float()))


def _plain_norm(s):
    x = s["x"]
    h = x if s["r"] is None else (x.float() + s["r"].float()).to(x.dtype)
    f = h.float()
    rstd = torch.rsqrt(f.square().mean(1) + 1e-5)
    y = f * rstd[:, None] * s["weight"]
    q, scales = _quantise(y) if s["checkpoint"] else (None, None)
    return dict(h=h, rstd=rstd, y=y.to(x.dtype) if s["y"] else None, q=q, scales=scales)


def _plain_norm_grad(s):
    rstd = s["rstd"][:, None]
    n = s["h"].float() * rstd
    dy = s["dy"].float()
    a = dy * s["weight"]
    dx = rstd * (a - n * (a * n).mean(1, keepdim=True))
    if s["dh_in"] is not None:
        dx = dx + s["dh_in"].float()
    return dict(dx=dx.to(s["h"].dtype), dweight=(dy * n).sum(0))


def _plain_weight_grad(s):
    g = s["dy"].float().t() @ _restore(s["q"], s["scales"])
    if not s["accumulate"]:
        return g.to(DTYPES[s["grad"]])
    return s["buffer"].copy_(g.add_(s["buffer"].float()))


# ---------------------------------------------------------------------------- the library's calls

def _own(s):
    import newton_schulz_13_b200 as ns
    op = s["op"]
    if op == "embedding":
        return ns.embedding(s["tokens"], s["table"], scale=s["scale"], out_dtype=DTYPES[s["out"]])
    if op == "embedding_grad":
        if s["accumulate"]:
            return ns.embedding_grad(s["tokens"], s["dy"], s["vocab"], scale=s["scale"], grad=s["buffer"], accumulate=True)
        return ns.embedding_grad(s["tokens"], s["dy"], s["vocab"], scale=s["scale"], grad_dtype=DTYPES[s["grad"]])
    if op == "norm":
        r = ns.rms_norm(s["x"], s["weight"], residual=s["r"], eps=1e-5, output=s["y"], checkpoint=s["checkpoint"])
        q, scales = r.checkpoint if s["checkpoint"] else (None, None)
        return dict(h=r.h, rstd=r.rstd, y=r.y, q=q, scales=scales)
    if op == "norm_grad":
        dx, dweight = ns.rms_norm_grad(s["dy"], s["h"], s["weight"], s["rstd"], dh=s["dh_in"])
        return dict(dx=dx, dweight=dweight)
    if op == "checkpoint":
        ck = ns.checkpoint_store(s["x"])
        return dict(q=ck.q, scales=ck.scales, x=ns.checkpoint_restore(ck, dtype=torch.bfloat16))
    ck = ns.ActCheckpoint(s["q"], s["scales"])
    if s["accumulate"]:
        return ns.weight_grad(s["dy"], ck, grad=s["buffer"], accumulate=True)
    return ns.weight_grad(s["dy"], ck, grad_dtype=DTYPES[s["grad"]])


def run(state):
    s = state
    if own:
        return _own(s)
    op = s["op"]
    if op == "embedding":
        return _plain_embedding(s)
    if op == "embedding_grad":
        return _plain_embedding_grad(s)
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_grad":
        return _plain_norm_grad(s)
    if op == "checkpoint":
        q, scales = _quantise(s["x"])
        return dict(q=q, scales=scales, x=_restore(q, scales).to(torch.bfloat16))
    return _plain_weight_grad(s)


# ---------------------------------------------------------------------------- what a pass cannot do without

def _distinct(n, vocab):
    """How many different ids n draws of prepare() hold on average."""
    edges = torch.log1p(torch.arange(vocab + 1, dtype=torch.float64)) / math.log(vocab + 1.0)
    p = edges[1:] - edges[:-1]
    return float((1.0 - torch.exp(n * torch.log1p(-p.clamp(max=1 - 1e-12)))).sum())


def work(case):
    c, op = case, case["op"]
    if op in ("embedding", "embedding_grad"):
        n, dim, ids = c["n"], c["dim"], 4 if c["ids"] == "int32" else 8
        valid = n - n // 64 if n > 64 else n
        used = min(valid, _distinct(valid, c["vocab"]))
        if op == "embedding":
            return dict(bytes=n * ids + used * dim * SIZE[c["table"]] + n * dim * SIZE[c["out"]], flops=n * dim)
        out = 2 * used if c["accumulate"] else c["vocab"]
        return dict(bytes=n * ids + valid * dim * SIZE[c["dy"]] + out * dim * SIZE[c["grad"]], flops=valid * dim)
    if op in ("norm", "norm_grad", "checkpoint"):
        t, d = c["rows"], c["dim"]
        e, packed = SIZE[c["x"]], 1 + 1 / BLOCK
        if op == "checkpoint":
            return dict(bytes=t * d * (e + packed + 2), flops=4 * t * d)
        if op == "norm":
            each = e + (2 * e if c["residual"] else 0) + (e if c["y"] else 0) + (packed if c["checkpoint"] else 0)
            return dict(bytes=t * d * each + 4 * d + 4 * t, flops=5 * t * d)
        return dict(bytes=t * d * (4 if c["dh"] else 3) * e + 8 * d + 4 * t, flops=10 * t * d)
    t, n, k = c["rows"], c["n"], c["k"]
    return dict(bytes=t * n * SIZE[c["dy"]] + t * k * (1 + 1 / BLOCK) + n * k * SIZE[c["grad"]] * (2 if c["accumulate"] else 1), flops=2.0 * t * n * k)


# ---------------------------------------------------------------------------- the definitions in 64 bits

def _exact_scale(y):
    """2^e of each block of y and of each of its elements, from the definition of e."""
    rows, dim = y.shape
    blocks = -(-dim // BLOCK)
    big = torch.zeros((rows, blocks * BLOCK), dtype=torch.float64, device=y.device)
    big[:, :dim] = y.abs()
    big = big.view(rows, blocks, BLOCK).max(dim=2).values
    part, e = torch.frexp(big / E4M3_MAX)                 # big / 448 = part 2^e with part in [1/2, 1)
    e = torch.where(part == 0.5, e - 1, e).clamp(E_LO, E_HI)
    s = torch.ldexp(torch.ones_like(big), e)
    return s, s[:, torch.arange(dim, device=y.device) // BLOCK]


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f64 = torch.float64
    if op == "embedding":
        rows = torch.zeros((case["n"], case["dim"]), dtype=f64, device="cuda")
        at = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["vocab"]))[:, 0]
        rows[at] = torch.index_select(s["table"], 0, s["tokens"][at].long()).to(f64)
        return rows * case["scale"]
    if op == "embedding_grad":
        at = torch.nonzero((s["tokens"] >= 0) & (s["tokens"] < case["vocab"]))[:, 0]
        ids, place = torch.unique(s["tokens"][at].long(), return_inverse=True)
        sums = torch.zeros((ids.numel(), case["dim"]), dtype=f64, device="cuda")
        sums.scatter_add_(0, place[:, None].expand(-1, case["dim"]), s["dy"][at].to(f64))
        g = s["buffer"].to(f64) if case["accumulate"] else torch.zeros((case["vocab"], case["dim"]), dtype=f64, device="cuda")
        g[ids] += case["scale"] * sums
        return g
    if op == "norm":
        h = s["x"].to(f64)
        if s["r"] is not None:
            h = (h + s["r"].to(f64)).to(s["x"].dtype).to(f64)   # the residual stream's own rounding
        rms = torch.sqrt((torch.linalg.vector_norm(h, dim=1) ** 2) / case["dim"] + 1e-5)
        y = h / rms[:, None] * s["weight"].to(f64)
        scale, each = _exact_scale(y) if case["checkpoint"] else (None, 1.0)
        return dict(h=h, rstd=1.0 / rms, y=y if case["y"] else None, q=y / each if case["checkpoint"] else None, scales=scale)
    if op == "norm_grad":
        r, w, dy = s["rstd"].to(f64), s["weight"].to(f64), s["dy"].to(f64)
        n = torch.einsum("td,t->td", s["h"].to(f64), r)
        inner = torch.einsum("td,td,d->t", dy, n, w) / case["dim"]
        dx = torch.einsum("td,d,t->td", dy, w, r) - torch.einsum("td,t,t->td", n, inner, r)
        return dict(dx=dx + (s["dh_in"].to(f64) if s["dh_in"] is not None else 0.0), dweight=torch.einsum("td,td->d", dy, n))
    if op == "checkpoint":
        x = s["x"].to(f64)
        scale, each = _exact_scale(x)
        q = x / each
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)   # 3 bits after the first
        q = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        return dict(q=q, scales=scale, x=q * each)
    x = s["q"].to(f64) * s["scales"].to(f64)[:, torch.arange(case["k"], device="cuda") // BLOCK]
    g = torch.einsum("tn,tk->nk", s["dy"].to(f64), x)
    return g + s["buffer"].to(f64) if case["accumulate"] else g
