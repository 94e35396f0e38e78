"""The operators that make the optimizer's gradients, against their formulas in 64 bits.

Tolerances count roundings, element by element: u(t) = eps(t) / 2 for the rounding of a result to
its type, and 2^-24 of the sum of the magnitudes for every fp32 addition on the longest path of a
sum (the bounds below take the number of terms, which no path exceeds)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, FP32: 2.0 ** -24}
E = 2.0 ** -24
DTS = [BF16, FP32]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(shape, dtype, seed, std=1.0, lo=0.1, hi=10.0):
    g = gen(seed)
    x = torch.randn(shape, generator=g, device="cuda") * std
    if len(shape) > 1:
        x = x * torch.exp(torch.rand(shape[-1], generator=g, device="cuda") * math.log(hi / lo) + math.log(lo))
    return x.to(dtype)


def strided(x, extra=0, offset=0):
    """The same values in a wider buffer: rows `extra` longer, beginning `offset` elements in."""
    rows, cols = x.shape
    buf = torch.full((rows * (cols + extra) + offset + 64,), float("nan"), dtype=x.dtype, device="cuda")
    v = buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
    v.copy_(x)
    return v


def within(got, want, tol, what=""):
    got = got.double()
    bad = ~((got - want).abs() <= tol) & ~(torch.isnan(got) & torch.isnan(want)) & (got != want)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first at {torch.nonzero(bad)[0].tolist()}, " \
        f"got {got[bad][0].item()}, want {want[bad][0].item()}"


class Guarded:
    """A buffer whose surroundings must not be written: `view` is a matrix within it."""

    def __init__(self, rows, cols, dtype, extra=0, offset=0, fill=7.0):
        self.buf = torch.full((offset + rows * (cols + extra) + 64,), fill, dtype=dtype, device="cuda")
        self.view = self.buf[offset:offset + rows * (cols + extra)].view(rows, cols + extra)[:, :cols]
        self.before = self.buf.clone()

    def check(self):
        mine = self.view.clone()
        self.view.copy_(torch.as_strided(self.before, self.view.shape, self.view.stride(), self.view.storage_offset()))
        same = torch.equal(self.buf.view(torch.uint8), self.before.view(torch.uint8))
        self.view.copy_(mine)
        assert same, "written outside the buffer"


# ---------------------------------------------------------------------------- embedding

EMBED = [(0, 50, 64), (1, 1, 1), (1, 128, 4096), (7, 1000, 33), (31, 5, 8), (33, 5, 768), (64, 1, 40), (1000, 300, 520),
         (4097, 50257, 96), (2500, 2049, 1536), (3000, 70000, 17)]


def tokens_of(n, vocab, seed, dtype):
    g = gen(seed)
    ids = (torch.exp(torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(vocab + 1.0)) - 1).long()
    ids.clamp_(0, vocab - 1)
    if n > 5:
        ids[torch.randint(n, (max(1, n // 20),), generator=g, device="cuda")] = -1
    return ids.to(dtype)


@pytest.mark.parametrize("table_dt", DTS)
@pytest.mark.parametrize("out_dt", DTS)
@pytest.mark.parametrize("n,vocab,dim", EMBED)
def test_embedding(n, vocab, dim, out_dt, table_dt):
    import newton_schulz_13_b200 as ns
    for ids_dt, extra, offset in ((torch.int64, 0, 0), (torch.int32, 8, 8), (torch.int64, 3, 1)):
        t = tokens_of(n, vocab, 3, ids_dt)
        table = strided(normal((vocab, dim), table_dt, 4, 0.02), extra, offset)
        scale = math.sqrt(dim)
        out = Guarded(n, dim, out_dt, extra, offset)
        got = ns.embedding(t, table, scale=scale, out=out.view)
        want = torch.where((t >= 0)[:, None], table.double()[t.long().clamp(min=0)] * float(torch.tensor(scale)), 0.0)
        within(got, want, want.abs() * (U[out_dt] + 2 * E))
        out.check()
        assert torch.equal(ns.embedding(t, table, scale=scale, out_dtype=out_dt), got)
    assert ns.check_status() == ns.OK


def test_embedding_ids_outside_the_vocabulary():
    import newton_schulz_13_b200 as ns
    table = normal((10, 64), FP32, 1)
    dy = normal((6, 64), FP32, 2)
    dy[[1, 3, 4, 5]] = float("nan")     # places that select no row must not reach the gradient
    for dt in (torch.int32, torch.int64):
        t = torch.tensor([9, -1, 0, 10, -2 ** 31, 2 ** 31 - 1], device="cuda").to(dt)
        y = ns.embedding(t, table)
        assert torch.equal(y[[0, 2]], table[[9, 0]]) and not y[[1, 3, 4, 5]].any()
        assert ns.check_status() == ns.WARN_TOKEN
        assert ns.check_status() == ns.OK
        g = ns.embedding_grad(t, dy, 10)
        assert torch.equal(g[[9, 0]], dy[[0, 2]]) and not g[1:9].any()
        assert ns.check_status() == ns.WARN_TOKEN
    t = torch.tensor([2 ** 40, -2 ** 40, 2 ** 32, 3, -1, -1], device="cuda")
    dy = torch.ones(6, 64, device="cuda")
    assert ns.embedding_grad(t, dy, 10).sum() == 64 and ns.check_status() == ns.WARN_TOKEN
    t = torch.tensor([-1, -5], device="cuda")
    assert not ns.embedding(t, table).any() and ns.check_status() == ns.OK


def embed_grad_want(t, dy, vocab, scale, old):
    keep = t >= 0
    idx = t.long()[keep]
    g = torch.zeros((vocab, dy.shape[1]), dtype=torch.float64, device="cuda")
    a = g.clone()
    g.index_add_(0, idx, dy[keep].double())
    a.index_add_(0, idx, dy[keep].double().abs())
    cnt = torch.bincount(idx, minlength=vocab).double()[:, None]
    scale = float(torch.tensor(scale))
    want = scale * g + (0.0 if old is None else old.double())
    tol = (cnt + 3) * E * (abs(scale) * a + (0.0 if old is None else old.double().abs()))
    return want, tol


@pytest.mark.parametrize("dy_dt", DTS)
@pytest.mark.parametrize("grad_dt", DTS)
@pytest.mark.parametrize("n,vocab,dim", EMBED)
def test_embedding_grad(n, vocab, dim, grad_dt, dy_dt):
    import newton_schulz_13_b200 as ns
    for ids_dt, extra, offset, acc in ((torch.int64, 0, 0, False), (torch.int32, 8, 8, True), (torch.int64, 3, 1, False),
                                       (torch.int32, 0, 0, True)):
        t = tokens_of(n, vocab, 5, ids_dt)
        dy = strided(normal((n, dim), dy_dt, 6, 1e-3), extra, offset)
        out = Guarded(vocab, dim, grad_dt, extra, offset)
        old = None
        if acc:
            old = normal((vocab, dim), grad_dt, 7, 1e-3)
            out.view.copy_(old)
        got = ns.embedding_grad(t, dy, vocab, scale=1.7, grad=out.view, accumulate=acc)
        want, tol = embed_grad_want(t, dy, vocab, 1.7, old)
        within(got, want, tol + U[grad_dt] * want.abs())
        out.check()
        if not acc:
            assert torch.equal(ns.embedding_grad(t, dy, vocab, scale=1.7, grad_dtype=grad_dt), got)
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("kind", ["one token", "two tokens", "runs of 33", "sorted down", "last id"])
def test_embedding_grad_long_runs(kind):
    """Runs of one token over many chunks, chunk borders on run borders, and every order of ids."""
    import newton_schulz_13_b200 as ns
    n, vocab, dim = 5000, 700, 72
    i = torch.arange(n, device="cuda")
    t = {"one token": i * 0 + 3, "two tokens": i % 2 * 699, "runs of 33": i // 33, "sorted down": 699 - i * 700 // n,
         "last id": i * 0 + 699}[kind]
    dy = normal((n, dim), FP32, 8)
    want, tol = embed_grad_want(t, dy, vocab, 1.0, None)
    first = ns.embedding_grad(t, dy, vocab)
    within(first, want, tol + E * want.abs())
    for _ in range(3):
        assert torch.equal(ns.embedding_grad(t, dy, vocab), first)     # one order of summation


def test_embedding_grad_many_ids():
    """More ids than one range per SM holds."""
    import newton_schulz_13_b200 as ns
    vocab = 400_000
    t = tokens_of(2000, vocab, 9, torch.int64)
    t[:4] = torch.tensor([vocab - 1, 0, vocab - 1, 1024], device="cuda")
    dy = normal((2000, 8), FP32, 10)
    want, tol = embed_grad_want(t, dy, vocab, 1.0, None)
    within(ns.embedding_grad(t, dy, vocab), want, tol + E * want.abs())


def test_embedding_grad_against_differences():
    """<dE, D> is the change of <dy, embedding(E)> along D (the operator is linear in E)."""
    import newton_schulz_13_b200 as ns
    t = tokens_of(200, 40, 11, torch.int64)
    table, d, dy = normal((40, 64), FP32, 12), normal((40, 64), FP32, 13), normal((200, 64), FP32, 14)
    f = lambda e: (ns.embedding(t, e, scale=3.0).double() * dy.double()).sum().item()  # noqa: E731
    g = ns.embedding_grad(t, dy, 40, scale=3.0).double()
    want = f(table + d) - f(table - d)
    terms = (ns.embedding(t, table.abs() + d.abs(), scale=3.0).double() * dy.double().abs()).sum().item()
    assert abs(2 * (g * d.double()).sum().item() - want) <= 210 * E * 2 * terms


# ---------------------------------------------------------------------------- 8-bit checkpoints

def mx_reference(x):
    """Codes and scales by the definition, in 64 bits."""
    x = x.double()
    rows, dim = x.shape
    nb = -(-dim // 32)
    v = torch.zeros((rows, nb * 32), dtype=torch.float64, device=x.device)
    v[:, :dim] = x
    v = v.view(rows, nb, 32)
    bad = ~torch.isfinite(v).all(2)
    v = torch.where(bad[:, :, None], 0.0, v)
    m, e = torch.frexp(v.abs().amax(2) / 448.0)
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(v.abs().amax(2) == 0, -117, e).clamp(-117, 119)
    q = torch.ldexp(v, -e[:, :, None]).clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(q / step) * step
    scale = torch.where(bad, float("nan"), torch.ldexp(torch.ones_like(m), e))
    q = torch.where(bad[:, :, None], float("nan"), q)
    return q.view(rows, nb * 32)[:, :dim], scale, bad


MX = [(0, 64), (1, 1), (1, 32), (3, 33), (5, 31), (17, 48), (64, 1536), (1023, 100), (130, 4096), (9, 14336), (2, 2047)]


@pytest.mark.parametrize("dtype", DTS)
@pytest.mark.parametrize("rows,dim", MX)
def test_checkpoint(rows, dim, dtype):
    import newton_schulz_13_b200 as ns
    for extra, offset in ((0, 0), (16, 16), (1, 1)):
        x = strided(normal((rows, dim), dtype, 20, 1.0, 1e-4, 1e3), extra, offset)
        q8 = Guarded(rows, dim, torch.uint8, extra, offset, 9)
        s8 = Guarded(rows, -(-dim // 32), torch.uint8, extra, offset, 9)
        out = ns.ActCheckpoint(q8.view.view(torch.float8_e4m3fn), s8.view.view(torch.float8_e8m0fnu))
        ck = ns.checkpoint_store(x, out=out)
        q8.check()
        s8.check()
        q, scale, _ = mx_reference(x)
        assert torch.equal(ck.q.double(), q) and torch.equal(ck.scales.double(), scale)
        for dt in DTS:
            back = Guarded(rows, dim, dt, extra, offset)
            got = ns.checkpoint_restore(ck, out=back.view)
            assert torch.equal(got.double(), q * scale.repeat_interleave(32, 1)[:, :dim])
            back.check()
        own = ns.checkpoint_store(x)
        assert torch.equal(own.q.view(torch.uint8), ck.q.view(torch.uint8))
        assert torch.equal(own.scales.view(torch.uint8), ck.scales.view(torch.uint8))


@pytest.mark.parametrize("dim", [96, 70])
def test_checkpoint_edge_values(dim):
    """Zeros, the largest and smallest numbers, values at a scale's border, ties, infinities, NaN."""
    import newton_schulz_13_b200 as ns
    for dtype in DTS:
        big = torch.finfo(dtype).max
        rows = [0.0, -0.0, big, -big, 2.0 ** -126, 2.0 ** -133, 2.0 ** -149, 448.0, 449.0, 452.0, 1.75 * 2 ** -60,
                3.5e38 if dtype == BF16 else 3.4e38, 2.0 ** -108, 2.0 ** -117, float("inf"), -float("inf"), float("nan")]
        x = torch.zeros((len(rows), dim), device="cuda")
        x[:, 33] = torch.tensor(rows, device="cuda")
        x[:, 34] = x[:, 33] * 0.0410      # lands between codes
        x[:, 35] = x[:, 33] * (1.0625 / 1.75)   # a tie under the scale of a 1.75 2^k maximum
        x = x.to(dtype)
        q, scale, bad = mx_reference(x)
        ck = ns.checkpoint_store(x)
        got_q, got_s = ck.q.double(), ck.scales.double()
        assert torch.equal(torch.isnan(got_s), bad)
        assert torch.equal(got_s[~bad], scale[~bad])
        assert torch.equal(torch.nan_to_num(got_q, nan=1e9), torch.nan_to_num(q, nan=1e9))
        for dt in DTS:
            r = ns.checkpoint_restore(ck, dtype=dt).double()
            w = q * scale.repeat_interleave(32, 1)[:, :dim]
            assert torch.equal(torch.nan_to_num(r, nan=1e9), torch.nan_to_num(w, nan=1e9))
            assert torch.isfinite(r[~bad.any(1)]).all()     # 3.5e38 is an infinity already in fp32


# ---------------------------------------------------------------------------- RMS norm

NORM = [(0, 64), (1, 1), (1, 4096), (3, 7), (5, 64), (33, 768), (130, 1537), (300, 2048), (17, 4096), (2, 8192), (3, 8200),
        (2, 14336), (4, 16391), (2, 32768), (2, 32767)]
SUM = 256        # additions on the longest path of a row sum: at most 32 per thread, then two warp trees


def norm_want(x, r, w, eps):
    h = x if r is None else (x.float() + r.float()).to(r.dtype)
    d = h.double()
    rstd = 1.0 / torch.sqrt((d * d).mean(1) + float(torch.tensor(eps)))
    return h, rstd, d * rstd[:, None] * w.double()


@pytest.mark.parametrize("x_dt", DTS)
@pytest.mark.parametrize("r_dt", [None, BF16, FP32])
@pytest.mark.parametrize("rows,dim", NORM)
def test_rms_norm(rows, dim, r_dt, x_dt):
    import newton_schulz_13_b200 as ns
    for extra, offset, w_dt, output, ckpt in ((0, 0, FP32, True, True), (8, 8, BF16, True, False), (1, 3, FP32, True, True),
                                              (0, 0, FP32, False, True)):
        x = strided(normal((rows, dim), x_dt, 30), extra, offset)
        r = None if r_dt is None else strided(normal((rows, dim), r_dt, 31, 2.0), extra, offset)
        w = (1.0 + 0.1 * torch.randn(dim, generator=gen(32), device="cuda")).to(w_dt)
        y = Guarded(rows, dim, x_dt, extra, offset) if output else None
        h = Guarded(rows, dim, r_dt, extra, offset) if r is not None else None
        got = ns.rms_norm(x, w, residual=r, eps=1e-5, output=output, checkpoint=ckpt, y=y.view if y else None,
                          h=h.view if h else None)
        want_h, want_rstd, want = norm_want(x, r, w, 1e-5)
        assert torch.equal(got.h, want_h)
        within(got.rstd, want_rstd, want_rstd * SUM * E, "rstd")
        if output:
            within(got.y, want, want.abs() * (SUM * E + U[x_dt]), "y")
            y.check()
        else:
            assert got.y is None
        if h:
            h.check()
        if ckpt:
            back = ns.checkpoint_restore(got.checkpoint, dtype=FP32)
            scale = got.checkpoint.scales.double()
            each = scale.repeat_interleave(32, 1)[:, :dim]
            within(back, want, want.abs() * (2.0 ** -4 + SUM * E) + each * 2.0 ** -10, "checkpoint")
            _, s, _ = mx_reference(want)
            differ = s != scale
            if differ.any():      # only where the block's largest value is at a scale's border
                nb = s.shape[1]
                v = torch.zeros((rows, nb * 32), dtype=torch.float64, device="cuda")
                v[:, :dim] = want.abs()
                top = (v.view(rows, nb, 32).amax(2) / torch.minimum(s, scale) / 448.0)[differ]
                assert ((top - 1).abs() <= 2 * SUM * E).all()
        else:
            assert got.checkpoint is None


def test_rms_norm_in_place_and_leading_dimensions():
    import newton_schulz_13_b200 as ns
    x, r = normal((2, 5, 64), BF16, 33), normal((2, 5, 64), BF16, 34)
    w = torch.ones(64, device="cuda")
    want = ns.rms_norm(x, w, residual=r, checkpoint=True)
    assert want.y.shape == (2, 5, 64) and want.rstd.shape == (2, 5) and want.checkpoint.scales.shape == (2, 5, 2)
    xi, ri = x.clone(), r.clone()
    got = ns.rms_norm(xi, w, residual=ri, h=ri, y=xi)
    assert got.h is ri and got.y is xi and torch.equal(ri, want.h) and torch.equal(xi, want.y)
    dy, dh = normal((2, 5, 64), BF16, 35), normal((2, 5, 64), BF16, 36)
    dx, dw = ns.rms_norm_grad(dy, want.h, w, want.rstd, dh=dh)
    for target in (0, 1, 2):
        a = [dy.clone(), want.h.clone(), dh.clone()]
        dx2, dw2 = ns.rms_norm_grad(a[0], a[1], w, want.rstd, dh=a[2], dx=a[target])
        assert dx2 is a[target] and torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_rms_norm_rows_of_zeros_infinities_and_nan():
    import newton_schulz_13_b200 as ns
    for dim in (128, 77):
        x = normal((5, dim), FP32, 37)
        x[1] = 0
        x[2, 5] = float("inf")
        x[3, 6] = float("nan")
        w = torch.ones(dim, device="cuda")
        got = ns.rms_norm(x, w, checkpoint=True)
        clean = x[[0, 1, 4]]
        ref = ns.rms_norm(clean, w, checkpoint=True)
        assert torch.equal(got.y[[0, 1, 4]], ref.y) and not got.y[1].any()
        assert torch.equal(got.checkpoint.q[[0, 1, 4]].view(torch.uint8), ref.checkpoint.q.view(torch.uint8))
        assert got.rstd[2] == 0 and torch.isnan(got.y[2, 5]) and not got.y[2, :5].any()
        assert torch.isnan(got.y[3]).all() and torch.isnan(got.checkpoint.scales[3].float()).all()
        got = ns.rms_norm(torch.zeros(2, dim, device="cuda"), w, eps=0.0)
        assert torch.isinf(got.rstd).all() and torch.isnan(got.y).all()


@pytest.mark.parametrize("dy_dt", DTS)
@pytest.mark.parametrize("h_dt", DTS)
@pytest.mark.parametrize("rows,dim", NORM + [(1500, 72), (2500, 33), (700, 1024)])
def test_rms_norm_grad(rows, dim, h_dt, dy_dt):
    import newton_schulz_13_b200 as ns
    for extra, offset, w_dt, with_dh, acc in ((0, 0, FP32, True, False), (8, 8, BF16, False, True), (1, 3, FP32, True, True)):
        h = strided(normal((rows, dim), h_dt, 40, 2.0), extra, offset)
        dy = strided(normal((rows, dim), dy_dt, 41, 1e-3), extra, offset)
        dh = strided(normal((rows, dim), h_dt, 42, 1e-3), extra, offset) if with_dh else None
        w = (1.0 + 0.1 * torch.randn(dim, generator=gen(43), device="cuda")).to(w_dt)
        rstd = (1.0 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
        old = normal((dim,), FP32, 44, 1e-2) if acc else None
        dx = Guarded(rows, dim, h_dt, extra, offset)
        dwb = Guarded(1, dim, FP32, 0, 1)
        dwv = dwb.view[0]
        if acc:
            dwv.copy_(old)
        got, dw = ns.rms_norm_grad(dy, h, w, rstd, dh=dh, dx=dx.view, dweight=dwv, accumulate=acc)
        r = rstd.double()[:, None]
        n, a = h.double() * r, dy.double() * w.double()
        want = r * (a - n * (a * n).mean(1, keepdim=True))
        mag = r * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True))
        if with_dh:
            want, mag = want + dh.double(), mag + dh.double().abs()
        within(got, want, SUM * E * mag + U[h_dt] * want.abs(), "dx")
        t = dy.double() * n
        want_w = t.sum(0) + (old.double() if acc else 0.0)
        within(dw, want_w, (rows + 8) * E * (t.abs().sum(0) + (old.double().abs() if acc else 0.0)), "dweight")
        dx.check()
        dwb.check()
        again, dw2 = ns.rms_norm_grad(dy, h, w, rstd, dh=dh)
        assert torch.equal(again, got)
        if not acc:
            assert torch.equal(dw2, dw)


def test_rms_norm_grad_against_differences():
    """The directional derivative of <dy, y> + <dh, h> by central differences in 64 bits of the
    formula, at fp32 inputs; the step's own error is of order step^2."""
    import newton_schulz_13_b200 as ns
    x, r, w = normal((20, 96), FP32, 50), normal((20, 96), FP32, 51), normal((96,), FP32, 52)
    dy, dh = normal((20, 96), FP32, 53), normal((20, 96), FP32, 54)
    d, dw_dir = normal((20, 96), FP32, 55, 1.0, 1.0, 1.0).double(), normal((96,), FP32, 56).double()
    fw = ns.rms_norm(x, w, residual=r, eps=1e-5)
    dx, dweight = ns.rms_norm_grad(dy, fw.h, w, fw.rstd, dh=dh)

    def f(h, weight):
        return (dy.double() * h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-5) * weight + dh.double() * h).sum().item()

    s, h0 = 1e-5, fw.h.double()
    num_x = (f(h0 + s * d, w.double()) - f(h0 - s * d, w.double())) / (2 * s)
    num_w = (f(h0, w.double() + s * dw_dir) - f(h0, w.double() - s * dw_dir)) / (2 * s)
    # fp32 gradients: SUM roundings of the terms; differences: 2^-52 of f's terms over the step
    mag = (dx.double().abs() * d.abs()).sum().item() + (dy.double().abs() * w.double().abs()).sum().item()
    assert abs((dx.double() * d).sum().item() - num_x) <= mag * (SUM * E + 2.0 ** -52 * 1920 / s)
    mag_w = (dweight.double().abs() * dw_dir.abs()).sum().item() + (dy.double().abs() * dw_dir.abs()).sum().item()
    assert abs((dweight.double() * dw_dir).sum().item() - num_w) <= mag_w * (SUM * E + 2.0 ** -52 * 1920 / s)


@pytest.mark.parametrize("rows,dim", [(4096, 4096), (9000, 520), (2000, 8192)])
def test_rms_norm_wait_limit(rows, dim):
    """With a limit of 1 ns a call either reports that a wait for a row ran out or, where every row
    was there in time, is right; the device stays usable."""
    import newton_schulz_13_b200 as ns
    x, r, w = normal((rows, dim), BF16, 57), normal((rows, dim), BF16, 58), torch.ones(dim, device="cuda")
    want = ns.rms_norm(x, w, residual=r, checkpoint=True)
    grad = ns.rms_norm_grad(x, want.h, w, want.rstd, dh=r)
    assert ns.check_status() == ns.OK
    out_of_cache = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for call, right in ((lambda: ns.rms_norm(x, w, residual=r, checkpoint=True)[:3], want[:3]),
                        (lambda: ns.rms_norm_grad(x, want.h, w, want.rstd, dh=r), grad)):
        for _ in range(5):
            out_of_cache.zero_()
            ns.set_wait_limit_ns(1)
            try:
                got = call()
                try:
                    assert ns.check_status() == ns.OK
                    assert all(torch.equal(a, b) for a, b in zip(got, right))
                    print("no wait ran out")
                except ns.MuonError as e:
                    assert e.code == ns.ERR_TIMEOUT
                    print("reported")
            finally:
                ns.set_wait_limit_ns(0)
    again = ns.rms_norm(x, w, residual=r, checkpoint=True)
    assert torch.equal(again.y, want.y) and torch.equal(again.checkpoint.q.view(torch.uint8), want.checkpoint.q.view(torch.uint8))
    assert all(torch.equal(a, b) for a, b in zip(ns.rms_norm_grad(x, want.h, w, want.rstd, dh=r), grad))
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("x_dt,r_dt", [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32), (BF16, None)])
@pytest.mark.parametrize("rows,dim", [(66000, 64), (17000, 264), (5462, 768), (1031, 4096), (600, 8192)])
def test_rms_norm_many_rows(rows, dim, x_dt, r_dt):
    """Sizes at which rows come through the ring, in shapes that leave its last groups idle."""
    import newton_schulz_13_b200 as ns
    x = normal((rows, dim), x_dt, 47)
    r = None if r_dt is None else normal((rows, dim), r_dt, 48, 2.0)
    w = 1.0 + 0.1 * torch.randn(dim, generator=gen(49), device="cuda")
    got = ns.rms_norm(strided(x, 8, 8), w, residual=r, eps=1e-5, checkpoint=True)
    want_h, want_rstd, want = norm_want(x, r, w, 1e-5)
    assert torch.equal(got.h, want_h)
    within(got.rstd, want_rstd, want_rstd * SUM * E, "rstd")
    within(got.y, want, want.abs() * (SUM * E + U[x_dt]), "y")
    back = ns.checkpoint_restore(got.checkpoint, dtype=FP32)
    each = got.checkpoint.scales.double().repeat_interleave(32, 1)[:, :dim]
    within(back, want, want.abs() * (2.0 ** -4 + SUM * E) + each * 2.0 ** -10, "checkpoint")
    xi, ri = x.clone(), None if r is None else r.clone()
    same = ns.rms_norm(xi, w, residual=ri, h=ri, y=xi, checkpoint=True)      # in place
    assert torch.equal(same.y, got.y) and (r is None or torch.equal(ri, got.h))
    assert ns.check_status() == ns.OK


# ---------------------------------------------------------------------------- weight gradient

WGRAD = [(0, 5, 40), (1, 1, 1), (1, 256, 256), (15, 48, 1536), (63, 80, 33), (64, 257, 300), (65, 256, 512), (130, 1536, 48),
         (1000, 300, 72), (1025, 80, 1536), (3001, 129, 264), (5000, 768, 768), (2048, 2304, 768)]


def wgrad_tol(dy, x, planes):
    """The tensor core adds 16 products at a time to a running sum that it truncates: 2^-22 of the
    magnitudes per step covers the alignment and truncation of its terms; a chunk has 64 steps, and
    chunks and parts add in fp32."""
    rows = dy.shape[0]
    steps = min(-(-rows * planes // 16), 64) + -(-rows * planes // 1024) + 70
    return steps * 2.0 ** -22 * (dy.double().abs().t() @ x.double().abs())


@pytest.mark.parametrize("grad_dt", DTS)
@pytest.mark.parametrize("dy_dt", DTS)
@pytest.mark.parametrize("rows,n,k", WGRAD)
def test_weight_grad(rows, n, k, dy_dt, grad_dt):
    import newton_schulz_13_b200 as ns
    for extra, offset, acc in ((0, 0, False), (16, 16, True), (1, 1, False), (3, 0, True)):
        x = normal((rows, k), FP32, 60)
        ck = ns.checkpoint_store(x)
        q = ck.q.view(torch.uint8)
        if extra:
            wide = torch.full((rows, k + extra), 255, dtype=torch.uint8, device="cuda")
            wide[:, :k] = q
            sc = torch.full((rows, ck.scales.shape[1] + 3), 255, dtype=torch.uint8, device="cuda")
            sc[:, :ck.scales.shape[1]] = ck.scales.view(torch.uint8)
            ck = ns.ActCheckpoint(wide[:, :k].view(torch.float8_e4m3fn), sc[:, :ck.scales.shape[1]].view(torch.float8_e8m0fnu))
        xr = ns.checkpoint_restore(ck, dtype=FP32)
        dy = strided(normal((rows, n), dy_dt, 61, 1e-3), extra, offset)
        out = Guarded(n, k, grad_dt, extra, offset)
        old = None
        if acc:
            old = normal((n, k), grad_dt, 62, 1e-2)
            out.view.copy_(old)
        got = ns.weight_grad(dy, ck, grad=out.view, accumulate=acc)
        want = dy.double().t() @ xr.double() + (old.double() if acc else 0.0)
        tol = wgrad_tol(dy, xr, 1 if dy_dt == BF16 else 3) + 2 * E * (old.double().abs() if acc else 0.0) + U[grad_dt] * want.abs()
        within(got, want, tol)
        out.check()
        if not acc:
            for _ in range(2):
                assert torch.equal(ns.weight_grad(dy, ck, grad_dtype=grad_dt), got)
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("shapes", [((8192, 768, 2304), (4096, 1536, 1536)), ((16384, 256, 256), (5000, 2304, 768))])
def test_weight_grad_joined_tiles_on_two_streams_and_in_graphs(shapes):
    """Calls whose tiles fall to several pairs, many at once on two streams, beside graphs of them:
    each gives what it gives alone."""
    import newton_schulz_13_b200 as ns
    sets = []
    for i, (rows, n, k) in enumerate(shapes):
        dy, ck = normal((rows, n), BF16, 140 + i), ns.checkpoint_store(normal((rows, k), BF16, 150 + i))
        sets.append((dy, ck, ns.weight_grad(dy, ck, grad_dtype=FP32)))
    graphs, outs = [], []
    for dy, ck, _ in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ns.weight_grad(dy, ck, grad_dtype=FP32))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for r in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(ns.weight_grad(sets[i][0], sets[i][1], grad_dtype=FP32))
                if r % 5 == 4:
                    graphs[i].replay()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(torch.equal(g, sets[i][2]) for g in got[i]) and torch.equal(outs[i], sets[i][2])
    assert ns.check_status() == ns.OK


def test_weight_grad_fp32_keeps_its_precision_over_many_rows():
    """The sum over 20,000 rows stays near fp32: 1e-5 of the norm is half of what fp32 outputs of
    such sums may be off by; the truncation of one long running sum would exceed it."""
    import newton_schulz_13_b200 as ns
    for dt in DTS:
        dy, x = normal((20000, 256), dt, 63, 1.0).abs(), normal((20000, 256), FP32, 64).abs()
        ck = ns.checkpoint_store(x)
        want = dy.double().t() @ ns.checkpoint_restore(ck, dtype=FP32).double()
        got = ns.weight_grad(dy, ck, grad_dtype=FP32).double()
        rel = ((got - want).norm() / want.norm()).item()
        print("relative error", rel)
        assert rel <= 1e-5


def test_weight_grad_infinities_and_nan():
    import newton_schulz_13_b200 as ns
    for dt in DTS:
        dy = normal((100, 70), dt, 65).abs() + 1
        x = normal((100, 96), FP32, 66).abs() + 1
        dy[7, 3] = float("inf")
        dy[9, 4] = float("nan")
        x[11, 40] = float("nan")        # its block of 32 becomes NaN
        g = ns.weight_grad(dy.to(dt), ns.checkpoint_store(x), grad_dtype=FP32)
        bad = torch.zeros(70, 96, dtype=torch.bool, device="cuda")
        bad[4] = True
        bad[:, 32:64] = True
        assert torch.equal(torch.isnan(g), bad)
        inf = torch.zeros_like(bad)
        inf[3] = True
        assert torch.equal(torch.isinf(g), inf & ~bad)
    # the largest finite fp32 values are not infinite in any of the three terms
    dy = torch.full((1, 8), torch.finfo(FP32).max, device="cuda")
    g = ns.weight_grad(dy, ns.checkpoint_store(torch.full((1, 32), 0.5, device="cuda")))
    assert torch.equal(g, torch.full((8, 32), torch.finfo(FP32).max / 2, device="cuda"))


def test_weight_grad_wait_limit():
    """A wait that runs out is reported, and the device stays usable."""
    import newton_schulz_13_b200 as ns
    dy, ck = normal((4096, 1024), BF16, 67), ns.checkpoint_store(normal((4096, 1024), BF16, 68))
    want = ns.weight_grad(dy, ck)
    assert ns.check_status() == ns.OK
    ns.set_wait_limit_ns(1)
    try:
        ns.weight_grad(dy, ck)
        with pytest.raises(ns.MuonError) as e:
            ns.check_status()
        assert e.value.code == ns.ERR_TIMEOUT
    finally:
        ns.set_wait_limit_ns(0)
    assert torch.equal(ns.weight_grad(dy, ck), want) and ns.check_status() == ns.OK


# ---------------------------------------------------------------------------- together

def _pass(ns, t, table, r, w, W, dh):
    """Embedding, norm with residual and checkpoint, a product, and every gradient."""
    x = ns.embedding(t, table, scale=4.0, out_dtype=BF16)
    f = ns.rms_norm(x, w, residual=r, checkpoint=True)
    out = f.y.float() @ W.t()
    d_out = (out * 1e-3).to(BF16)                       # the gradient of 5e-4 |out|^2
    dW = ns.weight_grad(d_out, f.checkpoint, grad_dtype=FP32)
    dy = (d_out.float() @ W).to(BF16)
    dx, dw = ns.rms_norm_grad(dy, f.h, w, f.rstd, dh=dh)
    dE = ns.embedding_grad(t, dx, table.shape[0], scale=4.0, grad_dtype=FP32)
    return dict(y=f.y, h=f.h, dW=dW, dx=dx, dw=dw, dE=dE, d_out=d_out, dy=dy)


def _inputs(seed, rows=300, vocab=500, dim=256, n=384):
    return (tokens_of(rows, vocab, seed, torch.int64), normal((vocab, dim), FP32, seed + 1, 0.02), normal((rows, dim), BF16, seed + 2),
            1.0 + 0.1 * normal((dim,), FP32, seed + 3), normal((n, dim), FP32, seed + 4, 0.02, 1.0, 1.0),
            normal((rows, dim), BF16, seed + 5, 1e-3))


def test_pass_and_optimizer_steps():
    """Forward and backward through the operators, then the steps that take their gradients: every
    gradient against 64 bits on the same intermediate values, and the steps against the oracle."""
    import numpy as np

    import newton_schulz_13_b200 as ns
    import oracle
    t, table, r, w, W, dh = _inputs(70)
    g = _pass(ns, t, table, r, w, W, dh)
    dim, vocab = 256, 500
    x = torch.where((t >= 0)[:, None], table.double()[t.clamp(min=0)] * 4.0, 0.0).to(BF16)
    h, rstd, y = norm_want(x, r, w, 1e-5)
    assert torch.equal(g["h"], h)
    # dW sees y through 8 bits: each value off by at most 2^-4 of itself or 2^-10 of its scale
    # (at most 2 max / 448), and by the norm's own roundings
    blocks = y.abs().view(300, dim // 32, 32).amax(2).repeat_interleave(32, 1)
    off = y.abs() * (2.0 ** -4 + SUM * E) + blocks * (2.0 / 448 * 2.0 ** -10)
    want_W = g["d_out"].double().t() @ y
    within(g["dW"], want_W, g["d_out"].double().abs().t() @ off + 100 * 2.0 ** -22 * (g["d_out"].double().abs().t() @ y.abs()))
    n, a, r64 = h.double() * rstd[:, None], g["dy"].double() * w.double(), rstd[:, None]
    want_x = r64 * (a - n * (a * n).mean(1, keepdim=True)) + dh.double()
    mag = r64 * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + dh.double().abs()
    within(g["dx"], want_x, 2 * SUM * E * mag + U[BF16] * want_x.abs())
    tt = g["dy"].double() * n
    within(g["dw"], tt.sum(0), (308 + SUM) * E * tt.abs().sum(0))
    want_E, tol = embed_grad_want(t, g["dx"], vocab, 4.0, None)
    within(g["dE"], want_E, tol + E * want_E.abs())

    W0, m = W.clone(), torch.zeros_like(W)
    ns.muon_step([W], [g["dW"]], [m], lr=0.02)
    ps, gs = [table, w], [g["dE"], g["dw"]]
    p0 = [p.double().cpu().numpy().ravel().copy() for p in ps]
    ms, vs = [torch.zeros_like(p) for p in ps], [torch.zeros_like(p) for p in ps]
    ns.adamw_step(ps, gs, ms, vs, step=1, lr=1e-3)
    assert ns.check_status() == ns.OK
    P, M = [W0.double().cpu().numpy()], [np.zeros(W.shape)]
    oracle.muon_step(P, [g["dW"].double().cpu().numpy()], M, lr=0.02, mu=0.95, nesterov=True, weight_decay=0.0, rms_mode=0,
                     coeffs=[ns.QUINTIC] * 5, zero_center=False, eps=1e-7, want_O=True)
    d_got, d_want = (W - W0).double().cpu().numpy(), P[0] - W0.double().cpu().numpy()
    assert np.linalg.norm(d_got - d_want) <= 3e-2 * np.linalg.norm(d_want)      # the step's bf16 tolerance
    o_m, o_v = [np.zeros(p.size) for p in p0], [np.zeros(p.size) for p in p0]
    oracle.adamw_step(p0, [x.double().cpu().numpy().ravel() for x in gs], o_m, o_v, step=1, lr=1e-3, beta1=0.9, beta2=0.95,
                      eps=1e-8, weight_decay=0.0)
    for p, want in zip(ps, p0):
        assert np.linalg.norm(p.double().cpu().numpy().ravel() - want) <= 1e-5 * np.linalg.norm(want)


def test_graphs_and_streams():
    """Two captured passes and eager ones, replayed in turn and on two streams at once: each gives
    what it gives alone."""
    import newton_schulz_13_b200 as ns
    sets = [_inputs(80), _inputs(90, rows=700, vocab=900, dim=520, n=200)]
    names = ("h", "dW", "dx", "dw", "dE")
    want = [{k: v.clone() for k, v in _pass(ns, *s).items()} for s in sets]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, st in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(_pass(ns, *s))
        graphs.append(g)
    for order in ([0, 1], [1, 0, 0], [0, 1, 1]):
        for i in order:
            graphs[i].replay()
            eager = _pass(ns, *sets[1 - i])
            torch.cuda.synchronize()
            for k in names:
                assert torch.equal(outs[i][k], want[i][k]), (order, i, k)
                assert torch.equal(eager[k], want[1 - i][k]), (order, i, k)
    # new inputs in the captured buffers
    fresh = _inputs(100)
    for a, b in zip(sets[0], fresh):
        a.copy_(b)
    graphs[0].replay()
    torch.cuda.synchronize()
    ref = _pass(ns, *fresh)
    for k in names:
        assert torch.equal(outs[0][k], ref[k]), k
    # eager calls on two streams at once
    got = [None, None]
    sets[0] = _inputs(80)
    torch.cuda.synchronize()
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _pass(ns, *sets[i])
        torch.cuda.synchronize()
        for i in (0, 1):
            for k in names:
                assert torch.equal(got[i][k], want[i][k]), (i, k)
    # the stream argument
    ev = torch.cuda.Event()
    t, table, r, w, W, dh = sets[0]
    y = ns.embedding(t, table, scale=4.0, out_dtype=BF16, stream=streams[0])
    ev.record(streams[0])
    torch.cuda.current_stream().wait_event(ev)
    assert torch.equal(y, ns.embedding(t, table, scale=4.0, out_dtype=BF16))
    f = ns.rms_norm(y, w, residual=r, checkpoint=True, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(f.h, want[0]["h"])
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("dim", [4096, 4095])
def test_offsets_past_32_bits(dim):
    """Matrices of over 2^31 elements: their last rows give what those rows give alone."""
    import newton_schulz_13_b200 as ns
    rows, tail = 530_000, 40
    last = normal((tail, dim), BF16, 130)
    x = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    x[-tail:] = last
    assert x.numel() > 1 << 31
    w = torch.ones(dim, device="cuda")
    ck, ref = ns.checkpoint_store(x), ns.checkpoint_store(last)
    assert torch.equal(ck.q[-tail:].view(torch.uint8), ref.q.view(torch.uint8))
    assert torch.equal(ck.scales[-tail:].view(torch.uint8), ref.scales.view(torch.uint8))
    back = ns.checkpoint_restore(ck)
    assert torch.equal(back[-tail:], ns.checkpoint_restore(ref)) and not back[:-tail].any()
    del back
    f, g = ns.rms_norm(x, w, checkpoint=True), ns.rms_norm(last, w, checkpoint=True)
    each = U[BF16] + SUM * E     # the two may take different kernels: the orders of their sums differ
    within(f.y[-tail:], g.y.double(), 2 * each * g.y.double().abs())
    assert not f.y[:-tail].any()
    dx, dw = ns.rms_norm_grad(x, x, w, f.rstd)
    want, want_w = ns.rms_norm_grad(last, last, w, f.rstd[-tail:])
    assert torch.equal(dx[-tail:], want) and not dx[:-tail].any()
    terms = (last.double() ** 2 * f.rstd[-tail:].double()[:, None]).sum(0)
    within(dw, want_w.double(), 2 * (tail + 8) * E * terms)
    del f, dx
    t = torch.arange(rows - tail, rows, device="cuda")
    assert torch.equal(ns.embedding(t, x), last)
    grad = ns.embedding_grad(t, last, rows)
    assert torch.equal(grad[-tail:], last) and not grad[:-tail].any()
    grad = ns.embedding_grad(t, last, rows, grad=grad, accumulate=True)
    assert torch.equal(grad[-tail:].float(), 2 * last.float())
    del grad
    # a checkpoint of ones: sums of ones are exact
    ones = ns.checkpoint_store(x.fill_(1.0))
    dy = torch.ones(rows, 8, dtype=BF16, device="cuda")
    assert torch.equal(ns.weight_grad(dy, ones, grad_dtype=FP32), torch.full((8, dim), float(rows), device="cuda"))
    assert ns.check_status() == ns.OK


def test_plain_calls_and_full_path_agree(monkeypatch):
    """Calls that take the extension's path give what the path through ctypes gives."""
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    from newton_schulz_13_b200 import gradients
    assert gradients._fast is not None
    x, r, w = normal((3, 50, 72), BF16, 120), normal((3, 50, 72), FP32, 121), normal((72,), FP32, 122)
    t = tokens_of(150, 40, 123, torch.int32).view(3, 50)
    table, dy = normal((40, 72), FP32, 124), normal((3, 50, 24), FP32, 125)
    ck = ns.checkpoint_store(x)
    buf_e, buf_w = normal((40, 72), FP32, 126), normal((24, 72), FP32, 127)
    f = ns.rms_norm(x, w, residual=r)
    calls = [
        lambda: [ns.embedding(t, table), ns.embedding(t, table, scale=2, out_dtype=BF16)],
        lambda: [ns.embedding_grad(t, x, 40), ns.embedding_grad(t, x, 40, scale=0.5, grad_dtype=FP32),
                 ns.embedding_grad(t, x, 40, grad=buf_e.clone(), accumulate=True), ns.embedding_grad(t, x, 40, grad=buf_e.clone())],
        lambda: [*ns.rms_norm(x, w)[:3], *ns.rms_norm(x, w, residual=r, eps=0.1)[:3]],
        lambda: [*ns.rms_norm(x, w, residual=r, checkpoint=True, output=False).checkpoint, *ns.rms_norm(r, w.to(BF16), checkpoint=True).checkpoint],
        lambda: [*ns.rms_norm_grad(x, f.h, w, f.rstd), *ns.rms_norm_grad(x, f.h, w, f.rstd, dh=r)],
        lambda: [*ns.checkpoint_store(x), *ns.checkpoint_store(r), ns.checkpoint_restore(ck), ns.checkpoint_restore(ck, dtype=FP32)],
        lambda: [ns.weight_grad(dy, ck), ns.weight_grad(dy.to(BF16), ck, grad_dtype=FP32),
                 ns.weight_grad(dy, ck, grad=buf_w.clone(), accumulate=True)],
        lambda: [ns.embedding(t[0, 0], table), ns.embedding(t[:0], table), *ns.checkpoint_store(x[:0]), *ns.rms_norm(x[:0], w)[:3]],
    ]
    for i, call in enumerate(calls):
        fast = call()
        with monkeypatch.context() as m:
            m.setattr(gradients, "_fast", None)
            full = call()
        for k, (a, b) in enumerate(zip(fast, full)):
            assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride(), (i, k)
            assert torch.equal(a.contiguous().view(torch.uint8) if a.dim() else a, b.contiguous().view(torch.uint8) if b.dim() else b), (i, k)
    assert ns.check_status() == ns.OK


def test_refusals_of_layouts_and_types():
    import newton_schulz_13_b200 as ns
    x = normal((6, 64), BF16, 110)
    w = torch.ones(64, device="cuda")
    t = torch.arange(6, device="cuda")
    ck = ns.checkpoint_store(x)
    f = ns.rms_norm(x, w)
    bad = [
        (ValueError, lambda: ns.rms_norm(x.t(), w)),
        (ValueError, lambda: ns.rms_norm(x, w[:32])),
        (ValueError, lambda: ns.rms_norm(x, w, residual=x[:3])),
        (ValueError, lambda: ns.rms_norm(x.cpu(), w)),
        (ValueError, lambda: ns.rms_norm(x, w.cpu())),
        (TypeError, lambda: ns.rms_norm(x.half(), w)),
        (TypeError, lambda: ns.rms_norm(x, w, y=x.float())),
        (TypeError, lambda: ns.rms_norm(x, w, residual=x, h=x.float())),
        (ValueError, lambda: ns.rms_norm(x, w, h=x)),
        (ValueError, lambda: ns.rms_norm(x, w, output=False)),
        (ns.MuonError, lambda: ns.rms_norm(x, w, eps=-1.0)),
        (ns.MuonError, lambda: ns.rms_norm(x, w, y=torch.as_strided(x, (6, 64), (60, 1)))),
        (ns.MuonError, lambda: ns.rms_norm(torch.zeros(1, 32769, device="cuda"), torch.ones(32769, device="cuda"))),
        (ValueError, lambda: ns.rms_norm_grad(x, f.h, w, f.rstd[:3])),
        (ValueError, lambda: ns.rms_norm_grad(x, f.h, w, f.rstd.double())),
        (ValueError, lambda: ns.rms_norm_grad(x, f.h, w, f.rstd, accumulate=True)),
        (TypeError, lambda: ns.rms_norm_grad(x, f.h, w, f.rstd, dh=x.float())),
        (TypeError, lambda: ns.rms_norm_grad(x, f.h, w, f.rstd, dx=x.float())),
        (TypeError, lambda: ns.rms_norm_grad(x, f.h, w, f.rstd, dweight=w.double())),
        (ValueError, lambda: ns.embedding(t[::2], x)),
        (TypeError, lambda: ns.embedding(t.float(), x)),
        (TypeError, lambda: ns.embedding(t, x.half())),
        (ValueError, lambda: ns.embedding(t, x[0])),
        (ns.MuonError, lambda: ns.embedding(t, x, scale=float("nan"))),
        (ns.MuonError, lambda: ns.embedding(t, x, out=x)),
        (ValueError, lambda: ns.embedding(t, x, out=torch.empty(5, 64, device="cuda"))),
        (ValueError, lambda: ns.embedding_grad(t, x[:5], 10)),
        (ValueError, lambda: ns.embedding_grad(t, x, 10, accumulate=True)),
        (ValueError, lambda: ns.embedding_grad(t, x, 10, grad=torch.empty(9, 64, device="cuda"))),
        (ns.MuonError, lambda: ns.embedding_grad(t, x, 0)),
        (ns.MuonError, lambda: ns.embedding_grad(t, x, 6, grad=x)),
        (TypeError, lambda: ns.embedding_grad(t, x, 10, grad_dtype=torch.float16)),
        (TypeError, lambda: ns.checkpoint_restore(ns.ActCheckpoint(ck.q, ck.scales.view(torch.uint8)))),
        (TypeError, lambda: ns.checkpoint_restore(x)),
        (ValueError, lambda: ns.checkpoint_restore(ns.ActCheckpoint(ck.q, ck.scales[:, :1]))),
        (TypeError, lambda: ns.checkpoint_restore(ck, dtype=torch.float16)),
        (TypeError, lambda: ns.checkpoint_store(x.double())),
        (ValueError, lambda: ns.weight_grad(x[:5], ck)),
        (TypeError, lambda: ns.weight_grad(x.half(), ck)),
        (ValueError, lambda: ns.weight_grad(x, ck, accumulate=True)),
        (ValueError, lambda: ns.weight_grad(x, ck, grad=torch.empty(64, 32, device="cuda"))),
        (TypeError, lambda: ns.weight_grad(x, ck, grad=torch.empty(64, 64, device="cuda"), grad_dtype=BF16)),
    ]
    for i, (kind, call) in enumerate(bad):
        with pytest.raises(kind):
            call()
            pytest.fail(f"call {i} was accepted")
    # side by side in one buffer is not an overlap
    both = torch.empty(6, 128, dtype=BF16, device="cuda")
    both[:, :64] = x
    assert torch.equal(ns.rms_norm(both[:, :64], w, y=both[:, 64:]).y, f.y)
    assert ns.check_status() == ns.OK
