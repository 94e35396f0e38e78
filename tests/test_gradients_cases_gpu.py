"""The gradient-making operators on calls with a history or a size of their own: sums onto a large
gradient, several warnings at once, buffers given as outputs, many tiles, tokens and rows.

Tolerances as in test_gradients_gpu: roundings counted element by element."""
import pytest
import torch

from .test_gradients_gpu import (BF16, DTS, E, FP32, SUM, U, Guarded, embed_grad_want, gen, norm_want, normal, strided,
                                 tokens_of, wgrad_tol, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------- weight gradient

@pytest.mark.parametrize("dy_dt", DTS)
@pytest.mark.parametrize("rows,n,k", [(16384, 256, 256), (16384, 100, 333), (16384, 512, 9472), (700, 512, 9472)])
def test_weight_grad_onto_a_large_gradient(rows, n, k, dy_dt):
    """Sums whose parts are each below half a step of the old gradient, but not the whole: the old
    value enters once. Every sum is a multiple of 2^-36 (2^-33 for 700 rows) below 2^24 of them, so
    exact, and so is 1 + 2^-22; 700 rows: their sum is 0.68 of the step above 1, and rounds to it."""
    import newton_schulz_13_b200 as ns
    ck = ns.checkpoint_store(torch.ones(rows, k, dtype=BF16, device="cuda"))
    unit, want = (2.0 ** -36, 1 + 2.0 ** -22) if rows == 16384 else (2.0 ** -33, 1 + 2.0 ** -23)
    dy = torch.full((rows, n), unit, dtype=dy_dt, device="cuda")
    for extra in (0, 1):
        out = Guarded(n, k, FP32, extra, extra, fill=1.0)
        got = ns.weight_grad(dy, ck, grad=out.view, accumulate=True)
        assert torch.equal(got, torch.full((n, k), want, device="cuda")), got.double().sub(1).abs().max().item()
        out.check()
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("dy_dt", DTS)
@pytest.mark.parametrize("rows,n,k", [(300, 2304, 2304), (4000, 2304, 2304), (2100, 2305, 4200)])
def test_weight_grad_more_tiles_than_pairs(rows, n, k, dy_dt, acc):
    """Several tiles per pair, and whole tiles followed by dealt-out ones."""
    import newton_schulz_13_b200 as ns
    ck = ns.checkpoint_store(normal((rows, k), FP32, 160))
    xr = ns.checkpoint_restore(ck, dtype=FP32)
    dy = normal((rows, n), dy_dt, 161, 1e-3)
    for grad_dt, extra in ((FP32, 0), (BF16, 3)):
        out = Guarded(n, k, grad_dt, extra, extra)
        old = normal((n, k), grad_dt, 162, 1e-2)
        out.view.copy_(old)
        got = ns.weight_grad(dy, ck, grad=out.view, accumulate=acc)
        want = dy.double().t() @ xr.double() + (old.double() if acc else 0.0)
        tol = wgrad_tol(dy, xr, 1 if dy_dt == BF16 else 3) + (E * want.abs() if acc else 0.0) + U[grad_dt] * want.abs()
        within(got, want, tol)
        out.check()
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("e", [-100, -110, -111, -120, -126, -140, -149])
def test_weight_grad_of_small_fp32_values(e):
    """Three truncated terms of 8 bits hold a number from 2^-110 on; below, the third ends at 2^-133,
    bf16's smallest number. One row, so that nothing else is rounded (2^20 keeps the products normal)."""
    import newton_schulz_13_b200 as ns
    ck = ns.checkpoint_store(torch.full((1, 32), 2.0 ** 20, device="cuda"))
    m = torch.randint(1 << 23, 2 << 23, (1, 512), generator=gen(193), device="cuda").double()
    dy = (m * 2.0 ** (e - 23) * torch.where(m % 2 == 0, 1.0, -1.0)).float()
    got = ns.weight_grad(dy, ck).double() * 2.0 ** -20
    off = (got - dy.double().t()).abs().max().item()
    assert off == 0.0 if e >= -110 else off < 2.0 ** -133


# ---------------------------------------------------------------------------- status

def test_a_token_warning_hides_no_other():
    """A batch with an id past the vocabulary and a NaN in an update matrix: both are reported, the
    graver first, whichever came first; and a time limit that ran out does not take the warning along."""
    import newton_schulz_13_b200 as ns
    table = normal((10, 64), FP32, 163)
    past = torch.tensor([3, 10], device="cuda")

    def token(grad):
        if grad:
            ns.embedding_grad(past, normal((2, 64), FP32, 164), 10)
        else:
            ns.embedding(past, table)

    def nan():
        g = normal((64, 64), FP32, 165)
        g[3, 4] = float("nan")
        ns.muon_step([normal((64, 64), FP32, 166)], [g], [torch.zeros(64, 64, device="cuda")], lr=0.02)

    assert ns.check_status() == ns.OK
    for grad in (False, True):
        for order in (0, 1):
            for call in ((lambda: token(grad)), nan) if order else (nan, (lambda: token(grad))):
                call()
            assert ns.check_status() == ns.WARN_NONFINITE
            assert ns.check_status() == ns.WARN_TOKEN
            assert ns.check_status() == ns.OK
    dy, ck = normal((4096, 1024), BF16, 167), ns.checkpoint_store(normal((4096, 1024), BF16, 168))
    token(False)
    ns.set_wait_limit_ns(1)
    try:
        ns.weight_grad(dy, ck)
        with pytest.raises(ns.MuonError) as e:
            ns.check_status()
        assert e.value.code == ns.ERR_TIMEOUT
    finally:
        ns.set_wait_limit_ns(0)
    assert ns.check_status() == ns.WARN_TOKEN
    assert ns.check_status() == ns.OK


# ---------------------------------------------------------------------------- table gradient

@pytest.mark.parametrize("n,vocab,dim", [(16385, 5000, 33), (20000, 50257, 72), (65536, 50257, 24), (70001, 700, 40),
                                         (140000, 128256, 8), (66000, 3, 264)])
def test_embedding_grad_many_tokens(n, vocab, dim):
    """More tokens than one reading of a sorting block holds, and more than 16-bit counts do."""
    import newton_schulz_13_b200 as ns
    for ids_dt, dt, grad_dt, acc in ((torch.int64, BF16, FP32, True), (torch.int32, FP32, BF16, False)):
        t = tokens_of(n, vocab, 170, ids_dt)
        dy = normal((n, dim), dt, 171, 1e-3)
        old = normal((vocab, dim), grad_dt, 172, 1e-3) if acc else None
        got = ns.embedding_grad(t, dy, vocab, scale=1.7, grad=old.clone() if acc else None, grad_dtype=None if acc else grad_dt,
                                accumulate=acc)
        want, tol = embed_grad_want(t, dy, vocab, 1.7, old)
        within(got, want, tol + U[grad_dt] * want.abs())
        again = ns.embedding_grad(t, dy, vocab, scale=1.7, grad=old.clone() if acc else None, grad_dtype=None if acc else grad_dt,
                                  accumulate=acc)
        assert torch.equal(again, got)
    assert ns.check_status() == ns.OK


# ---------------------------------------------------------------------------- RMS norm

def test_rms_norm_output_over_the_input():
    """Where y takes x's place and there is no residual, no h remains to be returned."""
    import newton_schulz_13_b200 as ns
    for shape in ((3, 5, 64), (1100, 4096), (9, 77)):
        x, w = normal(shape, BF16, 173), normal(shape[-1:], FP32, 174)
        want = ns.rms_norm(x, w)
        assert want.h is x
        for alias in (lambda b: b, lambda b: b.view(shape), lambda b: b.detach()):
            buf = x.clone()
            got = ns.rms_norm(buf, w, y=alias(buf))
            assert torch.equal(got.y, want.y) and torch.equal(got.rstd, want.rstd)
            assert got.h is None
        other = torch.empty_like(x)
        assert ns.rms_norm(x, w, y=other).h is x and torch.equal(other, want.y)
        buf, res = x.clone(), normal(shape, FP32, 175)
        got, ref = ns.rms_norm(buf, w, residual=res, y=buf), ns.rms_norm(x, w, residual=res)
        assert torch.equal(got.h, ref.h) and torch.equal(buf, ref.y)
    x = torch.empty(0, 64, device="cuda")
    assert ns.rms_norm(x, torch.ones(64, device="cuda"), y=torch.empty(0, 64, device="cuda")).h is x      # nothing overwritten
    assert ns.check_status() == ns.OK


PAIRS = [(BF16, BF16), (BF16, FP32), (FP32, BF16), (FP32, FP32), (BF16, None), (FP32, None)]


@pytest.mark.parametrize("x_dt,r_dt", PAIRS)
@pytest.mark.parametrize("rows,dim", [(140000, 31), (66000, 65), (17000, 263), (5500, 771), (1100, 4093), (1031, 4096), (600, 8191)])
def test_rms_norm_many_unaligned_rows(rows, dim, x_dt, r_dt):
    """The ring with rows of any alignment: each tensor has a stride and an offset of its own."""
    import newton_schulz_13_b200 as ns
    x = strided(normal((rows, dim), x_dt, 176), 1, 3)
    r = None if r_dt is None else strided(normal((rows, dim), r_dt, 177, 2.0), 3, 1)
    w = 1.0 + 0.1 * torch.randn(dim, generator=gen(178), device="cuda")
    y = Guarded(rows, dim, x_dt, 5, 1)
    h = None if r is None else Guarded(rows, dim, r_dt, 2, 5)
    got = ns.rms_norm(x, w, residual=r, eps=1e-5, checkpoint=True, y=y.view, h=None if h is None else h.view)
    want_h, want_rstd, want = norm_want(x, r, w, 1e-5)
    assert torch.equal(got.h, want_h)
    within(got.rstd, want_rstd, want_rstd * SUM * E, "rstd")
    within(got.y, want, want.abs() * (SUM * E + U[x_dt]), "y")
    back = ns.checkpoint_restore(got.checkpoint, dtype=FP32)
    scale = got.checkpoint.scales.double()
    each = scale.repeat_interleave(32, 1)[:, :dim]
    within(back, want, want.abs() * (2.0 ** -4 + SUM * E) + each * 2.0 ** -10, "checkpoint")
    y.check()
    if h is not None:
        h.check()
    # in place, in buffers whose gaps must stay
    xb = Guarded(rows, dim, x_dt, 1, 3)
    xb.view.copy_(x)
    rb = None if r is None else Guarded(rows, dim, r_dt, 3, 1)
    if rb is not None:
        rb.view.copy_(r)
    same = ns.rms_norm(xb.view, w, residual=None if rb is None else rb.view, eps=1e-5, checkpoint=True, y=xb.view,
                       h=None if rb is None else rb.view)
    assert torch.equal(xb.view, got.y) and torch.equal(same.rstd, got.rstd)
    assert torch.equal(same.checkpoint.q.view(torch.uint8), got.checkpoint.q.view(torch.uint8))
    xb.check()
    if rb is not None:
        assert torch.equal(rb.view, got.h)
        rb.check()
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("x_dt,r_dt", PAIRS)
@pytest.mark.parametrize("rows,dim", [(11000, 384), (8200, 512), (9000, 520), (2100, 2048), (1900, 2304), (1030, 4104), (900, 5120),
                                      (600, 8192)])
def test_rms_norm_many_aligned_rows(rows, dim, x_dt, r_dt):
    """On both sides of every bound of the choice between the ring and the threads' own loads."""
    import newton_schulz_13_b200 as ns
    x, r = normal((rows, dim), x_dt, 190), None if r_dt is None else normal((rows, dim), r_dt, 191, 2.0)
    w = 1.0 + 0.1 * torch.randn(dim, generator=gen(192), device="cuda")
    got = ns.rms_norm(x, w, residual=r, eps=1e-5, checkpoint=True)
    want_h, want_rstd, want = norm_want(x, r, w, 1e-5)
    assert torch.equal(got.h, want_h)
    within(got.rstd, want_rstd, want_rstd * SUM * E, "rstd")
    within(got.y, want, want.abs() * (SUM * E + U[x_dt]), "y")
    each = got.checkpoint.scales.double().repeat_interleave(32, 1)[:, :dim]
    within(ns.checkpoint_restore(got.checkpoint, dtype=FP32), want, want.abs() * (2.0 ** -4 + SUM * E) + each * 2.0 ** -10, "checkpoint")
    xi, ri = x.clone(), None if r is None else r.clone()
    same = ns.rms_norm(xi, w, residual=ri, h=ri, y=xi, checkpoint=True)
    assert torch.equal(xi, got.y) and (r is None or torch.equal(ri, got.h))
    assert torch.equal(same.checkpoint.q.view(torch.uint8), got.checkpoint.q.view(torch.uint8))
    assert ns.check_status() == ns.OK


@pytest.mark.parametrize("dy_dt", DTS)
@pytest.mark.parametrize("h_dt", DTS)
@pytest.mark.parametrize("rows,dim", [(20000, 72), (20000, 71), (6000, 1024), (6000, 1023), (3000, 4096), (3000, 4093), (1500, 8192),
                                      (1500, 8191), (700, 8200), (700, 8201), (700, 16391)])
def test_rms_norm_grad_many_rows(rows, dim, h_dt, dy_dt):
    """Enough rows per group for the ring's stages to be filled again several times, with dh; then
    with dx in the place of each tensor of its type."""
    import newton_schulz_13_b200 as ns
    pad = 0 if dim % 8 == 0 else 1
    h = strided(normal((rows, dim), h_dt, 180, 2.0), 8 if pad == 0 else 1, 8 if pad == 0 else 3)
    dy = strided(normal((rows, dim), dy_dt, 181, 1e-3), 0 if pad == 0 else 2, pad)
    dh = strided(normal((rows, dim), h_dt, 182, 1e-3), 16 if pad == 0 else 5, 2 * pad)
    w = 1.0 + 0.1 * torch.randn(dim, generator=gen(183), device="cuda")
    rstd = (1.0 / torch.sqrt(h.double().square().mean(1) + 1e-5)).float()
    dx = Guarded(rows, dim, h_dt, 8 if pad == 0 else 3, 8 if pad == 0 else 1)
    got, dw = ns.rms_norm_grad(dy, h, w, rstd, dh=dh, dx=dx.view)
    r = rstd.double()[:, None]
    n, a = h.double() * r, dy.double() * w.double()
    want = r * (a - n * (a * n).mean(1, keepdim=True)) + dh.double()
    mag = r * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + dh.double().abs()
    within(got, want, SUM * E * mag + U[h_dt] * want.abs(), "dx")
    t = dy.double() * n
    within(dw, t.sum(0), (rows + 8) * E * t.abs().sum(0), "dweight")
    dx.check()
    for place in ("h", "dh", "dy") if dy_dt == h_dt else ("h", "dh"):
        bufs = {}
        for name, src, extra, offset in (("h", h, 8 if pad == 0 else 1, 8 if pad == 0 else 3), ("dy", dy, 0 if pad == 0 else 2, pad),
                                         ("dh", dh, 16 if pad == 0 else 5, 2 * pad)):
            bufs[name] = Guarded(rows, dim, src.dtype, extra, offset)
            bufs[name].view.copy_(src)
        _, dw2 = ns.rms_norm_grad(bufs["dy"].view, bufs["h"].view, w, rstd, dh=bufs["dh"].view, dx=bufs[place].view)
        assert torch.equal(bufs[place].view, got) and torch.equal(dw2, dw), place
        for b in bufs.values():
            b.check()
    assert ns.check_status() == ns.OK


# ---------------------------------------------------------------------------- arguments

@pytest.mark.parametrize("plain", [True, False])
def test_arguments_without_a_truth_value(plain, monkeypatch):
    """An argument whose truth value cannot be had raises its own error."""
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    from newton_schulz_13_b200 import gradients
    if not plain:
        monkeypatch.setattr(gradients, "_fast", None)

    class Unsure:
        def __bool__(self):
            raise ZeroDivisionError("unsure")

        __int__ = __index__ = __bool__

    x, w = normal((4, 64), BF16, 169), torch.ones(64, device="cuda")
    t = torch.arange(4, device="cuda")
    grad, ck = torch.zeros(64, 64, device="cuda"), ns.checkpoint_store(x)
    for call in (lambda: ns.rms_norm(x, w, output=Unsure()), lambda: ns.rms_norm(x, w, checkpoint=Unsure()),
                 lambda: ns.embedding_grad(t, x, 64, grad=grad, accumulate=Unsure()),
                 lambda: ns.weight_grad(x, ck, grad=grad, accumulate=Unsure())):
        with pytest.raises(ZeroDivisionError):
            call()
    assert ns.check_status() == ns.OK
