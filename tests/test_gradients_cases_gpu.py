"""The gradient-making operators on calls with a history or a size of their own.

Tolerances as in test_gradients_gpu: roundings counted element by element."""
import pytest
import torch

from .test_gradients_gpu import BF16, DTS, FP32, Guarded, normal

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
