"""The gradient-making operators without a GPU: bad arguments are refused before a device is looked
for, good ones fail loudly where there is none, and the binding refuses tensors off the device."""
import os

import pytest

A, B, C, D, F, G, H, S, T = (0x100000000 * (i + 1) for i in range(9))     # pointers nobody reads
WS = 0x10000000000
BIG = 1 << 40


def _embedding(ns, tokens=A, bits=64, n=4, table=B, tdt=1, ts=8, vocab=10, dim=8, scale=1.0, out=C, odt=1, os_=8):
    return ns.lib.muon_embedding(tokens, bits, n, table, tdt, ts, vocab, dim, scale, out, odt, os_, None)


def _embedding_grad(ns, tokens=A, bits=64, n=4, dy=B, ddt=1, ds=8, vocab=10, dim=8, scale=1.0, grad=C, gdt=1, gs=8, acc=0,
                    ws=WS, wb=BIG):
    return ns.lib.muon_embedding_grad(tokens, bits, n, dy, ddt, ds, vocab, dim, scale, grad, gdt, gs, acc, ws, wb, None)


def _norm(ns, x=A, xdt=0, xs=64, r=B, rdt=0, rs=64, w=C, wdt=1, rows=4, dim=64, eps=1e-5, h=D, hs=64, y=F, ys=64, q=G, qs=64,
          sc=H, ss=2, rstd=S):
    return ns.lib.muon_rms_norm(x, xdt, xs, r, rdt, rs, w, wdt, rows, dim, eps, h, hs, y, ys, q, qs, sc, ss, rstd, None)


def _norm_grad(ns, dy=A, ddt=0, ds=64, h=B, hdt=0, hs=64, w=C, wdt=1, rstd=D, dh=F, dhs=64, rows=4, dim=64, dx=G, xs=64, dw=H,
               acc=0, ws=WS, wb=BIG):
    return ns.lib.muon_rms_norm_grad(dy, ddt, ds, h, hdt, hs, w, wdt, rstd, dh, dhs, rows, dim, dx, xs, dw, acc, ws, wb, None)


def _store(ns, x=A, xdt=0, xs=64, rows=4, dim=64, q=B, qs=64, sc=C, ss=2):
    return ns.lib.muon_checkpoint_store(x, xdt, xs, rows, dim, q, qs, sc, ss, None)


def _restore(ns, q=B, qs=64, sc=C, ss=2, rows=4, dim=64, x=A, xdt=0, xs=64):
    return ns.lib.muon_checkpoint_restore(q, qs, sc, ss, rows, dim, x, xdt, xs, None)


def _wgrad(ns, dy=A, ddt=0, ds=64, q=B, qs=96, sc=C, ss=3, rows=4, n=64, k=96, grad=D, gdt=0, gs=96, acc=0, ws=WS, wb=BIG):
    return ns.lib.muon_weight_grad(dy, ddt, ds, q, qs, sc, ss, rows, n, k, grad, gdt, gs, acc, ws, wb, None)


CALLS = [_embedding, _embedding_grad, _norm, _norm_grad, _store, _restore, _wgrad]
BAD = [
    (_embedding, dict(bits=16), "token_bits"), (_embedding, dict(n=-1), "n must"), (_embedding, dict(n=1 << 31), "n must"),
    (_embedding, dict(tokens=None), "tokens"), (_embedding, dict(tokens=A + 4), "aligned"),
    (_embedding, dict(tdt=2), "table_dtype"), (_embedding, dict(odt=-1), "out_dtype"),
    (_embedding, dict(vocab=0), "vocab"), (_embedding, dict(vocab=1 << 31), "vocab"), (_embedding, dict(dim=0), "dim"),
    (_embedding, dict(dim=(1 << 20) + 1, ts=1 << 21, os_=1 << 21), "dim"), (_embedding, dict(scale=float("inf")), "scale"),
    (_embedding, dict(ts=7), "stride"), (_embedding, dict(table=None), "table"), (_embedding, dict(out=None), "out"),
    (_embedding, dict(out=B + 64), "overlaps"), (_embedding, dict(out=A), "overlaps"), (_embedding, dict(table=B + 2), "aligned"),
    (_embedding_grad, dict(bits=8), "token_bits"), (_embedding_grad, dict(ddt=3), "dy_dtype"),
    (_embedding_grad, dict(gdt=3), "grad_dtype"), (_embedding_grad, dict(gs=3), "stride"), (_embedding_grad, dict(dy=None), "dy"),
    (_embedding_grad, dict(grad=None), "grad"), (_embedding_grad, dict(ws=None), "workspace"),
    (_embedding_grad, dict(ws=WS + 16), "aligned"), (_embedding_grad, dict(wb=0), "workspace_bytes"),
    (_embedding_grad, dict(grad=B), "overlaps"), (_embedding_grad, dict(ws=C), "overlaps"), (_embedding_grad, dict(ws=A), "overlaps"),
    (_embedding_grad, dict(scale=float("nan")), "scale"),
    (_norm, dict(xdt=9), "x_dtype"), (_norm, dict(rdt=9), "r_dtype"), (_norm, dict(wdt=9), "w_dtype"), (_norm, dict(rows=-1), "rows"),
    (_norm, dict(dim=0), "dim"), (_norm, dict(dim=32769), "dim"), (_norm, dict(eps=-1.0), "eps"), (_norm, dict(eps=float("nan")), "eps"),
    (_norm, dict(h=None), "together"), (_norm, dict(r=None), "together"), (_norm, dict(q=None), "together"),
    (_norm, dict(y=None, q=None, sc=None), "must be given"), (_norm, dict(x=None), "x must"), (_norm, dict(xs=63), "stride"),
    (_norm, dict(hs=63), "stride"), (_norm, dict(ys=63), "stride"), (_norm, dict(qs=63), "stride"), (_norm, dict(ss=1), "stride"),
    (_norm, dict(rstd=None), "rstd"), (_norm, dict(h=A + 64), "overlap"), (_norm, dict(h=B, hs=65), "overlap"),
    (_norm, dict(y=B), "overlap"), (_norm, dict(y=D), "overlap"), (_norm, dict(q=A), "overlap"), (_norm, dict(sc=G + 1), "overlap"),
    (_norm, dict(rstd=F), "overlap"), (_norm, dict(w=None), "weight"),
    (_norm_grad, dict(ddt=4), "dy_dtype"), (_norm_grad, dict(hdt=4), "h_dtype"), (_norm_grad, dict(wdt=4), "w_dtype"),
    (_norm_grad, dict(rows=-2), "rows"), (_norm_grad, dict(dim=40000), "dim"), (_norm_grad, dict(dw=None), "dweight"),
    (_norm_grad, dict(dy=None), "dy"), (_norm_grad, dict(dx=None), "dx"), (_norm_grad, dict(rstd=None), "rstd"),
    (_norm_grad, dict(dhs=1), "stride"), (_norm_grad, dict(ws=None), "workspace"), (_norm_grad, dict(wb=1), "workspace_bytes"),
    (_norm_grad, dict(dx=A + 2), "overlap"), (_norm_grad, dict(dx=C), "overlap"), (_norm_grad, dict(dw=G), "overlap"),
    (_norm_grad, dict(ws=B), "overlap"), (_norm_grad, dict(dx=A, ddt=1), "overlap"),
    (_store, dict(xdt=2), "dtype"), (_store, dict(rows=-1), "rows"), (_store, dict(dim=0), "dim"), (_store, dict(x=None), "x must"),
    (_store, dict(q=None), "codes"), (_store, dict(sc=None), "codes"), (_store, dict(qs=3), "stride"), (_store, dict(ss=1), "stride"),
    (_store, dict(q=A + 4), "overlap"), (_store, dict(sc=B), "overlap"),
    (_restore, dict(xdt=2), "dtype"), (_restore, dict(x=B), "overlap"), (_restore, dict(xs=63), "stride"),
    (_wgrad, dict(ddt=2), "dy_dtype"), (_wgrad, dict(gdt=2), "grad_dtype"), (_wgrad, dict(rows=-1), "rows"),
    (_wgrad, dict(rows=(1 << 29) + 1), "rows"), (_wgrad, dict(n=0), "n and k"), (_wgrad, dict(k=(1 << 20) + 1), "n and k"),
    (_wgrad, dict(dy=None), "dy"), (_wgrad, dict(q=None), "codes"), (_wgrad, dict(sc=None), "codes"), (_wgrad, dict(grad=None), "grad"),
    (_wgrad, dict(gs=95), "stride"), (_wgrad, dict(qs=95), "stride"), (_wgrad, dict(ss=2), "stride"), (_wgrad, dict(ds=63), "stride"),
    (_wgrad, dict(grad=A), "overlap"), (_wgrad, dict(grad=B + 32), "overlap"), (_wgrad, dict(wb=0), "workspace"),
]


@pytest.mark.parametrize("call,kw,needle", BAD)
def test_bad_arguments_are_refused(call, kw, needle):
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint     # loads the calls' signatures
    assert call(ns, **kw) == ns.ERR_INVALID_ARG
    assert needle in ns.last_error(), ns.last_error()


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="checks the no-device path")
@pytest.mark.parametrize("call", CALLS)
def test_no_device_fails_loudly(call):
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    assert call(ns) == ns.ERR_UNSUPPORTED
    assert ns.last_error()


def test_nothing_to_do_needs_no_device():
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    assert _embedding(ns, n=0, tokens=None, out=None) == ns.OK
    assert _embedding_grad(ns, n=0, tokens=None, dy=None, acc=1) == ns.OK
    assert _norm(ns, rows=0) == ns.OK
    assert _norm_grad(ns, rows=0, acc=1) == ns.OK
    assert _store(ns, rows=0) == ns.OK and _restore(ns, rows=0) == ns.OK
    assert _wgrad(ns, rows=0, dy=None, q=None, sc=None, acc=1) == ns.OK


def test_side_by_side_columns_are_no_overlap():
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    # y in the right half of the buffer whose left half is x: only the missing device is reported
    rc = _norm(ns, x=A, xs=128, y=A + 128, ys=128)
    assert rc != ns.ERR_INVALID_ARG, ns.last_error()
    assert _norm(ns, x=A, xs=128, y=A + 126, ys=128) == ns.ERR_INVALID_ARG


def test_workspace_sizes():
    import newton_schulz_13_b200 as ns
    ns.ActCheckpoint
    f, g, w = ns.lib.muon_embedding_grad_workspace, ns.lib.muon_rms_norm_grad_workspace, ns.lib.muon_weight_grad_workspace
    assert f(0, 1, 1) > 0 and f(16384, 128256, 4096) < 1 << 28
    assert f(-1, 1, 1) == ns.ERR_INVALID_ARG and f(1, 0, 1) == ns.ERR_INVALID_ARG and f(1, 1, 0) == ns.ERR_INVALID_ARG
    assert g(0, 8) >= 0 and g(-1, 8) == ns.ERR_INVALID_ARG and g(1, 32769) == ns.ERR_INVALID_ARG
    assert w(100, 64, 96, 0) >= 0 and w(100, 64, 96, 2) == ns.ERR_INVALID_ARG and w((1 << 29) + 1, 1, 1, 0) == ns.ERR_INVALID_ARG
    for n in (1, 1000, 100000):     # sizes do not shrink as a call grows
        assert f(n + 1, 100, 64) >= f(n, 100, 64)
    # the largest sizes neither overflow nor ask for less than the parts they hold
    assert f((1 << 31) - 1, (1 << 31) - 1, 1 << 20) > (1 << 31) * 8


def test_binding_refuses_tensors_off_the_device():
    import torch

    import newton_schulz_13_b200 as ns
    x, w, t = torch.zeros(4, 64), torch.ones(64), torch.zeros(4, dtype=torch.int64)
    ck = ns.ActCheckpoint(torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8).view(torch.float8_e8m0fnu))
    for call in (lambda: ns.embedding(t, x), lambda: ns.embedding_grad(t, x, 5), lambda: ns.rms_norm(x, w),
                 lambda: ns.rms_norm_grad(x, x, w, w[:4]), lambda: ns.checkpoint_store(x), lambda: ns.checkpoint_restore(ck),
                 lambda: ns.weight_grad(x, ck)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_unknown_attribute():
    import newton_schulz_13_b200 as ns
    with pytest.raises(AttributeError):
        ns.no_such_operator
