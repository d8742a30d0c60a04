"""Argument checks of the norms around a residual sum, without a GPU: every call is refused, or is empty, before any CUDA call."""
import pytest
import torch


@pytest.fixture(scope="module")
def kq():
    from quantized_decode_gemv_block_gb300 import build
    build.build()
    import quantized_decode_gemv_block_gb300 as m
    m.load_library()
    return m


FAKE = 1 << 20  # never dereferenced


def test_refusals(kq):
    L = kq.lib()
    good = dict(yd=kq.BF16, y=FAKE, ys=64, hd=kq.F32, h=FAKE + 4096, hs=64, ho=FAKE + 8192, hos=64, g=FAKE + 256, gs=0, sc=1.0, wd=kq.F32,
                post=FAKE, pre=FAKE, eps=1e-6, xd=kq.BF16, x=FAKE + 16384, xs=64, T=4, H=64, fl=kq.KQ_NORM_POST)

    def call(**kw):
        a = dict(good, **kw)
        return L.kq_residual_norm(a["yd"], a["y"], a["ys"], a["hd"], a["h"], a["hs"], a["ho"], a["hos"], a["g"], a["gs"], a["sc"], a["wd"],
                                  a["post"], a["pre"], a["eps"], a["xd"], a["x"], a["xs"], a["T"], a["H"], a["fl"], None)
    for kw in (dict(yd=0), dict(hd=3), dict(wd=7), dict(xd=-1)):
        assert call(**kw) == kq.KQ_ERR_UNSUPPORTED, kw
    for kw in (dict(fl=4), dict(T=-1), dict(T=(1 << 30) + 1), dict(H=0), dict(H=32769), dict(y=None, h=None), dict(y=None), dict(fl=0),
               dict(x=None), dict(ho=None, x=None, pre=None), dict(ys=63), dict(hs=1), dict(hos=0), dict(xs=63), dict(gs=63), dict(y=FAKE + 1),
               dict(h=FAKE + 2), dict(ho=FAKE + 2), dict(g=FAKE + 1), dict(post=FAKE + 2), dict(pre=FAKE + 1), dict(x=FAKE + 16385),
               dict(ho=FAKE + 4096, hos=65), dict(x=FAKE + 4096), dict(x=FAKE + 8192), dict(ho=FAKE), dict(x=FAKE, xs=65),
               dict(x=FAKE, xd=kq.F32)):
        assert call(**kw) == kq.KQ_ERR_ARG, kw
        assert L.kq_last_error().decode() != ""
    assert call(T=0, y=None, h=None) == 0 and L.kq_last_error().decode() == ""


def test_binding_refusals(kq):
    h, w = torch.zeros((4, 64)), torch.ones(64)
    for args, kw, match in (((None, None), {}, "one of h and y"), ((h[0], None), {}, "tokens, H"), ((h, h[:3]), {}, "must be"),
                            ((h, h.t().contiguous().t()), {}, "contiguous rows"), ((h, h[:1].expand(4, 64)), {}, "row of its own"),
                            ((h, h), dict(pre=w[:60]), "weights"), ((h, h), dict(post=w, pre=w.bfloat16()), "agree in type"),
                            ((h, h), dict(gate=w.bfloat16()), "y's type"), ((h, h), dict(gate=w[:9]), "gate"),
                            ((h, h), dict(h_out=h.bfloat16()), "h's type"), ((h, h), dict(x_out=h), "without pre"),
                            ((h, h), dict(pre=w, x_out=h, x_dtype=torch.bfloat16), "x_dtype"), ((h, h), dict(h_out=h[:, :60]), "must be")):
        with pytest.raises(ValueError, match=match):
            kq.residual_norm(*args, stream=0, **kw)
    with pytest.raises(TypeError):
        kq.residual_norm(h.half(), h.half(), stream=0)
    with pytest.raises(ValueError, match="gradient"):
        kq.residual_norm(h, h.clone().requires_grad_(), stream=0)
    with pytest.raises(ValueError, match="gradient"):
        kq.residual_norm(h, h, pre=w.clone().requires_grad_(), stream=0)
