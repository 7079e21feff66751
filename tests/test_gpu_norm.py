"""The block norms (dg_norm_residual) against the definition in 64 bits:
widths around vectors and thread counts, both kinds, every optional input,
fp32 residual streams, odd alignment, aliasing, rows that are constant or zero."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import quantized_skinny_gemm_gb300 as dg
from gpu_util import DEV, need_gpu, sync

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def _case(rows, N, ftype, h32, gate, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda shape, std, dt: (torch.randn(shape, generator=g) * std).to(dt)
    dt = DT[ftype]
    return {"h": n((rows, N), 2.0, torch.float32 if h32 else dt), "y": n((rows, N), 0.7, dt),
            "w_pre": n((N,), 0.2, dt), "b_pre": n((N,), 0.1, dt), "w_post": n((N,), 0.2, dt),
            "b_post": n((N,), 0.1, dt),
            "gate": n((rows, N), 0.5, dt) if gate == 1 else n((N,), 0.5, dt) if gate == 2 else None}


def _run_and_check(t, ftype, h32, kind, alpha=1.0, beta=1.0, eps=1e-6, w_offset=1.0, what="norm",
                   h_out=True, x_out=True):
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    rows, N = (t["h"] if t["h"] is not None else t["y"]).shape
    ho = torch.full((rows, N), 3.0, dtype=torch.float32 if h32 else DT[ftype], device=DEV)
    xo = torch.full((rows, N), 3.0, dtype=DT[ftype], device=DEV)
    dg.norm_residual(dg.norm(d["h"], ho if h_out else None, xo if x_out else None, d["w_pre"],
                             b_pre=d["b_pre"], y=d["y"], w_post=d["w_post"], b_post=d["b_post"],
                             gate=d["gate"], alpha=alpha, beta=beta, eps=eps, w_offset=w_offset, kind=kind))
    sync()
    f = {k: None if v is None else ref.f64(v) for k, v in t.items()}
    a32, b32, e32, o32 = (float(np.float32(v)) for v in (alpha, beta, eps, w_offset))
    rh, rx, bh, bx = ref.norm(f["h"], f["y"], f["w_pre"], f["b_pre"], f["w_post"], f["b_post"], f["gate"],
                              a32, b32, e32, o32, kind == dg.NORM_LAYER, ftype, h32)
    if h_out:
        ref.check(ref.f64(ho), rh, bh, what + " h")
    if x_out:
        ref.check(ref.f64(xo), rx, bx, what + " x")
    return ho, xo


@pytest.mark.parametrize("N", [1, 2, 7, 8, 100, 255, 1000, 1536, 4095, 4096, 8192, 8200, 16384, 32767, 32768])
@pytest.mark.parametrize("ftype,kind,h32,gate", [("f16", 0, 0, 0), ("bf16", 1, 1, 1), ("bf16", 0, 0, 2)])
def test_widths(N, ftype, kind, h32, gate):
    need_gpu()
    t = _case(5, N, ftype, h32, gate, N)
    _run_and_check(t, ftype, h32, kind, alpha=0.9, beta=0.5, what="N=%d" % N)


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("drop", [("w_post", "b_post"), ("b_post",), ("b_pre",), ("gate",), ("h",),
                                  ("y", "w_post", "b_post", "gate"), ("w_post", "b_post", "b_pre", "gate")])
@pytest.mark.parametrize("h32", [0, 1])
def test_optional_inputs(kind, drop, h32):
    need_gpu()
    t = _case(9, 640, "f16", h32, 1, 7)
    for k in drop:
        t[k] = None
    _run_and_check(t, "f16", h32 if t["h"] is not None else 0 if not h32 else 1, kind, alpha=1.25,
                   beta=-0.5, w_offset=0.0, eps=1e-5, what=str(drop))


@pytest.mark.parametrize("h_out,x_out", [(True, False), (False, True)])
def test_one_output(h_out, x_out):
    need_gpu()
    ho, xo = _run_and_check(_case(3, 513, "bf16", 0, 0, 8), "bf16", 0, 0, h_out=h_out, x_out=x_out)
    assert h_out or (ho == 3.0).all()
    assert x_out or (xo == 3.0).all()


@pytest.mark.parametrize("rows", [1, 2, 3000])
def test_row_counts_are_independent_rows(rows):
    need_gpu()
    t = _case(rows, 1536, "f16", 0, 2, 9)
    ho, xo = _run_and_check(t, "f16", 0, 0)
    one = {k: v[rows - 1:] if v is not None and v.dim() == 2 else v for k, v in t.items()}
    h1, x1 = _run_and_check(one, "f16", 0, 0)
    assert torch.equal(h1[0], ho[-1]) and torch.equal(x1[0], xo[-1])


def test_in_place_and_unaligned():
    need_gpu()
    t = _case(4, 1024, "f16", 0, 1, 10)
    ho, xo = _run_and_check(t, "f16", 0, 1, w_offset=0.0)
    d = {k: v.to(DEV) for k, v in t.items()}
    kw = dict(b_pre=d["b_pre"], w_post=d["w_post"], b_post=d["b_post"], gate=d["gate"], kind=1)
    h, y = d["h"].clone(), d["y"].clone()
    dg.norm_residual(dg.norm(h, h, y, d["w_pre"], y=y, **kw))
    sync()
    assert torch.equal(h, ho) and torch.equal(y, xo)
    h, y = d["h"].clone(), d["y"].clone()
    dg.norm_residual(dg.norm(h, y, h, d["w_pre"], y=y, **kw))     # the other way round
    sync()
    assert torch.equal(y, ho) and torch.equal(h, xo)
    # one element off a 16-byte boundary
    off = lambda v: torch.cat((v.flatten()[:1], v.flatten()))[1:].view(v.shape)
    h2, x2 = torch.empty_like(ho), torch.empty_like(xo)
    e = {k: off(v) for k, v in d.items()}
    assert e["h"].data_ptr() % 16
    dg.norm_residual(dg.norm(e["h"], h2, x2, e["w_pre"], y=e["y"], b_pre=e["b_pre"], w_post=e["w_post"],
                             b_post=e["b_post"], gate=e["gate"], kind=1))
    sync()
    _, rx, _, bx = ref.norm(*(ref.f64(t[k]) for k in ("h", "y", "w_pre", "b_pre", "w_post", "b_post", "gate")),
                            1.0, 1.0, float(np.float32(1e-6)), 0.0, True, "f16", 0)
    ref.check(ref.f64(x2), rx, bx, "unaligned")
    assert (ref.f64(h2) == ref.f64(ho)).mean() > 0.99


@pytest.mark.parametrize("kind", [0, 1])
def test_zero_constant_and_non_finite_rows(kind):
    need_gpu()
    h = torch.randn(5, 300, generator=torch.Generator().manual_seed(11)).half()
    h[0] = 0
    h[1] = 2.0
    h[2, 7] = float("nan")
    h[3] *= 30000.0 / h[3].abs().max()
    t = {"h": h, "y": None, "w_pre": torch.ones(300).half(), "b_pre": None, "w_post": None, "b_post": None,
         "gate": None}
    d = h.to(DEV)
    xo = torch.empty_like(d)
    dg.norm_residual(dg.norm(d, None, xo, t["w_pre"].to(DEV), kind=kind, eps=1e-5))
    sync()
    assert (xo[0] == 0).all() and torch.isnan(xo[2]).all()
    if kind == dg.NORM_LAYER:
        assert (xo[1] == 0).all()
    keep = [0, 3, 4] if kind == dg.NORM_LAYER else [0, 1, 3, 4]
    f = ref.f64(h)[keep]
    _, rx, _, bx = ref.norm(f, None, np.ones(300), None, None, None, None, 1.0, 1.0,
                            float(np.float32(1e-5)), 0.0, kind == dg.NORM_LAYER, "f16", 0)
    ref.check(ref.f64(xo)[keep], rx, bx, "rows")


@pytest.mark.parametrize("N", [1, 5, 8, 113, 114, 121, 128, 129, 242, 243, 256, 263, 1537, 2056])
@pytest.mark.parametrize("ftype,kind,h32,gate", [("f16", 0, 0, 2), ("bf16", 1, 1, 1), ("bf16", 1, 0, 0)])
def test_many_rows(N, ftype, kind, h32, gate):
    """More rows than run at once, so that each team takes several."""
    need_gpu()
    t = _case(20011 if N < 300 else 2003, N, ftype, h32, gate, N)
    _run_and_check(t, ftype, h32, kind, alpha=0.9, beta=0.5, what="many N=%d" % N)


@pytest.mark.parametrize("rows,N", [(331, 8185), (331, 8186), (331, 8193), (317, 8192), (160, 16371), (9, 16371),
                                    (157, 32749), (157, 32752), (3, 32753)])
@pytest.mark.parametrize("bare", [False, True])
def test_wide_rows(rows, N, bare):
    """Few and many rows of widths around the vectors a thread holds; with all
    weights and with one alone, which shared memory holds."""
    need_gpu()
    t = _case(rows, N, "bf16", 0, 1, N)
    if bare:
        t["w_post"] = t["b_post"] = t["b_pre"] = None
    _run_and_check(t, "bf16", 0, 1, alpha=0.9, beta=0.5, what="wide N=%d" % N)


def test_rows_in_place():
    """h' over h, x over y: odd rows share 16-byte vectors with their neighbours."""
    need_gpu()
    t = _case(5003, 333, "f16", 0, 0, 3)
    d = {k: None if v is None else v.to(DEV) for k, v in t.items()}
    dg.norm_residual(dg.norm(d["h"], d["h"], d["y"], d["w_pre"], b_pre=d["b_pre"], y=d["y"], w_post=d["w_post"],
                             b_post=d["b_post"]))
    sync()
    ho, xo = _run_and_check(t, "f16", 0, 0, eps=1e-6, w_offset=0.0)
    assert torch.equal(d["h"], ho) and torch.equal(d["y"], xo)
