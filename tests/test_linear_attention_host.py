"""Argument checks of the linear attention and group norm entry points that
need no GPU: every refusal comes before any device work (the pointers here
are never dereferenced)."""
import ctypes

import pytest


def _lib():
    import long_sequence_fft_b200 as lsf
    return lsf, lsf.library()


def _shape(**kw):
    from long_sequence_fft_b200.linear_attention import _Shape
    f = dict(B=2, T=100, nseq=0, H=4, Hq=4, Hk=2, Hv=2, K=64, V=64, dtype=2, scale=1.0, zero_rest=0)
    f.update(kw)
    s = _Shape()
    for n, x in f.items():
        setattr(s, n, x)
    for n, h, d in (("q_stride", s.Hq, s.K), ("k_stride", s.Hk, s.K), ("v_stride", s.Hv, s.V), ("o_stride", s.H, s.V)):
        if n not in kw:
            getattr(s, n)[:] = [s.T * h * d, h * d, d]
    return s


# far apart, aligned, never read
Q, K, V, O, LD, ST, CU, WS = (i << 36 for i in range(1, 9))


def _call(s, q=Q, k=K, v=V, ld=LD, init=None, cu=None, o=O, fin=None, ws=WS, n=1 << 40):
    _, lib = _lib()
    return lib.fftconv_linear_attention(ctypes.byref(s) if s is not None else None, q, k, v, ld, init, cu, o, fin, ws,
                                        n, None)


@pytest.mark.parametrize("shape,args,status", [
    (None, {}, -1),
    (dict(B=-1), {}, -1),
    (dict(H=0), {}, -1),
    (dict(H=4, Hk=3), {}, -1),
    (dict(dtype=0), {}, -2),
    (dict(dtype=9), {}, -1),
    (dict(K=0), {}, -1),
    (dict(K=136), {}, -2),
    (dict(V=20), {}, -2),
    (dict(nseq=2), {}, -1),                                  # packed needs B = 1
    (dict(B=1, nseq=2), {}, -1),                             # ... and offsets
    ({}, dict(cu=CU), -1),                                   # offsets without packed sequences
    (dict(T=1 << 31), {}, -2),
    ({}, dict(q=None), -1),
    ({}, dict(o=None), -1),
    ({}, dict(ld=None), -1),
    ({}, dict(q=Q + 8), -3),
    ({}, dict(o=O + 2), -3),
    ({}, dict(init=ST + 4), -3),
    (dict(q_stride=[0, 256, 64]), {}, -3),                   # expanded
    (dict(k_stride=[12800, 132, 64]), {}, -3),               # not 16-byte rows
    ({}, dict(o=Q), -1),
    ({}, dict(o=V + 64), -1),
    ({}, dict(init=ST, fin=ST + 1024), -1),
    (dict(B=1, T=1 << 16, H=1, Hq=1, Hk=1, Hv=1), dict(n=16), -1),        # cut along time: workspace too small
    (dict(B=1, T=1 << 16, H=1, Hq=1, Hk=1, Hv=1), dict(ws=WS + 16), -3),
    (dict(B=1, T=1 << 16, H=1, Hq=1, Hk=1, Hv=1), dict(ws=None), -1),
])
def test_linear_attention_refusals(shape, args, status):
    lsf, lib = _lib()
    s = None if shape is None else _shape(**{k: v for k, v in shape.items() if not k.endswith("stride")})
    for n, x in (shape or {}).items():
        if n.endswith("stride"):
            getattr(s, n)[:] = x
    assert _call(s, **args) == status
    assert lib.fftconv_last_error()


@pytest.mark.parametrize("args,status", [
    (dict(dinit=ST), -1),                                    # dk and dv both read dfinal
    (dict(dinit=ST + 1024), -1), (dict(dinit=WS + 2), -3), (dict(dq=O), -1), (dict(dk=K), -1), (dict(dv=None), -1),
    (dict(dq=(9 << 36) + 4), -3), (dict(dk=9 << 36), -1), (dict(ws=None), -1),
])
def test_linear_attention_backward_refusals(args, status):
    _, lib = _lib()
    a = dict(dq=9 << 36, dk=10 << 36, dv=11 << 36, dinit=None, ws=WS)
    a.update(args)
    s = _shape(Hk=2)                                          # (shared heads: partial sums need the workspace)
    rc = lib.fftconv_linear_attention_backward(ctypes.byref(s), Q, K, V, LD, None, None, O, ST, a["dq"], a["dk"],
                                               a["dv"], a["dinit"], a["ws"], 1 << 40, None)
    assert rc == status and lib.fftconv_last_error()


def test_linear_attention_workspace():
    """None where a call fills the GPU by its sequences and heads; segment
    states where it is cut along time; fp32 partial sums of shared heads."""
    _, lib = _lib()
    w = lambda s, b=0: lib.fftconv_linear_attention_workspace_bytes(ctypes.byref(s), b)   # noqa: E731
    assert w(_shape(B=64, H=16, Hq=16, Hk=16, Hv=16, T=4096)) == 0
    assert w(_shape(B=64, H=16, Hq=16, Hk=16, Hv=16, T=4096), 1) == 0
    assert w(_shape(B=1, H=2, Hq=2, Hk=2, Hv=2, T=65536)) > 0
    assert w(_shape(B=64, H=16, Hq=16, Hk=4, Hv=16, T=4096), 1) == 64 * 4096 * 16 * 64 * 4
    assert w(_shape(dtype=0)) == 0 and w(_shape(T=0)) == 0


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), -1), (dict(Hk=3), -1), (dict(dtype=0), -2), (dict(K=12), -2), (dict(V=256), -2), (dict(pool=3), -1),
    (dict(q=None), -1), (dict(state=None), -1), (dict(q=Q + 2), -3), (dict(state=ST + 4), -3), (dict(o=Q), -1),
    (dict(o=ST), -1), (dict(qs=(0, 64)), -1), (dict(qs=None), -1),
])
def test_step_refusals(change, status):
    _, lib = _lib()
    a = dict(q=Q, k=K, v=V, ld=LD, state=ST, slots=None, o=O, B=2, pool=2, H=4, Hq=4, Hk=4, Hv=4, K=64, V=64, dtype=1,
             qs=(256, 64))
    a.update(change)
    st = lambda x: None if x is None else (ctypes.c_int64 * 2)(*x)           # noqa: E731
    rc = lib.fftconv_linear_attention_step(a["q"], a["k"], a["v"], a["ld"], a["state"], a["slots"], a["o"], a["B"],
                                           a["pool"], a["H"], a["Hq"], a["Hk"], a["Hv"], a["K"], a["V"], a["dtype"],
                                           1.0, st(a["qs"]), st((256, 64)), st((256, 64)), None)
    assert rc == status and lib.fftconv_last_error()


@pytest.mark.parametrize("change,status", [
    (dict(G=5), -1), (dict(C=0), -1), (dict(N=-1), -1), (dict(dtype=7), -1), (dict(wdtype=1), -1), (dict(act=3), -1),
    (dict(b=None), -1), (dict(mean=None), -1), (dict(x=None), -1), (dict(x=Q + 2), -3), (dict(ldx=60), -1),
    (dict(gate=K, ldg=8), -1), (dict(y=Q), -1), (dict(ws=None), -1), (dict(n=8), -1), (dict(ws=WS + 16), -3),
])
def test_group_norm_refusals(change, status):
    _, lib = _lib()
    a = dict(x=Q, gate=None, w=V, b=LD, y=O, mean=ST, rstd=CU, N=4, S=3, C=64, G=4, ldx=64, ldg=64, dtype=2, wdtype=0,
             act=1, ws=WS, n=1 << 30)
    a.update(change)
    rc = lib.fftconv_group_norm(a["x"], a["gate"], a["w"], a["b"], a["y"], a["mean"], a["rstd"], a["N"], a["S"],
                                a["C"], a["G"], a["ldx"], a["ldg"], a["dtype"], a["wdtype"], a["act"], 1e-5, a["ws"],
                                a["n"], None)
    assert rc == status and lib.fftconv_last_error()
    # the backward call's own: gradients that overlap, or that nothing asks for
    back = lambda dx=O, dgate=None, dw=None, db=None, dy=K: lib.fftconv_group_norm_backward(   # noqa: E731
        Q, None, None, None, dy, ST, CU, dx, dgate, dw, db, 4, 3, 64, 4, 64, 0, 64, 2, 2, 1, WS, 1 << 30, None)
    assert back(dx=Q) == -1 and back(dw=V, db=LD) == -1 and back(dgate=V) == -1 and back(dy=None) == -1


@pytest.mark.parametrize("N,C", [(1, 65535 * 256 + 1), (1 << 20, 1 << 12)])
def test_group_norm_sizes_beyond_a_grid(N, C):
    _, lib = _lib()
    rc = lib.fftconv_group_norm(Q, None, None, None, O, None, None, N, 1, C, C, C, 0, 2, 2, 1, 1e-5, WS, 1 << 50, None)
    assert rc == -2 and lib.fftconv_last_error()


def test_python_refuses_cpu_tensors():
    import torch
    import long_sequence_fft_b200 as lsf
    t = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lsf.linear_attention(t, t, t, torch.zeros(2))
    with pytest.raises(ValueError):
        lsf.linear_attention_step(t[0], t[0], t[0], torch.zeros(2), torch.zeros((4, 2, 64, 64)))
    with pytest.raises(ValueError):
        lsf.group_norm(torch.zeros((2, 8)), 2)
    with pytest.raises(ValueError):
        lsf.linear_attention(t[0], t[0], t[0], torch.zeros(2))
