"""GPU tests of group norm against its fp64 definition.

Bounds: y and the gradients are fp32 expressions rounded once: u times the
value, plus fp32 errors relative to the size of the terms: |n| <= |xh w| + |b|
and its mean and sums.  The statistics' own errors are a few 2^-24 of
max|x| rstd (the mean's rounding, seen in units of the normalised value); 2^-20
of (1 + max|x| rstd) times the terms' scale covers them, the activations'
fast exponential and the reductions (16 binary levels)."""
import pytest

from mixer_reference import group_norm as reference

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(shape, dtype, seed, gate, affine, wdtype=None, mean=0.5):
    g, dt = _gen(seed), DT[dtype]
    r = lambda *s: torch.randn(s, generator=g, device="cuda")                # noqa: E731
    C = shape[-1]
    x = dict(x=(r(*shape) * 1.5 + mean).to(dt), dy=r(*shape).to(dt), gate=r(*shape).mul(2).to(dt) if gate else None,
             weight=None, bias=None)
    if affine:
        wd = DT[wdtype or "f32"]
        x["weight"], x["bias"] = (1 + 0.3 * r(C)).to(wd), (0.3 * r(C)).to(wd)
    return x


def _run(x, G, act, eps=1e-5):
    import long_sequence_fft_b200 as lsf
    names = [n for n in ("x", "gate", "weight", "bias") if x[n] is not None]
    leaves = {n: x[n].clone().requires_grad_() for n in names}
    y = lsf.group_norm(leaves["x"], G, leaves.get("weight"), leaves.get("bias"), gate=leaves.get("gate"),
                       activation=act, eps=eps)
    got = {"y": y.detach()}
    for n, gr in zip(names, torch.autograd.grad(y, list(leaves.values()), x["dy"])):
        got["d" + n] = gr
    with torch.no_grad():
        y2 = lsf.group_norm(x["x"], G, x["weight"], x["bias"], gate=x["gate"], activation=act, eps=eps)
    assert torch.equal(y2, got["y"])
    return got


def _check(got, x, G, act, eps=1e-5, what=""):
    ref = reference(x["x"], G, x["weight"], x["bias"], x["gate"], act, eps, x["dy"])
    # sizes of the terms behind each value
    xd = x["x"].double()
    N, C = xd.shape[0], xd.shape[-1]
    rows = xd.reshape(N, -1, G, C // G)
    rstd = 1 / torch.sqrt(rows.var(dim=(1, 3), unbiased=False) + eps)                        # [N, G]
    ratio = float((rows.abs().amax(dim=(1, 3)) * rstd).max())
    w = 1.0 if x["weight"] is None else float(x["weight"].abs().max())
    b = 0.0 if x["bias"] is None else float(x["bias"].abs().max())
    n = ratio * w + b
    gate = 1.0 if x["gate"] is None else float(x["gate"].abs().max())
    dn = float(x["dy"].abs().max()) * max(1.1, gate)
    count = xd.numel() // C
    scale = {"y": n * max(1.0, gate), "dgate": dn * n * 1.1, "dx": float(rstd.max()) * dn * w * (1 + ratio) * 2,
             "dweight": dn * ratio * count ** 0.5 * 4, "dbias": dn * count ** 0.5 * 4}
    for name, t in got.items():
        u = torch.finfo(t.dtype).eps / 2
        err = (t.double() - ref[name]).abs()
        bound = u * ref[name].abs() + 2.0 ** -20 * (1 + ratio) * scale[name] + torch.finfo(t.dtype).smallest_normal * u
        worst = (err - bound).max().item()
        assert worst <= 0, f"{what} {name}: {err.max().item():.3e} beyond its bound by {worst:.3e}"


SHAPES = [
    ((1, 8), 1), ((8, 768), 12), ((5, 760), 8), ((33, 2048), 16), ((3, 4096), 1), ((700, 64), 4), ((9, 35), 7),
    ((4, 90), 3), ((2, 6000), 2),                                            # one position a sample
    ((2, 3, 8), 4), ((1, 100, 64), 1), ((3, 257, 760), 8), ((2, 1000, 36), 4), ((2, 7, 5, 48), 3), ((1, 4097, 24), 24),
    ((2, 40, 4104), 3), ((5, 2, 6), 1),
]


@pytest.mark.parametrize("shape,G", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("gate,act,affine", [(False, "silu", True), (True, "silu", True), (True, "sigmoid", False),
                                             (False, "none", True), (True, "none", False)])
def test_forward_and_gradients(shape, G, dtype, gate, act, affine):
    x = _inputs(shape, dtype, seed=sum(shape) + G, gate=gate, affine=affine)
    _check(_run(x, G, act), x, G, act, what=f"{shape} G={G} {dtype}")


@pytest.mark.parametrize("shape,G", [((5003, 768), 12), ((20011, 96), 4), ((9001, 1024), 2), ((4100, 35), 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True])
def test_more_rows_than_the_gpu_holds(shape, G, dtype, gate):
    """Blocks that walk down many rows, the last of them beyond the end."""
    x = _inputs(shape, dtype, seed=shape[0], gate=gate, affine=True)
    _check(_run(x, G, "silu"), x, G, "silu", what=f"{shape} G={G} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_parameters_in_the_tensors_type(dtype):
    x = _inputs((40, 256), dtype, seed=3, gate=True, affine=True, wdtype=dtype)
    got = _run(x, 4, "silu")
    assert got["dweight"].dtype == DT[dtype]
    _check(got, x, 4, "silu")


def test_far_mean_and_constant_groups():
    """A mean far from zero (two passes over the values, or joined squares,
    not a difference of squares), and groups without variance."""
    for shape in ((20, 256), (2, 500, 256)):
        x = _inputs(shape, "f32", seed=5, gate=False, affine=True, mean=300.0)
        _check(_run(x, 4, "none"), x, 4, "none", what=f"far mean {shape}")
        x["x"] = torch.full(shape, 3.25, device="cuda")
        got = _run(x, 4, "none")
        assert torch.equal(got["y"], x["bias"].expand(shape))


def test_extreme_gates_and_values():
    """Gates and values where the exponential over- or underflows."""
    import long_sequence_fft_b200 as lsf
    x = torch.randn((4, 64), generator=_gen(1), device="cuda")
    gate = torch.tensor([-1e30, -200.0, -88.0, -87.0, 0.0, 87.0, 200.0, 1e30], device="cuda").repeat(4, 8)
    for act in ("silu", "sigmoid"):
        got = lsf.group_norm(x, 4, gate=gate, activation=act)
        ref = reference(x, 4, gate=gate, act=act)["y"]
        ref = torch.where(gate < -80, torch.zeros_like(ref), ref)            # below 1e-33 of the values
        assert torch.isfinite(got).all()
        assert ((got.double() - ref).abs() <= 1e-5 * ref.abs() + 1e-30).all(), act


def test_strided_rows_streams_and_graphs():
    """x and the gate as slices of one projection; a side stream; a captured
    forward and backward pass replayed on new inputs."""
    import long_sequence_fft_b200 as lsf
    wide = torch.randn((50, 3, 256), generator=_gen(2), device="cuda").bfloat16()
    x, gate = wide[:, 0], wide[:, 2]
    ref = lsf.group_norm(x.contiguous(), 4, gate=gate.contiguous(), activation="silu")
    assert torch.equal(lsf.group_norm(x, 4, gate=gate, activation="silu"), ref)
    odd = torch.randn((50, 261), generator=_gen(3), device="cuda").half()    # rows that are no multiple of 16 bytes
    a = lsf.group_norm(odd[:, :256], 4, activation="silu")
    b = lsf.group_norm(odd[:, :256].contiguous(), 4, activation="silu")
    # another order of the same fp32 sums, then one rounding each
    assert ((a.double() - b.double()).abs() <= 2 * 2.0 ** -11 * b.double().abs() + 1e-5).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lsf.group_norm(x, 4, gate=gate, activation="silu", stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, ref)
    out = torch.empty_like(ref)
    assert lsf.group_norm(x, 4, gate=gate, activation="silu", out=out) is out and torch.equal(out, ref)
    for shape in ((64, 256), (2, 300, 256)):
        p = _inputs(shape, "bf16", seed=6, gate=True, affine=True)
        leaves = {n: p[n].clone().requires_grad_() for n in ("x", "gate", "weight", "bias")}
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            y = lsf.group_norm(leaves["x"], 4, leaves["weight"], leaves["bias"], gate=leaves["gate"], activation="silu")
            grads = torch.autograd.grad(y, list(leaves.values()), p["dy"])
        new = _inputs(shape, "bf16", seed=7, gate=True, affine=True)
        with torch.no_grad():
            for n in leaves:
                leaves[n].copy_(new[n])
        g.replay()
        torch.cuda.synchronize()
        new["dy"] = p["dy"]
        _check(dict(y=y.detach(), **{"d" + n: t for n, t in zip(leaves, grads)}), new, 4, "silu", what="replayed")


def test_repeats_bit_for_bit_and_empty_calls():
    import long_sequence_fft_b200 as lsf
    for shape in ((300, 512), (3, 700, 96)):
        x = _inputs(shape, "bf16", seed=8, gate=True, affine=True)
        a, b = _run(x, 4, "silu"), _run(x, 4, "silu")
        for n in a:
            assert torch.equal(a[n], b[n]), n
    for shape in ((0, 64), (3, 0, 64)):
        x = torch.zeros(shape, device="cuda", requires_grad=True)
        w = torch.ones(64, device="cuda", requires_grad=True)
        y = lsf.group_norm(x, 4, w, torch.zeros(64, device="cuda"))
        y.sum().backward()
        assert y.shape == shape and not w.grad.any()


def test_gradients_against_differences():
    """Central differences of the fp64 definition along random directions."""
    for shape, gate in (((12, 128), True), ((2, 30, 48), False)):
        x = _inputs(shape, "f32", seed=9, gate=gate, affine=True)
        got = _run(x, 4, "silu")
        for name in ("x", "gate", "weight", "bias"):
            if x[name] is None:
                continue
            d = torch.randn(x[name].shape, generator=_gen(len(name)), device="cuda").double()

            def loss(e):
                y = {**x, name: x[name].double() + e * d}
                r = reference(y["x"], 4, y["weight"], y["bias"], y["gate"], "silu")["y"]
                return (r * x["dy"].double()).sum().item()

            h = 1e-5
            fd = (loss(h) - loss(-h)) / (2 * h)
            an = (got["d" + name].double() * d).sum().item()
            size = (got["d" + name].double() ** 2).sum().sqrt().item()
            # h^2 of the third derivative, 2^-52 / h of the loss, and the
            # gradient's fp32 errors against the directions
            assert abs(fd - an) <= 1e-4 * size + 1e-6, (name, fd, an)


def test_refusals():
    import long_sequence_fft_b200 as lsf
    x = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    bad = lambda *a, **kw: pytest.raises(ValueError, lsf.group_norm, *a, **kw)   # noqa: E731
    bad(x[0], 4)
    bad(x, 5)
    bad(x, 0)
    bad(x.double(), 4)
    bad(x.cpu(), 4)
    bad(x, 4, w)
    bad(x, 4, w, w.half())
    bad(x, 4, w.cpu(), w.cpu())
    bad(x, 4, w[:32], w[:32])
    bad(x, 4, activation="relu")
    bad(x, 4, gate=x[:2])
    bad(x, 4, gate=x.half())
    bad(x[:, ::2], 4)
    bad(x[:1].expand(4, 64), 4)
    bad(x, 4, out=torch.empty((4, 32), device="cuda"))
    bad(x, 4, out=torch.empty((4, 128), device="cuda")[:, :64])
    with pytest.raises(NotImplementedError):
        lsf.group_norm(x.clone().requires_grad_(), 4, out=torch.empty_like(x))
    with pytest.raises(lsf.FFTConvError):
        lsf.group_norm(x, 4, out=x)
