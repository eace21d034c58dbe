"""GPU tests of group norm's sample form where its samples go through the
passes some at a time, and where groups lie across blocks of channels; the
bounds are those of test_gpu_group_norm."""
import pytest

from test_gpu_group_norm import _check, _inputs, _run

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("shape,G,dtype,gate,affine", [
    ((9001, 2048), 2, "bf16", False, True),    # one position, groups of over 512 channels: three times 3001 rows
    ((9001, 2048), 2, "f32", True, True),
    ((4500, 4104), 3, "f16", True, False),     # ... that are no whole blocks
    ((13001, 1290), 2, "bf16", False, True),   # ... nor whole vectors
    ((120001, 2, 96), 32, "bf16", False, True),
    ((30011, 3, 512), 512, "f32", True, True),  # as many groups as channels
    ((3001, 5, 2304), 2304, "f16", False, True),
])
def test_some_samples_at_a_time(shape, G, dtype, gate, affine):
    import long_sequence_fft_b200 as lsf
    N, S, C = shape[0], shape[1] if len(shape) == 3 else 1, shape[-1]
    assert lsf.library().fftconv_group_norm_workspace_bytes(N, S, C, G, 1) > 16 << 20
    x = _inputs(shape, dtype, seed=N, gate=gate, affine=affine)
    _check(_run(x, G, "silu"), x, G, "silu", what=f"{shape} G={G} {dtype}")


@pytest.mark.parametrize("shape,G", [((3, 7, 6000), 40), ((2, 5, 4104), 27), ((2, 3, 16384), 16384), ((2, 9, 8200), 1),
                                     ((4, 50, 2056), 257)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [False, True])
def test_groups_across_blocks_of_channels(shape, G, dtype, gate):
    x = _inputs(shape, dtype, seed=G, gate=gate, affine=True)
    _check(_run(x, G, "silu"), x, G, "silu", what=f"{shape} G={G} {dtype}")


def test_some_samples_at_a_time_in_rows_of_wider_tensors():
    """Strides of x, gate and gradient that differ, over several rounds; the
    same call captured; sums that repeat bit for bit."""
    import long_sequence_fft_b200 as lsf
    N, C, G = 9001, 2048, 2
    x = _inputs((N, C), "bf16", seed=3, gate=True, affine=True)
    wide = torch.empty((N, 3, C), device="cuda", dtype=torch.bfloat16)
    wide[:, 0], wide[:, 2] = x["x"], x["gate"]

    def call(whole, w, b):
        y = lsf.group_norm(whole[:, 0], G, w, b, gate=whole[:, 2], activation="silu")
        dy = torch.cat([x["dy"], x["dy"]], 1)[:, :C]
        return [y, *torch.autograd.grad(y, [whole, w, b], dy)]

    leaves = lambda: [t.clone().requires_grad_() for t in (wide, x["weight"], x["bias"])]    # noqa: E731
    got, mine = _run(x, G, "silu"), leaves()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        captured = call(*mine)
    g.replay()
    torch.cuda.synchronize()
    for y, dwide, dw, db in (call(*leaves()), captured):
        for a, e in ((y, "y"), (dwide[:, 0], "dx"), (dwide[:, 2], "dgate"), (dw, "dweight"), (db, "dbias")):
            assert torch.equal(a, got[e]), e


@pytest.mark.parametrize("dtype,size", [("f32", 1e20), ("f32", -3e37), ("bf16", 1e30)])
@pytest.mark.parametrize("shape", [(2, 300, 64), (3, 5, 4104), (2, 6000)])
def test_values_whose_square_overflows(dtype, size, shape):
    """Far from zero, but near to each other: the variance is finite."""
    import long_sequence_fft_b200 as lsf
    x = _inputs(shape, dtype, seed=1, gate=False, affine=True)
    x["x"] = torch.full(shape, size, device="cuda").to(x["x"].dtype)
    got = _run(x, 2, "none")
    assert torch.equal(got["y"], x["bias"].to(got["y"].dtype).expand(shape))
    if dtype == "f32" and size == 1e20:
        # deviations of 1e16: every value is exact to 2^-24 of 1e20, 6e-4 of a deviation
        x["x"] = (1e20 + 1e16 * x["dy"]).float()
        d = x["x"].double() - x["x"].double().reshape(shape[0], -1, 2, shape[-1] // 2).mean((1, 3)).repeat_interleave(
            shape[-1] // 2, 1).reshape(shape[0], *[1] * (len(shape) - 2), shape[-1])
        rstd = 1 / (d.reshape(shape[0], -1, 2, shape[-1] // 2) ** 2).mean((1, 3)).sqrt().repeat_interleave(
            shape[-1] // 2, 1).reshape(shape[0], *[1] * (len(shape) - 2), shape[-1])
        ref = d * rstd
        y = lsf.group_norm(x["x"], 2).double()
        # the mean is off by a few 2^-24 of 1e20 (joined over blocks): 16 of them, in deviations
        assert (y - ref).abs().max() <= 16 * 2.0 ** -24 * 1e4 * 1.1 + 1e-5 * ref.abs().max()


@pytest.mark.parametrize("D,G", [(17, 500000), (16, 800000), (1, 65535 * 256)])
def test_the_most_groups_of_a_launch(D, G):
    """The last group of the widest rows that a launch takes."""
    import long_sequence_fft_b200 as lsf
    x = torch.randn((1, D * G), generator=torch.Generator(device="cuda").manual_seed(D), device="cuda")
    y = lsf.group_norm(x, G)[:, -1024 * D:].double()
    t = x[:, -1024 * D:].double().view(1024, D)
    d = t - t.mean(1, keepdim=True)
    ref = (d / (d * d).mean(1, keepdim=True).add(1e-5).sqrt()).view(1, -1)
    assert (y - ref).abs().max() <= 2.0 ** -20 * 8
