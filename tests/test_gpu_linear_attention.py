"""GPU tests of linear attention (prompt form, backward pass, single-token
form) against its fp64 definition; the bounds are derived in
mixer_reference."""
import math

import pytest

from mixer_reference import attention, check_attention, magnitudes

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _case(B, T, heads, K, V, dtype, seed, n=None, initial=True, decays=None, scale_k=1.0):
    H, Hq, Hk, Hv = heads
    g, dt = _gen(seed), DT[dtype]
    r = lambda *s: torch.randn(s, generator=g, device="cuda")                # noqa: E731
    x = dict(q=r(B, T, Hq, K).to(dt), k=(r(B, T, Hk, K) * scale_k).to(dt), v=r(B, T, Hv, V).to(dt),
             do=r(B, T, H, V).to(dt))
    n = B if n is None else n
    x["initial"] = r(n, H, K, V) if initial else None
    x["dstate"] = r(n, H, K, V)
    if decays is None:
        decays = [-(2.0 ** -(1 + 8 * h / max(1, H - 1))) for h in range(H)]
    x["log_decay"] = torch.tensor(decays, dtype=torch.float32, device="cuda")
    return x


def _status_ok():
    import long_sequence_fft_b200 as lsf
    assert lsf.linear_attention_status() == 0


def _run(x, cu=None, scale=None, grads=True):
    import long_sequence_fft_b200 as lsf
    leaves = {n: x[n].clone().requires_grad_(grads) for n in ("q", "k", "v", "initial") if x[n] is not None}
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, s = lsf.linear_attention(leaves["q"], leaves["k"], leaves["v"], x["log_decay"],
                                initial_state=leaves.get("initial"), cu_seqlens=cud, return_state=True, scale=scale)
    got = {"o": o.detach(), "state": s.detach()}
    if grads:
        for n, gr in zip(leaves, torch.autograd.grad([o, s], list(leaves.values()), [x["do"], x["dstate"]])):
            got["d" + n] = gr
    _status_ok()
    return got


def _both(x, cu=None, scale=None):
    a = scale if scale is not None else x["q"].shape[3] ** -0.5
    args = (x["q"], x["k"], x["v"], x["log_decay"], a, x["initial"], x["do"], x["dstate"], cu)
    return attention(*args), magnitudes(*args)


MHA, KV, QK, ONE = (2, 2, 2, 2), (4, 4, 2, 2), (6, 2, 2, 6), (3, 1, 1, 1)


@pytest.mark.parametrize("B,T,heads,K,V,dtype", [
    (1, 1, MHA, 64, 64, "bf16"),            # one token
    (2, 15, MHA, 8, 8, "f16"),              # below one MMA step, smallest widths
    (1, 128, MHA, 64, 64, "f16"),           # exactly one tile
    (2, 129, KV, 64, 128, "bf16"),          # one token past a tile, keys and values shared
    (1, 300, QK, 128, 64, "f16"),           # queries and keys shared
    (3, 257, ONE, 128, 128, "bf16"),        # everything shared
    (1, 517, MHA, 40, 72, "bf16"),          # widths inside a tile
    (2, 255, KV, 120, 104, "f16"),
    (1, 1030, MHA, 128, 128, "f16"),
])
@pytest.mark.parametrize("initial", [False, True])
def test_forward_and_gradients(B, T, heads, K, V, dtype, initial):
    x = _case(B, T, heads, K, V, dtype, seed=T + K + V, initial=initial)
    ref, mag = _both(x)
    check_attention(_run(x), ref, mag, DT[dtype], f"B={B} T={T} heads={heads} K={K} V={V}")


@pytest.mark.parametrize("T,heads,K,V,dtype", [
    (4100, (1, 1, 1, 1), 64, 64, "bf16"),   # few heads: the sequence is cut along time
    (5000, (2, 2, 1, 1), 128, 128, "bf16"),
    (3333, (2, 1, 1, 2), 128, 64, "f16"),
])
def test_long_sequences_cut_along_time(T, heads, K, V, dtype):
    x = _case(1, T, heads, K, V, dtype, seed=T)
    ref, mag = _both(x)
    check_attention(_run(x), ref, mag, DT[dtype], f"T={T}")


@pytest.mark.parametrize("lens,heads,K,V,dtype", [
    ([1, 200, 0, 128, 371], MHA, 64, 64, "bf16"),
    ([0, 0, 5], MHA, 64, 128, "f16"),
    ([130, 1, 127, 129], KV, 128, 128, "f16"),
    ([3000, 7, 2500, 1], (1, 1, 1, 1), 64, 64, "bf16"),
    ([3] * 70, QK, 24, 16, "bf16"),
])
def test_packed_sequences(lens, heads, K, V, dtype):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = _case(1, cu[-1], heads, K, V, dtype, seed=sum(lens), n=len(lens))
    ref, mag = _both(x, cu)
    check_attention(_run(x, cu), ref, mag, DT[dtype], f"lens={lens[:6]}")


@pytest.mark.parametrize("heads", [(5, 5, 5, 5), (6, 2, 2, 6)])
@pytest.mark.parametrize("K,V", [(128, 64), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_mixed_widths_that_fill_the_gpu(heads, K, V, dtype):
    """More sequences and heads than SMs: the three gradients come from two
    launches of different widths."""
    x = _case(10, 600, heads, K, V, dtype, seed=K + heads[1])
    ref, mag = _both(x)
    check_attention(_run(x), ref, mag, DT[dtype], f"K={K} V={V}")


@pytest.mark.parametrize("K,V", [(128, 64), (64, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_repeats_wait_for_nothing(K, V, dtype):
    """Long walks on every SM, many times over: no bounded wait may give up, and
    the results stay the same."""
    import long_sequence_fft_b200 as lsf
    x = _case(8, 2048, (12, 12, 12, 12), K, V, dtype, seed=1, initial=False)
    leaves = [x[n].requires_grad_() for n in "qkv"]
    want = None
    for _ in range(25):
        o = lsf.linear_attention(*leaves, x["log_decay"])
        got = [o.detach(), *torch.autograd.grad(o, leaves, x["do"])]
        if want is None:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _status_ok()


@pytest.mark.parametrize("lens,heads,K,V,dtype", [
    ([40] * 33 + [1700, 0, 900] + [5] * 10 + [641], KV, 128, 128, "bf16"),
    ([1300, 1, 0, 513, 512, 511, 1024, 256, 257] + [9] * 30, MHA, 64, 128, "f16"),
    ([700, 2048, 33, 0, 1535], QK, 128, 64, "bf16"),
])
def test_packed_sequences_cut_along_time(lens, heads, K, V, dtype):
    """Long and brief pieces of many sequences, in the order of their lengths."""
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = _case(1, cu[-1], heads, K, V, dtype, seed=len(lens), n=len(lens))
    ref, mag = _both(x, cu)
    check_attention(_run(x, cu), ref, mag, DT[dtype], f"lens={lens[:6]}")


@pytest.mark.parametrize("T,cu", [(300, None), (3000, None), (3000, [0, 700, 700, 2900, 3000])])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_final_states_in_place_of_initial_ones(T, cu, K, V):
    """The C interface lets final_state be initial_state itself, for sequences
    in one piece and for those cut along time."""
    import ctypes

    import long_sequence_fft_b200 as lsf
    from long_sequence_fft_b200.linear_attention import _Shape
    n = 1 if cu is None else len(cu) - 1
    x = _case(1, T, MHA, K, V, "bf16", seed=T, n=n)
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    want, state = lsf.linear_attention(x["q"], x["k"], x["v"], x["log_decay"], initial_state=x["initial"],
                                       cu_seqlens=cud, return_state=True)
    o, both = torch.empty_like(want), x["initial"].clone()
    H = 2
    rows = lambda d: (T * H * d, H * d, d)                                   # noqa: E731
    shape = _Shape(1, T, 0 if cu is None else n, H, H, H, H, K, V, lsf.BF16, K ** -0.5, 1, rows(K), rows(K), rows(V),
                   rows(V))
    lib = lsf.library()
    size = lib.fftconv_linear_attention_workspace_bytes(ctypes.byref(shape), 0)
    assert (size > 0) == (T > 1000)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    rc = lib.fftconv_linear_attention(ctypes.byref(shape), x["q"].data_ptr(), x["k"].data_ptr(), x["v"].data_ptr(),
                                      x["log_decay"].data_ptr(), both.data_ptr(),
                                      None if cud is None else cud.data_ptr(), o.data_ptr(), both.data_ptr(),
                                      ws.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    _status_ok()
    assert torch.equal(o, want) and torch.equal(both, state)


def test_rows_outside_packed_sequences():
    """Tokens in front of and behind the packed sequences: unused whatever they
    hold (NaN here, in inputs and gradients), zero in new outputs and
    gradients, left as they were in `out`."""
    import long_sequence_fft_b200 as lsf
    cu, T = [5, 105, 105, 250], 300
    for heads in (MHA, KV):
        x = _case(1, T, heads, 64, 64, "bf16", seed=9, n=3)
        clean = _run(x, cu)
        bad = dict(x)
        for name in ("q", "k", "v", "do"):
            bad[name] = x[name].clone()
            bad[name][:, :5] = float("nan")
            bad[name][:, 250:] = float("inf")
        got = _run(bad, cu)
        for name in got:
            assert torch.equal(got[name], clean[name]), name
        for name in ("o", "dq", "dk", "dv"):
            assert not got[name][:, :5].any() and not got[name][:, 250:].any(), name
        out = torch.full_like(got["o"], 7.0)
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        # (with the state asked for, as in the run it is compared with: without
        # it the carried state is a 16-bit quantity only)
        lsf.linear_attention(bad["q"], bad["k"], bad["v"], x["log_decay"], initial_state=x["initial"], cu_seqlens=cud,
                             return_state=True, out=out)
        assert torch.equal(out[:, 5:250], got["o"][:, 5:250])
        assert (out[:, :5] == 7.0).all() and (out[:, 250:] == 7.0).all()


def test_packed_neighbours_do_not_leak():
    """A sequence of NaN between two others, inside their tiles."""
    cu = [0, 70, 140, 200]
    x = _case(1, 200, MHA, 64, 128, "f16", seed=4, n=3)
    clean = _run(x, cu)
    for name in ("q", "k", "v", "do"):
        x[name][:, 70:140] = float("nan")
    got = _run(x, cu)
    for name in ("o", "dq", "dk", "dv"):
        assert torch.equal(got[name][:, :70], clean[name][:, :70]), name
        assert torch.equal(got[name][:, 140:], clean[name][:, 140:]), name
    for name in ("state", "dinitial"):
        assert torch.equal(got[name][[0, 2]], clean[name][[0, 2]]), name


def test_offsets_out_of_range_are_clamped():
    import long_sequence_fft_b200 as lsf
    x = _case(1, 200, MHA, 64, 64, "bf16", seed=2, n=2, initial=False)
    cu = torch.tensor([-50, 100, 1 << 30], dtype=torch.int32, device="cuda")
    o = lsf.linear_attention(x["q"], x["k"], x["v"], x["log_decay"], cu_seqlens=cu)
    ref = lsf.linear_attention(x["q"], x["k"], x["v"], x["log_decay"],
                               cu_seqlens=torch.tensor([0, 100, 200], dtype=torch.int32, device="cuda"))
    assert torch.equal(o, ref)
    _status_ok()


@pytest.mark.parametrize("decays", [[0.0, -1e-6], [-float("inf"), -200.0], [-30.0, -5.0]])
def test_extreme_decays(decays):
    """No decay at all, decays that underflow inside a tile, and no memory
    (-inf: o_t = a (q_t . k_t) v_t)."""
    x = _case(1, 400, MHA, 64, 64, "bf16", seed=11, decays=decays)
    ref, mag = _both(x)
    check_attention(_run(x), ref, mag, torch.bfloat16, f"decays={decays}")


@pytest.mark.parametrize("size", [1e-4, 300.0])
def test_fp16_ranges(size):
    """Keys whose weighted products leave fp16's range on either side: scaled
    by exact powers of two inside, so the bounds are the usual ones."""
    x = _case(1, 300, MHA, 64, 64, "f16", seed=13, scale_k=size)
    x["v"] = (x["v"] / size).half()
    x["do"] = (x["do"] / 64).half()
    x["dstate"] = x["dstate"] / 64
    x["initial"] = x["initial"] * 1e3
    ref, mag = _both(x)
    got = _run(x)
    # an output below fp16's normal range is off by half a subnormal step
    check_attention({n: t for n, t in got.items() if n != "dv" or size > 1}, ref, mag, torch.float16, f"size={size}")


def test_strided_inputs_and_outputs():
    """q, k and v as slices of one projection, the output into a slice."""
    import long_sequence_fft_b200 as lsf
    g = _gen(21)
    B, T, H, D = 2, 190, 3, 64
    qkv = torch.randn((B, T, 3, H, D), generator=g, device="cuda").bfloat16()
    ld = torch.full((H,), -0.05, device="cuda")
    q, k, v = qkv.unbind(2)
    wide = torch.full((B, T, H, 2, D), 3.0, device="cuda").bfloat16()
    o = lsf.linear_attention(q, k, v, ld, out=wide[:, :, :, 1])
    ref = lsf.linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), ld)
    assert torch.equal(o, ref) and torch.equal(wide[:, :, :, 1], ref) and (wide[:, :, :, 0] == 3.0).all()
    # heads in front of tokens
    t = lambda a: a.transpose(1, 2).contiguous().transpose(1, 2)             # noqa: E731
    assert torch.equal(lsf.linear_attention(t(q), t(k), t(v), ld), ref)


def test_a_prompt_in_two_calls_and_then_single_tokens():
    """The state carries on: prompt halves, then steps, against the whole
    prompt's outputs and state."""
    import long_sequence_fft_b200 as lsf
    x = _case(2, 150, KV, 64, 128, "bf16", seed=5)
    ref, mag = _both(x)
    q, k, v, ld = x["q"], x["k"], x["v"], x["log_decay"]
    o1, s = lsf.linear_attention(q[:, :77], k[:, :77], v[:, :77], ld, initial_state=x["initial"], return_state=True)
    o2, s = lsf.linear_attention(q[:, 77:140], k[:, 77:140], v[:, 77:140], ld, initial_state=s, return_state=True)
    steps = [lsf.linear_attention_step(q[:, t], k[:, t], v[:, t], ld, s) for t in range(140, 150)]
    o = torch.cat([o1, o2, torch.stack(steps, 1)], 1)
    check_attention({"o": o, "state": s}, ref, mag, torch.bfloat16, "carried")


@pytest.mark.parametrize("B,heads,K,V,dtype", [
    (1, (1, 1, 1, 1), 8, 8, "bf16"), (3, KV, 64, 128, "f16"), (5, QK, 128, 72, "bf16"), (2, ONE, 40, 24, "f16"),
    (37, MHA, 128, 128, "bf16"),
])
@pytest.mark.parametrize("pooled", [False, True])
def test_step(B, heads, K, V, dtype, pooled):
    import long_sequence_fft_b200 as lsf
    x = _case(B, 1, heads, K, V, dtype, seed=B + K)
    ref, mag = _both(x)
    s = x["initial"].clone()
    slots = None
    if pooled:
        pool = torch.full((B + 4,) + s.shape[1:], 5.0, device="cuda")
        slots = torch.randperm(B + 4, generator=_gen(1), device="cuda")[:B].to(torch.int32)
        pool[slots.long()] = s
        s = pool
    o = lsf.linear_attention_step(x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["log_decay"], s, slots=slots)
    state = s if slots is None else s[slots.long()]
    # every product and sum is fp32: the output's own rounding, and 2^-15 M for the sums
    u = torch.finfo(DT[dtype]).eps / 2
    err = (o.double() - ref["o"][:, 0]).abs()
    assert (err <= u * ref["o"][:, 0].abs() + 2.0 ** -15 * mag["o"][:, 0]).all()
    assert ((state.double() - ref["state"]).abs() <= 2.0 ** -18 * mag["state"]).all()
    if pooled:
        rest = torch.ones(B + 4, dtype=torch.bool, device="cuda")
        rest[slots.long()] = False
        assert (s[rest] == 5.0).all()


def test_step_idle_rows():
    """Slots outside the pool, and a slot that an earlier row names already:
    zero output, no state touched; the first row of a slot counts."""
    import long_sequence_fft_b200 as lsf
    x = _case(6, 1, MHA, 64, 64, "bf16", seed=3)
    pool = torch.randn((4, 2, 64, 64), generator=_gen(8), device="cuda")
    slots = torch.tensor([2, -1, 0, 2, 4, 1 << 30], dtype=torch.int32, device="cuda")
    new = pool.clone()
    a = (x["q"][:, 0], x["k"][:, 0], x["v"][:, 0], x["log_decay"])
    o = lsf.linear_attention_step(*a, new, slots=slots, out=torch.full((6, 2, 64), 9.0, device="cuda").bfloat16())
    assert not o[[1, 3, 4, 5]].any()
    both = pool[[2, 0]].clone()
    oo = lsf.linear_attention_step(*(t[[0, 2]] for t in a[:3]), a[3], both)
    assert torch.equal(o[[0, 2]], oo) and torch.equal(new[[2, 0]], both)
    assert torch.equal(new[[1, 3]], pool[[1, 3]])


def test_repeats_bit_for_bit_and_empty_calls():
    import long_sequence_fft_b200 as lsf
    x = _case(1, 2000, (4, 2, 2, 4), 64, 64, "f16", seed=6)
    a, b = _run(x), _run(x)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    e = _case(2, 0, MHA, 64, 64, "f16", seed=1)
    got = _run(e)
    assert got["o"].shape == (2, 0, 2, 64)
    assert torch.equal(got["state"], e["initial"]) and torch.equal(got["dinitial"], e["dstate"])
    z = _case(0, 10, MHA, 64, 64, "f16", seed=1)
    assert _run(z)["o"].shape == (0, 10, 2, 64)
    s = torch.zeros((0, 2, 64, 64), device="cuda")
    assert lsf.linear_attention_step(z["q"][:, 0], z["k"][:, 0], z["v"][:, 0], z["log_decay"], s).shape == (0, 2, 64)


def test_gradients_against_differences():
    """The kernel's gradients along random directions against central
    differences of the fp64 definition (its own truncation: the loss is
    trilinear in q, k and v, so a difference in one of them is exact)."""
    x = _case(1, 260, KV, 64, 64, "f16", seed=17)
    got = _run(x)

    def loss(**change):
        y = {**x, **change}
        r = attention(y["q"], y["k"], y["v"], y["log_decay"], 0.125, y["initial"])
        return ((r["o"] * x["do"].double()).sum() + (r["state"] * x["dstate"].double()).sum()).item()

    for name in ("q", "k", "v", "initial"):
        d = torch.randn(x[name].shape, generator=_gen(len(name)), device="cuda").double()
        fd = (loss(**{name: x[name].double() + d}) - loss(**{name: x[name].double() - d})) / 2
        an = (got["d" + name].double() * d).sum().item()
        # the roundings of n gradients, each within 2u of its value's scale,
        # add up like a random walk against the directions
        size = (got["d" + name].double() ** 2).sum().sqrt().item()
        assert abs(fd - an) <= 6 * 2 * 2.0 ** -11 * size + 1e-3, (name, fd, an)


def test_autograd_layouts_and_partial_gradients():
    """An expanded gradient (from a sum), a transposed one, only some leaves,
    no gradient for the state, and the state's alone."""
    import long_sequence_fft_b200 as lsf
    x = _case(2, 140, KV, 64, 64, "bf16", seed=19)
    q, k, v = (x[n].clone().requires_grad_() for n in "qkv")
    lsf.linear_attention(q, k, v, x["log_decay"]).sum().backward()
    ones = torch.ones_like(x["do"])
    args = (x["q"], x["k"], x["v"], x["log_decay"], 0.125, None, ones, None)
    ref, mag = attention(*args), magnitudes(*args)
    check_attention({"dq": q.grad, "dk": k.grad, "dv": v.grad}, ref, mag, torch.bfloat16, "sum")
    o = lsf.linear_attention(x["q"], k, x["v"], x["log_decay"])
    do = x["do"].transpose(1, 2).contiguous().transpose(1, 2)
    g1, = torch.autograd.grad(o, k, do)
    o = lsf.linear_attention(x["q"], k, x["v"], x["log_decay"])
    g2, = torch.autograd.grad(o, k, x["do"])
    assert torch.equal(g1, g2)
    o, s = lsf.linear_attention(x["q"], k, x["v"], x["log_decay"], return_state=True)
    gs, = torch.autograd.grad(s, k, x["dstate"])
    args = (x["q"], x["k"], x["v"], x["log_decay"], 0.125, None, 0 * x["do"], x["dstate"])
    check_attention({"dk": gs}, attention(*args), magnitudes(*args), torch.bfloat16, "state only")


def test_streams_and_graphs():
    """Another stream than the current one; a captured call replayed on new
    inputs, with its backward pass; two graphs at once."""
    import long_sequence_fft_b200 as lsf
    x = _case(1, 3000, (2, 2, 2, 2), 64, 64, "bf16", seed=23)
    a = (x["q"], x["k"], x["v"], x["log_decay"])
    ref = lsf.linear_attention(*a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lsf.linear_attention(*a, stream=side)
    raw = lsf.linear_attention(*a, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, ref) and torch.equal(raw, ref)

    graphs = []
    for _ in range(2):
        leaves = [t.clone().requires_grad_() for t in a[:3]]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            o = lsf.linear_attention(*leaves, a[3])
            grads = torch.autograd.grad(o, leaves, x["do"])
        graphs.append((g, leaves, o, grads))
    y = _case(1, 3000, (2, 2, 2, 2), 64, 64, "bf16", seed=24)
    with torch.no_grad():
        for t, n in zip(graphs[0][1], "qkv"):
            t.copy_(y[n])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[1][0].replay()
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for (g, leaves, o, grads), src in zip(graphs, (y, x)):
        args = (src["q"], src["k"], src["v"], a[3], 0.125, None, x["do"], None)
        check_attention(dict(o=o.detach(), dq=grads[0], dk=grads[1], dv=grads[2]), attention(*args), magnitudes(*args),
                        torch.bfloat16, "replayed")
    _status_ok()


def test_captured_packed_call_with_other_offsets():
    """The segments are planned on the device: a captured call takes the
    offsets that it finds when it is replayed, and two graphs run at once."""
    import long_sequence_fft_b200 as lsf
    T = 4000
    x = _case(1, T, KV, 64, 64, "bf16", seed=31, n=4, initial=False)
    first, other = [0, 100, 3000, 3001, 4000], [0, 1700, 1700, 1764, 3999]
    graphs = []
    for _ in range(2):
        cu = torch.tensor(first, dtype=torch.int32, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            o, s = lsf.linear_attention(x["q"], x["k"], x["v"], x["log_decay"], cu_seqlens=cu, return_state=True)
        graphs.append((g, cu, o, s))
    graphs[1][1].copy_(torch.tensor(other, dtype=torch.int32))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graphs[0][0].replay()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    for (_, _, o, s), offsets in zip(graphs, (first, other)):
        want, state = lsf.linear_attention(x["q"], x["k"], x["v"], x["log_decay"], return_state=True,
                                           cu_seqlens=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        assert torch.equal(o, want) and torch.equal(s, state)
    _status_ok()


def test_more_sequences_than_one_look_of_the_plan():
    """Over 1024 sequences, some cut, against the same ones one by one."""
    import long_sequence_fft_b200 as lsf
    lens = ([3] * 700 + [1500] + [0, 17]) * 2
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    x = _case(1, cu[-1], MHA, 64, 64, "bf16", seed=5, n=len(lens))
    got = _run(x, cu)
    ref, mag = _both(x, cu)
    check_attention(got, ref, mag, torch.bfloat16, "many sequences")
    o, s = lsf.linear_attention(x["q"], x["k"], x["v"], x["log_decay"], initial_state=x["initial"], return_state=True,
                                cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert torch.equal(o, got["o"]) and torch.equal(s, got["state"])


def test_refusals():
    import long_sequence_fft_b200 as lsf
    x = _case(1, 64, MHA, 64, 64, "bf16", seed=1)
    q, k, v, ld = x["q"], x["k"], x["v"], x["log_decay"]
    bad = lambda e, *a, **kw: pytest.raises(e, lsf.linear_attention, *a, **kw)  # noqa: E731
    bad(ValueError, q.float(), k, v, ld)
    bad(ValueError, q, k.half(), v, ld)
    bad(ValueError, q, k[:, :32], v, ld)
    bad(ValueError, q.cpu(), k, v, ld)
    bad(ValueError, q, k, v.cpu(), ld)
    bad(ValueError, q, k, v, ld.cpu())
    bad(ValueError, q, k, v, ld.half())
    bad(ValueError, q, k, v, torch.zeros(3, device="cuda"))                  # 2 heads do not divide 3
    bad(ValueError, q[..., ::2], k[..., ::2], v, ld)                         # last index strided
    bad(ValueError, q[:, :1].expand(1, 64, 2, 64), k, v, ld)                 # expanded
    bad(ValueError, q, k, v, ld, initial_state=torch.zeros((1, 2, 64, 64), device="cuda").half())
    bad(ValueError, q, k, v, ld, initial_state=torch.zeros((2, 2, 64, 64), device="cuda"))
    bad(ValueError, q, k, v, ld, cu_seqlens=torch.tensor([0, 64], device="cuda"))            # int64
    bad(ValueError, q, k, v, ld, cu_seqlens=torch.tensor([0], dtype=torch.int32, device="cuda"))
    bad(ValueError, q, k, v, ld, out=torch.zeros((1, 64, 2, 32), device="cuda").bfloat16())
    with pytest.raises(NotImplementedError):
        lsf.linear_attention(q, k, v, ld.clone().requires_grad_())
    with pytest.raises(NotImplementedError):
        lsf.linear_attention(q.clone().requires_grad_(), k, v, ld, out=torch.empty_like(v))
    r = lambda *s: torch.zeros(s, device="cuda").bfloat16()                  # noqa: E731
    for K, V in ((136, 64), (64, 136), (12, 64), (64, 20)):
        with pytest.raises((lsf.FFTConvError, ValueError)):
            lsf.linear_attention(r(1, 8, 1, K), r(1, 8, 1, K), r(1, 8, 1, V), ld[:1].contiguous())
    b2 = r(2, 8, 2, 64)
    bad(ValueError, b2, b2, b2, ld, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32, device="cuda"))
    with pytest.raises(lsf.FFTConvError):
        lsf.linear_attention(q, k, v, ld, out=q)                             # overlaps an input
    s = torch.zeros((1, 2, 64, 64), device="cuda")
    step = (q[:, 0], k[:, 0], v[:, 0], ld)
    for state, kw in ((s.half(), {}), (s[:, :1], {}), (s, {"slots": torch.zeros(1, device="cuda")}),
                      (s.expand(2, 2, 64, 64), {})):
        with pytest.raises(ValueError):
            lsf.linear_attention_step(*step, state, **kw)
    with pytest.raises(NotImplementedError):
        lsf.linear_attention_step(q[:, 0].clone().requires_grad_(), *step[1:], s)
    assert math.isfinite(float(lsf.linear_attention(q, k, v, ld).float().sum()))
