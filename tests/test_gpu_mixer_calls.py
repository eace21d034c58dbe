"""GPU tests of how torch calls linear attention and group norm: gradients as
autograd hands them out, tensors that are saved and written, derivatives that
the operators do not have."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(seed, *shape):
    return torch.randn(shape, generator=_gen(seed), device="cuda")


def _behind(t, n):
    """t flattened behind n other values: the gradient of t is a contiguous
    piece of the whole's gradient, n elements from its start."""
    return torch.cat([t.new_zeros(n), t.flatten()])


@pytest.mark.parametrize("shape,G,dtype", [((3, 35), 7, "float32"), ((5, 64), 4, "bfloat16"),
                                           ((2, 30, 48), 4, "float16"), ((40, 256), 2, "float32")])
@pytest.mark.parametrize("n", [1, 3])
def test_norm_gradient_at_any_address(shape, G, dtype, n):
    import long_sequence_fft_b200 as lsf
    dt = getattr(torch, dtype)
    C = shape[-1]
    leaves = [_randn(1, *shape).to(dt), (1 + 0.1 * _randn(2, C)).to(dt), _randn(3, C).to(dt), _randn(4, *shape).to(dt)]
    leaves = [t.requires_grad_() for t in leaves]

    def call():
        return lsf.group_norm(leaves[0], G, leaves[1], leaves[2], gate=leaves[3], activation="silu")

    dy = _randn(5, *shape).to(dt)
    want = torch.autograd.grad(call(), leaves, dy)
    got = torch.autograd.grad(_behind(call(), n), leaves, _behind(dy, n))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("cu", [None, [0, 50, 50, 130]])
@pytest.mark.parametrize("n", [1, 3])
def test_attention_gradients_at_any_address(cu, n):
    """Of the outputs, of the final states, and of both."""
    import long_sequence_fft_b200 as lsf
    B, T, H, K, V = (1 if cu else 2), 130, 2, 64, 40
    seqs = len(cu) - 1 if cu else B
    leaves = [_randn(1, B, T, H, K).bfloat16(), _randn(2, B, T, H, K).bfloat16(), _randn(3, B, T, H, V).bfloat16(),
              _randn(4, seqs, H, K, V)]
    leaves = [t.requires_grad_() for t in leaves]
    ld = torch.tensor([-0.3, -0.01], device="cuda")
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")

    def call():
        return lsf.linear_attention(*leaves[:3], ld, initial_state=leaves[3], cu_seqlens=cud, return_state=True)

    do, ds = _randn(5, B, T, H, V).bfloat16(), _randn(6, seqs, H, K, V)
    want = torch.autograd.grad(call(), leaves, (do, ds))
    o, s = call()
    got = torch.autograd.grad((_behind(o, n), _behind(s, n)), leaves, (_behind(do, n), _behind(ds, n)))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_backward_through_an_overwritten_tensor_raises():
    """What a call writes in place counts as written: a backward pass that
    saved it must not go on with other values."""
    import long_sequence_fft_b200 as lsf
    q, k, v = (_randn(i, 1, 20, 2, 64).bfloat16() for i in range(3))
    ld = torch.tensor([-0.3, -0.01], device="cuda")
    step = (q[:, 0], k[:, 0], v[:, 0], ld)
    state = _randn(5, 1, 2, 64, 64)

    def saved_by_attention():
        return lsf.linear_attention(q.clone().requires_grad_(), k, v, ld, initial_state=state)

    o = saved_by_attention()
    o.sum().backward()                                       # (nothing written in between)
    o = saved_by_attention()
    before = state._version
    lsf.linear_attention_step(*step, state)
    assert state._version > before
    with pytest.raises(RuntimeError, match="inplace operation"):
        o.sum().backward()
    # a pool, through a view of it
    pool = _randn(6, 3, 2, 64, 64)
    o = lsf.linear_attention(q.clone().requires_grad_(), k, v, ld, initial_state=pool[1:2])
    lsf.linear_attention_step(*step, pool, slots=torch.tensor([1], dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError, match="inplace operation"):
        o.sum().backward()

    # out= of each operator, saved by a product
    w = torch.ones((), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    x = _randn(7, 20, 128).bfloat16()
    for out, call in ((torch.zeros((1, 20, 2, 64), device="cuda", dtype=torch.bfloat16),
                       lambda out: lsf.linear_attention(q, k, v, ld, out=out)),
                      (torch.zeros((1, 2, 64), device="cuda", dtype=torch.bfloat16),
                       lambda out: lsf.linear_attention_step(*step, state, out=out)),
                      (torch.zeros((20, 128), device="cuda", dtype=torch.bfloat16),
                       lambda out: lsf.group_norm(x, 4, out=out))):
        y = out * w
        assert call(out) is out
        with pytest.raises(RuntimeError, match="inplace operation"):
            y.sum().backward()


def test_inference_mode():
    """Tensors without a version, and ordinary ones written in inference mode."""
    import long_sequence_fft_b200 as lsf
    ordinary = torch.zeros((1, 2, 64, 64), device="cuda")
    with torch.inference_mode():
        q, k, v = (_randn(i, 1, 20, 2, 64).bfloat16() for i in range(3))
        ld = torch.tensor([-0.3, -0.01], device="cuda")
        o, state = lsf.linear_attention(q, k, v, ld, return_state=True, out=torch.empty_like(q))
        for s in (state, ordinary):
            o = lsf.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], ld, s, out=torch.empty_like(q[:, 0]))
        x = o.view(1, 128)
        y = lsf.group_norm(x, 2, out=torch.empty_like(x))
    assert torch.isfinite(y).all() and ordinary.any()


def test_forward_mode_derivatives_are_refused():
    """A dual tensor in any place raises, with and without reverse mode; inside
    a level, tensors without tangents are computed as ever."""
    from torch.autograd import forward_ad

    import long_sequence_fft_b200 as lsf
    q, k, v = (_randn(i, 1, 20, 2, 64).bfloat16() for i in range(3))
    ld, s = torch.tensor([-0.3, -0.01], device="cuda"), _randn(4, 1, 2, 64, 64)
    x, gate, w, b = _randn(5, 6, 64), _randn(6, 6, 64), _randn(7, 64), _randn(8, 64)
    calls = [
        (lambda q, k, v, ld, s: lsf.linear_attention(q, k, v, ld, initial_state=s), [q, k, v, ld, s]),
        (lambda q, k, v, ld, s: lsf.linear_attention_step(q, k, v, ld, s), [q[:, 0], k[:, 0], v[:, 0], ld, s.clone()]),
        (lambda x, gate, w, b: lsf.group_norm(x, 4, w, b, gate=gate), [x, gate, w, b]),
    ]
    for call, args in calls:
        want = call(*[a.clone() for a in args])
        with forward_ad.dual_level():
            assert torch.equal(call(*[a.clone() for a in args]), want)
            for i, a in enumerate(args):
                dual = list(args)
                dual[i] = forward_ad.make_dual(a, torch.ones_like(a))
                with pytest.raises(NotImplementedError):
                    call(*dual)
                with torch.no_grad(), pytest.raises(NotImplementedError):
                    call(*dual)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x.clone().requires_grad_(), torch.ones_like(x))
        with pytest.raises(NotImplementedError):
            lsf.group_norm(dual, 4)


def test_packed_training_batch_of_many_short_sequences():
    """What a call takes beside its tensors does not grow with the number of
    sequences; the gradients are those of the sequences one by one."""
    import long_sequence_fft_b200 as lsf
    lens = [64] * 500 + [3000] + [1] * 40
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T, H, D = cu[-1], 16, 128
    q, k, v, do = (_randn(i, 1, T, H, D).bfloat16() for i in range(4))
    ld = torch.linspace(-0.3, -0.001, H, device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v)]
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    o = lsf.linear_attention(*leaves, ld, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    got = torch.autograd.grad(o, leaves, do)
    torch.cuda.synchronize()
    # the output, three gradients, and states of a few segments (541 would be 1.7 GB)
    assert torch.cuda.max_memory_allocated() - held < 4 * q.numel() * 2 + (100 << 20)
    for i in (0, 499, 500, 540):
        a, e = cu[i], cu[i + 1]
        part = [t[:, a:e].detach().clone().requires_grad_() for t in leaves]
        one = lsf.linear_attention(*part, ld)
        for x, y in zip([o, *got], [one, *torch.autograd.grad(one, part, do[:, a:e].contiguous())]):
            x, y = x[:, a:e].double(), y.double()
            # two roundings of each side (mixer_reference)
            assert ((x - y).norm() / y.norm()).item() <= 2 * 0.85 * 2.0 ** -8
    assert lsf.linear_attention_status() == 0


def test_offsets_that_decrease():
    """Not a meaning, but no access outside either: the workspace's lists keep
    their bounds, and a call after it is right."""
    import long_sequence_fft_b200 as lsf
    T, H = 6000, 2
    q, k, v = (_randn(i, 1, T, H, 64).bfloat16() for i in range(3))
    ld = torch.tensor([-0.3, -0.01], device="cuda")
    good = torch.tensor([0, 3000, 3100, 6000], dtype=torch.int32, device="cuda")
    want = lsf.linear_attention(q, k, v, ld, cu_seqlens=good, return_state=True)
    for bad in ([0, 6000, 0, 6000], [5000, 100, 6000, 0], [0, 6000] * 40, [6000, 0] * 30):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, s = lsf.linear_attention(q, k, v, ld, cu_seqlens=cu, return_state=True)
        assert o.shape == v.shape and s.shape[0] == len(bad) - 1
        assert lsf.linear_attention_status() == 0
    for a, b in zip(lsf.linear_attention(q, k, v, ld, cu_seqlens=good, return_state=True), want):
        assert torch.equal(a, b)


def test_a_failed_call_leaves_nothing_behind():
    """The error of one call (here: a plan that finds no memory) is not the next
    one's, of any operator."""
    import long_sequence_fft_b200 as lsf
    q, k, v, do = (_randn(i, 1, 300, 4, 64).bfloat16() for i in range(4))
    k2, v2 = k[:, :, :2], v[:, :, :2]
    ld, x = torch.full((4,), -0.1, device="cuda"), _randn(5, 6, 64)
    big = _randn(6, 2, 300, 64)
    cu = torch.tensor([10, 100, 200], dtype=torch.int32, device="cuda")

    def fail():
        torch.cuda.empty_cache()
        free, _ = torch.cuda.mem_get_info()
        for spare in (256, 320, 384, 448):                   # (what cannot be had in one piece)
            try:
                hold = torch.empty(free - (spare << 20), dtype=torch.uint8, device="cuda")
                break
            except torch.cuda.OutOfMemoryError:
                hold = None
        if hold is None:
            pytest.skip("the device's memory cannot be held")
        with pytest.raises(lsf.FFTConvError):
            lsf.Plan(1 << 20, 2, "bf16", order=5)            # (its workspace: 512 MB)
        del hold
        torch.cuda.empty_cache()

    def train(f, *leaves):
        leaves = [t.clone().requires_grad_() for t in leaves]
        y = f(*leaves)
        torch.autograd.grad(y, leaves, torch.ones_like(y))

    for call in (lambda: lsf.group_norm(x, 4), lambda: lsf.group_norm(big, 4),
                 lambda: train(lambda x: lsf.group_norm(x, 4), x),
                 lambda: lsf.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], ld, torch.zeros((1, 4, 64, 64), device="cuda")),
                 lambda: lsf.linear_attention(q, k, v, ld), lambda: lsf.linear_attention(q, k, v, ld, cu_seqlens=cu),
                 lambda: train(lambda q, k, v: lsf.linear_attention(q, k, v, ld), q, k2, v2),
                 lambda: lsf.linear_attention_status()):
        fail()
        call()
    fail()
    assert lsf.linear_attention_status() == 0


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("log_decay,T,scale", [(1.0, 60, 1e-25), (0.8, 90, 1e-30), (0.69, 128, 1e-37), (2.0, 44, 1e-37),
                                               (0.05, 300, 1e-5)])
def test_growth(dtype, log_decay, T, scale):
    """g above 1: powers that leave fp32's range behind the last token do not
    reach it, and weights above 1 count in fp16's scales."""
    import long_sequence_fft_b200 as lsf
    from mixer_reference import attention, magnitudes
    dt = getattr(torch, dtype)
    x = [_randn(i, 1, T, 2, 64).to(dt) for i in range(4)]
    ld = torch.tensor([log_decay, -0.1], device="cuda")
    leaves = [t.clone().requires_grad_() for t in x[:3]]
    o = lsf.linear_attention(*leaves, ld, scale=scale)
    got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(o, leaves, x[3])), o=o.detach())
    args = (*x[:3], ld, scale, None, x[3], None)
    ref, mag = attention(*args), magnitudes(*args)
    # The growing head's (the other one's are below the type's normal range),
    # element by element as in mixer_reference.  Its 2-norm is no statistic
    # here: with g = 2 the last row holds most of it, and in that row two terms
    # P_ij v_j, whose P_ij (one rounding, up to u) all 64 channels share: up to
    # u + u for the norm as for an element.
    u = torch.finfo(dt).eps / 2
    for n, t in got.items():
        r, m = ref[n][:, :, :1], mag[n][:, :, :1]
        bound = u * r.abs() + (u + 2.0 ** -15) * m + torch.finfo(dt).smallest_normal * u
        assert ((t[:, :, :1].double() - r).abs() <= bound).all(), n


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("B,T,H,Hk,K,V,cu", [(1, 1, 1, 1, 128, 128, None), (3, 1, 6, 6, 64, 128, None),
                                             (2, 5, 4, 2, 128, 64, None), (1, 19, 3, 1, 64, 64, [0, 2, 4, 4, 10, 19]),
                                             (1, 128, 2, 2, 40, 72, None), (9, 33, 2, 1, 128, 128, None),
                                             (2, 77, 2, 2, 24, 120, None)])
@pytest.mark.parametrize("state_in,state_out", [(False, False), (True, False), (True, True), (False, True)])
def test_short_prompts_are_rounded_once(dtype, B, T, H, Hk, K, V, cu, state_in, state_out):
    """Sequences within a tile: nothing but the results is rounded to 16 bits
    (the weighted scores and the state coming in keep two parts of 8 or 11
    bits, 2^-17 at most), so beside that rounding only the fp32 sums' bound is
    left."""
    import long_sequence_fft_b200 as lsf
    from mixer_reference import attention, magnitudes
    dt = getattr(torch, dtype)
    n = B if cu is None else len(cu) - 1
    x = [_randn(i, B, T, h, d).to(dt) for i, (h, d) in enumerate(((H, K), (Hk, K), (Hk, V), (H, V)))]
    ld = -torch.logspace(-3, -0.3, H, dtype=torch.float32, device="cuda")
    initial = _randn(7, n, H, K, V) if state_in else None
    dstate = _randn(8, n, H, K, V) if state_out else None
    leaves = [t.clone().requires_grad_() for t in x[:3] + ([initial] if state_in else [])]
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, s = lsf.linear_attention(*leaves[:3], ld, initial_state=leaves[3] if state_in else None, cu_seqlens=cud,
                                return_state=True)
    out = [o, s] if state_out else [o]
    got = dict(zip(("dq", "dk", "dv", "dinitial"), torch.autograd.grad(out, leaves, [x[3], dstate][:len(out)])))
    got.update(o=o.detach(), state=s.detach())
    alone = lsf.linear_attention(*x[:3], ld, initial_state=initial, cu_seqlens=cud)
    args = (*x[:3], ld, K ** -0.5, initial, x[3], dstate, cu)
    ref, mag = attention(*args), magnitudes(*args)
    u = torch.finfo(dt).eps / 2
    for n, t in [*got.items(), ("o", alone)]:
        if t.dtype == torch.float32:
            bound = 2.0 ** -18 * mag[n] + 1e-37
        else:
            bound = u * ref[n].abs() + 2.0 ** -15 * mag[n] + torch.finfo(dt).smallest_normal * u
        assert ((t.double() - ref[n]).abs() <= bound).all(), n
