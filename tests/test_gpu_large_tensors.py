"""GPU tests of the mixer operators on tensors of more than 2^31 elements: the
last rows against the same rows by themselves."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("shape,G", [(((1 << 20) + 37, 2056), 8), (((1 << 20) + 37, 2050), 5), ((3, 350001, 2056), 2),
                                     ((1100000, 2, 1032), 3)])
def test_norm(shape, G):
    import long_sequence_fft_b200 as lsf
    x = torch.ones(shape, device="cuda", dtype=BF)
    assert x.numel() > 1 << 31
    dy = torch.zeros(shape, device="cuda", dtype=BF)
    tail = 2 if len(shape) == 3 and shape[0] > 3 else 1 if len(shape) == 3 else 64
    x[-tail:], dy[-tail:] = _randn(1, tail, *shape[1:]).to(BF), _randn(2, tail, *shape[1:]).to(BF)
    w, b = _randn(3, shape[-1]).requires_grad_(), _randn(4, shape[-1]).requires_grad_()

    def call(x, dy):
        x = x.requires_grad_()
        y = lsf.group_norm(x, G, w, b, activation="silu")
        return y, *torch.autograd.grad(y, [x, w, b], dy)

    y, dx, dw, db = call(x, dy)
    y2, dx2, dw2, db2 = call(x[-tail:].detach().clone(), dy[-tail:].clone())
    # (other chunks of a sample: other orders of the same fp32 sums)
    for a, c in ((y[-tail:], y2), (dx[-tail:], dx2)):
        assert ((a.double() - c.double()).norm() / c.double().norm()).item() <= 2.0 ** -8
        assert (a.double() - c.double()).abs().max() <= 2.0 ** -6 * c.double().abs().max()
    for a, c in ((dw, dw2), (db, db2)):
        assert (a - c).abs().max() <= 1e-4 * c.abs().max()
    first = torch.nn.functional.silu(b.detach().double())     # (a constant sample: its bias)
    assert (y[0].flatten()[:shape[-1]].double() - first).abs().max() <= 2.0 ** -7 * first.abs().max()


@pytest.mark.parametrize("Hk", [128, 32])
@pytest.mark.parametrize("packed", [False, True])
def test_attention(Hk, packed):
    """A strong decay: the last 300 tokens do not see the others."""
    import long_sequence_fft_b200 as lsf
    T, H, D, n = 140000, 128, 128, 300
    ld = torch.full((H,), -1.0, device="cuda")
    mk = lambda s, h: torch.cat([torch.zeros((1, T - n, h, D), device="cuda", dtype=BF),     # noqa: E731
                                 _randn(s, 1, n, h, D).to(BF)], 1).requires_grad_()
    q, k, v = mk(1, H), mk(2, Hk), mk(3, Hk)
    do = mk(4, H).detach()
    assert q.numel() > 1 << 31
    cu = torch.tensor([0, T - n, T], dtype=torch.int32, device="cuda") if packed else None
    o = lsf.linear_attention(q, k, v, ld, cu_seqlens=cu)
    got = [o, *torch.autograd.grad(o, [q, k, v], do)]
    part = [t[:, -n:].detach().clone().requires_grad_() for t in (q, k, v)]
    o2 = lsf.linear_attention(*part, ld)
    want = [o2, *torch.autograd.grad(o2, part, do[:, -n:].contiguous())]
    assert lsf.linear_attention_status() == 0
    for a, c in zip(got, want):
        a, c = a[:, -n:].double(), c.double()
        # two roundings of each side (mixer_reference)
        assert ((a - c).norm() / c.norm()).item() <= 2 * 0.85 * 2.0 ** -8
    for a in got:
        assert not a[:, :1000].any()


def test_attention_strides():
    """Batches more than 2^31 elements apart, in inputs and output."""
    import long_sequence_fft_b200 as lsf
    T, H, D, far = 200, 2, 64, (1 << 31) + 64
    stores = [torch.zeros(far + 3 * T * H * D, device="cuda", dtype=BF) for _ in range(2)]
    at = lambda s, i: s.as_strided((2, T, H, D), (far, H * D, D, 1), i * T * H * D)          # noqa: E731
    q, k, v, o = *(at(stores[0], i) for i in range(3)), at(stores[1], 1)
    for i, t in enumerate((q, k, v)):
        t.copy_(_randn(i, 2, T, H, D).to(BF))
    ld = torch.tensor([-0.1, -0.01], device="cuda")
    assert lsf.linear_attention(q, k, v, ld, out=o) is o
    assert torch.equal(o, lsf.linear_attention(q.contiguous(), k.contiguous(), v.contiguous(), ld))
    assert not stores[1][:T * H * D].any() and not stores[1][-T * H * D:].any()


def test_step_of_a_large_pool():
    import long_sequence_fft_b200 as lsf
    pool, H, D = 8500, 16, 128
    states = torch.zeros((pool, H, D, D), device="cuda")
    assert states.numel() > 1 << 31
    states[-2:] = _randn(1, 2, H, D, D)
    q, k, v = (_randn(i, 3, H, D).to(BF) for i in range(3))
    ld = torch.linspace(-1, -0.01, H, device="cuda")
    slots = torch.tensor([pool - 1, 3, pool - 2], dtype=torch.int32, device="cuda")
    alone = states[slots.long()].clone()
    o = lsf.linear_attention_step(q, k, v, ld, states, slots=slots)
    assert torch.equal(o, lsf.linear_attention_step(q, k, v, ld, alone))
    assert torch.equal(states[slots.long()], alone) and not states[4:8].any()
