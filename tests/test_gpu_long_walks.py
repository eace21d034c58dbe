"""GPU tests of linear attention's states over tens of thousands of tokens with
slow decays, where what is rounded at each chunk or segment adds up.

Bounds.  The states here are sums of positive terms, e(x) = (state - exact) /
exact.  A walk of n chunks rounds every element n times, by up to 2^-24 each,
independently: over the 4096 or more elements of a head their mean has a
deviation below 2^-24 sqrt(n / 4096) / sqrt(3), 2^-26 for 512 chunks.  What
remains in a head's mean is what all elements share, the weights: a few
roundings of single powers (2^-24 each, at most eight), and the error of the
exponential of the decay over the whole walk, X: 2 X 2^-23.  One power of g
rounded at every chunk, in the same direction, would be up to n 2^-25."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _states(T, H, K, V, dtype, early, rev, cu=None):
    """State (or its gradient, backward in time) after T tokens of which the
    first 100 (in the direction) have keys, from an initial one."""
    import long_sequence_fft_b200 as lsf
    g = torch.Generator(device="cuda").manual_seed(T + H)
    r = lambda *s: 1 + torch.rand(s, generator=g, device="cuda")             # noqa: E731
    n = 100 if early else 0
    z = lambda d: torch.zeros((1, T, H, d), device="cuda", dtype=dtype)      # noqa: E731
    k, v = z(K), z(V)
    k[:, :n], v[:, :n] = r(1, n, H, K).to(dtype), r(1, n, H, V).to(dtype)
    start = r(1, H, K, V)
    ld = -torch.logspace(-6, -4.5, H, dtype=torch.float32, device="cuda")
    cud = None if cu is None else torch.tensor([0, T], dtype=torch.int32, device="cuda")
    if rev:
        # dS backward in time: its "keys" are q, its "values" do, scaled by 1
        k, v = k.flip(1), v.flip(1)
        init = torch.zeros_like(start).requires_grad_()
        o, s = lsf.linear_attention(k, z(K), z(V), ld, initial_state=init, cu_seqlens=cud, return_state=True, scale=1.0)
        got, = torch.autograd.grad([o, s], [init], [v, start])
        behind = torch.arange(T, T - n, -1, device="cuda")                   # dinitial = g dS_0
        k, v = k.flip(1), v.flip(1)
    else:
        _, got = lsf.linear_attention(z(K), k, v, ld, initial_state=start, cu_seqlens=cud, return_state=True)
        behind = T - 1 - torch.arange(n, device="cuda")
    assert lsf.linear_attention_status() == 0
    ld = ld.double()
    want = torch.exp(ld * T)[None, :, None, None] * start.double()
    w = torch.exp(ld[None] * behind[:, None].double())
    want += torch.einsum("th,thk,thv->hkv", w, k[0, :n].double(), v[0, :n].double())[None]
    return ((got.double() - want) / want)[0], -ld * T


@pytest.mark.parametrize("K,V,dtype", [(64, 64, torch.bfloat16), (128, 128, torch.float16), (64, 64, torch.float16),
                                       (128, 64, torch.bfloat16)])
@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("rev", [False, True])
def test_walks_in_one_piece(K, V, dtype, early, rev):
    """As many heads as SMs: every sequence is one walk of 256 chunks."""
    T, H = 32768, torch.cuda.get_device_properties(0).multi_processor_count
    e, X = _states(T, H, K, V, dtype, early, rev)
    mean = e.mean(dim=(1, 2)).abs()
    bound = 2.0 ** -26 + 8 * 2.0 ** -24 + X * 2.0 ** -22
    assert (mean <= bound).all(), (mean - bound).max()
    # one element: every rounding at its worst
    assert (e.abs().amax(dim=(1, 2)) <= bound + 256 * 2.0 ** -24).all()


@pytest.mark.parametrize("T,K,V,dtype,packed", [(65536, 64, 64, torch.bfloat16, False),
                                                (150001, 128, 128, torch.float16, False),
                                                (100003, 64, 128, torch.bfloat16, True)])
@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("rev", [False, True])
def test_walks_in_segments(T, K, V, dtype, packed, early, rev):
    """Few heads: segments' own states, joined over the segments."""
    e, X = _states(T, 2, K, V, dtype, early, rev, cu=packed or None)
    mean = e.mean(dim=(1, 2)).abs()
    bound = 2.0 ** -26 + 8 * 2.0 ** -24 + X * 2.0 ** -22
    assert (mean <= bound).all(), (mean - bound).max()
