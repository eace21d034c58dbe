"""The operators together, as a layer uses them: linear attention over a
prompt, its heads normalised and gated, then the same layer token by token
from the state; and a training step through both."""
import pytest

from mixer_reference import attention, group_norm

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def _layer(B, T, H, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")                # noqa: E731
    x = {n: r(B, T, H, D).bfloat16() for n in ("q", "k", "v")}
    x["gate"] = r(B, T, H * D).bfloat16()
    x["weight"], x["bias"] = 1 + 0.1 * r(H * D), 0.1 * r(H * D)
    x["log_decay"] = torch.log1p(-(2.0 ** -torch.linspace(5, 9, H, device="cuda")))
    x["dy"] = r(B * T, H * D).bfloat16()
    return x


def _reference(x, H, D):
    """The exact layer on the bf16 inputs, and on the same inputs the layer
    with its attention rounded to bf16 in between (what any bf16 layer has)."""
    o = attention(x["q"], x["k"], x["v"], x["log_decay"], D ** -0.5)["o"]
    rows = lambda t: t.reshape(-1, H * D)                                     # noqa: E731
    return group_norm(rows(o), H, x["weight"], x["bias"], rows(x["gate"]), "silu")["y"]


def test_prompt_then_tokens():
    import long_sequence_fft_b200 as lsf
    B, T, H, D = 2, 150, 4, 64
    x = _layer(B, T, H, D, seed=1)
    ref = _reference(x, H, D).reshape(B, T, H * D)
    n = 140
    norm = lambda o, gate: lsf.group_norm(o.reshape(-1, H * D), H, x["weight"], x["bias"],       # noqa: E731
                                          gate=gate.reshape(-1, H * D), activation="silu")
    o, state = lsf.linear_attention(x["q"][:, :n], x["k"][:, :n], x["v"][:, :n], x["log_decay"], return_state=True)
    y = [norm(o, x["gate"][:, :n]).view(B, n, H * D)]
    for t in range(n, T):
        o = lsf.linear_attention_step(x["q"][:, t], x["k"][:, t], x["v"][:, t], x["log_decay"], state)
        y.append(norm(o, x["gate"][:, t]).view(B, 1, H * D))
    y = torch.cat(y, 1)
    # o carries at most sqrt(2) roundings' worth (0.85 u in 2-norm), the norm
    # keeps relative sizes, y is rounded once more (0.58 u): below 1.1 u
    rel = ((y.double() - ref).norm() / ref.norm()).item()
    assert rel <= 1.1 * 2.0 ** -8, rel
    assert lsf.linear_attention_status() == 0


def test_training_step_beside_the_long_convolution():
    """One layer of each mixer in a row, one backward pass through all three
    operators; gradients of the last ones against their formulas on the
    values the kernels produced."""
    import long_sequence_fft_b200 as lsf
    B, T, H, D = 2, 1024, 2, 64
    x = _layer(B, T, H, D, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = (torch.randn((H * D, T), generator=g, device="cuda") / T ** 0.5).bfloat16().requires_grad_()
    u = torch.randn((B, H * D, T), generator=g, device="cuda").bfloat16().requires_grad_()
    conv = lsf.fftconv(u, k)                                                 # [B, H D, T]
    v = conv.transpose(1, 2).contiguous().view(B, T, H, D)
    v.retain_grad()
    q = x["q"].clone().requires_grad_()
    gate = x["gate"].clone().requires_grad_()
    o = lsf.linear_attention(q, x["k"], v, x["log_decay"])
    o.retain_grad()
    y = lsf.group_norm(o.view(B * T, H * D), H, x["weight"], x["bias"], gate=gate.view(B * T, H * D),
                       activation="silu")
    y.backward(x["dy"])
    u_bf = 2.0 ** -8
    ref = group_norm(o.detach().view(B * T, H * D), H, x["weight"], x["bias"], x["gate"].view(B * T, H * D), "silu",
                     dy=x["dy"])
    for got, want in ((o.grad.view(B * T, H * D), ref["dx"]), (gate.grad.view(B * T, H * D), ref["dgate"])):
        assert ((got.double() - want).norm() / want.norm()).item() <= 0.6 * u_bf
    a = attention(x["q"], x["k"], v.detach(), x["log_decay"], D ** -0.5, do=o.grad)
    for got, want in ((q.grad, a["dq"]), (v.grad, a["dv"])):
        assert ((got.double() - want).norm() / want.norm()).item() <= 0.85 * u_bf
    assert u.grad is not None and k.grad is not None and torch.isfinite(u.grad).all()
