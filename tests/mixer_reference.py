"""Plain fp64 forms of linear attention and group norm for the tests, written
as the sums that define them, and the error bounds the kernels are held to.

Bounds.  With u = finfo(t).eps / 2 a rounding to t is off by at most u times
the value.  An output of linear attention is sum_s w_ts (q_t . k_s) v_s with
w_ts >= 0.  The kernel rounds the weighted q_t . k_s (or the carried state)
once, sums in fp32 and rounds the result, so with

    M = sum_s w_ts (|q_t| . |k_s|) |v_s|        (the same sum of magnitudes)

every element is within u |o| + u M of the exact one, plus the fp32 sums:
at most 256 terms a product, each partial sum off by at most 2^-23 of M,
hence 2^-15 M.  The gradients are sums of the same kind, with M from the same
formulas on magnitudes.  States are fp32 sums of exact products (weights in
24 bits): 2^-18 M covers 16 truncated partial sums of a chunk, the decays
(a few ulp each) and their accumulation over the chunks of a test.
Over many elements the roundings are independent: the relative 2-norm of two
of them stays below sqrt(2) u / sqrt(3) < 0.85 u.
"""
import torch


def attention(q, k, v, log_decay, scale, initial=None, do=None, dstate=None, cu=None):
    """dict(o, state[, dq, dk, dv, dinitial]) in fp64 on q's device."""
    H, K, V = log_decay.shape[0], q.shape[3], v.shape[3]
    B, T = q.shape[:2]
    seqs = [(b, 0, T) for b in range(B)] if cu is None else [(0, cu[i], cu[i + 1]) for i in range(len(cu) - 1)]
    q, k, v, log_decay = q.double(), k.double(), v.double(), log_decay.double()
    z = lambda *s: torch.zeros(s, dtype=torch.float64, device=q.device)      # noqa: E731
    out = {"o": z(B, T, H, V), "state": z(len(seqs), H, K, V)}
    if do is not None:
        out.update(dq=z(*q.shape), dk=z(*k.shape), dv=z(*v.shape), dinitial=z(len(seqs), H, K, V))
    for i, (b, a, e) in enumerate(seqs):
        n = e - a
        t = torch.arange(n, dtype=torch.float64, device=q.device)
        gap = t[:, None] - t[None]
        for h in range(H):
            hq, hk, hv = (h // (H // x.shape[2]) for x in (q, k, v))
            Q, Kk, Vv = q[b, a:e, hq], k[b, a:e, hk], v[b, a:e, hv]
            ld = max(float(log_decay[h]), -1e4)
            S0 = initial[i, h].double() if initial is not None else z(K, V)
            w = torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), 0.0) * scale
            rise, left = torch.exp(ld * (t + 1))[:, None], torch.exp(ld * (n - 1 - t))[:, None]
            whole = float(torch.exp(torch.tensor(ld * n, dtype=torch.float64)))
            P = w * (Q @ Kk.T)
            out["o"][b, a:e, h] = P @ Vv + scale * rise * (Q @ S0)
            out["state"][i, h] = (Kk * left).T @ Vv + whole * S0
            if do is None:
                continue
            G = do[b, a:e, h].double()
            dS = dstate[i, h].double() if dstate is not None else z(K, V)
            dP = w * (G @ Vv.T)
            out["dq"][b, a:e, hq] += dP @ Kk + scale * rise * (G @ S0.T)
            out["dk"][b, a:e, hk] += dP.T @ Q + left * (Vv @ dS.T)
            out["dv"][b, a:e, hv] += P.T @ G + left * (Kk @ dS)
            out["dinitial"][i, h] = scale * (Q * rise).T @ G + whole * dS
    return out


def magnitudes(q, k, v, log_decay, scale, initial=None, do=None, dstate=None, cu=None):
    a = lambda x: None if x is None else x.double().abs()                    # noqa: E731
    return attention(a(q), a(k), a(v), log_decay, abs(scale), a(initial), a(do), a(dstate), cu)


def check_attention(got, ref, mag, dtype, what=""):
    """Element-wise bounds of every output in `got` (see above), and the 2-norm
    over outputs large enough for it to be a statistic."""
    u = torch.finfo(dtype).eps / 2
    for name, x in got.items():
        if x is None:
            continue
        r, m = ref[name], mag[name]
        err = (x.double() - r).abs()
        if x.dtype == torch.float32:
            bound = 2.0 ** -18 * m + 1e-37
        else:
            bound = u * r.abs() + (u + 2.0 ** -15) * m + torch.finfo(dtype).smallest_normal * u
        worst = (err - bound).max().item() if err.numel() else -1.0
        assert worst <= 0, f"{what} {name}: error {err.max().item():.3e} beyond its bound by {worst:.3e}"
        if x.dtype != torch.float32 and x.numel() >= 4096:
            rel = (err.norm() / r.norm()).item()
            assert rel <= 0.85 * u, f"{what} {name}: relative 2-norm {rel:.3e} > {0.85 * u:.3e}"


def activation(x, act):
    s = 1 / (1 + torch.exp(-x))
    return {"none": (x, torch.ones_like(x)), "sigmoid": (s, s * (1 - s)), "silu": (x * s, s * (1 + x * (1 - s)))}[act]


def group_norm(x, groups, weight=None, bias=None, gate=None, act="none", eps=1e-5, dy=None):
    """dict(y[, dx, dgate, dweight, dbias]) in fp64."""
    shape, C = x.shape, x.shape[-1]
    N, D = shape[0], C // groups
    one = torch.ones(C, dtype=torch.float64, device=x.device)
    w, b = (one, 0 * one) if weight is None else (weight.double(), bias.double())
    rows = lambda t: t.reshape(N, -1, groups, D).transpose(1, 2).reshape(N * groups, -1)          # noqa: E731
    back = lambda t: t.reshape(N, groups, -1, D).transpose(1, 2).reshape(shape)                   # noqa: E731
    mean_of = lambda t: back(rows(t).mean(1, keepdim=True).expand(-1, rows(t).shape[1]))          # noqa: E731
    x = x.double()
    d = x - mean_of(x)
    rstd = 1 / torch.sqrt(mean_of(d * d) + eps)
    xh = d * rstd
    n = xh * w + b
    val, slope = activation(n if gate is None else gate.double(), act)
    out = {"y": val if gate is None else n * val}
    if dy is not None:
        dy = dy.double()
        dn = dy * (slope if gate is None else val)
        dnw = dn * w
        out["dgate"] = None if gate is None else dy * n * slope
        out["dweight"], out["dbias"] = (dn * xh).reshape(-1, C).sum(0), dn.reshape(-1, C).sum(0)
        out["dx"] = rstd * (dnw - mean_of(dnw) - xh * mean_of(dnw * xh))
    return out
