"""Measured cases of the recurrent mixers and the norm beside the long convolution.

The operators: linear attention with a decay for each head (prompt form,
forward and backward; single-token form) and group normalisation with an
activation or an activated gate, channels last (forward and backward).
``run`` computes a case in its plain form, elementary torch operations in 32
bits rounded once at the end, or, where ``own`` is true, through the package.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # a short request at the smallest model sizes: one prompt of 37 tokens
        {"name": "prompt_short", "op": "attention", "B": 1, "T": 37, "lens": "", "H": 8, "Hq": 8, "Hk": 8, "Hv": 8,
         "K": 64, "V": 64, "dtype": "f16", "decay": "slow", "initial": False, "state": True, "train": False},
        # a batch of requests prefilled together, packed, lengths from one token to a few thousand
        {"name": "prompt_packed", "op": "attention", "B": 1, "T": 8192, "lens": "1,2305,64,777,129,3001,0,1500,415",
         "H": 16, "Hq": 16, "Hk": 4, "Hv": 4, "K": 128, "V": 128, "dtype": "bf16", "decay": "slow", "initial": True,
         "state": True, "train": False},
        # one long document read at once, the state kept for what follows
        {"name": "prompt_long", "op": "attention", "B": 1, "T": 65536, "lens": "", "H": 16, "Hq": 16, "Hk": 16, "Hv": 16,
         "K": 128, "V": 128, "dtype": "bf16", "decay": "slow", "initial": False, "state": True, "train": False},
        # a training step's mixer at 4096 tokens and 768 channels, heads of 64
        {"name": "train_4k", "op": "attention", "B": 16, "T": 4096, "lens": "", "H": 12, "Hq": 12, "Hk": 12, "Hv": 12,
         "K": 64, "V": 64, "dtype": "bf16", "decay": "slow", "initial": False, "state": False, "train": True},
        # training on an odd length, keys and queries shared by groups of heads, a state carried in and out
        {"name": "train_shared_odd", "op": "attention", "B": 2, "T": 2047, "lens": "", "H": 16, "Hq": 4, "Hk": 4, "Hv": 16,
         "K": 128, "V": 64, "dtype": "f16", "decay": "fast", "initial": True, "state": True, "train": True},
        # one user's next token
        {"name": "step_one", "op": "step", "B": 1, "H": 12, "Hq": 12, "Hk": 12, "Hv": 12, "K": 64, "V": 64,
         "dtype": "f16", "decay": "slow", "pool": 0, "idle": 0},
        # a serving batch's next tokens, states in a pool, a few rows idle
        {"name": "step_batch", "op": "step", "B": 250, "H": 16, "Hq": 16, "Hk": 4, "Hv": 4, "K": 128, "V": 128,
         "dtype": "bf16", "decay": "slow", "pool": 320, "idle": 6},
        # the head norm and gate behind one step of a small batch
        {"name": "norm_step", "op": "norm", "N": 8, "S": 1, "C": 768, "G": 12, "dtype": "bf16", "act": "silu",
         "gate": True, "affine": True, "train": False},
        # the head norm and gate of a training step
        {"name": "norm_train", "op": "norm", "N": 32768, "S": 1, "C": 2048, "G": 16, "dtype": "bf16", "act": "silu",
         "gate": True, "affine": True, "train": True},
        # features of whole samples, normalised over positions, odd sizes
        {"name": "norm_sample", "op": "norm", "N": 16, "S": 4095, "C": 760, "G": 8, "dtype": "f16", "act": "silu",
         "gate": False, "affine": True, "train": False},
        {"name": "norm_sample_train", "op": "norm", "N": 8, "S": 4096, "C": 768, "G": 32, "dtype": "f32", "act": "silu",
         "gate": False, "affine": True, "train": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng, most):
    H = rng.choice([h for h in (1, 2, 3, 4, 6, 8, 12, 16, 24, 32) if h <= most])
    share = rng.choice([d for d in (1, 1, 2, 3, 4, 8) if H % d == 0])
    kind = rng.choice(("all", "kv", "qk"))
    Hs = H // share
    return {"all": (H, H, H, H), "kv": (H, H, Hs, Hs), "qk": (H, Hs, Hs, H)}[kind]


def draw(rng):
    kind = rng.choice(("attention", "attention", "attention", "step", "norm", "norm"))
    if kind == "attention":
        H, Hq, Hk, Hv = _heads(rng, 32)
        train = rng.random() < 0.4
        tokens = max(1, min(65536, (1 << 20) // H) // (4 if train else 1))
        K, V = rng.choice(((64, 64), (128, 128), (64, 128), (128, 64), (8 * rng.randint(2, 16), 8 * rng.randint(2, 16))))
        lens = ""
        if rng.random() < 0.4:
            T = _log_int(rng, 2, tokens)
            n = rng.randint(1, min(24, T))
            cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
            parts = [b - a for a, b in zip([0] + cuts, cuts + [T])]
            B, lens = 1, ",".join(map(str, parts))
        else:
            B = _log_int(rng, 1, 16)
            T = _log_int(rng, 1, max(1, tokens // B))
        return {"op": "attention", "B": B, "T": T, "lens": lens, "H": H, "Hq": Hq, "Hk": Hk, "Hv": Hv, "K": K, "V": V,
                "dtype": rng.choice(("bf16", "f16")), "decay": rng.choice(("slow", "fast")),
                "initial": rng.random() < 0.5, "state": rng.random() < 0.5, "train": train}
    if kind == "step":
        H, Hq, Hk, Hv = _heads(rng, 32)
        K, V = rng.choice(((64, 64), (128, 128), (64, 128), (128, 64), (8 * rng.randint(2, 16), 8 * rng.randint(2, 16))))
        B = _log_int(rng, 1, 250)
        pool = rng.choice((0, B + rng.randint(0, 64)))
        return {"op": "step", "B": B, "H": H, "Hq": Hq, "Hk": Hk, "Hv": Hv, "K": K, "V": V,
                "dtype": rng.choice(("bf16", "f16")), "decay": rng.choice(("slow", "fast")), "pool": pool,
                "idle": rng.randint(0, B // 8) if pool else 0}
    G = rng.choice((1, 2, 3, 4, 8, 12, 16, 32))
    train = rng.random() < 0.5
    if rng.random() < 0.5:
        S, C = 1, G * rng.choice((rng.randint(4, 256), 8 * rng.randint(1, 32)))
        N = _log_int(rng, 1, max(1, (1 << 25) // C))
    else:
        C = G * rng.choice((rng.randint(1, 64), 8 * rng.randint(1, 12)))
        S = _log_int(rng, 8, 16384)
        N = _log_int(rng, 1, max(1, min(64, (1 << 25) // (C * S))))
    return {"op": "norm", "N": N, "S": S, "C": C, "G": G, "dtype": rng.choice(("bf16", "f16", "f32")),
            "act": rng.choice(("none", "silu", "sigmoid")), "gate": rng.random() < 0.5, "affine": rng.random() < 0.8,
            "train": train}


def _log_decay(case):
    """slow: 1 - 2^-5 .. 1 - 2^-9 over the heads; fast: exp(-2^-1) .. exp(-2^-6)."""
    H = case["H"]
    x = [h / max(1, H - 1) for h in range(H)]
    if case["decay"] == "slow":
        return [math.log1p(-2.0 ** (-5 - 4 * t)) for t in x]
    return [-2.0 ** (-1 - 5 * t) for t in x]


def _lens(case):
    return [int(n) for n in case["lens"].split(",")] if case["lens"] else [case["T"]] * case["B"]


def work(case):
    b = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "attention":
        tok, H, K, V = case["B"] * case["T"], case["H"], case["K"], case["V"]
        ins = tok * (case["Hq"] * K + case["Hk"] * K + case["Hv"] * V) * b
        state = len(_lens(case)) * H * K * V * 4
        nbytes = ins + tok * H * V * b + state * (case["initial"] + case["state"])
        flops = 4.0 * tok * H * K * V
        if case["train"]:
            nbytes += 2 * ins + tok * H * V * b + state * (case["initial"] * 2 + case["state"])
            flops += 10.0 * tok * H * K * V
        return {"bytes": float(nbytes), "flops": flops}
    if case["op"] == "step":
        rows, H, K, V = case["B"] - case["idle"], case["H"], case["K"], case["V"]
        io = case["B"] * (case["Hq"] * K + case["Hk"] * K + case["Hv"] * V + H * V) * b
        return {"bytes": float(rows * H * K * V * 8 + io), "flops": 5.0 * rows * H * K * V}
    n = case["N"] * case["S"] * case["C"]
    passes = 2 + case["gate"]
    if case["train"]:
        passes += 3 + 2 * case["gate"]
    return {"bytes": float(n * b * passes), "flops": float(n * (10 + (20 if case["train"] else 0)))}


# ----------------------------------------------------------------- inputs ---

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * scale + mean).to(dtype)

    s = {"case": case}
    if case["op"] == "norm":
        lead = (case["N"], case["C"]) if case["S"] == 1 else (case["N"], case["S"], case["C"])
        s["x"] = normal(*lead, scale=1.5, mean=0.5)
        s["gate"] = normal(*lead) if case["gate"] else None
        s["weight"] = normal(case["C"], scale=0.2, mean=1.0, dtype=torch.float32) if case["affine"] else None
        s["bias"] = normal(case["C"], scale=0.2, dtype=torch.float32) if case["affine"] else None
        if case["train"]:
            s["dy"] = normal(*lead)
            for n in ("x", "gate", "weight", "bias"):
                if s[n] is not None:
                    s[n].requires_grad_()
        return s
    H, K, V = case["H"], case["K"], case["V"]
    s["log_decay"] = torch.tensor(_log_decay(case), dtype=torch.float32, device="cuda")
    if case["op"] == "step":
        B = case["B"]
        s["q"], s["k"], s["v"] = normal(B, case["Hq"], K), normal(B, case["Hk"], K), normal(B, case["Hv"], V)
        s["state"] = normal(case["pool"] or B, H, K, V, scale=3.0, dtype=torch.float32)
        s["slots"] = None
        if case["pool"]:
            slots = torch.randperm(case["pool"], generator=gen, device="cuda")[:B].to(torch.int32)
            if case["idle"]:
                slots[torch.randperm(B, generator=gen, device="cuda")[:case["idle"]]] = -1
            s["slots"] = slots
        return s
    B, T = case["B"], case["T"]
    s["q"] = normal(B, T, case["Hq"], K)
    s["k"] = normal(B, T, case["Hk"], K)
    s["v"] = normal(B, T, case["Hv"], V, mean=0.1)
    lens = _lens(case)
    s["cu"] = None
    if case["lens"]:
        s["cu"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    s["initial"] = normal(len(lens), H, K, V, dtype=torch.float32) if case["initial"] else None
    if case["train"]:
        s["do"] = normal(B, T, H, V)
        s["dstate"] = normal(len(lens), H, K, V, scale=0.3, dtype=torch.float32) if case["state"] else None
        for n in ("q", "k", "v", "initial"):
            if s[n] is not None:
                s[n].requires_grad_()
    return s


# -------------------------------------------------------------- the passes ---

def run(s):
    case = s["case"]
    return {"attention": _run_attention, "step": _run_step, "norm": _run_norm}[case["op"]](s, case)


def _run_attention(s, case):
    if own:
        import long_sequence_fft_b200 as lsf
        o = lsf.linear_attention(s["q"], s["k"], s["v"], s["log_decay"], initial_state=s["initial"], cu_seqlens=s["cu"],
                                 return_state=case["state"])
        o, last = o if case["state"] else (o, None)
    else:
        o, last = _plain_attention(s, case)
    out = {"o": o}
    if last is not None:
        out["state"] = last
    if case["train"]:
        names = [n for n in ("q", "k", "v", "initial") if s[n] is not None]
        outs, grads = ([o], [s["do"]]) if last is None else ([o, last], [s["do"], s["dstate"]])
        for n, g in zip(names, torch.autograd.grad(outs, [s[n] for n in names], grads)):
            out["d" + n] = g
    return out


def _plain_attention(s, case):
    """Chunks of 128 tokens: products inside a chunk, each chunk's own state,
    and the states at the chunks' starts as one product over the chunks."""
    H, K, V, dt = case["H"], case["K"], case["V"], s["q"].dtype
    q, k, v = (s[n].float().repeat_interleave(H // s[n].shape[2], dim=2) for n in ("q", "k", "v"))
    lens = _lens(case)
    longest = max(lens)
    if s["cu"] is None:
        n = torch.full((case["B"],), case["T"], device=q.device)
    else:
        # the packed sequences as rows of a padded batch
        cu = s["cu"].long()
        n = cu[1:] - cu[:-1]
        pos = torch.arange(longest, device=q.device)
        valid = pos[None] < n[:, None]
        at = (cu[:-1, None] + pos[None]).clamp(max=case["T"] - 1)
        q, k, v = (torch.where(valid[..., None, None], x[0][at], 0.0) for x in (q, k, v))
    B, T = q.shape[:2]
    scale = K ** -0.5
    C = min(128, T)
    nc = -(-T // C)
    pad = nc * C - T
    chunks = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(B, nc, C, H, -1).permute(0, 3, 1, 2, 4)  # noqa: E731
    ld = s["log_decay"].double()
    power = lambda e: torch.exp(ld.view(-1, *[1] * e.dim()) * e).float()                                           # noqa: E731
    i = torch.arange(C, device=q.device, dtype=torch.float64)
    c = torch.arange(nc, device=q.device, dtype=torch.float64)
    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    inside = torch.where(i[:, None] >= i[None], power((i[:, None] - i[None]).clamp(min=0)), 0.0)          # [H, C, C]
    o = ((qc @ kc.transpose(-1, -2)) * inside[:, None]) @ vc
    local = (kc * power(C - 1 - i)[:, None, :, None]).transpose(-1, -2) @ vc                             # [B, H, nc, K, V]
    carry = torch.where(c[:, None] > c[None], power((C * (c[:, None] - 1 - c[None])).clamp(min=0)), 0.0)  # [H, nc, nc]
    start = (carry @ local.reshape(B, H, nc, K * V)).view(B, H, nc, K, V)
    if s["initial"] is not None:
        start = start + s["initial"][:, :, None] * power(C * c)[:, :, None, None]
    o = o + (qc * power(i + 1)[:, None, :, None]) @ start
    o = (o * scale).permute(0, 2, 3, 1, 4).reshape(B, nc * C, H, V)[:, :T]
    last = None
    if case["state"]:
        left = n[:, None] - 1 - torch.arange(T, device=q.device)[None]                                   # [B, T]
        w = torch.where(left >= 0, power(left.clamp(min=0).double()), 0.0).permute(1, 0, 2)              # [B, H, T]
        last = (k.permute(0, 2, 1, 3) * w[..., None]).transpose(-1, -2) @ v.permute(0, 2, 1, 3)
        if s["initial"] is not None:
            last = last + s["initial"] * power(n.double()).t()[..., None, None]
    if s["cu"] is not None:
        o = o[valid][None]
    return o.to(dt), last


def _run_step(s, case):
    if own:
        import long_sequence_fft_b200 as lsf
        o = lsf.linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], slots=s["slots"])
        return {"o": o, "state": s["state"]}
    H, K, dt = case["H"], case["K"], s["q"].dtype
    q, k, v = (s[n].float().repeat_interleave(H // s[n].shape[1], dim=1) for n in ("q", "k", "v"))
    g = torch.exp(s["log_decay"])[None, :, None, None]
    if s["slots"] is None:
        s["state"].mul_(g).add_(k[..., :, None] * v[..., None, :])
        o = (q[..., None, :] @ s["state"])[..., 0, :] * K ** -0.5
        return {"o": o.to(dt), "state": s["state"]}
    live = s["slots"] >= 0
    rows = s["slots"].long()[live]
    new = s["state"][rows] * g + k[live][..., :, None] * v[live][..., None, :]
    s["state"][rows] = new
    o = torch.zeros((case["B"], H, case["V"]), device=q.device)
    o[live] = (q[live][..., None, :] @ new)[..., 0, :] * K ** -0.5
    return {"o": o.to(dt), "state": s["state"]}


def _act(x, act):
    return x * torch.sigmoid(x) if act == "silu" else torch.sigmoid(x) if act == "sigmoid" else x


def _run_norm(s, case):
    if own:
        import long_sequence_fft_b200 as lsf
        y = lsf.group_norm(s["x"], case["G"], s["weight"], s["bias"], gate=s["gate"], activation=case["act"], eps=EPS)
    else:
        x = s["x"].float().view(case["N"], case["S"], case["G"], -1)
        d = x - x.mean(dim=(1, 3), keepdim=True)
        n = d * torch.rsqrt((d * d).mean(dim=(1, 3), keepdim=True) + EPS)
        n = n.view(s["x"].shape)
        if s["weight"] is not None:
            n = n * s["weight"] + s["bias"]
        y = _act(n, case["act"]) if s["gate"] is None else n * _act(s["gate"].float(), case["act"])
        y = y.to(s["x"].dtype)
    out = {"y": y}
    if case["train"]:
        names = [n for n in ("x", "gate", "weight", "bias") if s[n] is not None]
        for n, g in zip(names, torch.autograd.grad(y, [s[n] for n in names], s["dy"])):
            out["d" + n] = g
    return out


# -------------------------------------------------------- in 64 bits, apart ---

def exact(case, seed):
    s = {n: x.detach().double() if isinstance(x, torch.Tensor) and x.is_floating_point() else x
         for n, x in prepare(case, seed).items()}
    return {"attention": _exact_attention, "step": _exact_step, "norm": _exact_norm}[case["op"]](s, case)


def _exact_attention(s, case):
    """The sums over all pairs of tokens, a sequence and a head at a time, in
    blocks of query tokens; gradients from their formulas."""
    H, K, V = case["H"], case["K"], case["V"]
    a, lens = K ** -0.5, _lens(case)
    z = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")   # noqa: E731
    B, T = case["B"], case["T"]
    out = {"o": z(B, T, H, V)}
    if case["state"]:
        out["state"] = z(len(lens), H, K, V)
    if case["train"]:
        out.update(dq=z(*s["q"].shape), dk=z(*s["k"].shape), dv=z(*s["v"].shape))
        if case["initial"]:
            out["dinitial"] = z(len(lens), H, K, V)
    at = 0
    for i, n in enumerate(lens):
        b, rows = (0, slice(at, at + n)) if case["lens"] else (i, slice(0, T))
        at += n
        t = torch.arange(n, dtype=torch.float64, device="cuda")
        for h in range(H):
            ld = s["log_decay"][h]
            hq, hk, hv = (h // (H // case[x]) for x in ("Hq", "Hk", "Hv"))
            q, k, v = s["q"][b, rows, hq], s["k"][b, rows, hk], s["v"][b, rows, hv]
            s0 = s["initial"][i, h] if case["initial"] else z(K, V)
            rise, left = torch.exp(ld * (t + 1))[:, None], torch.exp(ld * (n - 1 - t))[:, None]
            whole = torch.exp(ld * n)
            if case["state"]:
                out["state"][i, h] = whole * s0 + (k * left).t() @ v
            if case["train"]:
                do = s["do"][b, rows, h]
                ds = s["dstate"][i, h] if case["state"] else z(K, V)
                out["dq"][b, rows, hq] += a * rise * (do @ s0.t())
                out["dk"][b, rows, hk] += left * (v @ ds.t())
                out["dv"][b, rows, hv] += left * (k @ ds)
                if case["initial"]:
                    out["dinitial"][i, h] = whole * ds + a * (q * rise).t() @ do
            out["o"][b, rows, h] = a * rise * (q @ s0)
            for r in range(0, n, 2048):
                e = min(n, r + 2048)
                gap = t[r:e, None] - t[None, :e]
                w = torch.where(gap >= 0, torch.exp(ld * gap.clamp(min=0)), 0.0) * a
                p = (q[r:e] @ k[:e].t()) * w
                out["o"][b, rows, h][r:e] += p @ v[:e]
                if case["train"]:
                    dp = (do[r:e] @ v[:e].t()) * w
                    out["dq"][b, rows, hq][r:e] += dp @ k[:e]
                    out["dk"][b, rows, hk][:e] += dp.t() @ q[r:e]
                    out["dv"][b, rows, hv][:e] += p.t() @ do[r:e]
    return out


def _exact_step(s, case):
    o = torch.zeros((case["B"], case["H"], case["V"]), dtype=torch.float64, device="cuda")
    state = s["state"]
    slots = s["slots"].tolist() if s["slots"] is not None else list(range(case["B"]))
    of = {x: [h // (case["H"] // case[x]) for h in range(case["H"])] for x in ("Hq", "Hk", "Hv")}
    for b, slot in enumerate(slots):
        if slot < 0:
            continue
        k, v = s["k"][b, of["Hk"]], s["v"][b, of["Hv"]]
        state[slot] = torch.exp(s["log_decay"])[:, None, None] * state[slot] + torch.einsum("hk,hv->hkv", k, v)
        o[b] = torch.einsum("hk,hkv->hv", s["q"][b, of["Hq"]], state[slot]) / math.sqrt(case["K"])
    return {"o": o, "state": state}


def _exact_norm(s, case):
    N, S, G, C = case["N"], case["S"], case["G"], case["C"]
    shape = s["x"].shape
    one, zero = (torch.full((C,), c, dtype=torch.float64, device="cuda") for c in (1.0, 0.0))
    w, b = (s["weight"], s["bias"]) if case["affine"] else (one, zero)
    x = s["x"].reshape(N, S, G, C // G).transpose(1, 2).reshape(N * G, -1)
    var, mean = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    back = lambda y: y.reshape(N, G, S, C // G).transpose(1, 2).reshape(shape)    # noqa: E731
    xh = back((x - mean) / torch.sqrt(var + EPS))
    n = xh * w + b
    arg = n if s["gate"] is None else s["gate"]
    sig = 1 / (1 + torch.exp(-arg))
    act, slope = {"none": (arg, torch.ones_like(arg)), "sigmoid": (sig, sig * (1 - sig)),
                  "silu": (arg * sig, sig * (1 + arg * (1 - sig)))}[case["act"]]
    out = {"y": act if s["gate"] is None else n * act}
    if case["train"]:
        dy = s["dy"]
        dn = dy * (slope if s["gate"] is None else act)
        if s["gate"] is not None:
            out["dgate"] = dy * n * slope
        if case["affine"]:
            out["dweight"], out["dbias"] = (dn * xh).reshape(-1, C).sum(0), dn.reshape(-1, C).sum(0)
        m = lambda y: back(y.reshape(N, S, G, C // G).transpose(1, 2).reshape(N * G, -1).mean(1, keepdim=True)  # noqa: E731
                           .expand(-1, S * (C // G)))
        out["dx"] = back((1 / torch.sqrt(var + EPS)).expand(-1, S * (C // G))) * (dn * w - m(dn * w) - xh * m(dn * w * xh))
    return out
