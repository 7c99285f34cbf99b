"""Measured cases of the selective scan, its short causal convolution and the norm around them.

Each case names one call a user makes: the selective state space scan over prompts
(``scan``), its gradients (``scan_backward``) and one token (``scan_step``); the short
causal convolution in front of it (``conv``, ``conv_backward``, ``conv_step``); the
root-mean-square norm with the residual's addition, in floats (``norm``), with its
gradients (``norm_backward``) or in 8-bit codes (``norm_codes``).  ``run`` computes it with
elementary torch operations in 32 bits, or, with ``own``, through the package's entry
points; ``exact`` in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # The prompts of eight sequences through a gated layer of width 2048: the largest scan.
        {"name": "scan_b8_t4096_d2048", "op": "scan", "B": 8, "T": 4096, "D": 2048, "N": 16, "G": 1, "dtype": "bf16", "gated": True,
         "ragged": False},
        # One very long prompt: few channels, so the work has to be split over time.
        {"name": "scan_b1_t65536_d1024", "op": "scan", "B": 1, "T": 65536, "D": 1024, "N": 16, "G": 1, "dtype": "bf16", "gated": True,
         "ragged": False},
        # A padded batch of short prompts that continue older states, odd sizes everywhere, two groups of channels.
        {"name": "scan_ragged_b5_t777_d200_n7", "op": "scan", "B": 5, "T": 777, "D": 200, "N": 7, "G": 2, "dtype": "fp32", "gated": False,
         "ragged": True},
        # The gradients of a training step on eight sequences.
        {"name": "scan_backward_b8_t2048_d1024", "op": "scan_backward", "B": 8, "T": 2048, "D": 1024, "N": 16, "G": 1, "dtype": "bf16",
         "gated": True, "ragged": False},
        # A small training batch of odd sizes in fp32.
        {"name": "scan_backward_b3_t1001_d192", "op": "scan_backward", "B": 3, "T": 1001, "D": 192, "N": 16, "G": 1, "dtype": "fp32",
         "gated": True, "ragged": True},
        # One token of each of 256 streams.
        {"name": "scan_step_b256_d2048", "op": "scan_step", "B": 256, "D": 2048, "N": 16, "G": 1, "dtype": "bf16", "gated": True},
        # One token of two streams: the smallest call, latency counts.
        {"name": "scan_step_b2_d512", "op": "scan_step", "B": 2, "D": 512, "N": 16, "G": 1, "dtype": "fp32", "gated": True},
        # The convolution in front of the largest scan.
        {"name": "conv_b8_t4096_d2048", "op": "conv", "B": 8, "T": 4096, "D": 2048, "K": 4, "dtype": "bf16", "ragged": False},
        # Its gradients in the training step.
        {"name": "conv_backward_b8_t2048_d1024", "op": "conv_backward", "B": 8, "T": 2048, "D": 1024, "K": 4, "dtype": "bf16",
         "ragged": False},
        # One token of each of 256 streams through the convolution.
        {"name": "conv_step_b256_d2048", "op": "conv_step", "B": 256, "D": 2048, "K": 4, "dtype": "bf16"},
        # The norm before an 8-bit projection, over a prefill of 256 sequences of 512 tokens.
        {"name": "norm_codes_131072x2048", "op": "norm_codes", "M": 131072, "D": 2048, "dtype": "bf16", "residual": "bf16"},
        # The norm's gradients in the training step, the residual stream in fp32.
        {"name": "norm_backward_16384x2048", "op": "norm_backward", "M": 16384, "D": 2048, "dtype": "bf16", "residual": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_backward", "scan_step", "conv", "conv_backward", "conv_step", "norm", "norm_codes", "norm_backward"])
    dtype = rng.choice(["fp32", "bf16"])
    if op in ("scan", "scan_backward"):
        G, N = rng.choice([1, 1, 2]), rng.choice([16, 16, rng.randint(1, 32)])
        D, B = G * _log(rng, 16, 2048 // G), _log(rng, 1, 16)
        most = (8 * 4096 * 2048 * 16 if op == "scan" else 8 * 2048 * 1024 * 16) // (B * D * N)
        T = _log(rng, 1, max(1, min(65536 if op == "scan" else 8192, most)))
        return {"op": op, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "gated": rng.random() < 0.7, "ragged": rng.random() < 0.4}
    if op == "scan_step":
        G = rng.choice([1, 1, 2])
        return {"op": op, "B": _log(rng, 1, 256), "D": G * _log(rng, 16, 2048 // G), "N": rng.choice([16, 16, rng.randint(1, 64)]), "G": G,
                "dtype": dtype, "gated": rng.random() < 0.7}
    if op in ("conv", "conv_backward"):
        B, D = _log(rng, 1, 16), _log(rng, 16, 4096)
        T = _log(rng, 1, max(1, min(65536, (8 * 4096 * 2048 if op == "conv" else 8 * 2048 * 1024) // (B * D))))
        return {"op": op, "B": B, "T": T, "D": D, "K": rng.choice([2, 3, 4, 4]), "dtype": dtype, "ragged": rng.random() < 0.4}
    if op == "conv_step":
        return {"op": op, "B": _log(rng, 1, 256), "D": _log(rng, 16, 4096), "K": rng.choice([2, 3, 4, 4]), "dtype": dtype}
    D = _log(rng, 16, 4096)
    rows = 131072 if op != "norm_backward" else 16384
    return {"op": op, "M": _log(rng, 1, min(rows, rows * 2048 // D)), "D": D, "dtype": dtype,
            "residual": rng.choice(["", dtype, "fp32"]) if op != "norm_backward" else rng.choice([dtype, "fp32"])}


# ------------------------------------------------------------- plain forms


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _softplus(x):
    return x.clamp(min=0) + torch.log1p(torch.exp(-x.abs()))


def _alive(lengths, T):
    """[B,T,1] truth values of the tokens in front of each sequence's end, or None."""
    return None if lengths is None else (torch.arange(T, device=DEV) < lengths[:, None])[..., None]


def _cut(x, L):
    """[B,T,..] in chunks of L tokens, [L,B,chunks,..]; zeros behind the end."""
    B, T = x.shape[:2]
    n = -(-T // L)
    x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, n * L - T))
    return x.reshape(B, n, L, *x.shape[2:]).movedim(2, 0)


def _join(x, T):
    """Back from chunks [L,B,chunks,..] to [B,T,..]."""
    x = x.movedim(0, 2)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :T]


class _Chunks:
    """The scan's inputs in chunks of about sqrt(T) tokens, in fp32, channels by group: [L,B,chunks,G,D/G].  A token behind a
    sequence's end has step 0, which leaves the state as it is."""

    def __init__(self, s):
        u = s["u"].float()
        self.B, self.T, self.D = u.shape
        self.G, self.N = s["Bm"].shape[2:]
        self.L = math.isqrt(self.T - 1) + 1
        self.x = s["delta"].float() + s["bias"]
        dt, alive = _softplus(self.x), _alive(s["lengths"], self.T)
        dt = dt if alive is None else torch.where(alive, dt, 0.0)
        group = lambda t: _cut(t.view(self.B, self.T, self.G, -1), self.L)  # noqa: E731
        self.u, self.dt = group(u)[..., None], group(dt)[..., None]
        self.Bm, self.Cm = (_cut(s[k].float(), self.L)[..., None, :] for k in ("Bm", "Cm"))
        self.A = s["A"].view(self.G, -1, self.N)
        h0 = torch.zeros((self.B, self.D, self.N), device=DEV) if s["h0"] is None else s["h0"]
        self.h0 = h0.view(self.B, self.G, -1, self.N)
        self.decay = torch.exp(self.A * self.dt.sum(0))  # over each whole chunk

    def step(self, h, i):
        return h * torch.exp(self.A * self.dt[i]) + self.dt[i] * self.u[i] * self.Bm[i]

    def starts(self):
        """The state in front of each chunk, and the one behind the last."""
        ends = torch.zeros((), device=DEV)
        for i in range(self.L):
            ends = self.step(ends, i)
        at = [self.h0]
        for c in range(ends.shape[1]):
            at.append(at[-1] * self.decay[:, c] + ends[:, c])
        return torch.stack(at[:-1], 1), at[-1].reshape(self.B, self.D, self.N)

    def flat(self, x):
        return _join(x, self.T).reshape(self.B, self.T, -1)


def _scan(s):
    c = _Chunks(s)
    h, last = c.starts()
    y = []
    for i in range(c.L):
        h = c.step(h, i)
        y.append((h * c.Cm[i]).sum(-1))
    u = s["u"].float()
    y = c.flat(torch.stack(y)) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    alive = _alive(s["lengths"], c.T)
    y = y if alive is None else torch.where(alive, y, 0.0)
    return y.to(s["u"].dtype), last


def _scan_backward(s):
    c = _Chunks(s)
    alive, dtype = _alive(s["lengths"], c.T), s["u"].dtype
    u, dy = s["u"].float(), s["dy"].float()
    dy = dy if alive is None else torch.where(alive, dy, 0.0)
    gate = 1.0 if s["z"] is None else s["z"].float() * _sigmoid(s["z"].float())
    ds = dy * gate
    dsc = _cut(ds.view(c.B, c.T, c.G, -1), c.L)[..., None]
    hs, y = [c.starts()[0]], []
    for i in range(c.L):
        hs.append(c.step(hs[-1], i))
        y.append((hs[-1] * c.Cm[i]).sum(-1))
    g = torch.zeros((), device=DEV)  # the gradient that each chunk's own outputs send in front of it
    for i in reversed(range(c.L)):
        g = (g + dsc[i] * c.Cm[i]) * torch.exp(c.A * c.dt[i])
    at = [torch.zeros((), device=DEV) if s["dlast"] is None else s["dlast"].view(c.h0.shape)]
    for k in reversed(range(g.shape[1])):
        at.append(at[-1] * c.decay[:, k] + g[:, k])
    dh0 = at.pop()
    g = torch.stack([a.expand(c.h0.shape) for a in reversed(at)], 1)
    du, ddt, dB, dC, dA = [], [], [], [], torch.zeros(c.A.shape, device=DEV)
    for i in reversed(range(c.L)):
        g = g + dsc[i] * c.Cm[i]
        dC.append((dsc[i] * hs[i + 1]).sum(-2))
        dB.append((g * (c.dt[i] * c.u[i])).sum(-2))
        through = (g * c.Bm[i]).sum(-1)
        g = g * torch.exp(c.A * c.dt[i])
        q = g * hs[i]
        du.append(through * c.dt[i][..., 0])
        ddt.append(through * c.u[i][..., 0] + (q * c.A).sum(-1))
        dA = dA + (q * c.dt[i]).sum((0, 1))
    du, ddt, dB, dC = (_join(torch.stack(v[::-1]), c.T) for v in (du, ddt, dB, dC))
    ddelta = ddt.reshape(u.shape) * _sigmoid(c.x)
    ddelta = ddelta if alive is None else torch.where(alive, ddelta, 0.0)
    out = {"du": (du.reshape(u.shape) + s["skip"] * ds).to(dtype), "ddelta": ddelta.to(dtype), "dA": dA.view(c.D, c.N), "dB": dB.to(dtype),
           "dC": dC.to(dtype), "dskip": (ds * u).sum((0, 1)), "dz": None, "dbias": ddelta.sum((0, 1)),
           "dh0": None if s["h0"] is None else dh0.reshape(c.B, c.D, c.N)}
    if s["z"] is not None:
        z = s["z"].float()
        y = c.flat(torch.stack(y)) + s["skip"] * u
        out["dz"] = (dy * y * _sigmoid(z) * (1 + z * (1 - _sigmoid(z)))).to(dtype)
    return out


def _scan_step(s):
    u, G, N = s["u"].float(), *s["Bm"].shape[1:]
    shape = (u.shape[0], G, -1, N)
    dt = _softplus(s["delta"].float() + s["bias"])
    h = s["h"] * torch.exp(dt[..., None] * s["A"])
    h = h.view(shape) + (dt * u).view(*shape[:3], 1) * s["Bm"].float()[:, :, None]
    y = (h * s["Cm"].float()[:, :, None]).sum(-1).view(u.shape) + s["skip"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * _sigmoid(z)
    return y.to(s["u"].dtype), h.view(s["h"].shape)


def _conv_sum(s):
    """The inputs with the state in front of them, and the convolution before its activation."""
    x, K = s["x"].float(), s["w"].shape[1]
    state = x.new_zeros((x.shape[0], K - 1, x.shape[2])) if s["state"] is None else s["state"].float()
    x = torch.cat([state, x], 1)
    T = x.shape[1] - K + 1
    return x, T, sum(x[:, j:j + T] * s["w"][:, j].float() for j in range(K)) + s["bias"].float()


def _ends(s, T):
    """Where each sequence's last K - 1 inputs stand behind its state: [B, K - 1, D] indexes."""
    B, K = s["x"].shape[0], s["w"].shape[1]
    n = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    return (n[:, None] + torch.arange(K - 1, device=DEV))[..., None].expand(B, K - 1, s["x"].shape[2])


def _conv(s):
    x, T, c = _conv_sum(s)
    y, alive = c * _sigmoid(c), _alive(s["lengths"], T)
    y = y if alive is None else torch.where(alive, y, 0.0)
    return y.to(s["x"].dtype), x.gather(1, _ends(s, T)).to(s["x"].dtype)


def _conv_backward(s):
    x, T, c = _conv_sum(s)
    K, dtype, alive = s["w"].shape[1], s["x"].dtype, _alive(s["lengths"], T)
    g = _sigmoid(c)
    dc = s["dy"].float() * g * (1 + c * (1 - g))
    dc = dc if alive is None else torch.where(alive, dc, 0.0)
    dx = torch.zeros_like(x)
    dx.scatter_add_(1, _ends(s, T), s["dlast"].float())
    dw = []
    for j in range(K):
        dx[:, j:j + T] += dc * s["w"][:, j].float()
        dw.append((dc * x[:, j:j + T]).sum((0, 1)))
    return {"dx": dx[:, K - 1:].to(dtype), "dw": torch.stack(dw, 1), "dbias": dc.sum((0, 1)),
            "dstate": None if s["state"] is None else dx[:, :K - 1].to(dtype)}


def _conv_step(s):
    x = torch.cat([s["state"], s["x"][:, None]], 1)
    c = (x.float() * s["w"].float().t()).sum(1) + s["bias"].float()
    return (c * _sigmoid(c)).to(s["x"].dtype), x[:, 1:].contiguous()


def _norm_parts(s):
    """What is normalised (the sum as it is stored), in fp32, and 1 / rms of each row."""
    t = s["x"] if s["r"] is None else (s["x"].float() + s["r"].float()).to(s["r"].dtype)
    f = t.float()
    return t, f, torch.rsqrt(f.square().mean(1, keepdim=True) + EPS)


def _norm(s):
    t, f, inv = _norm_parts(s)
    return (f * inv * s["w"].float()).to(s["x"].dtype), None if s["r"] is None else t


def _norm_codes(s):
    t, f, inv = _norm_parts(s)
    y = f * inv * s["w"].float()
    scale = y.abs().amax(1) / 127
    values = torch.round(y / torch.where(scale > 0, scale, 1.0)[:, None]) * scale[:, None]
    return values.to(torch.bfloat16), scale, None if s["r"] is None else t


def _norm_backward(s):
    t = s["t"].float()
    inv = torch.rsqrt(t.square().mean(1, keepdim=True) + EPS)
    dy, n = s["dy"].float(), t * inv
    g = dy * s["w"].float()
    dx = (g - n * (g * n).mean(1, keepdim=True)) * inv + s["dt"].float()
    return dx.to(s["t"].dtype), (dy * n).sum(0)


_PLAIN = {"scan": _scan, "scan_backward": _scan_backward, "scan_step": _scan_step, "conv": _conv, "conv_backward": _conv_backward,
          "conv_step": _conv_step, "norm": _norm, "norm_codes": _norm_codes, "norm_backward": _norm_backward}


def _called(s):
    import scan_linear_rnn_amd as sr

    op = s["op"]
    if op.startswith("scan"):
        given = {"skip": s["skip"], "z": s["z"], "delta_bias": s["bias"], "delta_softplus": True}
        args = (s["u"], s["delta"], s["A"], s["Bm"], s["Cm"])
        if op == "scan":
            return sr.selective_scan_forward(*args, h0=s["h0"], lengths=s["lengths"], return_last=True, **given)
        if op == "scan_step":
            return sr.selective_step(*args, h_prev=s["h"], **given)
        names = ("du", "ddelta", "dA", "dB", "dC", "dskip", "dz", "dbias", "dh0")
        return dict(zip(names, sr.selective_scan_backward(*args, s["dy"], h0=s["h0"], lengths=s["lengths"], dh_last=s["dlast"], **given)))
    if op.startswith("conv"):
        if op == "conv":
            return sr.causal_conv_forward(s["x"], s["w"], s["bias"], silu=True, state=s["state"], lengths=s["lengths"], return_last=True)
        if op == "conv_step":
            return sr.causal_conv_step(s["x"], s["w"], s["bias"], silu=True, state=s["state"])
        return dict(zip(("dx", "dw", "dbias", "dstate"), sr.causal_conv_backward(
            s["x"], s["w"], s["dy"], s["bias"], silu=True, state=s["state"], lengths=s["lengths"], dlast=s["dlast"])))
    if op == "norm_backward":
        return sr.rms_norm_backward(s["t"], s["w"], s["dy"], dtotal=s["dt"], eps=EPS)
    if op == "norm":
        y = sr.rms_norm_forward(s["x"], s["w"], s["r"], eps=EPS)
        return (y, None) if s["r"] is None else y
    q, scale, *total = sr.rms_norm_quantize(s["x"], s["w"], s["r"], eps=EPS)
    values = torch.empty(s["x"].shape, dtype=torch.bfloat16, device=DEV)  # codes as the values they stand for
    torch.mul(q[:, :s["x"].shape[1]], scale[:, None], out=values)
    return values, scale, total[0] if total else None


def run(state):
    return _called(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- inputs


def _lengths(g, B, T):
    """Lengths of a padded batch: one full, one of a single token and one empty where there are three or more."""
    n = torch.randint(0, T + 1, (B,), device=DEV, generator=g).to(torch.int32)
    n[:1] = T
    if B > 2:
        n[1], n[2] = min(1, T), 0
    return n


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, dtype = case["op"], DTYPES[case["dtype"]]
    s = {"op": op}

    def normal(*shape, std=1.0, dtype=dtype):
        return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(dtype)

    if op.startswith("scan"):
        B, D, N, G = case["B"], case["D"], case["N"], case["G"]
        lead = (B,) if op == "scan_step" else (B, case["T"])
        s["u"], s["delta"], s["z"] = normal(*lead, D), normal(*lead, D, std=0.5), normal(*lead, D) if case["gated"] else None
        s["Bm"], s["Cm"] = normal(*lead, G, N), normal(*lead, G, N)
        # rates near 1 .. N and steps of 0.001 .. 0.1, as such layers start and stay near
        s["A"] = -torch.arange(1, N + 1, device=DEV).float() * torch.exp(normal(D, N, std=0.1, dtype=torch.float32))
        step = torch.exp(torch.empty(D, device=DEV).uniform_(math.log(1e-3), math.log(0.1), generator=g))
        s["bias"] = torch.log(torch.expm1(step))
        s["skip"] = 1 + normal(D, std=0.1, dtype=torch.float32)
        if op == "scan_step":
            s["h"] = normal(B, D, N, dtype=torch.float32)
        else:
            s["lengths"] = _lengths(g, B, case["T"]) if case["ragged"] else None
            s["h0"] = normal(B, D, N, dtype=torch.float32) if case["ragged"] else None
            if op == "scan_backward":
                s["dy"] = normal(*lead, D)
                s["dlast"] = normal(B, D, N, dtype=torch.float32) if case["ragged"] else None
    elif op.startswith("conv"):
        B, D, K = case["B"], case["D"], case["K"]
        lead = (B,) if op == "conv_step" else (B, case["T"])
        s["x"], s["w"], s["bias"] = normal(*lead, D), normal(D, K, std=K ** -0.5), normal(D, std=0.1)
        s["state"] = normal(B, K - 1, D) if op == "conv_step" or case["ragged"] else None
        if op != "conv_step":
            s["lengths"] = _lengths(g, B, case["T"]) if case["ragged"] else None
            if op == "conv_backward":
                s["dy"], s["dlast"] = normal(*lead, D), normal(B, K - 1, D)
    else:
        M, D = case["M"], case["D"]
        rdtype = DTYPES[case["residual"]] if case["residual"] else None
        s["w"] = 1 + normal(D, std=0.1)
        if op == "norm_backward":
            s["t"], s["dy"], s["dt"] = normal(M, D, std=3.0, dtype=rdtype), normal(M, D), normal(M, D, dtype=rdtype)
        else:
            # a residual stream with a few loud channels, and a layer's output to be added to it
            s["x"], s["r"] = normal(M, D), normal(M, D, std=3.0, dtype=rdtype) if rdtype else None
            loud = torch.randint(0, D, (max(1, D // 256),), device=DEV, generator=g)
            (s["x"] if s["r"] is None else s["r"])[:, loud] *= 8.0
    return s


def work(case):
    op, size = case["op"], {"fp32": 4, "bf16": 2}
    e = size[case["dtype"]]
    if op.startswith("scan"):
        B, D, N, G = case["B"], case["D"], case["N"], case["G"]
        T, gated = case.get("T", 1), int(case["gated"])
        x, bc, states, weights = e * B * T * D, e * B * T * G * N, 4 * B * D * N, 4 * (D * N + 2 * D)
        if op == "scan_backward":  # u, delta, dy, z; du, ddelta, dz; B, C and their gradients
            kept = 3 * case["ragged"]  # h0 and the gradients of both states
            return {"bytes": x * (5 + 2 * gated) + 4 * bc + states * kept + 2 * weights, "flops": 20 * B * T * D * N}
        # u, delta, z and y; B and C; the states
        kept = 2 if op == "scan_step" else 1 + case["ragged"]
        return {"bytes": x * (3 + gated) + 2 * bc + states * kept + weights, "flops": 7 * B * T * D * N}
    if op.startswith("conv"):
        B, D, K = case["B"], case["D"], case["K"]
        x, state, weights = e * B * case.get("T", 1) * D, e * B * (K - 1) * D, e * D * (K + 1)
        n = x // e
        if op == "conv_backward":
            return {"bytes": 3 * x + (1 + 2 * case["ragged"]) * state + weights + 4 * D * (K + 1), "flops": (6 * K + 10) * n}
        kept = 2 if op == "conv_step" else 1 + case["ragged"]
        return {"bytes": 2 * x + kept * state + weights, "flops": (2 * K + 5) * n}
    n, D = case["M"] * case["D"], case["D"]
    r = size.get(case["residual"], 0)
    if op == "norm_backward":
        return {"bytes": n * (e + 3 * r) + e * D + 4 * D, "flops": 10 * n}
    out = e if op == "norm" else 1
    return {"bytes": n * (e + 2 * r + out) + e * D + (0 if op == "norm" else 4 * case["M"]), "flops": (4 if op == "norm" else 7) * n}


# -------------------------------------------------------------------- exact


def _exact_scan(s, backward):
    """Token after token in 64 bits."""
    f = lambda t: None if t is None else t.double()  # noqa: E731
    u, delta, A, Bm, Cm, skip, z = (f(s[k]) for k in ("u", "delta", "A", "Bm", "Cm", "skip", "z"))
    B, T, D = u.shape
    N, per = A.shape[1], D // Bm.shape[2]
    x = delta + f(s["bias"])
    dt = torch.logaddexp(x, torch.zeros_like(x))
    spread = lambda t: t.repeat_interleave(per, 1)  # noqa: E731  [B,G,N] to the channels
    n = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    h = torch.zeros((B, D, N), device=DEV, dtype=torch.float64) if s["h0"] is None else f(s["h0"])
    kept = torch.empty((T + 1, B, D, N), device=DEV, dtype=torch.float64) if backward else None
    y = torch.zeros_like(u)
    whole = s["lengths"] is None
    for t in range(T):
        if backward:
            kept[t] = h
        new = torch.exp(dt[:, t, :, None] * A) * h + (dt[:, t] * u[:, t])[..., None] * spread(Bm[:, t])
        h = new if whole else torch.where((t < n)[:, None, None], new, h)
        y[:, t] = (h * spread(Cm[:, t])).sum(2)
    y += skip * u
    seen = (torch.arange(T, device=DEV)[None] < n[:, None])[..., None].double()
    gate = 1.0 if z is None else z / (1 + torch.exp(-z))
    if not backward:
        return y * gate * seen, h
    kept[T] = h
    dy = f(s["dy"]) * seen
    ds = dy * gate
    du, ddt, dB, dC = skip * ds, torch.zeros_like(u), torch.zeros_like(Bm), torch.zeros_like(Cm)
    dA = torch.zeros_like(A)
    G = torch.zeros_like(h) if s["dlast"] is None else f(s["dlast"])
    for t in range(T - 1, -1, -1):
        on = seen[:, t, :, None]
        grown = G + ds[:, t, :, None] * spread(Cm[:, t])
        a = torch.exp(dt[:, t, :, None] * A)
        dC[:, t] = (ds[:, t, :, None] * kept[t + 1]).view(B, -1, per, N).sum(2)
        dB[:, t] = (on * grown * (dt[:, t] * u[:, t])[..., None]).view(B, -1, per, N).sum(2)
        write = (on * grown * spread(Bm[:, t])).sum(2)
        du[:, t] += dt[:, t] * write
        far = on * grown * a * kept[t]
        ddt[:, t] = u[:, t] * write + (far * A).sum(2)
        dA += (far * dt[:, t, :, None]).sum(0)
        G = G * (1 - on) + grown * a * on
    ddelta = ddt / (1 + torch.exp(-x))
    dz = None
    if z is not None:
        p = 1 / (1 + torch.exp(-z))
        dz = dy * y * (p + z * p * (1 - p))
    return {"du": du, "ddelta": ddelta, "dA": dA, "dB": dB, "dC": dC, "dskip": (ds * u).sum((0, 1)), "dz": dz, "dbias": ddelta.sum((0, 1)),
            "dh0": None if s["h0"] is None else G}


def _exact_step(s):
    u, delta = s["u"].double(), s["delta"].double() + s["bias"].double()
    dt, per = torch.logaddexp(delta, torch.zeros_like(delta)), u.shape[1] // s["Bm"].shape[1]
    Bm, Cm = (s[k].double().repeat_interleave(per, 1) for k in ("Bm", "Cm"))
    h = torch.exp(dt[..., None] * s["A"].double()) * s["h"].double() + (dt * u)[..., None] * Bm
    y = (h * Cm).sum(2) + s["skip"].double() * u
    if s["z"] is not None:
        y = y * s["z"].double() / (1 + torch.exp(-s["z"].double()))
    return y, h


def _exact_conv(s, backward):
    """Each output from the inputs that it sees, found by their index; a token in front of the sequence is the state's or zero."""
    x, w = s["x"].double(), s["w"].double()
    B, T, D = x.shape
    K = w.shape[1]
    n = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    front = torch.zeros((B, K - 1, D), device=DEV, dtype=torch.float64) if s["state"] is None else s["state"].double()
    line = torch.cat([front, x], 1)
    seen = (torch.arange(T, device=DEV)[None] < n[:, None])[..., None].double()
    windows = line.unfold(1, K, 1)  # [B,T,D,K]
    c = (windows * w).sum(3) + s["bias"].double()
    p = 1 / (1 + torch.exp(-c))
    at = n[:, None] + torch.arange(K - 1, device=DEV)[None]
    rows = torch.arange(B, device=DEV)[:, None]
    if not backward:
        return c * p * seen, line[rows, at]
    dc = s["dy"].double() * (p + c * p * (1 - p)) * seen
    dline = torch.zeros_like(line)
    dline[rows, at] = s["dlast"].double()
    ahead = torch.nn.functional.pad(dc, (0, 0, K - 1, K - 1)).unfold(1, K, 1)  # what the tokens from each place on return to it
    dline += (ahead * w.flip(1)).sum(3)
    return {"dx": dline[:, K - 1:], "dw": (dc[..., None] * windows).sum((0, 1)), "dbias": dc.sum((0, 1)),
            "dstate": None if s["state"] is None else dline[:, :K - 1]}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("scan", "scan_backward"):
        return _exact_scan(s, op == "scan_backward")
    if op == "scan_step":
        return _exact_step(s)
    if op in ("conv", "conv_backward"):
        return _exact_conv(s, op == "conv_backward")
    w = s["w"].double()
    if op == "conv_step":
        line = torch.cat([s["state"], s["x"].unsqueeze(1)], 1).double()
        c = torch.einsum("bkd,dk->bd", line, w) + s["bias"].double()
        return c / (1 + torch.exp(-c)), line[:, 1:]
    if op == "norm_backward":
        t, dy = s["t"].double(), s["dy"].double()
        ms = (t * t).sum(1, keepdim=True) / case["D"] + EPS
        g = dy * w
        dx = g / ms.sqrt() - t * (g * t).sum(1, keepdim=True) / (case["D"] * ms.sqrt() ** 3) + s["dt"].double()
        return dx, (dy * t / ms.sqrt()).sum(0)
    # the norm is of the sum as it is stored, whose rounding is part of the definition
    t = s["x"].double()
    if s["r"] is not None:
        t = (s["x"].float() + s["r"].float()).to(s["r"].dtype).double()
    y = t / ((t * t).sum(1, keepdim=True) / case["D"] + EPS).sqrt() * w
    total = None if s["r"] is None else s["x"].double() + s["r"].double()
    if op == "norm":
        return y, total
    scale = y.abs().max(1).values / 127
    return None, scale, total
