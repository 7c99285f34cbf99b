"""Measured cases of the 8-bit products and the AdamW step.

Each case names one call a user makes: codes and scales of activations
(``rows``) or of a weight (``columns``), the 8-bit integer product with a scale
per token and per output channel (``product``), the single-token minGRU step on
8-bit weights (``step``), and the AdamW step over many tensors (``adamw``).
``run`` computes it with elementary torch operations in 32 bits, or, with
``own``, through the package's entry points; ``exact`` in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
PAD = 128        # stored rows of codes are a multiple of this many bytes, zeros behind the data
BLOCK = 256      # elements that share a scale of the 8-bit AdamW states
TOP = 448.0      # largest float8 e4m3 value
TINY = 2.0 ** -9  # smallest positive one
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
HYPER = {"lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.01}


def listed():
    return [
        # The activations of a prefill of 256 sequences of 512 tokens, width 2048.
        {"name": "rows_prefill_131072x2048", "op": "rows", "M": 131072, "K": 2048, "dtype": "fp32"},
        # One token of each of 256 streams of the same layer.
        {"name": "rows_decode_256x2048", "op": "rows", "M": 256, "K": 2048, "dtype": "bf16"},
        # The layer's input projection, quantised after a training step changed it.
        {"name": "columns_2048x4096", "op": "columns", "K": 2048, "N": 4096, "dtype": "fp32"},
        # A single stream's token through the input projection: the smallest call, latency counts.
        {"name": "product_1x2048x4096", "op": "product", "M": 1, "K": 2048, "N": 4096, "out": "fp32"},
        # 256 streams decoding through the input projection.
        {"name": "product_256x2048x4096", "op": "product", "M": 256, "K": 2048, "N": 4096, "out": "fp32"},
        # Ragged everywhere: rows, depth and columns that end inside a tile.
        {"name": "product_2047x1000x1537", "op": "product", "M": 2047, "K": 1000, "N": 1537, "out": "fp32"},
        # The prefill's projection, [k | p] in bf16 for the scan: the largest product.
        {"name": "product_131072x2048x4096", "op": "product", "M": 131072, "K": 2048, "N": 4096, "out": "bf16"},
        # The decode step over 256 streams, with the output projection.
        {"name": "step_256_d2048", "op": "step", "B": 256, "D_in": 2048, "D_h": 2048, "D_out": 2048, "dtype": "bf16"},
        # Two streams of the width-512 layer without an output projection, fp32 activations.
        {"name": "step_2_d512", "op": "step", "B": 2, "D_in": 512, "D_h": 512, "D_out": 0, "dtype": "fp32"},
        # The weights of 8 layers of width 2048, everything in fp32.
        {"name": "adamw_fp32_8x_d2048", "op": "adamw", "sizes": "2048x4096,2048x2048", "repeat": 8, "param": "fp32",
         "grad": "fp32", "bits": 32},
        # The same weights with bf16 gradients and states in 8 bits.
        {"name": "adamw_8bit_8x_d2048", "op": "adamw", "sizes": "2048x4096,2048x2048", "repeat": 8, "param": "fp32",
         "grad": "bf16", "bits": 8},
        # Many small tensors of odd sizes (widths 16 and 192, decay rates, a lone value), bf16 weights.
        {"name": "adamw_8bit_small", "op": "adamw", "sizes": "16x32,16x16,192x384,192x192,192,1001,1", "repeat": 7,
         "param": "bf16", "grad": "bf16", "bits": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "columns", "product", "product", "step", "adamw"])
    if op == "rows":
        K = _log(rng, 16, 4096)
        return {"op": op, "M": _log(rng, 1, min(131072, 131072 * 2048 // K)), "K": K, "dtype": rng.choice(["fp32", "bf16"])}
    if op == "columns":
        return {"op": op, "K": _log(rng, 16, 4096), "N": _log(rng, 16, 8192), "dtype": rng.choice(["fp32", "bf16"])}
    if op == "product":
        K, N = _log(rng, 16, 4096), _log(rng, 16, 8192)
        out = rng.choice(["fp32", "bf16"])
        M = _log(rng, 1, min(131072, 131072 * 2048 * 4096 // (K * N), (1 << 28 if out == "fp32" else 1 << 29) // N))
        return {"op": op, "M": M, "K": K, "N": N, "out": out}
    if op == "step":
        dtype = rng.choice(["fp32", "bf16"])
        D_out = _log(rng, 16, 4096) if dtype == "bf16" else 0
        return {"op": op, "B": _log(rng, 1, 1024), "D_in": _log(rng, 16, 4096), "D_h": _log(rng, 16, 4096),
                "D_out": D_out, "dtype": dtype}
    n, repeat = rng.randint(1, 7), rng.randint(1, 7)
    rows = [_log(rng, 1, 2048) for _ in range(n)]
    most = 8 * 2048 * 6144 // (n * repeat)
    sizes = ",".join("%dx%d" % (r, _log(rng, 1, min(4096, most // r))) for r in rows)
    return {"op": op, "sizes": sizes, "repeat": repeat, "param": rng.choice(["fp32", "bf16"]),
            "grad": rng.choice(["fp32", "bf16"]), "bits": rng.choice([8, 32])}


def _pad(k):
    return -(-k // PAD) * PAD


def _shapes(case):
    one = [tuple(int(n) for n in s.split("x")) for s in case["sizes"].split(",")]
    return one * case["repeat"]


def _offsets(shapes):
    """Where each tensor's states start in the flat state buffers, and their length: every tensor at a multiple of BLOCK."""
    at, total = [], 0
    for s in shapes:
        at.append(total)
        total += -(-math.prod(s) // BLOCK) * BLOCK
    return at, total


# ------------------------------------------------------------- plain forms


def _codes(x):
    """Symmetric 8-bit codes of the rows of x [M, K], zero-padded, and the scale of each row."""
    x = x.float()
    top = x.abs().amax(dim=1)
    scale = top / torch.full_like(top, 127.0)  # a true division: by a number it would be a product with a rounded 1/127
    live = torch.isfinite(scale) & (scale > 0)
    q = torch.round(x / torch.where(live, scale, 1.0)[:, None]).clamp(-127, 127)
    q = torch.where(live[:, None], q, 0.0).to(torch.int8)
    q = torch.nn.functional.pad(q, (0, _pad(x.shape[1]) - x.shape[1])).contiguous()
    return q, torch.where(torch.isfinite(scale), scale, torch.nan)


def _product(a, sa, b, sb):
    return (a.float() @ b.float().t()) * (sa[:, None] * sb)


def _block_encode(x, positive):
    """float8 e4m3 codes of x (flat, a multiple of BLOCK) and a scale for each block."""
    x = x.view(-1, BLOCK)
    scale = x.abs().amax(dim=1) / TOP
    y = torch.where(scale[:, None] == 0, 0.0, x / torch.where(scale == 0, 1.0, scale)[:, None])
    if positive:  # a positive second moment never becomes zero
        y = torch.where(x > 0, y.clamp(min=TINY), y)
    return y.to(torch.float8_e4m3fn).view(-1), scale


def _block_decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw_tensor(s, i, t):
    p, g, at = s["params"][i], s["grads"][i], s["at"][i]
    n = p.numel()
    end = at + -(-n // BLOCK) * BLOCK
    eight = s["m_scale"] is not None
    (b1, b2), lr = HYPER["betas"], HYPER["lr"]
    g = g.float().view(-1)
    m, v = s["m"][at:end], s["v"][at:end]
    if eight:
        ms, vs = s["m_scale"][at // BLOCK:end // BLOCK], s["v_scale"][at // BLOCK:end // BLOCK]
        m_old, v_old = _block_decode(m, ms)[:n], _block_decode(v, vs)[:n].square()
    else:
        m_old, v_old = m[:n], v[:n]
    m_new = m_old * b1 + g * (1 - b1)
    v_new = v_old * b2 + g * g * (1 - b2)
    step = m_new / (v_new.sqrt() / math.sqrt(1 - b2 ** t) + HYPER["eps"])
    p.copy_((p.float().view(-1) * (1 - lr * HYPER["weight_decay"]) - step * (lr / (1 - b1 ** t))).view(p.shape))
    if eight:
        grow = lambda x: torch.nn.functional.pad(x, (0, end - at - n))  # noqa: E731
        mc, mz = _block_encode(grow(m_new), False)
        vc, vz = _block_encode(grow(v_new.sqrt()), True)
        m.copy_(mc), v.copy_(vc), ms.copy_(mz), vs.copy_(vz)
    else:
        m[:n].copy_(m_new), v[:n].copy_(v_new)


def _plain(s):
    op = s["op"]
    if op == "rows":
        return _codes(s["x"])
    if op == "columns":
        return _codes(s["W"].t())
    if op == "product":
        return _product(s["a"], s["sa"], s["b"], s["sb"]).to(s["out"])
    if op == "step":
        kp = _product(*_codes(s["x"]), s["W_in"], s["s_in"])
        k, p = kp.chunk(2, dim=1)
        g = torch.where(p >= 0, p + 0.5, torch.sigmoid(p))
        h = s["h"] + torch.sigmoid(k) * (g - s["h"])
        if s["W_out"] is None:
            return h
        return _product(*_codes(h), s["W_out"], s["s_out"]).to(s["x"].dtype), h
    s["t"] += 1
    [_adamw_tensor(s, i, s["t"]) for i in range(len(s["params"]))]
    return _adamw_out(s)


def _adamw_out(s):
    return {k: s[k] for k in ("params", "m", "v", "m_scale", "v_scale")}


def _called(s):
    import scan_linear_rnn_amd as sr

    op = s["op"]
    if op == "rows":
        return sr.quantize_rows(s["x"])
    if op == "columns":
        return sr.quantize_columns(s["W"])
    if op == "product":
        return sr.matmul_i8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=s["out"])
    if op == "step":
        y, h = sr.mingru_step_i8(s["x"], s["W_in"], s["s_in"], s["W_out"], s["s_out"], h_prev=s["h"])
        return h if s["W_out"] is None else (y, h)
    s["t"] += 1
    sr.adamw_step(s["params"], s["grads"], s["m"], s["v"], m_scale=s["m_scale"], v_scale=s["v_scale"], step=s["t"], **HYPER)
    return _adamw_out(s)


def run(state):
    return _called(state) if own else _plain(state)


# ------------------------------------------------------------------- inputs


def _activations(g, M, K, dtype):
    """Tokens of a layer: unit normal, with a few channels eight times as large, as trained layers have."""
    x = torch.empty((M, K), device=DEV).normal_(generator=g)
    loud = torch.randint(0, K, (max(1, K // 256),), device=DEV, generator=g)
    x[:, loud] *= 8.0
    return x.to(dtype)


def _weight(g, K, N):
    return torch.empty((K, N), device=DEV).normal_(0.0, K ** -0.5, generator=g)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"op": op}
    if op == "rows":
        s["x"] = _activations(g, case["M"], case["K"], DTYPES[case["dtype"]])
    elif op == "columns":
        s["W"] = _weight(g, case["K"], case["N"]).to(DTYPES[case["dtype"]])
    elif op == "product":
        s["a"], s["sa"] = _codes(_activations(g, case["M"], case["K"], torch.float32))
        s["b"], s["sb"] = _codes(_weight(g, case["K"], case["N"]).t())
        s["out"] = DTYPES[case["out"]]
    elif op == "step":
        s["x"] = _activations(g, case["B"], case["D_in"], DTYPES[case["dtype"]])
        s["W_in"], s["s_in"] = _codes(_weight(g, case["D_in"], 2 * case["D_h"]).t())
        s["W_out"] = s["s_out"] = None
        if case["D_out"]:
            s["W_out"], s["s_out"] = _codes(_weight(g, case["D_h"], case["D_out"]).t())
        s["h"] = torch.empty((case["B"], case["D_h"]), device=DEV).normal_(generator=g)
    else:
        shapes = _shapes(case)
        s["at"], total = _offsets(shapes)
        s["t"] = 9
        # weights of scale fan_in^-1/2; gradients a few orders apart from tensor to tensor
        s["params"] = [torch.empty(z, device=DEV).normal_(0.0, z[0] ** -0.5, generator=g).to(DTYPES[case["param"]]) for z in shapes]
        s["grads"] = [torch.empty(z, device=DEV).normal_(0.0, 10.0 ** -(2 + i % 3), generator=g).to(DTYPES[case["grad"]])
                      for i, z in enumerate(shapes)]
        m, r = torch.zeros(total, device=DEV), torch.zeros(total, device=DEV)
        for i, (z, at) in enumerate(zip(shapes, s["at"])):
            n = math.prod(z)
            m[at:at + n].normal_(0.0, 0.2 * 10.0 ** -(2 + i % 3), generator=g)
            r[at:at + n].normal_(0.0, 10.0 ** -(2 + i % 3), generator=g).abs_()
        s["m"], s["v"], s["m_scale"], s["v_scale"] = m, r.square(), None, None
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _block_encode(m, False)
            s["v"], s["v_scale"] = _block_encode(r, True)
    return s


def work(case):
    op = case["op"]
    if op == "rows" or op == "columns":
        M, K = (case["M"], case["K"]) if op == "rows" else (case["N"], case["K"])
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": M * K * size + M * _pad(K) + 4 * M, "flops": 3 * M * K}
    if op == "product":
        M, K, N = case["M"], case["K"], case["N"]
        size = 4 if case["out"] == "fp32" else 2
        return {"bytes": M * K + N * K + 4 * (M + N) + size * M * N, "flops": 2 * M * K * N}
    if op == "step":
        B, I, H, O = case["B"], case["D_in"], case["D_h"], case["D_out"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": size * B * (I + O) + 8 * B * H + 2 * H * I + O * H + 4 * (2 * H + O),
                "flops": 2 * B * H * (2 * I + O)}
    n = sum(math.prod(z) for z in _shapes(case))
    size = {"fp32": 4, "bf16": 2}
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (2 * size[case["param"]] + size[case["grad"]] + state), "flops": 16 * n}


# -------------------------------------------------------------------- exact


def _exact_scale(x):
    """A row's scale is an fp32 number by definition, the nearest to its largest magnitude over 127; so is the quotient that is
    rounded to a code, which matters where bf16 values lie on the ties."""
    return (x.abs().max(dim=1).values / 127).float().double()


def _exact_codes(x):
    scale = _exact_scale(x)
    q = torch.zeros_like(x)
    live = scale > 0
    q[live] = torch.round((x[live] / scale[live].unsqueeze(1)).float()).double()
    return q, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rows" or op == "columns":
        x = (s["x"] if op == "rows" else s["W"].t()).double()
        return None, _exact_scale(x)
    if op == "product":
        b = (s["b"].double() * s["sb"].double().unsqueeze(1)).t().contiguous()
        return torch.cat([(a.double() * sa.double().unsqueeze(1)) @ b for a, sa in zip(s["a"].split(16384), s["sa"].split(16384))])
    if op == "step":
        H = case["D_h"]
        q, sx = _exact_codes(s["x"].double())
        w = s["W_in"].double()[:, :case["D_in"]] * s["s_in"].double().unsqueeze(1)
        kp = (q * sx.unsqueeze(1)) @ w.t().contiguous()
        z, p = 1 / (1 + torch.exp(-kp[:, :H])), kp[:, H:]
        cand = torch.where(p >= 0, p + 0.5, 1 / (1 + torch.exp(-p)))
        h = (1 - z) * s["h"].double() + z * cand
        if not case["D_out"]:
            return h
        q, sh = _exact_codes(h)
        w = s["W_out"].double()[:, :H] * s["s_out"].double().unsqueeze(1)
        return (q * sh.unsqueeze(1)) @ w.t().contiguous(), h
    t, (b1, b2) = s["t"] + 1, HYPER["betas"]
    params = []
    m_all, v_all = s["m"].double(), s["v"].double()
    if case["bits"] == 8:
        m_all = (m_all.view(-1, BLOCK) * s["m_scale"].double().unsqueeze(1)).view(-1)
        v_all = (v_all.view(-1, BLOCK) * s["v_scale"].double().unsqueeze(1)).view(-1) ** 2
    for p, g, at in zip(s["params"], s["grads"], s["at"]):
        n = p.numel()
        g = g.double().reshape(-1)
        m_all[at:at + n] = b1 * m_all[at:at + n] + (1 - b1) * g
        v_all[at:at + n] = b2 * v_all[at:at + n] + (1 - b2) * g ** 2
        m_hat, v_hat = m_all[at:at + n] / (1 - b1 ** t), v_all[at:at + n] / (1 - b2 ** t)
        old = p.double().reshape(-1)
        new = old - HYPER["lr"] * HYPER["weight_decay"] * old - HYPER["lr"] * m_hat / (torch.sqrt(v_hat) + HYPER["eps"])
        params.append(new.view(p.shape))
    if case["bits"] == 32:
        return {"params": params, "m": m_all, "v": v_all, "m_scale": None, "v_scale": None}
    scales = {k: (x.view(-1, BLOCK).abs().max(dim=1).values / TOP) for k, x in (("m_scale", m_all), ("v_scale", v_all.sqrt()))}
    return {"params": params, "m": None, "v": None, **scales}
