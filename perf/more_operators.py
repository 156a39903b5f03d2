"""Workloads of the norm beside the projections, of projections on 8-bit rows, and of the gradients through
frozen NVFP4 weights.

Five operators, each with its plain form (elementary torch operations in 32 bits, rounded once at the end) and
its call of the library:

  norm         the residual's sum and the root-mean-square norm:  s = x + r,  y = s / sqrt(mean(s^2) + eps) * w,
               y in 16 bits or in 8 bits with a scale per row (q = e4m3(y / scale), scale = max |y| / 448)
  norm_grad    its gradient:  dx = ds + (g - s mean(g s) / (mean(s^2) + eps)) / sqrt(mean(s^2) + eps),  g = w dy,
               dw = sum over the rows of dy s / sqrt(mean(s^2) + eps)
  rows         the channel-FP8 projection of such 8-bit rows:  y = scale_m c_n sum over k of xq W
  grad         a projection's gradient towards its input:  dx = dy W,  W in NVFP4
  swiglu_grad  the gated projection's gradient towards its gate and up rows, g and u computed again from x:
               dgate = dh u sigma(g) (1 + g (1 - sigma(g))),  dup = dh g sigma(g)

Hidden sizes and projection shapes are the library's own workloads (hidden sizes 2048 and 5120; dense projection
4352 x 5120; the gated MLP's packed 4352 x 5120 gate/up rows and 5120 x 2176 down projection).
"""
import torch

own = False

DEVICE = "cuda"
EPS = 1e-6

# E4M3 bytes of 2^-8 .. 2^-4, the block scales of the library's synthetic weights.
SCALE_BYTES = (0x02, 0x04, 0x08, 0x10, 0x18)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _norm(name, m, k, *, residual, bits):
    return {"name": name, "op": "norm", "m": m, "k": k, "residual": residual, "bits": bits}


def _norm_grad(name, m, k, *, residual):
    return {"name": name, "op": "norm_grad", "m": m, "k": k, "residual": residual}


def _product(name, op, m, n, k, layout=0):
    return {"name": name, "op": op, "m": m, "n": n, "k": k, "layout": layout}


def listed():
    return [
        # one decode step of a single request: what counts is the latency
        _norm("norm_decode1", 1, 2048, residual=True, bits=16),
        # a ragged prompt in front of a projection that reads 8-bit rows
        _norm("norm_333_8bit", 333, 5120, residual=True, bits=8),
        # a prefill batch
        _norm("norm_prefill8192", 8192, 2048, residual=True, bits=16),
        # the gradient of a short training micro-batch of odd length
        _norm_grad("norm_grad_333", 333, 5120, residual=True),
        # a training batch
        _norm_grad("norm_grad_8192", 8192, 2048, residual=True),
        # a decode batch of 13 requests on the channel-FP8 projection
        _product("rows_decode13", "rows", 13, 4352, 5120),
        # a ragged prompt
        _product("rows_333", "rows", 333, 4352, 5120),
        # a prefill batch on it
        _product("rows_prefill8192", "rows", 8192, 4352, 5120),
        # the last tokens of a few short sequences, back through the projection
        _product("grad_24", "grad", 24, 4352, 5120),
        # a training batch, back through the gated MLP's down projection
        _product("grad_4096", "grad", 4096, 5120, 2176),
        # a short training micro-batch of odd length through the gated projection, interleaved rows
        _product("swiglu_grad_333", "swiglu_grad", 333, 4352, 5120, layout=1),
        # a training batch
        _product("swiglu_grad_4096", "swiglu_grad", 4096, 4352, 5120),
    ]


def _between(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = low * (high / low) ** rng.random()
    return min(high // step * step, max(-(-low // step) * step, round(v / step) * step))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "rows", "grad", "swiglu_grad"))
    if op in ("norm", "norm_grad"):
        k = _between(rng, 64, 16384, 8)
        m = _between(rng, 1, min(16384, 8192 * 5120 // k))
        c = {"op": op, "m": m, "k": k, "residual": rng.random() < 0.7}
        return {**c, "bits": rng.choice((8, 16))} if op == "norm" else c
    n, k = _between(rng, 64, 8192, 32), _between(rng, 128, 8192, 128)
    m = _between(rng, 1, max(1, min(8192, 4096 * 4352 * 5120 // (n * k))))
    return {"op": op, "m": m, "n": n, "k": k, "layout": rng.randint(0, 1) if op == "swiglu_grad" else 0}


# ---- inputs ----------------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(torch.float16)


def _out(*shape, dtype=torch.float16):
    return torch.empty(shape, dtype=dtype, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_grad"):
        # a residual stream has a few columns that are much larger than the others
        columns = torch.exp(0.5 * torch.randn((k,), generator=g, device=DEVICE))
        s["w"] = (1.0 + 0.2 * torch.randn((k,), generator=g, device=DEVICE)).to(torch.float16)
        s["x"] = (torch.randn((m, k), generator=g, device=DEVICE) * columns).to(torch.float16)
        if op == "norm":
            s["r"] = _normal(g, m, k, scale=0.3) if case["residual"] else None
            s["s"] = _out(m, k) if case["residual"] else None
            s["y"] = _out(m, k) if case["bits"] == 16 else None
            s["q"] = _out(m, k, dtype=torch.uint8) if case["bits"] == 8 else None
            s["q_scale"] = _out(m, dtype=torch.float32) if case["bits"] == 8 else None
        else:
            s["dy"] = _normal(g, m, k)
            s["ds"] = _normal(g, m, k) if case["residual"] else None
            s["dx"], s["dw"] = _out(m, k), _out(k, dtype=torch.float32)
    elif op == "rows":
        n = case["n"]
        x = torch.randn((m, k), generator=g, device=DEVICE)
        s["x_scale"] = x.abs().amax(dim=1) / 448.0
        s["xq"] = (x / s["x_scale"][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        w = torch.randn((n, k), generator=g, device=DEVICE) * k ** -0.5
        s["c_scale"] = w.abs().amax(dim=1) / 448.0
        s["codes"] = (w / s["c_scale"][:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["y"] = _out(m, n)
    else:
        n = case["n"]
        s["codes"] = torch.randint(0, 256, (1, n, k // 2), generator=g, device=DEVICE, dtype=torch.uint8)
        pick = torch.randint(0, len(SCALE_BYTES), (1, n, k // 16), generator=g, device=DEVICE)
        s["scales"] = torch.tensor(SCALE_BYTES, dtype=torch.uint8, device=DEVICE)[pick]
        s["gscale"] = torch.full((1,), 0.37, device=DEVICE)
        if op == "grad":
            s["dy"], s["dx"] = _normal(g, m, n), _out(m, k)
        else:
            s["x"], s["dh"], s["dz"] = _normal(g, m, k, scale=0.5), _normal(g, m, n // 2), _out(m, n)
    if own:
        import gemm_nvfp4_amd as G
        if op == "norm_grad":
            s["ws"] = _out(max(16, G.nvfp4_add_rms_norm_grad_ws_bytes(m, k)), dtype=torch.uint8)
        elif op == "rows":
            s["weights"] = G.FP8ChannelTensor(s["codes"], s["c_scale"])
        elif op != "norm":
            s["weights"] = G.NVFP4Tensor(s["codes"], s["scales"], s["gscale"])
            size = G.nvfp4_linear_grad_ws_bytes if op == "grad" else G.nvfp4_linear_swiglu_grad_ws_bytes
            s["ws"] = _out(max(16, size(m, n, k)), dtype=torch.uint8)
    return s


# ---- one pass --------------------------------------------------------------------------------------

def run(s):
    return _library(s) if own else _plain(s)


def _library(s):
    import gemm_nvfp4_amd as G
    c = s["case"]
    op = c["op"]
    if op == "norm":
        stream, y, q, q_scale = G.nvfp4_add_rms_norm(s["x"], s["w"], residual=s["r"], eps=EPS, s=s["s"], y=s["y"], q=s["q"],
                                                     q_scale=s["q_scale"], want_y=c["bits"] == 16, want_q=c["bits"] == 8)
        return (stream, y) if c["bits"] == 16 else (stream, q.view(torch.float8_e4m3fn), q_scale)
    if op == "norm_grad":
        return G.nvfp4_add_rms_norm_grad(s["x"], s["dy"], s["w"], ds=s["ds"], eps=EPS, dx=s["dx"], dweight=s["dw"],
                                         ws=s["ws"])
    if op == "rows":
        return G.nvfp4_linear_fp8_rows(s["xq"], s["x_scale"], s["weights"], y=s["y"])
    if op == "grad":
        return G.nvfp4_linear_grad(s["dy"], s["weights"], dx=s["dx"], ws=s["ws"])
    return G.nvfp4_linear_swiglu_grad(s["x"], s["dh"], s["weights"], c["layout"], dz=s["dz"], ws=s["ws"])


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "norm":
        t = s["x"].float()
        if c["residual"]:
            t = t + s["r"].float()
        y = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS) * s["w"].float()
        stream = t.to(torch.float16) if c["residual"] else None
        if c["bits"] == 16:
            return stream, y.to(torch.float16)
        scale = y.abs().amax(dim=1) / 448.0
        return stream, (y / scale[:, None]).to(torch.float8_e4m3fn), scale
    if op == "norm_grad":
        t, dy = s["x"].float(), s["dy"].float()
        rstd = torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS)
        g = dy * s["w"].float()
        dx = rstd * (g - t * (rstd * rstd * (g * t).mean(dim=1, keepdim=True)))
        if c["residual"]:
            dx = dx + s["ds"].float()
        return dx.to(torch.float16), (dy * t * rstd).sum(dim=0)
    if op == "rows":
        x, w = s["xq"].view(torch.float8_e4m3fn).float(), s["codes"].view(torch.float8_e4m3fn).float()
        return (x @ w.t() * s["x_scale"][:, None] * s["c_scale"][None, :]).to(torch.float16)
    if op == "grad":
        return (s["dy"].float() @ _weights(s)).to(torch.float16)
    z = s["x"].float() @ _weights(s).t()
    half = c["n"] // 2
    gate, up = (z[:, 0::2], z[:, 1::2]) if c["layout"] else (z[:, :half], z[:, half:])
    dh = s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dgate, dup = dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig
    return (torch.stack((dgate, dup), dim=2).flatten(1) if c["layout"] else torch.cat((dgate, dup), dim=1)).to(torch.float16)


def _weights(s):
    """The NVFP4 weight in 32 bits: a code's value times its 16-column block's scale times the global scale."""
    codes = s["codes"][0].long()
    table = torch.tensor(E2M1, device=DEVICE)
    w = torch.stack((table[codes & 15], table[codes >> 4]), dim=-1).view(codes.shape[0], -1, 16)
    return (w * s["scales"][0].view(torch.float8_e4m3fn).float()[:, :, None]).view(codes.shape[0], -1) * s["gscale"]


# ---- what a pass cannot do without, and its result in 64 bits --------------------------------------

def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "norm":
        rows = 2 * (3 if case["residual"] else 1) * k
        return {"bytes": m * (rows + (2 * k if case["bits"] == 16 else k + 4)) + 2 * k, "flops": 5 * m * k}
    if op == "norm_grad":
        return {"bytes": 2 * m * k * (4 if case["residual"] else 3) + 6 * k, "flops": 11 * m * k}
    n = case["n"]
    if op == "rows":
        return {"bytes": n * k + 4 * n + m * k + 4 * m + 2 * m * n, "flops": 2 * m * n * k}
    weights = n * k * 9 // 16 + 4
    if op == "grad":
        return {"bytes": weights + 2 * m * (n + k), "flops": 2 * m * n * k}
    return {"bytes": weights + 2 * m * k + m * n + 2 * m * n, "flops": 2 * m * n * k + 6 * m * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        t, w = s["x"].double(), s["w"].double()
        if op == "norm" and case["residual"]:
            t = t + s["r"].double()
        length = torch.sqrt(t.square().mean(dim=1) + EPS)[:, None]
        if op == "norm":
            y = t / length * w
            stream = t if case["residual"] else None
            if case["bits"] == 16:
                return stream, y
            scale = y.abs().amax(dim=1) / 448
            return stream, y / scale[:, None], scale
        dy = s["dy"].double()
        unit = t / length
        # the part of w dy along the unit row does not reach x, but for what eps leaves of it
        along = (w * dy * unit).mean(dim=1)[:, None]
        dx = (w * dy - unit * along) / length
        return (dx + s["ds"].double() if case["residual"] else dx), (dy * unit).sum(dim=0)
    if op == "rows":
        y = _e4m3(s["xq"]) @ _e4m3(s["codes"]).t()
        return y * s["x_scale"].double()[:, None] * s["c_scale"].double()
    w = _exact_weights(s)
    if op == "grad":
        return s["dy"].double() @ w
    x, dh = s["x"].double(), s["dh"].double()
    half = case["n"] // 2
    rows = torch.arange(case["n"], device=DEVICE)
    gates, ups = (rows[0::2], rows[1::2]) if case["layout"] else (rows[:half], rows[half:])
    gate, up = x @ w[gates].t(), x @ w[ups].t()
    sig = torch.sigmoid(gate)
    dz = torch.empty((case["m"], case["n"]), dtype=torch.float64, device=DEVICE)
    dz[:, gates] = dh * up * (sig + gate * sig * torch.sigmoid(-gate))
    dz[:, ups] = dh * gate * sig
    return dz


def _e4m3(bytes_):
    """Values of E4M3 bytes in 64 bits from the format's definition: sign, exponent and mantissa fields."""
    b = bytes_.long()
    exp, man = (b // 8) % 16, (b % 8).double()
    v = torch.where(exp == 0, man * 2.0 ** -9, torch.exp2((exp - 7).double()) * (1.0 + man / 8.0))
    return torch.where(b >= 128, -v, v)


def _exact_weights(s):
    """The NVFP4 weight in 64 bits from the formats' definition."""
    codes = s["codes"][0].long()
    nib = torch.stack((codes % 16, codes // 16), dim=2).flatten(1)
    exp, man = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(exp == 0, man * 0.5, torch.exp2((exp - 1).double()) * (1.0 + man * 0.5))
    value = torch.where(nib >= 8, -mag, mag)
    return value * _e4m3(s["scales"][0]).repeat_interleave(16, dim=1) * s["gscale"].double()
