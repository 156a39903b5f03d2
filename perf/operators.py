"""Workloads of the routing plan's row operators and of the low-rank adapters beside the projections.

Six operators, each with its plain form (elementary torch operations in 32 bits, rounded once at the
end) and its call of the library:

  permute    tokens sorted by expert:           xs[j] = w[p] x[t],  row j = bucket-order position of pair p = (t, k)
  unpermute  expert rows back to their tokens:  out[t] = sum over k of w[t, k] ys[pos(t, k)]
  combine_grad  the gradient of that sum:       dys[j] = w[p] dout[t],  dw[t, k] = dout[t] . ys[pos(t, k)]
  linear     NVFP4 projection with adapters:    y = x W^T + s_a (x A_a^T) B_a^T,  a = the token's adapter
  swiglu     the gated projection with them:    h = silu(g) u,  g and u as y above on the gate and up rows
  add        adapters on a finished result:     out = y + s_a (x A_a^T) B_a^T, rows in token or bucket order

Hidden sizes, expert counts and projection shapes are the library's own workloads (512 experts, top-10,
hidden size 2048; dense projection 4352 x 5120; the gated MLP's packed 4352 x 5120 gate/up rows).
"""
import torch

own = False

DEVICE = "cuda"

# E4M3 bytes of 2^-8 .. 2^-4, the block scales of the library's synthetic weights.
SCALE_BYTES = (0x02, 0x04, 0x08, 0x10, 0x18)
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _rows(name, op, m, topk, experts, k, *, weighted, skipped=0, skew=0.0):
    return {"name": name, "op": op, "m": m, "topk": topk, "experts": experts, "k": k, "weighted": weighted,
            "skipped": skipped, "skew": skew}


def _dense(name, op, m, n, k, rank, adapters, *, without=0, layout=0):
    return {"name": name, "op": op, "m": m, "n": n, "k": k, "rank": rank, "adapters": adapters, "without": without,
            "layout": layout}


def _add(name, m, topk, n, k, rank, adapters, *, bucket, without=0):
    return {"name": name, "op": "add", "m": m, "topk": topk, "n": n, "k": k, "rank": rank, "adapters": adapters,
            "bucket": bucket, "without": without}


def listed():
    return [
        # one decode step of 16 requests, five of whose pairs are padding: what counts is the latency
        _rows("permute_decode16", "permute", 16, 10, 512, 2048, weighted=False, skipped=5),
        # a prefill batch with a skewed router
        _rows("permute_prefill8192", "permute", 8192, 10, 512, 2048, weighted=False, skew=1.0),
        # a single request's decode step
        _rows("unpermute_decode1", "unpermute", 1, 10, 512, 2048, weighted=True),
        # the prefill batch's expert results on their way back
        _rows("unpermute_prefill8192", "unpermute", 8192, 10, 512, 2048, weighted=True),
        # a short training micro-batch of odd length, few experts, a wide hidden size
        _rows("combine_grad_333", "combine_grad", 333, 2, 8, 5120, weighted=True, skipped=7),
        # a training batch
        _rows("combine_grad_8192", "combine_grad", 8192, 10, 512, 2048, weighted=True),
        # one request with an adapter on the dense projection
        _dense("linear_adapters_1", "linear", 1, 4352, 5120, 16, 32),
        # 32 requests, each with an adapter of its own but four that use the shared weights alone
        _dense("linear_adapters_32", "linear", 32, 4352, 5120, 16, 32, without=4),
        # the gated MLP's packed rows, 13 requests over three adapters, interleaved rows
        _dense("swiglu_adapters_13", "swiglu", 13, 4352, 5120, 32, 3, layout=1),
        # a full decode batch on the gated MLP
        _dense("swiglu_adapters_64", "swiglu", 64, 4352, 5120, 16, 16),
        # prompts of eight requests in one prefill batch, one of them without an adapter
        _add("add_prompts_4096", 4096, 1, 4352, 5120, 64, 7, bucket=False, without=512),
        # adapters of the experts, on rows that the plan sorted
        _add("add_experts_6000", 750, 8, 1024, 2048, 16, 64, bucket=True, without=40),
    ]


def _between(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = low * (high / low) ** rng.random()
    return min(high // step * step, max(-(-low // step) * step, round(v / step) * step))


def draw(rng):
    op = rng.choice(("permute", "unpermute", "combine_grad", "linear", "swiglu", "add"))
    if op in ("permute", "unpermute", "combine_grad"):
        k = _between(rng, 128, 8192, 8)
        topk = rng.randint(1, 16)
        experts = _between(rng, max(8, topk), 512)
        m = _between(rng, 1, max(1, min(8192, 8192 * 10 * 2048 // (topk * k))))
        skipped = rng.choice((0, 0, m * topk // 7))
        weighted = op == "combine_grad" or rng.random() < 0.5
        return {"op": op, "m": m, "topk": topk, "experts": experts, "k": k, "weighted": weighted, "skipped": skipped,
                "skew": rng.choice((0.0, 0.0, 1.0))}
    n, k, rank = _between(rng, 64, 8192, 32), _between(rng, 128, 8192, 128), _between(rng, 8, 128, 8)
    adapters = _between(rng, 1, 64)
    if op == "add":
        bucket = rng.random() < 0.5
        topk = rng.randint(1, min(8, adapters)) if bucket else 1
        m = _between(rng, 1, 4096 // topk)
        return {"op": op, "m": m, "topk": topk, "n": n, "k": k, "rank": rank, "adapters": adapters, "bucket": bucket,
                "without": rng.choice((0, m * topk // 5))}
    m = _between(rng, 1, 96)
    return {"op": op, "m": m, "n": n, "k": k, "rank": rank, "adapters": adapters, "without": rng.choice((0, m // 4)),
            "layout": rng.randint(0, 1) if op == "swiglu" else 0}


# ---- inputs ----------------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(torch.float16)


def _routing(g, m, topk, experts, skipped, skew=0.0):
    """Distinct experts per token, drawn by popularity (rank ** -skew), with `skipped` pairs set to -1."""
    rank = torch.randperm(experts, generator=g, device=DEVICE) + 1
    gumbel = -torch.log(-torch.log(torch.rand((m, experts), generator=g, device=DEVICE).clamp_(1e-20, 1 - 1e-7)))
    ids = torch.topk(gumbel - skew * torch.log(rank.float()), topk, dim=1).indices.to(torch.int32)
    pairs = ids.view(-1)
    pairs[torch.randperm(m * topk, generator=g, device=DEVICE)[:skipped]] = -1
    return ids


def _sorted(ids, experts):
    """The stable order of the pairs by expert (skipped ones last) and each pair's place in it."""
    flat = ids.view(-1).long()
    order = torch.argsort(torch.where(flat >= 0, flat, experts), stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEVICE)
    return order, place


def _adapter_ids(g, case):
    """One adapter per row, every adapter used where there are rows enough, `without` rows having none. Rows of
    a large batch are prompts (runs of one adapter), those of a small one single tokens in any order."""
    m, with_one = case["m"], case["m"] - case["without"]
    ids = torch.full((m,), -1, dtype=torch.int32, device=DEVICE)
    if m > 128:
        ids[:with_one] = (torch.arange(with_one, device=DEVICE) * case["adapters"] // max(1, with_one)).to(torch.int32)
    else:
        places = torch.randperm(m, generator=g, device=DEVICE)[:with_one]
        ids[places] = (torch.arange(with_one, device=DEVICE) % case["adapters"]).to(torch.int32)
    return ids.view(m, 1)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": dict(case)}
    if op in ("permute", "unpermute", "combine_grad"):
        experts, pairs = case["experts"], m * case["topk"]
        s["ids"] = _routing(g, m, case["topk"], experts, case["skipped"], case["skew"])
        s["weights"] = torch.softmax(torch.randn((m, case["topk"]), generator=g, device=DEVICE), dim=1)
        if op == "permute":
            s["x"], s["xs"] = _normal(g, m, k), torch.zeros((pairs, k), dtype=torch.float16, device=DEVICE)
        else:
            s["ys"] = _normal(g, pairs, k)
            s["out"] = torch.empty((m, k), dtype=torch.float16, device=DEVICE)
        if op == "combine_grad":
            s["dout"] = _normal(g, m, k)
            s["dys"] = torch.zeros((pairs, k), dtype=torch.float16, device=DEVICE)
            s["dw"] = torch.empty((m, case["topk"]), device=DEVICE)
    else:
        n, rank, experts = case["n"], case["rank"], case["adapters"]
        rows = m * case.get("topk", 1)
        if op == "add":
            s["ids"] = _routing(g, m, case["topk"], experts, case["without"]) if case["bucket"] else _adapter_ids(g, case)
            s["y"], s["out"] = _normal(g, rows, n), torch.zeros((rows, n), dtype=torch.float16, device=DEVICE)
        else:
            s["ids"] = _adapter_ids(g, case)
            s["codes"] = torch.randint(0, 256, (1, n, k // 2), generator=g, device=DEVICE, dtype=torch.uint8)
            pick = torch.randint(0, len(SCALE_BYTES), (1, n, k // 16), generator=g, device=DEVICE)
            s["scales"] = torch.tensor(SCALE_BYTES, dtype=torch.uint8, device=DEVICE)[pick]
            s["gscale"] = torch.full((1,), 0.37, device=DEVICE)
            s["out"] = torch.empty((m, n // 2 if op == "swiglu" else n), dtype=torch.float16, device=DEVICE)
        s["x"] = _normal(g, rows, k)
        s["a"] = _normal(g, experts, rank, k, scale=k ** -0.5)
        s["b"] = _normal(g, experts, n, rank, scale=0.1)
        s["scale"] = torch.rand((experts,), generator=g, device=DEVICE) + 0.5
    s["order"], s["place"] = _sorted(s["ids"], experts)
    if own:
        import gemm_nvfp4_amd as G
        s["plan"] = G.nvfp4_moe_plan(s["ids"], experts)
        if "a" in s:
            s["lora"] = G.LoRATensor(s["a"], s["b"], s["scale"])
            if op == "add":
                need = G.nvfp4_lora_add_ws_bytes(rows, k, rank)
            else:
                s["w"] = G.NVFP4Tensor(s["codes"], s["scales"], s["gscale"])
                need = G.nvfp4_linear_lora_ws_bytes(m, n, k, rank)
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device=DEVICE)
    return s


# ---- one pass --------------------------------------------------------------------------------------

def run(s):
    return _library(s) if own else _plain(s)


def _library(s):
    import gemm_nvfp4_amd as G
    c = s["case"]
    op, m = c["op"], c["m"]
    if op == "permute":
        return G.nvfp4_moe_permute(s["plan"], m, c["topk"], c["experts"], s["x"], s["weights"] if c["weighted"] else None,
                                   xs=s["xs"])
    if op == "unpermute":
        return G.nvfp4_moe_unpermute(s["plan"], m, c["topk"], c["experts"], s["ys"],
                                     s["weights"] if c["weighted"] else None, out=s["out"])
    if op == "combine_grad":
        return G.nvfp4_moe_unpermute_grad(s["plan"], m, c["topk"], c["experts"], s["dout"], s["ys"], s["weights"],
                                          dys=s["dys"], dweights=s["dw"])
    if op == "linear":
        return G.nvfp4_linear_lora(s["plan"], s["x"], s["w"], s["lora"], y=s["out"], ws=s["ws"])
    if op == "swiglu":
        return G.nvfp4_linear_swiglu_lora(s["plan"], s["x"], s["w"], s["lora"], c["layout"], h=s["out"], ws=s["ws"])
    return G.nvfp4_lora_add(s["plan"], m, c["topk"], s["x"], s["lora"], s["y"], order=int(c["bucket"]), out=s["out"],
                            ws=s["ws"])


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("permute", "unpermute", "combine_grad"):
        m, topk, k = c["m"], c["topk"], c["k"]
        order, place = s["order"][:m * topk - c["skipped"]], s["place"].view(m, topk)
        w = s["weights"] if c["weighted"] else None
        if op == "permute":
            xs = torch.zeros_like(s["xs"])
            rows = s["x"][order // topk]
            xs[:order.numel()] = rows if w is None else (rows.float() * w.view(-1)[order, None]).to(torch.float16)
            return xs
        there = (s["ids"] >= 0)[:, :, None]
        rows = torch.where(there, s["ys"][place].float(), 0.0)
        if op == "unpermute":
            return (rows if w is None else rows * w[:, :, None]).sum(dim=1).to(torch.float16)
        dout = s["dout"].float()
        dys = torch.zeros_like(s["dys"])
        dys[:order.numel()] = (dout[order // topk] * w.view(-1)[order, None]).to(torch.float16)
        return dys, (rows * dout[:, None, :]).sum(dim=2)
    x = s["x"].float()
    if op == "add":
        if c["bucket"]:
            valid = c["m"] * c["topk"] - c["without"]
            out = torch.zeros_like(s["y"])
            ids = s["ids"].view(-1)[s["order"]]
            out[:valid] = (s["y"].float() + _low_rank(s, x, ids))[:valid].to(torch.float16)
            return out
        return (s["y"].float() + _low_rank(s, x, s["ids"].view(-1))).to(torch.float16)
    y = x @ _weights(s).t() + _low_rank(s, x, s["ids"].view(-1))
    if op == "linear":
        return y.to(torch.float16)
    half = c["n"] // 2
    gate, up = (y[:, 0::2], y[:, 1::2]) if c["layout"] else (y[:, :half], y[:, half:])
    return (gate / (1.0 + torch.exp(-gate)) * up).to(torch.float16)


def _weights(s):
    """The NVFP4 weight in 32 bits: a code's value times its 16-column block's scale times the global scale."""
    codes = s["codes"][0].long()
    table = torch.tensor(E2M1, device=DEVICE)
    w = torch.stack((table[codes & 15], table[codes >> 4]), dim=-1).view(codes.shape[0], -1, 16)
    return (w * s["scales"][0].view(torch.float8_e4m3fn).float()[:, :, None]).view(codes.shape[0], -1) * s["gscale"]


def _low_rank(s, x, ids):
    """s_a (x A_a^T) B_a^T for every row's adapter a: all adapters' products at once, the others masked."""
    a, b = s["a"].float(), s["b"].float()
    adapters, rank, k = a.shape
    v = (x @ a.view(adapters * rank, k).t()).view(-1, adapters, rank)
    mine = ids[:, None] == torch.arange(adapters, device=DEVICE)[None, :]
    v = torch.where(mine[:, :, None], v * s["scale"][None, :, None], 0.0)
    return v.view(-1, adapters * rank) @ b.permute(0, 2, 1).reshape(adapters * rank, -1)


# ---- what a pass cannot do without, and its result in 64 bits --------------------------------------

def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op in ("permute", "unpermute", "combine_grad"):
        pairs = m * case["topk"]
        rows = pairs - case["skipped"]
        weights = 4 * pairs if case["weighted"] else 0
        moved = {"permute": 2 * k * (m + rows), "unpermute": 2 * k * (m + rows),
                 "combine_grad": 2 * k * (m + 2 * rows) + 4 * pairs}[op]
        flops = {"permute": rows * k * case["weighted"], "unpermute": 2 * rows * k, "combine_grad": 3 * rows * k}[op]
        return {"bytes": moved + weights + 4 * pairs, "flops": flops}
    n, rank = case["n"], case["rank"]
    rows = m * case.get("topk", 1)
    used = rows - case["without"]
    adapters = min(case["adapters"], used) * (2 * rank * (n + k) + 4)
    flops = 2 * used * rank * (n + k)
    if op == "add":
        given = used if case["bucket"] else rows
        return {"bytes": 2 * used * k + 4 * given * n + adapters + 4 * rows, "flops": flops + used * n}
    out = n // 2 if op == "swiglu" else n
    return {"bytes": n * k * 9 // 16 + 4 + 2 * m * k + 2 * m * out + adapters + 4 * rows, "flops": flops + 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op in ("permute", "unpermute", "combine_grad"):
        topk, k = case["topk"], case["k"]
        ids = s["ids"].view(-1).cpu()
        w = s["weights"].double().view(-1) if case["weighted"] else torch.ones(m * topk, dtype=torch.float64, device=DEVICE)
        # pairs by expert, one expert after the other
        lists = [torch.nonzero(ids == e).view(-1) for e in range(case["experts"])]
        pairs = torch.cat(lists).to(DEVICE)
        token, count = torch.div(pairs, topk, rounding_mode="floor"), pairs.numel()
        if op == "permute":
            out = torch.zeros((m * topk, k), dtype=torch.float64, device=DEVICE)
            out[:count] = s["x"].double()[token] * w[pairs, None]
            return out
        ys = s["ys"][:count].double()
        if op == "unpermute":
            out = torch.zeros((m, k), dtype=torch.float64, device=DEVICE)
            return out.index_add_(0, token, ys * w[pairs, None])
        dout = s["dout"].double()
        dys = torch.zeros((m * topk, k), dtype=torch.float64, device=DEVICE)
        dys[:count] = dout[token] * w[pairs, None]
        dw = torch.zeros(m * topk, dtype=torch.float64, device=DEVICE)
        dw[pairs] = (dout[token] * ys).sum(dim=1)
        return dys, dw.view(m, topk)
    x, a, b = s["x"].double(), s["a"].double(), s["b"].double()
    ids = s["ids"].view(-1).long()
    if op == "add":
        y = s["y"].double()
        if case["bucket"]:
            ids = torch.cat([ids[ids == e] for e in range(case["adapters"])])
            x, y = x[:ids.numel()], y[:ids.numel()]
    else:
        y = x @ _exact_weights(s).t()
    for e in range(case["adapters"]):
        mine = torch.nonzero(ids == e).view(-1)
        y[mine] += s["scale"][e].double() * ((x[mine] @ a[e].t()) @ b[e].t())
    if op == "add" and case["bucket"]:
        return torch.cat((y, torch.zeros((m * case["topk"] - y.shape[0], case["n"]), dtype=y.dtype, device=DEVICE)))
    if op != "swiglu":
        return y
    rows = y.view(m, -1, 2).unbind(2) if case["layout"] else y.chunk(2, dim=1)
    return rows[0] * torch.sigmoid(rows[0]) * rows[1]


def _exact_weights(s):
    """The weight in 64 bits from the formats' definition: sign, exponent and mantissa fields."""
    codes, scales = s["codes"][0].long(), s["scales"][0].long()
    nib = torch.stack((codes % 16, codes // 16), dim=2).flatten(1)
    exp, man = (nib // 2) % 4, (nib % 2).double()
    mag = torch.where(exp == 0, man * 0.5, torch.exp2((exp - 1).double()) * (1.0 + man * 0.5))
    value = torch.where(nib >= 8, -mag, mag)
    sexp, sman = (scales // 8) % 16, (scales % 8).double()
    block = torch.where(sexp == 0, sman * 2.0 ** -9, torch.exp2((sexp - 7).double()) * (1.0 + sman / 8.0))
    block = torch.where(scales >= 128, -block, block)
    return value * block.repeat_interleave(16, dim=1) * s["gscale"].double()
