"""The operators around the grouped GEMM of a mixture-of-experts layer: cases, inputs, plain forms and exact values.

Four operators are measured, each on its own:

* ``gate``    router logits to the k experts of each token and their weights; with ``train`` also the gradient of
              the logits from the gradient of the weights;
* ``unroute`` rows packed by expert back to the tokens' order, weighted and summed over a token's slots; with
              ``train`` also the gradients of the packed rows and of the weights;
* ``swiglu8`` SiLU-and-mul between the two expert products, which keeps its input in 8 bits (e4m3, one power-of-two
              scale for 32 columns), and the backward pass that starts from those 8 bits;
* ``rows8``   packed rows to the same 8-bit form and back: a product's input kept for its weight gradient.

``run`` computes them in plain torch operations, or calls ``moe_grouped_gemm_ragged_b200`` where ``own`` is true.
"""
import torch

own = False

BLOCK = 32          # columns that share a scale
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -118, 120


# ----------------------------------------------------------------------------------------------- the cases

def listed():
    gate = {"op": "gate", "bias": False, "padded": 0, "masked": False}
    unroute = {"op": "unroute", "weights": True, "residual": False, "dropped": 0.0, "train": False}
    return [
        # one decoded token: the gate's latency
        {"name": "gate_decode", **gate, "T": 1, "E": 64, "k": 8, "score": "softmax", "renorm": True, "scale": 1.0,
         "dtype": "bf16", "train": False},
        # a training step's tokens, probabilities over all the experts
        {"name": "gate_train", **gate, "T": 32768, "E": 64, "k": 8, "score": "softmax", "renorm": False, "scale": 1.0,
         "dtype": "bf16", "train": True},
        # sigmoid scores, chosen with a balancing bias, fp32 logits, some experts masked, a padded batch
        {"name": "gate_bias", **gate, "T": 16411, "E": 256, "k": 6, "score": "sigmoid", "renorm": True, "scale": 2.5,
         "dtype": "fp32", "train": True, "bias": True, "padded": 37, "masked": True},
        # one decoded token on its way back, added to the residual stream
        {"name": "unroute_decode", **unroute, "T": 1, "k": 8, "E": 64, "N": 2048, "residual": True},
        # few tokens, a ragged width and dropped slots
        {"name": "unroute_ragged", **unroute, "T": 777, "k": 3, "E": 33, "N": 1160, "dropped": 0.1, "train": True},
        # the gate-up workload's 32768 packed rows in training
        {"name": "unroute_train", **unroute, "T": 4096, "k": 8, "E": 64, "N": 2048, "train": True},
        # the large workload's 262144 packed rows without weights: the gradient of the routing itself
        {"name": "unroute_large", **unroute, "T": 32768, "k": 8, "E": 16, "N": 6144, "weights": False},
        # one token's eight rows
        {"name": "swiglu8_few", "op": "swiglu8", "T": 1, "k": 8, "E": 64, "N": 1536, "concat": True, "weights": False,
         "dropped": 0.0},
        # the gate-up workload: gate and up interleaved, an unused tail
        {"name": "swiglu8_gateup", "op": "swiglu8", "T": 4096, "k": 8, "E": 64, "N": 1536, "concat": False,
         "weights": False, "dropped": 0.01},
        # the down projection's input: [gate | up] halves, the routing weights applied before the down product
        {"name": "swiglu8_down", "op": "swiglu8", "T": 16384, "k": 4, "E": 32, "N": 4096, "concat": True,
         "weights": True, "dropped": 0.0},
        # a small product's input of an odd width
        {"name": "rows8_ragged", "op": "rows8", "R": 1001, "C": 1160, "tail": 29},
        # the large workload's input of its first product
        {"name": "rows8_large", "op": "rows8", "R": 262144, "C": 6144, "tail": 0},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over the logarithm."""
    return min(high, max(low, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["gate", "unroute", "swiglu8", "rows8"])
    if op == "gate":
        E = rng.choice([8, 16, 33, 60, 64, 128, 160, 256, 384])
        score = rng.choice(["softmax", "sigmoid"])
        T = _spread(rng, 1, 32768)
        return {"op": op, "T": T, "E": E, "k": rng.randint(1, 8), "score": score, "renorm": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["bf16", "fp32"]), "train": rng.random() < 0.5,
                "bias": score == "sigmoid" and rng.random() < 0.6, "padded": rng.randint(0, T // 4),
                "masked": rng.random() < 0.3}
    if op == "unroute":
        k = rng.randint(1, 8)
        return {"op": op, "T": _spread(rng, 1, 131072 // k), "k": k, "E": rng.choice([16, 33, 64]),
                "N": 8 * _spread(rng, 16, 768), "weights": rng.random() < 0.7, "residual": rng.random() < 0.5,
                "dropped": rng.choice([0.0, 0.0, 0.05]), "train": rng.random() < 0.5}
    if op == "swiglu8":
        k = rng.randint(1, 8)
        concat = rng.random() < 0.5
        return {"op": op, "T": _spread(rng, 1, 65536 // k), "k": k, "E": rng.choice([32, 33, 64]),
                "N": 16 * _spread(rng, 8, 256) if concat else 256 * rng.randint(1, 16), "concat": concat,
                "weights": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.05])}
    R = _spread(rng, 1, 262144)
    return {"op": op, "R": R, "C": 8 * _spread(rng, 8, 768), "tail": rng.randint(0, R // 8)}


# ---------------------------------------------------------------------------------------------- the inputs

def _randn(shape, gen, std=1.0):
    """N(0, std^2) in bf16, drawn in pieces so that the draws of a large tensor need little room."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for piece in flat.split(1 << 28):
        piece.copy_(torch.randn(piece.shape, generator=gen, device="cuda").mul_(std))
    return out


def _packed(T, k, E, dropped, gen):
    """(row_of [T*k], offs [E]) of tokens that choose k experts each: a stable sort by expert, dropped slots -1."""
    ids = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].reshape(-1)
    ids = torch.where(torch.rand(T * k, generator=gen, device="cuda") < dropped, E, ids)
    order = ids.argsort(stable=True)
    row_of = torch.empty_like(order)
    row_of[order] = torch.arange(T * k, device="cuda")
    row_of = torch.where(ids < E, row_of, -1).to(torch.int32)
    offs = torch.bincount(ids, minlength=E + 1)[:E].cumsum(0).to(torch.int32)
    return row_of, offs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        popular = torch.randn(E, generator=gen, device="cuda")
        x = torch.randn((T, E), generator=gen, device="cuda") + 0.5 * popular
        if case["masked"]:  # some experts out of reach of some tokens, and every 97th token without any
            x = x.masked_fill(torch.rand((T, E), generator=gen, device="cuda") < 0.2, float("-inf"))
            x[96::97] = float("-inf")
        s["logits"] = x.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["bias"] = -0.1 * popular if case["bias"] else None
        s["num_tokens"] = torch.tensor([T - case["padded"]], dtype=torch.int32, device="cuda")
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
        if case["train"]:
            s["dw"] = torch.randn((T, k), generator=gen, device="cuda")
            s["dx"] = torch.empty_like(s["logits"])
    elif case["op"] == "unroute":
        T, k, N = case["T"], case["k"], case["N"]
        s["row_of"], s["offs"] = _packed(T, k, case["E"], case["dropped"], gen)
        s["Y"] = _randn((T * k, N), gen)
        s["w"] = torch.rand((T, k), generator=gen, device="cuda") / k if case["weights"] else None
        s["res"] = _randn((T, N), gen) if case["residual"] else None
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        if case["train"]:
            s["dout"] = _randn((T, N), gen)
            s["dY"] = torch.zeros_like(s["Y"])  # rows behind the last sequence of rows stay as they are
            s["dw"] = torch.empty_like(s["w"]) if case["weights"] else None
    elif case["op"] == "swiglu8":
        T, k, N = case["T"], case["k"], case["N"]
        R, half = T * k, N // 2
        s["row_of"], s["offs"] = _packed(T, k, case["E"], case["dropped"], gen)
        s["H"], s["dact"] = _randn((R, N), gen, 1.5), _randn((R, half), gen)
        s["w"] = torch.rand((T, k), generator=gen, device="cuda") / k if case["weights"] else None
        s["act"], s["again"] = torch.zeros_like(s["dact"]), torch.zeros_like(s["dact"])
        s["dH"] = torch.zeros_like(s["H"])
        s["dw"] = torch.empty_like(s["w"]) if case["weights"] else None
        blocks = 2 * (-(-half // BLOCK))
        s["H8"] = torch.empty((R, N), dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.empty((R, blocks), dtype=torch.float8_e8m0fnu, device="cuda")
    else:
        R, C = case["R"], case["C"]
        s["X"] = _randn((R, C), gen)
        s["offs"] = torch.tensor([R - case["tail"]], dtype=torch.int32, device="cuda")
        s["X8"] = torch.empty((R, C), dtype=torch.float8_e4m3fn, device="cuda")
        s["scale"] = torch.zeros((R, -(-C // BLOCK)), dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        s["back"] = torch.zeros_like(s["X"])
    return s


# --------------------------------------------------------------------------------------------- plain forms

def _used(s):
    """[R, 1] whether a packed row is in use."""
    rows = (s["Y"] if "Y" in s else s["H"] if "H" in s else s["X"]).shape[0]
    return (torch.arange(rows, device="cuda") < s["offs"][-1])[:, None]


def _gate_plain(s):
    c, x = s["case"], s["logits"].float()
    T, k = c["T"], c["k"]
    x = x.masked_fill(torch.arange(T, device="cuda")[:, None] >= s["num_tokens"], float("-inf"))
    if s["bias"] is None:
        order = x  # either score grows with the logit
    else:  # values next to a border decide which expert is chosen
        order = torch.sigmoid(x.double()) + s["bias"].double()
        order = order.masked_fill(x == float("-inf"), float("-inf"))
    top, ids = order.sort(dim=1, descending=True, stable=True)
    ids, live = ids[:, :k], top[:, :k] > float("-inf")
    if c["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True).clamp_min(-3e38))
        p = e / e.sum(1, keepdim=True).clamp_min(1e-38)
    else:
        p = torch.sigmoid(x)
    v = p.gather(1, ids) * live
    total = v.sum(1, keepdim=True).clamp_min(1e-38)
    w = c["scale"] * (v / total if c["renorm"] else v)
    out = [torch.where(live, ids, -1).to(torch.int32), w]
    if c["train"]:
        g = c["scale"] * s["dw"] * live
        if c["renorm"]:
            g = (g - (g * v / total).sum(1, keepdim=True)) / total * live
        dp = torch.zeros_like(p).scatter(1, ids, g)
        if c["score"] == "softmax":
            dx = p * (dp - (dp * p).sum(1, keepdim=True))
        else:
            dx = dp * p * (1 - p)
        out.append(dx.to(s["logits"].dtype))
    return out


def _unroute_plain(s):
    c = s["case"]
    T, k, N = c["T"], c["k"], c["N"]
    row, live = s["row_of"].long().clamp_min(0), (s["row_of"] >= 0)[:, None]
    y = torch.where(live, s["Y"][row].float(), 0.0).view(T, k, N)
    o = (y * s["w"][:, :, None]).sum(1) if c["weights"] else y.sum(1)
    out = [(o + s["res"].float() if c["residual"] else o).to(torch.bfloat16)]
    if c["train"]:
        d = s["dout"].float()[:, None, :]
        g = d * s["w"][:, :, None] if c["weights"] else d.expand(T, k, N)
        dY = torch.zeros((T * k + 1, N), dtype=torch.bfloat16, device="cuda")
        dY[torch.where(s["row_of"] >= 0, s["row_of"].long(), T * k)] = g.reshape(T * k, N).to(torch.bfloat16)
        out.append(dY[:-1])
        if c["weights"]:
            out.append((y * d).sum(2))
    return out


def _halves(H, concat):
    """Gate and up columns of [R, N] rows: halves, or blocks of 128 in turn."""
    if concat:
        return H.chunk(2, dim=1)
    b = H.view(H.shape[0], -1, 2, 128)
    return b[:, :, 0].flatten(1), b[:, :, 1].flatten(1)


def _joined(g, u, concat):
    if concat:
        return torch.cat([g, u], 1)
    return torch.stack([g.view(g.shape[0], -1, 128), u.view(u.shape[0], -1, 128)], 2).flatten(1)


def _eight(x):
    """(values that the 8-bit form of fp32 rows stands for, biased exponents of its scales): e4m3 times the least
    power of two that brings a block of 32 columns into range."""
    R, C = x.shape
    b = torch.nn.functional.pad(x, (0, -C % BLOCK)).view(R, -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(2, keepdim=True))
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(MIN_EXP, MAX_EXP)  # 448 = 0.875 * 2^9
    e = torch.where(m == 0, MIN_EXP, e)
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).view(R, -1)[:, :C], (e + 127).view(R, -1)


def _swiglu8_plain(s):
    c = s["case"]
    used, H = _used(s), torch.where(_used(s), s["H"].float(), 0.0)
    g, u = _halves(H, c["concat"])
    if c["weights"]:
        flat = s["w"].view(-1, 1)
        row = torch.where(s["row_of"] >= 0, s["row_of"].long(), flat.shape[0])
        scale = torch.zeros((flat.shape[0] + 1, 1), device="cuda")
        scale[row] = flat
        scale = scale[:-1]
    else:
        scale = 1.0
    act = (g * torch.sigmoid(g) * u * scale).to(torch.bfloat16)
    g, u = _eight(g)[0], _eight(u)[0]
    d = torch.where(used, s["dact"].float(), 0.0)
    sig = torch.sigmoid(g)
    a = g * sig * u
    dg = d * scale * u * sig * (1 + g * (1 - sig))
    dH = _joined(dg, d * scale * g * sig, c["concat"]).to(torch.bfloat16)
    out = [act, (a * scale).to(torch.bfloat16), dH]
    if c["weights"]:
        dw = (d * a).sum(1)
        out.append(torch.where(s["row_of"] >= 0, dw[s["row_of"].long().clamp_min(0)], 0.0).view(c["T"], c["k"]))
    return out


def _rows8_plain(s):
    used = _used(s)
    back, e = _eight(torch.where(used, s["X"].float(), 0.0))
    return [back.to(torch.bfloat16), torch.where(used, e, 0)]


# --------------------------------------------------------------------------------------- the library's calls

def _gate_own(s):
    import moe_grouped_gemm_ragged_b200 as gg
    c = s["case"]
    how = {"score": gg.GATE_SOFTMAX if c["score"] == "softmax" else gg.GATE_SIGMOID, "renorm": c["renorm"],
           "scale": c["scale"]}
    gg.gate_topk(s["logits"], c["k"], bias=s["bias"], num_tokens=s["num_tokens"], topk_ids=s["ids"], weights=s["w"],
                 **how)
    out = [s["ids"], s["w"]]
    if c["train"]:
        out.append(gg.gate_topk_backward(s["logits"], s["ids"], s["dw"], s["dx"], **how))
    return out


def _unroute_own(s):
    import moe_grouped_gemm_ragged_b200 as gg
    c = s["case"]
    out = [gg.unroute(s["Y"], s["row_of"], c["k"], s["out"], weights=s["w"], residual=s["res"])]
    if c["train"]:
        gg.unroute_backward(s["dout"], s["row_of"], c["k"], s["dY"], Y=s["Y"] if c["weights"] else None,
                            weights=s["w"], dweights=s["dw"])
        out += [s["dY"], s["dw"]] if c["weights"] else [s["dY"]]
    return out


def _swiglu8_own(s):
    import moe_grouped_gemm_ragged_b200 as gg
    c = s["case"]
    how = {"offs": s["offs"], "gate_up_concat": c["concat"], "weights": s["w"],
           "row_of": s["row_of"] if c["weights"] else None}
    gg.silu_mul(s["H"], s["act"], H8=s["H8"], H8_scale=s["scale"], **how)
    gg.silu_mul_backward(s["dact"], s["dH"], H8=s["H8"], H8_scale=s["scale"], act=s["again"], dweights=s["dw"], **how)
    return [s["act"], s["again"], s["dH"]] + ([s["dw"]] if c["weights"] else [])


def _rows8_own(s):
    import moe_grouped_gemm_ragged_b200 as gg
    gg.pack8(s["X"], s["X8"], s["scale"], offs=s["offs"])
    gg.unpack8(s["X8"], s["scale"], s["back"], offs=s["offs"])
    return [s["back"], s["scale"].view(torch.uint8).to(torch.int32)]


def run(state):
    if own:
        return {"gate": _gate_own, "unroute": _unroute_own, "swiglu8": _swiglu8_own,
                "rows8": _rows8_own}[state["case"]["op"]](state)
    return {"gate": _gate_plain, "unroute": _unroute_plain, "swiglu8": _swiglu8_plain,
            "rows8": _rows8_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- what a pass has to do

def work(case):
    """Bytes of each input and output once, and operations, of one pass."""
    if case["op"] == "gate":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        live = (T - case["padded"]) / T
        bytes_, flops = T * E * size * live + T * k * 8, 8.0 * T * E * live
        if case["train"]:
            bytes_, flops = bytes_ + T * E * size + T * k * 4, 2 * flops
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "unroute":
        T, k, N = case["T"], case["k"], case["N"]
        rows = T * k * (1 - case["dropped"]) * N
        bytes_ = 2 * rows + 2 * T * N * (2 if case["residual"] else 1) + T * k * (8 if case["weights"] else 4)
        flops = 2 * rows
        if case["train"]:  # the packed rows are read once for both directions
            bytes_ += 2 * rows + 2 * T * N + T * k * 4 * bool(case["weights"])
            flops += rows * (3 if case["weights"] else 0)
        return {"bytes": bytes_, "flops": flops}
    if case["op"] == "swiglu8":
        rows = case["T"] * case["k"] * (1 - case["dropped"])
        n = rows * case["N"]
        # H once, both activations, the 8-bit form out and in, the two gradients, the weights and theirs
        return {"bytes": n * (2 + 1 + 1 + 2 * 33 / 32 + 1 + 2) + 16 * rows * bool(case["weights"]), "flops": 20 * n}
    n = (case["R"] - case["tail"]) * case["C"]
    return {"bytes": n * (2 + 2 * 33 / 32 + 2), "flops": 4 * n}


# ------------------------------------------------------------------------------------------- exact, 64 bits

def _exact_gate(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    x = s["logits"].to(torch.float64).clone()
    x[int(s["num_tokens"]):] = -torch.inf
    key = x if s["bias"] is None else (1 / (1 + torch.exp(-x))).add(s["bias"].to(torch.float64))
    key = torch.where(torch.isneginf(x), x, key)
    ids = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    xs = torch.gather(x, 1, ids)
    live = ~torch.isneginf(xs)
    log_score = xs if c["score"] == "softmax" else -torch.nn.functional.softplus(-xs)
    whole = torch.logsumexp(x, 1, keepdim=True)
    if c["renorm"]:
        base = torch.logsumexp(log_score, 1, keepdim=True)
    else:
        base = whole if c["score"] == "softmax" else torch.zeros_like(whole)
    v = torch.where(live, torch.exp(log_score - torch.where(torch.isneginf(base), 0, base)), 0)
    out = [torch.where(live, ids, -1).to(torch.int32), c["scale"] * v]
    if not c["train"]:
        return out
    g = c["scale"] * s["dw"].to(torch.float64)
    mean = (g * v).sum(1, keepdim=True)
    dx = torch.zeros_like(x)
    if c["score"] == "softmax":
        if not c["renorm"]:  # every probability falls with the chosen ones' gains
            dx = -mean * torch.where(torch.isneginf(whole), 0, torch.exp(x - torch.where(torch.isneginf(whole), 0, whole)))
            mean = torch.zeros_like(mean)
        inner = torch.ones_like(v)
    else:
        inner = 1 / (1 + torch.exp(xs))
        if not c["renorm"]:
            mean = torch.zeros_like(mean)
    dx.scatter_add_(1, ids, torch.where(live, v * inner * (g - mean), 0))
    return out + [dx]


def _exact_unroute(s):
    c = s["case"]
    T, k, N = c["T"], c["k"], c["N"]
    row = s["row_of"].view(T, k)
    total = s["res"].double() if c["residual"] else torch.zeros((T, N), dtype=torch.float64, device="cuda")
    dY = torch.zeros((T * k, N), dtype=torch.float64, device="cuda") if c["train"] else None
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    for j in range(k):
        t = (row[:, j] >= 0).nonzero()[:, 0]
        r = row[t, j].long()
        w = s["w"][t, j].double()[:, None] if c["weights"] else 1.0
        y = s["Y"][r].double()
        total.index_add_(0, t, y * w)
        if c["train"]:
            d = s["dout"][t].double()
            dY[r] = d * w
            dw[t, j] = (d * y).sum(1)
    return [total] + ([dY] if c["train"] else []) + ([dw] if c["train"] and c["weights"] else [])


def _exact_eight(x):
    """Nearest e4m3 values (ties to an even last bit) under the blocks' scales, by their spacing."""
    R, C = x.shape
    out = torch.zeros_like(x)
    codes = torch.zeros((R, -(-C // BLOCK)), dtype=torch.int64, device=x.device)
    for j in range(codes.shape[1]):
        b = x[:, j * BLOCK:(j + 1) * BLOCK]
        top = b.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, 1) / E4M3_MAX) - 1e-12)
        e = torch.where(top > 0, e, MIN_EXP).clamp(MIN_EXP, MAX_EXP)
        v = b / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        out[:, j * BLOCK:(j + 1) * BLOCK] = torch.round(v / step) * step * torch.exp2(e)
        codes[:, j] = (e[:, 0] + 127).long()
    return out, codes


def _exact_swiglu8(s):
    c = s["case"]
    T, k, N = c["T"], c["k"], c["N"]
    R, half, n = T * k, N // 2, int(s["offs"][-1])
    col = torch.arange(half, device="cuda")
    at_g = col if c["concat"] else col // 128 * 256 + col % 128
    at_u = at_g + (half if c["concat"] else 128)
    w = torch.ones((n, 1), dtype=torch.float64, device="cuda")
    live = (s["row_of"] >= 0).nonzero()[:, 0]
    row = s["row_of"][live].long()
    if c["weights"]:
        w[row, 0] = s["w"].view(-1)[live].double()
    H = s["H"][:n].double()
    g, u = H[:, at_g], H[:, at_u]
    act, again = (torch.zeros((R, half), dtype=torch.float64, device="cuda") for _ in range(2))
    dH = torch.zeros((R, N), dtype=torch.float64, device="cuda")
    act[:n] = w * g / (1 + torch.exp(-g)) * u
    g, u = _exact_eight(g)[0], _exact_eight(u)[0]
    d, q = s["dact"][:n].double(), 1 / (1 + torch.exp(-g))
    again[:n] = w * g * q * u
    dH[:n, at_g] = w * d * u * (q + g * q * (1 - q))
    dH[:n, at_u] = w * d * g * q
    out = [act, again, dH]
    if c["weights"]:
        dw = torch.zeros(R, dtype=torch.float64, device="cuda")
        dw[live] = (d * g * q * u).sum(1)[row]
        out.append(dw.view(T, k))
    return out


def _exact_rows8(s):
    n = int(s["offs"][-1])
    back = torch.zeros(s["X"].shape, dtype=torch.float64, device="cuda")
    codes = torch.zeros(s["scale"].shape, dtype=torch.int32, device="cuda")
    for at in range(0, n, 32768):
        end = min(n, at + 32768)
        value, code = _exact_eight(s["X"][at:end].double())
        back[at:end], codes[at:end] = value, code.to(torch.int32)
    return [back, codes]


def exact(case, seed):
    return {"gate": _exact_gate, "unroute": _exact_unroute, "swiglu8": _exact_swiglu8,
            "rows8": _exact_rows8}[case["op"]](prepare(case, seed))
