"""Measured cases of the operators around the all-reduce of one mixture-of-experts layer.

A tensor-parallel layer sums its partial outputs (the all-reduce), adds the sum to the
residual stream and normalises it, sends every token to its top-K experts, multiplies
each expert's rows with that expert's weights, and brings the results back to the
tokens, each with its gate weight.  Five operators follow that path:

  norm       root-mean-square norm with the residual's addition; the output in the
             inputs' type, or in 8 bits (E4M3) with a scale for each 128 elements
  norm_grad  its gradient: of the sum, and of the weight
  dispatch   the tokens' rows sorted by expert (the order, and the rows themselves)
  back       the experts' rows back at their tokens, weighted; for training with the
             gradients of the rows and of the weights
  matmul8    products of E4M3 rows, a scale for each 128 elements of a row, with E4M3
             weights, a scale for each block of 128 x 128, for one matrix or grouped by
             expert

`run` computes a case in plain torch (binary32), or, where `own` is true, through this
repository's entry points.  `exact` is the same from the definitions in binary64.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = 128                      # elements per scale, along a row and down the weights
TOP = 448.0                      # the largest E4M3 value
LEAST = 2.0 ** -96               # a block's largest magnitude counts as at least this
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def _blocks(n):
    return -(-n // BLOCK)


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one token of a decode step, hidden 8192: latency
        _norm("norm, one token to 8 bits", 1, 8192, "bf16", "e4m3"),
        # a ragged batch of a model with an odd width, rows inside a wider buffer
        _norm("norm, odd width and strides", 333, 4099, "fp16", "fp16", pad=5),
        # a prefill of 8192 tokens, quantised for the expert products
        _norm("norm, prefill to 8 bits", 8192, 8192, "bf16", "e4m3"),
        # a training step on few long rows, binary32
        _norm_grad("norm gradient, small", 130, 4104, "fp32"),
        # a training step at the prefill's size
        _norm_grad("norm gradient, large", 8192, 8192, "bf16"),
        # decode: 16 sequences, top 8 of 64 experts
        _dispatch("dispatch, decode", 16, 8, 64, 8192, "bf16"),
        # prefill on one of two expert-parallel ranks: half of the experts are elsewhere
        _dispatch("dispatch, prefill in 8 bits", 4096, 8, 64, 8192, "e4m3", parts=2),
        # decode: the experts' rows of 16 sequences back at their tokens
        _back("back, decode", 16, 8, 64, 8192, "bf16"),
        # training: forward and gradients at 4096 tokens
        _back("back, training", 4096, 8, 64, 8192, "bf16", train=True),
        # one token's projection: the weights are read once
        _matmul("matmul8, one token", 1, 8192, 8192, 0),
        # 512 tokens to the top 8 of 64 experts: 64 rows an expert on average, uneven
        _matmul("matmul8, experts", 4096, 2048, 8192, 64),
        # a dense prefill projection
        _matmul("matmul8, prefill", 8192, 8192, 8192, 0),
    ]


def _norm(name, T, H, dtype, out, pad=0, residual=True):
    return {"name": name, "op": "norm", "T": T, "H": H, "dtype": dtype, "out": out, "pad": pad,
            "residual": residual}


def _norm_grad(name, T, H, dtype, through=True):
    return {"name": name, "op": "norm_grad", "T": T, "H": H, "dtype": dtype, "through": through}


def _dispatch(name, T, K, E, H, dtype, parts=1):
    return {"name": name, "op": "dispatch", "T": T, "K": K, "E": E, "H": H, "dtype": dtype,
            "parts": parts}


def _back(name, T, K, E, H, dtype, train=False, parts=1):
    return {"name": name, "op": "back", "T": T, "K": K, "E": E, "H": H, "dtype": dtype,
            "train": train, "parts": parts}


def _matmul(name, M, N, K, E, out="bf16"):
    # E = 0: one matrix for all rows
    return {"name": name, "op": "matmul8", "M": M, "N": N, "K": K, "E": E, "out": out}


def _spread(rng, low, high):
    """A whole number between low and high, evenly over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A row width: half of them 4 or 5 times a power of two, the others any number."""
    n = _spread(rng, low, high)
    if rng.random() < 0.5:
        return n
    five = rng.random() < 0.3 and n >= 5
    power = 1 << ((n // 5 if five else n).bit_length() - 1)
    return 5 * power if five else power


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "dispatch", "back", "matmul8"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("norm", "norm_grad"):
        T, H = _spread(rng, 1, 8192), _width(rng, 64, 16384)
        T = min(T, (1 << 25) // H)
        if op == "norm_grad":
            return _unnamed(_norm_grad("", T, H, dtype, through=rng.random() < 0.5))
        return _unnamed(_norm("", T, H, dtype, rng.choice([dtype, "e4m3"]),
                              pad=rng.choice([0, 0, 8, rng.randrange(1, 40)]),
                              residual=rng.random() < 0.75))
    if op in ("dispatch", "back"):
        T, E = _spread(rng, 1, 4096), _spread(rng, 2, 256)
        K = rng.randrange(1, min(E, 8) + 1)
        H = _width(rng, 64, 16384)
        parts = rng.choice([1, 1, 2, 4])
        T = max(1, min(T, (1 << 27) // (K * H)))
        if op == "dispatch":
            return _unnamed(_dispatch("", T, K, E, H, rng.choice([dtype, "e4m3"]), parts))
        return _unnamed(_back("", T, K, E, H, dtype, train=rng.random() < 0.5, parts=parts))
    M, N, K = _spread(rng, 1, 8192), _width(rng, 16, 8192), _width(rng, 32, 8192)
    E = rng.choice([0, 0, _spread(rng, 2, 64)])
    if E and E * N * K > 1 << 29:
        N = max(16, (1 << 29) // (E * K))
    return _unnamed(_matmul("", M, N, K, E, rng.choice(["bf16", "fp16", "fp32"])))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


# ---- what a pass has to read, write and compute -----------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad"):
        n, s = case["T"] * case["H"], SIZE[case["dtype"]]
        if op == "norm_grad":
            return {"bytes": n * s * (4 if case["through"] else 3) + case["H"] * (s + 4),
                    "flops": 9 * n}
        out = n * SIZE[case["out"]]
        if case["out"] == "e4m3":
            out += 4 * case["T"] * _blocks(case["H"])
        return {"bytes": n * s * (3 if case["residual"] else 1) + out + case["H"] * s,
                "flops": 5 * n}
    if op in ("dispatch", "back"):
        # with parts of the experts elsewhere only that share of the rows is here
        T, H, s = case["T"], case["H"], SIZE[case["dtype"]]
        pairs = T * case["K"]
        rows = pairs / case["parts"]
        if op == "dispatch":
            row = H * s + (4 * _blocks(H) if case["dtype"] == "e4m3" else 0)
            return {"bytes": T * row + rows * row + 12 * pairs, "flops": 0}
        forward = rows * H * s + T * H * s + 8 * pairs
        grads = T * H * s + 2 * rows * H * s + 12 * pairs if case["train"] else 0
        return {"bytes": forward + grads, "flops": (5 if case["train"] else 2) * rows * H}
    M, N, K, E = case["M"], case["N"], case["K"], case["E"]
    return {"bytes": M * K + max(E, 1) * N * K + M * N * SIZE[case["out"]]
            + 4 * M * _blocks(K) + 4 * max(E, 1) * _blocks(N) * _blocks(K),
            "flops": 2 * M * N * K}


# ---- inputs ----------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return {"norm": _prepare_norm, "norm_grad": _prepare_norm_grad, "dispatch": _prepare_dispatch,
            "back": _prepare_back, "matmul8": _prepare_matmul}[case["op"]](case, g)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE)


def _hidden(g, T, H):
    """Hidden states: normal values, a few channels much larger than the others."""
    channel = 1 + 20 * (torch.rand(H, generator=g, device=DEVICE) < 0.004)
    return _normal(g, T, H) * channel


def _prepare_norm(case, g):
    T, H, pad, dt = case["T"], case["H"], case["pad"], TYPES[case["dtype"]]

    def rows(values):
        wide = torch.zeros(T, H + pad, dtype=dt, device=DEVICE)
        wide[:, :H] = values
        return wide[:, :H]

    def empty(kind):
        return torch.zeros(T, H + (pad if kind is not TYPES["e4m3"] else 0), dtype=kind,
                           device=DEVICE)[:, :H]
    return {"case": case, "x": rows(_normal(g, T, H)),
            "residual": rows(_hidden(g, T, H)) if case["residual"] else None,
            "gamma": (1 + 0.1 * _normal(g, H)).to(dt),
            "sum": empty(dt) if case["residual"] else None, "y": empty(TYPES[case["out"]]),
            "scale": torch.zeros(T, _blocks(H), device=DEVICE) if case["out"] == "e4m3" else None}


def _prepare_norm_grad(case, g):
    T, H, dt = case["T"], case["H"], TYPES[case["dtype"]]
    s = _hidden(g, T, H).to(dt)
    state = {"case": case, "sum": s, "gamma": (1 + 0.1 * _normal(g, H)).to(dt),
             "rstd": torch.rsqrt(s.float().square().mean(1) + EPS),
             "dy": (1e-3 * _normal(g, T, H)).to(dt),
             "dsum": (1e-3 * _normal(g, T, H)).to(dt) if case["through"] else None,
             "dx": torch.zeros(T, H, dtype=dt, device=DEVICE),
             "dgamma": torch.zeros(H, device=DEVICE),
             # where partial weight gradients are joined
             "work": torch.zeros(_GRAD_WORK_ROWS * H, device=DEVICE)}
    return state


_GRAD_WORK_ROWS = 512            # rows of partial weight gradients a caller sets aside


def _choices(case, g):
    """The router's choices: K different experts a token, some chosen far more often, of
    `parts` times E experts in all; the first E are here."""
    n = case["E"] * case["parts"]
    score = _normal(g, case["T"], n) + 0.7 * _normal(g, n)
    return torch.topk(score, case["K"], dim=1).indices.to(torch.int32)


def _order(ids, E):
    """(offsets, row_of, src) of the stable order of the pairs by expert."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    _, order = torch.sort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(n, device=flat.device)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=flat.device))
    here = key < E
    return (offsets.int(), torch.where(here, place, -1).int().reshape(ids.shape),
            torch.where(key[order] < E, order, -1).int())


def _prepare_dispatch(case, g):
    T, K, E, H = (case[k] for k in ("T", "K", "E", "H"))
    eight, n = case["dtype"] == "e4m3", T * K
    x = _normal(g, T, H)
    if eight:
        x = (x * 110).clamp(-TOP, TOP)
    return {"case": case, "ids": _choices(case, g), "x": x.to(TYPES[case["dtype"]]),
            "xscale": (0.01 * torch.rand(T, _blocks(H), generator=g, device=DEVICE)
                       if eight else None),
            "offsets": torch.zeros(E + 1, dtype=torch.int32, device=DEVICE),
            "row_of": torch.zeros(T, K, dtype=torch.int32, device=DEVICE),
            "src": torch.zeros(n, dtype=torch.int32, device=DEVICE),
            "rows": torch.zeros(n, H, dtype=TYPES[case["dtype"]], device=DEVICE),
            "rscale": torch.zeros(n, _blocks(H), device=DEVICE) if eight else None}


def _prepare_back(case, g):
    T, K, H, dt = case["T"], case["K"], case["H"], TYPES[case["dtype"]]
    ids = _choices(case, g)
    state = {"case": case, "row_of": _order(ids, case["E"])[1],
             "rows": _normal(g, T * K, H).to(dt),
             "w": torch.softmax(_normal(g, T, K), dim=1),
             "out": torch.zeros(T, H, dtype=dt, device=DEVICE)}
    if case["train"]:
        state |= {"dout": (1e-2 * _normal(g, T, H)).to(dt),
                  "drows": torch.zeros(T * K, H, dtype=dt, device=DEVICE),
                  "dw": torch.zeros(T, K, device=DEVICE)}
    return state


def _codes(g, rows, K):
    """E4M3 rows, 16-byte aligned, of values that were scaled to the format's range."""
    wide = torch.empty(rows, -(-K // 16) * 16, dtype=torch.bfloat16, device=DEVICE)
    wide.normal_(0, 110, generator=g)
    return wide.clamp_(-TOP, TOP).to(TYPES["e4m3"])[:, :K]


def _most(case):
    """The most rows one expert gets."""
    return min(case["M"], 4 * -(-case["M"] // case["E"]))


def _prepare_matmul(case, g):
    M, N, K, E = case["M"], case["N"], case["K"], case["E"]
    groups = max(E, 1)
    state = {"case": case, "a": _codes(g, M, K),
             "sa": 0.02 * torch.rand(M, _blocks(K), generator=g, device=DEVICE) + 1e-3,
             "b": _codes(g, groups * N, K).unflatten(0, (groups, N)),
             "sb": 2e-4 * torch.rand(groups, _blocks(N), _blocks(K), generator=g,
                                     device=DEVICE) + 1e-5,
             "d": torch.zeros(M, N, dtype=TYPES[case["out"]], device=DEVICE), "offsets": None}
    if E:
        # every row picks an expert, some far more often than others; what an expert gets
        # beyond its most stays unassigned, at the buffer's end
        pick = torch.multinomial(torch.softmax(_normal(g, E), 0), M, replacement=True, generator=g)
        count = torch.bincount(pick, minlength=E).clamp(max=_most(case))
        state["offsets"] = torch.cat([count.new_zeros(1), count.cumsum(0)]).int()
    return state


# ---- one pass ----------------------------------------------------------------------

def run(state):
    table = _OWN if own else _PLAIN
    return table[state["case"]["op"]](state)


def _own_norm(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_rmsnorm(s["x"], s["residual"], s["gamma"], EPS, s["sum"], s["y"], s["scale"], None,
                  c["T"], c["H"], c["dtype"], c["out"], ldx=s["x"].stride(0),
                  ldres=s["residual"].stride(0) if c["residual"] else 0,
                  ldsum=s["sum"].stride(0) if c["residual"] else 0, ldy=s["y"].stride(0))
    return {"sum": s["sum"], "y": s["y"], "scale": s["scale"]}


def _own_norm_grad(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_rmsnorm_grad(s["dy"], s["dsum"], s["sum"], s["gamma"], s["rstd"], s["dx"], s["dgamma"],
                       s["work"], 4 * s["work"].numel(), c["T"], c["H"], c["dtype"])
    return {"dx": s["dx"], "dgamma": s["dgamma"]}


def _own_dispatch(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    n = c["T"] * c["K"]
    ar.ar_moe_route(s["ids"], c["T"], c["K"], c["E"], s["offsets"], s["row_of"], s["src"])
    ar.ar_moe_dispatch(s["x"], s["xscale"], s["row_of"], s["rows"], s["rscale"], n, c["T"],
                       c["K"], c["H"], c["dtype"])
    return {k: s[k] for k in ("offsets", "row_of", "src", "rows", "rscale")}


def _own_back(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    n = c["T"] * c["K"]
    ar.ar_moe_return(s["rows"], n, s["row_of"], s["w"], s["out"], c["T"], c["K"], c["H"],
                     c["dtype"])
    if not c["train"]:
        return {"out": s["out"]}
    ar.ar_moe_return_grad(s["dout"], s["rows"], n, s["row_of"], s["w"], s["drows"], s["dw"],
                          c["T"], c["K"], c["H"], c["dtype"])
    return {"out": s["out"], "drows": s["drows"], "dw": s["dw"]}


def _own_matmul(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_matmul8(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], max(c["E"], 1), s["d"],
                  c["M"], c["N"], c["K"], c["out"], lda=s["a"].stride(0), ldb=s["b"].stride(1))
    return s["d"]


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "dispatch": _own_dispatch,
        "back": _own_back, "matmul8": _own_matmul}


def _plain_norm(s):
    c = s["case"]
    T, H, dt = c["T"], c["H"], TYPES[c["dtype"]]
    v = s["x"].float()
    if c["residual"]:
        v = v + s["residual"].float()
    y = v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * s["gamma"].float()
    total = v.to(dt) if c["residual"] else None
    if c["out"] != "e4m3":
        return {"sum": total, "y": y.to(dt), "scale": None}
    nb = _blocks(H)
    blocks = torch.zeros(T, nb * BLOCK, device=y.device)
    blocks[:, :H] = y
    blocks = blocks.view(T, nb, BLOCK)
    scale = blocks.abs().amax(2).clamp(min=LEAST) / TOP
    q = (blocks / scale[:, :, None]).to(TYPES["e4m3"]).view(T, nb * BLOCK)[:, :H]
    return {"sum": total, "y": q, "scale": scale}


def _plain_norm_grad(s):
    v, dy, g = s["sum"].float(), s["dy"].float(), s["gamma"].float()
    r = s["rstd"][:, None]
    hat = v * r
    dx = r * (g * dy - hat * (g * dy * hat).mean(1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.to(s["sum"].dtype), "dgamma": (dy * hat).sum(0)}


def _plain_dispatch(s):
    c = s["case"]
    n = c["T"] * c["K"]
    offsets, row_of, src = _order(s["ids"], c["E"])
    to = torch.where(row_of < 0, n, row_of).long()       # one more row takes what is elsewhere

    def spread(x):
        out = x.new_zeros(n + 1, x.shape[1])
        out[to] = x[:, None].expand(-1, c["K"], -1)
        return out[:n]
    if c["dtype"] != "e4m3":
        return {"offsets": offsets, "row_of": row_of, "src": src, "rows": spread(s["x"]),
                "rscale": None}
    return {"offsets": offsets, "row_of": row_of, "src": src,
            "rows": spread(s["x"].view(torch.uint8)).view(TYPES["e4m3"]),
            "rscale": spread(s["xscale"])}


def _plain_back(s):
    c = s["case"]
    n = c["T"] * c["K"]
    here = s["row_of"] >= 0
    at = s["row_of"].clamp(min=0).long()
    picked = s["rows"][at].float() * here[:, :, None]                    # T, K, H
    out = (picked * s["w"][:, :, None]).sum(1).to(s["rows"].dtype)
    if not c["train"]:
        return {"out": out}
    d = s["dout"].float()
    drows = s["rows"].new_zeros(n + 1, c["H"])
    drows[torch.where(here, at, n)] = (d[:, None] * s["w"][:, :, None]).to(drows.dtype)
    return {"out": out, "drows": drows[:n], "dw": (picked * d[:, None]).sum(2)}


def _scaled(codes, scale, down):
    """E4M3 codes times their scales, binary32; `down` rows share a scale."""
    s = scale.repeat_interleave(BLOCK, -1)[..., : codes.shape[-1]]
    if down > 1:
        s = s.repeat_interleave(down, -2)[..., : codes.shape[-2], :]
    return codes.float() * s


def _plain_matmul(s):
    c = s["case"]
    a, b = _scaled(s["a"], s["sa"], 1), _scaled(s["b"], s["sb"], BLOCK)
    out = TYPES[c["out"]]
    if not c["E"]:
        return (a @ b[0].t()).to(out)
    M, E, most = c["M"], c["E"], _most(c)
    r = torch.arange(M, device=a.device)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)       # E: unassigned
    at = e * most + torch.where(e < E, r - s["offsets"].long()[e.clamp(max=E - 1)], 0)
    padded = a.new_zeros(E * most + 1, c["K"])                           # the last: unassigned
    padded[at] = a
    d = torch.bmm(padded[:-1].view(E, most, -1), b.transpose(1, 2)).view(E * most, -1)
    return torch.where((e < E)[:, None], d[at.clamp(max=E * most - 1)], 0).to(out)


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dispatch": _plain_dispatch,
          "back": _plain_back, "matmul8": _plain_matmul}


# ---- the definitions in binary64 ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double()
        if s["residual"] is not None:
            v = v + s["residual"].double()
        y = v / torch.sqrt((v * v).sum(1, keepdim=True) / case["H"] + EPS) * s["gamma"].double()
        total = v if s["residual"] is not None else None
        if s["scale"] is None:
            return {"sum": total, "y": y, "scale": None}
        scale = torch.stack([part.abs().amax(1) for part in y.split(BLOCK, dim=1)], 1)
        scale = scale.clamp(min=LEAST) / TOP
        column = torch.arange(case["H"], device=y.device) // BLOCK
        return {"sum": total, "y": y / scale[:, column], "scale": scale}
    if case["op"] == "norm_grad":
        v, dy, g, r = (s[k].double() for k in ("sum", "dy", "gamma", "rstd"))
        inner = torch.einsum("th,h,th->t", dy, g, v)
        dx = r[:, None] * g * dy - (r ** 3 / case["H"] * inner)[:, None] * v
        if s["dsum"] is not None:
            dx += s["dsum"].double()
        return {"dx": dx, "dgamma": torch.einsum("th,th,t->h", dy, v, r)}
    if case["op"] == "dispatch":
        # by counting: a pair's row is the number of pairs that go before it
        flat = s["ids"].reshape(-1).long()
        onehot = torch.nn.functional.one_hot(flat.clamp(0, case["E"]), case["E"] + 1).int()
        count = onehot.sum(0)
        first = torch.cat([count.new_zeros(1), count.cumsum(0)])
        before = onehot.cumsum(0, dtype=torch.int32).gather(1, flat.clamp(0, case["E"])[:, None])
        row = first[flat.clamp(0, case["E"])] + before[:, 0].long() - 1
        src = torch.empty_like(row)
        src[row] = torch.arange(row.numel(), device=row.device)
        here = int(first[case["E"]])
        src[here:] = -1
        rows = torch.zeros(row.numel(), case["H"], dtype=torch.float64, device=row.device)
        rows[:here] = s["x"].double()[src[:here] // case["K"]]
        rscale = None
        if s["rscale"] is not None:
            rscale = torch.zeros(s["rscale"].shape, dtype=torch.float64, device=row.device)
            rscale[:here] = s["xscale"].double()[src[:here] // case["K"]]
        return {"offsets": first[: case["E"] + 1].int(),
                "row_of": torch.where(flat < case["E"], row, -1).int().view(s["ids"].shape),
                "src": src.int(), "rows": rows, "rscale": rscale}
    if case["op"] == "back":
        T, K, H = case["T"], case["K"], case["H"]
        out = torch.zeros(T, H, dtype=torch.float64, device=DEVICE)
        train = case["train"]
        if train:
            drows = torch.zeros(T * K, H, dtype=torch.float64, device=DEVICE)
            dw = torch.zeros(T, K, dtype=torch.float64, device=DEVICE)
            d = s["dout"].double()
        for k in range(K):
            t = torch.nonzero(s["row_of"][:, k] >= 0)[:, 0]
            row = s["row_of"][t, k].long()
            y, w = s["rows"][row].double(), s["w"][t, k].double()[:, None]
            out[t] += w * y
            if train:
                drows[row] = w * d[t]
                dw[t, k] = (y * d[t]).sum(1)
        return {"out": out, "drows": drows, "dw": dw} if train else {"out": out}
    # matmul8, one 128-wide slice of the inner axis at a time, expert by expert
    M, N, K = case["M"], case["N"], case["K"]
    if 2 * M * N * K > 1.5e13:
        return None
    d = torch.zeros(M, N, dtype=torch.float64, device=DEVICE)
    ends = s["offsets"].tolist() if case["E"] else [0, M]
    columns = torch.arange(N, device=DEVICE) // BLOCK
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        for kb in range(_blocks(K) if hi > lo else 0):
            part = slice(kb * BLOCK, (kb + 1) * BLOCK)
            p = s["a"][lo:hi, part].double() @ s["b"][e, :, part].double().t()
            d[lo:hi] += p * s["sa"][lo:hi, kb, None].double() * s["sb"][e, columns, kb].double()
    return d
