"""Measured cases of the operators of one decode step of a tensor-parallel layer.

Between two all-reduces a generated token goes through attention over what came before
it, kept in a paged cache, or through the experts of its layer.  Four operators:

  write   new keys and values into the pages of their sequences, as they are or in
          8 bits (E4M3) with a scale for each token and head
  read    back out of the pages, in the inputs' type
  attend  attention of one new token a sequence over its pages
  moe     a whole mixture-of-experts layer for a few tokens: gated first product,
          second product, sum over the choices; E4M3 weights with block scales

`run` computes a case in plain torch (binary32), or, where `own` is true, through this
repository's entry points.  `exact` is the same from the definitions in binary64.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
BLOCK = 128                      # weights that share a scale, down and along
TOP = 448.0                      # the largest E4M3 value
LEAST = 2.0 ** -96               # a row's largest magnitude counts as at least this
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32,
         "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


def _blocks(n):
    return -(-n // BLOCK)


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # a decode step of 16 sequences, 8 heads of keys and values on this rank: latency
        _write("write, decode", 0, 16, 4096, 8, 128, 64, "bf16", "e4m3"),
        # a prefill of 8192 tokens in 5 requests, some behind a cached prefix
        _write("write, prefill", 8192, 5, 2000, 8, 128, 64, "bf16", "e4m3"),
        # a short prefix back for another prefill; small pages, an unusual head
        _read("read, short prefix", 1000, 3, 0, 6, 80, 16, "fp16", "e4m3"),
        # one long document back in bf16
        _read("read, long", 65536, 1, 0, 8, 128, 64, "bf16", "e4m3"),
        # one short conversation on one of eight ranks: latency
        _attend("attend, short", 1, 500, 8, 1, 128, 64, "bf16", "bf16"),
        # one long document, all heads on one device
        _attend("attend, one long", 1, 131072, 64, 8, 128, 64, "bf16", "bf16"),
        # a batch of very different lengths over the 8-bit cache, some places idle
        _attend("attend, batch in 8 bits", 64, 16384, 64, 8, 128, 64, "bf16", "e4m3", idle=3),
        # no shared heads, an unusual head, small pages, a sliding window
        _attend("attend, window", 13, 5000, 24, 24, 80, 16, "fp16", "fp16", window=1000),
        # one head of keys and values for all
        _attend("attend, one shared head", 32, 8192, 32, 1, 256, 32, "bf16", "bf16"),
        # one token, top 8 of 64 experts: the experts' weights are read once
        _moe("moe, one token", 1, 8, 64, 8192, 2048, "bf16"),
        # four tokens, small experts of odd sizes, half of them on another rank
        _moe("moe, small", 4, 2, 8, 1000, 520, "fp16", parts=2),
        # sixteen tokens: most of the experts have one or two of them
        _moe("moe, sixteen tokens", 16, 8, 64, 8192, 1024, "bf16"),
    ]


def _cache(name, op, T, B, longest, heads, D, page, dtype, cache):
    # T new rows in all (0: one a sequence, a decode step)
    return {"name": name, "op": op, "T": T, "B": B, "longest": longest, "heads": heads, "D": D,
            "page": page, "dtype": dtype, "cache": cache}


def _write(name, T, B, longest, heads, D, page, dtype, cache):
    return _cache(name, "write", T, B, longest, heads, D, page, dtype, cache)


def _read(name, T, B, longest, heads, D, page, dtype, cache):
    return _cache(name, "read", T, B, longest, heads, D, page, dtype, cache)


def _attend(name, B, longest, heads, kv_heads, D, page, dtype, cache, window=0, idle=0):
    # the last `idle` places of the batch hold no sequence
    return _cache(name, "attend", 0, B, longest, kv_heads, D, page, dtype, cache) | {
        "q_heads": heads, "window": window, "idle": idle}


def _moe(name, T, K, E, H, F, dtype, parts=1):
    # E experts here, of parts times E in all
    return {"name": name, "op": "moe", "T": T, "K": K, "E": E, "H": H, "F": F, "dtype": dtype,
            "parts": parts}


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
    return max(low, 5 * power if five else power)


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "moe"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "moe":
        T, E = _spread(rng, 1, 64), _spread(rng, 2, 128)
        K = rng.randrange(1, min(E, 8) + 1)
        H, F = _width(rng, 64, 8192), _width(rng, 32, 4096)
        E = max(K, min(E, (1 << 30) // (H * F)))
        most = max(1, int(1.2e9 / (3 * H * F)))               # experts' weights a pass may read
        T = max(1, min(T, most // K if E > most else T))
        return _unnamed(_moe("", T, K, E, H, F, dtype, parts=rng.choice([1, 1, 2, 4])))
    cache = rng.choice([dtype, "e4m3"])
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256, rng.randrange(1, 257)])
    page = rng.choice([16, 32, 64, 64, 128, rng.randrange(1, 100)])
    heads = rng.choice([1, 2, 4, 8, rng.randrange(1, 25)])
    if op == "attend":
        group = rng.choice([1, 4, 8, 8, 16, rng.randrange(1, 33)])
        B, longest = _spread(rng, 1, 256), _spread(rng, 1, 131072)
        # elements of keys, as for the longest listed case
        longest = max(1, min(longest, (1 << 26) // (B * heads * D)))
        return _unnamed(_attend("", B, longest, heads * group, heads, D, page, dtype, cache,
                                window=rng.choice([0, 0, 0, _spread(rng, 1, 8192)]),
                                idle=rng.choice([0, 0, B // 5])))
    B = _spread(rng, 1, 64)
    T = rng.choice([0, _spread(rng, B, 32768)])
    T = min(T, (1 << 24) // (heads * D))
    T = T if T >= B else 0
    longest = _spread(rng, 1, 4096)
    longest = max(1, min(longest, (1 << 24) // (B * heads * D)))
    return _unnamed(_cache("", op, T, B, longest, heads, D, page, dtype, cache))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def _lengths(case):
    """Tokens of each sequence that were there before, or, for a decode step, with its
    new token: between a 64th of the longest and the longest, most of them short."""
    r = random.Random(case["longest"] * 1009 + case["B"])
    top = case["longest"]
    n = [top] + [max(1, int(top * 64 ** -r.random())) for _ in range(case["B"] - 1)]
    for i in range(case.get("idle", 0)):
        n[-1 - i] = 0
    return [min(top, x) for x in n]


def _shares(case):
    """New rows of each sequence; they add up to T."""
    T, B = case["T"], case["B"]
    r = random.Random(T * 1013 + B)
    cuts = sorted(r.randrange(T - B + 1) for _ in range(B - 1))
    return [hi - lo + 1 for lo, hi in zip([0] + cuts, cuts + [T - B])]


def _layout(case):
    """(lens, new rows) of the sequences."""
    before = _lengths(case)
    if case["T"] == 0:
        return before, [1] * case["B"]
    new = _shares(case)
    if case["longest"] == 0:
        return new, new
    return [b + n for b, n in zip(before, new)], new


# ---- what a pass has to read, write and compute -----------------------------------

def work(case):
    s = SIZE[case["dtype"]]
    if case["op"] == "moe":
        T, K, E, H, F = (case[k] for k in ("T", "K", "E", "H", "F"))
        # experts that a token of uniform choices goes to, and its pairs that are here
        active = E * (1 - (1 - K / (E * case["parts"])) ** T)
        pairs = T * K / case["parts"]
        scales = 4 * _blocks(H) * (_blocks(2 * F) + _blocks(F))
        return {"bytes": active * (3 * F * H + scales) + 2 * T * H * s + 8 * T * K,
                "flops": 6 * F * H * pairs}
    lens, new = _layout(case)
    heads, D = case["heads"], case["D"]
    held = D * SIZE[case["cache"]] + (4 if case["cache"] == "e4m3" else 0)
    if case["op"] == "attend":
        n = sum(min(x, case["window"]) if case["window"] else x for x in lens)
        q = case["B"] * case["q_heads"]
        return {"bytes": 2 * n * heads * held + 2 * q * D * s + 4 * q + 4 * case["B"],
                "flops": 4 * n * case["q_heads"] * D}
    rows = sum(new) * heads
    return {"bytes": 2 * rows * (D * s + held) + 4 * case["B"], "flops": 2 * rows * D}


# ---- inputs ----------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    return _prepare_moe(case, g) if case["op"] == "moe" else _prepare_cache(case, g)


def _normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEVICE).normal_(0, std, generator=g)


def _codes(g, *shape):
    """E4M3 values that were scaled to the format's range."""
    return _normal(g, *shape, std=110).clamp_(-TOP, TOP).to(TYPES["e4m3"])


def _prepare_cache(case, g):
    B, heads, D, page = (case[k] for k in ("B", "heads", "D", "page"))
    dt, eight = TYPES[case["dtype"]], case["cache"] == "e4m3"
    lens, new = _layout(case)
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    pages = sum(need) + 3                                    # the pool has some free
    order = torch.randperm(pages, generator=g, device=DEVICE).int()
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    place = torch.full((B, width), -1, dtype=torch.long)
    for b, n in enumerate(need):
        place[b, :n] = torch.arange(at, at + n)
        at += n
    place = place.to(DEVICE)
    table = torch.where(place >= 0, order[place.clamp(min=0)], -1).int()

    def pool():
        return _codes(g, pages, heads, page, D) if eight else _normal(g, pages, heads, page,
                                                                      D).to(dt)

    def scales():
        return (0.005 + 0.01 * torch.rand(pages, heads, page, generator=g, device=DEVICE)
                if eight else None)
    state = {"case": case, "lens": torch.tensor(lens, dtype=torch.int32, device=DEVICE),
             "host_lens": lens, "table": table, "pages": pages, "width": width,
             "kcache": pool(), "vcache": pool(), "kscale": scales(), "vscale": scales()}
    if case["op"] == "attend":
        q = case["q_heads"]
        state |= {"q": (2 * _normal(g, B, q, D)).to(dt),
                  "out": torch.zeros(B, q, D, dtype=dt, device=DEVICE),
                  "lse": torch.zeros(B, q, device=DEVICE),
                  # where the parts of a split sequence are joined
                  "work": torch.zeros(_WORK_ROWS * (D + 2), device=DEVICE)}
        return state
    T = sum(new)
    offsets = None
    if case["T"]:
        ends = torch.tensor([0] + new).cumsum(0)
        offsets = ends.int().to(DEVICE)
    # queries (four heads for each of keys), keys and values lie side by side in one row
    # of a layer's first product
    rows = _normal(g, T, 6 * heads * D).to(dt)
    if case["op"] == "read":
        rows.zero_()
    state |= {"T": T, "offsets": offsets, "k": rows[:, 4 * heads * D:5 * heads * D],
              "v": rows[:, 5 * heads * D:]}
    return state


_WORK_ROWS = 16384               # rows of partial results a caller sets aside


def _prepare_moe(case, g):
    T, K, E, H, F = (case[k] for k in ("T", "K", "E", "H", "F"))
    dt = TYPES[case["dtype"]]
    score = torch.rand(T, E * case["parts"], generator=g, device=DEVICE)
    wide = -(-H // 16) * 16, -(-F // 16) * 16                # rows on 16-byte boundaries

    def weights(rows, columns, padded):
        codes = torch.empty(E, rows, padded, dtype=TYPES["e4m3"], device=DEVICE)
        for e in range(E):
            codes[e] = _codes(g, rows, padded)
        return codes[:, :, :columns]

    def scales(rows, columns):
        r = torch.rand(E, _blocks(rows), _blocks(columns), generator=g, device=DEVICE)
        return (0.5 + r) * (columns ** -0.5 / 110)
    return {"case": case, "x": _normal(g, T, H).to(dt),
            "ids": torch.topk(score, K, dim=1).indices.int(),
            "w": torch.softmax(_normal(g, T, K).float(), dim=1),
            "up": weights(2 * F, H, wide[0]), "up_scale": scales(2 * F, H),
            "down": weights(H, F, wide[1]), "down_scale": scales(H, F),
            "out": torch.zeros(T, H, dtype=dt, device=DEVICE),
            "work": torch.zeros(T * K * (F + BLOCK), device=DEVICE)}


# ---- one pass ----------------------------------------------------------------------

def run(state):
    table = _OWN if own else _PLAIN
    return table[state["case"]["op"]](state)


def _own_write(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_cache_write(s["k"], s["v"], s["kcache"], s["vcache"], s["kscale"], s["vscale"],
                      s["pages"], c["page"], s["table"], s["width"], s["lens"], s["offsets"],
                      s["T"], c["B"], c["heads"], c["D"], c["dtype"], c["cache"],
                      ldk=s["k"].stride(0), ldv=s["v"].stride(0))
    return {k: s[k] for k in ("kcache", "vcache", "kscale", "vscale")}


def _own_read(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_cache_read(s["kcache"], s["vcache"], s["kscale"], s["vscale"], s["pages"], c["page"],
                     s["table"], s["width"], s["lens"], s["offsets"], s["k"], s["v"], s["T"],
                     c["B"], c["heads"], c["D"], c["dtype"], c["cache"], ldk=s["k"].stride(0),
                     ldv=s["v"].stride(0))
    return {"k": s["k"], "v": s["v"]}


def _own_attend(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_cache_attention(s["q"], s["kcache"], s["vcache"], s["kscale"], s["vscale"], s["pages"],
                          c["page"], s["table"], s["width"], s["lens"], c["D"] ** -0.5, s["out"],
                          s["lse"], s["work"], 4 * s["work"].numel(), c["B"], c["q_heads"],
                          c["heads"], c["D"], c["dtype"], c["cache"], window=c["window"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_moe(s):
    import all_reduce_reduction_gb300 as ar
    c = s["case"]
    ar.ar_moe_layer(s["x"], s["ids"], s["w"], s["up"], s["up_scale"], s["down"], s["down_scale"],
                    s["out"], s["work"], 4 * s["work"].numel(), c["T"], c["K"], c["E"], c["H"],
                    c["F"], c["dtype"], ldup=s["up"].stride(1), lddown=s["down"].stride(1))
    return s["out"]


_OWN = {"write": _own_write, "read": _own_read, "attend": _own_attend, "moe": _own_moe}


def _places(s):
    """(page, slot) of every row of k and v."""
    c = s["case"]
    row = torch.arange(s["T"], device=DEVICE)
    lens, table = s["lens"].long(), s["table"].long()
    if s["offsets"] is None:
        b, position = row, lens - 1
    else:
        off = s["offsets"].long()
        b = torch.searchsorted(off[1:], row, right=True)
        position = lens[b] - off[b + 1] + row
    return table[b, position // c["page"]], position % c["page"]


def _plain_write(s):
    c = s["case"]
    at, slot = _places(s)
    for x, cache, scale in ((s["k"], s["kcache"], s["kscale"]),
                            (s["v"], s["vcache"], s["vscale"])):
        x = x.view(s["T"], c["heads"], c["D"])
        if scale is None:
            cache[at, :, slot] = x
            continue
        x = x.float()
        top = x.abs().amax(2).clamp(min=LEAST) / TOP
        scale[at, :, slot] = top
        codes = (x / top[:, :, None]).to(TYPES["e4m3"])
        cache.view(torch.uint8)[at, :, slot] = codes.view(torch.uint8)
    return {k: s[k] for k in ("kcache", "vcache", "kscale", "vscale")}


def _plain_read(s):
    c = s["case"]
    at, slot = _places(s)
    for x, cache, scale in ((s["k"], s["kcache"], s["kscale"]),
                            (s["v"], s["vcache"], s["vscale"])):
        if scale is None:
            rows = cache[at, :, slot]
        else:
            codes = cache.view(torch.uint8)[at, :, slot].view(TYPES["e4m3"])
            rows = codes.float() * scale[at, :, slot][:, :, None]
        x.copy_(rows.reshape(s["T"], -1))
    return {"k": s["k"], "v": s["v"]}


def _sequence(cache, scale, pages, lo, hi):
    """Positions [lo, hi) of one sequence: heads, tokens, D in binary32."""
    page = cache.shape[2]
    pages = pages[lo // page:-(-hi // page)].long()
    if scale is None:
        x = cache[pages].float()
    else:
        x = cache.view(torch.uint8)[pages].view(TYPES["e4m3"]).float() * scale[pages][..., None]
    x = x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])
    first = lo - lo // page * page
    return x[:, first:first + hi - lo]


def _plain_attend(s):
    c = s["case"]
    B, q_heads, heads, D = c["B"], c["q_heads"], c["heads"], c["D"]
    out = torch.zeros(B, q_heads, D, dtype=s["q"].dtype, device=DEVICE)
    lse = torch.full((B, q_heads), -math.inf, device=DEVICE)
    for b, n in enumerate(s["host_lens"]):
        if n == 0:
            continue
        lo = max(0, n - c["window"]) if c["window"] else 0
        k = _sequence(s["kcache"], s["kscale"], s["table"][b], lo, n)
        v = _sequence(s["vcache"], s["vscale"], s["table"][b], lo, n)
        q = s["q"][b].float().view(heads, q_heads // heads, D)
        score = (q @ k.transpose(1, 2)) * D ** -0.5
        top = score.amax(2, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(2, keepdim=True)
        out[b] = ((p @ v) / total).reshape(q_heads, D).to(out.dtype)
        lse[b] = (top + torch.log(total)).reshape(q_heads)
    return {"out": out, "lse": lse}


def _scaled(codes, scale):
    """E4M3 weights times the scales of their blocks, binary32."""
    n, k = codes.shape[-2:]
    s = scale.repeat_interleave(BLOCK, -1)[..., :k].repeat_interleave(BLOCK, -2)[..., :n, :]
    return codes.float() * s


def _plain_moe(s):
    c = s["case"]
    T, K, E, F = c["T"], c["K"], c["E"], c["F"]
    out = torch.zeros(T, c["H"], device=DEVICE)
    up, down = s["up"].view(torch.uint8), s["down"].view(torch.uint8)
    for t in range(T):
        x = s["x"][t].float()
        for k in range(K):
            e = s["ids"][t, k:k + 1].long()
            here = e < E
            e = e.clamp(max=E - 1)
            w1 = _scaled(up[e][0].view(TYPES["e4m3"]), s["up_scale"][e][0])
            w2 = _scaled(down[e][0].view(TYPES["e4m3"]), s["down_scale"][e][0])
            both = w1 @ x
            gate, value = both[:F], both[F:]
            y = w2 @ (gate / (1 + torch.exp(-gate)) * value)
            out[t] += torch.where(here, s["w"][t, k] * y, 0)
    return out.to(s["x"].dtype)


_PLAIN = {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "moe": _plain_moe}


# ---- the definitions in binary64 ---------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "moe":
        return _exact_moe(s)
    held = {}
    for name in ("k", "v"):
        held[name] = s[name + "cache"].double()
        if s[name + "scale"] is not None and case["op"] != "write":
            held[name] *= s[name + "scale"].double()[..., None]
    lens, new = _layout(case)
    page, heads, D = case["page"], case["heads"], case["D"]
    tables = s["table"].tolist()

    def where(b, j):
        return tables[b][j // page], j % page
    if case["op"] == "attend":
        q_heads = case["q_heads"]
        out = torch.zeros(case["B"], q_heads, D, dtype=torch.float64, device=DEVICE)
        lse = torch.full((case["B"], q_heads), -math.inf, dtype=torch.float64, device=DEVICE)
        for b, n in enumerate(lens):
            lo = n - case["window"] if 0 < case["window"] < n else 0
            if n == 0:
                continue
            j = torch.arange(lo, n, device=DEVICE)
            at, slot = s["table"][b].long()[j // page], j % page
            k, v = held["k"][at, :, slot], held["v"][at, :, slot]          # n, heads, D
            q = s["q"][b].double().view(heads, -1, D) / math.sqrt(D)
            score = torch.einsum("hgd,nhd->hgn", q, k)
            lse[b] = torch.logsumexp(score, 2).reshape(-1)
            out[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(score, 2), v).reshape(q_heads, D)
        return {"out": out, "lse": lse}
    rows = [where(b, n - m + i) for b, (n, m) in enumerate(zip(lens, new)) for i in range(m)]
    at = torch.tensor([r[0] for r in rows], device=DEVICE)
    slot = torch.tensor([r[1] for r in rows], device=DEVICE)
    if case["op"] == "read":
        return {n: held[n][at, :, slot].reshape(len(rows), -1) for n in ("k", "v")}
    result = {"kscale": None, "vscale": None}
    for name in ("k", "v"):
        x = s[name].double().reshape(len(rows), heads, D)
        if s[name + "scale"] is not None:
            scale = x.abs().amax(2).clamp(min=LEAST) / TOP
            x = x / scale[..., None]
            result[name + "scale"] = s[name + "scale"].double()
            result[name + "scale"][at, :, slot] = scale
        held[name][at, :, slot] = x
        result[name + "cache"] = held[name]
    return result


def _exact_moe(s):
    c = s["case"]
    F, H = c["F"], c["H"]
    if 6 * F * H * c["T"] * c["K"] > 1e12:
        return None
    out = torch.zeros(c["T"], H, dtype=torch.float64, device=DEVICE)
    across, inner = torch.arange(H, device=DEVICE) // BLOCK, torch.arange(F, device=DEVICE) // BLOCK
    both = torch.arange(2 * F, device=DEVICE) // BLOCK
    for e in set(s["ids"].flatten().tolist()):
        if e >= c["E"]:
            continue
        t, k = torch.nonzero(s["ids"] == e, as_tuple=True)
        x = s["x"][t].double()
        w1 = s["up"][e].double() * s["up_scale"][e].double()[both][:, across]
        w2 = s["down"][e].double() * s["down_scale"][e].double()[across][:, inner]
        gate, value = (x @ w1[:F].t()), (x @ w1[F:].t())
        y = (gate * torch.sigmoid(gate) * value) @ w2.t()
        out.index_add_(0, t, s["w"][t, k, None].double() * y)
    return out
