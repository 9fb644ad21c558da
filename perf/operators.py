"""Cases of the slot router and of the packed (8- and 4-bit) bank.

Five operators: ``route`` (scores to slots and weights), ``route_backward`` (the
weights' gradient to the scores), ``pack`` (rows quantised as they are written
to a bank), ``gather`` (weighted sums of a packed bank's rows) and
``weight_grad`` (the gradient of a gather's weights). With ``own`` false, ``run``
computes them from elementary torch operations; with ``own`` true it calls
``sparse_delta_rule_amd``.
"""

import math

import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max
BLOCK = 32  # columns that share a scale in a packed row

# ------------------------------------------------------------------ cases


def _route(name, tokens, keys, k, score, *, dtype="f32", bias=False, groups=1, kept=1, top=1, normalise=False,
           scale=1.0, stream_slots=0, masked=0.0, w="f32", idx="i64"):
    return {"name": name, "op": "route", "tokens": tokens, "keys": keys, "k": k, "score": score, "dtype": dtype,
            "bias": bias, "groups": groups, "kept": kept, "top": top, "normalise": normalise, "scale": scale,
            "stream_slots": stream_slots, "masked": masked, "w": w, "idx": idx}


def _backward(name, tokens, keys, k, score, *, dtype="f32", normalise=False, scale=1.0, stream_slots=0, masked=0.0,
              w="f32", idx="i64"):
    return {"name": name, "op": "route_backward", "tokens": tokens, "keys": keys, "k": k, "score": score,
            "dtype": dtype, "normalise": normalise, "scale": scale, "stream_slots": stream_slots, "masked": masked,
            "w": w, "idx": idx}


def _pack(name, rows, slots, head_dim, *, dtype="bf16", packed="mx8", scattered=False, idx="i64"):
    return {"name": name, "op": "pack", "rows": rows, "slots": slots, "head_dim": head_dim, "dtype": dtype,
            "packed": packed, "scattered": scattered, "idx": idx}


def _gather(name, op, tokens, chunk, valid_low, width0, width1, slots, head_dim, *, packed="mx8", idx="i32", w="bf16"):
    return {"name": name, "op": op, "tokens": tokens, "chunk": chunk, "valid_low": valid_low, "width0": width0,
            "width1": width1, "slots": slots, "head_dim": head_dim, "packed": packed, "idx": idx, "w": w}


def listed():
    return [
        # One new token of one conversation chooses 8 of 256 experts: nothing but latency.
        _route("route one token", 1, 256, 8, "sigmoid", bias=True, groups=8, kept=4, top=2, normalise=True, scale=2.5),
        # The tokens of a training step or of a batch of prompts choose their experts, with a balancing bias.
        _route("route experts", 32768, 256, 8, "sigmoid", bias=True, groups=8, kept=4, top=2, normalise=True, scale=2.5),
        # One decode step of workload c2: every stream chooses 64 slots of its own 16384.
        _route("route slots c2", 4096, 16384, 64, "softmax", dtype="bf16", stream_slots=16384),
        # One decode step of workload c4: 256 of 2048 slots, the widest choice, some slots not yet in use.
        _route("route slots c4", 512, 2048, 256, "softmax", normalise=True, stream_slots=2048, masked=0.05),
        # The training step's way back through the experts' weights: few chosen, a dense gradient.
        _backward("route grad experts", 32768, 256, 8, "sigmoid", normalise=True, scale=2.5),
        # The same through a full softmax over c2's slots.
        _backward("route grad slots c2", 4096, 16384, 64, "softmax", dtype="bf16", stream_slots=16384),
        # The rows that c2's streams wrote in one step go to their slots of the packed copy.
        _pack("pack written rows", 4096 * 64, 1 << 20, 128, scattered=True),
        # A whole float32 bank of workload c4 is packed to 4 bits; rows of 100 columns end inside a block.
        _pack("pack bank c4", 512 * 2048, 512 * 2048, 100, dtype="f32", packed="mx4"),
        # One chunk of one sequence reads the memory while a model answers.
        _gather("gather one chunk", "gather", 64, 64, 64, 64, 64, 1 << 20, 128),
        # Workload c3's tokens over its 16M slots, at a byte a value.
        _gather("gather c3", "gather", 32768, 64, 32, 64, 64, 1 << 24, 128),
        # The router is trained through a frozen memory: gradients of c3's first operand's weights.
        _gather("weight grad c3", "weight_grad", 32768, 64, 32, 64, 0, 1 << 24, 128, w="f32"),
        # A short batch over a small 4-bit memory whose rows do not fill their blocks.
        _gather("weight grad short", "weight_grad", 1000, 50, 17, 48, 20, 100000, 100, packed="mx4", idx="i64"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


_MOST_SCORES = 4096 * 16384  # scores of a route case: the largest listed one's
_MOST_ROWS = 512 * 2048      # rows of a pack case


def draw(rng):
    op = rng.choice(["route", "route_backward", "pack", "gather", "weight_grad"])
    if op in ("route", "route_backward"):
        keys = _log(rng, 8, 65536)
        tokens = _log(rng, 1, min(32768, _MOST_SCORES // keys))
        k = _log(rng, 1, min(256, keys))
        common = dict(dtype=rng.choice(["f32", "bf16"]), normalise=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                      stream_slots=rng.choice([0, keys]), masked=rng.choice([0.0, 0.1, 0.5]),
                      w=rng.choice(["f32", "bf16"]), idx=rng.choice(["i32", "i64"]))
        score = rng.choice(["softmax", "sigmoid"])
        if op == "route_backward":
            if common["normalise"]:
                k = max(k, 2)  # a single renormalised weight is constant: its gradient is 0
            c = _backward("", tokens, keys, k, score, **common)
        else:
            groups = rng.choice([1, 1, 2, 4, 8, 16])
            if keys < 4 * groups:
                groups = 1
            keys -= keys % groups
            common["stream_slots"] = min(common["stream_slots"], keys)
            k = min(k, keys)
            kept = rng.randint(-(-k * groups // keys), groups)
            c = _route("", tokens, keys, k, score, bias=rng.random() < 0.5, groups=groups, kept=kept,
                       top=rng.choice([1, 2]), **common)
    elif op == "pack":
        head_dim = _log(rng, 16, 512)
        rows = _log(rng, 64, min(_MOST_ROWS, _MOST_ROWS * 64 // head_dim))
        c = _pack("", rows, rows + rng.randint(0, rows), head_dim, dtype=rng.choice(["f32", "bf16"]),
                  packed=rng.choice(["mx8", "mx4"]), scattered=rng.random() < 0.5, idx=rng.choice(["i32", "i64"]))
    else:
        chunk = _log(rng, 1, 256)
        head_dim = _log(rng, 16, 512)
        width0 = _log(rng, 1, 256)
        width1 = rng.choice([0, _log(rng, 1, 256)])
        most = 32768 * 128 * 128 if op == "gather" else 32768 * 64 * 128
        chunks = _log(rng, 1, max(1, min(32768, most // (head_dim * (width0 + width1))) // chunk))
        c = _gather("", op, chunks * chunk, chunk, rng.randint(0, chunk), width0, width1, _log(rng, 1000, 1 << 21),
                    head_dim, packed=rng.choice(["mx8", "mx4"]), idx=rng.choice(["i32", "i64"]),
                    w=rng.choice(["f32", "bf16"]))
    c.pop("name")
    return c


_ES = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}


def _code_bytes(c):
    return c["head_dim"] if c["packed"] == "mx8" else (c["head_dim"] + 1) // 2


def _scale_bytes(c):
    return -(-c["head_dim"] // BLOCK)


def work(c):
    if c["op"] in ("route", "route_backward"):
        scores, chosen = c["tokens"] * c["keys"], c["tokens"] * c["k"]
        dense, pair = scores * _ES[c["dtype"]], chosen * (_ES[c["idx"]] + _ES[c["w"]])
        if c["op"] == "route":
            return {"bytes": dense + pair + (4 * c["keys"] if c["bias"] else 0), "flops": 4 * scores}
        whole = c["score"] == "softmax" and not c["normalise"]
        return {"bytes": dense + pair + (dense if whole else chosen * _ES[c["dtype"]]),
                "flops": 8 * chosen + (6 * scores if whole else 0)}
    if c["op"] == "pack":
        slot = _ES[c["idx"]] if c["scattered"] else 0
        return {"bytes": c["rows"] * (c["head_dim"] * _ES[c["dtype"]] + _code_bytes(c) + _scale_bytes(c) + slot),
                "flops": 2 * c["rows"] * c["head_dim"]}
    width, operands = c["width0"] + c["width1"], 1 + (c["width1"] > 0)
    live = c["tokens"] * (c["valid_low"] + c["chunk"]) / (2 * c["chunk"])
    row = _code_bytes(c) + _scale_bytes(c)
    flops = 3 * live * width * c["head_dim"]
    if c["op"] == "gather":
        return {"bytes": live * width * (row + _ES[c["idx"]] + _ES[c["w"]]) + c["tokens"] * operands * c["head_dim"] * 4,
                "flops": flops}
    return {"bytes": live * width * (row + _ES[c["idx"]]) + live * operands * c["head_dim"] * 4
            + c["tokens"] * width * _ES[c["w"]], "flops": flops}


# ------------------------------------------------------------------ inputs


class _State:
    pass


def _packed_bank(c, gen):
    """A bank of rows N(0, 0.02^2), packed: the values' bytes, and a scale byte for each block."""
    n, hd = c["slots"], c["head_dim"]
    codes = torch.zeros((n, _row_bytes(c)), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((n, _scale_row_bytes(c)), dtype=torch.uint8, device=DEV)
    for r in range(0, n, 1 << 20):
        rows = torch.randn((min(1 << 20, n - r), hd), generator=gen, device=DEV) * 0.02
        codes[r:r + len(rows)], scales[r:r + len(rows)] = _pack_rows(c, rows)
    return codes, scales


def _row_bytes(c):
    """Bytes from one row's values to the next row's: rounded up to 16."""
    return -(-_code_bytes(c) // 16) * 16


def _scale_row_bytes(c):
    """Bytes from one row's scales to the next row's: rounded up to 4."""
    return -(-_scale_bytes(c) // 4) * 4


def prepare(c, seed):
    s = _State()
    s.c = c
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if c["op"] in ("route", "route_backward"):
        T, N = c["tokens"], c["keys"]
        x = torch.randn((T, N), generator=gen, device=DEV) * 2
        if c["masked"]:  # keys that may not be chosen: the same ones for a run of 16 tokens
            out = torch.rand((-(-T // 16), N), generator=gen, device=DEV) < c["masked"]
            x.masked_fill_(out.repeat_interleave(16, 0)[:T], -math.inf)
        s.logits = x.to(_TORCH[c["dtype"]])
        if c["op"] == "route":
            s.bias = (torch.rand((N,), generator=gen, device=DEV) - 0.5) * 0.2 if c["bias"] else None
        else:
            s.idx = torch.topk(s.logits, c["k"], dim=-1).indices + _first_slots(c)
            s.idx = s.idx.to(_TORCH[c["idx"]])
            s.dw = torch.randn((T, c["k"]), generator=gen, device=DEV).to(_TORCH[c["w"]])
        return s
    if c["op"] == "pack":
        n, hd = c["rows"], c["head_dim"]
        s.rows = (torch.randn((n, hd), generator=gen, device=DEV) * 0.02).to(_TORCH[c["dtype"]])
        s.slots = None
        if c["scattered"]:
            s.slots = torch.randperm(c["slots"], generator=gen, device=DEV)[:n].to(_TORCH[c["idx"]])
        s.codes = torch.zeros((c["slots"], _row_bytes(c)), dtype=torch.uint8, device=DEV)
        s.scales = torch.zeros((c["slots"], _scale_row_bytes(c)), dtype=torch.uint8, device=DEV)
    else:
        T, chunk = c["tokens"], c["chunk"]
        s.codes, s.scales = _packed_bank(c, gen)
        s.valid = torch.randint(c["valid_low"], chunk + 1, (T // chunk,), generator=gen, device=DEV).to(torch.int32)
        s.idx, s.w, s.dout = [], [], []
        for width in (c["width0"], c["width1"]):
            if width:
                s.idx.append(torch.randint(0, c["slots"], (T, width), generator=gen, device=DEV).to(_TORCH[c["idx"]]))
                s.w.append(torch.randn((T, width), generator=gen, device=DEV).to(_TORCH[c["w"]]))
                s.dout.append(torch.randn((T, c["head_dim"]), generator=gen, device=DEV))
    if own:
        import sparse_delta_rule_amd as sdm
        s.bank = sdm.PackedBank(s.codes, s.scales, c["head_dim"], c["packed"])
    return s


def run(s):
    c = s.c
    if own:
        return _RUN_OWN[c["op"]](c, s)
    return _RUN_PLAIN[c["op"]](c, s)


# ------------------------------------------------------------------ the framework's operators


def _own_route(c, s):
    import sparse_delta_rule_amd as sdm
    return sdm.sdm_route(s.logits, c["k"], score=c["score"], bias=s.bias, groups=c["groups"], kept_groups=c["kept"],
                         group_top=c["top"], normalise=c["normalise"], scale=c["scale"],
                         stream_slots=c["stream_slots"], idx_dtype=_TORCH[c["idx"]], w_dtype=_TORCH[c["w"]])


def _own_route_backward(c, s):
    import sparse_delta_rule_amd as sdm
    return sdm.sdm_route_backward(s.logits, s.idx, s.dw, score=c["score"], normalise=c["normalise"], scale=c["scale"],
                                  stream_slots=c["stream_slots"])


def _own_pack(c, s):
    import sparse_delta_rule_amd as sdm
    sdm.sdm_bank_pack(s.bank, s.rows, slots=s.slots)
    return _as_values(c, s.codes), s.scales


def _own_gather(c, s):
    import sparse_delta_rule_amd as sdm
    second = dict(idx1=s.idx[1], w1=s.w[1]) if c["width1"] else {}
    return sdm.sdm_gather_packed(s.bank, s.idx[0], s.w[0], chunk=c["chunk"], chunk_valid=s.valid, **second)


def _own_weight_grad(c, s):
    import sparse_delta_rule_amd as sdm
    second = dict(idx1=s.idx[1], dout1=s.dout[1]) if c["width1"] else {}
    return sdm.sdm_gather_weight_grad(s.bank, s.idx[0], s.dout[0], chunk=c["chunk"], chunk_valid=s.valid,
                                      w_dtype=_TORCH[c["w"]], **second)


_RUN_OWN = {"route": _own_route, "route_backward": _own_route_backward, "pack": _own_pack, "gather": _own_gather,
            "weight_grad": _own_weight_grad}


# ------------------------------------------------------------------ the plain forms


def _first_slots(c):
    """The first slot of each row's stream: every row of these cases is a stream of its own."""
    return torch.arange(c["tokens"], device=DEV)[:, None] * c["stream_slots"]


def _scores(c, x):
    """Scores of x (64 bits, masked keys -inf)."""
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-FLT_MAX))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-300)


def _clean(logits):
    x = logits.double()
    return torch.where(torch.isnan(x), -math.inf, x).clamp(max=FLT_MAX)


def _chosen_scores(c, x):
    """Scores of the chosen keys, up to a factor of their row where the weights are normalised."""
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    return torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-FLT_MAX))


def _plain_route(c, s):
    T, N, k = c["tokens"], c["keys"], c["k"]
    x = _clean(s.logits)  # 64 bits: which key is chosen may not depend on a rounding
    score = _scores(c, x)
    eligible = x > -math.inf
    value = x
    if s.bias is not None:
        eligible = eligible & (s.bias > -math.inf)
        value = torch.where(eligible, score + s.bias.double(), -math.inf)
    keys = torch.arange(N, device=DEV).expand(T, N)
    if c["groups"] > 1:
        G, size = c["groups"], N // c["groups"]
        by = torch.where(eligible, score if s.bias is None else value, -math.inf).view(T, G, size)
        best = torch.topk(by, min(c["top"], size), dim=-1).values
        none = best[..., 0] == -math.inf
        worth = torch.where(none, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(-1))
        kept = torch.sort(worth, dim=-1, descending=True, stable=True).indices[:, :c["kept"]]
        kept = torch.sort(kept, dim=-1).values
        keys = (kept[..., None] * size + torch.arange(size, device=DEV)).view(T, -1)
        value = torch.gather(value, 1, keys)
    order = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :k]
    key = torch.gather(keys, 1, order)
    chosen = torch.gather(eligible, 1, key)
    if c["normalise"]:
        at = torch.where(chosen, torch.gather(x, 1, key), -math.inf)
        u = torch.where(chosen, _chosen_scores(c, at), 0.0)
        total = u.sum(-1, keepdim=True)
        w = torch.where(total > 0, c["scale"] * u / total, 0.0)
    else:
        w = c["scale"] * torch.where(chosen, torch.gather(score, 1, key), 0.0)
    return (key + _first_slots(c)).to(_TORCH[c["idx"]]), w.to(_TORCH[c["w"]])


def _plain_route_backward(c, s):
    key = s.idx.long() - _first_slots(c)
    x, dw = s.logits.float(), s.dw.float()
    at, d = torch.gather(x, 1, key).double(), s.dw.double()  # 64 bits: both differences below cancel
    if c["score"] == "sigmoid" or c["normalise"]:
        u = _chosen_scores(c, at)
        if c["normalise"]:
            w = u / u.sum(-1, keepdim=True).clamp(min=1e-300)
            d = d - (d * w).sum(-1, keepdim=True)
        else:
            w = u
        if c["score"] == "sigmoid":
            d = d / (1 + torch.exp(at))
        return torch.zeros_like(x).scatter_add_(1, key, (c["scale"] * w * d).float()).to(s.logits.dtype)
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-FLT_MAX))
    p = e / e.sum(-1, keepdim=True).clamp(min=1e-37)
    du = torch.zeros_like(x).scatter_add_(1, key, c["scale"] * dw)
    return (p * (du - (c["scale"] * dw * torch.gather(p, 1, key)).sum(-1, keepdim=True))).to(s.logits.dtype)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _pack_rows(c, rows):
    """Value bytes [n, row bytes] and scale bytes [n, scale row bytes] of float rows."""
    n, hd = rows.shape
    nb = _scale_bytes(c)
    x = torch.zeros((n, nb * BLOCK), device=DEV)
    x[:, :hd] = rows
    x = x.view(n, nb, BLOCK)
    most = x.abs().amax(-1)
    m, e = torch.frexp(most)  # most = m 2^e, m in [0.5, 1)
    mantissa, top = (0.875, 9) if c["packed"] == "mx8" else (0.75, 3)  # the largest value: 448 = 0.875 2^9, 6 = 0.75 2^3
    e = torch.where(most > 0, e - top + (m > mantissa), -127).clamp(-127, 127)
    y = torch.ldexp(x.double(), -e[..., None]).float()
    scales = torch.zeros((n, _scale_row_bytes(c)), dtype=torch.uint8, device=DEV)
    scales[:, :nb] = (e + 127).to(torch.uint8)
    codes = torch.zeros((n, _row_bytes(c)), dtype=torch.uint8, device=DEV)
    y = y.view(n, nb * BLOCK)
    if c["packed"] == "mx8":
        codes[:, :hd] = y.to(torch.float8_e4m3fn).view(torch.uint8)[:, :hd]
    else:
        a = y.abs()
        up = [a > 0.25, a >= 0.75, a > 1.25, a >= 1.75, a > 2.5, a >= 3.5, a > 5.0]  # ties to the even code
        code = sum(u.to(torch.uint8) for u in up) | (torch.signbit(y).to(torch.uint8) << 3)
        code = code.view(n, -1, 2)
        codes[:, :(hd + 1) // 2] = (code[..., 0] | (code[..., 1] << 4))[:, :(hd + 1) // 2]
    return codes, scales


def _as_values(c, codes):
    """8-bit codes as the values they stand for; a byte of 4-bit codes holds two and stays a byte."""
    return codes.view(torch.float8_e4m3fn) if c["packed"] == "mx8" else codes


def _plain_pack(c, s):
    codes, scales = _pack_rows(c, s.rows.float())
    where = torch.arange(c["rows"], device=DEV) if s.slots is None else s.slots.long()
    s.codes[where], s.scales[where] = codes, scales
    return _as_values(c, s.codes), s.scales


def _unpack(c, s, slots):
    """Values of the rows at `slots`: [..., head_dim], which 32 bits hold exactly."""
    hd = c["head_dim"]
    codes = s.codes[slots]
    if c["packed"] == "mx8":
        v = codes.view(torch.float8_e4m3fn)[..., :hd].float()
    else:
        both = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)[..., :hd]
        values = torch.tensor(_E2M1 + [-x for x in _E2M1], device=DEV)
        v = values[both.int()]
    scale = torch.exp2(s.scales[slots][..., :_scale_bytes(c)].double() - 127).float()
    return v * scale.repeat_interleave(BLOCK, dim=-1)[..., :hd]


def _live(c, s):
    t = torch.arange(c["tokens"], device=DEV)
    return t % c["chunk"] < s.valid.long()[t // c["chunk"]]


def _plain_gather(c, s):
    live, out = _live(c, s), []
    for idx, w in zip(s.idx, s.w):
        sums = (_unpack(c, s, idx.long()) * w.float()[..., None]).sum(1)
        out.append(torch.where(live[:, None], sums, 0.0))
    return tuple(out) + (None,) * (2 - len(out))


def _plain_weight_grad(c, s):
    live, out = _live(c, s), []
    for idx, dout in zip(s.idx, s.dout):
        dots = (_unpack(c, s, idx.long()) * dout[:, None]).sum(-1)
        out.append(torch.where(live[:, None], dots, 0.0).to(_TORCH[c["w"]]))
    return tuple(out) + (None,) * (2 - len(out))


_RUN_PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "pack": _plain_pack,
              "gather": _plain_gather, "weight_grad": _plain_weight_grad}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _exact_route(c, s):
    """Chooses one key at a time: the largest value left, the lowest key among equals."""
    T, N = c["tokens"], c["keys"]
    x = s.logits.to(torch.float64)
    x = torch.nan_to_num(x, nan=-math.inf, posinf=FLT_MAX, neginf=-math.inf)
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
    able = ~torch.isneginf(x)
    if s.bias is not None:
        able &= ~torch.isneginf(s.bias)
    c_of = x.clone() if s.bias is None else p + s.bias.double()
    c_of[~able] = -math.inf
    worth_of = c_of if s.bias is not None else torch.where(able, p, -math.inf)
    left = torch.ones((T, N), dtype=torch.bool, device=DEV)
    if c["groups"] > 1:
        worth = worth_of.reshape(T, c["groups"], -1).sort(-1).values[..., -c["top"]:]
        worth = torch.where(torch.isneginf(worth[..., -1]), -math.inf, worth.masked_fill(torch.isneginf(worth), 0).sum(-1))
        keep = torch.zeros_like(worth, dtype=torch.bool)
        ids = torch.arange(c["groups"], device=DEV)
        for _ in range(c["kept"]):
            most = worth.masked_fill(keep, -math.inf).amax(-1, keepdim=True)
            first = torch.where(~keep & (worth == most), ids, c["groups"]).amin(-1, keepdim=True)
            keep.scatter_(1, first, True)
        left &= keep.repeat_interleave(N // c["groups"], dim=1)
    ids, chosen = torch.arange(N, device=DEV), []
    for _ in range(c["k"]):
        most = c_of.masked_fill(~left, -math.inf).amax(-1, keepdim=True)
        first = torch.where(left & (c_of == most), ids, N).amin(-1, keepdim=True)
        left.scatter_(1, first, False)
        chosen.append(first)
    key = torch.cat(chosen, 1)
    u = (p * able).gather(1, key)
    if c["normalise"]:
        u = torch.nan_to_num(u / u.sum(-1, keepdim=True), nan=0.0)
    return None, c["scale"] * u


def _exact_route_backward(c, s):
    """Through the definition, by the chain rule in 64 bits."""
    key = s.idx.long() - torch.arange(c["tokens"], device=DEV)[:, None] * c["stream_slots"]
    x = s.logits.double().requires_grad_()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, -1)
    u = p.gather(1, key)
    w = u / u.sum(-1, keepdim=True) if c["normalise"] else u
    (c["scale"] * w * s.dw.double()).sum().backward()
    return torch.nan_to_num(x.grad, nan=0.0)  # a row of masked keys has weights 0


def _e4m3_values():
    """The value of each 8-bit code: sign, 4 bits of exponent (bias 7), 3 of fraction; 127 and 255 are no numbers."""
    v = [(b % 8 / 8 + (b // 8 > 0)) * 2.0 ** (max(b // 8, 1) - 7) for b in range(128)]
    return v[:127] + [math.nan]


def _exact_pack(c, s):
    """The nearest 8-bit value of each element over its block's power of two. (Bytes of two 4-bit codes have none.)"""
    if c["packed"] != "mx8":
        return None
    hd, table = c["head_dim"], torch.tensor(_e4m3_values()[:127], dtype=torch.float64, device=DEV)
    where = torch.arange(c["rows"], device=DEV) if s.slots is None else s.slots.long()
    out = torch.zeros(s.codes.shape, dtype=torch.float64, device=DEV)
    for b in range(0, hd, BLOCK):
        x = s.rows[:, b:b + BLOCK].double()
        e = torch.ceil(torch.log2(x.abs().amax(1, keepdim=True) / 448)).clamp(-127, 127)
        a = x.abs() / torch.exp2(e)
        low = (torch.searchsorted(table, a.contiguous(), right=True) - 1).clamp(max=125)
        below, above = a - table[low], table[low + 1] - a
        up = (above < below) | ((above == below) & (low % 2 == 1))
        value = table[low + up] * torch.sign(x)
        out[:, b:b + x.shape[1]] = out[:, b:b + x.shape[1]].index_copy(0, where, value)
    return out, None


def _decoded(c, s, slots):
    """Values of the rows at `slots` from the bits of their codes and scales, in 64 bits."""
    hd = c["head_dim"]
    if c["packed"] == "mx8":
        table = _e4m3_values()
        codes = s.codes[slots][..., :hd].int()
    else:  # sign, 2 bits of exponent (bias 1), 1 of fraction; the even column in the low half
        table = [(b % 2 / 2 + (b // 2 > 0)) * 2.0 ** (max(b // 2, 1) - 1) for b in range(8)]
        col = torch.arange(hd, device=DEV)
        codes = (s.codes[slots][..., col // 2] >> (col % 2 * 4)).int() & 15
    v = torch.tensor(table + [-t for t in table], dtype=torch.float64, device=DEV)[codes]
    e = s.scales[slots][..., torch.arange(hd, device=DEV) // BLOCK]
    return torch.ldexp(v, e.int() - 127)


def _in_parts(c, s, what):
    """`what` of each operand's slots, rows and factors, for few tokens at a time, in 64 bits; padding tokens give 0."""
    step, out = max(1, (1 << 27) // ((c["width0"] + c["width1"]) * c["head_dim"])), []
    t = torch.arange(c["tokens"], device=DEV)
    live = (t % c["chunk"] < s.valid.long()[t // c["chunk"]])[:, None]
    for o in range(len(s.idx)):
        parts = []
        for a in range(0, c["tokens"], step):
            rows = _decoded(c, s, s.idx[o][a:a + step].long())
            parts.append(what(o, rows, slice(a, a + step)) * live[a:a + step])
        out.append(torch.cat(parts))
    return tuple(out) + (None,) * (2 - len(out))


def _exact_gather(c, s):
    return _in_parts(c, s, lambda o, rows, at: (rows * s.w[o][at].double()[..., None]).sum(1))


def _exact_weight_grad(c, s):
    return _in_parts(c, s, lambda o, rows, at: (rows * s.dout[o][at].double()[:, None]).sum(2))


def exact(c, seed):
    s = prepare(c, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "pack": _exact_pack,
            "gather": _exact_gather, "weight_grad": _exact_weight_grad}[c["op"]](c, s)
