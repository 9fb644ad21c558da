"""Cases of what trains a router and a bank.

Five operators: ``balance`` (how often a route chose each key, and the loss that
keeps the choice even), ``balance_grad`` (its gradient to the scores), ``lookup``
(scaled rows of a table, with dropout), ``lookup_grad`` (its gradient to the
table) and ``bank_grad`` (the gradient of a gather's weighted sums to the bank).
With ``own`` false, ``run`` computes them from elementary torch operations; with
``own`` true it calls ``sparse_delta_rule_amd``.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
FLT_MAX = torch.finfo(torch.float32).max
BLOCK = 32  # columns that share a scale in a packed row

# ------------------------------------------------------------------ cases


def _balance(name, op, tokens, keys, k, score, *, dtype="f32", chunk=0, valid_low=None, per_chunk=False, scale=0.01,
             stream_slots=0, masked=0.0, idx="i64"):
    chunk = chunk or tokens
    return {"name": name, "op": op, "tokens": tokens, "keys": keys, "k": k, "score": score, "dtype": dtype, "chunk": chunk,
            "valid_low": chunk if valid_low is None else valid_low, "per_chunk": per_chunk, "scale": scale,
            "stream_slots": stream_slots, "masked": masked, "idx": idx}


def _lookup(name, n, slots, head_dim, *, bank="bf16", out="bf16", scale=1.0, dropout=0.0, skewed=False, unused=0.0,
            idx="i64"):
    return {"name": name, "op": "lookup", "n": n, "slots": slots, "head_dim": head_dim, "bank": bank, "out": out,
            "scale": scale, "dropout": dropout, "skewed": skewed, "unused": unused, "idx": idx}


def _lookup_grad(name, n, slots, head_dim, *, bank="f32", out="bf16", scale=1.0, dropout=0.0, skewed=True, unused=0.0,
                 idx="i64"):
    return {**_lookup(name, n, slots, head_dim, bank=bank, out=out, scale=scale, dropout=dropout, skewed=skewed,
                      unused=unused, idx=idx), "op": "lookup_grad"}


def _bank_grad(name, tokens, chunk, valid_low, width0, width1, slots, head_dim, *, bank="f32", skewed=False, idx="i32",
               w="bf16"):
    return {"name": name, "op": "bank_grad", "tokens": tokens, "chunk": chunk, "valid_low": valid_low, "width0": width0,
            "width1": width1, "slots": slots, "head_dim": head_dim, "bank": bank, "skewed": skewed, "idx": idx, "w": w}


def listed():
    return [
        # A training step's 8 sequences, padded at their ends, each balanced over 256 experts on its own.
        _balance("balance experts", "balance", 32768, 256, 8, "sigmoid", chunk=4096, valid_low=3000, per_chunk=True),
        # All streams of workload c2 together, over the 16384 slots that each of them chose 64 from.
        _balance("balance slots c2", "balance", 4096, 16384, 64, "softmax", dtype="bf16", stream_slots=16384),
        # One short prompt and few experts: nothing but latency.
        _balance("balance short", "balance", 333, 100, 6, "softmax", dtype="bf16", idx="i32"),
        # The way back of the first two.
        _balance("balance grad experts", "balance_grad", 32768, 256, 8, "sigmoid", chunk=4096, valid_low=3000,
                 per_chunk=True),
        _balance("balance grad slots c2", "balance_grad", 4096, 16384, 64, "softmax", dtype="bf16", stream_slots=16384),
        # The next token of 64 streams becomes 64 rows of the model's input.
        _lookup("lookup one step", 64, 50000, 1024, scale=32.0),
        # The tokens of a training step, with dropout.
        _lookup("lookup training", 32768, 50000, 1024, scale=32.0, dropout=0.1, skewed=True),
        # Rows of a 4-bit table that do not fill their blocks, some of the tokens padding.
        _lookup("lookup packed", 65521, 100000, 100, bank="mx4", out="f32", unused=0.05, idx="i32"),
        # The training step's way back: few tokens are very frequent, most of the table is not named at all.
        _lookup_grad("lookup grad training", 32768, 50000, 1024, scale=32.0, dropout=0.1),
        # A short batch of a small table.
        _lookup_grad("lookup grad short", 500, 1000, 100, out="f32", unused=0.05, idx="i32"),
        # Workload c3's tokens, both operands, through a memory that learns.
        _bank_grad("bank grad c3", 32768, 64, 32, 64, 64, 1 << 21, 128),
        # One chunk of one sequence.
        _bank_grad("bank grad one chunk", 64, 64, 48, 64, 64, 1 << 17, 128, w="f32", idx="i64"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


_MOST_SCORES = 4096 * 16384  # scores of a balance case: the largest listed one's
_MOST_VALUES = 1 << 28       # values of a gradient to a bank
_MOST_TERMS = 32768 * 128 * 128


def draw(rng):
    op = rng.choice(["balance", "balance_grad", "lookup", "lookup_grad", "bank_grad"])
    if op in ("balance", "balance_grad"):
        keys = _log(rng, 8, 65536)
        tokens = _log(rng, 1, min(32768, _MOST_SCORES // keys))
        chunk = _log(rng, max(1, tokens // 64), tokens)
        tokens -= tokens % chunk
        k = _log(rng, 1, min(256, keys // 2))  # with every key chosen by every token the counts are equal: no gradient
        c = _balance("", op, tokens, keys, k, rng.choice(["softmax", "sigmoid"]),
                     dtype=rng.choice(["f32", "bf16"]), chunk=chunk, valid_low=rng.randint(0, chunk),
                     per_chunk=rng.random() < 0.5, scale=rng.choice([0.001, 0.01, 1.0]),
                     stream_slots=rng.choice([0, keys]), masked=rng.choice([0.0, 0.1, 0.5]),
                     idx=rng.choice(["i32", "i64"]))
    elif op in ("lookup", "lookup_grad"):
        head_dim = _log(rng, 16, 8192)
        n = _log(rng, 1, min(131072, 32768 * 1024 // head_dim))
        slots = _log(rng, 1000, min(1 << 20, 50000 * 1024 // head_dim))
        common = dict(scale=rng.choice([1.0, 32.0, 0.7]), dropout=rng.choice([0.0, 0.1, 0.5]),
                      unused=rng.choice([0.0, 0.05, 0.5]), skewed=rng.random() < 0.5, out=rng.choice(["f32", "bf16"]),
                      idx=rng.choice(["i32", "i64"]))
        if op == "lookup":
            c = _lookup("", n, slots, head_dim, bank=rng.choice(["f32", "bf16", "mx8", "mx4"]), **common)
        else:
            c = _lookup_grad("", n, slots, head_dim, bank=rng.choice(["f32", "bf16"]), **common)
    else:
        chunk = _log(rng, 1, 256)
        head_dim = _log(rng, 16, 512)
        width0 = _log(rng, 1, 256)
        width1 = rng.choice([0, _log(rng, 1, 256)])
        chunks = _log(rng, 1, max(1, min(32768, _MOST_TERMS // (head_dim * (width0 + width1))) // chunk))
        c = _bank_grad("", chunks * chunk, chunk, rng.randint(0, chunk), width0, width1,
                       _log(rng, 1000, min(1 << 21, _MOST_VALUES // head_dim)), head_dim,
                       bank=rng.choice(["f32", "bf16"]), skewed=rng.random() < 0.5, idx=rng.choice(["i32", "i64"]),
                       w=rng.choice(["f32", "bf16"]))
    c.pop("name")
    return c


_ES = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
_TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}


def _row_size(c):
    """Bytes of a table's row without its padding."""
    hd = c["head_dim"]
    if c["bank"] in _ES:
        return hd * _ES[c["bank"]]
    return (hd if c["bank"] == "mx8" else (hd + 1) // 2) + -(-hd // BLOCK)


def work(c):
    if c["op"] in ("balance", "balance_grad"):
        live = (c["valid_low"] + c["chunk"]) / (2 * c["chunk"])
        scores, segments = c["tokens"] * c["keys"], (c["tokens"] // c["chunk"] if c["per_chunk"] else 1)
        dense = scores * _ES[c["dtype"]]
        if c["op"] == "balance":
            return {"bytes": live * (dense + c["tokens"] * c["k"] * _ES[c["idx"]]) + segments * (8 * c["keys"] + 4),
                    "flops": 5 * live * scores}
        return {"bytes": live * dense + dense + segments * 4 * c["keys"], "flops": 8 * live * scores}
    hd = c["head_dim"]
    if c["op"] in ("lookup", "lookup_grad"):
        named = c["n"] * (1 - c["unused"])
        dense = hd * _ES[c["out"]]
        if c["op"] == "lookup":
            rows = c["slots"] * -math.expm1(named * math.log1p(-1 / c["slots"]))  # different ones, of even draws
            return {"bytes": rows * _row_size(c) + c["n"] * (dense + _ES[c["idx"]]), "flops": 2 * named * hd}
        return {"bytes": named * dense + c["n"] * _ES[c["idx"]] + c["slots"] * hd * _ES[c["bank"]], "flops": 2 * named * hd}
    width, operands = c["width0"] + c["width1"], 1 + (c["width1"] > 0)
    live = c["tokens"] * (c["valid_low"] + c["chunk"]) / (2 * c["chunk"])
    return {"bytes": live * (width * (_ES[c["idx"]] + _ES[c["w"]]) + operands * hd * 4) + c["slots"] * hd * _ES[c["bank"]],
            "flops": 2 * live * width * hd}


# ------------------------------------------------------------------ inputs


class _State:
    pass


def _slots(c, gen, shape):
    """Slots drawn evenly, or (skewed) so that the r-th most frequent has a chance of about 1 / r."""
    if not c["skewed"]:
        return torch.randint(0, c["slots"], shape, generator=gen, device=DEV)
    rank = torch.exp(torch.rand(shape, generator=gen, device=DEV, dtype=torch.float64) * math.log(c["slots"])).long() - 1
    return torch.randperm(c["slots"], generator=gen, device=DEV)[rank.clamp(0, c["slots"] - 1)]


def _packed_table(c, gen):
    """A packed table's codes and scales: any codes but those of no number, scales about 2^-6."""
    n, hd = c["slots"], c["head_dim"]
    size = hd if c["bank"] == "mx8" else (hd + 1) // 2
    codes = torch.zeros((n, -(-size // 16) * 16), dtype=torch.uint8, device=DEV)
    codes[:, :size] = torch.randint(0, 256, (n, size), generator=gen, device=DEV).to(torch.uint8)
    if c["bank"] == "mx8":
        codes -= ((codes & 127) == 127).to(torch.uint8)
    blocks = -(-hd // BLOCK)
    scales = torch.zeros((n, -(-blocks // 4) * 4), dtype=torch.uint8, device=DEV)
    scales[:, :blocks] = torch.randint(117, 126, (n, blocks), generator=gen, device=DEV).to(torch.uint8)
    return codes, scales


def prepare(c, seed):
    s = _State()
    s.c = c
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    if c["op"] in ("balance", "balance_grad"):
        T, N = c["tokens"], c["keys"]
        x = torch.randn((T, N), generator=gen, device=DEV) * 2
        x += torch.randn((N,), generator=gen, device=DEV)  # some keys are liked by all: what the loss is against
        if c["masked"]:  # keys that may not be chosen: the same ones for a run of 16 tokens
            out = torch.rand((-(-T // 16), N), generator=gen, device=DEV) < c["masked"]
            x.masked_fill_(out.repeat_interleave(16, 0)[:T], -math.inf)
        s.logits = x.to(_TORCH[c["dtype"]])
        key = torch.topk(s.logits, c["k"], dim=-1).indices
        s.idx = (key + torch.arange(T, device=DEV)[:, None] * c["stream_slots"]).to(_TORCH[c["idx"]])
        s.valid = torch.randint(c["valid_low"], c["chunk"] + 1, (T // c["chunk"],), generator=gen, device=DEV).to(torch.int32)
        s.dloss = torch.rand((), generator=gen, device=DEV) + 0.5
        if c["op"] == "balance_grad":  # as the loss gave them
            s.counts = _plain_counts(c, s).to(torch.int32)
            s.coef = _coef(c, s).to(torch.float32)
        return s
    if c["op"] in ("lookup", "lookup_grad"):
        s.idx = _slots(c, gen, (c["n"],))
        if c["unused"]:
            s.idx[torch.rand((c["n"],), generator=gen, device=DEV) < c["unused"]] = -1
        s.idx = s.idx.to(_TORCH[c["idx"]])
        s.rng = torch.randint(0, 1 << 62, (2,), generator=gen, device=DEV) if c["dropout"] else None
        if c["op"] == "lookup_grad":
            s.dout = torch.randn((c["n"], c["head_dim"]), generator=gen, device=DEV).to(_TORCH[c["out"]])
        elif c["bank"] in _ES:
            s.bank = (torch.randn((c["slots"], c["head_dim"]), generator=gen, device=DEV) * 0.02).to(_TORCH[c["bank"]])
        else:
            s.codes, s.scales = _packed_table(c, gen)
            if own:
                import sparse_delta_rule_amd as sdm
                s.bank = sdm.PackedBank(s.codes, s.scales, c["head_dim"], c["bank"])
        return s
    T, chunk = c["tokens"], c["chunk"]
    s.valid = torch.randint(c["valid_low"], chunk + 1, (T // chunk,), generator=gen, device=DEV).to(torch.int32)
    s.idx, s.w, s.dout = [], [], []
    for width in (c["width0"], c["width1"]):
        if width:
            s.idx.append(_slots(c, gen, (T, width)).to(_TORCH[c["idx"]]))
            s.w.append(torch.randn((T, width), generator=gen, device=DEV).to(_TORCH[c["w"]]))
            s.dout.append(torch.randn((T, c["head_dim"]), generator=gen, device=DEV))
    return s


def run(s):
    c = s.c
    if own:
        return _RUN_OWN[c["op"]](c, s)
    return _RUN_PLAIN[c["op"]](c, s)


# ------------------------------------------------------------------ the framework's operators


def _own_balance(c, s):
    import sparse_delta_rule_amd as sdm
    return sdm.sdm_route_balance(s.logits, s.idx, score=c["score"], chunk=c["chunk"], chunk_valid=s.valid,
                                 per_chunk=c["per_chunk"], scale=c["scale"], stream_slots=c["stream_slots"])


def _own_balance_grad(c, s):
    import sparse_delta_rule_amd as sdm
    return sdm.sdm_route_balance_backward(s.logits, s.counts, s.coef, dloss=s.dloss, score=c["score"], chunk=c["chunk"],
                                          chunk_valid=s.valid, per_chunk=c["per_chunk"])


def _own_lookup(c, s):
    import sparse_delta_rule_amd as sdm
    return sdm.sdm_lookup(s.bank, s.idx, scale=c["scale"], dropout=c["dropout"], rng=s.rng, out_dtype=_TORCH[c["out"]])


def _own_lookup_grad(c, s):
    import sparse_delta_rule_amd as sdm
    return sdm.sdm_lookup_grad(s.idx, s.dout, c["slots"], scale=c["scale"], dropout=c["dropout"], rng=s.rng,
                               bank_dtype=_TORCH[c["bank"]])


def _own_bank_grad(c, s):
    import sparse_delta_rule_amd as sdm
    second = dict(idx1=s.idx[1], w1=s.w[1], dout1=s.dout[1]) if c["width1"] else {}
    return sdm.sdm_gather_bank_grad(s.idx[0], s.w[0], s.dout[0], c["slots"], chunk=c["chunk"], chunk_valid=s.valid,
                                    bank_dtype=_TORCH[c["bank"]], **second)


_RUN_OWN = {"balance": _own_balance, "balance_grad": _own_balance_grad, "lookup": _own_lookup,
            "lookup_grad": _own_lookup_grad, "bank_grad": _own_bank_grad}


# ------------------------------------------------------------------ the plain forms


def _live(c, s):
    t = torch.arange(c["tokens"], device=DEV)
    return t % c["chunk"] < s.valid.long()[t // c["chunk"]]


def _segments(c):
    return c["tokens"] // c["chunk"] if c["per_chunk"] else 1


def _live_counts(c, s):
    """Live tokens of each sequence, 64 bits."""
    n = s.valid.double()
    return n if c["per_chunk"] else n.sum().view(1)


def _coef(c, s):
    """What each sequence's sum of counts times sums of scores is multiplied by."""
    n = _live_counts(c, s)
    return torch.where(n > 0, c["scale"] * c["keys"] / (c["k"] * n.clamp(min=1) ** 2 * (n > 0).sum().clamp(min=1)), 0.0)


def _plain_counts(c, s):
    key = s.idx.long() - torch.arange(c["tokens"], device=DEV)[:, None] * c["stream_slots"]
    live = _live(c, s)[:, None] & (key >= 0) & (key < c["keys"])
    segment = (torch.arange(c["tokens"], device=DEV) // c["chunk"] if c["per_chunk"] else
               torch.zeros(c["tokens"], dtype=torch.int64, device=DEV))
    counts = torch.zeros(_segments(c) * c["keys"], dtype=torch.int64, device=DEV)
    at = (segment[:, None] * c["keys"] + key.clamp(0, c["keys"] - 1)).view(-1)
    return counts.scatter_add_(0, at, live.long().view(-1)).view(-1, c["keys"])


def _plain_scores(c, s):
    """Each row's scores over their sum, and 1 - s of a sigmoid (32 bits)."""
    x = s.logits.float()
    x = torch.where(torch.isnan(x), -math.inf, x).clamp(max=FLT_MAX)
    if c["score"] == "sigmoid":
        u = 1 / (1 + torch.exp(-x))
        return u / u.sum(-1, keepdim=True).clamp(min=1e-37), 1 / (1 + torch.exp(x))
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-FLT_MAX))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-37), None


def _plain_balance(c, s):
    p, _ = _plain_scores(c, s)
    p = torch.where(_live(c, s)[:, None], p, 0.0)
    total = p.view(_segments(c), -1, c["keys"]).sum(1, dtype=torch.float64)  # a long sum
    mean = total / _live_counts(c, s).clamp(min=1)[:, None]
    counts, coef = _plain_counts(c, s), _coef(c, s)
    loss = (coef * (counts * total).sum(-1)).sum()
    return loss.float(), counts.to(torch.int32), mean.float(), coef.float()


def _plain_balance_grad(c, s):
    p, rest = _plain_scores(c, s)
    f = (s.counts.float() * (s.dloss * s.coef)[:, None]).repeat_interleave(c["tokens"] // _segments(c), 0)
    d = p * (f - (f * p).sum(-1, keepdim=True))
    if rest is not None:
        d = d * rest
    return torch.where(_live(c, s)[:, None], d, 0.0).to(s.logits.dtype)


_U32 = 0xffffffff


def _philox(c0, c1, c2, c3, k0, k1):
    """Philox4x32-10 in 64-bit integers, whose low 64 bits of a product are right also where they wrap."""
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & _U32) ^ c1 ^ k0, p1 & _U32, ((p0 >> 32) & _U32) ^ c3 ^ k1, p0 & _U32
        k0, k1 = (k0 + 0x9E3779B9) & _U32, (k1 + 0xBB67AE85) & _U32
    return c0, c1, c2, c3


def _dropped(c):
    """Of 65536 equally likely values of a column, those that drop it."""
    return int(round(c["dropout"] * 65536))


def _factor(c):
    return c["scale"] * 65536 / (65536 - _dropped(c))


def _plain_mask(c, s):
    """[n, head_dim] truth values: the columns that stay."""
    row = torch.arange(c["n"], device=DEV)[:, None]
    octet = torch.arange(-(-c["head_dim"] // 8), device=DEV)[None]
    seed, offset = s.rng[0], s.rng[1]
    zero = torch.zeros_like(row + octet)
    words = _philox(octet + zero, row + zero, (offset & _U32) + zero, (offset >> 32 & _U32) + zero, seed & _U32,
                    seed >> 32 & _U32)
    both = torch.stack([half for w in words for half in (w & 0xffff, w >> 16)], -1)
    return both.view(c["n"], -1)[:, :c["head_dim"]] >= _dropped(c)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _plain_rows(c, s, slots):
    """Rows of the table as 32-bit values."""
    if c["bank"] in _ES:
        return s.bank[slots].float()
    hd, codes = c["head_dim"], s.codes[slots]
    if c["bank"] == "mx8":
        v = codes.view(torch.float8_e4m3fn)[..., :hd].float()
    else:
        both = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)[..., :hd]
        v = torch.tensor(_E2M1 + [-x for x in _E2M1], device=DEV)[both.int()]
    scale = torch.exp2(s.scales[slots][..., :-(-hd // BLOCK)].float() - 127)
    return v * scale.repeat_interleave(BLOCK, dim=-1)[..., :hd]


def _plain_lookup(c, s):
    at = s.idx.long()
    stays = ((at >= 0) & (at < c["slots"]))[:, None]
    if c["dropout"]:
        stays = stays & _plain_mask(c, s)
    return torch.where(stays, _plain_rows(c, s, at.clamp(0, c["slots"] - 1)) * _factor(c), 0.0).to(_TORCH[c["out"]])


def _plain_lookup_grad(c, s):
    at = s.idx.long()
    stays = ((at >= 0) & (at < c["slots"]))[:, None]
    if c["dropout"]:
        stays = stays & _plain_mask(c, s)
    terms = torch.where(stays, s.dout.double(), 0.0)  # 64 bits: a frequent token's sum is long
    total = torch.zeros((c["slots"], c["head_dim"]), dtype=torch.float64, device=DEV)
    total.index_add_(0, at.clamp(0, c["slots"] - 1), terms)
    return (total * _factor(c)).to(_TORCH[c["bank"]])


def _plain_bank_grad(c, s):
    live = _live(c, s)[:, None]
    total = torch.zeros((c["slots"], c["head_dim"]), dtype=torch.float64, device=DEV)  # 64 bits: long sums
    for idx, w, dout in zip(s.idx, s.w, s.dout):
        w = torch.where(live, w.float(), 0.0)
        step = max(1, (1 << 27) // (idx.shape[1] * c["head_dim"]))
        for a in range(0, c["tokens"], step):
            terms = w[a:a + step, :, None].double() * dout[a:a + step, None].double()
            total.index_add_(0, idx[a:a + step].long().view(-1), terms.view(-1, c["head_dim"]))
    return total.to(_TORCH[c["bank"]])


_RUN_PLAIN = {"balance": _plain_balance, "balance_grad": _plain_balance_grad, "lookup": _plain_lookup,
              "lookup_grad": _plain_lookup_grad, "bank_grad": _plain_bank_grad}


# ------------------------------------------------------------------ from the definitions, in 64 bits


def _groups(c, s):
    """For each sequence, its live tokens' numbers."""
    valid, chunk = s.valid.tolist(), c["chunk"]
    runs = [torch.arange(g * chunk, g * chunk + v, device=DEV) for g, v in enumerate(valid)]
    return runs if c["per_chunk"] else [torch.cat(runs)]


def _shares(c, logits):
    """A row's scores as shares of their sum (64 bits)."""
    x = torch.nan_to_num(logits.double(), nan=-math.inf, posinf=FLT_MAX, neginf=-math.inf)
    if c["score"] == "softmax":
        return torch.nan_to_num(torch.softmax(x, -1), nan=0.0)
    score = torch.sigmoid(x)
    return torch.nan_to_num(score / score.sum(-1, keepdim=True), nan=0.0)


def _exact_balance(c, s):
    first = torch.arange(c["tokens"], device=DEV)[:, None] * c["stream_slots"]
    means, sums, sizes = [], [], []
    for tokens in _groups(c, s):
        total = torch.zeros(c["keys"], dtype=torch.float64, device=DEV)
        for part in tokens.split(2048):
            total += _shares(c, s.logits[part]).sum(0)
        count = torch.bincount((s.idx.long() - first)[tokens].flatten(), minlength=c["keys"]).double()
        means.append(total / max(len(tokens), 1))
        sums.append(torch.dot(count, total))
        sizes.append(len(tokens))
    some = max(sum(n > 0 for n in sizes), 1)
    coef = [c["scale"] * c["keys"] / c["k"] / n / n / some if n else 0.0 for n in sizes]
    loss = sum(a * b for a, b in zip(coef, sums))
    return loss, None, torch.stack(means), torch.tensor(coef, dtype=torch.float64, device=DEV)


def _exact_balance_grad(c, s):
    """Through the mean scores, by the chain rule in 64 bits."""
    out = torch.zeros((c["tokens"], c["keys"]), dtype=torch.float64, device=DEV)
    for g, tokens in enumerate(_groups(c, s)):
        for part in tokens.split(2048):
            x = s.logits[part].double().requires_grad_()
            to = s.counts[g].double() * (s.coef[g].double() * s.dloss.double())
            if c["score"] == "softmax":
                share = torch.softmax(x, -1)
            else:
                score = torch.sigmoid(x)
                share = score / score.sum(-1, keepdim=True)
            (share @ to).sum().backward()
            out[part] = torch.nan_to_num(x.grad, nan=0.0)  # a row of masked keys has no part in the mean
    return out


def _exact_mask(c, s):
    """[n, head_dim]: 1 where a column stays, by Philox4x32-10 in unsigned integers on the host."""
    if not c["dropout"]:
        return 1.0
    seed, offset = (int(v) for v in s.rng.tolist())
    octets, low = -(-c["head_dim"] // 8), np.uint64(0xffffffff)
    shape = (c["n"], octets)
    a = np.broadcast_to(np.arange(octets, dtype=np.uint64), shape)
    b = np.broadcast_to(np.arange(c["n"], dtype=np.uint64)[:, None], shape)
    d, e = np.uint64(offset & 0xffffffff), np.uint64(offset >> 32)
    key = [seed & 0xffffffff, seed >> 32]
    for _ in range(10):
        first, third = a * np.uint64(0xD2511F53), d * np.uint64(0xCD9E8D57)
        a, b, d, e = ((third >> np.uint64(32)) ^ b ^ np.uint64(key[0]), third & low,
                      (first >> np.uint64(32)) ^ e ^ np.uint64(key[1]), first & low)
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack([np.broadcast_to(w, shape) for w in (a, b, d, e)], -1).astype("<u4")
    values = words.view("<u2").reshape(c["n"], -1)[:, :c["head_dim"]]
    return torch.from_numpy(values >= round(c["dropout"] * 65536)).to(DEV).double()


def _e4m3_values():
    """The value of each 8-bit code: sign, 4 bits of exponent (bias 7), 3 of fraction."""
    v = [(b % 8 / 8 + (b // 8 > 0)) * 2.0 ** (max(b // 8, 1) - 7) for b in range(128)]
    return v[:127] + [math.nan]


def _exact_lookup(c, s):
    hd, named = c["head_dim"], (s.idx >= 0) & (s.idx < c["slots"])
    at = torch.where(named, s.idx, 0).long()
    if c["bank"] in _ES:
        rows = s.bank.double()[at]
    else:
        col = torch.arange(hd, device=DEV)
        if c["bank"] == "mx8":
            table, codes = _e4m3_values(), s.codes[at][:, :hd].int()
        else:  # sign, 2 bits of exponent (bias 1), 1 of fraction; the even column in the low half
            table = [(b % 2 / 2 + (b // 2 > 0)) * 2.0 ** (max(b // 2, 1) - 1) for b in range(8)]
            codes = (s.codes[at][:, col // 2] >> (col % 2 * 4)).int() & 15
        values = torch.tensor(table + [-t for t in table], dtype=torch.float64, device=DEV)
        rows = torch.ldexp(values[codes], s.scales[at][:, col // BLOCK].int() - 127)
    keep = 1 - round(c["dropout"] * 65536) / 65536
    return rows * _exact_mask(c, s) * named[:, None] * (c["scale"] / keep)


def _by_sorted(slots, entries, total, weight):
    """total[s] += the entries of slot s, by a sort and sums over the runs of equal slots."""
    order = torch.sort(slots, stable=True).indices
    kinds, sizes = torch.unique_consecutive(slots[order], return_counts=True)
    ends = sizes.cumsum(0)
    for a in range(0, len(kinds), 1 << 17):
        lo = int(ends[a] - sizes[a])
        hi = int(ends[min(a + (1 << 17), len(kinds)) - 1])
        number = torch.repeat_interleave(torch.arange(len(sizes[a:a + (1 << 17)]), device=DEV), sizes[a:a + (1 << 17)])
        part = torch.zeros((len(sizes[a:a + (1 << 17)]), total.shape[1]), dtype=torch.float64, device=DEV)
        for b in range(lo, hi, 1 << 19):
            e = order[b:min(b + (1 << 19), hi)]
            part.index_add_(0, number[b - lo:b - lo + len(e)], weight(e)[:, None] * entries(e))
        total[kinds[a:a + (1 << 17)]] += part


def _exact_lookup_grad(c, s):
    total = torch.zeros((c["slots"], c["head_dim"]), dtype=torch.float64, device=DEV)
    rows = s.dout.double() * _exact_mask(c, s)
    there = torch.nonzero((s.idx >= 0) & (s.idx < c["slots"])).flatten()
    factor = torch.full((len(there),), c["scale"] / (1 - round(c["dropout"] * 65536) / 65536), dtype=torch.float64, device=DEV)
    _by_sorted(s.idx[there].long(), lambda e: rows[there[e]], total, lambda e: factor[e])
    return total


def _exact_bank_grad(c, s):
    total = torch.zeros((c["slots"], c["head_dim"]), dtype=torch.float64, device=DEV)
    t = torch.arange(c["tokens"], device=DEV)
    tokens = torch.nonzero(t % c["chunk"] < s.valid.long()[t // c["chunk"]]).flatten()
    for idx, w, dout in zip(s.idx, s.w, s.dout):
        width = idx.shape[1]
        flat = w[tokens].double().flatten()
        _by_sorted(idx[tokens].long().flatten(), lambda e: dout[tokens[e // width]].double(), total, lambda e: flat[e])
    return total


def exact(c, seed):
    s = prepare(c, seed)
    return {"balance": _exact_balance, "balance_grad": _exact_balance_grad, "lookup": _exact_lookup,
            "lookup_grad": _exact_lookup_grad, "bank_grad": _exact_bank_grad}[c["op"]](c, s)
