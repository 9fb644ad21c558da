"""What trains a router and a bank, run together as a training step has it: tokens looked
up with dropout, a router over the memory's slots with its balance loss, a gather of the
chosen rows, and the way back to the scores, the memory and the table; on several
streams at once, and captured in a graph."""

import numpy as np
import pytest
import torch

import train_ref as ref
import sparse_delta_rule_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
T, CHUNK, V, SLOTS, HD, K = 96, 24, 50, 64, 40, 6


def inputs(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    tokens = torch.randint(0, V, (T,), generator=g, device=DEV)
    tokens[::17] = -1
    return dict(table=rand(V, HD), bank=rand(SLOTS, HD), proj=rand(HD, SLOTS) * 0.3, tokens=tokens, target=rand(T, HD),
                rng=torch.tensor([seed, seed * 3 + 1], device=DEV),
                cv=torch.randint(0, CHUNK + 1, (T // CHUNK,), generator=g, device=DEV).to(torch.int32),
                dloss=torch.tensor(0.5, device=DEV))


def step(s):
    """Outputs, losses and gradients of sum over live tokens of (read - target)^2 / 2 plus dloss times the balance loss."""
    x = sdm.sdm_lookup(s["table"], s["tokens"], scale=2.0, dropout=0.25, rng=s["rng"])
    logits = x @ s["proj"]
    idx, w = sdm.sdm_route(logits, K, normalise=True)
    loss, counts, mean, coef = sdm.sdm_route_balance(logits, idx, chunk=CHUNK, chunk_valid=s["cv"], per_chunk=True, scale=0.1)
    out, _, _ = sdm.sdm_gather(s["bank"], idx, w, chunk=CHUNK, chunk_valid=s["cv"], with_stash=False)
    live = torch.arange(T, device=DEV) % CHUNK < s["cv"].repeat_interleave(CHUNK)
    dout = torch.where(live[:, None], out - s["target"], 0.0)
    dbank = sdm.sdm_gather_bank_grad(idx, w, dout, SLOTS, chunk=CHUNK, chunk_valid=s["cv"])
    dw, _ = sdm.sdm_gather_weight_grad(s["bank"], idx, dout, chunk=CHUNK, chunk_valid=s["cv"])
    dlogits = sdm.sdm_route_backward(logits, idx, dw, normalise=True)
    sdm.sdm_route_balance_backward(logits, counts, coef, dloss=s["dloss"], chunk=CHUNK, chunk_valid=s["cv"], per_chunk=True,
                                   dlogits=dlogits, accumulate=True)
    dtable = sdm.sdm_lookup_grad(s["tokens"], dlogits @ s["proj"].t().contiguous(), V, scale=2.0, dropout=0.25, rng=s["rng"])
    return x, idx, w, loss, counts, out, dbank, dlogits, dtable


def test_a_training_step():
    s = inputs(1)
    x, idx, w, loss, counts, out, dbank, dlogits, dtable = step(s)
    # by the chain rule in 64 bits, through the definitions and the same choice
    table, bank = (s[n].double().cpu().requires_grad_() for n in ("table", "bank"))
    tok, cv = s["tokens"].cpu(), s["cv"].cpu()
    mask = torch.from_numpy(ref.kept(T, HD, 0.25, s["rng"].tolist()))
    y = torch.where((tok >= 0)[:, None] & mask, table[tok.clamp(min=0)] * 2 / 0.75, 0.0)
    z = y @ s["proj"].double().cpu()
    z.retain_grad()
    key = idx.cpu()
    u = torch.softmax(z.gather(1, key), 1)
    read = (u[..., None] * bank[key]).sum(1)
    live = torch.arange(T) % CHUNK < cv.long().repeat_interleave(CHUNK)
    p = torch.softmax(z, 1)
    balance, some = 0, int((cv > 0).sum())
    for g in range(T // CHUNK):
        n = int(cv[g])
        if n:
            rows = slice(g * CHUNK, g * CHUNK + n)
            c = torch.bincount(key[rows].flatten(), minlength=SLOTS).double()
            assert torch.equal(counts[g].cpu().double(), c)
            balance = balance + 0.1 * SLOTS / K / n / n / some * (c * p[rows].sum(0)).sum()
    total = (((read - s["target"].double().cpu()) ** 2).sum(1) * live).sum() / 2 + 0.5 * balance
    total.backward()
    assert loss.item() == pytest.approx(balance.item(), rel=1e-5)
    # The route's choice is exact for its own float32 logits; those differ from z by 40 roundings of terms of
    # about 1 to 10, some 1e-5: what follows is compared to a hundred times that, relative to each array's largest.
    for got, want in ((x, y), (out, torch.where(live[:, None], read, 0.0)), (dbank, bank.grad), (dlogits, z.grad),
                      (dtable, table.grad)):
        assert (got.double().cpu() - want).abs().max() <= 1e-3 * want.abs().max()
    assert not dtable[~torch.isin(torch.arange(V), tok)].any()


def same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


def test_calls_on_several_streams_at_once():
    jobs = [inputs(seed) for seed in range(4)]
    want = [step(s) for s in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in jobs]
    for _ in range(5):
        got = []
        for s, stream in zip(jobs, streams):
            with torch.cuda.stream(stream):
                got.append(step(s))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_a_graph_replayed_between_eager_calls():
    s, others = inputs(5), [inputs(seed) for seed in (6, 7, 8)]
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s)  # a first call outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(s)
    for new in (others[0], others[1], others[0], others[2], inputs(5)):
        for name, t in new.items():
            s[name].copy_(t)
        want = step(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(held, want)
        graph.replay()  # twice over the same memory
        step(others[1])
        torch.cuda.synchronize()
        assert same(held, want)


def test_the_current_stream_orders_the_calls():
    """Work on a side stream that waits for nothing but its own stream's calls."""
    g = torch.Generator(device=DEV).manual_seed(1)
    idx = torch.randint(0, 5000, (20000,), generator=g, device=DEV)
    dout = torch.randn((20000, 64), generator=g, device=DEV)
    want = sdm.sdm_lookup_grad(idx, dout, 5000)
    late = torch.zeros_like(dout)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(DEV)
    with torch.cuda.stream(side):
        big = torch.randn((4096, 4096), device=DEV)
        for _ in range(4):
            big = big @ big * 1e-3
        late.copy_(dout)
        got = sdm.sdm_lookup_grad(idx, late, 5000)
    side.synchronize()
    assert torch.equal(got, want)
