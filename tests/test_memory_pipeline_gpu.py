"""The slot router and the packed bank as they are used together, with the decode
and the gather: a memory layer's step that serves, and one that trains its
router; on several streams at once, and captured in a graph."""

import numpy as np
import pytest
import torch

import memory_ref as ref
import sparse_delta_rule_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def layer(seed, streams=48, slots=512, hd=128, W=16):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    bank = (rand(streams * slots, hd) * 0.02).to(torch.bfloat16)
    steps = []
    for _ in range(3):
        steps.append(dict(write=rand(streams, slots).to(torch.bfloat16), read=rand(streams, slots).to(torch.bfloat16),
                          v=rand(streams, hd), beta=torch.rand((streams, 1), generator=g, device=DEV),
                          g=-0.1 * torch.rand((streams, 1), generator=g, device=DEV)))
    return bank, sdm.PackedBank.empty(streams * slots, hd, "mx8", DEV), steps, dict(W=W, slots=slots)


def serve(bank, packed, step, W, slots):
    """One token of every stream: choose slots, write and read the bank, bring its packed
    copy up to date, and read that with the same weights."""
    k_idx, k_val = sdm.sdm_route(step["write"], W, normalise=True, stream_slots=slots)
    q_idx, q_val = sdm.sdm_route(step["read"], W, score="sigmoid", stream_slots=slots)
    readings = sdm.sdm_decode_step(bank, k_idx, k_val, step["v"], step["beta"], step["g"], q_idx, q_val)
    sdm.sdm_bank_pack(packed, bank, slots=k_idx, row_idx=k_idx)
    out, _ = sdm.sdm_gather_packed(packed, q_idx, q_val, chunk=1)
    return k_idx, q_idx, q_val, readings, out


def test_a_layer_that_serves():
    bank, packed, steps, sizes = layer(1)
    sdm.sdm_bank_pack(packed, bank)
    for step in steps:
        k_idx, q_idx, q_val, readings, out = serve(bank, packed, step, **sizes)
        first = sizes["slots"] * np.arange(48)[:, None]
        for name, idx, kw in (("write", k_idx, {}), ("read", q_idx, dict(score="sigmoid"))):
            keys, _ = ref.route(step[name].double().cpu().numpy(), sizes["W"], **kw)
            assert np.array_equal(idx.cpu().numpy(), keys + first)
        # the packed copy is the bank as it is now
        codes, scales = ref.pack(bank.float().cpu().numpy(), "mx8")
        assert np.array_equal(packed.codes.cpu().numpy(), codes) and np.array_equal(packed.scales.cpu().numpy(), scales)
        # e4m3 values are within half a step, 2^-4, of theirs (or 2^-10 of the block's scale, at most
        # 2^-8 of its largest value over 448): the two readings differ by at most that of each term
        rows = bank.float()[q_idx].double()
        most = rows.unflatten(-1, (4, 32)).abs().amax(-1, keepdim=True).expand(-1, -1, 4, 32).flatten(-2)
        each = torch.maximum(rows.abs() * 2.0 ** -4, 2.0 ** -9 * most / 224)
        far = (q_val.double().abs()[..., None] * each).sum(1)
        # and the decode's own roundings of q_val and of its reading to bfloat16, and of 16 float32 sums
        terms = (q_val.double().abs()[..., None] * rows.abs()).sum(1)
        far = far + (2 * 2.0 ** -8 + 2.0 ** -18) * terms
        assert ((readings.double() - out.double()).abs() <= far).all()


def train(logits, packed, target, slots):
    """A router through a frozen packed memory: its outputs, and the gradient of
    sum (out - target)^2 / 2 with respect to its scores."""
    idx, w = sdm.sdm_route(logits, 8, normalise=True, stream_slots=slots)
    out, _ = sdm.sdm_gather_packed(packed, idx, w, chunk=1)
    dw, _ = sdm.sdm_gather_weight_grad(packed, idx, out - target, chunk=1)
    return idx, out, sdm.sdm_route_backward(logits, idx, dw, normalise=True, stream_slots=slots)


def test_a_router_that_trains():
    bank, packed, steps, sizes = layer(2, streams=6, slots=64, hd=40)
    bank *= 50
    sdm.sdm_bank_pack(packed, bank)
    logits = steps[0]["write"].float()
    target = torch.randn((6, 40), device=DEV)
    idx, out, grad = train(logits, packed, target, 64)
    values = torch.from_numpy(ref.unpack(packed.codes.cpu().numpy(), packed.scales.cpu().numpy(), 40, "mx8"))
    # by the chain rule in 64 bits
    x = logits.double().cpu().requires_grad_()
    keys = idx.cpu() - 64 * torch.arange(6)[:, None]
    w = torch.softmax(x.gather(1, keys), 1)
    y = (w[..., None] * values[idx.cpu()]).sum(1)
    ((y - target.double().cpu()) ** 2).sum().div(2).backward()
    # float32 sums of 8 and of 40 terms between the two: 2^-24 each, of terms at most `size`
    d = (y - target.double().cpu()).detach().abs() + 10 * 2.0 ** -24 * values[idx.cpu()].abs().amax(1)
    size = (d[:, None] * values[idx.cpu()].abs()).sum(2).amax(1, keepdim=True)
    assert ((grad.double().cpu() - x.grad).abs() <= 2 * 60 * 2.0 ** -24 * size).all()
    assert ((grad != 0).sum(1) <= 8).all()


def test_calls_on_several_streams_at_once():
    jobs = []
    for seed in range(4):
        bank, packed, steps, sizes = layer(seed + 10)
        sdm.sdm_bank_pack(packed, bank)
        want_bank, want_packed = bank.clone(), sdm.PackedBank(packed.codes.clone(), packed.scales.clone(), 128)
        want = [serve(want_bank, want_packed, s, **sizes) for s in steps]
        jobs.append((bank, packed, steps, sizes, want, want_bank, want_packed))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in jobs]
    got = [[] for _ in jobs]
    for i in range(3):
        for n, (bank, packed, steps, sizes, *_) in enumerate(jobs):
            with torch.cuda.stream(streams[n]):
                got[n].append(serve(bank, packed, steps[i], **sizes))
    torch.cuda.synchronize()
    for n, (bank, packed, _, _, want, want_bank, want_packed) in enumerate(jobs):
        for a, b in zip(got[n], want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert torch.equal(bank, want_bank) and torch.equal(packed.codes, want_packed.codes)
        assert torch.equal(packed.scales, want_packed.scales)


def test_a_graph_replayed_between_eager_calls():
    bank, packed, steps, sizes = layer(3)
    sdm.sdm_bank_pack(packed, bank)
    step = {k: v.clone() for k, v in steps[0].items()}
    logits, target = steps[1]["write"].float(), torch.randn((48, 128), device=DEV)
    start = bank.clone(), packed.codes.clone(), packed.scales.clone()

    def all_of_it():
        return serve(bank, packed, step, **sizes) + train(logits, packed, target, sizes["slots"])

    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_of_it()  # a first call outside the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = all_of_it()
    other = layer(4)
    for new in (steps[0], steps[1], steps[2], steps[1]):
        for name, t in new.items():
            step[name].copy_(t)
        logits.copy_(new["read"])
        now = bank.clone(), packed.codes.clone(), packed.scales.clone()
        want = [t.clone() for t in all_of_it()]
        after = bank.clone(), packed.codes.clone(), packed.scales.clone()
        for t, s in zip((bank, packed.codes, packed.scales), now):
            t.copy_(s)
        graph.replay()
        for t, s in zip((bank, packed.codes, packed.scales), after):
            assert torch.equal(t, s)
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        serve(other[0], other[1], other[2][0], **sizes)  # eager work between the replays
        torch.cuda.synchronize()
    assert not torch.equal(start[0], bank)


def test_the_current_stream_orders_the_calls():
    """Work on a side stream that waits for nothing but its own stream's calls."""
    x = torch.randn((512, 4096), device=DEV)
    want = sdm.sdm_route(x, 32)
    torch.cuda.synchronize()
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream(DEV)
    with torch.cuda.stream(side):
        big = torch.randn((4096, 4096), device=DEV)
        for _ in range(4):
            big = big @ big * 1e-3
        y.copy_(x)
        got = sdm.sdm_route(y, 32)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
