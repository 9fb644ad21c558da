"""sdm_route_balance and its gradient against the plain implementation of
tests/train_ref.py: counts exactly, sums and gradients within what float32 allows."""

import numpy as np
import pytest
import torch

import train_ref as ref
import sparse_delta_rule_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = float("inf"), float("nan")
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def choices(seed, T, N, k, stray=0.05):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, N, (T, k), generator=g)
    idx[torch.rand((T, k), generator=g) < stray] = -1  # not a key of its token
    return idx


def logits_like(seed, T, N, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, N), generator=g) * spread + torch.randn((N,), generator=g)).to(dtype)


def check(x, idx, *, score="softmax", scale=1.0, stream_slots=0, index=torch.int64, dloss=1.5, tokens=None, **kw):
    """Both directions of a call; returns its results."""
    T, N = x.shape
    np_kw = {k: (v.numpy() if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    gpu_kw = {k: (v.to(DEV) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    slots = idx + stream_slots * torch.arange(T)[:, None] if stream_slots else idx
    xd = x.to(DEV)
    loss, counts, mean, coef = sdm.sdm_route_balance(xd, slots.to(index).to(DEV), score=score, scale=scale,
                                                     stream_slots=stream_slots, **gpu_kw)
    want, (far, off) = ref.balance(x.float().numpy(), idx.numpy(), score=score, scale=scale, **np_kw)
    assert np.array_equal(counts.cpu().numpy(), want[1])
    assert (np.abs(mean.double().cpu().numpy() - want[2]) <= off).all()
    assert (np.abs(coef.double().cpu().numpy() - want[3]) <= 2.0 ** -23 * np.abs(want[3])).all()
    assert abs(loss.item() - want[0]) <= far
    d = sdm.sdm_route_balance_backward(xd, counts, coef, dloss=torch.tensor(dloss, device=DEV), score=score, **gpu_kw)
    g, size = ref.balance_backward(x.float().numpy(), want[1], coef.cpu().numpy(), dloss=float(np.float32(dloss)),
                                   score=score, **np_kw)
    assert d.dtype == x.dtype
    got = d.double().cpu().numpy()
    # half a step of the type, and of its least normal number (a score below 2^-126 may count as 0)
    bound = size + EPS[x.dtype] * (np.abs(g) + size) + 2.0 ** -126
    assert (np.abs(got - g) <= bound).all(), np.abs(got - g).max()
    return loss, counts, mean, coef, d


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 16, 100, 127, 128, 129, 256, 257, 500, 512, 513, 1000, 1024])
def test_keys(N, dtype, score):
    check(logits_like(N, 70, N, dtype), choices(N, 70, N, min(N, 6)), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [1025, 1032, 4096, 8192, 8193, 16384, 16400, 20001, 32768, 40000, 65535, 65536])
def test_many_keys(N, dtype, score):
    check(logits_like(N, 5, N, dtype), choices(N, 5, N, 64), score=score, scale=0.3)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 511, 512, 513, 1025, 3001])
def test_tokens(T):
    check(logits_like(T, T, 40), choices(T, T, 40, 4), index=torch.int32)
    check(logits_like(T, T, 40, torch.bfloat16), choices(T, T, 40, 40), score="sigmoid", scale=-2.0)


def test_more_tokens_than_a_piece_holds():
    """More than 512 * 255 tokens: pieces of 255, choices of 256 keys each by every token."""
    T = 512 * 255 + 300
    x, idx = torch.zeros((T, 2)), torch.zeros((T, 2), dtype=torch.int64)
    loss, counts, mean, coef = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV))
    assert counts.tolist() == [[2 * T, 0]] and mean.tolist() == [[0.5, 0.5]] and loss.item() == 1.0
    x, idx = torch.zeros((3000, 300)), torch.arange(256).expand(3000, 256).contiguous()
    idx[:, 100:] = 7  # a key named many times by one token counts as often
    _, counts, _, _ = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV), chunk=1500, per_chunk=True)
    assert counts[:, 7].tolist() == [1500 * 157] * 2 and counts[:, 99].tolist() == [1500] * 2
    assert counts.sum().item() == 3000 * 256


@pytest.mark.parametrize("per_chunk", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("chunk,valid", [(1, None), (6, 4), (60, None), (60, 0), (150, 149), (300, 300)])
def test_chunks(chunk, valid, score, per_chunk):
    x, idx = logits_like(3, 300, 33), choices(4, 300, 33, 5)
    check(x, idx, score=score, chunk=chunk, valid=valid, per_chunk=per_chunk, scale=0.01)


@pytest.mark.parametrize("per_chunk", [False, True])
@pytest.mark.parametrize("N", [60, 1100])
def test_ragged_chunks(per_chunk, N):
    g = torch.Generator().manual_seed(8)
    for chunk in (10, 25, 100):
        cv = torch.randint(0, chunk + 1, (200 // chunk,), generator=g).to(torch.int32)
        cv[0] = 0
        x, idx = logits_like(chunk, 200, N), choices(chunk, 200, N, 3)
        x[3], idx[3] = NAN, 1 << 40  # padding: whatever it holds
        _, _, _, _, d = check(x, idx, chunk=chunk, chunk_valid=cv, per_chunk=per_chunk, scale=0.7)
        out = torch.full((200, N), 3.0, device=DEV)
        counts = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV), chunk=chunk, chunk_valid=cv.to(DEV), per_chunk=per_chunk,
                                       scale=0.7)
        got = sdm.sdm_route_balance_backward(x.to(DEV), counts[1], counts[3], chunk=chunk, chunk_valid=cv.to(DEV),
                                             per_chunk=per_chunk, dloss=torch.tensor([1.5], device=DEV), dlogits=out,
                                             accumulate=True)
        assert got is out
        live = torch.from_numpy(ref.live(200, chunk, chunk_valid=cv.numpy())).to(DEV)
        assert torch.equal(out[~live], torch.full_like(out[~live], 3.0))
        assert torch.equal(out[live], 3.0 + d[live])


def test_chunk_counts_past_the_chunk_are_the_chunk():
    x, idx = logits_like(3, 40, 16), choices(4, 40, 16, 2)
    cv = torch.tensor([-5, 10, 99, 3], dtype=torch.int32)
    a = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV), chunk=10, chunk_valid=cv.to(DEV), per_chunk=True)
    b = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV), chunk=10, chunk_valid=cv.clamp(0, 10).to(DEV), per_chunk=True)
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and a[3][0].item() == 0 and a[1][0].sum().item() == 0


@pytest.mark.parametrize("per_chunk", [False, True])
def test_no_tokens(per_chunk):
    out = sdm.sdm_route_balance(torch.empty((0, 300), device=DEV), torch.empty((0, 5), dtype=torch.int64, device=DEV),
                                loss=torch.full((), 7.0, device=DEV), chunk=4, per_chunk=per_chunk)
    n = 0 if per_chunk else 1
    assert out[0].item() == 0 and [list(t.shape) for t in out[1:]] == [[n, 300], [n, 300], [n]]
    assert not any(t.any() for t in out)
    all_padding = sdm.sdm_route_balance(torch.zeros((8, 300), device=DEV), torch.zeros((8, 5), dtype=torch.int64, device=DEV),
                                        chunk=4, valid=0, per_chunk=per_chunk)
    assert not any(t.any() for t in all_padding)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [50, 200, 600, 3000, 20000, 40000])
def test_masked_and_extreme_logits(N, score):
    x = logits_like(9, 24, N)
    g = torch.Generator().manual_seed(5)
    x[torch.rand(x.shape, generator=g) < 0.3] = -INF
    x[2], x[3] = -INF, NAN
    x[4, ::3] = NAN
    x[5, 7] = INF
    x[6, 7] = x[6, 9] = INF
    x[7] = torch.finfo(torch.float32).min
    x[8] = x[8] * 1e4 - 1e6
    x[9] = x[9] * 50
    x[10] = -70 - x[10].abs()
    x[11] = -63.9
    x[12], x[12, 5] = -200.0, -64.0
    x[13] = 1e30
    x[14, :] = -INF
    x[14, N - 1] = -3e38
    x[15] = 60 + x[15]
    _, _, mean, _, d = check(x, choices(9, 24, N, 4), score=score)
    assert not d[torch.isneginf(x).to(DEV) | torch.isnan(x).to(DEV)].any()
    assert torch.isfinite(mean).all() and not d[2].any() and not d[3].any()


@pytest.mark.parametrize("N", [64, 2048, 16384, 20001, 40000, 65535])
@pytest.mark.parametrize("gap", [5.0, 20.0, 40.0, 80.0])
def test_one_key_far_above_the_rest(N, gap):
    """Its gradient is of the others' size times their shares: differences to its own count cancel nothing."""
    x = torch.zeros((4, N))
    x[:, 3] = gap
    idx = torch.full((4, 2), 3)
    idx[1, 0], idx[2, 0] = 5, 9
    _, counts, _, coef, d = check(x, idx)
    want, _ = ref.balance_backward(x.numpy(), counts.cpu().numpy(), coef.cpu().numpy(), dloss=1.5)
    # a sum of like signs but for keys 5 and 9, which are less than a thirtieth of the terms: 8 u for each
    # of at most 120 roundings, and (4 + 3 gap) u of the shares
    assert np.allclose(d[:, 3].cpu(), want[:, 3], rtol=(8 * 120 + 4 * gap) * 2.0 ** -24, atol=2.0 ** -126)
    assert want[0, 3] > 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [40, 300, 900, 5000, 33000])
def test_confident_rows(N, score, dtype):
    """Rows one of whose keys has more, or nearly, 4/5 of the share, beside even ones."""
    x = logits_like(3, 40, N, torch.float32, 0.5)
    for t in range(40):
        if t % 3:
            level = np.log(max(N - 1, 1) * (3.5 + t / 20))  # shares about 0.78 to 0.85
            x[t] = x[t] * 0.01 - (30 if score == "sigmoid" else 0)
            x[t, (t * 7) % N] += float(level)
    check(x.to(dtype), choices(4, 40, N, 4), score=score, chunk=10, chunk_valid=torch.tensor([10, 7, 0, 9], dtype=torch.int32),
          per_chunk=True)


def test_counts_that_are_all_alike_or_large():
    """The gradient of equal counts is 0 up to the differences' own roundings; counts past 2^24 keep their differences."""
    x = logits_like(5, 16, 64).to(DEV)
    coef = torch.ones(1, device=DEV)
    same = torch.full((1, 64), 123456, dtype=torch.int32, device=DEV)
    assert not sdm.sdm_route_balance_backward(x, same, coef).any()
    big = same + (1 << 28)
    big[0, ::2] += 3
    small = torch.zeros_like(same)
    small[0, ::2] = 3
    a, b = (sdm.sdm_route_balance_backward(x, c, coef) for c in (big, small))
    want, size = ref.balance_backward(x.cpu().numpy(), small.cpu().numpy(), [1.0])
    for d in (a, b):
        assert (np.abs(d.double().cpu().numpy() - want) <= size + 2.0 ** -23 * np.abs(want)).all()


def test_streams_and_index_types():
    x, idx = logits_like(1, 24, 50), choices(2, 24, 50, 7)
    check(x, idx, stream_slots=50, index=torch.int32)
    check(x, idx, stream_slots=1000)
    # [steps, streams, keys] as a sequence of decodes' routes have them
    x3 = x.view(4, 6, 50).to(DEV)
    slots, _ = sdm.sdm_route(x3, 7, stream_slots=64)
    a = sdm.sdm_route_balance(x3, slots, stream_slots=64)
    keys = slots.cpu() - 64 * torch.arange(6)[None, :, None]
    b = sdm.sdm_route_balance(x.to(DEV), keys.view(24, 7).to(DEV))
    assert all(torch.equal(u, v) for u, v in zip(a, b)) and a[1].sum().item() == 24 * 7


@pytest.mark.parametrize("dtype,off", [(torch.float32, 1), (torch.bfloat16, 1), (torch.bfloat16, 4)])
@pytest.mark.parametrize("N", [64, 2048])
def test_unaligned_logits(dtype, off, N):
    x, idx = logits_like(1, 20, N, dtype), choices(2, 20, N, 4)
    flat = torch.cat([torch.zeros(off, dtype=dtype), x.flatten()]).to(DEV)
    a = sdm.sdm_route_balance(flat[off:].view(20, N), idx.to(DEV))
    b = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV))
    assert torch.equal(a[1], b[1]) and torch.allclose(a[2], b[2], rtol=1e-4)
    out = torch.zeros(20 * N + off, dtype=dtype, device=DEV)
    sdm.sdm_route_balance_backward(flat[off:].view(20, N), a[1], a[3], dlogits=out[off:].view(20, N))
    want = sdm.sdm_route_balance_backward(x.to(DEV), b[1], b[3])
    assert torch.allclose(out[off:].view(20, N).float(), want.float(), rtol=1e-2 if dtype == torch.bfloat16 else 1e-4, atol=1e-7)
    assert not out[:off].any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("N", [50, 256, 1500])
def test_added_to_the_routes_own_gradient(N, dtype):
    x = logits_like(6, 30, N, dtype).to(DEV)
    idx, w = sdm.sdm_route(x, 5, normalise=True)
    base = sdm.sdm_route_backward(x, idx, torch.randn(w.shape, device=DEV), normalise=True)
    loss, counts, mean, coef = sdm.sdm_route_balance(x, idx, scale=0.5)
    alone = sdm.sdm_route_balance_backward(x.float(), counts, coef)
    got = sdm.sdm_route_balance_backward(x, counts, coef, dlogits=base.clone(), accumulate=True)
    # the same values, their sum rounded once
    assert torch.equal(got, (base.float() + alone).to(dtype)) or dtype == torch.bfloat16
    far = (got.double() - (base.double() + alone.double())).abs()
    assert (far <= EPS[dtype] * (base.double() + alone.double()).abs() + 2.0 ** -24 * (base.double().abs() + alone.abs())).all()


def test_gradients_that_are_not_finite_stay_in_their_rows():
    x, idx = logits_like(1, 10, 40), choices(2, 10, 40, 4)
    x[3, 5] = -INF
    x[4] = -INF
    _, counts, _, coef = sdm.sdm_route_balance(x.to(DEV), idx.to(DEV), chunk=5, per_chunk=True)
    d = sdm.sdm_route_balance_backward(x.to(DEV), counts, coef, chunk=5, per_chunk=True, dloss=torch.tensor(INF, device=DEV))
    assert d[3, 5].item() == 0 and not d[4].any() and not torch.isfinite(d[0]).all()
    assert torch.isfinite(sdm.sdm_route_balance_backward(x.to(DEV), counts, coef, chunk=5, per_chunk=True)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [40, 200, 600, 3000, 20000, 40000])
def test_gradients_near_the_largest_float32(N, score):
    """With a factor of 1e35 some gradients are past float32: those are infinite, the others as they are, and a key without a
    score has none."""
    x = logits_like(N, 6, N)
    x[:, ::3] -= 60.0  # shares of 1e-26
    x[:, 5], x[2], x[3, :] = -INF, -INF, -80.0
    x[3, 7] = -INF
    x[1] -= 30.0
    x[1, 1] = x[1].max() + np.log(N)  # the key of the large count, with half of the share or more
    counts = torch.randint(0, 50, (1, N), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    counts[0, 1] = 1 << 24
    coef, dloss = torch.tensor([1e5], device=DEV), np.float32(1e30)
    d = sdm.sdm_route_balance_backward(x.to(DEV), counts.to(DEV), coef, dloss=torch.tensor(float(dloss), device=DEV), score=score)
    got = d.double().cpu().numpy()
    want, size = ref.balance_backward(x.numpy(), counts.numpy(), [1e5], dloss=float(dloss), score=score)
    most = float(torch.finfo(torch.float32).max)
    # f is rounded twice more here. A score below 2^-126 (a softmax's and a deep sigmoid's relative to the row's
    # largest) may count as 0: a share of 2^-126 over the row's sum, which is at least its largest score, times a
    # difference below 2^25.
    top = x.double().numpy().max(1, keepdims=True)
    least = 1 / (1 + np.exp(-top)) if score == "sigmoid" else np.ones_like(top)
    least[top <= -64] = 1
    bound = size + 4 * 2.0 ** -24 * (np.abs(want) + size) + 2.0 ** -126 / least * 2.0 ** 25 * 1e35
    inside, past = np.abs(want) + bound < most, np.abs(want) - bound > most
    assert inside.any() and past.any() and not d[torch.isneginf(x).to(DEV)].any()
    assert (np.abs(got - want)[inside] <= bound[inside]).all() and (got[past] == np.sign(want[past]) * INF).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [8, 100, 200, 400, 1000, 3000])
def test_a_rows_gradient_is_its_own(N, score, dtype):
    """The same bits whatever the rows beside it hold: a key above the rest, none, very large ones, very small scores."""
    T = 4096  # eight rows and more of a workgroup
    x = logits_like(N, T, N, torch.float32, 0.5)
    counts = torch.randint(0, 50, (1, N), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    counts[0, N // 2] = 1 << 20
    beside = x.clone()
    beside[1::6], beside[3::6], beside[5::6] = 0.0, 3e30, -63.9  # every other row; e^63.9 times dloss passes float32
    beside[1::6, N // 3] = 12.0 + np.log(N)
    beside[51] = -INF
    coef, dloss = torch.ones(1, device=DEV), torch.tensor(1e15, device=DEV)
    for add in (False, True):
        got = [sdm.sdm_route_balance_backward(v.to(dtype).to(DEV), counts.to(DEV), coef, dloss=dloss, score=score,
                                              dlogits=torch.zeros((T, N), dtype=dtype, device=DEV), accumulate=add)[::2] for v in (x, beside)]
        assert torch.isfinite(got[0]).all() and got[0].any() and torch.equal(*got)


def test_given_outputs_and_workspace_and_repeats():
    x, idx = logits_like(1, 3000, 300).to(DEV), choices(2, 3000, 300, 8).to(DEV)
    first = sdm.sdm_route_balance(x, idx, scale=0.1)
    size = sdm.library().sdm_route_balance_workspace(3000, 300, 3000, 0)
    ws = torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
    outs = [torch.full_like(t, 77) for t in first]
    for _ in range(3):
        got = sdm.sdm_route_balance(x, idx, scale=0.1, loss=outs[0], counts=outs[1], mean=outs[2], coef=outs[3], workspace=ws)
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(got, outs, first))
    with pytest.raises(sdm.SdmError, match="bytes"):
        sdm.sdm_route_balance(x, idx, workspace=ws[:size - 16])
