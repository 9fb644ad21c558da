"""sdm_route and sdm_route_backward against the plain implementations of
tests/memory_ref.py: the same keys in the same order, always, and weights and
gradients within what their roundings allow."""

import numpy as np
import pytest
import torch

import memory_ref as ref
from sparse_delta_rule_amd import SdmError, sdm_route, sdm_route_backward

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = float("inf"), float("nan")
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def softmax_slack(x: np.ndarray) -> float:
    """How far a softmax whose row sum is float32 may be off, relatively: 2^-24 for each
    addition that a term passes through (a lane's own terms, at most keys / 64 and one,
    and 12 levels of a tree), 4 for its exponential and |x - max| <= 64 that its rounded
    argument is multiplied by (terms further down are below 2^-90 and lost in the rest)."""
    return 2.0 ** -24 * (x.shape[-1] / 64 + 1 + 12 + 4 + 64)


def within(got: torch.Tensor, want: np.ndarray, slack):
    far = np.abs(got.double().cpu().numpy() - want)
    bad = int((~(far <= slack)).sum())  # a NaN is never within
    assert bad == 0, f"{bad} of {far.size} values are off, the worst by {np.nanmax(far / np.maximum(slack, 1e-300)):.3g} of its slack"


def check_route(logits: torch.Tensor, k, *, idx_dtype=torch.int64, w_dtype=torch.float32, bias=None, **kw):
    names = dict(kept="kept_groups", top="group_top")
    idx, w = sdm_route(logits.to(DEV), k, bias=None if bias is None else bias.to(DEV), idx_dtype=idx_dtype,
                       w_dtype=w_dtype, **{names.get(a, a): v for a, v in kw.items()})
    x = logits.double().numpy()
    keys, want = ref.route(x, k, bias=None if bias is None else bias.numpy(), **kw)
    assert idx.dtype == idx_dtype and w.dtype == w_dtype
    assert np.array_equal(idx.cpu().numpy(), keys)
    slack = HALF_STEP[w_dtype] * (1 + 1e-6) + 2.0 ** -24 * 1.01
    if kw.get("score", "softmax") == "softmax" and not kw.get("normalise"):
        slack += softmax_slack(x)
    # 2^-149: a denormal result's step; half of it for bfloat16's, 2^-134
    within(w, want, slack * np.abs(want) + (2.0 ** -149 if w_dtype == torch.float32 else 2.0 ** -134))
    return idx, w


def scores_like(kind: str, T: int, N: int, seed: int) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, N), generator=g) * 2
    if kind == "levels":  # many ties
        x = (x * 2).round() / 2
    elif kind == "equal":
        x = torch.full((T, N), 0.75)
    elif kind == "up":
        x = torch.linspace(-9, 9, N).repeat(T, 1)
    elif kind == "down":
        x = torch.linspace(9, -9, N).repeat(T, 1)
    elif kind == "strided":  # the large ones all 64, 256 or 1024 apart
        x -= 100 * (torch.arange(N) % (64, 256, 1024)[seed % 3] != 5 % N)
    elif kind == "front":  # the large ones next to one another
        x -= 100 * (torch.arange(N) >= max(1, N // 16))
    elif kind == "masked":
        x[torch.rand((T, N), generator=g) < 0.7] = -INF
        x[0] = -INF
    elif kind == "odd":
        x[torch.rand((T, N), generator=g) < 0.1] = NAN
        x[torch.rand((T, N), generator=g) < 0.05] = INF
        x[torch.rand((T, N), generator=g) < 0.1] = 3.4e38
        x[torch.rand((T, N), generator=g) < 0.1] = -3.4e38
        x[torch.rand((T, N), generator=g) < 0.1] = 1e-42
        x[torch.rand((T, N), generator=g) < 0.3] = 0.0
        x[torch.rand((T, N), generator=g) < 0.3] = -0.0
    return x


SIZES = [(1, 1, 1), (3, 2, 1), (5, 7, 7), (4, 64, 8), (7, 65, 3), (3, 100, 100), (2, 255, 17), (9, 256, 8), (2, 257, 1),
         (3, 256, 256), (4, 512, 16), (2, 1000, 64), (3, 2048, 256), (2, 4099, 32), (2, 16384, 64), (1, 30001, 256),
         (1, 65536, 100)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score,normalise", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                             ("sigmoid", True)])
@pytest.mark.parametrize("T,N,k", SIZES)
def test_route_sizes(T, N, k, score, normalise, dtype):
    x = scores_like("normal", T, N, N + k).to(dtype)
    check_route(x, k, score=score, normalise=normalise, scale=2.5 if normalise else 1.0)


@pytest.mark.parametrize("kind", ["levels", "equal", "up", "down", "strided", "front", "masked", "odd"])
@pytest.mark.parametrize("T,N,k", [(4, 61, 8), (3, 256, 8), (3, 300, 128), (2, 2048, 256), (2, 5000, 33),
                                   (2, 16384, 256)])
def test_route_distributions(kind, T, N, k):
    x = scores_like(kind, T, N, N)
    check_route(x, k, score="softmax", normalise=True)
    check_route(x, k, score="sigmoid", w_dtype=torch.bfloat16, idx_dtype=torch.int32)
    if kind in ("levels", "masked", "strided"):
        check_route(x.to(torch.bfloat16), k, score="softmax")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["normal", "levels", "masked", "odd"])
@pytest.mark.parametrize("T,N,k", [(5, 64, 6), (4, 256, 8), (3, 257, 100), (2, 3001, 256), (2, 16384, 64)])
def test_route_with_a_bias(T, N, k, kind, score):
    g = torch.Generator().manual_seed(N)
    bias = (torch.rand(N, generator=g) - 0.5) * 0.2
    check_route(scores_like(kind, T, N, 3), k, score=score, bias=bias, normalise=True, scale=2.5)
    bias[::5], bias[1::7], bias[2::11] = -INF, NAN, INF
    check_route(scores_like(kind, T, N, 4), k, score=score, bias=bias, normalise=True)
    check_route(scores_like(kind, T, N, 5).to(torch.bfloat16), k, score=score, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,N,k", [(3, 200, 8), (3, 256, 8), (2, 1000, 64), (2, 6000, 200)])
def test_route_scores_that_float32_cannot_tell_apart(T, N, k, score):
    # The bias undoes the score up to its own rounding, so that score + bias differ by
    # about 2^-26 and less: only more than 32 bits put the keys in their order.
    x = scores_like("normal", 1, N, N + 1)
    s = ref.scores(x[0].double().numpy(), score)
    bias = torch.from_numpy((0.5 - s).astype(np.float32))
    check_route(x.repeat(T, 1), k, score=score, bias=bias)
    check_route(x.repeat(T, 1), k, score=score, bias=bias, normalise=True)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("kind", ["normal", "levels", "masked", "equal"])
@pytest.mark.parametrize("N,groups,kept,top,k", [(64, 8, 3, 2, 8), (256, 8, 4, 2, 8), (256, 8, 4, 1, 128), (256, 256, 9, 2, 9),
                                                 (160, 2, 1, 2, 80), (1200, 12, 5, 1, 64), (4096, 16, 16, 2, 256),
                                                 (20000, 100, 31, 2, 100), (30, 3, 2, 2, 20)])
def test_route_in_groups(N, groups, kept, top, k, kind, with_bias):
    bias = (torch.rand(N, generator=torch.Generator().manual_seed(N)) - 0.5) * 0.2 if with_bias else None
    x = scores_like(kind, 3, N, groups)
    for score in ("softmax", "sigmoid"):
        check_route(x, k, score=score, bias=bias, groups=groups, kept=kept, top=top, normalise=True)


@pytest.mark.parametrize("T", [1, 5, 64, 1000])
def test_route_many_tokens(T):
    x = scores_like("normal", T, 256, T)
    bias = (torch.rand(256, generator=torch.Generator().manual_seed(1)) - 0.5) * 0.2
    check_route(x, 8, score="sigmoid", bias=bias, groups=8, kept=4, top=2, normalise=True, scale=2.5)


def test_route_slots_of_streams():
    x = scores_like("normal", 24, 96, 1).view(2, 3, 4, 96)
    keys, _ = ref.route(x.view(24, 96).double().numpy(), 6)
    idx, w = sdm_route(x.to(DEV), 6, stream_slots=1000)
    assert idx.shape == w.shape == (2, 3, 4, 6)
    want = keys.reshape(2, 3, 4, 6) + 1000 * np.arange(4)[:, None]
    assert np.array_equal(idx.cpu().numpy(), want)
    far = sdm_route(x.to(DEV), 6, stream_slots=1 << 40)[0]
    assert np.array_equal(far.cpu().numpy(), keys.reshape(2, 3, 4, 6) + (np.arange(4)[:, None] << 40))
    with pytest.raises(SdmError, match="does not fit"):
        sdm_route(x.to(DEV), 6, stream_slots=1 << 30, idx_dtype=torch.int32)


def test_route_of_no_tokens_and_given_outputs():
    x = torch.zeros((0, 8), device=DEV)
    idx, w = sdm_route(x, 2)
    assert idx.shape == w.shape == (0, 2)
    x = scores_like("normal", 3, 8, 1).to(DEV)
    idx, w = torch.empty((3, 2), dtype=torch.int32, device=DEV), torch.empty((3, 2), dtype=torch.bfloat16, device=DEV)
    got = sdm_route(x, 2, idx=idx, w=w)
    assert got[0] is idx and got[1] is w
    assert torch.equal(idx.long(), sdm_route(x, 2)[0])
    assert sdm_route_backward(torch.zeros((0, 8), device=DEV), idx[:0], w[:0]).shape == (0, 8)


def test_route_of_unaligned_rows():
    """Logits that begin anywhere an element may, and rows of odd lengths."""
    for dtype in (torch.float32, torch.bfloat16):
        for N in (257, 256, 4099):
            flat = scores_like("normal", 1, 3 * N + 1, N)[0].to(dtype)
            x = flat.to(DEV)[1:].view(3, N)
            assert x.data_ptr() % 16
            idx, _ = sdm_route(x, 16)
            assert np.array_equal(idx.cpu().numpy(), ref.route(flat[1:].view(3, N).double().numpy(), 16)[0])
            dw = torch.randn((3, 16), device=DEV)
            out = torch.empty(3 * N + 1, dtype=dtype, device=DEV)[1:].view(3, N)
            assert torch.equal(sdm_route_backward(x, idx, dw, normalise=True, dlogits=out),
                               sdm_route_backward(x.clone(), idx, dw, normalise=True))
            # A full softmax's float32 sum is taken in another order: both hold to the definition.
            for got in (sdm_route_backward(x, idx, dw, dlogits=out), sdm_route_backward(x.clone(), idx, dw)):
                check_backward(flat[1:].view(3, N), 16, idx=idx.cpu(), dw=dw.cpu(), got=got)


def test_route_of_a_large_call():
    """More scores than 2^31: offsets past 32 bits."""
    T, N = 40000, 65536
    x = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
    rng = torch.Generator(device=DEV).manual_seed(3)
    hot = torch.randint(0, N, (T,), generator=rng, device=DEV)
    x[torch.arange(T, device=DEV), hot] = 3.0
    idx, w = sdm_route(x, 2, normalise=True)
    assert torch.equal(idx[:, 0], hot)
    assert torch.equal(idx[:, 1], (hot == 0).long())
    d = sdm_route_backward(x, idx, torch.ones((T, 2), device=DEV) * torch.tensor([1.0, 0.0], device=DEV),
                           normalise=True)
    p = 1 / (1 + np.exp(-3.0))
    want = p * (1 - p)
    top = d[torch.arange(T, device=DEV), hot].double()
    assert ((top - want).abs() <= 2.0 ** -8 * want * 1.001).all()
    assert (d != 0).sum().item() == 2 * T


@pytest.mark.parametrize("N,k", [(64, 8), (256, 12), (1000, 40), (5000, 64), (16384, 256)])
def test_route_of_signalling_nans(N, k):
    """Every kind of NaN counts as -inf, also those that no arithmetic makes."""
    for dtype, bits, plain in ((torch.float32, torch.int32, (0x7f800001, -0x7fffff, 0x7fc00000)),
                               (torch.bfloat16, torch.int16, (0x7f81, -0x7f, 0x7fc0))):
        x = scores_like("normal", 3, N, N).to(dtype)
        for i, pattern in enumerate(plain):
            x.view(bits)[i, i::3] = pattern
        assert x.isnan().sum() >= N - 3
        check_route(x, k)
        check_route(x, k, score="sigmoid", bias=torch.zeros(N), normalise=True)
        check_backward(x, k)
        check_backward(x, k, score="sigmoid", normalise=True)


# ------------------------------------------------------------------ backward


def check_backward(x: torch.Tensor, k, *, w_dtype=torch.float32, bias=None, seed=0, idx=None, dw=None, repeats=1, got=None,
                   **kw):
    dev_bias = None if bias is None else bias.to(DEV)
    if idx is None:
        idx = sdm_route(x.to(DEV), k, bias=dev_bias, **kw)[0].cpu()
    if dw is None:
        dw = torch.randn(idx.shape, generator=torch.Generator().manual_seed(seed)).to(w_dtype)
    if got is None:
        got = sdm_route_backward(x.to(DEV), idx.to(DEV), dw.to(DEV), bias=dev_bias, **kw)
    want, size = ref.route_backward(x.double().numpy(), idx.numpy(), dw.double().numpy(),
                                    bias=None if bias is None else bias.numpy(), **kw)
    # The result's rounding, and where a row's softmax is float32 the roundings of its
    # score, of its two terms and of their difference, each relative to the terms.
    slack = HALF_STEP[x.dtype] * 1.001 * np.abs(want) + 2.0 ** -24 * 1.01 * np.abs(want)
    # A key given `repeats` times adds as many terms, each rounded to float32 and each
    # sum too, relative to the terms.
    slack = slack + (2 * (repeats - 1) * 2.0 ** -24 * 1.01 + 1e-14) * size + (2.0 ** -149 if x.dtype == torch.float32 else 2.0 ** -134)
    if kw.get("score", "softmax") == "softmax" and not kw.get("normalise"):
        slack = slack + (softmax_slack(x) + 6 * 2.0 ** -24) * size
        # A score below the smallest normal float32 counts as anything up to that (its exponential
        # may be 0), and is multiplied by a difference of at most sum |dw| twice.
        slack = slack + 2.0 ** -126 * 2 * abs(kw.get("scale", 1.0)) * np.abs(dw.double().numpy()).sum(1, keepdims=True)
    assert got.dtype == x.dtype
    within(got, want, slack)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("score,normalise", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                             ("sigmoid", True)])
@pytest.mark.parametrize("T,N,k", SIZES)
def test_route_backward_sizes(T, N, k, score, normalise, dtype):
    check_backward(scores_like("normal", T, N, N).to(dtype), k, score=score, normalise=normalise, scale=2.5,
                   w_dtype=torch.bfloat16 if N % 2 else torch.float32)


@pytest.mark.parametrize("score,normalise", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                             ("sigmoid", True)])
@pytest.mark.parametrize("kind", ["levels", "equal", "masked", "odd", "front"])
def test_route_backward_distributions(kind, score, normalise):
    for T, N, k in ((4, 61, 8), (3, 256, 8), (2, 5000, 256)):
        bias = torch.zeros(N)
        bias[::3], bias[1::7] = -INF, NAN
        x = scores_like(kind, T, N, 7)
        check_backward(x, k, score=score, normalise=normalise)
        check_backward(x, k, score=score, normalise=normalise, bias=bias)


def test_route_backward_of_rows_without_a_key_is_zero():
    x = torch.full((2, 40), -INF, device=DEV)
    idx, w = sdm_route(x, 4)
    assert torch.equal(idx.cpu(), torch.arange(4).repeat(2, 1)) and not w.any()
    dw = torch.full((2, 4), NAN, device=DEV)
    for score in ("softmax", "sigmoid"):
        for normalise in (False, True):
            assert not sdm_route_backward(x, idx, dw, score=score, normalise=normalise).any()


def test_route_backward_ignores_foreign_slots_and_adds_repeated_ones():
    x = scores_like("normal", 2, 50, 3)
    for score, normalise in (("sigmoid", False), ("softmax", False)):
        idx = torch.tensor([[3, -1, 3, 1 << 40], [50, 49, 0, 0]])
        check_backward(x, 4, score=score, normalise=normalise, idx=idx, seed=2, repeats=2)


def test_route_backward_through_streams():
    x = scores_like("normal", 12, 33, 2).view(3, 4, 33).to(DEV)
    idx, _ = sdm_route(x, 5, stream_slots=64)
    flat, _ = sdm_route(x, 5)
    dw = torch.randn(idx.shape, device=DEV)
    assert torch.equal(sdm_route_backward(x, idx, dw, stream_slots=64), sdm_route_backward(x, flat, dw))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalise", [False, True])
def test_route_gradient_against_differences(score, normalise):
    """The weights of sdm_route itself, at logits moved by h, against its gradient."""
    torch.manual_seed(1)
    x = (torch.randn((4, 40)) * 2).to(DEV)
    idx, w = sdm_route(x, 6, score=score, normalise=normalise)
    dw = torch.randn(w.shape, device=DEV)
    grad = sdm_route_backward(x, idx, dw, score=score, normalise=normalise)
    h = 2.0 ** -7
    for i in range(40):
        up, down = x.clone(), x.clone()
        up[:, i] += h
        down[:, i] -= h

        def loss(y):  # the weights of the same keys: the route's own, put in the order of idx
            j, v = sdm_route(y, 40, score=score)
            s = torch.zeros((4, 40), dtype=torch.float64, device=DEV).scatter_(1, j, v.double()).gather(1, idx)
            return ((s / s.sum(1, keepdim=True) if normalise else s) * dw.double()).sum(1)

        slope = (loss(up) - loss(down)) / (2 * h)
        # a third derivative below 1 a weight times h^2 / 6, and float32 weights' roundings over 2 h
        far = dw.double().abs().sum(1) * (h * h / 6 + (2.0 ** -23 + 2 * softmax_slack(x[:1].cpu().numpy())) / (2 * h))
        assert ((slope - grad[:, i].double()).abs() <= far).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,groups,kept,top,k", [(72, 2, 1, 2, 7), (80, 8, 2, 2, 16), (34, 2, 1, 1, 6), (995, 5, 3, 2, 30), (33, 33, 7, 1, 5),
                                                 (1120, 16, 8, 2, 18), (9000, 90, 3, 2, 150), (40000, 10, 4, 2, 256)])
@pytest.mark.parametrize("kind", ["normal", "masked"])
def test_route_in_groups_that_float32_cannot_tell_apart(N, groups, kept, top, k, kind, score):
    """Groups of any size, whose values a bias makes equal but for its own rounding."""
    x = scores_like(kind, 2, N, N)
    s = ref.scores(np.where(np.isfinite(x[1].double().numpy()), x[1].double().numpy(), -1e30), score)
    bias = torch.from_numpy((0.25 - s).astype(np.float32))
    check_route(x, k, score=score, bias=bias, groups=groups, kept=kept, top=top, normalise=True)
    check_route(x, k, score=score, groups=groups, kept=kept, top=top)


@pytest.mark.parametrize("N,k", [(2048, 64), (5000, 256), (20000, 32)])
def test_route_of_equal_scores_with_a_bias(N, k):
    """More equal keys than a workgroup holds candidates: a router before its first step."""
    x = torch.zeros((2, N))
    x[1, 7::13] = -INF
    check_route(x, k, score="sigmoid", bias=torch.zeros(N), normalise=True)
    check_route(x, k, score="softmax", bias=torch.zeros(N), groups=4, kept=3, top=2)


@pytest.mark.parametrize("size", [3e2, 7e4, 1e9, 1e15, 1e25, 1e37])
@pytest.mark.parametrize("T,N,k", [(5, 64, 6), (3, 256, 8), (2, 3000, 200), (2, 16384, 64)])
def test_route_of_large_logits(T, N, k, size):
    """Logits far from 0, all of them and by turns, where a term's exponent is a difference of large numbers."""
    near = torch.randn((T, N), generator=torch.Generator().manual_seed(N)) * 0.25 + 1
    for x in (near * size, near * -size, near * size * (torch.arange(N) % 3 - 1)):
        for score in ("softmax", "sigmoid"):
            for normalise in (False, True):
                check_route(x, k, score=score, normalise=normalise)
                check_backward(x, k, score=score, normalise=normalise)
        check_route(x, k, score="softmax", bias=torch.linspace(-0.1, 0.1, N), normalise=True)


def test_route_of_the_most_tokens():
    """2^21 tokens, as many as a call takes, in both kernels: the last ones as the first."""
    T = 1 << 21
    for N in (12, 1100):
        x = torch.zeros((T, N), dtype=torch.bfloat16, device=DEV)
        hot = torch.arange(T, device=DEV) * 7919 % N
        x[torch.arange(T, device=DEV), hot] = 2.0
        idx, w = sdm_route(x, 1, idx_dtype=torch.int32)
        assert torch.equal(idx[:, 0].long(), hot)
        d = sdm_route_backward(x, idx, torch.ones_like(w))
        top = d[torch.arange(T, device=DEV), hot]
        assert (top == top[0]).all() and (top > 0).all()
        assert (d != 0).sum().item() == T * N
    with pytest.raises(SdmError, match="at most 2"):
        sdm_route(torch.zeros((T + 1, 4), device=DEV), 1)


# Every wavefront kernel (16, 32 and 64 lanes a row, 4 to 16 keys a lane) with groups that
# are not whole lanes, and enough rows that several wavefronts share each compute unit.
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("score,top,with_bias", [("softmax", 1, True), ("sigmoid", 1, False), ("softmax", 2, False), ("sigmoid", 2, True)])
@pytest.mark.parametrize("N,groups,kept,k", [(60, 12, 5, 4), (96, 16, 13, 4), (240, 16, 7, 6), (240, 15, 11, 20), (384, 16, 13, 4),
                                             (432, 4, 3, 1), (448, 16, 11, 8), (504, 8, 5, 20), (505, 5, 2, 8), (768, 16, 9, 8),
                                             (1000, 40, 31, 4)])
def test_route_in_groups_of_many_rows(N, groups, kept, k, score, top, with_bias, dtype):
    g = torch.Generator().manual_seed(N + groups)
    x = (torch.randn((4099, N), generator=g) * 1.5).to(dtype)
    x[torch.rand((4099, N), generator=g) < 0.3] = -INF
    bias = torch.rand(N, generator=g) * 0.5 if with_bias else None
    kw = dict(score=score, groups=groups, kept=kept, top=top, normalise=top == 1)
    idx, w = check_route(x, k, bias=bias, **kw)
    for _ in range(3):
        i2, w2 = sdm_route(x.to(DEV), k, bias=None if bias is None else bias.to(DEV), score=score, groups=groups,
                           kept_groups=kept, group_top=top, normalise=top == 1)
        assert torch.equal(i2, idx) and torch.equal(w2, w)


# Logits whose float64 scores are equal though they are not: a sigmoid of 37 and more is 1,
# a softmax's terms 746 below the largest are 0. Groups of equal scores go by their number.
@pytest.mark.parametrize("score", ("softmax", "sigmoid"))
@pytest.mark.parametrize("top", (1, 2))
@pytest.mark.parametrize("T,N,groups,kept,k", [(1500, 64, 8, 3, 4), (40, 256, 8, 4, 8), (1500, 256, 8, 4, 8), (1500, 384, 16, 5, 4),
                                               (40, 1000, 40, 11, 8), (20, 2000, 20, 7, 8), (7, 8192, 256, 100, 32)])
def test_route_in_groups_of_saturated_scores(T, N, groups, kept, k, top, score):
    x = torch.randn((T, N), generator=torch.Generator().manual_seed(N + T)) * 1e3
    check_route(x, k, score=score, groups=groups, kept=kept, top=top, normalise=True)
    check_route(x.bfloat16(), k, score=score, groups=groups, kept=kept, top=top)


@pytest.mark.parametrize("k", [1, 3])
@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
def test_route_of_a_near_tie_behind_equal_keys(k, dtype):
    """Two keys of equal logit and bias, and a third of a far larger score whose value is nearly
    theirs: neighbours in the order of a float32 softmax's sum that are equal tell nothing of it."""
    wrong = []
    for seed in range(150):
        g = torch.Generator().manual_seed(seed)
        N = 2048
        x = torch.randn((1, N), generator=g).to(dtype)
        low, far, first = 300 + seed, 1500 - seed, torch.tensor([40, 1900])
        x[0, far] = 6.0 + 0.01 * seed  # a score of a tenth to a third
        x[0, low] = x[0, low + 700] = -2.0
        bias = torch.full((N,), -3.0)  # the other keys: far from the best
        s = ref.scores(x[0].double().numpy(), "softmax")
        bias[far] = 0.25
        bias[low] = bias[low + 700] = float(s[far] + 0.25 - s[low])  # within 2^-25 of a tie
        if k == 3:
            bias[first] = torch.tensor([3.0, 2.5])
        idx, _ = sdm_route(x.to(DEV), k, bias=bias.to(DEV))
        keys, _ = ref.route(x.double().numpy(), k, bias=bias.numpy())
        if not np.array_equal(idx.cpu().numpy(), keys):
            wrong.append(seed)
    assert wrong == []


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,N,groups", [(3, 64, 2), (1500, 64, 8), (3, 90, 5), (1500, 256, 8), (3, 1000, 10), (3, 3000, 6)])
def test_route_in_groups_at_the_lowest_bias(T, N, groups, score):
    """A mask of the type's lowest value: two such keys sum to more than float32 holds, and still
    go before a group that has no eligible key."""
    size = N // groups
    x = scores_like("normal", T, N, N)
    lowest = -float(np.finfo(np.float32).max)
    bias = torch.full((N,), -INF)
    bias[(groups - 1) * size:] = lowest
    check_route(x, 2, score=score, bias=bias, groups=groups, kept=1, top=2, normalise=True)
    bias[:size] = lowest  # equal values but for float64: the lower group
    check_route(x, 2, score=score, bias=bias, groups=groups, kept=1, top=2)
    bias[size] = lowest  # one such key is more than two
    check_route(x, 1, score=score, bias=bias, groups=groups, kept=1, top=2)
    bias[:size] = lowest / 2 * 1.5
    check_route(x, 2, score=score, bias=bias, groups=groups, kept=1, top=2)
    bias[1::2] = -INF
    check_route(x, 4, score=score, bias=bias, groups=groups, kept=2, top=2)


@pytest.mark.parametrize("T,N", [(6000, 64), (6000, 256), (1024, 1000), (6000, 3000)])
def test_route_of_scores_that_a_large_bias_makes_equal(T, N):
    """Two keys of a bias of 1e9, a step of which in float64 is 2^-23: scores nearer than that are equal
    or not by where a step falls, which a float32 softmax's sum does not tell."""
    g = torch.Generator().manual_seed(N)
    x = torch.randn((T, N), generator=g)
    at = torch.randperm(N, generator=g)[:2].sort().values
    x[:, at] = float(4 + np.log(N / 64)) + torch.rand((T, 1), generator=g) + torch.tensor([0, 2.0 ** -21])
    bias = torch.zeros(N)
    bias[at] = 1e9
    idx, _ = sdm_route(x.to(DEV), 1, bias=bias.to(DEV))
    X = x.double().numpy()
    e = np.exp(X - X.max(1, keepdims=True))
    v = (e / e.sum(1, keepdims=True))[:, at.numpy()] + 1e9
    want = at.numpy()[(v[:, 1] > v[:, 0]).astype(int)]
    bad = (idx[:, 0].cpu().numpy() != want).sum()
    assert bad == 0, f"{bad} of {T} rows"


@pytest.mark.parametrize("bad", [INF, -INF, NAN], ids=["inf", "-inf", "nan"])
@pytest.mark.parametrize("T,N,k", [(4, 61, 8), (3, 256, 8), (2, 5001, 200), (2, 16384, 64), (1, 40000, 256)])
@pytest.mark.parametrize("score,normalise", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_route_backward_of_a_gradient_that_is_not_finite(T, N, k, bad, score, normalise):
    """A key at -inf has the gradient 0 whatever the others' is; a full softmax's other keys are none of them finite."""
    x = scores_like("masked", T, N, N)
    x[0] = scores_like("normal", 1, N, 1)[0]
    x[0, ::3] = -INF
    for dtype in (torch.float32, torch.bfloat16):
        d = x.to(dtype).to(DEV)
        idx, _ = sdm_route(d, k, score=score, normalise=normalise)
        dw = torch.randn(idx.shape, generator=torch.Generator().manual_seed(1)).to(DEV)
        dw[:, 0] = bad
        got = sdm_route_backward(d, idx, dw, score=score, normalise=normalise)
        masked = d == -INF
        assert not (got[masked] != 0).any()
        chosen = torch.zeros_like(masked).scatter_(1, idx, True)
        if normalise or score == "sigmoid":
            assert not (got[~chosen] != 0).any()
            assert not got.gather(1, idx)[:, 0].isfinite().any()
        else:
            assert not got[~masked].isfinite().any()


def test_route_backward_where_the_weights_sum_to_zero():
    """Renormalised sigmoid scores that are all 0 in float64: the gradient is 0, also of an infinite one."""
    x = torch.full((3, 50), -800.0)
    x[1] = -3e38
    x[2, 7] = 1.0  # a row whose sum is not 0
    for dtype in (torch.float32, torch.bfloat16):
        d = x.to(dtype).to(DEV)
        idx, w = sdm_route(d, 4, score="sigmoid", normalise=True)
        assert not w[:2].any()
        for bad in (INF, NAN, 1.0):
            dw = torch.full((3, 4), bad, device=DEV)
            got = sdm_route_backward(d, idx, dw, score="sigmoid", normalise=True)
            assert not (got[:2] != 0).any()
            assert got[2, 7].isnan() == (bad != 1.0)


@pytest.mark.parametrize("dtype", (torch.float32, torch.bfloat16))
@pytest.mark.parametrize("T,N,k", [(3, 200, 8), (2, 5000, 64), (2, 16384, 64), (1, 40000, 256)])
def test_route_backward_of_large_gradients(T, N, k, dtype):
    """Sums of du s past float32's range, with gradients inside it."""
    x = (scores_like("normal", T, N, N) * 0.1).to(dtype)
    check_backward(x, k, scale=2.0 ** 127, dw=torch.full((T, k), N / 16.0))  # a sum of about 2^127 k / 16

    # And where the keys of the largest scores get gradients past it themselves: k + 1 of them,
    # all but one chosen, and masked keys and some 60 below behind them.
    x = scores_like("normal", T, N, N).to(dtype)
    x[:, :N // 2] = -INF
    x[:, :k + 1] = torch.linspace(60, 50, k + 1).to(dtype)
    idx = torch.arange(1, k + 1).repeat(T, 1)
    idx[:, 0] = 0
    du = 2.0 ** 100
    want, _ = ref.route_backward(x.double().numpy(), idx.numpy(), np.full((T, k), du), scale=du)
    got = sdm_route_backward(x.to(DEV), idx.to(DEV), torch.full((T, k), du, device=DEV), scale=du).double().cpu().numpy()
    assert (got[:, 0] == np.inf).all()
    want, got, X = want[:, k + 1:], got[:, k + 1:], x.double().numpy()[:, k + 1:]
    assert 0 < np.abs(want).max() < 2.0 ** 126
    # A float32 exponential of a distance d: 2.25 d 2^-24 (the distance's rounding, the product with log2 e
    # and that constant's own) and 4 2^-24, in the key's own term and in the row's sum; six roundings
    # of their product; and the result's.
    eps = 2.0 ** -24 * (2.25 * (60 - X[np.isfinite(X)].min()) + 8)
    assert (np.abs(got - want) <= (2 * eps + 6 * 2.0 ** -24 + HALF_STEP[dtype] * 1.001) * np.abs(want)).all()


@pytest.mark.parametrize("peak", [10, 17, 20, 24, 30, 40])
@pytest.mark.parametrize("T,N,k", [(2, 256, 1), (3, 255, 4), (2, 1000, 8), (2, 5000, 33), (2, 16384, 64), (1, 40000, 256)])
def test_route_backward_of_a_peaked_row(T, N, k, peak):
    """One chosen key far above the rest: 1 - s is what the others' scores sum to, and keeps its
    relative precision, so a chosen key's gradient is right relative to what cancels in exact
    arithmetic only, B_j = |du_j| (1 - s_j) + sum over m != j of |du_m| s_m, times s_j."""
    x = scores_like("normal", T, N, N) * 0.5
    hot = torch.arange(T) * 37 + 5
    x[torch.arange(T), hot] = x.amax(1) + peak
    idx = sdm_route(x.to(DEV), k)[0].cpu()
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(peak))
    got = sdm_route_backward(x.to(DEV), idx.to(DEV), dw.to(DEV), scale=1.5).double().cpu().numpy()
    X = x.double().numpy()
    # A float32 exponential of a distance d: 2.25 d 2^-24 (the distance's rounding, the product with
    # log2 e and that constant's own), 4 2^-24 itself, again 4 where a wavefront's sum is moved to
    # the row's largest. The row's sum then is off by at most eps of what the other keys add, in
    # relation to all by eps (1 - s_max), and s_j (du_j - dot) by at most 2 eps s_j B_j.
    eps = 2.0 ** -24 * (2.25 * (X.max() - X.min()) + 8)
    for t in range(T):
        e = np.exp(X[t] - X[t].max())
        rest = np.array([np.delete(e, j).sum() for j in idx[t].numpy()])
        z, s = e.sum(), e / e.sum()
        d, at = 1.5 * dw[t].double().numpy(), idx[t].numpy()
        other = np.array([np.delete(d * s[at], j).sum() for j in range(k)])
        size = np.array([np.delete(np.abs(d) * s[at], j).sum() for j in range(k)])
        want = s[at] * (d * (rest / z) - other)
        B = s[at] * (np.abs(d) * (rest / z) + size)
        # the result's rounding, and float64's own where 1 - s is taken as a difference: at most 64 additions
        # of a lane, 6 levels of lanes, 16 wavefronts and a division, 2^-53 each
        slack = 2.0 ** -24 * 1.01 * np.abs(want) + 2 * eps * B + 2.0 ** -46 * s[at] * np.abs(d)
        far = np.abs(got[t][at] - want)
        assert (far <= slack).all(), (t, (far / slack).max())
        dot = (d * s[at]).sum()
        out = np.setdiff1d(np.arange(N), at)
        assert (np.abs(got[t][out] + s[out] * dot) <= 2 * eps * s[out] * (np.abs(d) * s[at]).sum() + 2.0 ** -149).all()
