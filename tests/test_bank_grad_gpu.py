"""sdm_lookup_grad and sdm_gather_bank_grad against the plain implementation of
tests/train_ref.py: bit for bit on small whole numbers, whose sums float32 holds exactly,
and within what float32 sums allow on others."""

import numpy as np
import pytest
import torch

import train_ref as ref
import sparse_delta_rule_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = float("inf"), float("nan")
EPS = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative
BOTH = [torch.float32, torch.bfloat16]


def slots_like(kind, n, slots, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "even":
        idx = torch.randint(0, slots, (n,), generator=g)
    elif kind == "skewed":
        idx = (torch.exp(torch.rand(n, generator=g, dtype=torch.float64) * np.log(slots)).long() - 1).clamp(0, slots - 1)
    elif kind == "one":
        idx = torch.full((n,), slots // 2)
    elif kind == "runs":  # of every length up to some hundreds
        idx = (torch.arange(n).double().sqrt() * 2).long() % slots
    elif kind == "falling":
        idx = (slots - 1 - torch.arange(n)) % slots
    else:  # most of them none
        idx = torch.where(torch.rand(n, generator=g) < 0.9, -1, torch.randint(0, slots, (n,), generator=g))
    return idx


def whole(shape, seed, most=3):
    return torch.randint(-most, most + 1, shape, generator=torch.Generator().manual_seed(seed)).float()


def lookup_case(n, slots, hd, kind, *, bank=torch.float32, out=torch.float32, index=torch.int64, add=False, p=0.0, scale=1.0,
                exactly=True, seed=0):
    idx = slots_like(kind, n, slots, seed + n)
    dout = (whole((n, hd), seed) if exactly else torch.randn((n, hd), generator=torch.Generator().manual_seed(seed))).to(out)
    rng = torch.tensor([seed * 77 + 1, (1 << 35) + n])
    mask = ref.kept(n, hd, p, rng.tolist())
    a = float(ref.factor(scale, p))
    v = np.where(mask, dout.double().numpy(), 0)
    want, size, count = ref.bank_grad(slots, idx.numpy(), lambda e: v[e], hd)
    old = whole((slots, hd), 5, 100).to(bank)
    dbank = old.clone().to(DEV) if add else None
    got = sdm.sdm_lookup_grad(idx.to(index).to(DEV), dout.to(DEV), slots, scale=scale, dropout=p, rng=rng.to(DEV),
                              bank_dtype=bank, dbank=dbank, accumulate=add)
    assert got.dtype == bank and (got is dbank or not add)
    check(got, want * a, size * abs(a), count, old.double().numpy() if add else None, exactly and a in (1.0, 2.0))


def check(got, want, size, count, old, exactly):
    total = want if old is None else want + old
    dtype = got.dtype
    got = got.double().cpu().numpy()
    if exactly and dtype == torch.float32:
        assert np.array_equal(got, total), np.argwhere(got != total)[:5]
        return
    # m terms: m additions of a sum at most `size`, the factor's product and the sum with what was there
    off = (count[:, None] + 2) * 2.0 ** -24 * size * (1 + 1e-3) + 2 * 2.0 ** -24 * np.abs(total)
    if exactly:
        off *= 0
    assert (np.abs(got - total) <= off + EPS[dtype] * (np.abs(total) + off) + 2.0 ** -140).all(), np.abs(got - total).max()
    unnamed = count == 0
    assert np.array_equal(got[unnamed], (np.zeros_like(total) if old is None else old)[unnamed])


@pytest.mark.parametrize("kind", ["even", "skewed", "one", "runs", "falling", "none"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 63, 64, 65, 500, 4095, 4096, 4097, 9000])
def test_lengths(n, kind):
    lookup_case(n, 300, 24, kind)
    lookup_case(n, 65537 if kind == "even" else 40, 3, kind, index=torch.int32, add=True)


@pytest.mark.parametrize("add", [False, True], ids=["write", "add"])
@pytest.mark.parametrize("out", BOTH, ids=["dout-f32", "dout-bf16"])
@pytest.mark.parametrize("bank", BOTH, ids=["f32", "bf16"])
@pytest.mark.parametrize("hd", [1, 2, 7, 8, 9, 40, 64, 100, 101, 128, 200, 256, 512, 513, 1024, 1032])
def test_columns(hd, bank, out, add):
    lookup_case(700, 50, hd, "skewed", bank=bank, out=out, add=add, index=torch.int32)
    lookup_case(700, 50, hd, "runs", bank=bank, out=out, add=add, exactly=False, scale=0.7)


@pytest.mark.parametrize("slots", [1, 2, 3, 255, 256, 257, 65535, 65536, 65537, (1 << 16) * 5, (1 << 24) - 1, 1 << 24, (1 << 24) + 1])
def test_slots(slots):
    """One to four passes of the sort, whose last digits are few or many."""
    lookup_case(5000, slots, 2, "even")
    lookup_case(5000, slots, 2, "skewed", add=True, index=torch.int32)


@pytest.mark.parametrize("kind", ["even", "skewed", "one", "runs", "falling", "none"])
@pytest.mark.parametrize("n", [15, 16, 17, 4096, 4097, 8192, 65536, 65537, 70001])
def test_banks_of_more_rows_than_entries(n, kind):
    """Zeroed beside the sort: of one workgroup, of up to 64 tiles, of more."""
    lookup_case(n, n, 4, kind, out=torch.bfloat16)
    lookup_case(n, n + 77777, 9 if n < 20000 else 2, kind, bank=torch.bfloat16, index=torch.int32)


@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
@pytest.mark.parametrize("n", [65537, 131072, 140001, 300000])
def test_more_entries_than_rows(n, kind):
    lookup_case(n, 5000, 4, kind)
    lookup_case(n, 300, 5, kind, add=True, exactly=kind != "one")


@pytest.mark.parametrize("n", [16 * 64 - 1, 16 * 64, 16 * 64 + 1, 16 * 65, 16 * 130 + 5, 16 * 1100])
@pytest.mark.parametrize("before", [0, 1, 15, 16, 17, 500])
def test_runs_over_many_blocks(n, before):
    """A run that begins anywhere in a block and goes on over windows of 64 of them, with other runs around it."""
    idx = torch.cat([torch.zeros(before, dtype=torch.int64), torch.full((n,), 5), torch.arange(6, 40), torch.full((300,), 41)])
    dout = whole((len(idx), 4), 3)
    for slots in (42, 100000):
        want = torch.zeros((slots, 4), dtype=torch.float64).index_add_(0, idx, dout.double())
        for add in (False, True):
            dbank = torch.full((slots, 4), 2.0, device=DEV)
            got = sdm.sdm_lookup_grad(idx.to(DEV), dout.to(DEV), slots, dbank=dbank, accumulate=add)
            assert torch.equal(got.double().cpu(), want + 2 if add else want)


@pytest.mark.parametrize("add", [False, True], ids=["write", "add"])
@pytest.mark.parametrize("hd,bank", [(64, torch.float32), (128, torch.float32), (256, torch.float32), (1000, torch.float32),
                                     (129, torch.float32), (128, torch.bfloat16), (512, torch.bfloat16)])
def test_columns_in_slices(hd, bank, add):
    """dout larger than an L2 cache: a row's columns on two, four and eight XCDs."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T, W, slots = (8 << 20) // hd // 2, 8, 3000
    idx = torch.randint(0, slots, (2, T, W), generator=g, device=DEV)
    idx[0, ::5] = 7
    w = torch.randint(-1, 2, (2, T, W), generator=g, device=DEV).float()
    dout = torch.randint(-1, 2, (2, T, hd), generator=g, device=DEV).float()
    dbank = torch.ones((slots, hd), dtype=bank, device=DEV)
    got = sdm.sdm_gather_bank_grad(idx[0], w[0], dout[0], slots, chunk=T, valid=T - 3, idx1=idx[1], w1=w[1], dout1=dout[1],
                                   dbank=dbank, accumulate=add)
    want = torch.full((slots, hd), float(add), dtype=torch.float64, device=DEV)
    for o in range(2):
        for c in range(W):
            want.index_add_(0, idx[o, :T - 3, c], (w[o, :T - 3, c, None] * dout[o, :T - 3]).double())
    assert torch.equal(got.double(), want.to(bank).double())


@pytest.mark.parametrize("out", BOTH, ids=["dout-f32", "dout-bf16"])
@pytest.mark.parametrize("hd", [5, 8, 64, 136])
@pytest.mark.parametrize("p", [0.1, 0.5])
def test_dropout(p, hd, out):
    """The lookup's own mask: with p = 1/2 the factor is 2 and everything exact."""
    lookup_case(400, 30, hd, "skewed", out=out, p=p, seed=3, exactly=p == 0.5)
    lookup_case(400, 30, hd, "even", out=out, p=p, seed=4, exactly=p == 0.5, bank=torch.bfloat16, add=True)


def test_dropped_columns_and_rows_outside_are_not_counted_whatever_they_hold():
    rng = torch.tensor([3, 4])
    mask = torch.from_numpy(ref.kept(50, 32, 0.5, rng.tolist()))
    dout = torch.where(mask, 1.0, NAN)
    idx = torch.arange(50) % 5
    idx[7], dout[7] = -1, INF
    idx[8], dout[8] = 5, NAN
    got = sdm.sdm_lookup_grad(idx.to(DEV), dout.to(DEV), 5, dropout=0.5, rng=rng.to(DEV)).cpu()
    want = torch.zeros((5, 32)).index_add_(0, idx.clamp(0, 4), torch.where(mask & (idx % 5 == idx)[:, None], 2.0, 0.0))
    assert torch.equal(got, want)
    bad = dout.clone()
    bad[11] = NAN  # of slot 1
    got = sdm.sdm_lookup_grad(idx.to(DEV), bad.to(DEV), 5, dropout=0.5, rng=rng.to(DEV)).cpu()
    assert torch.isnan(got[1]).any() and torch.equal(got[[0, 2, 3, 4]], want[[0, 2, 3, 4]])


@pytest.mark.parametrize("bank", BOTH, ids=["f32", "bf16"])
@pytest.mark.parametrize("slots", [40, 4000])  # fewer rows than entries, and more
def test_rows_that_no_entry_names_are_plus_zero(slots, bank):
    """Also where the factor is negative, or the largest that float32 holds."""
    idx = (torch.arange(300) % 20).to(DEV)
    for scale in (-1.0, 3e38, -3e38):
        for hd in (16, 33):
            dout = torch.zeros((300, hd), device=DEV)
            got = sdm.sdm_lookup_grad(idx, dout, slots, scale=scale, bank_dtype=bank)
            assert not got.any() and not torch.signbit(got[20:]).any()


@pytest.mark.parametrize("n", [0, 3])
def test_nothing_to_add(n):
    idx, dout = torch.full((n,), -1, device=DEV), torch.ones((n, 9), device=DEV)
    got = sdm.sdm_lookup_grad(idx, dout, 70000)
    assert got.shape == (70000, 9) and not got.any()
    kept = torch.full((70000, 9), 4.0, device=DEV)
    assert (sdm.sdm_lookup_grad(idx, dout, 70000, dbank=kept, accumulate=True) == 4).all()


def test_a_lookup_and_its_gradient_are_adjoint():
    """<lookup(B), D> = <B, lookup_grad(D)> for B and D of small whole numbers, through the same mask."""
    B, D = whole((60, 48), 1), whole((4, 70, 48), 2)
    idx = slots_like("skewed", 280, 60, 3).view(4, 70)
    rng = torch.tensor([9, 10], device=DEV)
    y = sdm.sdm_lookup(B.to(DEV), idx.to(DEV), scale=4.0, dropout=0.5, rng=rng)
    d = sdm.sdm_lookup_grad(idx.to(DEV), D.to(DEV), 60, scale=4.0, dropout=0.5, rng=rng)
    assert y.shape == (4, 70, 48) and (y.double().cpu() * D).sum().item() == (d.double().cpu() * B).sum().item() != 0


def gather_case(tokens, chunk, W0, W1, slots, hd, kind, *, valid=None, cv=None, bank=torch.float32, w=torch.float32,
                index=torch.int64, add=False, exactly=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    alive = ref.live(tokens, chunk, valid, None if cv is None else cv.numpy())
    want, size, count = 0, 0, 0
    args = []
    for o, W in enumerate((W0, W1)):
        if W == 0:
            continue
        idx = slots_like(kind, tokens * W, slots, seed + o).view(tokens, W)
        weights = (whole((tokens, W), seed + 2 + o) if exactly else torch.randn((tokens, W), generator=g)).to(w)
        dout = whole((tokens, hd), seed + 4 + o) if exactly else torch.randn((tokens, hd), generator=g)
        idx[~alive], weights[~alive], dout[~alive] = 1 << 20, NAN, NAN  # padding: not read
        flat, flat_w = np.where(alive[:, None], idx.numpy(), -1).ravel(), weights.double().numpy().ravel()
        r, s, c = ref.bank_grad(slots, flat, lambda e: flat_w[e][:, None] * dout.double().numpy()[e // W], hd)
        want, size, count = want + r, size + s, count + c
        args.append((idx.to(index).to(DEV), weights.to(DEV), dout.to(DEV)))
    second = dict(idx1=args[1][0], w1=args[1][1], dout1=args[1][2]) if W1 else {}
    old = whole((slots, hd), 5, 100).to(bank)
    dbank = old.clone().to(DEV) if add else None
    got = sdm.sdm_gather_bank_grad(*args[0], slots, chunk=chunk, valid=valid, chunk_valid=None if cv is None else cv.to(DEV),
                                   bank_dtype=bank, dbank=dbank, accumulate=add, **second)
    check(got, want, size, count, old.double().numpy() if add else None, exactly)


@pytest.mark.parametrize("kind", ["even", "skewed", "one", "runs"])
@pytest.mark.parametrize("W0,W1", [(1, 0), (3, 0), (1, 1), (8, 5), (64, 64), (256, 1)])
def test_gather_widths(W0, W1, kind):
    gather_case(60, 12, W0, W1, 500, 40, kind, valid=7)
    gather_case(60, 60, W0, W1, 500, 128, kind, index=torch.int32, w=torch.bfloat16, add=True)


@pytest.mark.parametrize("bank", BOTH, ids=["f32", "bf16"])
@pytest.mark.parametrize("w", BOTH, ids=["w-f32", "w-bf16"])
@pytest.mark.parametrize("hd", [1, 7, 64, 100, 128, 520])
def test_gather_types(hd, w, bank):
    cv = torch.tensor([0, 10, 3, 9, 1], dtype=torch.int32)
    gather_case(50, 10, 16, 9, 77, hd, "even", cv=cv, bank=bank, w=w)
    gather_case(50, 10, 16, 9, 77, hd, "skewed", cv=cv, bank=bank, w=w, add=True, exactly=False, index=torch.int32)


def test_gather_of_nothing_but_padding():
    gather_case(40, 8, 5, 2, 30, 16, "even", valid=0)
    gather_case(40, 8, 5, 2, 30, 16, "even", valid=0, add=True)


def test_a_gather_and_its_gradient_are_adjoint():
    B, D0, D1 = whole((90, 64), 1), whole((32, 64), 2), whole((32, 64), 3)
    idx, w = torch.randint(0, 90, (32, 12), device=DEV), whole((32, 12), 4).to(DEV)
    cv = torch.tensor([8, 0, 5, 2], dtype=torch.int32, device=DEV)
    out0, _, out1 = sdm.sdm_gather(B.to(DEV), idx, w, chunk=8, chunk_valid=cv, idx1=idx, w1=2 * w, with_stash=False)
    d = sdm.sdm_gather_bank_grad(idx, w, D0.to(DEV), 90, chunk=8, chunk_valid=cv, idx1=idx, w1=2 * w, dout1=D1.to(DEV))
    lhs = (out0.double().cpu() * D0).sum() + (out1.double().cpu() * D1).sum()
    assert lhs.item() == (d.double().cpu() * B).sum().item() != 0


def test_the_gradient_by_differences():
    """Of sum (out - target)^2 / 2 in float64 through the gather's definition."""
    g = torch.Generator().manual_seed(1)
    B, w, y = torch.randn((20, 8), generator=g), torch.randn((16, 4), generator=g), torch.randn((16, 8), generator=g)
    idx = torch.randint(0, 20, (16, 4), generator=g)

    def loss(bank):
        return ((((bank[idx].double() * w.double()[..., None]).sum(1)) - y) ** 2).sum().item() / 2

    out, _, _ = sdm.sdm_gather(B.to(DEV), idx.to(DEV), w.to(DEV), chunk=16, with_stash=False)
    d = sdm.sdm_gather_bank_grad(idx.to(DEV), w.to(DEV), out - y.to(DEV), 20, chunk=16).cpu()
    B = B.double()
    for s, c in ((0, 0), (7, 3), (19, 7)):
        up, down = B.clone(), B.clone()
        up[s, c] += 1e-4
        down[s, c] -= 1e-4
        # a quadratic: its central difference is exact but for roundings, 2^-52 of a loss of some hundreds over 1e-4
        assert d[s, c].item() == pytest.approx((loss(up) - loss(down)) / 2e-4, abs=1e-4)


@pytest.mark.parametrize("off", [1, 2, 4])
def test_any_alignment(off):
    n, hd, slots = 200, 64, 20
    idx = slots_like("skewed", n, slots, 1)
    for out in BOTH:
        for bank in BOTH:
            flat = whole((n * hd + off,), 2).to(out).to(DEV)
            dbank = torch.full((slots * hd + off + 1,), 9.0, dtype=bank, device=DEV)
            got = sdm.sdm_lookup_grad(idx.to(DEV), flat[off:].view(n, hd), slots, dbank=dbank[off:-1].view(slots, hd))
            want = torch.zeros((slots, hd)).index_add_(0, idx, flat[off:].view(n, hd).float().cpu())
            assert torch.equal(got.float().cpu(), want.to(bank).float())
            assert (dbank[:off] == 9).all() and dbank[-1].item() == 9


@pytest.mark.parametrize("kind", ["skewed", "one"])
def test_the_same_inputs_give_the_same_bits(kind):
    n, slots, hd = 100000, 1000, 72
    idx = slots_like(kind, n, slots, 1).to(DEV)
    dout = torch.randn((n, hd), device=DEV)
    first = sdm.sdm_lookup_grad(idx, dout, slots)
    size = sdm.library().sdm_bank_grad_workspace(n, slots, hd)
    for fill in (0, 0xff, 0x7f):
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(sdm.sdm_lookup_grad(idx, dout, slots, workspace=ws), first)
    count = torch.bincount(idx, minlength=slots).cpu().numpy()
    want, size = np.zeros((slots, hd)), np.zeros((slots, hd))
    d = dout.double().cpu().numpy()
    np.add.at(want, idx.cpu().numpy(), d)
    np.add.at(size, idx.cpu().numpy(), np.abs(d))
    check(first, want, size, count, None, False)
    with pytest.raises(sdm.SdmError, match="bytes"):
        sdm.sdm_lookup_grad(idx, dout, slots, workspace=ws[:1024])


@pytest.mark.parametrize("add", [False, True], ids=["write", "add"])
@pytest.mark.parametrize("hd", [40, 128, 129])
@pytest.mark.parametrize("terms", ["alike", "any"])
def test_long_sums_lose_no_more_than_short_ones(terms, hd, add):
    """2^20 terms of one slot, and some of others. Alike: each term's lowest bits are less than half a step of a sum of 512
    blocks of 32, so that a float32 sum of those would lose them every time."""
    T, W, slots = 4096, 256, 50
    g = torch.Generator(device=DEV).manual_seed(1)
    idx = torch.where(torch.rand((T, W), generator=g, device=DEV) < 0.01, torch.randint(0, slots, (T, W), generator=g, device=DEV), 7)
    w = torch.full((T, W), 1 + 1.5 * 2.0 ** -16, device=DEV) if terms == "alike" else torch.rand((T, W), generator=g, device=DEV)
    dout = torch.ones((T, hd), device=DEV) if terms == "alike" else torch.rand((T, hd), generator=g, device=DEV)
    got = sdm.sdm_gather_bank_grad(idx, w, dout, slots, chunk=T, dbank=torch.zeros((slots, hd), device=DEV), accumulate=add)
    matrix = torch.zeros((slots, T), dtype=torch.float64, device=DEV)
    matrix.index_put_((idx.flatten(), torch.arange(T, device=DEV).repeat_interleave(W)), w.flatten().double(), accumulate=True)
    want = matrix @ dout.double()
    # at most 48 roundings of a block's terms and 16 of up to 17 blocks, or one of more of them; one of the sum with what
    # was there; terms are positive
    assert ((got.double() - want).abs() <= (48 + 16 + 1) * 2.0 ** -24 * want).all()
    long = (got.double() - want)[7].abs() / want[7]
    assert (long <= (48 + 1 + 1) * 2.0 ** -24).all()


@pytest.mark.slow
def test_a_bank_past_32_bit_offsets():
    slots, hd = (1 << 25) + 5, 136  # 4.56e9 values
    idx = torch.tensor([slots - 1, 0, slots - 1, 1 << 24, slots - 2])
    dout = torch.arange(1, 6, dtype=torch.float32)[:, None].expand(5, hd).contiguous()
    got = sdm.sdm_lookup_grad(idx.to(DEV), dout.to(DEV), slots, bank_dtype=torch.bfloat16)
    assert got[[slots - 1, 0, 1 << 24, slots - 2]][:, 135].tolist() == [4, 2, 4, 5]
    assert (got != 0).any(1).sum().item() == 4


@pytest.mark.slow
def test_the_widest_rows():
    """As many slices of the columns as the last pass's grid holds, and a run over several blocks of entries."""
    hd, n = 65535 * 256, 40
    idx = torch.ones(n, dtype=torch.int64, device=DEV)
    idx[7] = 0
    dout = (torch.arange(hd, device=DEV) % 5 - 2).to(torch.bfloat16).expand(n, hd).contiguous()
    got = sdm.sdm_lookup_grad(idx, dout, 3)
    assert torch.equal(got[0], dout[0].float()) and torch.equal(got[1], 39 * dout[0].float()) and not got[2].any()
    add = sdm.sdm_lookup_grad(idx, dout, 3, dbank=got.clone(), accumulate=True)
    assert torch.equal(add, 2 * got)
    with pytest.raises(sdm.SdmError, match="head_dim must be at most"):
        sdm.sdm_lookup_grad(idx[:1], torch.zeros((1, hd + 1), device=DEV), 1)


@pytest.mark.slow
def test_many_entries():
    """Several hundred tiles of the sort, both kinds of slots, and a run over thousands of blocks."""
    g = torch.Generator(device=DEV).manual_seed(1)
    T, W, slots = 40000, 64, 1 << 20
    idx = torch.randint(0, slots, (T, W), generator=g, device=DEV)
    idx[::3] = 12345
    w = torch.randint(0, 3, (T, W), generator=g, device=DEV).float()
    dout = torch.randint(-2, 3, (T, 16), generator=g, device=DEV).float()
    got = sdm.sdm_gather_bank_grad(idx, w, dout, slots, chunk=40)
    want = torch.zeros((slots, 16), dtype=torch.float64, device=DEV)
    want.index_add_(0, idx.flatten(), (w[..., None] * dout[:, None]).view(-1, 16).double())
    assert torch.equal(got.double(), want)


@pytest.mark.slow
@pytest.mark.parametrize("hd", [4160, 4163])
@pytest.mark.parametrize("kind", ["even", "skewed", "one"])
def test_columns_in_turns(hd, kind):
    """2^20 entries of so many columns that the sums of blocks are made for 4096 of them at a time."""
    T, W, slots = 4096, 256, 64
    idx = slots_like(kind, T * W, slots, 1).view(T, W).to(DEV)
    w = whole((T, W), 2, 1).to(DEV)
    dout = whole((T, hd), 3, 1).to(DEV)
    assert sdm.library().sdm_bank_grad_workspace(T * W, slots, hd) < 27 * T * W + (1 << 30) + (1 << 20) < 24 * T * W + T * W // 4 * hd
    matrix = torch.zeros((slots, T), dtype=torch.float64, device=DEV)
    matrix.index_put_((idx.flatten(), torch.arange(T, device=DEV).repeat_interleave(W)), w.flatten().double(), accumulate=True)
    want = matrix @ dout.double()  # whole numbers below 2^21
    got = sdm.sdm_gather_bank_grad(idx, w, dout, slots, chunk=T)
    assert torch.equal(got.double(), want)
    got = sdm.sdm_gather_bank_grad(idx, w, dout, slots, chunk=T, dbank=got, accumulate=True)
    assert torch.equal(got.double(), 2 * want)
    large = sdm.sdm_gather_bank_grad(idx + 7, w, dout, T * W + 9, chunk=T, bank_dtype=torch.bfloat16)  # zeroed beside the sort
    assert torch.equal(large[7:71], want.to(torch.bfloat16)) and not large[:7].any() and not large[71:].any()
    del large
    torch.cuda.empty_cache()


@pytest.mark.slow
def test_dropout_in_turns():
    n, slots, hd = 1 << 20, 33, 4160
    idx = slots_like("skewed", n, slots, 1).to(DEV)
    rng = torch.tensor([11, 12], device=DEV)
    dout = torch.randint(-1, 2, (n, hd), device=DEV, dtype=torch.int8, generator=torch.Generator(device=DEV).manual_seed(1)).to(torch.bfloat16)
    got = sdm.sdm_lookup_grad(idx, dout, slots, dropout=0.5, rng=rng)
    mask = sdm.sdm_lookup(torch.ones((slots, hd), device=DEV, dtype=torch.bfloat16), idx, dropout=0.5, rng=rng)  # 0 or 2
    want = torch.zeros((slots, hd), device=DEV, dtype=torch.float64)
    for a in range(0, n, 1 << 17):
        at = slice(a, a + (1 << 17))
        one_hot = torch.zeros((slots, 1 << 17), dtype=torch.float32, device=DEV)
        one_hot[idx[at], torch.arange(1 << 17, device=DEV)] = 1
        want += (one_hot @ (mask[at] * dout[at]).float()).double()  # whole numbers, of less than 2^18
    assert torch.equal(got.double(), want)
    del dout, mask
    torch.cuda.empty_cache()


def test_refusals():
    idx, dout = torch.zeros(3, dtype=torch.int64, device=DEV), torch.ones((3, 8), device=DEV)
    with pytest.raises(ValueError, match="dbank to add to"):
        sdm.sdm_lookup_grad(idx, dout, 4, accumulate=True)
    with pytest.raises(ValueError, match="dbank must be"):
        sdm.sdm_lookup_grad(idx, dout, 4, dbank=torch.empty((5, 8), device=DEV))
    with pytest.raises(TypeError, match="bank_dtype"):
        sdm.sdm_lookup_grad(idx, dout, 4, bank_dtype=torch.float16)
    with pytest.raises(sdm.SdmError, match="empty bank"):
        sdm.sdm_lookup_grad(idx, dout, 0)
    with pytest.raises(ValueError, match="w0 must be"):
        sdm.sdm_gather_bank_grad(idx[:, None], torch.ones((3, 2), device=DEV), dout, 4, chunk=3)
