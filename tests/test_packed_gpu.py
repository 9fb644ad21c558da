"""Packed banks: sdm_bank_pack bit for bit against the plain implementation of
tests/memory_ref.py, sdm_gather_packed bit for bit against sdm_gather on the
values, sdm_gather_weight_grad within what its roundings allow."""

import copy
import pickle

import numpy as np
import pytest
import torch

import memory_ref as ref
from helpers import gamma
from sparse_delta_rule_amd import PackedBank, sdm_bank_pack, sdm_gather, sdm_gather_packed, sdm_gather_weight_grad

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = float("inf"), float("nan")
KINDS = ["mx8", "mx4"]


def rows_like(n, hd, seed, dtype=torch.float32, spread=12):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, hd), generator=g) * 0.02
    if spread:  # blocks of very different sizes, some of zeros
        e = torch.randint(-spread, spread + 1, (n, -(-hd // 32)), generator=g).float()
        x = x * torch.exp2(e).repeat_interleave(32, 1)[:, :hd]
        x[torch.rand(x.shape, generator=g) < 0.05] = 0.0
        x[torch.rand(x.shape, generator=g) < 0.05] *= -0.0
    return x.to(dtype)


def same(bank: PackedBank, rows: torch.Tensor, slots=None):
    codes, scales = ref.pack(rows.float().numpy(), bank.kind)
    at = slice(None) if slots is None else slots
    assert np.array_equal(bank.scales.cpu().numpy()[at], scales)
    assert np.array_equal(bank.codes.cpu().numpy()[at], codes)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("hd", [1, 2, 7, 8, 15, 16, 31, 32, 33, 63, 64, 65, 96, 100, 101, 127, 128, 130, 200, 256, 500, 1000,
                                2047, 2048, 2080, 5000])
def test_pack_sizes(hd, dtype, kind):
    rows = rows_like(37, hd, hd, dtype)
    bank = PackedBank.empty(37, hd, kind, DEV)
    bank.codes.fill_(0xa5)
    bank.scales.fill_(0xa5)
    assert sdm_bank_pack(bank, rows.to(DEV)) is bank
    same(bank, rows)


@pytest.mark.parametrize("kind", KINDS)
def test_pack_every_code_border_and_tie(kind):
    """Every midpoint between two codes, and its float32 neighbours, at small, ordinary and large scales."""
    table = np.array(ref.E4M3 if kind == "mx8" else ref.E2M1)
    mid = (table[1:] + table[:-1]) / 2
    x = np.concatenate([table, mid]).astype(np.float32)
    x = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(1e9))])
    x = np.concatenate([x, -x])
    most = table[-1]
    x = x[np.abs(x) <= most]
    x = np.pad(x, (0, -len(x) % 31)).reshape(-1, 31)
    x = np.concatenate([np.full((len(x), 1), most, np.float32), x], 1)  # pins the block's scale
    x = np.concatenate([np.ldexp(x, e).astype(np.float32) for e in (-127, -126, -120, -60, -1, 0, 1, 60, 118, 119)])
    bank = PackedBank.empty(len(x), 32, kind, DEV)
    sdm_bank_pack(bank, torch.from_numpy(x).to(DEV))
    same(bank, torch.from_numpy(x))


@pytest.mark.parametrize("kind", KINDS)
def test_pack_scale_borders_and_extremes(kind):
    """Blocks whose largest magnitude lies at, above and below a scale's border, denormal and near the largest float32."""
    most = np.float32(448 if kind == "mx8" else 6)
    tops = []
    for e in (-149, -140, -137, -136, -135, -130, -129, -128, -127, -126, -100, -9, 0, 9, 100, 118, 119, 120):
        with np.errstate(over="ignore"):
            a = np.float32(np.ldexp(np.float64(most), e))
        tops += [a, np.nextafter(a, np.float32(0)), np.nextafter(a, np.float32(3e38))]
    tops += [np.float32(3.4028235e38), np.float32(1e-45), np.float32(0)]
    tops = np.array([t for t in tops if np.isfinite(t)], np.float32)
    x = tops[:, None] * np.linspace(-1, 1, 33, dtype=np.float32)[None]
    bank = PackedBank.empty(len(x), 33, kind, DEV)
    sdm_bank_pack(bank, torch.from_numpy(x).to(DEV))
    same(bank, torch.from_numpy(x))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_pack_what_is_not_finite(kind, dtype):
    x = rows_like(64, 100, 5, dtype)
    g = torch.Generator().manual_seed(1)
    for v in (NAN, INF, -INF):
        x[torch.rand(x.shape, generator=g) < 0.01] = v
    x[0] = INF
    x[1, 5] = NAN
    bank = PackedBank.empty(64, 100, kind, DEV)
    sdm_bank_pack(bank, x.to(DEV))
    same(bank, x)
    # and it reads back as not-a-number, the rest as packed
    back, _ = sdm_gather_packed(bank, torch.arange(64, device=DEV)[:, None], torch.ones((64, 1), device=DEV), chunk=1)
    want = ref.unpack(*ref.pack(x.float().numpy(), kind), 100, kind)
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("kind", KINDS)
def test_pack_to_slots_and_from_rows(kind, index):
    n, slots, hd = 300, 1000, 100
    rows = rows_like(n, hd, 1)
    g = torch.Generator().manual_seed(2)
    at = torch.randperm(slots, generator=g)[:n]
    at[5], at[77], at[200] = -1, slots, -(1 << 31) if index == torch.int32 else 1 << 40  # store nothing
    named = (at >= 0) & (at < slots)
    bank = PackedBank.empty(slots, hd, kind, DEV)
    bank.codes.fill_(7)
    bank.scales.fill_(9)
    sdm_bank_pack(bank, rows.to(DEV), slots=at.to(index).to(DEV))
    same(bank, rows[named], at[named].numpy())
    left = np.setdiff1d(np.arange(slots), at[named].numpy())
    assert (bank.codes.cpu().numpy()[left] == 7).all() and (bank.scales.cpu().numpy()[left] == 9).all()
    # rows of a bank brought up to date in its packed copy, some of them named many times
    src = torch.randint(0, n, (2000,), generator=g)
    src[3], src[9] = -5, n
    copy = PackedBank.empty(n, hd, kind, DEV)
    sdm_bank_pack(copy, rows.to(DEV), row_idx=src.to(index).to(DEV), slots=src.to(index).to(DEV))
    done = np.unique(src[(src >= 0) & (src < n)].numpy())
    same(copy, rows[done], done)
    # row_idx alone: consecutive slots
    some = PackedBank.empty(50, hd, kind, DEV)
    sdm_bank_pack(some, rows.to(DEV), row_idx=src[100:150].to(index).to(DEV))
    same(some, rows[src[100:150]])


@pytest.mark.parametrize("dtype,off", [(torch.float32, 1), (torch.float32, 2), (torch.bfloat16, 1), (torch.bfloat16, 2),
                                       (torch.bfloat16, 4)])
def test_pack_rows_at_any_alignment(dtype, off):
    flat = rows_like(1, 20 * 128 + off, 3, dtype, spread=0)[0]
    bank = PackedBank.empty(20, 128, "mx8", DEV)
    sdm_bank_pack(bank, flat.to(DEV)[off:].view(20, 128))
    same(bank, flat[off:].view(20, 128))


def test_pack_many_rows():
    """A grid's loop over rows: more rows than one pass of the largest grid would hold at one a workgroup."""
    n, hd = 1 << 20, 2064
    rows = torch.zeros((1, hd), device=DEV)
    rows[0, 5], rows[0, -1] = 3.0, -448.0
    idx = torch.zeros(n + 3, dtype=torch.int32, device=DEV)
    at = torch.arange(n + 3, dtype=torch.int32, device=DEV) % 4096
    at[-1] = 4100
    bank = PackedBank.empty(4101, hd, "mx8", DEV)
    sdm_bank_pack(bank, rows, row_idx=idx, slots=at)
    want, scale = ref.pack(rows.cpu().numpy(), "mx8")
    for s in (0, 1, 4095, 4100):
        assert np.array_equal(bank.codes[s].cpu().numpy(), want[0]) and np.array_equal(bank.scales[s].cpu().numpy(), scale[0])
    assert not bank.codes[4096:4100].any()


def test_pack_of_nothing():
    bank = PackedBank.empty(4, 16, "mx8", DEV)
    sdm_bank_pack(bank, torch.zeros((0, 16), device=DEV))
    sdm_bank_pack(bank, torch.ones((2, 16), device=DEV), slots=torch.zeros(0, dtype=torch.int32, device=DEV))
    assert not bank.codes.any()


# ------------------------------------------------------------------ gather


def packed(n, hd, kind, seed, spread=6):
    rows = rows_like(n, hd, seed, spread=spread)
    bank = PackedBank.empty(n, hd, kind, DEV)
    sdm_bank_pack(bank, rows.to(DEV))
    codes, scales = ref.pack(rows.numpy(), kind)
    return bank, torch.from_numpy(ref.unpack(codes, scales, hd, kind)).float().to(DEV)


def draws(seed, T, width, n, index, w_dtype):
    g = torch.Generator().manual_seed(seed)
    return (torch.randint(0, n, (T, width), generator=g).to(index).to(DEV),
            torch.randn((T, width), generator=g).to(w_dtype).to(DEV))


def bits(t):
    return t.contiguous().view(torch.int32)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hd", [1, 3, 4, 16, 17, 32, 40, 64, 100, 101, 127, 128, 129, 256, 400, 1000, 1024, 1025, 2500])
def test_gather_head_dims(hd, kind):
    bank, values = packed(300, hd, kind, hd)
    for T, W0, W1 in ((6, 5, 0), (24, 64, 9), (40, 1, 256)):
        i0, w0 = draws(1, T, W0, 300, torch.int32, torch.float32)
        kw = {}
        if W1:
            i1, w1 = draws(2, T, W1, 300, torch.int32, torch.float32)
            kw = dict(idx1=i1, w1=w1)
        out0, out1 = sdm_gather_packed(bank, i0, w0, chunk=T, **kw)
        want0, _, want1 = sdm_gather(values, i0, w0, chunk=T, with_stash=False, **kw)
        assert torch.equal(bits(out0), bits(want0))
        assert out1 is None if not W1 else torch.equal(bits(out1), bits(want1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("index,w_dtype", [(torch.int32, torch.bfloat16), (torch.int64, torch.float32)])
@pytest.mark.parametrize("T,chunk,W0,W1", [(1, 1, 1, 1), (64, 64, 64, 64), (60, 20, 7, 0), (300, 3, 33, 8), (4096, 64, 64, 64),
                                           (5000, 50, 12, 255), (33000, 11, 3, 5)])
def test_gather_tokens_and_padding(T, chunk, W0, W1, index, w_dtype, kind):
    hd = 128 if T % 3 else 100
    bank, values = packed(2000, hd, kind, T)
    g = torch.Generator().manual_seed(T)
    counts = torch.randint(0, chunk + 1, (T // chunk,), generator=g).to(torch.int32)
    alive = torch.from_numpy(ref.live(T, chunk, chunk_valid=counts.numpy())).to(DEV)
    i0, w0 = draws(1, T, W0, 2000, index, w_dtype)
    i0[~alive], w0[~alive] = -1, NAN  # padding is not read
    kw = dict(chunk=chunk)
    if W1:
        i1, w1 = draws(2, T, W1, 2000, index, w_dtype)
        i1[~alive] = 1 << 30
        kw.update(idx1=i1, w1=w1)
    for padding in (dict(chunk_valid=counts.to(DEV)), dict(valid=0)):
        got = sdm_gather_packed(bank, i0, w0, **kw, **padding)
        want = sdm_gather(values, i0, w0, with_stash=False, **kw, **padding)
        assert torch.equal(bits(got[0]), bits(want[0]))
        if W1:
            assert torch.equal(bits(got[1]), bits(want[2]))


def test_gather_into_outputs_at_any_alignment():
    for hd in (64, 50, 33):
        bank, values = packed(64, hd, "mx8", 3)
        i0, w0 = draws(1, 8, 20, 64, torch.int64, torch.float32)
        want = sdm_gather(values, i0, w0, chunk=8, with_stash=False)[0]
        for off in (1, 2, 4):
            flat = torch.full((8 * hd + off + 4,), 5.0, device=DEV)
            out = flat[off:off + 8 * hd].view(8, hd)
            assert sdm_gather_packed(bank, i0, w0, chunk=8, out0=out)[0] is out
            assert torch.equal(bits(out), bits(want))
            assert (flat[:off] == 5).all() and (flat[off + 8 * hd:] == 5).all()


def test_gather_weights_that_are_not_finite():
    bank, values = packed(50, 64, "mx8", 3)
    i0, w0 = draws(1, 8, 20, 50, torch.int64, torch.float32)
    w0[0, 3], w0[1, 0], w0[2, 19], w0[3] = INF, -INF, NAN, 3e38
    got = sdm_gather_packed(bank, i0, w0, chunk=8)[0]
    want = sdm_gather(values, i0, w0, chunk=8, with_stash=False)[0]
    assert torch.equal(torch.nan_to_num(got, nan=1.5), torch.nan_to_num(want, nan=1.5))


def test_gather_past_32_bits():
    """A packed bank of more than 2^32 bytes."""
    n, hd = (1 << 32) // 256 + 4096, 256
    bank = PackedBank.empty(n, hd, "mx8", DEV)
    rows = rows_like(8, hd, 1)
    at = torch.tensor([0, 1, n // 2, (1 << 31) // 256, (1 << 32) // 256 - 1, (1 << 32) // 256, n - 2, n - 1])
    sdm_bank_pack(bank, rows.to(DEV), slots=at.to(DEV))
    values = torch.from_numpy(ref.unpack(*ref.pack(rows.numpy(), "mx8"), hd, "mx8")).float().to(DEV)
    back = sdm_gather_packed(bank, at.to(DEV)[:, None], torch.ones((8, 1), device=DEV), chunk=8)[0]
    assert torch.equal(back, values)
    dout = torch.randn((1, hd), device=DEV)
    dw = sdm_gather_weight_grad(bank, at.to(DEV)[None], dout, chunk=1)[0]
    assert torch.equal(dw, sdm_gather_weight_grad(PackedBank(bank.codes[at.to(DEV)], bank.scales[at.to(DEV)], hd), torch.arange(
        8, device=DEV)[None], dout, chunk=1)[0])


# ------------------------------------------------------------------ weight gradient


def banks(kind, n, hd, seed):
    """(a bank of the kind, its values in float64 on the host)."""
    if kind in KINDS:
        bank, values = packed(n, hd, kind, seed)
        return bank, values.double().cpu().numpy()
    rows = rows_like(n, hd, seed, torch.bfloat16 if kind == "bf16" else torch.float32)
    return rows.to(DEV), rows.double().numpy()


def check_weight_grad(bank, values, i, dout, alive, got):
    want, size = ref.weight_grad(values, i.cpu().numpy(), dout.cpu().numpy(), alive)
    hd = values.shape[1]
    # hd products and sums in float32 in some order, then a rounding to the weights' type
    slack = gamma(hd + 1) * size + 2.0 ** -149
    if got.dtype == torch.bfloat16:
        slack = slack * 1.01 + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got.double().cpu().numpy() - want) <= slack).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"] + KINDS)
@pytest.mark.parametrize("hd", [1, 3, 8, 16, 31, 64, 100, 101, 126, 128, 129, 256, 1000, 1025, 4100])
def test_weight_grad_head_dims(hd, kind):
    bank, values = banks(kind, 100, hd, hd)
    for T, W0, W1 in ((5, 3, 0), (12, 64, 9), (4, 1, 256)):
        i0, _ = draws(1, T, W0, 100, torch.int32, torch.float32)
        i1, _ = draws(2, T, max(W1, 1), 100, torch.int32, torch.float32)
        d0, d1 = torch.randn((T, hd), device=DEV), torch.randn((T, hd), device=DEV)
        kw = dict(idx1=i1, dout1=d1) if W1 else {}
        dw0, dw1 = sdm_gather_weight_grad(bank, i0, d0, chunk=T, **kw)
        alive = np.ones(T, bool)
        check_weight_grad(bank, values, i0, d0, alive, dw0)
        if W1:
            check_weight_grad(bank, values, i1, d1, alive, dw1)
        else:
            assert dw1 is None


@pytest.mark.parametrize("kind", ["f32", "bf16"] + KINDS)
@pytest.mark.parametrize("T,chunk,W0,W1", [(1, 1, 1, 1), (64, 64, 64, 64), (60, 20, 7, 0), (300, 3, 33, 8), (1000, 50, 48, 20)])
def test_weight_grad_padding(T, chunk, W0, W1, kind):
    hd = 128 if T % 3 else 100
    bank, values = banks(kind, 500, hd, T)
    g = torch.Generator().manual_seed(T)
    counts = torch.randint(0, chunk + 1, (T // chunk,), generator=g).to(torch.int32)
    alive = ref.live(T, chunk, chunk_valid=counts.numpy())
    dead = ~torch.from_numpy(alive).to(DEV)
    i0, _ = draws(1, T, W0, 500, torch.int64, torch.float32)
    d0 = torch.randn((T, hd), device=DEV)
    i0[dead], d0[dead] = -1, NAN
    kw = {}
    if W1:
        i1, _ = draws(2, T, W1, 500, torch.int64, torch.float32)
        d1 = torch.randn((T, hd), device=DEV)
        kw = dict(idx1=i1.masked_fill(dead[:, None], 1 << 50), dout1=d1)
    dw0, dw1 = sdm_gather_weight_grad(bank, i0, d0, chunk=chunk, chunk_valid=counts.to(DEV), w_dtype=torch.bfloat16, **kw)
    assert not dw0[dead].any()
    check_weight_grad(bank, values, i0, d0.nan_to_num(), alive, dw0)
    if W1:
        assert not dw1[dead].any()
        check_weight_grad(bank, values, i1, d1, alive, dw1)
    assert not sdm_gather_weight_grad(bank, i0, d0, chunk=chunk, valid=0)[0].any()


def test_weight_grad_against_differences():
    """The slope of <out, dout> in one weight, from sdm_gather_packed itself."""
    bank, values = packed(100, 96, "mx8", 1, spread=0)
    i0, w0 = draws(1, 6, 10, 100, torch.int64, torch.float32)
    dout = torch.randn((6, 96), device=DEV)
    dw = sdm_gather_weight_grad(bank, i0, dout, chunk=6)[0]
    for n in range(10):
        loss = []
        for h in (0.5, -0.5):
            w = w0.clone()
            w[:, n] += h
            loss.append((sdm_gather_packed(bank, i0, w, chunk=6)[0].double() * dout.double()).sum(1))
        # the loss is linear in the weight: only the roundings of 10 products and of w + h are left
        far = ((w0.double().abs() + 1)[:, :, None] * values.double()[i0].abs() * dout.double().abs()[:, None]).sum((1, 2))
        assert ((loss[0] - loss[1] - dw[:, n].double()).abs() <= 2 * gamma(12) * far).all()


def test_a_bank_keeps_its_arrays():
    """Calls go by the arrays that the bank was made of: another one, or another size, is another bank."""
    packed = PackedBank.empty(16, 128, "mx8", DEV)
    for name, other in (("codes", packed.codes.clone()), ("scales", packed.scales.clone()), ("head_dim", 64),
                        ("num_slots", 32), ("dtype", 5)):
        with pytest.raises(AttributeError, match="cannot be replaced"):
            setattr(packed, name, other)
    assert packed.head_dim == 128 and packed.num_slots == 16 and packed.kind == "mx8" and packed.codes.shape == (16, 128)
    packed.name = "notes"  # a caller's own field goes along
    rows = torch.randn((16, 128), device=DEV)
    sdm_bank_pack(packed, rows)
    for copied in (copy.deepcopy(packed), pickle.loads(pickle.dumps(packed))):
        assert copied._head[:2] == (copied.codes.data_ptr(), copied.scales.data_ptr())
        assert copied.codes.data_ptr() != packed.codes.data_ptr() and copied._head[2:] == packed._head[2:]
        assert torch.equal(copied.codes, packed.codes) and torch.equal(copied.scales, packed.scales)
        assert type(copied) is PackedBank and copied.name == "notes"
        idx, w = torch.arange(16, device=DEV)[:, None], torch.ones((16, 1), device=DEV)
        before = sdm_gather_packed(packed, idx, w, chunk=1)[0]
        sdm_bank_pack(copied, rows * 2)  # and leaves the first one as it is
        assert torch.equal(sdm_gather_packed(packed, idx, w, chunk=1)[0], before)
        assert torch.equal(sdm_gather_packed(copied, idx, w, chunk=1)[0], 2 * before)


@pytest.mark.parametrize("kind", KINDS)
def test_every_code_with_every_scale(kind):
    """A bank's bytes may be the caller's own: each code's value times each scale, as float32, past its
    range infinite, and the scale 255 not-a-number."""
    lines = np.zeros((256, 256), np.uint8)
    lines[:] = np.arange(256)  # mx8: each code; mx4: each pair of codes
    hd = 256 if kind == "mx8" else 512
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], ref.scale_bytes(hd), 1)
    bank = PackedBank(torch.from_numpy(lines).to(DEV), torch.from_numpy(scales).to(DEV), hd, kind)
    with np.errstate(over="ignore", invalid="ignore"):
        want = ref.unpack(lines, scales, hd, kind).astype(np.float32)
    every = torch.arange(256, device=DEV)[:, None]
    for n in (256, 256 * 40):  # few and many columns a lane
        back, _ = sdm_gather_packed(bank, every.repeat(n // 256, 1), torch.ones((n, 1), device=DEV), chunk=n)
        assert np.array_equal(back[-256:].cpu().numpy(), want, equal_nan=True)
    # rows of four blocks, whose scales come with the entry
    short = PackedBank(torch.from_numpy(lines[:, 96:160] if kind == "mx4" else lines[:, 64:192]).contiguous().to(DEV),
                       torch.from_numpy(scales[:, :4]).contiguous().to(DEV), 128, kind)
    part = want[:, 192:320] if kind == "mx4" else want[:, 64:192]
    for n in (256, 256 * 400):
        back, _ = sdm_gather_packed(short, every.repeat(n // 256, 1), torch.ones((n, 1), device=DEV), chunk=n)
        assert np.array_equal(back[-256:].cpu().numpy(), part, equal_nan=True)
