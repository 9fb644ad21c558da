"""sdm_lookup bit for bit against the plain implementation of tests/train_ref.py."""

import numpy as np
import pytest
import torch

import memory_ref
import train_ref as ref
import sparse_delta_rule_amd as sdm

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
INF, NAN = float("inf"), float("nan")


def rng_of(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64)


def same(got, want, dtype):
    """Bit for bit but for a NaN's payload."""
    want = torch.from_numpy(want).to(dtype)
    assert got.dtype == dtype and torch.equal(torch.isnan(got.cpu()), torch.isnan(want))
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    a, b = torch.nan_to_num(got.cpu(), nan=0.0, posinf=INF, neginf=-INF), torch.nan_to_num(want, nan=0.0, posinf=INF, neginf=-INF)
    assert torch.equal(a.view(bits) * (a != 0), b.view(bits) * (b != 0))  # a zero of either sign


def bank_of(kind, slots, hd, seed):
    """A bank as the call takes it, and its float32 values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((slots, hd), generator=g) * 0.3
    if kind in ("f32", "bf16"):
        t = x.to(torch.float32 if kind == "f32" else torch.bfloat16)
        return t.to(DEV), t.float().numpy()
    p = sdm.sdm_bank_pack(sdm.PackedBank.empty(slots, hd, kind, DEV), x.to(DEV))
    return p, memory_ref.unpack(p.codes.cpu().numpy(), p.scales.cpu().numpy(), hd, kind).astype(np.float32)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["f32", "bf16", "mx8", "mx4"])
@pytest.mark.parametrize("hd", [1, 3, 4, 7, 8, 9, 16, 31, 33, 64, 100, 101, 128, 136, 520, 1000, 2048, 2056, 5003])
def test_sizes(hd, kind, out):
    bank, values = bank_of(kind, 50, hd, hd)
    g = torch.Generator().manual_seed(1)
    for n, index in ((1, torch.int64), (61, torch.int32)):
        idx = torch.randint(-3, 53, (n,), generator=g).to(index)
        for scale, p in ((1.0, 0.0), (0.7, 0.0), (32.0, 0.3)):
            rng = rng_of(12345678901234567, (1 << 40) + hd)
            mask = ref.kept(n, hd, p, rng.tolist()) if p and hd <= 600 or n == 1 else None
            if p and mask is None:
                continue
            got = sdm.sdm_lookup(bank, idx.to(DEV), scale=scale, dropout=p, rng=rng.to(DEV), out_dtype=out)
            same(got, ref.lookup(values, idx.numpy(), scale, mask, p), out)


def test_many_rows_take_several_a_thread():
    bank, values = bank_of("bf16", 300, 100, 3)
    idx = torch.randint(-1, 301, (200000,), generator=torch.Generator().manual_seed(2))
    same(sdm.sdm_lookup(bank, idx.to(DEV), scale=3.0), ref.lookup(values, idx.numpy(), 3.0), torch.bfloat16)
    bank, values = bank_of("f32", 40, 2056, 3)
    idx = torch.randint(-1, 41, (2050,), generator=torch.Generator().manual_seed(2))
    same(sdm.sdm_lookup(bank, idx.to(DEV)), ref.lookup(values, idx.numpy()), torch.float32)


def test_index_shapes_and_values():
    bank, values = bank_of("f32", 10, 12, 1)
    idx = torch.tensor([[0, 9, 10], [-1, -(1 << 40), 1 << 33]])
    got = sdm.sdm_lookup(bank, idx.to(DEV))
    assert got.shape == (2, 3, 12)
    assert torch.equal(got[0, :2].cpu(), torch.from_numpy(values[[0, 9]])) and not got[0, 2].any() and not got[1].any()
    assert sdm.sdm_lookup(bank, torch.tensor(4, device=DEV)).shape == (12,)
    assert sdm.sdm_lookup(bank, torch.empty((0, 3), dtype=torch.int32, device=DEV)).shape == (0, 3, 12)


def test_dropped_and_missing_columns_are_zero_whatever_the_bank_holds():
    bank = torch.full((4, 64), NAN, device=DEV)
    bank[0] = INF
    rng = rng_of(1, 2)
    idx = torch.tensor([0, 1, 2, 3, -1])
    got = sdm.sdm_lookup(bank, idx.to(DEV), dropout=0.5, rng=rng.to(DEV)).cpu()
    mask = torch.from_numpy(ref.kept(5, 64, 0.5, rng.tolist()))
    assert not got[~mask].any() and not got[4].any()
    assert torch.isnan(got[1:4][mask[1:4]]).all() and torch.isinf(got[0][mask[0]]).all()


@pytest.mark.parametrize("p", [2.0 ** -16, 0.1, 0.5, 0.9, 1 - 2.0 ** -16])
def test_masks(p):
    """Every seed and offset has its own mask, all of it as defined; without a threshold nothing is dropped."""
    bank = torch.ones((1, 72), device=DEV)
    idx = torch.zeros(200, dtype=torch.int64)
    seen = []
    for seed, offset in ((0, 0), (1, 0), (0, 1), (-1, -1), (1 << 32, 0), (0, 1 << 32)):
        rng = rng_of(seed, offset)
        got = sdm.sdm_lookup(bank, idx.to(DEV), dropout=p, rng=rng.to(DEV)).cpu()
        mask = ref.kept(200, 72, p, rng.tolist())
        assert np.array_equal(got.numpy(), np.where(mask, ref.factor(1.0, p), 0).astype(np.float32))
        seen.append(mask)
    if p in (0.1, 0.5, 0.9):
        assert not any(np.array_equal(a, b) for i, a in enumerate(seen) for b in seen[:i])
    tiny = sdm.sdm_lookup(bank, idx.to(DEV), dropout=2.0 ** -18)  # nearest to no dropout: no rng needed
    assert torch.equal(tiny, torch.ones_like(tiny))


def test_the_share_of_dropped_columns():
    bank = torch.ones((1, 1024), device=DEV)
    got = sdm.sdm_lookup(bank, torch.zeros(4096, dtype=torch.int32, device=DEV), dropout=0.1, rng=rng_of(7, 8).to(DEV))
    n, q = got.numel(), ref.threshold(0.1) / 65536
    # five standard deviations of a fair draw, over all, a row and a column
    assert abs((got == 0).sum().item() - n * q) < 5 * (n * q * (1 - q)) ** 0.5
    for dim, m in ((0, 4096), (1, 1024)):
        assert ((got == 0).sum(dim) - m * q).abs().max().item() < 6.5 * (m * q * (1 - q)) ** 0.5
    # of neighbours, both dropped
    both = ((got[:, 1:] == 0) & (got[:, :-1] == 0)).sum().item() / (4096 * 1023)
    assert abs(both - q * q) < 5 * (q * q / (4096 * 1023)) ** 0.5


@pytest.mark.parametrize("kind,off", [("f32", 1), ("bf16", 1), ("bf16", 4)])
def test_any_alignment(kind, off):
    dtype = torch.float32 if kind == "f32" else torch.bfloat16
    flat = (torch.randn(30 * 64 + off, generator=torch.Generator().manual_seed(4)) * 2).to(dtype)
    bank = flat.to(DEV)[off:].view(30, 64)
    idx = torch.arange(29, -1, -1)
    for out_dtype in (torch.float32, torch.bfloat16):
        out = torch.full((30 * 64 + off + 1,), 9.0, dtype=out_dtype, device=DEV)
        view = out[off:off + 30 * 64].view(30, 64)
        assert sdm.sdm_lookup(bank, idx.to(DEV), scale=2.0, out=view) is view
        same(view, ref.lookup(flat[off:].view(30, 64).float().numpy(), idx.numpy(), 2.0), out_dtype)
        assert (out[:off] == 9).all() and out[-1].item() == 9


@pytest.mark.slow
def test_a_bank_past_32_bit_offsets():
    bank = torch.zeros(((1 << 25) + 5, 136), dtype=torch.bfloat16, device=DEV)  # 4.56e9 values
    last = len(bank) - 1
    at = torch.tensor([last, 0, 1 << 24, last - 1])
    bank[at.to(DEV)] = torch.arange(1, 5, device=DEV, dtype=torch.bfloat16)[:, None].expand(4, 136)
    assert sdm.sdm_lookup(bank, at.to(DEV))[:, 135].tolist() == [1, 2, 3, 4]


@pytest.mark.slow
def test_more_rows_than_a_grid_holds():
    """70 M rows of 1032 columns, 144 GB: the rows past 2^24 - 1 workgroups of four, too, and their own masks."""
    n, hd = 70_000_000, 1032
    bank = torch.arange(1, 4, device=DEV, dtype=torch.bfloat16)[:, None].expand(3, hd).contiguous()
    idx = (torch.arange(n, device=DEV) % 4).to(torch.int32)  # a fourth of them none
    out = sdm.sdm_lookup(bank, idx)
    assert out.shape == (n, hd)
    for a in range(0, n, 1 << 22):
        rows, at = out[a:a + (1 << 22)], idx[a:a + (1 << 22)]
        assert (rows == torch.where(at < 3, at + 1, 0).to(torch.bfloat16)[:, None]).all()
    rng = rng_of(5, 6)
    sdm.sdm_lookup(bank, idx, dropout=0.5, rng=rng.to(DEV), out=out)
    edge = 4 * ((1 << 24) - 1)
    for i in (0, edge - 1, edge, edge + 6, n - 3):
        keep = torch.tensor([[w >> 16 * (j % 2) & 0xffff for j in range(8) for w in [ref.philox((o, i, 6, 0), (5, 0))[j // 2]]]
                             for o in range(hd // 8)]).flatten() >= 1 << 15
        assert torch.equal(out[i].cpu().float(), torch.where(keep, 2.0 * (i % 4 + 1), 0.0) * (i % 4 < 3)), i
    del out, rows
    torch.cuda.empty_cache()


def test_refusals():
    bank, idx = torch.ones((4, 8), device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(sdm.SdmError, match="needs rng"):
        sdm.sdm_lookup(bank, idx, dropout=0.5)
    with pytest.raises(sdm.SdmError, match="dropout must be"):
        sdm.sdm_lookup(bank, idx, dropout=1.0)
    with pytest.raises(ValueError, match="contiguous"):
        sdm.sdm_lookup(bank.t(), idx)
    with pytest.raises(ValueError, match="out must be"):
        sdm.sdm_lookup(bank, idx, out=torch.empty((4, 8), device=DEV))
    with pytest.raises(TypeError, match="rng"):
        sdm.sdm_lookup(bank, idx, dropout=0.5, rng=torch.zeros(2, device=DEV))
