"""include/sdm_train.h without a GPU: what it declares is exported, and bad
arguments are turned into status codes on the host before any HIP call (fake,
never dereferenced device addresses; no call here reaches a launch)."""

import os
import re
import subprocess

import pytest
import torch

import sparse_delta_rule_amd as sdm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sdm_train.h")

OK, E_DTYPE, E_SHAPE, E_RANGE, E_ALIGN, E_OVERLAP, E_NULL = 0, 1, 2, 3, 4, 5, 6
F32, BF16, I32, I64, MX8, MX4 = 0, 1, 2, 3, 4, 5
A = 0x10000000
MB = 1 << 20
NAN, INF = float("nan"), float("inf")


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sdm_[a-z_0-9]+)\s*\(", text)))
    assert names == ["sdm_bank_grad_workspace", "sdm_gather_bank_grad", "sdm_lookup", "sdm_lookup_grad",
                     "sdm_route_balance", "sdm_route_balance_backward", "sdm_route_balance_workspace"]
    for name in names:
        assert hasattr(sdm.library(), name), name
    for name in names:
        if "workspace" not in name:
            assert callable(getattr(sdm, name))


@pytest.mark.parametrize("compiler,std", [("gcc", "-std=c11"), ("g++", "-std=c++17")])
def test_the_header_is_plain_c(compiler, std, tmp_path):
    name = tmp_path / ("a.c" if compiler == "gcc" else "a.cpp")
    name.write_text('#include "sdm_train.h"\nint64_t (*f)(int64_t, int64_t, int64_t) = sdm_bank_grad_workspace;\n'
                    "int g(void) { return SDM_GRAD_WRITE + SDM_GRAD_ADD + (SDM_MAX_GRAD_ENTRIES > 0); }\n")
    r = subprocess.run([compiler, std, "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(name)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def call(fn, args):
    lib = sdm.library()
    rc = getattr(lib, fn)(*args.values())
    return rc, lib.sdm_last_error().decode()


def with_changes(args, changes):
    assert set(changes) <= set(args)
    return {**args, **changes}


def rejects(fn, args, kw, code, msg):
    rc, got = call(fn, with_changes(args, kw))
    assert rc == code and msg in got and got.startswith(fn + ": "), (rc, got)


# ------------------------------------------------------------------ balance
BALANCE = dict(logits=A, logit_dtype=F32, tokens=16, keys=256, k=8, score=0, chunk=4, valid=4, chunk_valid=A + 4 * MB,
               per_chunk=1, scale=1.0, streams=16, stream_slots=256, idx=A + 16 * MB, idx_dtype=I64, counts=A + 24 * MB,
               mean=A + 32 * MB, coef=A + 40 * MB, loss=A + 48 * MB, workspace=A + 64 * MB, workspace_bytes=MB, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(logit_dtype=I32), E_DTYPE, "logits must be"),
    (dict(idx_dtype=F32), E_DTYPE, "idx must be"),
    (dict(tokens=-4), E_SHAPE, "tokens = -4"),
    (dict(tokens=(1 << 21) + 4), E_SHAPE, "at most 2^21 tokens"),
    (dict(keys=0), E_RANGE, "keys must be"),
    (dict(keys=65537), E_RANGE, "keys must be"),
    (dict(k=0), E_RANGE, "k must be"),
    (dict(k=257, keys=1000), E_RANGE, "k must be"),
    (dict(k=9, keys=8), E_RANGE, "at most the 8 keys"),
    (dict(score=2), E_RANGE, "score must be"),
    (dict(chunk=0), E_SHAPE, "whole number of chunks"),
    (dict(chunk=5), E_SHAPE, "whole number of chunks"),
    (dict(valid=5), E_SHAPE, "valid lie in"),
    (dict(valid=-1), E_SHAPE, "valid lie in"),
    (dict(scale=NAN), E_RANGE, "scale must be finite"),
    (dict(streams=0), E_SHAPE, "streams = 0"),
    (dict(streams=1 << 40, stream_slots=1 << 40), E_SHAPE, "overflow"),
    (dict(logits=None), E_NULL, "required"),
    (dict(idx=None), E_NULL, "required"),
    (dict(loss=None), E_NULL, "required"),
    (dict(coef=None), E_NULL, "required"),
    (dict(workspace=None), E_NULL, "workspace is required"),
    (dict(workspace_bytes=100), E_SHAPE, "100 bytes"),
    (dict(workspace=A + 64 * MB + 8), E_ALIGN, "16-byte"),
    (dict(logits=A + 2), E_ALIGN, "aligned"),
    (dict(chunk_valid=A + 4 * MB + 1), E_ALIGN, "aligned"),
    (dict(counts=A + 32 * MB), E_OVERLAP, "counts and mean"),
    (dict(loss=A + 40 * MB + 12), E_OVERLAP, "coef and loss"),
    (dict(mean=A + 16 * 256 * 4 - 4), E_OVERLAP, "mean and logits"),
    (dict(workspace=A + 16 * MB), E_OVERLAP, "workspace and idx"),
    (dict(chunk_valid=A + 64 * MB), E_OVERLAP, "workspace and chunk_valid"),
])
def test_balance_rejects(kw, code, msg):
    rejects("sdm_route_balance", BALANCE, kw, code, msg)


def test_balance_workspace():
    f = sdm.library().sdm_route_balance_workspace
    assert f(0, 8, 1, 0) > 0 and f(0, 8, 1, 1) > 0
    assert f(-1, 8, 1, 0) == f(10, 8, 3, 0) == f(10, 0, 5, 0) == f(10, 70000, 5, 0) == f(1 << 22, 8, 1, 0) == f(4, 8, 0, 0) == 0
    # sums of 4 bytes and counts of 2 for each key of each piece, and at most 512 + sequences pieces for few tokens
    assert f(1 << 21, 65536, 1, 1) > (1 << 37) * 6
    assert f(4096, 16384, 4096, 0) < 513 * 16384 * 6 + 8 * 256 + 4 * 513 + 100


BACKWARD = dict(logits=A, logit_dtype=BF16, tokens=16, keys=256, score=1, chunk=16, valid=16, chunk_valid=None, per_chunk=0,
                counts=A + 24 * MB, coef=A + 40 * MB, dloss=A + 48 * MB, accumulate=0, dlogits=A + 64 * MB, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(logit_dtype=MX8), E_DTYPE, "logits must be"),
    (dict(tokens=-1), E_SHAPE, "tokens = -1"),
    (dict(keys=-3), E_RANGE, "keys must be"),
    (dict(score=7), E_RANGE, "score must be"),
    (dict(chunk=3), E_SHAPE, "whole number"),
    (dict(counts=None), E_NULL, "required"),
    (dict(coef=None), E_NULL, "required"),
    (dict(dlogits=None), E_NULL, "required"),
    (dict(dlogits=A + 1), E_ALIGN, "aligned"),
    (dict(dloss=A + 2), E_ALIGN, "aligned"),
    (dict(dlogits=A), E_OVERLAP, "dlogits and logits"),
    (dict(dlogits=A + 24 * MB - 2), E_OVERLAP, "dlogits and counts"),
    (dict(dloss=A + 64 * MB), E_OVERLAP, "dlogits and dloss"),
])
def test_balance_backward_rejects(kw, code, msg):
    rejects("sdm_route_balance_backward", BACKWARD, kw, code, msg)


def test_balance_backward_of_nothing():
    assert call("sdm_route_balance_backward", with_changes(BACKWARD, dict(tokens=0, logits=None, dlogits=None))) == (OK, "")


# ------------------------------------------------------------------ lookups
LOOKUP = dict(bank=A, scales=A + 64 * MB, bank_dtype=MX8, num_slots=1000, head_dim=100, n=300, idx=A + 128 * MB, idx_dtype=I64,
              scale=1.0, dropout=0.5, rng=A + 160 * MB, out=A + 200 * MB, out_dtype=BF16, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(bank_dtype=I32), E_DTYPE, "the bank must be"),
    (dict(idx_dtype=BF16), E_DTYPE, "idx must be"),
    (dict(out_dtype=MX8), E_DTYPE, "out must be"),
    (dict(num_slots=0), E_SHAPE, "empty bank"),
    (dict(head_dim=0), E_SHAPE, "empty bank"),
    (dict(head_dim=1 << 29), E_RANGE, "head_dim must be"),
    (dict(head_dim=65535 * 256 + 1), E_RANGE, "head_dim must be at most 16776960"),
    (dict(num_slots=1 << 60), E_SHAPE, "overflow"),
    (dict(n=-1), E_SHAPE, "n must be"),
    (dict(n=1 << 31), E_SHAPE, "n must be"),
    (dict(scale=INF), E_RANGE, "scale must be finite"),
    (dict(dropout=1.0), E_RANGE, "dropout must be"),
    (dict(dropout=-0.1), E_RANGE, "dropout must be"),
    (dict(dropout=NAN), E_RANGE, "dropout must be"),
    (dict(rng=None), E_NULL, "needs rng"),
    (dict(rng=A + 160 * MB + 4), E_ALIGN, "rng must be 8-byte"),
    (dict(bank=None), E_NULL, "required"),
    (dict(scales=None), E_NULL, "required"),
    (dict(idx=None), E_NULL, "required"),
    (dict(out=None), E_NULL, "required"),
    (dict(bank=A + 8), E_ALIGN, "codes must be 16-byte"),
    (dict(bank_dtype=F32, bank=A + 2), E_ALIGN, "element size"),
    (dict(out=A + 200 * MB + 1), E_ALIGN, "element size"),
    (dict(out=A + 1000 * 112 - 2), E_OVERLAP, "out and codes"),
    (dict(out=A + 128 * MB + 8), E_OVERLAP, "out and idx"),
    (dict(rng=A + 200 * MB), E_OVERLAP, "out and rng"),
    (dict(n=(1 << 31) - 1, head_dim=2048, idx=A + (1 << 50), out=A + (1 << 51)), E_SHAPE, "exceed the grid"),
])
def test_lookup_rejects(kw, code, msg):
    rejects("sdm_lookup", LOOKUP, kw, code, msg)


@pytest.mark.parametrize("head_dim", [513, 1024, 1025, 1032, 5000])
def test_rows_of_a_lookup(head_dim):
    """As many as the header says, and one more; the call stops at the shared memory that it finds, or at the grid."""
    most = (1 << 28) * max(1, 256 // -(-head_dim // 8))
    args = with_changes(LOOKUP, dict(bank_dtype=BF16, scales=None, head_dim=head_dim, idx=A + (1 << 50), out=A))
    rejects("sdm_lookup", args, dict(n=most), E_OVERLAP, "out and bank")
    rejects("sdm_lookup", args, dict(n=most + 1, out=A + (1 << 51)), E_SHAPE, "exceed the grid")


def test_lookup_of_nothing():
    assert call("sdm_lookup", with_changes(LOOKUP, dict(n=0, bank=None, idx=None, out=None, rng=None))) == (OK, "")


GRAD = dict(n=300, idx=A, idx_dtype=I32, dout=A + 64 * MB, dout_dtype=BF16, scale=1.0, dropout=0.5, rng=A + 160 * MB,
            dbank=A + 200 * MB, bank_dtype=F32, num_slots=1000, head_dim=100, mode=0, workspace=A + 256 * MB,
            workspace_bytes=16 * MB, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(idx_dtype=F32), E_DTYPE, "idx must be"),
    (dict(dout_dtype=I64), E_DTYPE, "dout must be"),
    (dict(bank_dtype=MX8), E_DTYPE, "dbank must be"),
    (dict(num_slots=0), E_SHAPE, "empty bank"),
    (dict(num_slots=1 << 31), E_RANGE, "at most 2^31 - 1 slots"),
    (dict(head_dim=-1), E_SHAPE, "empty bank"),
    (dict(head_dim=65535 * 256 + 1, num_slots=2), E_RANGE, "head_dim must be at most 16776960"),
    (dict(mode=2), E_RANGE, "mode must be"),
    (dict(n=-1), E_SHAPE, "n must be"),
    (dict(n=1 << 31), E_SHAPE, "n must be"),
    (dict(scale=NAN), E_RANGE, "scale must be"),
    (dict(dropout=0.99999), E_RANGE, "dropout must be"),
    (dict(rng=None), E_NULL, "needs rng"),
    (dict(idx=None), E_NULL, "required"),
    (dict(dout=None), E_NULL, "required"),
    (dict(dbank=None), E_NULL, "required"),
    (dict(n=0, dbank=None), E_NULL, "required"),
    (dict(dout=A + 64 * MB + 1), E_ALIGN, "element size"),
    (dict(workspace=None), E_NULL, "workspace is required"),
    (dict(workspace_bytes=1000), E_SHAPE, "1000 bytes"),
    (dict(workspace=A + 256 * MB + 4), E_ALIGN, "16-byte"),
    (dict(dbank=A + 64 * MB), E_OVERLAP, "dbank and dout"),
    (dict(workspace=A + 200 * MB), E_OVERLAP, "dbank and workspace"),
    (dict(workspace=A), E_OVERLAP, "workspace and idx"),
    (dict(rng=A + 200 * MB + 8), E_OVERLAP, "dbank and rng"),
    (dict(num_slots=(1 << 31) - 1, head_dim=16384, dbank=A + (1 << 50)), E_SHAPE, "exceed the grid"),
])
def test_lookup_grad_rejects(kw, code, msg):
    rejects("sdm_lookup_grad", GRAD, kw, code, msg)


@pytest.mark.parametrize("scale,dropout,ok", [(3e38, 0.5, False), (-3e38, 0.2, False), (6e33, 1 - 2.0 ** -16, False),
                                              (3e38, 0.0, True), (1.5e38, 0.5, True), (5e33, 1 - 2.0 ** -16, True)])
def test_a_factor_past_float32_is_refused(scale, dropout, ok):
    """scale / (1 - dropout); a call that passes this check stops at the pointer that it lacks."""
    for fn, args in (("sdm_lookup", with_changes(LOOKUP, dict(bank=None))), ("sdm_lookup_grad", with_changes(GRAD, dict(dout=None)))):
        rejects(fn, args, dict(scale=scale, dropout=dropout), *((E_NULL, "required") if ok else (E_RANGE, "finite in float32")))


def test_lookup_grad_of_nothing():
    assert call("sdm_lookup_grad", with_changes(GRAD, dict(n=0, mode=1, idx=None, dout=None, dbank=None, rng=None))) == (OK, "")


BANK = dict(tokens=64, chunk=16, valid=16, chunk_valid=A + 8 * MB, idx_dtype=I64, w_dtype=BF16, idx0=A, w0=A + 16 * MB,
            dout0=A + 32 * MB, width0=32, idx1=A + 64 * MB, w1=A + 80 * MB, dout1=A + 96 * MB, width1=16, dbank=A + 200 * MB,
            bank_dtype=F32, num_slots=1000, head_dim=128, mode=0, workspace=A + 256 * MB, workspace_bytes=16 * MB, stream=None)
ONE = dict(idx1=None, w1=None, dout1=None, width1=0)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(idx_dtype=F32), E_DTYPE, "slots must be"),
    (dict(w_dtype=I32), E_DTYPE, "weights must be"),
    (dict(bank_dtype=MX4), E_DTYPE, "dbank must be"),
    (dict(num_slots=-1), E_SHAPE, "empty bank"),
    (dict(mode=-1), E_RANGE, "mode must be"),
    (dict(tokens=65), E_SHAPE, "whole number"),
    (dict(tokens=-16), E_SHAPE, "whole number"),
    (dict(valid=17), E_SHAPE, "valid lie in"),
    (dict(idx1=None), E_NULL, "in part"),
    (dict(w1=None), E_NULL, "in part"),
    (dict(dout1=None), E_NULL, "in part"),
    (dict(width0=0), E_RANGE, "width0 must be"),
    (dict(width0=257), E_RANGE, "width0 must be"),
    (dict(width1=0), E_RANGE, "width1 must be"),
    (dict(width1=300), E_RANGE, "width1 must be"),
    (dict(tokens=1 << 26), E_SHAPE, "at most 2^31 - 1 entries"),
    (dict(dbank=None), E_NULL, "required"),
    (dict(w0=None), E_NULL, "required"),
    (dict(dout0=A + 32 * MB + 2), E_ALIGN, "element size"),
    (dict(chunk_valid=A + 8 * MB + 2), E_ALIGN, "element size"),
    (dict(workspace=None), E_NULL, "workspace is required"),
    (dict(workspace_bytes=0), E_SHAPE, "0 bytes"),
    (dict(dbank=A + 96 * MB), E_OVERLAP, "dbank and dout"),
    (dict(workspace=A + 80 * MB), E_OVERLAP, "workspace and w"),
    (dict(dbank=A + 256 * MB), E_OVERLAP, "dbank and workspace"),
    (dict(dbank=A + 8 * MB), E_OVERLAP, "dbank and chunk_valid"),
])
def test_bank_grad_rejects(kw, code, msg):
    rejects("sdm_gather_bank_grad", BANK, kw, code, msg)


def test_bank_grad_of_nothing():
    assert call("sdm_gather_bank_grad", with_changes(BANK, dict(ONE, tokens=0, mode=1, idx0=None, dbank=None))) == (OK, "")


def test_bank_grad_workspace():
    f = sdm.library().sdm_bank_grad_workspace
    assert f(0, 1, 1) > 0
    assert f(-1, 1, 1) == f(1, 0, 1) == f(1, 1, 0) == f(1 << 31, 1, 1) == f(1, 1 << 31, 1) == f(1, 1, 1 << 29) == 0
    for n in (1, 1000, 1 << 20):
        for hd in (1, 8, 128, 1024):
            # two arrays of 12 bytes an entry, sums of at most two runs for each 16 entries, counts of digits
            least, rows = 24 * n, 2 * -(-n // 16) * 4 * (hd + 7) // 8 * 8
            assert least < f(n, 1 << 20, hd) < least + rows + 64 * 1024 + n


@pytest.mark.parametrize("entries,slots,head_dim", [
    (32768 * 512, 32768, 8192), ((1 << 20) * 512, 1 << 20, 1024), (1 << 20, 64, 4160), (33024, 3, 65535 * 256), (40, 3, 65535 * 256),
    ((1 << 31) - 1, 1 << 21, 128), ((1 << 31) - 1, (1 << 31) - 1, 1), ((1 << 31) - 1, 1 << 27, 40), (5000, 1 << 27, 20000)])
def test_bank_grad_workspace_of_many_entries(entries, slots, head_dim):
    """The header's bound: sums of runs do not grow with entries times columns."""
    size = sdm.library().sdm_bank_grad_workspace(entries, slots, head_dim)
    assert 24 * entries < size <= 27 * entries + max(1 << 30, 16 * entries) + MB


@pytest.mark.parametrize("entries,over", [(300, True), (4096, True), (5000, False)])
def test_the_largest_written_bank(entries, over):
    """Sizes alone: a call within them stops at the memory that dbank and dout share."""
    args = with_changes(GRAD, dict(n=entries, num_slots=1 << 22, head_dim=16384, dout=A + (1 << 45), dbank=A + (1 << 46), workspace=A + (1 << 44),
                                   workspace_bytes=1 << 40))
    if over:
        rejects("sdm_lookup_grad", args, {}, E_SHAPE, "exceed the grid")
    rejects("sdm_lookup_grad", args, dict(num_slots=(1 << 22) - 2, dout=A + (1 << 46)), E_OVERLAP, "dbank and dout")


# ------------------------------------------------------------------ the binding's own checks
def test_the_binding_checks_its_tensors():
    """Host tensors: every call stops before the library."""
    x, i = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int64)
    for f in (lambda: sdm.sdm_route_balance(x, i), lambda: sdm.sdm_lookup(x, i), lambda: sdm.sdm_lookup_grad(i[:, 0], x, 9),
              lambda: sdm.sdm_gather_bank_grad(i, x[:, :2].contiguous(), x, 9, chunk=4),
              lambda: sdm.sdm_route_balance_backward(x, i[:1].int(), x[0, :1])):
        with pytest.raises(ValueError, match="device -1"):
            f()
    with pytest.raises(TypeError, match="dtype"):
        sdm.sdm_lookup(x.half(), i)
    with pytest.raises(ValueError, match="none of them"):
        sdm.sdm_gather_bank_grad(i, x[:, :2].contiguous(), x, 9, chunk=4, idx1=i)


def test_a_lookups_out_and_its_type_agree():
    x, i = torch.zeros((4, 8)), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="out is torch.bfloat16, out_dtype torch.float32"):
        sdm.sdm_lookup(x, i, out=x.bfloat16(), out_dtype=torch.float32)
    with pytest.raises(ValueError, match="device -1"):  # which they do here
        sdm.sdm_lookup(x, i, out=x.bfloat16(), out_dtype=torch.bfloat16)
