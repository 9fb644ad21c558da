"""include/sdm_memory.h without a GPU: what it declares is exported, and bad
arguments are turned into status codes on the host before any HIP call (fake,
never dereferenced device addresses; no call here reaches a launch)."""

import os
import re
import subprocess

import pytest
import torch

import memory_ref as ref
import sparse_delta_rule_amd as sdm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "sdm_memory.h")

OK, E_DTYPE, E_SHAPE, E_RANGE, E_ALIGN, E_OVERLAP, E_NULL = 0, 1, 2, 3, 4, 5, 6
F32, BF16, I32, I64, MX8, MX4 = 0, 1, 2, 3, 4, 5
A = 0x10000000
MB = 1 << 20
GB = 1 << 30


def test_every_declared_function_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(sdm_[a-z_0-9]+)\s*\(", text)))
    assert names == ["sdm_bank_pack", "sdm_gather_packed", "sdm_gather_weight_grad", "sdm_packed_row_bytes",
                     "sdm_packed_scale_bytes", "sdm_route", "sdm_route_backward"]
    for name in names:
        assert hasattr(sdm.library(), name), name


@pytest.mark.parametrize("compiler,std", [("gcc", "-std=c11"), ("g++", "-std=c++17")])
def test_the_header_is_plain_c(compiler, std, tmp_path):
    name = tmp_path / ("a.c" if compiler == "gcc" else "a.cpp")
    name.write_text('#include "sdm_memory.h"\nint (*f)(void*, void*, int, int64_t, int64_t, const void*, int, int64_t, int64_t,'
                    " const void*, const void*, int, void*) = sdm_bank_pack;\n")
    r = subprocess.run([compiler, std, "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.dirname(HEADER), str(name)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_constants_match_the_header():
    text = open(HEADER).read()
    for name in ("SDM_MX8", "SDM_MX4"):
        assert int(re.search(rf"\b{name} = (\d+)", text).group(1)) == getattr(sdm, name)
    assert int(re.search(r"#define SDM_MAX_KEYS (\d+)", text).group(1)) == sdm.SDM_MAX_KEYS


@pytest.mark.parametrize("hd", [1, 2, 16, 17, 31, 32, 33, 100, 128, 129, 1000])
def test_packed_row_sizes(hd):
    for kind in ("mx8", "mx4"):
        assert sdm.PackedBank.row_bytes(hd, kind) == (ref.row_bytes(hd, kind), ref.scale_bytes(hd))
    lib = sdm.library()
    assert lib.sdm_packed_row_bytes(F32, hd) == 0 and lib.sdm_packed_scale_bytes(I64, hd) == 0
    assert lib.sdm_packed_row_bytes(MX8, 0) == 0 and lib.sdm_packed_row_bytes(MX8, (1 << 30) + 1) == 0
    with pytest.raises(ValueError, match="out of range"):
        sdm.PackedBank.row_bytes(0)
    with pytest.raises(ValueError, match="kind"):
        sdm.PackedBank.row_bytes(8, "mx2")


def call(fn, args):
    lib = sdm.library()
    rc = getattr(lib, fn)(*args.values())
    return rc, lib.sdm_last_error().decode()


def with_changes(args, changes):
    assert set(changes) <= set(args)
    return {**args, **changes}


# ------------------------------------------------------------------ route
ROUTE = dict(logits=A, logit_dtype=F32, tokens=16, keys=256, k=8, score=0, bias=A + 8 * MB, groups=8, kept=4, top=2,
             normalise=1, scale=1.0, streams=16, stream_slots=256, idx=A + 16 * MB, idx_dtype=I64, w=A + 24 * MB,
             w_dtype=F32, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(logit_dtype=I32), E_DTYPE, "logits must be"),
    (dict(logit_dtype=9), E_DTYPE, "logits must be"),
    (dict(idx_dtype=F32), E_DTYPE, "idx must be"),
    (dict(w_dtype=I64), E_DTYPE, "weights must be"),
    (dict(tokens=-1), E_SHAPE, "tokens = -1"),
    (dict(keys=0), E_RANGE, "keys must be in 1..65536"),
    (dict(keys=65544), E_RANGE, "keys must be in 1..65536"),
    (dict(keys=1 << 40), E_RANGE, "keys must be"),
    (dict(k=0), E_RANGE, "k must be in 1..256"),
    (dict(k=257, kept=8, keys=1024), E_RANGE, "k must be in 1..256"),
    (dict(k=129), E_RANGE, "at most the 128 keys to choose from"),
    (dict(score=2), E_RANGE, "score must be"),
    (dict(groups=0), E_RANGE, "groups must be in 1..256"),
    (dict(groups=257), E_RANGE, "groups must be in 1..256"),
    (dict(kept=0), E_RANGE, "kept_groups in 1..groups"),
    (dict(kept=9), E_RANGE, "kept_groups in 1..groups"),
    (dict(top=3), E_RANGE, "group_top must be 1 or 2"),
    (dict(groups=7, kept=7), E_SHAPE, "7 groups do not divide 256 keys"),
    (dict(scale=float("inf")), E_RANGE, "scale must be finite"),
    (dict(scale=float("nan")), E_RANGE, "scale must be finite"),
    (dict(streams=0), E_SHAPE, "streams = 0"),
    (dict(stream_slots=-1), E_SHAPE, "stream_slots = -1"),
    (dict(streams=1 << 40, stream_slots=1 << 40), E_SHAPE, "overflow"),
    (dict(tokens=(1 << 21) + 1), E_SHAPE, "at most 2^21 tokens"),
    (dict(stream_slots=1 << 28, idx_dtype=I32), E_RANGE, "does not fit"),
    (dict(logits=None), E_NULL, "required"),
    (dict(idx=None), E_NULL, "required"),
    (dict(w=None), E_NULL, "required"),
    (dict(logits=A + 2), E_ALIGN, "aligned"),
    (dict(bias=A + 8 * MB + 1), E_ALIGN, "aligned"),
    (dict(idx=A + 16 * MB + 4), E_ALIGN, "aligned"),
    (dict(w=A + 24 * MB + 2), E_ALIGN, "aligned"),
    (dict(idx=A + 16 * 256 * 4 - 8), E_OVERLAP, "idx and logits"),
    (dict(w=A + 8 * MB), E_OVERLAP, "w and bias"),
    (dict(w=A + 16 * MB), E_OVERLAP, "idx and w"),
])
def test_route_rejects(kw, code, msg):
    rc, got = call("sdm_route", with_changes(ROUTE, kw))
    assert rc == code and msg in got and got.startswith("sdm_route: "), got


def test_route_slots_that_just_fit():
    last = dict(streams=1 << 40, tokens=0)  # the streams that occur count, not all that are named
    assert call("sdm_route", with_changes(ROUTE, dict(last, stream_slots=1 << 22, idx_dtype=I32)))[0] == OK
    assert call("sdm_route", with_changes(ROUTE, dict(tokens=0, logits=None, idx=None, w=None))) == (OK, "")


BACKWARD = dict(logits=A, logit_dtype=BF16, tokens=16, keys=256, k=8, score=1, bias=None, normalise=1, scale=1.0,
                streams=16, stream_slots=256, idx=A + 16 * MB, idx_dtype=I32, dw=A + 24 * MB, w_dtype=BF16,
                dlogits=A + 32 * MB, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(logit_dtype=MX8), E_DTYPE, "logits must be"),
    (dict(idx_dtype=BF16), E_DTYPE, "idx must be"),
    (dict(w_dtype=I32), E_DTYPE, "weights must be"),
    (dict(tokens=-5), E_SHAPE, "tokens = -5"),
    (dict(keys=70000), E_RANGE, "keys must be"),
    (dict(k=300), E_RANGE, "k must be"),
    (dict(keys=4), E_RANGE, "at most the 4 keys"),
    (dict(score=-1), E_RANGE, "score must be"),
    (dict(scale=float("-inf")), E_RANGE, "finite"),
    (dict(streams=-1), E_SHAPE, "streams = -1"),
    (dict(dw=None), E_NULL, "required"),
    (dict(dlogits=None), E_NULL, "required"),
    (dict(dw=A + 24 * MB + 1), E_ALIGN, "aligned"),
    (dict(dlogits=A + 32 * MB + 1), E_ALIGN, "aligned"),
    (dict(dlogits=A), E_OVERLAP, "dlogits and logits"),
    (dict(dlogits=A + 24 * MB - 2), E_OVERLAP, "dlogits and dw"),
    (dict(idx=A + 32 * MB + 16 * 256 * 2 - 4), E_OVERLAP, "dlogits and idx"),
])
def test_route_backward_rejects(kw, code, msg):
    rc, got = call("sdm_route_backward", with_changes(BACKWARD, kw))
    assert rc == code and msg in got and got.startswith("sdm_route_backward: "), got


def test_route_backward_of_nothing():
    assert call("sdm_route_backward", with_changes(BACKWARD, dict(tokens=0, logits=None, dlogits=None))) == (OK, "")


# ------------------------------------------------------------------ packed banks
PACK = dict(codes=A, scales=A + 64 * MB, packed_dtype=MX8, num_slots=1000, head_dim=100, rows=A + 128 * MB, row_dtype=BF16,
            num_rows=500, n=300, row_idx=A + 256 * MB, slots=A + 320 * MB, idx_dtype=I64, stream=None)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(packed_dtype=BF16), E_DTYPE, "SDM_MX8 or SDM_MX4"),
    (dict(row_dtype=MX4), E_DTYPE, "rows must be"),
    (dict(idx_dtype=F32), E_DTYPE, "row_idx and slots must be"),
    (dict(num_slots=0), E_SHAPE, "empty bank"),
    (dict(head_dim=0), E_SHAPE, "empty bank"),
    (dict(head_dim=(1 << 28) + 1), E_RANGE, "would exceed"),
    (dict(n=-1), E_SHAPE, "n = -1"),
    (dict(num_rows=-1), E_SHAPE, "num_rows = -1"),
    (dict(num_slots=1 << 60), E_SHAPE, "overflow"),
    (dict(n=1 << 62), E_SHAPE, "overflow"),
    (dict(row_idx=None, n=501), E_SHAPE, "n = 501 rows of 500"),
    (dict(slots=None, n=1001, num_rows=2000), E_SHAPE, "into 1000 slots"),
    (dict(codes=None), E_NULL, "required"),
    (dict(scales=None), E_NULL, "required"),
    (dict(rows=None), E_NULL, "required"),
    (dict(codes=A + 8), E_ALIGN, "codes must be 16-byte"),
    (dict(scales=A + 64 * MB + 2), E_ALIGN, "scales 4-byte"),
    (dict(rows=A + 128 * MB + 1), E_ALIGN, "element size"),
    (dict(slots=A + 320 * MB + 4), E_ALIGN, "element size"),
    (dict(scales=A + 1000 * 112 - 4), E_OVERLAP, "codes and scales"),
    (dict(rows=A + 64 * MB + 3998), E_OVERLAP, "scales and rows"),
    (dict(slots=A + 111992), E_OVERLAP, "codes and slots"),
])
def test_pack_rejects(kw, code, msg):
    rc, got = call("sdm_bank_pack", with_changes(PACK, kw))
    assert rc == code and msg in got and got.startswith("sdm_bank_pack: "), got


def test_pack_of_nothing():
    assert call("sdm_bank_pack", with_changes(PACK, dict(n=0, codes=None, rows=None))) == (OK, "")
    assert call("sdm_bank_pack", with_changes(PACK, dict(num_rows=0, rows=None))) == (OK, "")


GATHER = dict(codes=A, scales=A + 64 * MB, dtype=MX8, num_slots=1000, head_dim=100, tokens=64, chunk=16, valid=16,
              chunk_valid=A + 100 * MB, idx_dtype=I32, w_dtype=BF16, idx0=A + 128 * MB, w0=A + 160 * MB, width0=32,
              out0=A + 192 * MB, idx1=A + 224 * MB, w1=A + 256 * MB, width1=16, out1=A + 288 * MB, stream=None)


@pytest.mark.parametrize("fn", ["sdm_gather_packed", "sdm_gather_weight_grad"])
@pytest.mark.parametrize("kw,code,msg", [
    (dict(dtype=I32), E_DTYPE, "SDM_MX8"),
    (dict(dtype=77), E_DTYPE, "SDM_MX8"),
    (dict(idx_dtype=F32), E_DTYPE, "slots must be"),
    (dict(w_dtype=MX8), E_DTYPE, "weights must be"),
    (dict(num_slots=0), E_SHAPE, "empty bank"),
    (dict(head_dim=-3), E_SHAPE, "empty bank"),
    (dict(head_dim=(1 << 28) + 1), E_RANGE, "head_dim"),
    (dict(tokens=-16), E_SHAPE, "whole number of chunks"),
    (dict(tokens=63), E_SHAPE, "whole number of chunks"),
    (dict(chunk=0), E_SHAPE, "whole number of chunks"),
    (dict(valid=17), E_SHAPE, "valid lie in"),
    (dict(valid=-1), E_SHAPE, "valid lie in"),
    (dict(width0=0), E_RANGE, "width0 must be in 1..256"),
    (dict(width0=257), E_RANGE, "width0 must be in 1..256"),
    (dict(width1=300), E_RANGE, "width1 must be in 1..256"),
    (dict(width1=0), E_RANGE, "width1 must be in 1..256"),
    (dict(idx1=None), E_NULL, "given in part"),
    (dict(w1=None), E_NULL, "given in part"),
    (dict(out1=None), E_NULL, "given in part"),
    (dict(num_slots=1 << 60), E_SHAPE, "overflow"),
    (dict(tokens=1 << 50, chunk=1 << 50), E_SHAPE, "overflow"),
    (dict(tokens=1 << 32, idx1=None, w1=None, out1=None, width1=0, head_dim=1, idx0=A + 2048 * GB,
          w0=A + 4096 * GB, out0=A + 8192 * GB, chunk_valid=A + 16384 * GB), E_SHAPE, "exceed the grid"),
    (dict(codes=None), E_NULL, "required"),
    (dict(scales=None), E_NULL, "required"),
    (dict(idx0=None), E_NULL, "required"),
    (dict(w0=None), E_NULL, "required"),
    (dict(out0=None), E_NULL, "required"),
    (dict(codes=A + 8), E_ALIGN, "codes must be 16-byte"),
    (dict(scales=A + 64 * MB + 1), E_ALIGN, "scales 4-byte"),
    (dict(idx0=A + 128 * MB + 2), E_ALIGN, "element size"),
    (dict(w1=A + 256 * MB + 1), E_ALIGN, "element size"),
    (dict(out0=A + 192 * MB + 1), E_ALIGN, "element size"),
    (dict(chunk_valid=A + 100 * MB + 2), E_ALIGN, "element size"),
    (dict(out0=A + 111996), E_OVERLAP, "codes"),
    (dict(out0=A + 64 * MB), E_OVERLAP, "scales"),
    (dict(out0=A + 128 * MB), E_OVERLAP, "idx"),
    (dict(out1=A + 256 * MB), E_OVERLAP, "share memory"),
    (dict(out1=A + 192 * MB), E_OVERLAP, "share memory"),
])
def test_gathers_reject(kw, code, msg, fn):
    rc, got = call(fn, with_changes(GATHER, kw))
    assert rc == code and msg in got and got.startswith(fn + ": "), got


def test_gathers_of_nothing_and_of_too_many_columns():
    for fn in ("sdm_gather_packed", "sdm_gather_weight_grad"):
        assert call(fn, with_changes(GATHER, dict(tokens=0, codes=None, idx0=None, idx1=None))) == (OK, "")
    rc, got = call("sdm_gather_packed", with_changes(GATHER, dict(head_dim=1 << 27)))
    assert rc == E_RANGE and "grid" in got


def test_weight_grad_of_a_float_bank_needs_no_scales_and_only_its_alignment():
    base = with_changes(GATHER, dict(dtype=BF16, scales=None, codes=A + 2))
    rc, got = call("sdm_gather_weight_grad", with_changes(base, dict(out0=A + 2 + 1000 * 200 - 2)))
    assert rc == E_OVERLAP and "bank" in got
    rc, got = call("sdm_gather_weight_grad", with_changes(base, dict(codes=A + 1)))
    assert rc == E_ALIGN
    rc, got = call("sdm_gather_packed", base)
    assert rc == E_DTYPE


# ------------------------------------------------------------------ the binding
def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 8))
    idx, w = torch.zeros((4, 2), dtype=torch.int64), torch.zeros((4, 2))
    for what in (lambda: sdm.sdm_route(x, 2), lambda: sdm.sdm_route_backward(x, idx, w),
                 lambda: sdm.PackedBank.empty(10, 8, "mx8", device="cpu"),
                 lambda: sdm.sdm_gather_weight_grad(x, idx, x, chunk=4)):
        with pytest.raises(ValueError, match="is on cpu"):
            what()


def test_binding_refuses_bad_shapes_and_types():
    x = torch.zeros((4, 8))
    with pytest.raises(TypeError, match="logits has unsupported dtype"):
        sdm.sdm_route(x.double(), 2)
    with pytest.raises(ValueError, match="keys"):
        sdm.sdm_route(torch.zeros(()), 2)
    with pytest.raises(ValueError, match="kind"):
        sdm.PackedBank(torch.zeros((4, 16), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), 8, "int8")
    with pytest.raises(ValueError, match="codes must be"):
        sdm.PackedBank(torch.zeros((4, 8), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), 8)
    with pytest.raises(ValueError, match="num_slots, row_bytes"):
        sdm.PackedBank(torch.zeros((4,), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8), 8)
    with pytest.raises(TypeError, match="codes has unsupported dtype"):
        sdm.PackedBank(torch.zeros((4, 16)), torch.zeros((4, 4), dtype=torch.uint8), 8)
    with pytest.raises(ValueError, match="bank must be"):
        sdm.sdm_gather_weight_grad(torch.zeros(8), torch.zeros((4, 2), dtype=torch.int64), x, chunk=4)
