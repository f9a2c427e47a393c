"""Host-side checks of the fused-epilogue, grouped and row operators, without a GPU: bad arguments are refused
before any CUDA call, outputs may not overlap other buffers, workspace sizes, and the plain forms' own pins."""

import ctypes

import numpy as np
import pytest

from tests import operators_plain as plain

BIG = 1 << 40


def far(i):
    """Distinct fake addresses, 64 GiB apart, never dereferenced."""
    return ctypes.c_void_p((i + 1) << 36)


MIS = ctypes.c_void_p((1 << 36) + 4)

LAYER = dict(packed=far(0), s=far(1), out=8, K=64, u=far(2), tokens=4, bias=far(3), act=4, glu=1, residual=far(4), o=far(5),
             o_dtype=1, workspace=far(6), bytes=BIG, stream=None)
GROUPED = dict(packed=far(0), s=far(1), experts=3, out=8, K=64, u=far(2), tokens=4, rows=far(3), offsets=far(4), n=8,
               bias=far(5), act=4, glu=1, o=far(6), o_dtype=0, workspace=far(7), bytes=BIG, stream=None)
GROUP = dict(ids=far(0), tokens=4, topk=2, experts=8, offsets=far(1), rows=far(2), slots=far(3), stream=None)
COMBINE = dict(y=far(0), dtype=1, n=8, width=16, slots=far(1), weights=far(2), tokens=4, topk=2, residual=far(3), o=far(4),
               stream=None)
BASE = {"lq_gemm_epilogue": LAYER, "lq_gemv_epilogue": LAYER, "lq_gemm_grouped": GROUPED, "lq_group_rows": GROUP,
        "lq_combine_rows": COMBINE}

BAD = [(fn, {key: None}) for fn, base in BASE.items() for key, v in base.items()
       if isinstance(v, ctypes.c_void_p) and (key not in ("bias", "residual", "rows") or fn == "lq_group_rows")]
BAD += [(fn, {key: MIS}) for fn, base in BASE.items() for key, v in base.items() if isinstance(v, ctypes.c_void_p)]
for fn in ("lq_gemm_epilogue", "lq_gemv_epilogue", "lq_gemm_grouped"):
    BAD += [(fn, c) for c in ({"out": 0}, {"out": 7}, {"K": 0}, {"K": 48}, {"K": -32}, {"tokens": 0}, {"act": -1}, {"act": 5}, {"glu": 2},
                              {"glu": -1}, {"o_dtype": 2}, {"bytes": 0}, {"workspace": ctypes.c_void_p((7 << 36) + 16)})]
BAD += [("lq_gemv_epilogue", {"tokens": 17}), ("lq_gemm_grouped", {"experts": 0}), ("lq_gemm_grouped", {"experts": 4097}),
        ("lq_gemm_grouped", {"n": 0}), ("lq_gemm_grouped", {"experts": 4096, "out": 1 << 20}),
        ("lq_gemm_grouped", {"rows": None, "n": 5}), ("lq_group_rows", {"tokens": 0}), ("lq_group_rows", {"topk": 0}),
        ("lq_group_rows", {"experts": 0}), ("lq_group_rows", {"experts": 4097}),
        ("lq_group_rows", {"tokens": 1 << 20, "topk": 1 << 12}), ("lq_combine_rows", {"dtype": 2}), ("lq_combine_rows", {"n": 0}),
        ("lq_combine_rows", {"width": 0}), ("lq_combine_rows", {"tokens": 0}), ("lq_combine_rows", {"topk": 0}),
        ("lq_combine_rows", {"tokens": 1 << 20, "topk": 1 << 12})]

LAST, PAST = 2 ** 31 - 4097, 2 ** 31 - 4096  # the largest count that is taken, and the next one
BAD += [("lq_gemm_epilogue", {"out": PAST, "K": 32}), ("lq_gemm_epilogue", {"K": PAST}), ("lq_gemm_epilogue", {"tokens": PAST}),
        ("lq_gemv_epilogue", {"K": PAST}), ("lq_gemm_grouped", {"experts": 1, "out": PAST}), ("lq_gemm_grouped", {"n": PAST}),
        ("lq_gemm_grouped", {"experts": 4096, "out": 2 ** 19}), ("lq_gemm_grouped", {"tokens": PAST}),
        ("lq_group_rows", {"tokens": 1, "topk": PAST}), ("lq_group_rows", {"tokens": PAST, "topk": 1}),
        ("lq_combine_rows", {"tokens": 1, "topk": PAST}), ("lq_combine_rows", {"n": PAST}), ("lq_combine_rows", {"width": PAST})]


def call(fn, **change):
    import bit_lifted_gemm_b200 as lq
    return getattr(lq.lib, fn)(*{**BASE[fn], **change}.values())


@pytest.mark.parametrize("fn,change", BAD, ids=lambda v: v if isinstance(v, str) else "-".join(f"{k}={x}" for k, x in v.items()))
def test_bad_arguments_refused(fn, change, monkeypatch):
    import bit_lifted_gemm_b200 as lq
    monkeypatch.setenv("LQ_FAULT", "launch")  # what is accepted by mistake launches nothing
    assert call(fn, **change) == lq.LQ_ERR_INVALID_ARG


@pytest.mark.parametrize("fn", list(BASE))
def test_good_arguments_pass_the_checks(fn, monkeypatch):
    import bit_lifted_gemm_b200 as lq
    monkeypatch.setenv("LQ_FAULT", "launch")
    assert call(fn) == lq.LQ_ERR_CUDA
    optional = [k for k in ("bias", "residual", "rows") if k in BASE[fn] and fn != "lq_group_rows"]
    change = {k: None for k in optional}
    if fn == "lq_gemm_grouped":
        change["tokens"] = 8
    assert call(fn, **change) == lq.LQ_ERR_CUDA


@pytest.mark.parametrize("fn,change", [("lq_gemm_grouped", {"tokens": LAST, "K": 32, "out": 2}), ("lq_group_rows", {"tokens": 1, "topk": LAST}),
                                       ("lq_combine_rows", {"tokens": 1, "topk": LAST}), ("lq_combine_rows", {"n": 1, "width": LAST, "tokens": 1})])
def test_largest_counts_pass_the_checks(fn, change, monkeypatch):
    import bit_lifted_gemm_b200 as lq
    monkeypatch.setenv("LQ_FAULT", "launch")
    # one TiB between the buffers
    apart = {k: ctypes.c_void_p((i + 1) << 40) for i, (k, v) in enumerate(BASE[fn].items()) if isinstance(v, ctypes.c_void_p)}
    assert call(fn, **apart, **change) == lq.LQ_ERR_CUDA


@pytest.mark.parametrize("fn,outputs", [("lq_gemm_epilogue", ["o", "workspace"]), ("lq_gemv_epilogue", ["o", "workspace"]),
                                        ("lq_gemm_grouped", ["o", "workspace"]),
                                        ("lq_group_rows", ["offsets", "rows", "slots"]), ("lq_combine_rows", ["o"])])
def test_outputs_may_not_overlap(fn, outputs, monkeypatch):
    import bit_lifted_gemm_b200 as lq
    monkeypatch.setenv("LQ_FAULT", "launch")
    for o in outputs:
        for key, v in BASE[fn].items():
            if isinstance(v, ctypes.c_void_p) and key != o:
                assert call(fn, **{o: v}) == lq.LQ_ERR_INVALID_ARG, (o, key)


def test_inputs_may_overlap(monkeypatch):
    import bit_lifted_gemm_b200 as lq
    monkeypatch.setenv("LQ_FAULT", "launch")
    assert call("lq_gemm_epilogue", bias=far(1)) == lq.LQ_ERR_CUDA
    assert call("lq_combine_rows", residual=far(0)) == lq.LQ_ERR_CUDA


def test_workspace_sizes():
    import bit_lifted_gemm_b200 as lq
    assert lq.gemm_epilogue_workspace_size(13824, 12288, 2048) >= 1
    assert lq.gemv_epilogue_workspace_size(13824, 12288, 16) >= 1
    assert lq.gemm_grouped_workspace_size(8, 4096, 10240, 8192) >= 1
    assert lq.gemm_epilogue_workspace_size(8, 48, 1) == 0
    assert lq.gemm_epilogue_workspace_size(0, 64, 1) == 0
    assert lq.gemv_epilogue_workspace_size(8, 64, 17) == 0
    assert lq.gemm_grouped_workspace_size(4097, 8, 64, 1) == 0
    assert lq.gemm_grouped_workspace_size(4, 8, 64, 0) == 0
    need = lq.gemv_epilogue_workspace_size(300, 1536, 5)
    import os
    os.environ["LQ_FAULT"] = "launch"
    try:
        big = dict(out=300, K=1536, tokens=5)
        assert call("lq_gemv_epilogue", bytes=need, **big) == lq.LQ_ERR_CUDA
        assert call("lq_gemv_epilogue", bytes=need - 1, **big) == lq.LQ_ERR_INVALID_ARG
    finally:
        del os.environ["LQ_FAULT"]


def test_plain_layer_against_hand_values():
    packed = np.array([[0b101], [0xFFFFFFFF]], np.uint32)
    u = np.zeros((1, 32))
    u[0, :3] = 1, 2, 4
    z = plain.layer(packed, np.array([2.0, 1.0]), u)[0]
    assert z.tolist() == [[2 * (1 - 2 + 4), 7.0]]
    assert plain.layer(packed, np.array([2.0, 1.0]), u, glu=True, bias=np.array([1.0, -1.0]))[0].tolist() == [[7.0 * 6.0]]


def test_plain_group_and_combine_against_hand_values():
    offsets, rows, slots = plain.group(np.array([[1, 0], [1, -1], [0, 5]]), 2)
    assert offsets.tolist() == [0, 2, 4] and rows.tolist() == [0, 2, 0, 1, -1, -1]
    assert slots.tolist() == [[2, 0], [3, -1], [1, -1]]
    y = np.arange(8.0).reshape(4, 2)
    o, _ = plain.combine(y, slots, np.full((3, 2), 0.5))
    assert o.tolist() == [[0.5 * 4 + 0, 0.5 * 5 + 0.5], [3.0, 3.5], [1.0, 1.5]]


def test_experts_block_checks_its_widths():
    import torch
    from bit_lifted_gemm_b200.experts import ExpertMLP, interleave_rows
    gate, up = torch.zeros((2, 8, 3), dtype=torch.int32), torch.ones((2, 8, 3), dtype=torch.int32)
    both = interleave_rows(gate, up)
    assert both.shape == (2, 16, 3) and both[0, :, 0].tolist() == [0, 1] * 8
    with pytest.raises(ValueError):
        interleave_rows(gate, up[:, :4])
    M = torch.zeros((10, 24))
    s = torch.zeros((2, 16))
    block = ExpertMLP(torch.zeros((2, 20, 3), dtype=torch.int32), torch.zeros((2, 20)),
                      torch.zeros((2, 40, 1), dtype=torch.int32), torch.zeros((2, 40)), M)
    x, ids, w = torch.zeros((5, 40), dtype=torch.bfloat16), torch.zeros((5, 2), dtype=torch.int32), torch.zeros((5, 2))
    for bad in ((x[:4], ids, w), (x, ids, w[:4]), (x, ids[:, 0], w[:, 0]), (x[:, :32], ids, w), (x.float(), ids, w)):
        with pytest.raises(ValueError, match="must be"):
            block.step(*bad)
    with pytest.raises(ValueError):  # model = 40 channels lift to 96 columns = 3 words, hidden = 8 is no multiple of d
        ExpertMLP(both, s, torch.zeros((2, 40, 1), dtype=torch.int32), s, M)


OVER = 2 ** 32 + 8  # as a C int this is 8, a count that the library takes


@pytest.mark.parametrize("which", ["gemm out", "gemm tokens", "gemv out", "grouped n", "grouped out", "ids", "experts", "y", "width", "slots"])
def test_counts_past_32_bits_are_refused(which):
    """The binding's own check, before it asks for a device: tensors without storage stand for the large ones."""
    import torch

    import bit_lifted_gemm_b200 as lq

    def t(shape, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="meta")

    i32, bf = torch.int32, torch.bfloat16
    call = {
        "gemm out": lambda: lq.gemm_epilogue(t((OVER, 1), i32), t((OVER,)), t((1, 32), bf)),
        "gemm tokens": lambda: lq.gemm_epilogue(t((4, 1), i32), t((4,)), t((OVER, 32), bf)),
        "gemv out": lambda: lq.gemv_epilogue(t((OVER, 1), i32), t((OVER,)), t((1, 32))),
        "grouped n": lambda: lq.gemm_grouped(t((2, 1, 1), i32), t((2, 1)), t((8, 32), bf), t((3,), i32), OVER),
        "grouped out": lambda: lq.gemm_grouped(t((2, OVER, 1), i32), t((2, OVER)), t((8, 32), bf), t((3,), i32), 8),
        "ids": lambda: lq.group_rows(t((OVER, 1), i32), 4),
        "experts": lambda: lq.group_rows(t((4, 2), i32), OVER),
        "y": lambda: lq.combine_rows(t((OVER, 1)), t((4, 2), i32), t((4, 2))),
        "width": lambda: lq.combine_rows(t((1, OVER)), t((4, 2), i32), t((4, 2))),
        "slots": lambda: lq.combine_rows(t((4, 1)), t((OVER, 1), i32), t((OVER, 1))),
    }[which]
    with pytest.raises(lq.LQError, match="LQ_ERR_INVALID_ARG"):
        call()


def test_workspace_sizes_of_counts_past_32_bits():
    import bit_lifted_gemm_b200 as lq
    for over in (OVER, -OVER):
        assert lq.gemm_epilogue_workspace_size(over, 64, 4) == lq.gemm_epilogue_workspace_size(8, 64, over) == 0
        assert lq.gemv_epilogue_workspace_size(over, 64, 4) == lq.gemv_epilogue_workspace_size(8, 64 + 2 * over, 4) == 0
        assert lq.gemm_grouped_workspace_size(2, over, 64, 4) == lq.gemm_grouped_workspace_size(2, 8, 64, over) == 0


def test_experts_block_checks_what_the_lift_reads():
    """M and the whitening blocks go to kernels that take their extents from the other tensors' shapes."""
    import torch

    from bit_lifted_gemm_b200.experts import ExpertMLP
    i32 = torch.int32
    layers = (torch.zeros((2, 40, 2), dtype=i32), torch.zeros((2, 40)), torch.zeros((2, 40, 2), dtype=i32), torch.zeros((2, 40)))
    M = torch.zeros((20, 24))  # model = 40 and hidden = 20 channels lift to 48 and 24 columns: 64 and 32
    layers = (layers[0], layers[1], layers[2][:, :, :1].contiguous(), layers[3])
    block = ExpertMLP(*layers, M, tinv_in=torch.zeros((5, 8, 8)), tinv_hidden=torch.zeros((5, 4, 4)))
    for bad in (M.double(), M.t().contiguous().t(), M[0]):
        with pytest.raises(ValueError):
            ExpertMLP(*layers, bad)
    z = torch.zeros
    for model, hidden in (((5, 4, 4), (5, 8, 8)), ((4, 8, 8), None), (None, (4, 4, 4)), ((40, 40), None), ((5, 8, 4), None),
                          ((1, 0, 0), None), ((3, 16, 16), None)):
        with pytest.raises(ValueError, match="tinv"):
            ExpertMLP(*layers, M, tinv_in=None if model is None else z(model), tinv_hidden=None if hidden is None else z(hidden))
    for bad in (z((5, 8, 8), dtype=torch.float64), z((5, 8, 8)).transpose(1, 2), z((5, 8, 8), device="meta")):
        with pytest.raises(ValueError, match="tinv"):
            ExpertMLP(*layers, M, tinv_in=bad)
    x, ids, w = z((5, 40), dtype=torch.bfloat16, device="meta"), z((5, 2), dtype=i32), z((5, 2))
    with pytest.raises(ValueError, match="device"):
        block.step(x, ids, w)


def _body(text, name):
    """The braces after the first definition of a function of this name."""
    import re
    start = next(m.end() for m in re.finditer(rf"\b{name}\s*\(", text)
                 if re.match(r"[^;{]*\)\s*\{", text[m.end():], re.S))
    at = text.index("{", start)
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at: i + 1]


def test_debug_build_checks_the_operators_kernels():
    """What the header says the debug build checks of these operators is checked, and every flag is read."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_lifted_gemm_b200", "csrc")

    def read(f):
        with open(os.path.join(csrc, f)) as h:
            return h.read()

    for f, functions in (("lq_epilogue.cuh", ["finish_row"]), ("lq_gemv.cu", ["widen_kernel"]), ("lq_grouped_mma.cu", ["mma_kernel"]),
                         ("lq_grouped_tc.cu", ["store_row", "gather_kernel", "tc_kernel"]),
                         ("lq_rows.cu", ["group_kernel", "combine_kernel"])):
        for name in functions:
            assert "LQ_IN_BOUNDS" in _body(read(f), name), (f, name)
    flags = set()
    for f in sorted(os.listdir(csrc)):
        text = read(f)
        if f.endswith(".cu"):
            shared = [h for h in re.findall(r'#include "(\w+\.cuh)"', text) if h != "lq_debug.cuh" and "LQ_IN_BOUNDS" in read(h)]
            if "LQ_IN_BOUNDS" in text or shared:
                flags |= set(re.findall(r"^LQ_DEBUG_FLAG_TAKE\((\w+)\)", text, re.M)) or {"none in " + f}
    for name in flags:
        assert f"lq::{name}()" in read("lq_api.cu") and f"unsigned {name}();" in read("lq_internal.h"), name


def test_grouped_workspace_without_rows(monkeypatch):
    """Only rows are copied to the workspace of a product of many slots an expert; without them it needs next to nothing."""
    import bit_lifted_gemm_b200 as lq
    monkeypatch.setenv("LQ_FAULT", "launch")
    for E, out, K, n in ((8, 4096, 10240, 8192), (3, 8, 64, 60), (5, 130, 1056, 70), (8, 11008, 10240, 2), (32, 2816, 4096, 128),
                         (4, 256, 40960, 4)):
        with_rows, without = lq.gemm_grouped_workspace_size(E, out, K, n), lq.gemm_grouped_workspace_size(E, out, K, n, rows=False)
        assert 256 <= without <= with_rows
        if n >= 9 * E:
            assert without == 256 and with_rows == max(256, n * K * 2)
        sizes = dict(experts=E, out=out, K=K, n=n, tokens=n)
        for rows, need in ((far(3), with_rows), (None, without)):
            assert call("lq_gemm_grouped", bytes=need, rows=rows, **sizes) == lq.LQ_ERR_CUDA
            assert call("lq_gemm_grouped", bytes=need - 1, rows=rows, **sizes) == lq.LQ_ERR_INVALID_ARG
    assert lq.gemm_grouped_workspace_size(4097, 8, 64, 1, rows=False) == 0
    assert lq.gemm_grouped_workspace_size(4, 8, 64, OVER, rows=False) == 0


def test_layer_workspace_stays_within_the_documented_bound():
    """include/lq.h states the most that a layer's partial sums take: every number of tiles, at steps of K from few to many.
    Nine to sixteen tokens of wide layers take the decode call's scratch beside u in fp32."""
    import os
    import re

    import bit_lifted_gemm_b200 as lq
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "lq.h")) as f:
        stated = [int(v.replace(",", "")) for v in re.findall(r"at most ([\d,]+)\s*\*?\s*bytes", f.read())]
    assert len(stated) == 1
    sizes = {(128 * blocks - 127 * ragged, K, tokens) for blocks in range(1, 300) for K in (64, 1056, 8192, 20480, 131072)
             for tokens in (17, 64, 100, 256, 300, 512, 1000) for ragged in (0, 1)}
    assert max(lq.gemm_epilogue_workspace_size(*size) for size in sizes) == stated[0]
    for out, K, tokens in ((18945, 20480, 16), (28672, 4096, 9), (131072, 131072, 12)):
        wide = 4 * K * tokens
        assert wide % 256 == 0
        assert lq.gemm_epilogue_workspace_size(out, K, tokens) == wide + lq.gemv_epilogue_workspace_size(out, K, tokens)


def _misses(got, z, act):
    want, tol = plain.activate_exact(z, act)
    return int((np.abs(got.astype(np.float64) - want) > tol + plain.U32 * np.abs(want)).sum())


def test_the_activations_bound_tells_forms_that_lose_the_tails():
    """The bound that the kernels' activations are held to lets fp32 evaluations of the exact forms pass and none that cancel
    or drop a tail."""
    import math
    f = np.float32
    z = np.linspace(-60, 60, 4001).astype(f)
    z64, tail = z.astype(np.float64), z < -3
    erf, erfc = (np.vectorize(v, otypes=[np.float64]) for v in (math.erf, math.erfc))
    x = f(0.70710678118654752) * z
    y = f(0.79788456080286536) * (z + f(0.044715) * z * z * z)
    with np.errstate(all="ignore"):
        assert _misses(f(0.5) * z * erfc(-x).astype(f), z64, "gelu") == 0
        assert _misses(z / (f(1) + np.exp(f(-2) * y)), z64, "gelu_tanh") == 0
        assert _misses(z / (f(1) + np.exp(-z)), z64, "silu") == 0
        assert _misses(f(0.5) * z * (f(1) + erf(x).astype(f)), z64, "gelu") > 100
        assert _misses(f(0.5) * z * (f(1) + np.tanh(y)), z64, "gelu_tanh") > 100
        for act, good in (("gelu", f(0.5) * z * erfc(-x).astype(f)), ("gelu_tanh", z / (f(1) + np.exp(f(-2) * y))),
                          ("silu", z / (f(1) + np.exp(-z)))):
            assert _misses(np.where(tail, f(0), good), z64, act) > 100
            assert _misses(good * f(1 + 2e-4), z64, act) > 1000
    # where float64 does not cancel both references are one
    near = np.abs(z64) < 3
    for act in ("gelu", "gelu_tanh", "silu", "relu", "none"):
        assert np.allclose(plain.activate_exact(z64, act)[0][near], plain.activate(z64, act)[near], rtol=1e-12, atol=0)
