"""Fused-epilogue products, grouped products, row grouping and row joining on the GPU against the plain float64
forms of operators_plain.py: sizes from one token and one word of K up, odd and unaligned ones, every
activation, gate, type, empty and uneven experts, indices and ids outside their range, NaN and Inf rows, mean-
shifted inputs, streams, graphs, workspaces in use by earlier calls, and the experts' block that runs them together."""

import numpy as np
import pytest

from tests import operators_plain as plain
from tests.gpu_common import dev, rel_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lq():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import bit_lifted_gemm_b200 as lq
    yield lq
    assert lq.get_device_status() == lq.LQ_OK


def bf16(x):
    """Rounded to bf16 (nearest even), as float32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return b.view(np.float32)


def gpu(x, as_bf16=False):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()
    return t.to(torch.bfloat16) if as_bf16 else t


def f64(t):
    return t.double().cpu().numpy()


def words(rng, shape):
    return rng.integers(0, 2 ** 32, shape, dtype=np.uint64).astype(np.uint32)


def ints(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def make_layer(rng, lead, out, K):
    return words(rng, lead + (out, K // 32)), rng.uniform(0.01, 0.03, lead + (out,)).astype(np.float32)


def run_layer(lq, rng, out, K, tokens, u_t, o_t, act, glu, with_bias, with_res, u=None, **kw):
    packed, s = make_layer(rng, (), out, K)
    u = rng.standard_normal((tokens, K)).astype(np.float32) if u is None else u
    u = bf16(u) if u_t == "bf16" else u
    bias = rng.standard_normal(out).astype(np.float32) if with_bias else None
    width = out // 2 if glu else out
    res = rng.standard_normal((tokens, width)).astype(np.float32) if with_res else None
    res = bf16(res) if with_res and o_t == "bf16" else res
    call = lq.gemv_epilogue if u_t == "f32" else lq.gemm_epilogue
    got = call(dev(packed), gpu(s), gpu(u, u_t == "bf16"), bias=None if bias is None else gpu(bias), act=act, glu=glu,
               residual=None if res is None else gpu(res, o_t == "bf16"), o_dtype=o_t, **kw)
    want, tol = plain.layer(packed, s.astype(np.float64), u, bias, act, glu, res)
    return got, want, tol


SIZES = [  # out, K, tokens
    (1, 32, 1), (2, 32, 1), (5, 64, 2), (16, 32, 3), (37, 96, 3), (33, 1024, 1), (128, 1024, 16), (129, 1056, 17),
    (510, 1568, 5), (1000, 2048, 8), (1000, 2048, 9), (640, 4096, 64), (1022, 3360, 65), (300, 1536, 130),
    (258, 2080, 300), (2050, 1536, 257), (4100, 512, 31), (96, 12288, 4), (130, 20480, 7), (512, 992, 1000)]


@pytest.mark.parametrize("out,K,tokens", SIZES)
@pytest.mark.parametrize("which", range(4))
def test_layer_epilogue(lq, out, K, tokens, which):
    rng = np.random.default_rng([1, out, K, tokens, which])
    acts = ["none", "relu", "gelu", "gelu_tanh", "silu", None]
    act = acts[(which + out + K // 32 + tokens) % 6]
    glu = out % 2 == 0 and which % 2 == 1
    u_t = "f32" if which >= 2 and tokens <= 16 else "bf16"
    o_t = ("bf16", "f32", "f32", "bf16")[which]
    got, want, tol = run_layer(lq, rng, out, K, tokens, u_t, o_t, act, glu, which != 1, which in (0, 3))
    plain.assert_close(f64(got), want, tol, o_t == "bf16")


@pytest.mark.parametrize("K", [32, 96, 160, 288, 384, 1056])
@pytest.mark.parametrize("tokens", [3, 8, 9, 64, 65, 128, 129, 260])
def test_many_tiles_of_few_steps(lq, K, tokens):
    """More tiles than the persistent kernels have CTAs, with one, odd and even numbers of k-steps each: the rings and
    their owners carry on from tile to tile."""
    out = 40000
    rng = np.random.default_rng([20, K, tokens])
    packed, s = make_layer(rng, (), out, K)
    u = bf16(rng.standard_normal((tokens, K)))
    rows = np.sort(rng.choice(out, 3000, replace=False))
    rows[-1], rows[0] = out - 1, 0
    want, tol = plain.layer(packed[rows], s[rows].astype(np.float64), u)
    args = dev(packed), gpu(s), gpu(u, True)
    first = lq.gemm_epilogue(*args)
    plain.assert_close(f64(first)[:, rows], want, tol, False)
    for _ in range(5):
        assert bool((lq.gemm_epilogue(*args) == first).all())


@pytest.mark.parametrize("each", [1, 5, 8, 20, 70, 150])
@pytest.mark.parametrize("K", [96, 288, 1120])
def test_many_experts_of_few_steps(lq, each, K):
    """The same over experts of uneven sizes, some empty."""
    rng = np.random.default_rng([21, each, K])
    E, out = 40, 1100
    sizes = rng.integers(0, 2 * each + 1, E)
    sizes[3], sizes[7] = 0, 2 * each
    case = grouped_case(rng, E, out, K, sizes, True)
    packed, s, offsets, n, rows, u = case
    got = call_grouped(lq, *case, o_dtype="f32")
    want, tol, _ = plain.grouped(packed, s.astype(np.float64), u, offsets, n, rows)
    plain.assert_close(f64(got), want, tol, False)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("glu", [False, True])
def test_activations_over_their_range(lq, act, glu):
    """z runs from -60 to 60 through the bias alone (u = 0): the activation's own accuracy, tails included."""
    out, K = 4096, 64
    rng = np.random.default_rng(2)
    bias = np.linspace(-60, 60, out).astype(np.float32)
    packed, s = make_layer(rng, (), out, K)
    for call, dt in ((lq.gemv_epilogue, False), (lq.gemm_epilogue, True)):
        got = call(dev(packed), gpu(s), gpu(np.zeros((2, K)), dt), bias=gpu(bias), act=act, glu=glu)
        want, tol = plain.layer(packed, s, np.zeros((2, K)), bias, act, glu)
        # float64 erf and tanh cancel below 2^-53: an absolute floor far under the fp32 step of the values near 0
        plain.assert_close(f64(got), want, tol + 1e-13, False)


@pytest.mark.parametrize("tokens", [1, 2, 7, 16, 17, 40, 64, 200, 300])
@pytest.mark.parametrize("u_t", ["f32", "bf16"])
def test_integer_inputs_are_exact(lq, tokens, u_t):
    """Integer u, s = 1: every partial sum is an integer below 2^24, so any order gives the exact result."""
    if u_t == "f32" and tokens > 16:
        pytest.skip("fp32 u is the decode form, at most 16 columns")
    out, K = 401, 2240
    rng = np.random.default_rng([3, tokens])
    packed = words(rng, (out, K // 32))
    u = rng.integers(-8, 9, (tokens, K)).astype(np.float32)
    call = lq.gemv_epilogue if u_t == "f32" else lq.gemm_epilogue
    got = call(dev(packed), gpu(np.ones(out)), gpu(u, u_t == "bf16"))
    assert np.array_equal(f64(got), u.astype(np.float64) @ plain.signs(packed).T)


@pytest.mark.parametrize("tokens", [1, 5, 16, 33, 100])
def test_mean_shifted_inputs(lq, tokens):
    """u = 1 + noise: the sums of the two signs are large and cancel. No order keeps every partial sum small, so
    the bound is 2^-23 (K/16 + 16) of the sum of |u|, times s."""
    out, K = 300, 4096
    rng = np.random.default_rng([4, tokens])
    packed, s = make_layer(rng, (), out, K)
    u = bf16(1 + 0.1 * rng.standard_normal((tokens, K)))
    want = (u.astype(np.float64) @ plain.signs(packed).T) * s
    for call, is_bf in ((lq.gemm_epilogue, True),) + (((lq.gemv_epilogue, False),) if tokens <= 16 else ()):
        got = f64(call(dev(packed), gpu(s), gpu(u, is_bf)))
        tol = (K / 16 + 16) * 2.0 ** -23 * s * np.abs(u).sum(1)[:, None]
        plain.assert_close(got, want, tol, False)
        assert rel_err(got, want) <= 1e-5


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1.0, 1e12, 1e30])
def test_fp32_decode_keeps_its_range(lq, scale):
    """fp32 u of any magnitude, with one element 10^4 times the rest, at fp32 accuracy."""
    out, K = 200, 2048
    rng = np.random.default_rng(5)
    packed, s = make_layer(rng, (), out, K)
    for batch in (1, 3, 16):
        u = (rng.standard_normal((batch, K)) * scale).astype(np.float32)
        u[:, 77] *= 1e4
        want, tol = plain.layer(packed, s.astype(np.float64), u)
        # the large element enters every partial sum: sqrt(sum u^2) in tol covers it
        plain.assert_close(f64(lq.gemv_epilogue(dev(packed), gpu(s), gpu(u))), want, tol, False)


@pytest.mark.parametrize("tokens", [3, 16, 40, 150])
def test_nan_and_inf_rows_stay_in_their_rows(lq, tokens):
    out, K = 260, 1056
    rng = np.random.default_rng([6, tokens])
    packed, s = make_layer(rng, (), out, K)
    clean = bf16(rng.standard_normal((tokens, K)))
    u = clean.copy()
    u[1, 500] = np.nan
    u[2, 7], u[2, 1000] = np.inf, -np.inf
    u[0, 3] = np.inf
    sg = plain.signs(packed)
    for call, is_bf in ((lq.gemm_epilogue, True),) + (((lq.gemv_epilogue, False),) if tokens <= 16 else ()):
        base = f64(call(dev(packed), gpu(s), gpu(clean, is_bf)))
        got = f64(call(dev(packed), gpu(s), gpu(u, is_bf)))
        assert np.array_equal(got[3:], base[3:])
        assert np.isnan(got[1]).all()
        assert np.array_equal(got[0], np.where(sg[:, 3] > 0, np.inf, -np.inf))
        opposed = sg[:, 7] == sg[:, 1000]  # +inf and -inf in one sum
        assert np.isnan(got[2][opposed]).all()
        assert np.array_equal(got[2][~opposed], np.where(sg[~opposed, 7] > 0, np.inf, -np.inf))


def grouped_case(rng, E, out, K, sizes, gather, tokens=None):
    packed, s = make_layer(rng, (E,), out, K)
    offsets = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    n = int(offsets[-1])
    tokens = (tokens or max(1, n // 2 + 1)) if gather else n
    rows = rng.integers(0, tokens, n).astype(np.int32) if gather else None
    u = bf16(rng.standard_normal((tokens, K)))
    return packed, s, offsets, n, rows, u


def call_grouped(lq, packed, s, offsets, n, rows, u, bias=None, **kw):
    return lq.gemm_grouped(dev(packed), gpu(s), gpu(u, True), ints(offsets), n, rows=None if rows is None else ints(rows),
                           bias=None if bias is None else gpu(bias), **kw)


GROUPS = [  # experts' sizes, out, K
    ([1], 1, 32), ([0, 1], 2, 32), ([1, 0, 0, 1], 50, 96), ([3, 5, 2, 0, 1, 7], 130, 1024), ([16, 17, 0, 1], 258, 1056),
    ([0, 0, 40], 300, 2080), ([8] * 16, 96, 512), ([100, 0, 3, 200], 512, 1536), ([1] * 40, 64, 2240),
    ([257, 1, 128, 0, 33], 254, 768), ([5, 300, 0, 0, 64, 65, 256], 1026, 992), ([2, 1], 2816, 10240),
    ([0, 600, 1], 384, 4096)]


@pytest.mark.parametrize("sizes,out,K", GROUPS)
@pytest.mark.parametrize("which", range(4))
def test_grouped(lq, sizes, out, K, which):
    rng = np.random.default_rng([7, out, K, which])
    case = grouped_case(rng, len(sizes), out, K, sizes, which % 2 == 0)
    bias = rng.standard_normal((len(sizes), out)).astype(np.float32) if which >= 2 else None
    glu = out % 2 == 0 and which in (0, 3)
    act, o_t = ("silu", None, "gelu", "relu")[which], ("bf16", "f32", "bf16", "f32")[which]
    got = call_grouped(lq, *case, bias=bias, act=act, glu=glu, o_dtype=o_t)
    packed, s, offsets, n, rows, u = case
    want, tol, written = plain.grouped(packed, s.astype(np.float64), u, offsets, n, rows, bias, act, glu)
    assert written.all()
    plain.assert_close(f64(got), want, tol, o_t == "bf16")


@pytest.mark.parametrize("K", [96, 1056])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_slots_and_rows_outside(lq, K, gather):
    """Slots of no expert keep their contents, offsets outside 0..n are cut, rows outside u count as zero rows."""
    import torch
    rng = np.random.default_rng([8, K])
    E, out, n = 5, 70, 90
    packed, s = make_layer(rng, (E,), out, K)
    bias = rng.standard_normal((E, out)).astype(np.float32)
    offsets = np.array([-3, 4, 4, 40, 70, 70 if gather else 500], np.int32)
    tokens = 20 if gather else n
    rows = rng.integers(-4, 26, n).astype(np.int32) if gather else None
    u = bf16(rng.standard_normal((tokens, K)))
    for o_t in ("f32", "bf16"):
        out_t = torch.full((n, out), 7.5, device="cuda", dtype=torch.float32 if o_t == "f32" else torch.bfloat16)
        call_grouped(lq, packed, s, offsets, n, rows, u, bias=bias, out=out_t)
        want, tol, written = plain.grouped(packed, s.astype(np.float64), u, offsets, n, rows, bias)
        got = f64(out_t)
        assert (got[~written] == 7.5).all()
        plain.assert_close(got[written], want[written], tol[written], o_t == "bf16")


def test_grouped_nothing_routed(lq):
    import torch
    rng = np.random.default_rng(9)
    packed, s = make_layer(rng, (3,), 64, 128)
    out_t = torch.full((10, 64), 2.0, device="cuda")
    call_grouped(lq, packed, s, np.zeros(4, np.int32), 10, np.full(10, -1), bf16(rng.standard_normal((4, 128))), out=out_t)
    assert bool((out_t == 2.0).all())


@pytest.mark.parametrize("out,K,tokens", [(130, 12288, 9), (1001, 8224, 64), (640, 10240, 100), (257, 16384, 130), (258, 20480, 300),
                                          (4096, 10240, 33), (2050, 20512, 512)])
def test_layers_cut_along_k(lq, out, K, tokens):
    """Few tiles and a long K: the parts of a tile are added in order, whatever the workspace held; values, gates, exact
    integers, and infinities that meet from different parts."""
    import torch
    rng = np.random.default_rng([25, out, K, tokens])
    need = lq.gemm_epilogue_workspace_size(out, K, tokens)
    assert need > 256
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    for act, glu, o_t in (("gelu", False, "f32"), ("silu", out % 2 == 0, "bf16")):
        got, want, tol = run_layer(lq, rng, out, K, tokens, "bf16", o_t, act, glu, True, True, workspace=ws)
        plain.assert_close(f64(got), want, tol, o_t == "bf16")
    packed, _ = make_layer(rng, (), out, K)
    weights = dev(packed), gpu(np.ones(out))
    u = rng.integers(-8, 9, (tokens, K)).astype(np.float32)
    got = lq.gemm_epilogue(*weights, gpu(u, True), workspace=ws)
    assert np.array_equal(f64(got), u.astype(np.float64) @ plain.signs(packed).T)
    x = gpu(rng.standard_normal((tokens, K)), True)
    first = lq.gemm_epilogue(*weights, x, workspace=ws)
    for _ in range(20):
        assert torch.equal(lq.gemm_epilogue(*weights, x, workspace=ws), first)
    u[1, 5], u[1, K - 3] = np.inf, -np.inf
    got = f64(lq.gemm_epilogue(*weights, gpu(u, True), workspace=ws))[1]
    sg = plain.signs(packed)
    opposed = sg[:, 5] == sg[:, K - 3]
    assert np.isnan(got[opposed]).all() and np.array_equal(got[~opposed], np.where(sg[~opposed, 5] > 0, np.inf, -np.inf))


def test_layers_cut_along_k_in_graphs_and_streams(lq):
    import torch
    rng = np.random.default_rng(26)
    out, K, tokens = 384, 12288, 64
    packed, s = make_layer(rng, (), out, K)
    weights = dev(packed), gpu(s)
    inputs = [gpu(rng.standard_normal((tokens, K)), True) for _ in range(2)]
    alone = [lq.gemm_epilogue(*weights, u) for u in inputs]
    spaces = [torch.empty(lq.gemm_epilogue_workspace_size(out, K, tokens), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(a) for a in alone]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            for _ in range(3):
                lq.gemm_epilogue(*weights, inputs[i], out=outs[i], workspace=spaces[i])
        graphs.append(g)
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i], alone[i])


def test_grouped_calls_without_slots_leave_the_next_call_alone(lq):
    """On one workspace: what calls without any slot prepare there must not come after what a call with slots does."""
    import torch
    rng = np.random.default_rng(24)
    E, out, K, n = 4, 256, 40960, 4
    packed, s, offsets, _, rows, u = grouped_case(rng, E, out, K, [1] * 4, True)
    weights = dev(packed), gpu(s)
    other, here = gpu(-u, True), gpu(u, True)
    none, each, at = ints(np.zeros(E + 1)), ints(offsets), ints(rows)
    alone = lq.gemm_grouped(*weights, here, each, n, rows=at)
    ws = torch.empty(lq.gemm_grouped_workspace_size(E, out, K, n), dtype=torch.uint8, device="cuda")
    unused = torch.full((n, out), 7.5, device="cuda")
    for _ in range(50):
        for _ in range(3):
            lq.gemm_grouped(*weights, other, none, n, rows=at, out=unused, workspace=ws)
        got = lq.gemm_grouped(*weights, here, each, n, rows=at, workspace=ws)
        assert torch.equal(got, alone)
    assert bool((unused == 7.5).all())


@pytest.mark.parametrize("sizes", [[3, 0, 9, 1], [30, 70, 5, 250]])
def test_grouped_integer_inputs_are_exact(lq, sizes):
    rng = np.random.default_rng(10)
    packed, s, offsets, n, rows, u = grouped_case(rng, 4, 129, 1120, sizes, True)
    u = rng.integers(-8, 9, u.shape).astype(np.float32)
    got = call_grouped(lq, packed, np.ones_like(s), offsets, n, rows, u)
    want, _, _ = plain.grouped(packed, np.ones_like(s), u, offsets, n, rows)
    assert np.array_equal(f64(got), want)


@pytest.mark.parametrize("K", [128, 1024, 1152, 4096, 1056])
@pytest.mark.parametrize("sizes", [[1], [0, 2, 0, 1, 0, 0, 1], [1] * 7 + [0] * 60, [9] + [0] * 40, [0, 70, 0, 3] + [0] * 60])
def test_grouped_few_slots(lq, sizes, K):
    """Fewer slots than experts, alone or several in one expert: a share of the SMs to each slot."""
    rng = np.random.default_rng([22, len(sizes), K])
    E, out = len(sizes), 150
    packed, s, offsets, n, rows, u = grouped_case(rng, E, out, K, sizes, True)
    bias = rng.standard_normal((E, out)).astype(np.float32)
    for act, glu, o_t in (("gelu", False, "f32"), ("silu", True, "bf16")):
        got = call_grouped(lq, packed, s, offsets, n, rows, u, bias=bias, act=act, glu=glu, o_dtype=o_t)
        want, tol, _ = plain.grouped(packed, s.astype(np.float64), u, offsets, n, rows, bias, act, glu)
        plain.assert_close(f64(got), want, tol, o_t == "bf16")


@pytest.mark.parametrize("K", [128, 20480])
def test_grouped_few_slots_outside(lq, K):
    """Slots of no expert keep their contents, rows outside u count as zero rows, NaN and Inf stay in their slots."""
    import torch
    rng = np.random.default_rng([23, K])
    E, out, n, tokens = 9, 2050, 6, 4
    packed, s = make_layer(rng, (E,), out, K)
    bias = rng.standard_normal((E, out)).astype(np.float32)
    u = bf16(rng.standard_normal((tokens, K)))
    u[1, 5], u[2, 7], u[2, 9] = np.nan, np.inf, np.inf
    rows = np.array([0, 1, 2, 4, -1, 3], np.int32)  # slot 5 belongs to no expert
    offsets = np.array([0, 0, 1, 3, 3, 3, 4, 5, 5, 5], np.int32)
    o = torch.full((n, out), 7.5, device="cuda")
    call_grouped(lq, packed, s, offsets, n, rows, u, bias=bias, out=o)
    got = f64(o)
    clean = np.where(np.isfinite(u), u, 0).astype(np.float32)
    want, tol, written = plain.grouped(packed, s.astype(np.float64), clean, offsets, n, rows, bias)
    assert written.tolist() == [True] * 5 + [False] and (got[5] == 7.5).all()
    for i in (0, 3, 4):
        plain.assert_close(got[i: i + 1], want[i: i + 1], tol[i: i + 1], False)
    assert np.isnan(got[1]).all()
    sg = plain.signs(packed[2])
    opposed = sg[:, 7] != sg[:, 9]
    assert np.isnan(got[2][opposed]).all()
    assert np.array_equal(got[2][~opposed], np.where(sg[~opposed, 7] > 0, np.inf, -np.inf))


def test_grouped_more_experts_than_a_warp(lq):
    rng = np.random.default_rng(11)
    sizes = rng.integers(0, 4, 300)
    packed, s, offsets, n, rows, u = grouped_case(rng, 300, 48, 160, sizes, True)
    got = call_grouped(lq, packed, s, offsets, n, rows, u, act="silu", glu=True)
    want, tol, _ = plain.grouped(packed, s.astype(np.float64), u, offsets, n, rows, None, "silu", True)
    plain.assert_close(f64(got), want, tol, False)


def test_outputs_past_32_bit_offsets(lq):
    """n * width over 2^31 elements: the last rows are right."""
    import torch
    out, K, n = 65536, 32, 33000
    rng = np.random.default_rng(12)
    packed, s = make_layer(rng, (2,), out, K)
    u = bf16(rng.standard_normal((n, K)))
    offsets = np.array([0, 16000, n], np.int32)
    o = torch.empty((n, out), dtype=torch.bfloat16, device="cuda")
    call_grouped(lq, packed, s, offsets, n, None, u, out=o)
    for at in (0, 15999, 16000, 32767, 32768, n - 1):
        want, tol = plain.layer(packed[int(at >= 16000)], s[int(at >= 16000)].astype(np.float64), u[at: at + 1])
        plain.assert_close(f64(o[at: at + 1]), want, tol, True)


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (1, 2, 8), (16, 2, 8), (33, 4, 300), (1000, 8, 128), (5, 3, 4096),
                                                 (4096, 2, 8), (20011, 7, 61), (70000, 2, 5), (300, 2, 40),
                                                 (5000, 8, 4096), (2000, 2, 4096)])
@pytest.mark.parametrize("outside", [False, True])
def test_group_rows(lq, tokens, topk, experts, outside):
    rng = np.random.default_rng([13, tokens])
    lo, hi = (-2, experts + 2) if outside else (0, experts)
    ids = rng.integers(lo, hi, (tokens, topk)).astype(np.int32)
    if outside and tokens == 16:
        ids[:] = -1  # nothing kept
    got = lq.group_rows(ints(ids), experts)
    for g, w in zip(got, plain.group(ids, experts)):
        assert np.array_equal(g.cpu().numpy(), w)


def test_group_rows_extreme_ids(lq):
    ids = np.array([[2 ** 31 - 1, -2 ** 31, 0, 1, 0, 0]], np.int32)
    for g, w in zip(lq.group_rows(ints(ids), 2), plain.group(ids, 2)):
        assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("tokens,topk,width,n", [(1, 1, 1, 1), (3, 2, 7, 5), (16, 2, 5120, 32), (100, 8, 1001, 700),
                                                 (257, 4, 1032, 1028), (9, 70, 36, 40)])
@pytest.mark.parametrize("o_t", ["f32", "bf16"])
@pytest.mark.parametrize("with_res", [False, True])
def test_combine_rows(lq, tokens, topk, width, n, o_t, with_res):
    rng = np.random.default_rng([14, tokens, width])
    r = bf16 if o_t == "bf16" else (lambda x: x.astype(np.float32))
    y, res = r(rng.standard_normal((n, width))), r(rng.standard_normal((tokens, width)))
    slots = rng.integers(-2, n + 2, (tokens, topk)).astype(np.int32)
    slots[0] = -1  # a token with no expert
    w = rng.uniform(-1, 1, (tokens, topk)).astype(np.float32)
    wn = np.where((slots >= 0) & (slots < n), w, np.nan).astype(np.float32)  # weights of skipped slots are not used
    got = lq.combine_rows(gpu(y, o_t == "bf16"), ints(slots), gpu(wn), residual=gpu(res, o_t == "bf16") if with_res else None)
    want, tol = plain.combine(y, slots, w, res if with_res else None)
    plain.assert_close(f64(got), want, tol, o_t == "bf16")


def expert_mlp(lq, rng, E, model, hidden, d, D):
    from bit_lifted_gemm_b200.experts import ExpertMLP, interleave_rows
    K1, K2 = lq.lifted_dim(model, d, D), lq.lifted_dim(hidden, d, D)
    gate, gs = make_layer(rng, (E,), hidden, K1)
    up, us = make_layer(rng, (E,), hidden, K1)
    down, ds = make_layer(rng, (E,), model, K2)
    M = (rng.standard_normal((d, D)) / np.sqrt(D)).astype(np.float32)
    mlp = ExpertMLP(interleave_rows(dev(gate), dev(up)), interleave_rows(gpu(gs), gpu(us)), dev(down), gpu(ds), gpu(M))
    return mlp, (gate, gs, up, us, down, ds, M)


def lift(x, M, K):
    d, D = M.shape
    u = np.zeros((x.shape[0], K))
    v = (x.reshape(x.shape[0], -1, d) @ M).reshape(x.shape[0], -1)
    u[:, : v.shape[1]] = v
    return u


def expert_mlp_plain(lq, parts, x, ids, w):
    """Rounded to bf16 where the block's tensors are bf16."""
    gate, gs, up, us, down, ds, M = (np.asarray(p) for p in parts)
    M = M.astype(np.float64)
    u = bf16(lift(x.astype(np.float64), M, gate.shape[2] * 32)).astype(np.float64)
    o = x.astype(np.float64)
    for t in range(x.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < gate.shape[0]:
                continue
            g, v = gs[e] * (plain.signs(gate[e]) @ u[t]), us[e] * (plain.signs(up[e]) @ u[t])
            h = bf16(plain.activate(g, "silu") * v).astype(np.float64)
            uh = bf16(lift(h[None], M, down.shape[2] * 32)).astype(np.float64)[0]
            o[t] = o[t] + float(w[t, j]) * bf16(ds[e] * (plain.signs(down[e]) @ uh))
    return o


@pytest.mark.parametrize("tokens,topk", [(1, 2), (9, 2), (70, 3)])
def test_experts_block(lq, tokens, topk):
    """The four operators and the lift as they run together. The plain form rounds to bf16 at the same places, so
    what differs is fp32 sums that fall on the other side of a rounding: one bf16 step (2^-7) in a few elements of h and
    of the lifted rows, averaged over the products that follow, and one step of the result: under three steps of the
    part that the experts add, plus half a step of o."""
    rng = np.random.default_rng([15, tokens])
    E, model, hidden = 6, 320, 200
    mlp, parts = expert_mlp(lq, rng, E, model, hidden, 10, 24)
    x = bf16(rng.standard_normal((tokens, model)))
    ids = np.argsort(rng.random((tokens, E)), axis=1)[:, :topk].astype(np.int32)
    ids[0, 0] = -1
    w = rng.uniform(0.1, 1, (tokens, topk)).astype(np.float32)
    got = f64(mlp.step(gpu(x, True), ints(ids), gpu(w)))
    want = expert_mlp_plain(lq, parts, x, ids, w)
    added = np.abs(want - x).max(1, keepdims=True)
    assert (np.abs(got - want) <= plain.UBF * np.abs(want) + 3 * 2.0 ** -7 * added).all()
    assert rel_err(got, want) <= 2 ** -8


def test_experts_block_in_a_graph_and_on_another_stream(lq):
    """Captured once, replayed on new inputs with other group sizes; and on a side stream: the same bits as eager."""
    import torch
    rng = np.random.default_rng(16)
    E, model, hidden, tokens, topk = 6, 320, 200, 24, 2
    mlp, _ = expert_mlp(lq, rng, E, model, hidden, 10, 24)

    def inputs():
        ids = rng.integers(-1, E, (tokens, topk)).astype(np.int32)
        return gpu(rng.standard_normal((tokens, model)), True), ints(ids), gpu(rng.uniform(0.1, 1, (tokens, topk)))

    x, ids, w = inputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = mlp.step(x, ids, w)
    on_side = mlp.step(x, ids, w, stream=side)
    side.synchronize()
    assert torch.equal(eager, on_side)
    graphs = []
    for _ in range(2):  # two graphs of the same block, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = mlp.step(x, ids, w)
        graphs.append((g, o))
    for _ in range(3):
        for new, old in zip(inputs(), (x, ids, w)):
            old.copy_(new)
        want = mlp.step(x, ids, w)
        for g, o in graphs:
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want)


@pytest.mark.parametrize("tokens,u_t", [(1, "f32"), (16, "f32"), (2, "bf16"), (16, "bf16"), (50, "bf16"), (300, "bf16")])
def test_workspace_contents_do_not_matter_and_results_repeat(lq, tokens, u_t):
    import torch
    rng = np.random.default_rng([17, tokens])
    out, K = 700, 2240
    packed, s = make_layer(rng, (), out, K)
    u = gpu(rng.standard_normal((tokens, K)), u_t == "bf16")
    size = (lq.gemv_epilogue_workspace_size if u_t == "f32" else lq.gemm_epilogue_workspace_size)(out, K, tokens)
    call = lq.gemv_epilogue if u_t == "f32" else lq.gemm_epilogue
    pk, sd = dev(packed), gpu(s)
    first = call(pk, sd, u)
    for fill in (0, 255, 0x7F):
        ws = torch.full((size + 64,), fill, dtype=torch.uint8, device="cuda")
        for _ in range(3):
            assert torch.equal(call(pk, sd, u, workspace=ws), first)
        assert bool((ws[size:] == fill).all())


def test_calls_after_calls_of_other_shapes_share_a_workspace(lq):
    """One workspace for a chain of calls of several shapes and kinds, in one stream."""
    import torch
    rng = np.random.default_rng(18)
    shapes = [(300, 1536, 1, "f32"), (700, 2240, 40, "bf16"), (64, 4096, 16, "f32"), (129, 96, 3, "bf16"), (300, 1536, 200, "bf16")]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    made = []
    for out, K, tokens, u_t in shapes * 2:
        packed, s = make_layer(rng, (), out, K)
        u = rng.standard_normal((tokens, K)).astype(np.float32)
        u = bf16(u) if u_t == "bf16" else u
        call = lq.gemv_epilogue if u_t == "f32" else lq.gemm_epilogue
        made.append((call(dev(packed), gpu(s), gpu(u, u_t == "bf16"), workspace=ws), packed, s, u))
    for got, packed, s, u in made:
        want, tol = plain.layer(packed, s.astype(np.float64), u)
        plain.assert_close(f64(got), want, tol, False)


def test_wrong_tensors_are_refused(lq):
    import torch
    rng = np.random.default_rng(19)
    packed, s = make_layer(rng, (2,), 64, 128)
    pk, sd, u = dev(packed), gpu(s), gpu(rng.standard_normal((4, 128)), True)
    off = ints([0, 2, 4])
    with pytest.raises(ValueError):
        lq.gemm_epilogue(pk[0], sd[0], u.float())
    with pytest.raises(ValueError):
        lq.gemv_epilogue(pk[0], sd[0], u)
    with pytest.raises(ValueError):
        lq.gemm_epilogue(pk[0], sd[0], u, bias=sd[0][:63])
    with pytest.raises(ValueError):
        lq.gemm_epilogue(pk[0], sd[0], u, act="tanh")
    with pytest.raises(ValueError):
        lq.gemm_epilogue(pk[0], sd[0], u, residual=torch.zeros((4, 64), device="cuda"), o_dtype="bf16")
    with pytest.raises(ValueError):
        lq.gemm_grouped(pk, sd, u, off.long(), 4)
    with pytest.raises(ValueError):
        lq.gemm_grouped(pk, sd, u.t().contiguous().t(), off, 4)
    with pytest.raises(lq.LQError):  # more slots than rows of u, and no rows
        lq.gemm_grouped(pk, sd, u, off, 5)
    with pytest.raises(lq.LQError):  # in place
        o = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
        lq.gemm_epilogue(dev(words(rng, (128, 4))), gpu(np.ones(128)), o, out=o)
    with pytest.raises(lq.LQError):  # pageable host memory through the C ABI
        import ctypes
        rc = lq.lib.lq_combine_rows(ctypes.c_void_p(np.zeros(64, np.float32).ctypes.data & ~15), 0, 1, 4, off.data_ptr(),
                                    sd.data_ptr(), 1, 1, None, pk.data_ptr(), None)
        lq._check(rc, "lq_combine_rows")
    with pytest.raises(lq.LQError):  # workspace too small
        lq.gemv_epilogue(pk[0], sd[0], u.float(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_two_threads_at_once(lq):
    """Calls of two host threads, each on a stream and workspaces of its own, give what they give alone."""
    import threading

    import torch
    rng = np.random.default_rng(27)
    work = []
    for out, K, tokens in ((300, 12288, 1), (514, 4096, 6), (384, 12288, 64), (1000, 1536, 300)):
        packed, s = make_layer(rng, (), out, K)
        work.append((dev(packed), gpu(s), gpu(rng.standard_normal((tokens, K)), True)))
    ids = ints(rng.integers(0, 40, (3000, 8)))

    def calls():
        return [lq.gemm_epilogue(*w, act="gelu") for w in work] + [lq.gemv_epilogue(*w[:2], w[2].float()) for w in work[:2]] + [
            t for t in lq.group_rows(ids, 40)]

    alone = calls()
    torch.cuda.synchronize()
    wrong = []

    def run():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = calls()
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, alone)):
                        wrong.append("results differ")
        except Exception as e:  # a thread's exception would be lost
            wrong.append(repr(e))

    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# tokens and type of u: the decode GEMV (fp32, and bf16 made fp32), its tcgen05 form, the mma.sync kernel, the tcgen05
# kernel, and the same cut along K
EPILOGUES = [(2, "f32", 64), (2, "bf16", 64), (16, "f32", 64), (5, "bf16", 64), (40, "bf16", 64), (300, "bf16", 64), (40, "bf16", 8192)]


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("tokens,u_t,K", EPILOGUES)
def test_activations_are_accurate_in_their_tails(lq, act, glu, tokens, u_t, K):
    """u = 0, so z is the bias exactly and the bound is the activation's own: down to where its value leaves fp32's
    normal range, at both ends of that range, and among the smallest numbers."""
    out = 1024
    z = np.linspace(-120, 120, out).astype(np.float32)
    z[:8] = [0.0, -0.0, 1e-30, -1e-30, 1e-40, -1e-40, 3e30, -3e30]
    if glu:  # gates in the even rows, factors around 1 in the odd ones
        bias = np.stack([z, np.linspace(-2, 2, out).astype(np.float32)], 1).reshape(-1)
    else:
        bias = z
    rng = np.random.default_rng(28)
    packed, s = make_layer(rng, (), bias.size, K)
    call = lq.gemv_epilogue if u_t == "f32" else lq.gemm_epilogue
    got = f64(call(dev(packed), gpu(s), gpu(np.zeros((tokens, K)), u_t == "bf16"), bias=gpu(bias), act=act, glu=glu))
    want, tol = plain.activate_exact(z.astype(np.float64), act)
    big = np.abs(z) > 1e30  # the bound's floor grows with |z|; the values are z and 0
    tol[big] = 2 * plain.U32 * np.abs(want[big])
    if glu:
        other = bias[1::2].astype(np.float64)
        want, tol = want * other, tol * np.abs(other) + 2.0 ** -150
    assert got.shape == (tokens, out)
    plain.assert_close(got, np.tile(want, (tokens, 1)), np.tile(tol, (tokens, 1)), False)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("tokens,u_t,K", EPILOGUES)
def test_activations_of_nan_and_inf(lq, act, glu, tokens, u_t, K):
    bias = np.full(256, 0.5, np.float32)
    step = 2 if glu else 1
    bias[20], bias[40], bias[60] = np.nan, np.inf, -np.inf
    rng = np.random.default_rng(29)
    packed, s = make_layer(rng, (), bias.size, K)
    call = lq.gemv_epilogue if u_t == "f32" else lq.gemm_epilogue
    got = f64(call(dev(packed), gpu(s), gpu(np.zeros((tokens, K)), u_t == "bf16"), bias=gpu(bias), act=act, glu=glu))
    low = {"none": -np.inf, "relu": 0.0}.get(act, np.nan)
    for at, want in ((20, np.nan), (40, np.inf), (60, low)):
        assert np.array_equal(got[:, at // step], np.full(tokens, want), equal_nan=True)
    rest = np.delete(got, [20 // step, 40 // step, 60 // step], axis=1)
    assert np.isfinite(rest).all() and (rest == rest[0, 0]).all()


@pytest.mark.parametrize("E,n", [(12, 60), (5, 90), (40, 30)])  # five slots an expert, eighteen, and one
@pytest.mark.parametrize("K", [96, 1056, 1152, 2048])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_rows_outside_read_nothing(lq, E, n, K, gather):
    """Rows outside u count as zero rows, whatever lies beside u in memory (NaN here); offsets outside 0..n are cut;
    slots of no expert keep their contents. At the sizes of each kernel, rows of words aligned and not."""
    import torch
    rng = np.random.default_rng([30, E, K])
    out, tokens = 134, 20 if gather else n
    packed, s = make_layer(rng, (E,), out, K)
    bias = rng.standard_normal((E, out)).astype(np.float32)
    u = bf16(rng.standard_normal((tokens, K)))
    beside = torch.full((tokens + 16, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    beside[8: 8 + tokens] = gpu(u, True)
    rows = rng.integers(-8, tokens + 8, n).astype(np.int32) if gather else None
    if gather:
        rows[:4] = [2 ** 31 - 1, -2 ** 31, -1, tokens]
    for last in (n - 7, n + 500):  # slots left over, and an offset past the end
        offsets = np.sort(rng.integers(0, n - 7, E + 1)).astype(np.int32)
        offsets[0], offsets[1], offsets[-1] = -3, 5, last
        offsets[1:] = np.maximum.accumulate(offsets[1:])
        for glu, o_t in ((False, "f32"), (True, "bf16")):
            width = out // 2 if glu else out
            o = torch.full((n, width), 7.5, device="cuda", dtype=torch.float32 if o_t == "f32" else torch.bfloat16)
            lq.gemm_grouped(dev(packed), gpu(s), beside[8: 8 + tokens], ints(offsets), n, rows=None if rows is None else ints(rows),
                            bias=gpu(bias), act="silu", glu=glu, out=o)
            want, tol, written = plain.grouped(packed, s.astype(np.float64), u, offsets, n, rows, bias, "silu", glu)
            got = f64(o)
            assert (got[~written] == 7.5).all() and written.sum() >= n - 7
            plain.assert_close(got[written], want[written], tol[written], o_t == "bf16")


@pytest.mark.parametrize("tokens", [9, 12, 16])
@pytest.mark.parametrize("K", [1056, 12288])
def test_wide_layers_hold_bf16_rows_to_21_bits(lq, tokens, K):
    """Layers of more than 18944 rows at 9 to 16 tokens: u may be off by 2^(E - 21), 2^E the power of two above the largest of
    its 32 elements, whatever the spread among them (here up to 2^24), and no more; all other sums as elsewhere."""
    out = 18945
    rng = np.random.default_rng([31, tokens, K])
    packed, s = make_layer(rng, (), out, K)
    u = bf16(rng.standard_normal((tokens, K)) * 2.0 ** rng.integers(-24, 1, (tokens, K)))
    rows = np.sort(rng.choice(out, 1500, replace=False))
    rows[0], rows[-1] = 0, out - 1
    want, tol = plain.layer(packed[rows], s[rows].astype(np.float64), u)
    largest = np.abs(u.astype(np.float64)).reshape(tokens, -1, 32).max(2)
    above = 2.0 ** (np.floor(np.log2(largest)) + 1)
    tol = tol + s[rows] * (32 * above * 2.0 ** -21).sum(1)[:, None]
    args = dev(packed), gpu(s), gpu(u, True)
    assert lq.gemm_epilogue_workspace_size(out, K, tokens) > lq.gemv_epilogue_workspace_size(out, K, tokens)  # that route
    plain.assert_close(f64(lq.gemm_epilogue(*args))[:, rows], want, tol, False)


def whitening(rng, channels, t):
    return np.stack([np.linalg.qr(rng.standard_normal((t, t)))[0] for _ in range(channels // t)]).astype(np.float32)


@pytest.mark.parametrize("tokens,topk,model,hidden,t_in,t_hidden", [(1, 2, 320, 200, 32, 8), (9, 2, 320, 200, None, 40),
                                                                    (100, 3, 640, 640, 128, 128)])
def test_experts_block_with_whitening_and_dropped_choices(lq, tokens, topk, model, hidden, t_in, t_hidden):
    """Each layer's own T^{-1}; most choices dropped, so that most slots of the inner tensors are never written, in memory that
    held NaN before. Tolerance as in test_experts_block."""
    import torch

    import oracle
    rng = np.random.default_rng([32, tokens])
    E = 6
    mlp, parts = expert_mlp(lq, rng, E, model, hidden, 10, 24)
    tinv = [None if t is None else whitening(rng, c, t) for c, t in ((model, t_in), (hidden, t_hidden))]
    mlp = type(mlp)(mlp.gate_up, mlp.gate_up_s, mlp.down, mlp.down_s, mlp.M, *(None if t is None else gpu(t) for t in tinv))
    x = bf16(rng.standard_normal((tokens, model)))
    ids = np.argsort(rng.random((tokens, E)), axis=1)[:, :topk].astype(np.int32)
    ids[rng.random(ids.shape) < 0.6] = -1
    ids[0, 0] = 3
    w = rng.uniform(0.1, 1, (tokens, topk)).astype(np.float32)
    gate, gs, up, us, down, ds, M = (np.asarray(p) for p in parts)

    def lifted(a, t, K):
        return bf16(lift(oracle.whiten(a, t), M.astype(np.float64), K)).astype(np.float64)

    u = lifted(x.astype(np.float64), tinv[0], gate.shape[2] * 32)
    want = x.astype(np.float64)
    for i, j in np.argwhere(ids >= 0):
        e = ids[i, j]
        g, v = gs[e] * (plain.signs(gate[e]) @ u[i]), us[e] * (plain.signs(up[e]) @ u[i])
        h = bf16(plain.activate(g, "silu") * v).astype(np.float64)
        want[i] += float(w[i, j]) * bf16(ds[e] * (plain.signs(down[e]) @ lifted(h[None], tinv[1], down.shape[2] * 32)[0]))
    args = gpu(x, True), ints(ids), gpu(w)
    torch.cuda.synchronize()
    poison = [torch.full((1 << b,), float("nan"), device="cuda") for b in range(6, 23)]
    del poison
    got = f64(mlp.step(*args))
    added = np.abs(want - x).max(1, keepdims=True)
    assert (np.abs(got - want) <= plain.UBF * np.abs(want) + 3 * 2.0 ** -7 * added).all()
    none = (ids < 0).all(1)
    assert np.array_equal(got[none], x[none].astype(np.float64))
