"""Paths of the row products that only larger or more uneven calls take: every
token-block count of the few-token kernel, its walk over several tiles, routed
gradients whose sum is split, and the give-up path of every format."""
import os
import subprocess
import sys

import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("group_scale_search_b200")

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
FMTS = list(ref.FMT)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tq.lib()


def rows(R, n, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((R, n), generator=gen) * scale).to(torch.bfloat16).cuda()


def scale_of(*ws):
    """What the kernel normalises by: the larger of the largest scales (NVFP4: the largest dequantized value / 15)."""
    if ws[0].fmt == "nvfp4":
        return max(w.dense().abs().max().item() for w in ws) * 448 / 15
    return max(w.largest_scale().max().item() for w in ws)


def check_loss(w, x, seed):
    """Loss and gradient by the few-token kernel."""
    R, V = x.shape[0], w.shape[1]
    gen = torch.Generator().manual_seed(seed)
    labels = torch.randint(0, V, (R,), generator=gen)
    labels[-1] = V - 1
    if R > 2:
        labels[1] = -100
    labels = labels.cuda()
    want, lse64, err = ref.head_loss(x, w, labels, True)
    loss, lse = tq.tq_head_loss(x, w.handle(tq), labels)
    ref.check(lse, lse64, err, FP32)
    ref.check(loss, want, err, FP32)
    dloss = torch.rand(R, generator=gen).cuda() + 0.5
    dx, err = ref.head_grad(dloss, x, w, labels, lse, True)
    ref.check(tq.tq_head_loss_backward(dloss, x, w.handle(tq), labels, lse), dx, err, BF16)


# ---------------------------------------------------------------- few tokens

# 17 to 32 rows take four blocks of 8 tokens, 9 to 16 two; rows of several
# slices of 128 columns with a remainder (and for one shape none)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,I", [(8, 904), (12, 904), (17, 904), (24, 1160), (31, 520), (32, 1024)])
def test_every_block_count(fmt, R, I):
    O = 333
    g, u = ref.Weights(fmt, 1, O, I, 1, "cuda"), ref.Weights(fmt, 1, O, I, 2, "cuda")
    x, d = rows(R, I, 3), rows(R, O, 4, 1e-3)
    z, err = ref.product_few(x, g)
    ref.check(tq.tq_dequant_matmul(x, g.handle(tq), out_dtype=torch.float32), z, err, FP32)
    ref.check(tq.tq_dequant_matmul(x, g.handle(tq)), z, err, BF16)
    h, err = ref.gated(x, g, u, "gelu", "few")
    ref.check(tq.tq_gated_ffn(x, g.handle(tq), u.handle(tq), act="gelu", out_dtype=torch.float32), h, err, FP32)
    dx, err = ref.gated_grad(d, x, g, u, "silu", scale_of(g, u), fmt == "nvfp4", few=True)
    ref.check(tq.tq_gated_ffn_backward(d, x, g.handle(tq), u.handle(tq)), dx, err, BF16)
    check_loss(g, x, 5)


# So many tiles of 32 weight rows that a block's groups of warps take several
# each: with one warp to a tile (more tiles than 2 x 148 blocks hold warps),
# and with two to eight (rows of many slices).
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,O,I", [(1, 100000, 520), (9, 80000, 264), (3, 26000, 4104), (8, 40000, 2184), (16, 30000, 2056)])
def test_several_tiles_of_a_warp(fmt, R, O, I):
    w = ref.Weights(fmt, 1, O, I, 6, "cuda")
    x = rows(R, I, 7)
    z, err = ref.product_few(x, w)
    ref.check(tq.tq_dequant_matmul(x, w.handle(tq), out_dtype=torch.float32), z, err, FP32)
    ref.check(tq.tq_dequant_matmul(x, w.handle(tq)), z, err, BF16)
    check_loss(w, x, 8)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R", [20, 32])
def test_several_tiles_of_four_token_blocks(fmt, R):
    """Fewer tiles of 128 rows than SMs, rows of so many slices that eight
    warps share a tile and take several (the last column range is short)."""
    O, I = 12800, 8072
    w = ref.Weights(fmt, 1, O, I, 9, "cuda")
    x = rows(R, I, 10)
    z, err = ref.product_few(x, w)
    ref.check(tq.tq_dequant_matmul(x, w.handle(tq), out_dtype=torch.float32), z, err, FP32)
    check_loss(w, x, 11)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,O,I", [(90, 2000, 264), (100, 1856, 1024), (5, 3000, 520)])
def test_several_tiles_over_experts(fmt, R, O, I):
    """A handful of rows over 100 experts: a group of warps walks from one
    matrix into the next."""
    E = 100
    g, u = ref.Weights(fmt, E, O, I, 12, "cuda"), ref.Weights(fmt, E, O, I, 13, "cuda")
    x, d = rows(R, I, 14), rows(R, O, 15, 1e-2)
    gen = torch.Generator().manual_seed(16)
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randint(0, R + 1, (E - 1,), generator=gen).sort().values,
                     torch.tensor([R])])
    o = off.to(torch.int32).cuda()
    y = tq.tq_dequant_matmul(x, g.handle(tq), offsets=o, out_dtype=torch.float32)
    h = tq.tq_gated_ffn(x, g.handle(tq), u.handle(tq), offsets=o, out_dtype=torch.float32)
    dx = tq.tq_gated_ffn_backward(d, x, g.handle(tq), u.handle(tq), offsets=o)
    tq.tq_sync()
    smax = scale_of(g, u)
    for e in range(E):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start == s.stop:
            continue
        a, b = one_matrix(g, e), one_matrix(u, e)
        z, err = ref.product_few(x[s], a)
        ref.check(y[s], z, err, FP32)
        z, err = ref.gated(x[s], a, b, "silu", "few")
        ref.check(h[s], z, err, FP32)
        z, err = ref.gated_grad(d[s], x[s], a, b, "silu", smax, fmt == "nvfp4", few=True)
        ref.check(dx[s], z, err, BF16)


def one_matrix(w, e):
    m = ref.Weights.__new__(ref.Weights)
    m.__dict__.update(w.__dict__)
    m.shape = (1, *w.shape[1:])
    m.packed = w.packed.view(w.shape[0], -1)[e]
    m.scales = w.scales[e:e + 1]
    m.zeros = None if w.zeros is None else w.zeros[e:e + 1]
    m.glob = None if w.glob is None else w.glob[e:e + 1]
    return m


# ---------------------------------------------------------------- routed gradients, split sums

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("I", [128, 200])
def test_routed_gradients_of_a_split_sum(fmt, gated, I):
    """Few tiles and a long sum over weight rows: its parts are joined for the
    rows of the ranges, the others stay, whatever the workspace holds."""
    E, O, R = 3, 6000, 60
    g, u = ref.Weights(fmt, E, O, I, 17, "cuda"), ref.Weights(fmt, E, O, I, 18, "cuda")
    x, d = rows(R + 9, I, 19), rows(R + 9, O, 20, 1e-3)
    smax = scale_of(g, u)
    for off in ([0, 20, 20, R + 9], [5, 3, -7, R + 5], [7, 7, 30, R], [4, 4, 4, 4], [R + 30, 1, 2, 3], [-3, 2, 90, 80]):
        clean = []
        for v in off:   # made monotone and within the rows
            clean.append(min(max(v, clean[-1] if clean else 0, 0), R + 9))
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")   # NaN of every type
        out = torch.full((R + 9, I + 3), 7.0, dtype=torch.bfloat16, device="cuda")
        if gated:
            tq.tq_gated_ffn_backward(d, x, g.handle(tq), u.handle(tq), offsets=o, out=out[:, :I], workspace=ws)
        else:
            tq.tq_dequant_matmul_backward(d, g.handle(tq), I, offsets=o, out=out[:, :I], workspace=ws)
        tq.tq_sync()
        assert (out[:clean[0]] == 7).all() and (out[clean[-1]:] == 7).all() and (out[:, I:] == 7).all()
        for e in range(E):
            s = slice(clean[e], clean[e + 1])
            if s.start >= s.stop:
                continue
            if gated:
                z, err = ref.gated_grad(d[s], x[s], g, u, "silu", smax, fmt == "nvfp4", e)
                few, err_few = ref.gated_grad(d[s], x[s], g, u, "silu", smax, fmt == "nvfp4", e, True)
                err = torch.maximum(err, err_few)   # (the projections are the few-token kernel's)
            else:
                ds = d[s].double()
                z, err = ref.gradient(ds, g.dense()[e], 2.0 ** -39 * ds.abs().amax(1, keepdim=True), g.largest_scale()[e])
            ref.check(out[s, :I], z, err, BF16)


# ---------------------------------------------------------------- other ranges

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R", [30, 250])
def test_one_matrix_and_a_range(fmt, R):
    """offsets may be given for a single matrix too: its range of the rows."""
    O, I = 150, 264
    g, u = ref.Weights(fmt, 1, O, I, 25, "cuda"), ref.Weights(fmt, 1, O, I, 26, "cuda")
    x, d = rows(R, I, 27), rows(R, O, 28, 1e-2)
    gh, uh = g.handle(tq), u.handle(tq)
    calls = [(O, lambda x, d, **kw: tq.tq_dequant_matmul(x, gh, **kw)), (O, lambda x, d, **kw: tq.tq_gated_ffn(x, gh, uh, **kw)),
             (I, lambda x, d, **kw: tq.tq_dequant_matmul_backward(d, gh, I, **kw)),
             (I, lambda x, d, **kw: tq.tq_gated_ffn_backward(d, x, gh, uh, **kw))]
    for lo, hi in ((0, R), (3, R - 2), (7, 7)):
        off = torch.tensor([lo, hi], dtype=torch.int32, device="cuda")
        for n, call in calls:
            out = torch.full((R, n), 7.0, dtype=torch.bfloat16, device="cuda")
            call(x, d, offsets=off, out=out)
            assert torch.equal(out[lo:hi], call(x, d)[lo:hi])   # (a row's result does not depend on the others)
            assert (out[:lo] == 7).all() and (out[hi:] == 7).all()


@pytest.mark.parametrize("fmt", ["int3", "int4g32", "nvfp4"])
@pytest.mark.parametrize("R", [700, 40000])
def test_as_many_matrices_as_there_may_be(fmt, R):
    E, O, I = 1024, 40, 72
    g, u = ref.Weights(fmt, E, O, I, 29, "cuda"), ref.Weights(fmt, E, O, I, 30, "cuda")
    x, d = rows(R, I, 31), rows(R, O, 32, 1e-2)
    expert = torch.randint(0, E, (R,), generator=torch.Generator().manual_seed(33)).sort().values.cuda()
    off = torch.searchsorted(expert, torch.arange(E + 1, device="cuda")).to(torch.int32)
    few = R < E
    W, A, s = g.dense(), g.spread(), g.largest_scale()[expert, None]
    x64 = x.double()
    z = torch.einsum("ri,roi->ro", x64, W[expert])
    tiny = 2.0 ** -30 * x64.abs().amax(1, keepdim=True) * W.abs().sum(2)[expert]
    y = tq.tq_dequant_matmul(x, g.handle(tq), offsets=off, out_dtype=torch.float32)
    size = torch.einsum("ri,roi->ro", x64.abs(), (A if few else W.abs())[expert])
    ref.check(y, z, (I / 16 + 2 * g.G + 32) * ref.U * size + tiny, FP32)
    d64 = d.double()
    dx = tq.tq_dequant_matmul_backward(d, g.handle(tq), I, offsets=off)
    size = torch.einsum("ro,roi->ri", d64.abs(), W.abs()[expert])
    tiny = 2.0 ** -39 * d64.abs().amax(1, keepdim=True) * W.abs().sum(1)[expert] + 2.0 ** -32 * s * d64.abs().sum(1, keepdim=True)
    ref.check(dx, torch.einsum("ro,roi->ri", d64, W[expert]), (2.0 ** -10 + (O / 16 + 32) * ref.U) * size + tiny, BF16)
    # the block and its gradient, by the norm of what they are off
    h = tq.tq_gated_ffn(x, g.handle(tq), u.handle(tq), offsets=off, out_dtype=torch.float32)
    p = ref.act("silu", z)[0] * torch.einsum("ri,roi->ro", x64, u.dense()[expert])
    assert (h.double() - p).norm() <= 1e-4 * p.norm()   # (fp32 sums of exact products)
    db = tq.tq_gated_ffn_backward(d, x, g.handle(tq), u.handle(tq), offsets=off)
    U_ = torch.einsum("ri,roi->ro", x64, u.dense()[expert])
    a, da = ref.act("silu", z)
    want = torch.einsum("ro,roi->ri", d64 * U_ * da, W[expert]) + torch.einsum("ro,roi->ri", d64 * a, u.dense()[expert])
    assert (db.double() - want).norm() <= (BF16 + 2.0 ** -9) * want.norm()   # (its rounding, and the operands' 11 bits)


def test_first_calls_inside_a_capture():
    """A process whose first row products are captured, each kind of kernel
    among them, and replayed: the same bits as plain calls."""
    code = f"""
import sys
sys.path[:0] = [{ROOT!r}, {os.path.join(ROOT, "tests")!r}]
import torch
import group_scale_search_b200 as tq, rows_ref as ref
torch.manual_seed(1)
x, d = (torch.randn(200, n, device="cuda").to(torch.bfloat16) for n in (256, 300))
g, u = (ref.Weights("int4g64", 1, 300, 256, s, "cuda") for s in (1, 2))
gh, uh = g.handle(tq), u.handle(tq)
lab, one = torch.arange(200, device="cuda"), torch.ones(200, device="cuda")
lse = torch.logsumexp(x.double() @ g.dense()[0].T, 1).float()
def run(R):
    return [tq.tq_dequant_matmul(x[:R], gh), tq.tq_dequant_matmul(x[:R], gh, out_dtype=torch.float32),
            tq.tq_gated_ffn(x[:R], gh, uh), tq.tq_dequant_matmul_backward(d[:R], gh, 256),
            tq.tq_gated_ffn_backward(d[:R], x[:R], gh, uh), tq.tq_head_loss(x[:R], gh, lab[:R])[0],
            tq.tq_head_loss_backward(one[:R], x[:R], gh, lab[:R], lse[:R])]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = run(5) + run(200)
graph.replay()
torch.cuda.synchronize()
tq.tq_sync()
assert all(torch.equal(a, b) for a, b in zip(outs, run(5) + run(200)))
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]


# ---------------------------------------------------------------- giving up

@pytest.mark.parametrize("fmt", FMTS)
def test_every_format_reports_a_given_up_wait(fmt):
    g, u = ref.Weights(fmt, 1, 300, 256, 21, "cuda"), ref.Weights(fmt, 1, 300, 256, 22, "cuda")
    x, d = rows(300, 256, 23), rows(300, 300, 24)
    gh, uh = g.handle(tq), u.handle(tq)
    calls = (lambda: tq.tq_dequant_matmul(x, gh), lambda: tq.tq_dequant_matmul(x[:60], gh, out_dtype=torch.float32),
             lambda: tq.tq_gated_ffn(x, gh, uh), lambda: tq.tq_dequant_matmul_backward(d, gh, 256))
    want = [call() for call in calls]
    tq.tq_sync()
    for call, right in zip(calls, want):
        tq.tq_debug_set_wait_limit(0)
        try:
            call()
        finally:
            tq.tq_debug_set_wait_limit(-1)
        with pytest.raises(tq.TQError):
            tq.tq_sync()
        tq.tq_sync()   # (reported once)
        assert torch.equal(call(), right)
