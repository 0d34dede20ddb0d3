"""Row products at the ends of their types' ranges: zero-points of any byte,
gates, tokens and norms far from one, tiles of the vocabulary that nothing is
left of."""
import math

import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("group_scale_search_b200")

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
FMTS = list(ref.FMT)
INT4 = [f for f in FMTS if f.startswith("int4")]
FEW_OR_NOT = [5, 90]   # rows for the few-token kernel, and for the other


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tq.lib()


def normal(R, n, seed, scale=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((R, n), generator=gen, dtype=torch.float64) * scale).to(torch.bfloat16).cuda()


def largest(*ws):
    """M of the header's bounds: the largest |s| max(z, 15 - z), int3 4 |s| (NVFP4: the largest |What|)."""
    m = 0.0
    for w in ws:
        if w.fmt == "nvfp4":
            k = w.dense().abs().max()
        elif w.fmt == "int3":
            k = 4 * w.scales.abs().max()
        else:
            z = w.zeros.double()
            k = (w.scales.double().abs() * torch.maximum(z, 15 - z)).max()
        m = max(m, k.item())
    return m


def scaled(w, by):
    """The same records with values `by` times as large."""
    if w.fmt == "nvfp4":
        w.glob *= by
    else:
        w.scales *= by
    return w


def check_all(g, u, x, d, act="silu", slack=0.0):
    """Every product and gradient of one pair of matrices against 64 bits."""
    R, (_, O, I) = x.shape[0], g.shape
    few, fmt = R <= 32, g.fmt
    gh, uh = g.handle(tq), u.handle(tq)
    M = largest(g, u)
    # 2^-31 M sum |x| is 2^-32 times 2 M as rows_ref takes it; of the gated bound's 15 smax, M
    z, err = ref.either(x, g, 0, "few" if few else None)
    ref.check(tq.tq_dequant_matmul(x, gh, out_dtype=torch.float32), z, err, FP32)
    if not few and fmt != "nvfp4":
        z, err = ref.product16(x, g.dense()[0], 2 * M)
    ref.check(tq.tq_dequant_matmul(x, gh), z, err, BF16)
    z, err = ref.gradient(d.double(), g.dense()[0], 2.0 ** -39 * d.double().abs().amax(1, keepdim=True), 2 * M)
    ref.check(tq.tq_dequant_matmul_backward(d, gh, I), z, err, BF16)
    h, err = ref.gated(x, g, u, act, "few" if few else None)
    ref.check(tq.tq_gated_ffn(x, gh, uh, act=act, out_dtype=torch.float32), h, err, FP32)
    if not few and fmt != "nvfp4":
        h, err = ref.gated(x, g, u, act, 2 * M)
    ref.check(tq.tq_gated_ffn(x, gh, uh, act=act), h, err, BF16)
    dx, err = ref.gated_grad(d, x, g, u, act, 2 * M, fmt == "nvfp4", few=few)
    got = tq.tq_gated_ffn_backward(d, x, gh, uh, act=act)
    ref.check(got, dx, err, BF16)
    # (rounding does far less than the bound's worst case)
    assert (got.double() - dx).norm() <= 0.01 * dx.norm() + slack


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("zero", [15, 16, 17, 31, 255])
@pytest.mark.parametrize("fmt", INT4)
def test_any_zero_point(fmt, zero, R):
    """A byte is a byte: a zero-point outside the codes' range, in groups whose
    scale is the matrix's largest, just below a power of two."""
    O, I = 150, 264
    g, u = ref.Weights(fmt, 1, O, I, 1, "cuda"), ref.Weights(fmt, 1, O, I, 2, "cuda")
    for w in (g, u):
        w.scales.clamp_(max=0.015)
        w.scales[:, 3::40] = 0.0156   # (below 2^-6)
        w.zeros[:, 3::40] = zero
    check_all(g, u, normal(R, I, 3), normal(R, O, 4, 1e-3))


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("fmt", INT4)
def test_scales_and_zeros_of_any_alignment(fmt, R):
    """Scales that start on an element, zero-points on a byte: the same bits."""
    O, I = 151, 264
    g, u = ref.Weights(fmt, 1, O, I, 22, "cuda"), ref.Weights(fmt, 1, O, I, 23, "cuda")
    x, d = normal(R, I, 24), normal(R, O, 25, 1e-3)

    def run():
        gh, uh = g.handle(tq), u.handle(tq)
        return [tq.tq_dequant_matmul(x, gh), tq.tq_gated_ffn(x, gh, uh), tq.tq_dequant_matmul_backward(d, gh, I),
                tq.tq_gated_ffn_backward(d, x, gh, uh)]

    want = run()
    for at_scales, at_zeros in ((1, 1), (2, 3), (0, 2), (3, 0)):
        for w in (g, u):
            for name, at in (("scales", at_scales), ("zeros", at_zeros)):
                t = getattr(w, name)
                buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
                view = buf[at:at + t.numel()].view(t.shape)
                setattr(w, name, view.copy_(t))
        for a, b in zip(want, run()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("fmt", FMTS)
def test_gates_whose_square_is_no_float(fmt, act, R):
    """Gates beyond 1.9e19: act(g) is g or 0, act'(g) 1 or 0."""
    O, I = 140, 200
    g, u = (ref.Weights(fmt, 1, O, I, s, "cuda") for s in (5, 6))
    x, d = normal(R, I, 7), normal(R, O, 8, 1e-3)
    for w, size in ((g, 4e19), (u, 4e17)):   # h up to 1e38
        scaled(w, size / (x.double() @ w.dense()[0].T).std().item())
    gate = x.double() @ g.dense()[0].T
    assert (gate > 2e19).any() and (gate < -2e19).any()
    # act' is a step for such gates: where the gate is within its own error of
    # zero it may be 0 or 1 (gelu: in [-0.13, 1.13]), which moves dg by up to
    # 1.26 |dh u|, and |dg Wg| by that times Wg's largest singular value; du
    # moves by |dh| times that error, less than the error of gates elsewhere
    Wg = g.dense()[0]
    z, err = ref.product16(x, Wg, 2 * largest(g, u)) if R > 32 and fmt != "nvfp4" else ref.either(x, g, 0, "few" if R <= 32 else None)
    step = torch.where(z.abs() <= err, (d.double() * (x.double() @ u.dense()[0].T)).abs(), 0.0)
    check_all(g, u, x, d, act, 1.26 * (step.norm() * torch.linalg.matrix_norm(Wg, 2)).item())


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("size", [1e-27, 1e-24, 1e20, 1e26])
def test_gated_gradient_of_rows_whose_square_is_no_float(fmt, size, R):
    """Tokens whose squares leave fp32, weights that bring gate and up back to
    about one."""
    O, I = 140, 200
    g, u = (scaled(ref.Weights(fmt, 1, O, I, s, "cuda"), 1 / size) for s in (10, 11))
    x, d = normal(R, I, 12, size), normal(R, O, 13, 1e-3)
    dx, err = ref.gated_grad(d, x, g, u, "silu", 2 * largest(g, u), fmt == "nvfp4", few=R <= 32)
    got = tq.tq_gated_ffn_backward(d, x, g.handle(tq), u.handle(tq))
    ref.check(got, dx, err, BF16)
    assert (got.double() - dx).norm() <= 0.01 * dx.norm()   # (rounding does far less than the bound's worst case)


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("fmt", FMTS)
def test_tokens_near_the_largest(fmt, R):
    """Tokens up to 2^119, weights that bring the products back."""
    O, I = 70, 200
    x = normal(R, I, 16, 2.0 ** 117)
    few = "few" if R <= 32 else None
    w = scaled(ref.Weights(fmt, 1, O, I, 14, "cuda"), 2.0 ** -100)
    z, err = ref.either(x, w, 0, few)
    ref.check(tq.tq_dequant_matmul(x, w.handle(tq), out_dtype=torch.float32), z, err, FP32)
    if fmt != "nvfp4" and few is None:
        z, err = ref.product16(x, w.dense()[0], 2 * largest(w))
    ref.check(tq.tq_dequant_matmul(x, w.handle(tq)), z, err, BF16)
    scaled(w, 2.0 ** -14)   # products of about ten
    h, err = ref.gated(x, w, w, "silu", few)
    ref.check(tq.tq_gated_ffn(x, w.handle(tq), w.handle(tq), out_dtype=torch.float32), h, err, FP32)
    labels = torch.arange(R, device="cuda") % O
    want, lse64, err = ref.head_loss(x, w, labels, few is not None)
    loss, lse = tq.tq_head_loss(x, w.handle(tq), labels)
    ref.check(lse, lse64, err, FP32)
    ref.check(loss, want, err, FP32)


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("fmt", ["int3", "int4g64"])
def test_a_tile_of_the_vocabulary_at_minus_infinity(fmt, R):
    """Entries masked by an infinite scale, whole tiles of them, beside logits
    far below zero: the sum is that of the others."""
    V, I = 700, 64
    w = ref.Weights(fmt, 1, V, I, 17, "cuda")
    w.packed.zero_()   # codes 0: every value -4 or -15 scales
    if w.zeros is not None:
        w.zeros.fill_(15)
    w.scales[:] = (torch.rand(1, V, 1, generator=torch.Generator().manual_seed(18)) + 1).cuda()
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[:256] = False
    keep[512:640] = False
    w.scales[0, ~keep] = float("inf")
    x = torch.rand((R, I), generator=torch.Generator().manual_seed(19)).add_(0.5).to(torch.bfloat16).cuda()
    labels = torch.full((R,), 300, device="cuda")
    one = ref.Weights.__new__(ref.Weights)
    one.__dict__.update(w.__dict__)
    one.scales = w.scales[:, keep]
    one.zeros = None if w.zeros is None else w.zeros[:, keep]
    one.packed = w.packed.view(V, -1)[keep].reshape(-1)
    one.shape = (1, int(keep.sum()), I)
    want, lse64, err = ref.head_loss(x, one, labels - 256, R <= 32)
    assert lse64.max() < -100
    loss, lse = tq.tq_head_loss(x, w.handle(tq), labels)
    ref.check(lse, lse64, err, FP32)
    ref.check(loss, want, err, FP32)


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("fmt", FMTS)
def test_gradient_of_small_probabilities(fmt, R):
    """Probabilities of about 2^-34.5 (the rest of the sum is elsewhere) and a
    label whose own row is zero: the gradient is theirs alone.  Each is held to
    2^-11 of itself or 2^-38, and |err W| <= |err| |W|, the largest singular
    value."""
    V, I = 300, 64
    w = ref.Weights(fmt, 1, V, I, 20, "cuda")
    w.scales[0, V - 1] = 0
    x = normal(R, I, 21, 0.1)
    labels = torch.full((R,), V - 1, device="cuda")
    lse = torch.full((R,), 34.5 * math.log(2), device="cuda")
    W = w.dense()[0]
    p = torch.exp(x.double() @ W.T - lse.double()[:, None])
    want = p[:, :-1] @ W[:-1]
    err = ((p * 2.0 ** -11).norm(dim=1) + V ** 0.5 * 2.0 ** -38) * torch.linalg.matrix_norm(W, 2)
    got = tq.tq_head_loss_backward(torch.ones(R, device="cuda"), x, w.handle(tq), labels, lse).double()
    off = (got - want).norm(dim=1)
    assert (off <= err * (1 + BF16) + 2.0 ** -9 * want.norm(dim=1)).all(), (off / want.norm(dim=1)).max()


@pytest.mark.parametrize("R", FEW_OR_NOT)
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 18, 2.0 ** 24])
@pytest.mark.parametrize("fmt", FMTS)
def test_a_token_far_above_its_row(fmt, size, R):
    """One column far above the others, whose weights are zero: what the f16
    copy keeps of the others, by the header's bounds (few rows: 2^-30 of the
    largest times s (q + z), since zero-points come from the groups' sums)."""
    O, I = 90, 264
    w = ref.Weights(fmt, 1, O, I, 26, "cuda")
    rec = w.packed.view(O, w.G, -1)
    if fmt == "int3":   # code 4: v = 0
        rec[:, 0, 0] &= 0xfc
        rec[:, 0, 16] |= 1
    else:               # the low nibble: the zero-point, or E2M1's zero
        rec[:, 0, 0] = (rec[:, 0, 0] & 0xf0) | (0 if w.zeros is None else w.zeros[0, :, 0])
    W = w.dense()[0]
    assert (W[:, 0] == 0).all()
    x = normal(R, I, 27)
    x[:, 0] = size
    top = 2.0 ** -30 * x.double().abs().amax(1, keepdim=True)
    if R <= 32:
        z, err = ref.product_few(x, w)
        err = err + top * (w.spread()[0].sum(1) - W.abs().sum(1))
    else:
        z, err = ref.product(x, W, w.G)
    ref.check(tq.tq_dequant_matmul(x, w.handle(tq), out_dtype=torch.float32), z, err, FP32)
    if size <= 2.0 ** 12:   # (what tokens may be in earnest: nothing is lost)
        got = tq.tq_dequant_matmul(x, w.handle(tq), out_dtype=torch.float32).double()
        exact = (I / 16 + 2 * w.G + 32) * ref.U * (x[:, 1:].double().abs() @ w.spread()[0][:, 1:].T + size * w.spread()[0][:, 0])
        assert ((got - z).abs() <= exact).all()
