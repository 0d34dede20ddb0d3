"""Row products whose records and token matrices pass 2^32 bytes: the far end
against the same rows by themselves."""
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("group_scale_search_b200")

BF16, FP32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tq.lib()


def rows(R, n, seed):
    return torch.randn((R, n), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.fixture(scope="module", params=["int4g32", "nvfp4"])
def big(request):
    """A matrix of 4.4e9 bytes of records whose last 300 rows are random, the
    others one row repeated; and those 300 rows by themselves."""
    fmt, I, tail = request.param, 8192, 300
    per = I // ref.GROUP[fmt] * ref.BYTES[fmt]
    O = int(4.4e9) // per
    end, one = ref.Weights(fmt, 1, tail, I, 1, "cuda"), ref.Weights(fmt, 1, 1, I, 2, "cuda")
    w = ref.Weights.__new__(ref.Weights)
    w.__dict__.update(one.__dict__)
    w.shape = (1, O, I)

    def fill(a, b):
        out = torch.empty((O, a.numel()), dtype=a.dtype, device="cuda")
        out[:] = a.reshape(1, -1)
        out[O - tail:] = b.reshape(tail, -1)
        return out

    w.packed = fill(one.packed, end.packed).view(-1)
    w.scales = fill(one.scales, end.scales)[None]
    w.zeros = None if one.zeros is None else fill(one.zeros, end.zeros)[None]
    end.glob = one.glob
    assert w.packed.numel() > 2 ** 32
    yield w, end, tail
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R", [3, 100])
def test_records_past_32_bits(big, R):
    w, end, tail = big
    O, I = w.shape[1:]
    wh = w.handle(tq)
    x = rows(R, I, 3)
    few = R <= 32
    z, err = ref.either(x, end, 0, "few" if few else None)
    y = tq.tq_dequant_matmul(x, wh, out_dtype=torch.float32)
    ref.check(y[:, O - tail:], z, err, FP32)
    # (the first of the equal rows and the last: the same sum)
    assert torch.equal(y[:, :1], y[:, O - tail - 1:O - tail]) and torch.equal(y[:, 1:O - tail], y[:, :O - tail - 1])
    h = tq.tq_gated_ffn(x, wh, wh, out_dtype=torch.float32)
    want, err = ref.gated(x, end, end, "silu", "few" if few else None)
    ref.check(h[:, O - tail:], want, err, FP32)
    labels = torch.arange(R, device="cuda") + O - tail
    loss, lse = tq.tq_head_loss(x, wh, labels)
    logits = y.double()
    assert (lse.double() - torch.logsumexp(logits, 1)).abs().max() <= 1e-4   # (up to 132 joined tiles in a row, 2^-21 each)
    assert (loss.double() - (lse.double() - logits.gather(1, labels[:, None])[:, 0])).abs().max() <= 1e-5
    # gradients of tokens that only the far rows move
    d = torch.zeros((R, O), dtype=torch.bfloat16, device="cuda")
    d[:, O - tail:] = rows(R, tail, 4)
    dx = tq.tq_dequant_matmul_backward(d, wh, I)
    far = d[:, O - tail:].double()
    smax = w.largest_scale().max().item() * 2 * 15   # 2^-31 M, as 2^-32 times 2 M; M <= 15 s
    z, err = ref.gradient(far, end.dense()[0], 2.0 ** -39 * far.abs().amax(1, keepdim=True), smax)
    # (the sum runs over all rows, in the tensor cores' 32 bits: the others add zeros)
    ref.check(dx, z, err, BF16)


@pytest.mark.parametrize("R", [5, 40])
def test_row_strides_past_32_bits(R):
    """Token rows and outputs so far apart that the last starts past 2^32 bytes."""
    ld = (2 ** 32 // 2 + 4096) // (R - 1) + 1
    w = ref.Weights("int4g64", 1, 100, 136, 5, "cuda")
    wh = w.handle(tq)
    x, d = rows(R, 136, 6), rows(R, 100, 7)
    wide = torch.empty((R, ld), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((R, ld), dtype=torch.bfloat16, device="cuda")
    assert (R - 1) * ld * 2 > 2 ** 32
    wide[:, 1:137] = x
    wide[:, 200:300] = d
    xs, ds = wide[:, 1:137], wide[:, 200:300]
    for call, args, plain, cols in ((tq.tq_dequant_matmul, (xs, wh), (x, wh), 100), (tq.tq_gated_ffn, (xs, wh, wh), (x, wh, wh), 100),
                                    (tq.tq_dequant_matmul_backward, (ds, wh, 136), (d, wh, 136), 136),
                                    (tq.tq_gated_ffn_backward, (ds, xs, wh, wh), (d, x, wh, wh), 136)):
        got = call(*args, out=out[:, 7:7 + cols])
        assert torch.equal(got, call(*plain))
