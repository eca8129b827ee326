"""The linear layer with 4-bit weights against the 64-bit definition.

Bound: products of 16-bit activations and 4-bit codes are exact in fp32; K of them, their group
scales, bias and residual are summed in fp32 in some order, at most (K + 8) units of 2^-24 of
the terms' magnitudes; then one rounding to the output type."""
import pytest
import torch

import int8_weight_quantized_gb300 as ck
import transformer_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(M, N, K, group, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn((M, K), generator=g, device=DEV).to(dtype)
    codes = torch.randint(-8, 8, (N, K), generator=g, device=DEV, dtype=torch.int8)
    scale = (torch.rand((N, K // group), generator=g, device=DEV) * 0.02 + 0.001).to(torch.bfloat16)
    return x, codes, scale


def expected(x, codes, scale, group, bias, residual, out_dtype):
    w = codes.double() * scale.double().repeat_interleave(group, 1)
    y = x.double() @ w.t()
    mag = x.double().abs() @ w.abs().t()
    for extra in (bias, residual):
        if extra is not None:
            y, mag = y + extra.double(), mag + extra.double().abs()
    fp32 = (x.shape[1] + 8) * ref.U32 * mag
    return y, fp32 + (y.abs() + fp32) * ref.unit(out_dtype) + ref.least(out_dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K,group", [
    (1, 8, 128, 32), (1, 8, 128, 128), (1, 512, 512, 128), (2, 24, 256, 256), (3, 1000, 384, 64), (7, 136, 1152, 128),
    (8, 512, 2048, 32), (9, 264, 640, 128), (16, 1024, 4096, 64), (17, 72, 256, 64), (33, 200, 896, 128),
    (65, 80, 384, 32), (1, 16384, 5376, 128), (130, 48, 256, 128),
])
def test_against_the_definition(M, N, K, group, dtype):
    x, codes, scale = make(M, N, K, group, dtype, seed=M + N)
    w4 = ck.ck_int4_pack(codes)
    y = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    ck.ck_int4_linear(x, w4, scale, y=y)
    want, tol = expected(x, codes, scale, group, None, None, dtype)
    ref.assert_within(y, want, tol, "y")


@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M", [1, 5, 24])
def test_bias_residual_and_output_types(M, out_dtype):
    N, K, group = 272, 768, 128
    for dtype in (torch.bfloat16, torch.float16):
        x, codes, scale = make(M, N, K, group, dtype, seed=M)
        bias = torch.randn(N, device=DEV).to(dtype)
        residual = torch.randn((M, N), device=DEV).to(out_dtype)
        w4 = ck.ck_int4_pack(codes)
        want, tol = expected(x, codes, scale, group, bias, residual, out_dtype)
        y = ck.ck_int4_linear(x, w4, scale, bias=bias, residual=residual, out_dtype=out_dtype)
        ref.assert_within(y, want, tol, "y")
        ck.ck_int4_linear(x, w4, scale, bias=bias, residual=residual, y=residual, out_dtype=out_dtype)  # in place
        assert torch.equal(y, residual)


def test_rows_do_not_depend_on_the_batch():
    """A row's result is the same bits alone and among up to eight rows (one tile of rows)."""
    x, codes, scale = make(8, 512, 1024, 128, torch.bfloat16, seed=4)
    w4 = ck.ck_int4_pack(codes)
    all_rows = ck.ck_int4_linear(x, w4, scale)
    for m in (0, 3, 7):
        assert torch.equal(ck.ck_int4_linear(x[m:m + 1], w4, scale), all_rows[m:m + 1])


def test_pack_layout():
    codes = torch.arange(-8, 8, dtype=torch.int8, device=DEV).repeat(8, 8)
    words = ck.ck_int4_pack(codes).cpu().to(torch.int64) & 0xFFFFFFFF
    c = codes.cpu().to(torch.int64) + 8
    want = sum(c[:, e::8] << (4 * (e // 2) + 16 * (e % 2)) for e in range(8))
    assert torch.equal(words, want)


@pytest.mark.parametrize("N,K,group", [(8, 128, 32), (40, 512, 64), (16, 1280, 128), (24, 768, 256)])
def test_prepared_weight(N, K, group):
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    W = torch.randn((N, K), generator=g, device=DEV) * 0.02
    W[0, :group] = 0
    w4, scale = ck.ck_int4_prepare_weight(W, group)
    Wc = W.cpu().view(N, -1, group)  # torch's CUDA division by a plain number is not the IEEE quotient
    want_scale = (Wc.abs().amax(-1) / 7).to(torch.bfloat16)
    assert torch.equal(scale.cpu(), want_scale)
    s = want_scale.float()[..., None]
    codes = torch.where(s > 0, (Wc / s.clamp_min(1e-38)).round().clamp(-7, 7), torch.zeros_like(s))
    assert torch.equal(w4, ck.ck_int4_pack(codes.view(N, K).to(torch.int8).to(DEV)))


def test_other_streams_and_graphs():
    x, codes, scale = make(4, 4096, 4096, 128, torch.bfloat16, seed=2)
    w4 = ck.ck_int4_pack(codes)
    want = ck.ck_int4_linear(x, w4, scale)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[ck.ck_int4_linear(x, w4, scale, stream=s) for _ in range(4)] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for per in outs for o in per)
    y = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ck.ck_int4_linear(x, w4, scale, y=y)
    x.mul_(-1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, -want)


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("group", [32, 64, 128, 256])
def test_groups_that_codes_cannot_hold_have_nan_scales(group, fill):
    """A NaN or infinite weight leaves no plausible group: its scale is NaN, and with it its row's
    outputs; the other groups are as they were."""
    N, K = 24, 512
    g = torch.Generator(device=DEV)
    g.manual_seed(5)
    W = torch.randn((N, K), generator=g, device=DEV) * 0.02
    w4, scale = ck.ck_int4_prepare_weight(W, group)
    bad = torch.zeros(scale.shape, dtype=torch.bool, device=DEV)
    for n, k in ((0, 0), (3, group - 1), (7, K - 1), (23, group + 9)):
        W[n, k % K] = fill
        bad[n, k % K // group] = True
    got4, got = ck.ck_int4_prepare_weight(W, group)
    assert torch.equal(got.isnan(), bad)
    assert torch.equal(got[~bad], scale[~bad])
    words = bad.repeat_interleave(group // 8, 1)
    assert torch.equal(got4[~words], w4[~words])
    y = ck.ck_int4_linear(torch.randn((2, K), generator=g, device=DEV).to(torch.bfloat16), got4, got)
    assert torch.equal(y.isnan().all(0), bad.any(1)) and torch.equal(y.isnan().any(0), bad.any(1))
