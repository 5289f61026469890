"""4-bit matrix-vector products with group scales against binary64 on the host:
group sizes, zero points, every batch, ragged rows and columns, wide ranges,
values that are not finite, fused norm / bias / residual, streams and graphs."""
import pytest
import torch

import activation_sparse_mlp_amd as spffn
from tests import attn_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def setup_module(module):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(rows, cols, group, zeros, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g)
    ng = -(-cols // group)
    scales = (torch.rand(rows, ng, generator=g) * 0.01 + 0.001).half()
    z = torch.randint(0, 16, (rows, ng), dtype=torch.uint8, generator=g) if zeros else None
    w = spffn.Q4Matrix(codes.to(DEV), scales.to(DEV), None if z is None else z.to(DEV),
                       group=group)
    return w, ref.q4_weights(codes, scales, z, group), g


SHAPES = [
    # rows, cols, group, B, zeros
    (1, 32, 32, 1, False),
    (17, 96, 32, 2, True),
    (100, 160, 128, 3, True),
    (33, 4128, 64, 8, False),
    (1029, 1056, 64, 9, True),
    (16, 128, 32, 16, False),
    (40, 2080, 128, 16, True),
    (8200, 256, 32, 1, True),      # enough row tiles for two per wave
    (8200, 288, 64, 5, False),
    (8193, 160, 128, 2, True),
    (8193, 416, 32, 12, True),
    (8209, 1024, 128, 7, False),
]


@pytest.mark.parametrize("rows,cols,group,B,zeros", SHAPES)
def test_product(rows, cols, group, B, zeros):
    w, wd, g = make(rows, cols, group, zeros, seed=rows + cols)
    x = torch.randn(B, cols, generator=g)
    x[:, ::7] *= 40.0
    y, bound = ref.q4_matvec(wd, x)
    ref.close(spffn.q4_matvec(w, x.to(DEV)).cpu(), y, bound)


@pytest.mark.parametrize("B", range(1, 17))
def test_every_batch_fused(B):
    rows, cols = 205, 736
    w, wd, g = make(rows, cols, 64, B % 2 == 0, seed=B)
    x = torch.randn(B, cols, generator=g) * 3.0
    bias, resid = torch.randn(rows, generator=g), torch.randn(B, rows, generator=g)
    y, bound = ref.q4_matvec(wd, x, bias, resid, rms_eps=1e-5)
    out = resid.to(DEV)
    got = spffn.q4_matvec(w, x.to(DEV), bias=bias.to(DEV), resid=out, rms_eps=1e-5, y=out)
    assert got is out  # the residual stream is updated in place
    ref.close(got.cpu(), y, bound)


def test_tokens_do_not_depend_on_each_other():
    rows, cols = 70, 512
    w, wd, g = make(rows, cols, 128, True, seed=3)
    x = torch.randn(16, cols, generator=g)
    x[3] *= 1e30
    x[4] *= 1e-30
    x[5] = 0.0
    x[6, 100] = float("inf")
    x[7, 3] = float("nan")
    x[8, 40:80] = float("-inf")
    x[9] *= 1e-44  # subnormal
    y, bound = ref.q4_matvec(wd, x)
    # any_odd: an infinity times the code and times the zero point are separate sums, and
    # inf - inf is NaN: which of the two comes out is not fixed, that it is not finite is.
    # Subnormal products are within a few of the smallest steps besides.
    bound = bound + cols * 2.0 ** -149 * 16
    for B in (16, 8):
        xs = x[:B] if B == 16 else x[2:10]
        ys, bs = (y[:B], bound[:B]) if B == 16 else (y[2:10], bound[2:10])
        ref.close(spffn.q4_matvec(w, xs.contiguous().to(DEV)).cpu(), ys, bs,
                  any_odd=True)
    for b in range(16):  # one token alone
        ref.close(spffn.q4_matvec(w, x[b].to(DEV)).cpu()[None], y[b:b + 1], bound[b:b + 1],
                  any_odd=True)


def test_small_values_next_to_an_outlier():
    rows, cols = 64, 256
    w, wd, g = make(rows, cols, 32, False, seed=4)
    x = torch.randn(2, cols, generator=g)
    x[0, 17] = 3e4
    x[1, :128] *= 2.0 ** -20
    x[1, 5] = 1.0
    y, bound = ref.q4_matvec(wd, x)
    ref.close(spffn.q4_matvec(w, x.to(DEV)).cpu(), y, bound)


def test_every_code_and_zero_point_is_exact():
    # one-hot activations read the weights back, rounded to fp32 once
    cols = 64
    codes = torch.arange(16, dtype=torch.uint8).repeat(16, 4)[:, :cols]  # code c % 16 in column c
    z = torch.arange(16, dtype=torch.uint8).view(16, 1)
    packed = (codes[:, 0::2] | codes[:, 1::2] << 4).contiguous()
    scales = (torch.arange(16).view(16, 1) * 0.0371 + 0.01).half()
    w = spffn.Q4Matrix(packed.to(DEV), scales.to(DEV), z.to(DEV), group=64)
    wd = ref.q4_weights(packed, scales, z, 64)
    for c0 in range(0, cols, 16):
        x = torch.zeros(16, cols)
        x[torch.arange(16), torch.arange(c0, c0 + 16)] = 1.0
        got = spffn.q4_matvec(w, x.to(DEV)).cpu()
        assert torch.equal(got.double(), wd[:, c0:c0 + 16].t())


def test_repeats_are_bitwise_equal_and_rows_before_after_untouched():
    rows, cols, B = 301, 1312, 6
    w, _, g = make(rows, cols, 64, True, seed=6)
    x = torch.randn(B, cols, generator=g).to(DEV)
    big = torch.full((B * rows + 64,), -7.0, device=DEV)
    y = big[32:32 + B * rows].view(B, rows)
    first = spffn.q4_matvec(w, x, y=y).clone()
    for _ in range(3):
        assert torch.equal(spffn.q4_matvec(w, x), first)
    assert bool((big[:32] == -7).all()) and bool((big[-32:] == -7).all())


def test_other_stream_and_graph():
    rows, cols, B = 530, 2048, 4
    w, _, g = make(rows, cols, 32, False, seed=7)
    x = torch.randn(B, cols, generator=g).to(DEV)
    y = torch.empty(B, rows, device=DEV)
    want = spffn.q4_matvec(w, x, rms_eps=1e-6)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        spffn.q4_matvec(w, x, rms_eps=1e-6, y=y)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spffn.q4_matvec(w, x, rms_eps=1e-6, y=y)
    for i in range(4):
        x.copy_(torch.randn(B, cols, generator=g))
        want = spffn.q4_matvec(w, x, rms_eps=1e-6)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


@pytest.mark.parametrize("B", [1, 2, 7, 16])
def test_views_that_are_only_aligned_to_an_element(B):
    rows, cols = 77, 416
    w, host, g = make(rows, cols, 32, True, seed=8)
    x = torch.randn(B, cols, generator=g)
    bias, resid = torch.randn(rows, generator=g), torch.randn(B, rows, generator=g)
    at = lambda t: torch.cat([t.new_zeros(1), t.flatten()]).to(DEV)[1:].view(t.shape)  # noqa: E731
    y = at(torch.zeros(B, rows))
    got = spffn.q4_matvec(w, x.to(DEV), bias=at(bias), resid=at(resid), y=y)
    want, bound = ref.q4_matvec(host, x, bias, resid)
    assert got is y
    ref.close(got.cpu(), want, bound)
