"""4-bit products whose values lie near the ends of their types, and values that are not finite in every part of an operand,
through both kernels; and which of the two takes a call."""
import math

import pytest
import torch

import decode_ref as ref
import tensor_core_gemm_tcgen05_gb300 as g
from serving_ref import TYPES
from test_decode_gpu import clean, w4_inputs

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ctx():
    with g.Context(0) as c:
        yield c


def on_tensor_memory(ctx, call):
    """Whether a call takes the kernel that waits for loads (w4_umma_kernel): held back, they let its waits run out."""
    g.gemm_set_timeout_ns(ctx, 2_000_000)
    g.gemm_set_debug(ctx, g.GEMM_DEBUG_WITHHOLD_FIRST_LOAD)
    try:
        call()
        torch.cuda.synchronize()
        status = g.gemm_last_device_error(ctx)[0]
    finally:
        g.gemm_set_debug(ctx, 0)
        g.gemm_set_timeout_ns(ctx, 2_000_000_000)
    assert status in (g.GEMM_OK, g.GEMM_ERR_TIMEOUT)
    return status == g.GEMM_ERR_TIMEOUT


# outputs, columns, group: one step; several; a last step in part (of 256 and of 128 columns, where the group allows), more pieces of
# A than go to the sums by shuffles from five rows on; columns that a cluster shares
SHAPES = [(64, 256, 32), (136, 2048, 64), (136, 2048, 128), (264, 4224, 32), (264, 4224, 64), (264, 4224, 128), (16, 16384, 64),
          (16, 16384, 128)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,k,group", SHAPES)
def test_w4_few_rows_and_many_take_a_kernel_each(ctx, dtype, n, k, group):
    """What the tests below rely on: up to eight rows of these shapes take w4_kernel, more the other one."""
    for m in (1, 3, 8, 9, 40):
        a, codes, scales, zeros, _ = (x if x is None else x.cuda() for x in w4_inputs(m, n, k, group, TYPES[dtype], True))
        assert on_tensor_memory(ctx, lambda: g.w4_gemm(ctx, a, codes, scales, zeros)) == (m > 8), m
    clean(ctx)


def wide_bound(a, scales, k, group):
    """Up to eight rows in BF16, code A and zero A are summed apart: roundings are relative to (128 + 15) scale |A|."""
    mag = a.double().abs() @ scales.double().abs().repeat_interleave(group, 1).T
    return 143 * mag * 2.0 ** -23 * (group + k // group + 16)


@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("m", [1, 3, 8, 40])
@pytest.mark.parametrize("kind", ["one", "group", "cancelling", "largest", "every", "edge"])
def test_w4_activations_near_the_end_of_bf16(ctx, m, n, k, group, kind):
    """Finite values of any size, in one row among ordinary ones: whatever (code - zero) scale A is in FP32's range comes out."""
    a, codes, scales, zeros, bias = w4_inputs(m, n, k, group, BF16, True, seed=m)
    scales = (scales.double() * 2.0 ** -30).to(BF16)
    row, last = m // 2, k - group   # (the last group, in the last slice and step)
    if kind == "one":
        a[row, last + 7] = 3e36
    elif kind == "group":
        a[row, last :] = 1e34
    elif kind == "cancelling":
        a[row, last : last + 16 : 2] = 1e37
        a[row, last + 1 : last + 16 : 2] = -1e37
    elif kind == "largest":
        a[row, 5] = torch.finfo(BF16).max
    elif kind == "every":   # the group's sum of (code - zero) A leaves FP32's range, scaled it does not
        a[row, last :] = 1e38
    else:   # the largest that is still summed with the codes as they are
        a[row, last :] = float(torch.tensor(0x77ff, dtype=torch.int16).view(BF16))
    y, slack = ref.w4(a, codes, scales, zeros, bias, "none")
    assert float(y.abs().max()) < 3e38   # (a case of the range, not past it)
    if m <= 8:   # (in slices of the columns without larger values)
        slack = slack + wide_bound(torch.where(a.abs() < 2.0 ** 113, a, 0), scales, k, group)
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda())
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (m, n, k, group, kind))


@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("m", [2, 8, 40])
def test_w4_codes_above_and_below_the_zero(ctx, m, n, k, group):
    """A single value of 3e36 times a weight of 0.01, codes 9 and 7 around the zero of 8: 3e34 and -3e34."""
    a = torch.zeros(m, k, dtype=BF16)
    a[1, k - 3] = 3e36
    codes = torch.full((n, k // 2), 0x88, dtype=torch.uint8)
    codes[0::2], codes[1::2] = 0x99, 0x77
    scales = torch.full((n, k // group), 0.01, dtype=BF16)
    y, slack = ref.w4(a, codes, scales, None, None, "none")
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda()).cpu()
    clean(ctx)
    ref.check_w4(got, y, slack, (m, n, k, group))
    assert bool((got[1, 0::2] > 2.9e34).all()) and bool((got[1, 1::2] < -2.9e34).all())


@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("m", [1, 8, 40])
@pytest.mark.parametrize("kind", ["large scales", "small scales"])
def test_w4_scales_near_the_ends_of_bf16(ctx, m, n, k, group, kind):
    """Scales of 2^120 to 2^126 for activations of 2^-100, and results of about 2^-110."""
    a, codes, scales, zeros, _ = w4_inputs(m, n, k, group, BF16, True, seed=m)
    gen = torch.Generator().manual_seed(2)
    if kind == "large scales":
        a, scales = a.double() * 2.0 ** -100, scales.double() * 2.0 ** torch.randint(123, 127, scales.shape, generator=gen)
    else:
        a, scales = a.double() * 2.0 ** -60, scales.double() * 2.0 ** -50
    a, scales = a.to(BF16), scales.to(BF16)
    y, slack = ref.w4(a, codes, scales, zeros, None, "none")
    # sums are kept in units of 2^12 beyond eight rows: FP32's smallest numbers are then 2^-149 2^12, half of it off for each group and CTA
    slack = slack + 2.0 ** -138 * (k // group + 8) + (wide_bound(a, scales, k, group) if m <= 8 else 0.0)
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda())
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (m, n, k, group, kind))


@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("m", [1, 5, 8, 40])
def test_w4_activations_at_the_end_of_fp16(ctx, m, n, k, group):
    """FP16's largest values all over a group, of one sign and of both."""
    a, codes, scales, zeros, bias = w4_inputs(m, n, k, group, F16, True, seed=m)
    scales = (scales.double() * 2.0 ** -14).to(F16)   # (results of up to 128 15 65504 2^-14 0.15 = 1152)
    top = torch.finfo(F16).max
    a[0, k - group :] = top
    a[m // 2, : group // 2], a[m // 2, group // 2 : group] = top, -top
    y, slack = ref.w4(a, codes, scales, zeros, bias, "none")
    # up to eight rows the codes as they are, 15 at most, in the place of code - zero
    mag = a.double().abs() @ scales.double().abs().repeat_interleave(group, 1).T
    slack = slack + (15 * mag * 2.0 ** -23 * (group + k // group + 16) if m <= 8 else 0.0)
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda())
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (m, n, k, group))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,k,group", SHAPES)
@pytest.mark.parametrize("m", [1, 3, 5, 8, 40])
@pytest.mark.parametrize("place", ["first", "last"])
def test_w4_not_finite_anywhere(ctx, dtype, m, n, k, group, place):
    """NaN and infinities in the first or last group stay in their row; an infinity times a weight of 0 is NaN."""
    dt = TYPES[dtype]
    a, codes, scales, zeros, _ = w4_inputs(m, n, k, group, dt, True, seed=m)
    row, col = m - 1, 3 if place == "first" else k - 2
    y, slack = ref.w4(a, codes, scales, zeros, None, "none")
    if m <= 8:   # (a slice without them sums codes as they are)
        mag = a.double().abs() @ scales.double().abs().repeat_interleave(group, 1).T
        slack = slack + (143 if dt == BF16 else 15) * mag * 2.0 ** -23 * (group + k // group + 16)
    keep = torch.arange(m) != row
    dev = [x.cuda() for x in (codes, scales, zeros)]
    a[row, col] = math.nan
    got = g.w4_gemm(ctx, a.cuda(), *dev).cpu()
    clean(ctx)
    assert bool(got[row].isnan().all())
    ref.check_w4(got[keep], y[keep], slack[keep], (dtype, m, n, k, group, place))
    for sign in (1, -1):
        a[row, col] = sign * math.inf
        got = g.w4_gemm(ctx, a.cuda(), *dev).cpu()
        clean(ctx)
        ref.check_w4(got[keep], y[keep], slack[keep], (dtype, m, n, k, group, place, sign))
        code = codes[:, col // 2] // 16 if col % 2 else codes[:, col // 2] % 16
        w = (code.float() - (zeros[:, col // group] % 16).float()) * scales[:, col // group].float()
        want, out = w * (sign * math.inf), got[row].float()
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out[~out.isnan()], want[~want.isnan()])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("n,k,group", SHAPES)
def test_w4_the_same_rows_through_both_kernels(ctx, dtype, n, k, group):
    """Rows alone and among others differ by what each kernel's sums may be off and the last rounding."""
    dt = TYPES[dtype]
    a, codes, scales, zeros, bias = w4_inputs(24, n, k, group, dt, True)
    a[2, k - group :] *= 2.0 ** 100 if dt == BF16 else 2.0 ** 4
    scales = (scales.double() * 2.0 ** -7).to(dt)
    dev = [x.cuda() for x in (codes, scales, zeros, bias)]
    many = g.w4_gemm(ctx, a.cuda(), *dev).cpu()[:8]
    few = g.w4_gemm(ctx, a[:8].cuda(), *dev).cpu()
    clean(ctx)
    y, slack = ref.w4(a[:8], codes, scales, zeros, bias, "none")
    ref.check_w4(many, y, slack, "many")
    mag = a[:8].double().abs() @ scales.double().abs().repeat_interleave(group, 1).T
    wide = slack + (143 if dt == BF16 else 15) * mag * 2.0 ** -23 * (group + k // group + 16)
    ref.check_w4(few, y, wide, "few")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("m,n,k,group", [(300, 520, 1152, 128), (1000, 136, 512, 64), (4133, 264, 256, 32)])
def test_w4_prompts(ctx, dtype, m, n, k, group):
    a, codes, scales, zeros, bias = w4_inputs(m, n, k, group, TYPES[dtype], True)
    y, slack = ref.w4(a, codes, scales, zeros, bias, "gelu")
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), zeros.cuda(), bias.cuda(), g.EPI_GELU)
    clean(ctx)
    ref.check_w4(got.cpu(), y, slack, (dtype, m, n, k, group))


@pytest.mark.parametrize("m", [9, 70])
@pytest.mark.parametrize("act", ["none", "gelu", "relu"])
def test_w4_many_rows_without_columns(ctx, m, act):
    """Without columns every row is act(bias)."""
    bias = torch.linspace(-3, 3, 24).to(F16)
    a, codes, scales = torch.empty(m, 0, dtype=F16), torch.empty(24, 0, dtype=torch.uint8), torch.empty(24, 0, dtype=F16)
    got = g.w4_gemm(ctx, a.cuda(), codes.cuda(), scales.cuda(), None, bias.cuda(), {"none": g.EPI_NONE, "gelu": g.EPI_GELU, "relu": g.EPI_RELU}[act])
    clean(ctx)
    y, slack = ref.w4(a, codes, scales, None, bias, act)
    ref.check_w4(got.cpu(), y.expand(m, 24), slack, (m, act))
