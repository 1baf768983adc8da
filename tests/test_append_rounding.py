"""The append's quantisation at every border.  On the CPU: the 12-bit rounding of its quotients, for every bf16 value, every
scale and a reciprocal as far off as an approximate one may be.  On the GPU: every bf16 value beside every scale
for which it lies among the codes' borders, and every value as its group's largest."""
import numpy as np
import pytest

from tests._util import to_dev
from tests.test_fp4_cache import sti  # noqa: F401  (the fixture)
from workloads import bf16_bits_to_f32

gpu = pytest.mark.gpu

FINITE = np.arange(0x7F80, dtype=np.uint32).astype(np.uint16)          # the finite values that are not negative
# a value past a border belongs to the code above it; on it, to the even one of the two
BORDERS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))
E4M3 = np.array([k * 2.0 ** -9 if k < 8 else (1 + k % 8 / 8) * 2.0 ** (k // 8 - 7) for k in range(127)])


def code_of(x, s):
    """E2M1 magnitude code of x / s (x >= 0, s > 0): x against border * s, both exact in fp64."""
    code = np.zeros(np.broadcast(x, s).shape, np.uint8)
    for border, upper in BORDERS:
        code += (x >= border * s) if upper else (x > border * s)
    return code


def round12(q):
    """The kernel's rounding of an fp32 value to 12 significant bits, ties away."""
    return ((q.view(np.uint32) + np.uint32(0x800)) & np.uint32(0xFFFFF000)).view(np.float32)


@pytest.mark.parametrize("ulps", [-2, -1, 0, 1, 2])
def test_codes_by_an_approximate_reciprocal(ulps):
    """x / s as fp32 x times a reciprocal of s that is up to two ulps off, rounded to 12 bits: the same code as by
    comparing x with the borders, for every finite x and every positive E4M3 scale."""
    x = bf16_bits_to_f32(FINITE)[None]
    s = E4M3[1:, None]
    r = (np.float32(1) / s.astype(np.float32)).view(np.int32) + np.int32(ulps)
    with np.errstate(over="ignore"):
        q = round12((x * r.view(np.float32)).astype(np.float32))
    np.testing.assert_array_equal(code_of(q.astype(np.float64), np.float64(1)), code_of(x.astype(np.float64), s))


def test_scale_byte_of_every_maximum():
    """E4M3(max / 6) by an fp32 product with 1/6 rounded to 12 bits: the nearest E4M3 value, ties to the even byte, 448 at
    most."""
    x = bf16_bits_to_f32(FINITE)
    with np.errstate(over="ignore"):
        q = round12(x * (np.float32(1) / np.float32(6))).astype(np.float64)
    x = x.astype(np.float64)

    def nearest(v, unit):       # v / unit among E4M3; unit: 6 compares v with 6 times the borders, exact in fp64
        border = (E4M3[:-1] + E4M3[1:]) / 2 * unit
        above = np.searchsorted(border, v, side="left")         # borders below v
        tie = (above < len(border)) & (v == border[np.minimum(above, len(border) - 1)])
        return np.where(tie & (above % 2 == 1), above + 1, above)

    np.testing.assert_array_equal(nearest(q, 1.0), nearest(x, 6.0))


def test_power_of_two_scale_of_every_maximum():
    """floor(log2 max) - 2 from the exponent field, subnormal values included; the quotient is exact."""
    x = bf16_bits_to_f32(FINITE[1:]).astype(np.float64)
    X = np.maximum(FINITE[1:].astype(int) // 128 - 129, -127)
    np.testing.assert_array_equal(X, np.clip(np.floor(np.log2(x)) - 2, -127, 127))
    r = np.ldexp(1.0, -X).astype(np.float32)
    np.testing.assert_array_equal((bf16_bits_to_f32(FINITE[1:]) * r).astype(np.float64), x * np.ldexp(1.0, -X))


def bits_of(v):
    """A value that bf16 holds exactly -> its pattern."""
    b = np.array([v], np.float32).view(np.uint32) >> 16
    assert bf16_bits_to_f32(b)[0] == v
    return b.astype(np.uint16)


def groups_with(values, top, group):
    """Groups that start with `top`, the rest filled with values (patterns), each with either sign."""
    both = np.concatenate([values, values | 0x8000])
    n = -(-len(both) // (group - 1))
    g = np.zeros((n, group), np.uint16)
    g[:, 0] = top
    g[:, 1:] = np.resize(both, (n, group - 1))
    return g


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e8m0"])
def test_append_every_value_beside_every_scale(sti, orc, fmt):  # noqa: F811
    import torch

    group = 16 if fmt == "e4m3" else 32
    f = bf16_bits_to_f32(FINITE).astype(np.float64)
    parts = []
    if fmt == "e4m3":
        for s in E4M3[1:]:
            parts.append(groups_with(FINITE[(f >= s / 8) & (f <= 6 * s)], bits_of(6 * s), group))
    else:
        for X in range(-127, 126):
            top = 2.0 ** (X + 2) * (2 - 2.0 ** -7)
            parts.append(groups_with(FINITE[(f >= 2.0 ** (X - 3)) & (f <= top)], bits_of(top), group))
    alone = np.zeros((2 * len(FINITE), group), np.uint16)               # every value as the largest
    alone[:, 5] = np.concatenate([FINITE, FINITE | 0x8000])
    x = np.concatenate(parts + [alone])
    x = np.concatenate([x, np.zeros((-len(x) % (64 // group), group), np.uint16)]).reshape(1, -1, 64)
    n = x.shape[1]
    codes = torch.zeros(1, n, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, n, 64 // group, dtype=torch.uint8, device="cuda")
    sti.kv_append_fp4(to_dev(x), torch.zeros(1, dtype=torch.int32, device="cuda"), n, 1, codes, scales)
    want_codes, want_scales = orc.fp4_rows(bf16_bits_to_f32(x), fmt)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)
    np.testing.assert_array_equal(codes.cpu().numpy(), want_codes)
    have = set(np.unique(want_scales).tolist())
    assert have >= (set(range(1, 127)) if fmt == "e4m3" else set(range(253)))
