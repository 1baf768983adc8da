"""The bounded 4-bit cache where its numbers or its callers are at an edge: rows far below a head's largest."""
import numpy as np
import pytest

from tests.test_fp4_cache import sti  # noqa: F401  (the fixture)

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("h, s, rows, at, gap", [
    (64, 304, 4096, 0, 14.0), (64, 304, 4096, 0, 17.5), (64, 304, 4096, 0, 19.0), (64, 304, 4095, 2000, 17.5),
    (8, 2432, 4096, 0, 17.5),           # eight queries share a tile
    (64, 160, 1 << 20, 0, 19.0),        # together the small rows weigh 0.6 %
])
def test_attend_rows_far_below_the_largest(sti, h, s, rows, at, gap):  # noqa: F811
    """One row scores `gap` above all the others and is zero where they are one: out there is their share,
    n e^-gap / (1 + n e^-gap), which lse and row_weight state too.  As many queries as SMs or more, so that a query's
    rows are one SM's.

    P is held relative to 2^-7 of the running maximum, so f16 takes at most 2^-32 (half its smallest step, 2^-25)
    or 2^-11 of each row's probability; scores: as in check_attention; the output rounds to bf16.  Running sums in
    fp32, each step off by at most half an ulp (2^-24) for l, one addition per 64 rows, and one ulp (2^-23) for the
    tensor core's, four per 64 rows."""
    import torch

    d, n = 64, rows - 1
    q = torch.zeros(1, s, h, d, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = 4.0
    codes = torch.full((1, rows, d // 2), 0x22, device="cuda", dtype=torch.uint8)       # ones ...
    codes[..., :8] = 0                                                                  # ... after the first group
    codes[0, at] = 0
    codes[0, at, 0] = 0x07                                                              # 6 in the first element
    scales = torch.full((1, rows, d // 16), 0x38, device="cuda", dtype=torch.uint8)     # 1
    start = torch.tensor([rows * 2 * s], device="cuda", dtype=torch.int32)
    lse = torch.empty(1, s, h, device="cuda")
    w = torch.zeros(1, rows, device="cuda")
    scale = float(np.float32(gap / 24))
    out = sti.attn_fp4kv(q, codes, scales, start, 2 * s, scale, lse=lse, row_weight=w).double().cpu().numpy()
    g = 24 * scale
    small = np.exp(-g)                       # of one row, next to the largest's 1
    total = 1 + n * small
    ds = (d / 16 + 2) * 2.0 ** -23 * g
    run = (rows + 63) // 64 * 2.0 ** -24
    want = np.zeros(d)
    want[0], want[16:] = 6 / total, n * small / total
    tol = want * (2.0 ** -8 + 2.0 ** -11 + 2 * ds + 2.0 ** -19 + 9 * run) + n * 2.0 ** -32 * (want > 0)
    err = np.abs(out - want).max(axis=(0, 1, 2))
    assert (err <= tol).all(), f"{(err[16:] / want[16:]).max():.3g} of the small rows' share, {err[0]:.3g} of the large row's"
    np.testing.assert_allclose(lse.double().cpu().numpy(), g + np.log(total), rtol=0, atol=ds + 2.0 ** -19 + 2.0 ** -21 * g + run)
    each = np.full(rows, h * s * small / total)
    each[at] = h * s / total
    rel = 2 * ds + 2.0 ** -19 * (1 + g) + 64 * s * 2.0 ** -24 + run
    np.testing.assert_allclose(w.double().cpu().numpy()[0], each, rtol=rel)
