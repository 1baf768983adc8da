"""The bounded 4-bit cache at the sizes where a call takes another way: how row weights are summed, how the parts of a
split query are joined, more sequences than a grid has rows."""
import numpy as np
import pytest

from tests._util import bf16_out_to_f64, to_dev, to_dev_any
from tests.test_fp4_cache import attend, check_attention, reference, sti  # noqa: F401  (the fixture among them)
from workloads import bf16_bits_to_f32, rng_for, to_bf16_bits

gpu = pytest.mark.gpu

WEIGHTS = {
    # name: b, s, h, d, rows, start_pos, prev.   `tiles`: of 64 rows, of all sequences
    # scores kept, 4096 tiles or more: a block takes four tiles.  Sequence 0 ends a row into the second tile of a block,
    # which only its last query sees; a query more sees each further row of sequence 1
    "kept_four_tiles_a_block": (2, 4, 64, 64, 131067, [64 * 1501 + 61, 131064], True),
    "kept_four_tiles_one_query": (33, 1, 40, 64, 8001, None, False),
    "kept_four_tiles_shared": (3, 20, 7, 64, 90001, [64 * 1200 + 40, 5, 200000], True),   # three groups, the last of two queries
    # computed again, by every CTA for all queries, 40 tiles a CTA: one chunk of 32 and one of the rest
    "again_one_split_long": (1, 3, 40, 64, 64 * 6000 - 7, [64 * 6000 - 9], True),
    # the same for many sequences of one tile
    "again_one_split_sequences": (2500, 9, 33, 64, 64, None, False),
    # computed again, CTAs split over the queries too: a query each, and several with pieces that cut sequences
    "again_split_each": (2, 20, 64, 64, 2560, [2540, 1000], True),
    "again_split_several": (3, 70, 64, 128, 9600, [9530, 4000, 70], False),
    "again_split_shared": (2, 41, 16, 64, 9000, [8960, 31], True),
}


def make(name, b, s, h, d, rows, sp, prev):
    """Random codes and scales 1/8 .. 7/4 (finite), scores of a few units."""
    rng = rng_for(9800 + len(name), rows + h)
    a = dict(q=to_bf16_bits(rng.standard_normal((b, s, h, d))), codes=rng.integers(0, 256, (b, rows, d // 2), np.uint8),
             scales=rng.integers(0x20, 0x3F, (b, rows, d // 16), np.uint8),
             start_pos=np.array(sp if sp is not None else rng.integers(0, rows, b), np.int32), ratio=1, scale=0.5 * d ** -0.5,
             sink=rng.standard_normal(h).astype(np.float32), dropped=None, prev_out=None, prev_lse=None)
    if prev:
        a["prev_out"] = to_bf16_bits(rng.standard_normal((b, s, h, d)))
        a["prev_lse"] = (8 + rng.standard_normal((b, s, h))).astype(np.float32)
    a["w0"] = rng.random((b, rows)).astype(np.float32)
    return a


def check(sti, orc, a):  # noqa: F811
    """check_attention, some sequences at a time.  The fp32 running sums of long rows come beside its tolerances: l
    takes one addition per 64 rows, each off by at most 2^-24 of the sum, so lse, and by e^lse the weights, may be off by
    `run` more; that much is taken off their errors first."""
    out, lse, w = attend(sti, a)
    out, lse, w = bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), w.cpu().numpy().astype(np.float64)
    b, rows = a["w0"].shape
    run = (rows + 63) // 64 * 2.0 ** -24

    def nearer(got, want, by):
        with np.errstate(invalid="ignore"):
            err = np.nan_to_num(got - want, posinf=np.inf, neginf=-np.inf)
            return np.where(np.abs(err) <= by, want, got - np.sign(err) * by)

    step = max(1, 200000 // rows)
    for i in range(0, b, step):
        at = slice(i, i + step)
        one = {k: v[at] if isinstance(v, np.ndarray) and k != "sink" else v for k, v in a.items()}
        ref = reference(orc, one)
        check_attention(out[at], nearer(lse[at], ref[1], run), ref, bf16_bits_to_f32(one["q"]), one["codes"], one["scales"],
                        a["scale"], nearer(w[at], one["w0"] + ref[2], run * ref[2]), one["w0"])


@gpu
@pytest.mark.parametrize("name", list(WEIGHTS))
def test_row_weights(sti, orc, name):  # noqa: F811
    check(sti, orc, make(name, *WEIGHTS[name]))


@gpu
@pytest.mark.parametrize("b", [2, 20, 60, 130])
def test_one_long_sequence_among_short_ones(sti, orc, b):  # noqa: F811
    """The long sequence's query is split between nearly all SMs, whatever the number of sequences suggests."""
    rows = 20000
    sp = [200 + 7 * i for i in range(b)]
    sp[b // 2] = rows - 1
    check(sti, orc, make("one_long", b, 1, 5, 64, rows, sp, True))


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e8m0"])
def test_append_more_sequences_than_a_grid_has_rows(sti, orc, fmt):  # noqa: F811
    import torch

    b, dim, rows = 65536 + 70, 64, 3
    rng = rng_for(9900, dim)
    bits = to_bf16_bits(rng.standard_normal((b, 1, dim)))
    start = rng.integers(0, 4 * rows, b).astype(np.int32)           # one token of four: every fourth completes a row
    per = dim // (16 if fmt == "e4m3" else 32)
    codes = torch.full((b, rows, dim // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((b, rows, per), 0xCD, dtype=torch.uint8, device="cuda")
    pos = torch.full((b, rows), -5, dtype=torch.int32, device="cuda")
    weight = torch.full((b, rows), 3.0, device="cuda")
    sti.kv_append_fp4(to_dev(bits), to_dev_any(start), 1, 4, codes, scales, row_pos=pos, row_weight=weight)
    want = [np.full(t.shape, v, t.cpu().numpy().dtype) for t, v in ((codes, 0xAB), (scales, 0xCD), (pos, -5), (weight, 3.0))]
    new_codes, new_scales = orc.fp4_rows(bf16_bits_to_f32(bits), fmt)
    done = np.flatnonzero(start % 4 == 3)
    row = start[done] // 4
    assert len(done) > 10000 and done[-1] >= 65536
    for t, v in zip(want, (new_codes[done, 0], new_scales[done, 0], row, 0.0)):
        t[done, row] = v
    for t, v in zip((codes, scales, pos, weight), want):
        np.testing.assert_array_equal(t.cpu().numpy(), v)


@gpu
def test_attend_more_sequences_than_a_grid_has_rows(sti, orc):  # noqa: F811
    """Row weights of 65,606 sequences (their scores do not fit the kept ones' room)."""
    import torch

    b, h, d, rows = 65536 + 70, 2, 64, 3
    a = make("many", b, 1, h, d, rows, None, False)
    out, lse, w = attend(sti, a)
    some = np.r_[0:40, 65500:65606]
    part = {k: v[some] if isinstance(v, np.ndarray) and k != "sink" else v for k, v in a.items()}
    ref = reference(orc, part)
    at = torch.tensor(some, device="cuda")
    check_attention(bf16_out_to_f64(out[at]), lse[at].cpu().numpy().astype(np.float64), ref, bf16_bits_to_f32(part["q"]),
                    part["codes"], part["scales"], a["scale"], w[at].cpu().numpy().astype(np.float64), part["w0"])
