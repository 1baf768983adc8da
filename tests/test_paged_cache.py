"""A paged cache of bf16 rows (rope_freqs, norm_rope, kv_append_paged, attn_paged) against the definitions in 64 bits."""
import ctypes
import math

import numpy as np
import pytest

from tests._util import bf16_out_to_f64, to_dev, to_dev_any
from tests.test_fp4_cache import FAKE, P, lib, sti  # noqa: F401  (fixtures among them)
from workloads import bf16_bits_to_f32, rng_for, to_bf16_bits

gpu = pytest.mark.gpu
NAN16 = np.uint16(0x7FC0)


def f64(bits):
    return bf16_bits_to_f32(bits).astype(np.float64)


def opt(v, up=to_dev_any):
    return None if v is None else up(v)


# ---------------------------------------------------------------------------------- definitions


def frequencies(rd, theta=10000.0, factor=1.0, orig=0, fast=32.0, slow=1.0):
    """Radians per position of each pair."""
    i = np.arange(rd // 2)
    f = theta ** (-2.0 * i / rd)
    if factor == 1.0:
        return f
    if orig == 0:
        return f / factor
    at = [rd * math.log(orig / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (fast, slow)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
    return f / factor * ramp + f * (1 - ramp)


def norm_rotate(x, pos, f, off, interleaved, inverse=False, gain=1.0, norm=True, weight=None, eps=1e-6):
    """x [..., h, d] at positions pos [...]; the result and the size that errors are relative to."""
    x = x.copy()
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight
    size = np.abs(x)
    if f is not None:
        rd = 2 * len(f)
        a = off + (np.arange(rd // 2) * 2 if interleaved else np.arange(rd // 2))
        b = a + (1 if interleaved else rd // 2)
        ang = pos[..., None] * f * (-1 if inverse else 1)
        c, s = np.cos(ang)[..., None, :] * gain, np.sin(ang)[..., None, :] * gain
        u, v = x[..., a], x[..., b]
        x[..., a], x[..., b] = u * c - v * s, v * c + u * s
        both = (size[..., a] + size[..., b]) * abs(gain)
        size[..., a] = size[..., b] = both
    return x, size


def check_rows(got, want, size):
    """bf16 rounding (2^-8 of the value) and fp32 arithmetic before it, on what the row's values are made of: the
    mean of up to 1024 squares summed in chains of at most 32 + 5 (37 2^-24, halved by the root), root, cos and sin to 2 ulp
    (2^-22 each), five products and sums (2^-24 each), an angle to 2^-24: below 2^-18 together, twice that here."""
    ok = np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * size
    assert ok.all(), f"{(~ok).sum()} of {ok.size} off, worst {np.abs(got - want).max():.3g}"


# ---------------------------------------------------------------------------------- frequencies (CPU)


@pytest.mark.parametrize("rd,theta,factor,orig", [(64, 1e4, 1, 0), (16, 1e4, 40, 4096), (128, 5e5, 8, 8192), (2, 1e4, 4, 0),
                                                  (1024, 1e6, 16, 65536), (64, 1e4, 0.5, 0), (64, 1e4, 16, 3)])
def test_frequencies(lib, rd, theta, factor, orig):  # noqa: F811
    turns = np.zeros(rd // 2, np.uint64)
    assert lib.sti_rope_freqs(rd, theta, factor, orig, 32.0, 1.0, turns.ctypes.data) == 0
    want = frequencies(rd, theta, factor, orig) / (2 * math.pi)
    # pow, a division and the ramp in 64 bits: a few 2^-53
    assert np.allclose(turns.astype(np.float64) * 2.0 ** -64, want % 1, rtol=2.0 ** -48, atol=2.0 ** -64)


def test_frequencies_refused(lib):  # noqa: F811
    t = np.zeros(512, np.uint64)
    good = dict(rd=64, theta=1e4, factor=1.0, orig=0, fast=32.0, slow=1.0, out=t.ctypes.data)
    call = lambda **k: lib.sti_rope_freqs(*{**good, **k}.values())  # noqa: E731
    assert call() == 0
    for kw in (dict(rd=0), dict(rd=63), dict(theta=1.0), dict(theta=float("nan")), dict(factor=0.0), dict(factor=float("inf")),
               dict(orig=-1), dict(fast=1.0), dict(slow=0.0), dict(out=None)):
        assert call(**kw) == 1, kw
    assert call(rd=1026) == 2


# ---------------------------------------------------------------------------------- norm and rotate


ROTATE = {
    # name: b, s, h, d, rd, off, interleaved, inverse, norm, weight, first positions, n_new, gain, factor
    "queries": (3, 2, 64, 512, 64, 448, True, False, True, False, [65534, 0, 9], None, 1.0, 16),
    "one_row": (1, 1, 1, 512, 64, 448, True, False, True, True, [5], None, 1.0, 1),
    "one_head_of_8": (5, 3, 1, 8, 8, 0, True, False, True, True, [1, 2, 3, 4, 5], None, 1.0, 1),
    "back": (2, 5, 20, 128, 128, 0, False, True, False, False, [1000000, 2 ** 31 - 6], None, 1.0, 1),
    "halves_mid": (2, 3, 5, 192, 32, 64, False, False, True, True, [77, 123456], None, 1.3, 40),
    "halves_across_chunks": (1, 7, 9, 512, 512, 0, False, False, True, True, [40000], None, 1.0, 4),
    "halves_16": (1, 7, 3, 40, 16, 24, False, False, True, True, [40000], None, 1.0, 4),
    "pairs_off_8": (2, 4, 3, 96, 72, 8, True, False, True, False, [0, 31], None, 0.7, 1),
    "d_1024": (1, 3, 10, 1024, 1024, 0, True, False, True, True, [7], None, 1.0, 1),
    "d_1024_halves": (1, 3, 7, 1024, 512, 512, False, False, True, True, [7], None, 1.0, 1),
    "no_rotation": (2, 3, 7, 320, 0, 0, True, False, True, True, [0, 3], None, 1.0, 1),
    "copy": (2, 3, 7, 64, 0, 0, True, False, False, False, [0, 3], None, 1.0, 1),
    "padded": (4, 37, 6, 64, 64, 0, True, False, True, False, [10, 20, 30, 40], [37, 0, 1, 36], 1.0, 1),
    "many_tokens": (2, 500, 3, 32, 16, 16, False, False, True, False, [0, 60000], [500, 499], 1.0, 8),
    "d_320": (2, 40, 5, 320, 64, 256, True, False, True, True, [3, 100000], [40, 33], 1.0, 1),
    "d_384": (1, 3, 50, 384, 128, 0, True, True, False, False, [9], None, 1.0, 1),
    "d_576": (3, 90, 1, 576, 64, 512, True, False, True, True, [0, 70, 8], [90, 0, 1], 1.0, 40),
    "d_768": (1, 5, 3, 768, 768, 0, True, False, True, False, [1], None, 1.0, 1),
    "d_576_halves": (3, 30, 1, 576, 48, 40, False, False, True, True, [0, 70, 8], [30, 2, 0], 1.0, 1),
    "d_320_halves": (2, 9, 8, 320, 304, 8, False, True, True, True, [3, 100000], None, 1.0, 1),
    "d_512_halves_mid": (2, 70, 3, 512, 16, 200, False, False, True, True, [3, 100000], None, 1.0, 1),
    "d_64_halves_all": (2, 700, 2, 64, 64, 0, False, False, True, True, [0, 9000], [700, 650], 1.0, 1),
    "d_128_many": (1, 3000, 8, 128, 96, 32, False, False, True, True, [17], None, 1.0, 1),
    "d_16_many": (7, 300, 1, 16, 16, 0, True, False, False, False, [0, 1, 2, 3, 4, 5, 6], None, 1.0, 1),
}


def make_rotate(name):
    b, s, h, d, rd, off, inter, inv, norm, weight, first, new, gain, factor = ROTATE[name]
    rng = rng_for(7100 + len(name), d + rd)
    x = to_bf16_bits(3 * rng.standard_normal((b, s, h, d)) * np.exp2(rng.integers(-20, 20, (b, s, h, 1))))
    w = to_bf16_bits(1 + 0.3 * rng.standard_normal(d)) if weight else None
    first = np.array(first, np.int32)
    pos = first[:, None].astype(np.int64) + np.arange(s)
    f = frequencies(rd, factor=factor, orig=4096 if factor != 1 else 0) if rd else None
    want, size = norm_rotate(f64(x), pos, f, off, inter, inv, gain, norm, None if w is None else f64(w))
    real = np.arange(s) < (np.array(new)[:, None] if new else s)
    return dict(x=x, w=w, first=first, want=want, size=size, real=np.broadcast_to(real, (b, s)),
                kw=dict(rope_off=off if rd else None, interleaved=inter, inverse=inv, gain=gain, norm=norm),
                n_new=None if new is None else np.array(new, np.int32), rd=rd,
                freqs=dict(factor=factor, orig_len=4096 if factor != 1 else 0))


@gpu
@pytest.mark.parametrize("name", list(ROTATE))
def test_rotate(sti, name):  # noqa: F811
    import torch

    a = make_rotate(name)
    freqs = sti.rope_freqs(a["rd"], **a["freqs"]) if a["rd"] else None
    x, out = to_dev(a["x"]), torch.full(a["x"].shape, -7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(weight=opt(a["w"], to_dev), n_new=opt(a["n_new"]), **a["kw"])
    got = sti.norm_rope(x, to_dev_any(a["first"]), freqs, out=out, **kw)
    assert got is out and (x == to_dev(a["x"])).all()
    y, real = bf16_out_to_f64(out), a["real"]
    check_rows(y[real], a["want"][real], a["size"][real])
    assert (y[~real] == -7).all()
    # positions token by token, and in place: the same bits
    each = to_dev_any((a["first"].astype(np.int64)[:, None] + np.arange(x.shape[1])).astype(np.int32))
    again = sti.norm_rope(x, each, freqs, out=x, **kw)
    assert again is x and (x[torch.from_numpy(real.copy())] == out[torch.from_numpy(real.copy())]).all()
    assert (x.cpu()[torch.from_numpy(~real)] == to_dev(a["x"]).cpu()[torch.from_numpy(~real)]).all()


@gpu
def test_rotate_strided(sti):  # noqa: F811
    """Parts of a fused projection [tokens, heads and latent]: queries in place beside the others, sequences and tokens in
    any order."""
    import torch

    b, s, h, d = 3, 5, 6, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    freqs, pos = sti.rope_freqs(32), torch.tensor([4, 5, 6], dtype=torch.int32, device="cuda")
    qkv = torch.randn(b, s, 3 * h * d, generator=g, device="cuda").bfloat16()
    keep = qkv.clone()
    part = lambda t, i: t[..., i * h * d:(i + 1) * h * d].unflatten(-1, (h, d))  # noqa: E731
    want = sti.norm_rope(part(keep, 0).contiguous(), pos, freqs)
    got = sti.norm_rope(part(qkv, 0), pos, freqs)
    assert (got == want).all() and (qkv == keep).all()
    sti.norm_rope(part(qkv, 0), pos, freqs, out=part(qkv, 2))
    assert (part(qkv, 2) == want).all() and (qkv[..., :2 * h * d] == keep[..., :2 * h * d]).all()
    tokens_first = part(keep, 0).transpose(0, 1).contiguous().transpose(0, 1)
    assert (sti.norm_rope(tokens_first, pos, freqs, out=tokens_first) == want).all()


@gpu
def test_rotate_there_and_back(sti):  # noqa: F811
    """Rotating back returns the row (two bf16 roundings of values of the pair's length, 2^-8 each)."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(2, 50, 4, 128, generator=g, device="cuda").bfloat16()
    pos, freqs = torch.tensor([0, 999999], dtype=torch.int32, device="cuda"), sti.rope_freqs(64)
    for inter in (True, False):
        there = sti.norm_rope(x, pos, freqs, interleaved=inter, norm=False)
        back = sti.norm_rope(there, pos, freqs, interleaved=inter, norm=False, inverse=True)
        r = x.float()[..., 64:]
        u, v = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :32], r[..., 32:])
        size = torch.hypot(u, v)
        size = torch.stack([size, size], -1).flatten(-2) if inter else torch.cat([size, size], -1)
        assert ((back.float()[..., 64:] - r).abs() <= (2 ** -8 * 2 ** 0.5 + 2 ** -8 + 2 ** -15) * size).all()
        assert (back[..., :64] == x[..., :64]).all()


@gpu
def test_rotate_special_rows(sti):  # noqa: F811
    """Rows of zeros stay zeros; a NaN stays in its row."""
    import torch

    x = torch.randn(1, 4, 3, 64, device="cuda").bfloat16()
    x[0, 1] = 0
    x[0, 2, 1, 5] = float("nan")
    pos = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sti.norm_rope(x, pos, sti.rope_freqs(32))
    assert (y[0, 1] == 0).all() and y[0, 2, 1].isnan().all()
    y[0, 2, 1] = 0
    assert y.isfinite().all()
    assert sti.norm_rope(x[:0], pos[:0], sti.rope_freqs(32)).shape == (0, 4, 3, 64)


# ---------------------------------------------------------------------------------- append


APPEND = {
    # name: b, s, d, rd, page, first positions, n_new, norm
    "decode": (6, 1, 512, 64, 64, [0, 63, 64, 127, 700, 5], None, True),
    "prompt": (2, 300, 512, 64, 64, [0, 130], None, True),
    "padded": (4, 50, 192, 64, 24, [0, 23, 24, 100], [50, 0, 1, 49], True),
    "as_they_are": (2, 33, 64, 0, 1, [0, 7], None, False),
    "page_100": (3, 70, 8, 8, 100, [99, 0, 50], None, True),
    "d_1024": (1, 9, 1024, 64, 7, [3], None, True),
}


def page_table(rng, b, need, spare=3):
    """need[i] pages of sequence i, anywhere in the pool; the table's other entries say so (-1)."""
    n = int(sum(need)) + spare
    order = rng.permutation(n).astype(np.int32)
    table = np.full((b, max(1, int(max(need)))), -1, np.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, n


@gpu
@pytest.mark.parametrize("name", list(APPEND))
def test_append(sti, name):  # noqa: F811
    import torch

    b, s, d, rd, page, first, new, norm = APPEND[name]
    rng = rng_for(7200 + len(name), d + page)
    first = np.array(first, np.int64)
    count = np.array(new if new else [s] * b)
    table, n = page_table(rng, b, -(-(first + s) // page))
    x = to_bf16_bits(2 * rng.standard_normal((b, s, d)))
    w = to_bf16_bits(1 + 0.3 * rng.standard_normal(d)) if norm else None
    f = frequencies(rd) if rd else None
    pairs = rd < 16                                         # (halves turn 16 dims at least)
    want, size = norm_rotate(f64(x)[:, :, None], first[:, None] + np.arange(s), f, d - rd, pairs, norm=norm,
                             weight=None if w is None else f64(w))
    pool = torch.full((n, page + 3, d + 0), -7.0, dtype=torch.bfloat16, device="cuda")
    pages = pool[:, :page]                                  # page strides of their own
    ws = sti.workspace(256)
    wide = torch.full((b, table.shape[1] + 2), -1, dtype=torch.int32, device="cuda")
    wide[:, :-2] = to_dev_any(table)
    sti.kv_append_paged(to_dev(x), to_dev_any(first.astype(np.int32)), pages, wide[:, :-2], sti.rope_freqs(rd) if rd else None,
                        interleaved=pairs, norm=norm, weight=opt(w, to_dev), n_new=None if new is None else to_dev_any(count.astype(np.int32)),
                        ws=ws)
    assert sti.read_device_status(ws) == 0
    got = bf16_out_to_f64(pool)
    for i in range(b):
        for t in range(count[i]):
            p = first[i] + t
            row = got[table[i, p // page], p % page]
            check_rows(row, want[i, t, 0], size[i, t, 0])
            got[table[i, p // page], p % page] = -7
    assert (got == -7).all()                                # nothing else was written


@gpu
def test_append_bad_pages(sti):  # noqa: F811
    """Rows past the table, or of pages that the pool does not have, are left out and reported."""
    import torch

    d, page = 64, 4
    x = torch.randn(4, 6, d, device="cuda").bfloat16()
    table = torch.tensor([[0, 1], [2, -1], [7, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    start = torch.tensor([4, 0, 0, 0], dtype=torch.int32, device="cuda")
    n_new = torch.tensor([6, 4, 6, 6], dtype=torch.int32, device="cuda")
    pages = torch.full((7, page, d), -7.0, dtype=torch.bfloat16, device="cuda")
    ws = sti.workspace(256)
    want = pages.clone()
    want[1], want[2], want[3, :2] = x[0, :4], x[1, :4], x[2, 4:6]
    sti.kv_append_paged(x, start, pages, table, ws=ws)
    assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
    assert (pages == want).all()
    sti.kv_append_paged(x[1:2], start[1:2], pages, table[1:2], n_new=n_new[1:2], ws=ws)
    assert sti.read_device_status(ws) == 0
    sti.kv_append_paged(x, start, pages, table)             # without a workspace: the same, unreported
    assert (pages == want).all()


# ---------------------------------------------------------------------------------- attention


ATTEND = {
    # name: b, s, h, d, page, start_pos, n_new, window, n_first, sink, prev
    "one_row": (1, 1, 64, 512, 64, [0], None, 0, 0, True, False),
    "one_row_window": (2, 1, 64, 512, 64, [0, 70], None, 1, 0, True, True),
    "one_tile_less": (2, 1, 64, 512, 64, [62, 10], None, 0, 0, True, False),
    "one_tile": (2, 1, 64, 512, 64, [63, 3], None, 0, 0, False, False),
    "one_tile_more": (2, 1, 64, 512, 64, [64, 63], None, 0, 0, False, True),
    "window_128": (3, 1, 64, 512, 64, [700, 127, 128], None, 128, 4, True, False),
    "window_over_all": (2, 1, 64, 512, 64, [99, 300], None, 5000, 64, True, False),
    "first_meets_window": (4, 1, 64, 128, 16, [105, 106, 107, 250], None, 100, 7, True, False),
    "first_past_the_start": (3, 1, 64, 64, 16, [99, 150, 260], None, 50, 200, True, True),
    "long_split": (1, 1, 64, 512, 64, [4998], None, 0, 0, True, True),
    "ragged": (6, 1, 64, 512, 100, [5000, 0, 1, 64, 1500, 4], None, 0, 0, True, True),
    "page_1": (2, 3, 64, 256, 1, [200, 0], None, 0, 0, True, False),
    "page_7": (2, 3, 64, 192, 7, [200, 90], None, 65, 3, True, False),
    "many_sequences": (200, 1, 64, 128, 16, None, None, 40, 2, True, False),
    "chunk": (2, 70, 64, 512, 64, [1200, 0], None, 0, 0, True, True),
    "chunk_window": (2, 300, 64, 512, 64, [1200, 0], None, 128, 4, True, False),
    "chunk_padded": (4, 40, 64, 320, 24, [300, 0, 77, 1], [40, 0, 1, 39], 30, 0, True, False),
    "long_queries": (1, 200, 64, 512, 64, [1300], None, 0, 0, True, False),
    "heads_33": (2, 2, 33, 320, 64, [399, 256], None, 0, 0, True, False),
    "few_heads": (3, 2, 5, 192, 24, [900, 333, 0], None, 0, 0, True, True),
    "one_head": (2, 3, 1, 64, 8, [250, 30], None, 20, 0, True, False),
    "packed_window": (2, 50, 5, 128, 16, [0, 333], None, 10, 3, True, True),
    "packed_first_inside": (2, 20, 3, 64, 16, [0, 90], None, 7, 95, True, False),
    "packed_window_1": (2, 100, 2, 64, 16, [0, 333], None, 1, 0, False, False),
    "packed_padded": (5, 9, 20, 128, 24, [0, 5, 900, 30, 2], [9, 0, 1, 8, 4], 33, 5, True, True),
    "packed_causal": (2, 300, 16, 128, 64, [0, 7], None, 0, 0, True, False),
    "packed_one_head": (3, 130, 1, 64, 64, [0, 5, 1], None, 0, 0, True, True),
    "packed_split": (1, 5, 12, 448, 64, [4990], None, 0, 0, True, True),
    # several queries per SM, each of a tile or two, for every number of 128-dim blocks
    "runs_d64": (2, 300, 64, 64, 16, [0, 90], None, 20, 0, True, False),
    "runs_d128_prev": (3, 250, 33, 128, 16, [5, 40, 0], [250, 0, 249], 64, 0, True, True),
    "runs_d256": (2, 400, 64, 256, 64, [70, 1], None, 60, 3, True, True),
    "runs_d384": (2, 350, 64, 384, 24, [300, 0], None, 100, 1, True, False),
    "runs_d448": (2, 300, 64, 448, 64, [64, 0], None, 1, 0, True, True),
    "runs_d512_prev": (2, 300, 64, 512, 64, [64, 0], None, 40, 2, False, True),
    "whole_16_tiles": (2, 90, 64, 192, 64, [900, 500], None, 940, 60, True, False),
    "pieces_of_4": (5, 1, 64, 320, 64, [1999, 0, 700, 64, 1300], None, 0, 0, True, True),
    "packed_runs_d320": (2, 700, 20, 320, 64, [0, 50], [700, 650], 33, 5, True, True),
    "packed_pairs_d448": (2, 5, 32, 448, 64, [380, 100], None, 0, 0, True, True),
    # lists cut into parts: few and many of them, of few and many queries, heads that fill no group of four
    "parts_13": (12, 1, 57, 64, 16, [1990 - 160 * i for i in range(12)], None, 0, 0, True, True),
    "parts_9_d512": (18, 1, 64, 512, 64, [1500, 3, 700] * 6, None, 0, 0, True, True),
    "parts_7_heads_33": (25, 1, 33, 448, 24, [1400 - 50 * i for i in range(25)], None, 0, 0, True, True),
    "parts_3": (60, 1, 64, 320, 64, [1500, 40, 900, 0] * 15, [1, 1, 0, 1] * 15, 0, 0, True, True),
    "parts_2_many_queries": (170, 1, 39, 128, 16, [1790 - 10 * i for i in range(170)], None, 0, 0, True, True),
    "parts_2_packed": (160, 3, 19, 64, 64, [1600, 900] * 80, [3, 0, 1, 2] * 40, 0, 0, True, True),
    "parts_many_one_head": (1, 1, 1, 64, 16, [9000], None, 0, 0, True, True),
    "parts_window": (3, 40, 64, 192, 64, [3000, 2500, 0], [40, 2, 40], 2000, 70, True, True),
}


def seen_by(P, window, first):
    """Positions that the query at P sees, as a mask over 0 .. P."""
    p = np.arange(P + 1)
    return (p > P - window) | (p < first) if window else p >= 0


def make_attend(name):
    b, s, h, d, page, start, new, window, first, sink, prev = ATTEND[name]
    rng = rng_for(7300 + len(name), d + h)
    start = np.array(start if start is not None else rng.integers(0, 300, b), np.int32)
    count = np.array(new if new else [s] * b, np.int32)
    need = -(-(start.astype(np.int64) + np.maximum(count, 1)) // page)
    table, n = page_table(rng, b, need)
    kv = [to_bf16_bits(rng.standard_normal((start[i] + count[i], d)) * np.exp2(rng.integers(-2, 2, (start[i] + count[i], 1))))
          for i in range(b)]
    pool = np.full((n, page, d), NAN16, np.uint16)          # rows that nothing sees hold NaN
    used = np.zeros((b, table.shape[1]), bool)
    for i in range(b):
        keep = np.zeros(start[i] + count[i], bool)
        for t in range(count[i]):
            keep[:start[i] + t + 1] |= seen_by(start[i] + t, window, first)
        for p in np.nonzero(keep)[0]:
            pool[table[i, p // page], p % page] = kv[i][p]
            used[i, p // page] = True
    table[~used] = -5                                       # and pages of which nothing is seen are not there
    a = dict(q=to_bf16_bits(2 * rng.standard_normal((b, s, h, d))), pool=pool, table=table, start=start, count=count,
             n_new=count if new else None, window=window, n_first=first, scale=d ** -0.5, kv=kv,
             sink=rng.standard_normal(h).astype(np.float32) if sink else None)
    a["prev_out"] = to_bf16_bits(rng.standard_normal((b, s, h, d))) if prev else None
    a["prev_lse"] = (4 + rng.standard_normal((b, s, h))).astype(np.float32) if prev else None
    if prev and h > 1:
        a["prev_lse"][0, 0, :2] = -np.inf                   # heads for which the other rows held nothing
    return a


def attend_reference(a, hidden=lambda i, p: np.zeros(len(p), bool)):
    """(out, lse, mass, largest sum |q k|) in 64 bits; hidden(i, positions): rows that do not exist."""
    q = f64(a["q"])
    b, s, h, d = q.shape
    out, lse = np.full((b, s, h, d), np.nan), np.full((b, s, h), np.nan)
    mass = np.zeros((b, s, h, d))
    sabs = 0.0
    for i in range(b):
        kv = f64(a["kv"][i])
        for t in range(a["count"][i]):
            p = np.nonzero(seen_by(a["start"][i] + t, a["window"], a["n_first"]))[0]
            p = p[~hidden(i, p)]
            k = kv[p]
            x = a["scale"] * q[i, t] @ k.T
            if len(p):
                sabs = max(sabs, a["scale"] * float((np.abs(q[i, t]) @ np.abs(k).T).max()))
            parts = [x]
            if len(p) and a["sink"] is not None:
                parts.append(a["sink"].astype(np.float64)[:, None])
            if a["prev_lse"] is not None:
                parts.append(a["prev_lse"][i, t].astype(np.float64)[:, None])
            z = np.concatenate(parts, 1)
            top = z.max(1, initial=-np.inf)
            ref = np.where(np.isinf(top), 0, top)
            with np.errstate(divide="ignore"):
                L = ref + np.log(np.exp(z - ref[:, None]).sum(1))
            pr = np.exp(x - np.where(np.isinf(L), 0, L)[:, None])
            o, m = pr @ k, pr @ np.abs(k)
            if a["prev_lse"] is not None:
                c = np.where(np.isinf(L), 0, np.exp(a["prev_lse"][i, t] - np.where(np.isinf(L), 0, L)))[:, None]
                o, m = o + c * f64(a["prev_out"][i, t]), m + c * np.abs(f64(a["prev_out"][i, t]))
            out[i, t], lse[i, t], mass[i, t] = o, L, m
    return out, lse, mass, sabs


def check_attention(a, got, got_lse, ref):
    """Element by element.  Score error ds: fp32 accumulation of d products, each step of 16 off by at most an ulp of the
    running sum, and the factor, product and difference of the exponent: (d / 16 + 6) 2^-23 of sum |q k|.  A
    probability is off by 2 ds (its own and the sum's) and bf16 rounding (2^-8), the exponential's 2 ulp and the
    sums' roundings (n / 16 + 16) 2^-23; the output by bf16 rounding (2^-8)."""
    out, lse, mass, sabs = ref
    d = out.shape[-1]
    n = max(len(k) for k in a["kv"])
    ds = (d / 16 + 6) * 2.0 ** -23 * sabs
    real = np.arange(out.shape[1]) < a["count"][:, None]
    err = np.abs(got - out)[real]
    tol = (2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * ds + (n / 16 + 16) * 2.0 ** -23) * mass)[real]
    assert (err <= tol).all(), f"out: {(err - tol).max():.3g} over, worst {err.max():.3g}"
    g, w = got_lse[real], lse[real]
    assert np.array_equal(np.isneginf(g), np.isneginf(w))
    fin = np.isfinite(w)
    lerr = np.abs(g[fin] - w[fin])
    assert (lerr <= ds + 2.0 ** -19 + 2.0 ** -21 * np.abs(w[fin])).all(), f"lse: {lerr.max():.3g}"
    assert (got[~real] == -7).all() and (got_lse[~real] == -7).all()


def attend(sti, a, **more):  # noqa: F811
    import torch

    out = torch.full(a["q"].shape, -7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(a["q"].shape[:3], -7.0, device="cuda")
    ws = more.pop("ws", None)
    ws = sti.workspace(sti.attn_paged_workspace_size(*a["q"].shape)) if ws is None else ws
    kw = dict(window=a["window"], n_first=a["n_first"], attn_sink=opt(a["sink"]), prev_out=opt(a["prev_out"], to_dev),
              prev_lse=opt(a["prev_lse"]), n_new=opt(a["n_new"]), out=out, lse=lse, ws=ws)
    sti.attn_paged(to_dev(a["q"]), to_dev(a["pool"]), to_dev_any(a["table"]), to_dev_any(a["start"]), a["scale"], **{**kw, **more})
    return out, lse, ws


@gpu
@pytest.mark.parametrize("name", list(ATTEND))
def test_attend(sti, name):  # noqa: F811
    a = make_attend(name)
    out, lse, ws = attend(sti, a)
    assert sti.read_device_status(ws) == 0
    check_attention(a, bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), attend_reference(a))
    again, lse2, _ = attend(sti, a, ws=ws)                  # the same bits, whatever the workspace held
    assert (again == out).all() and (lse2 == lse).all()
    if a["prev_out"] is not None and a["n_new"] is None:
        po = to_dev(a["prev_out"])
        attend(sti, a, prev_out=po, out=po, lse=None)       # in place of prev_out, without lse
        assert (po == out).all()


@gpu
@pytest.mark.parametrize("h,s", [(64, 1), (6, 5), (32, 2)])
def test_attend_bad_pages(sti, h, s):  # noqa: F811
    """Pages outside the pool and positions past the table count as rows that nothing sees, and are reported; a query left
    without rows keeps what it had (prev), or gives 0 and -inf."""
    import torch

    b, d, page = 4, 64, 16
    rng = rng_for(7400, h)
    start = np.array([90, 100, 40, 15], np.int32)
    table, n = page_table(rng, b, [7, 7, 7, 7])
    kv = [to_bf16_bits(rng.standard_normal((112, d))) for _ in range(b)]
    pool = np.zeros((n, page, d), np.uint16)
    for i in range(b):
        for p in range(112):
            pool[table[i, p // page], p % page] = kv[i][p]
    table[0, 2], table[0, 5] = -1, n
    table[2] = [n, -2, 2 ** 31 - 1, -2 ** 31, -1, -1, -1]
    a = dict(q=to_bf16_bits(2 * rng.standard_normal((b, s, h, d))), pool=pool, table=table, start=start,
             count=np.full(b, s, np.int32), n_new=None, window=0, n_first=0, scale=d ** -0.5, kv=kv,
             sink=rng.standard_normal(h).astype(np.float32), prev_out=None, prev_lse=None)

    def hidden(i, p):
        return np.isin(p // page, [2, 5]) if i == 0 else np.full(len(p), i == 2)

    for prev in (False, True):
        if prev:
            a["prev_out"] = to_bf16_bits(rng.standard_normal((b, s, h, d)))
            a["prev_lse"] = (4 + rng.standard_normal((b, s, h))).astype(np.float32)
        out, lse, ws = attend(sti, a)
        assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
        check_attention(a, bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), attend_reference(a, hidden))
        if not prev:
            assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    # a table that ends before the queries do: the positions behind it are not seen
    cut = dict(a, table=np.ascontiguousarray(a["table"][:, :3]))
    out, lse, ws = attend(sti, cut)
    assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
    check_attention(cut, bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64),
                    attend_reference(cut, lambda i, p: hidden(i, p) | (p >= 48)))
    none = dict(a, table=np.zeros((b, 0), np.int32))
    out, lse, ws = attend(sti, none)
    assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
    assert (out == to_dev(a["prev_out"])).all() and (lse == to_dev_any(a["prev_lse"])).all()


@gpu
@pytest.mark.parametrize("h,s,window", [(8, 8, 0), (8, 20, 5), (64, 6, 0), (64, 6, 3)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_attend_non_finite_row(sti, h, s, window, value):  # noqa: F811
    """A row with a NaN or infinity changes nothing for the queries that do not see it, also where those that do share
    their tiles."""
    import torch

    d, page, at = 128, 16, 37
    g = torch.Generator(device="cuda").manual_seed(s)
    q = torch.randn(1, s, h, d, generator=g, device="cuda").bfloat16()
    pages = torch.randn(4, page, d, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[2, 0, 3, 1]], dtype=torch.int32, device="cuda")
    start = torch.tensor([35], dtype=torch.int32, device="cuda")
    want = sti.attn_paged(q, pages, table, start, d ** -0.5, window=window)
    pages[3, at - 32, 5] = value
    lse = torch.empty(1, s, h, device="cuda")
    got = sti.attn_paged(q, pages, table, start, d ** -0.5, window=window, lse=lse)
    P = 35 + torch.arange(s)
    sees = (P >= at) & ((P - at < window) | (window == 0))
    assert (got[0, ~sees] == want[0, ~sees]).all() and lse[0, ~sees].isfinite().all()
    assert got[0, sees].isnan().any(-1).all()


@gpu
@pytest.mark.parametrize("h", [64, 4])
def test_attend_extreme_scores(sti, h):  # noqa: F811
    """Scores whose largest grows along the rows by more than a bf16 P could hold, and rows far below it."""
    rng = rng_for(7500, h)
    d, n = 64, 700
    kv = rng.standard_normal((n, d)) * 0.05
    kv[:, 0] += np.linspace(-60, 60, n)
    q = rng.standard_normal((1, 2, h, d)) * 0.1
    q[..., 0] = np.where(np.arange(h) % 2, 40.0, -40.0)
    kvb = to_bf16_bits(kv)
    pool = np.zeros((n // 100, 100, d), np.uint16)
    pool.reshape(-1, d)[:] = kvb
    a = dict(q=to_bf16_bits(q), pool=pool, table=np.arange(7, dtype=np.int32)[None], start=np.array([n - 2], np.int32),
             count=np.array([2], np.int32), n_new=None, window=0, n_first=0, scale=d ** -0.5, kv=[kvb], sink=None,
             prev_out=None, prev_lse=None)
    out, lse, _ = attend(sti, a)
    check_attention(a, bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), attend_reference(a))


@gpu
def test_attend_far_pages(sti):  # noqa: F811
    """A pool whose last pages lie past 2^31 elements, and a page stride of its own."""
    import torch

    d, page, n = 512, 64, 66000
    pool = torch.empty(n, page + 1, d, dtype=torch.bfloat16, device="cuda")      # 4.4 GB
    pages = pool[:, :page]
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn(1, 200, d, generator=g, device="cuda").bfloat16()
    q = torch.randn(1, 1, 64, d, generator=g, device="cuda").bfloat16()
    last = torch.tensor([199], dtype=torch.int32, device="cuda")
    near = torch.zeros(4, page, d, dtype=torch.bfloat16, device="cuda")
    out = []
    for where, ids in ((near, [0, 1, 2, 3]), (pages, [n - 1, 65999 - 40, n - 7, 65600])):
        table = torch.tensor([ids], dtype=torch.int32, device="cuda")
        sti.kv_append_paged(rows, last * 0, where, table, sti.rope_freqs(64), norm=True)
        out.append(sti.attn_paged(q, where, table, last, d ** -0.5))
    assert (out[0] == out[1]).all()


# ---------------------------------------------------------------------------------- together


def layer_step(sti, st, x, n_new=None):  # noqa: F811
    """One step of a layer: queries and rows from x [b, s, (h + 1) d], both normed and rotated, the rows appended, the
    window attended, joined with the attention over the older rows' 4-bit copies, rotated back."""
    h, d = st["h"], st["d"]
    b, s, _ = x.shape
    q = sti.norm_rope(x[..., :h * d].unflatten(-1, (h, d)), st["pos"], st["freqs"], n_new=n_new)
    sti.kv_append_paged(x[..., h * d:], st["pos"], st["pages"], st["table"], st["freqs"], norm=True, weight=st["w"], n_new=n_new)
    prev = lse = None
    if st["codes"] is not None:
        import torch

        lse = torch.empty(b, s, h, device=x.device)
        prev = sti.attn_fp4kv(q, st["codes"], st["scales"], st["seen"], 1, st["scale"], lse=lse)
    o = sti.attn_paged(q, st["pages"], st["table"], st["pos"], st["scale"], window=st["window"], n_first=st["first"],
                       attn_sink=st["sink"], prev_out=prev, prev_lse=lse, n_new=n_new)
    o = sti.norm_rope(o, st["pos"], st["freqs"], inverse=True, norm=False, n_new=n_new)
    st["pos"] += s if n_new is None else n_new
    return o


def layer_state(sti, b, h, d, page, most, window, first, older=0):  # noqa: F811
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)
    st = dict(h=h, d=d, window=window, first=first, scale=d ** -0.5, freqs=sti.rope_freqs(32),
              pos=torch.zeros(b, dtype=torch.int32, device="cuda"), w=torch.rand(d, generator=g, device="cuda").bfloat16() + 0.5,
              sink=torch.randn(h, generator=g, device="cuda"), codes=None,
              pages=torch.full((b * most, page, d), float("nan"), dtype=torch.bfloat16, device="cuda"),
              table=torch.randperm(b * most, generator=g, device="cuda").int().view(b, most))
    if older:
        st["codes"] = torch.randint(0, 256, (b, older, d // 2), generator=g, device="cuda", dtype=torch.uint8)
        st["scales"] = torch.randint(40, 56, (b, older, d // 16), generator=g, device="cuda", dtype=torch.uint8)
        st["seen"] = torch.full((b,), older - 1, dtype=torch.int32, device="cuda")
    return st


@gpu
@pytest.mark.parametrize("window,first", [(0, 0), (20, 3)])
def test_prompt_chunks_tokens_agree(sti, window, first):  # noqa: F811
    """A whole prompt, the same in padded chunks, and token by token give the same outputs up to the order of sums (P
    rounded to bf16 relative to other maxima: 2^-8 of sum p |row| each, rows within 4, and the output's 2^-8, twice each and
    rotated, which mixes two dims)."""
    import torch

    b, h, d, n = 2, 12, 64, 61
    x = torch.randn(b, n, (h + 1) * d, generator=torch.Generator(device="cuda").manual_seed(6), device="cuda").bfloat16()
    whole = layer_step(sti, layer_state(sti, b, h, d, 8, 8, window, first), x).float()
    tokens = layer_state(sti, b, h, d, 8, 8, window, first)
    one = torch.cat([layer_step(sti, tokens, x[:, t:t + 1]) for t in range(n)], 1).float()
    chunks = layer_state(sti, b, h, d, 8, 8, window, first)
    got = torch.zeros_like(whole)
    at = [0, 0]
    for sizes in ((10, 7), (1, 0), (0, 25), (25, 25), (25, 4)):
        pad = torch.full((b, 25, (h + 1) * d), float("nan"), dtype=torch.bfloat16, device="cuda")
        for i in range(b):
            pad[i, :sizes[i]] = x[i, at[i]:at[i] + sizes[i]]
        o = layer_step(sti, chunks, pad, torch.tensor(sizes, dtype=torch.int32, device="cuda"))
        for i in range(b):
            got[i, at[i]:at[i] + sizes[i]] = o[i, :sizes[i]]
            at[i] += sizes[i]
    assert at == [n, n]
    for other in (one, got):
        assert (other - whole).abs().max() <= 2 * (4 + 4) * 2 ** -8 * 2 ** 0.5 + 4 * 2 ** -8
    assert (tokens["pages"].nan_to_num() == chunks["pages"].nan_to_num()).all()


@gpu
def test_layer_against_definition(sti):  # noqa: F811
    """Two steps of a layer against the definitions, the rows' bf16 values taken as appended."""
    import torch

    import oracle

    b, h, d, page, window, first, older = 2, 20, 64, 16, 24, 2, 90
    st = layer_state(sti, b, h, d, page, 6, window, first, older)
    g = torch.Generator(device="cuda").manual_seed(9)
    f = frequencies(32)
    old = oracle.kvfp4_decode(st["codes"].cpu().numpy(), st["scales"].cpu().numpy(), d).astype(np.float64)
    start = 0
    for s in (50, 3):
        x = torch.randn(b, s, (h + 1) * d, generator=g, device="cuda").bfloat16()
        o = bf16_out_to_f64(layer_step(sti, st, x))
        q = bf16_out_to_f64(sti.norm_rope(x[..., :h * d].unflatten(-1, (h, d)), st["pos"] - s, st["freqs"]))
        pages, table = bf16_out_to_f64(st["pages"]), st["table"].cpu().numpy()
        sink = st["sink"].cpu().numpy().astype(np.float64)
        for i in range(b):
            for t in range(s):
                p = np.nonzero(seen_by(start + t, window, first))[0]
                rows = np.concatenate([pages[table[i, p // page], p % page], old[i]])
                z = st["scale"] * q[i, t] @ rows.T
                e = np.exp(z)
                pr = e / (e.sum(1) + np.exp(sink))[:, None]
                ref, _ = norm_rotate((pr @ rows)[None], np.array([start + t]), f, d - 32, True, inverse=True, norm=False)
                mass = (pr @ np.abs(rows))
                # bf16 roundings: P of both parts, prev_out, the output and the rotated output, 2^-8 each; the rotation
                # adds two dims' errors
                tol = 5 * 2.0 ** -8 * 2 * mass.max(-1, keepdims=True)
                assert (np.abs(o[i, t] - ref[0]) <= tol).all()
        start += s


@gpu
def test_layer_captured_and_replayed(sti):  # noqa: F811
    """A decode step of the layer captured once and replayed leaves the same pages and outputs as the calls made one by
    one."""
    import torch

    h, d, steps = 64, 512, 9
    xs = torch.randn(steps, 3, 1, (h + 1) * d, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    one = layer_state(sti, 3, h, d, 4, 3, 5, 1, older=200)
    want = [layer_step(sti, one, x) for x in xs]
    two, x = layer_state(sti, 3, h, d, 4, 3, 5, 1, older=200), torch.zeros_like(xs[0])
    pos = two["pos"].clone()
    layer_step(sti, two, x)                                 # (warm: what torch allocates)
    two["pos"].copy_(pos)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer_step(sti, two, x)
    two["pos"].copy_(pos)
    for i in range(steps):
        x.copy_(xs[i])
        graph.replay()
        assert (out == want[i]).all(), i
    assert (one["pages"].nan_to_num() == two["pages"].nan_to_num()).all()


@gpu
def test_two_streams(sti):  # noqa: F811
    """Calls of different sizes on two streams at once, each with its workspace: what each gives alone."""
    import torch

    cases = [make_attend("long_split"), make_attend("packed_padded"), make_attend("chunk_window")]
    want = [attend(sti, a)[:2] for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    dev = [[to_dev(a["q"]), to_dev(a["pool"]), to_dev_any(a["table"]), to_dev_any(a["start"])] for a in cases]
    kws = [dict(window=a["window"], n_first=a["n_first"], attn_sink=opt(a["sink"]), prev_out=opt(a["prev_out"], to_dev),
                prev_lse=opt(a["prev_lse"]), n_new=opt(a["n_new"]),
                ws=sti.workspace(sti.attn_paged_workspace_size(*a["q"].shape)),
                out=torch.full(a["q"].shape, -7.0, dtype=torch.bfloat16, device="cuda"),
                lse=torch.full(a["q"].shape[:3], -7.0, device="cuda")) for a in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, s, t, kw in zip(cases, streams, dev, kws):
            sti.attn_paged(*t, a["scale"], stream=s, **kw)
    torch.cuda.synchronize()
    for (o, l), kw in zip(want, kws):
        assert (kw["out"] == o).all() and (kw["lse"] == l).all()


# ---------------------------------------------------------------------------------- refusals (CPU)


def test_norm_rope_refusals(lib):  # noqa: F811
    n = 4 * 64

    def call(x=P(FAKE), xb=10 * n, xt=n, pos=P(FAKE), each=0, new=None, b=2, s=10, h=4, d=64, norm=1, w=None, eps=1e-6,
             turns=P(FAKE), rd=32, off=32, flags=0, gain=1.0, y=P(FAKE * 64), yb=10 * n, yt=n):
        return lib.sti_norm_rope(x, xb, xt, pos, each, new, b, s, h, d, norm, w, eps, turns, rd, off, flags, gain, y, yb, yt,
                                 None)

    for kw in (dict(x=None), dict(x=P(FAKE + 8)), dict(xb=10 * n + 4), dict(xt=n + 4), dict(pos=None), dict(b=-1), dict(s=0),
               dict(h=0), dict(d=0), dict(turns=None), dict(turns=P(FAKE + 4)), dict(off=40), dict(off=-8), dict(flags=4),
               dict(y=None), dict(y=P(FAKE * 64 + 2)), dict(yt=n - 8), dict(yb=9 * n), dict(w=P(FAKE + 8)),
               dict(w=P(FAKE), norm=0), dict(eps=-1.0), dict(eps=float("nan")),
               dict(y=P(FAKE), yb=20 * n), dict(y=P(FAKE + 16)), dict(y=P(FAKE + 2 * n))):
        assert call(**kw) == 1, kw
    for kw in (dict(d=60, rd=32, off=0), dict(d=1032), dict(rd=20), dict(rd=24, flags=1), dict(off=4), dict(s=0x7FFFFFFF)):
        assert call(**kw) == 2, kw
    assert call(b=0) == 0


def test_append_refusals(lib):  # noqa: F811
    def call(x=P(FAKE), xb=10 * 64, xt=64, pos=P(FAKE), b=2, s=10, d=64, rd=32, off=32, flags=0, pages=P(FAKE * 64),
             stride=16 * 64, n=9, page=16, table=P(FAKE), ts=3, most=3, ws=None):
        return lib.sti_kv_append_paged(x, xb, xt, pos, None, b, s, d, 0, None, 0.0, P(FAKE), rd, off, flags, 1.0, pages, stride, n,
                                       page, table, ts, most, ws, None)

    for kw in (dict(x=None), dict(pages=None), dict(pages=P(FAKE * 64 + 8)), dict(stride=16 * 64 - 8), dict(stride=16 * 64 + 4),
               dict(n=-1), dict(page=0), dict(table=None), dict(ts=2), dict(most=-1), dict(ws=P(FAKE + 8)), dict(flags=2),
               dict(pos=None), dict(pages=P(FAKE)), dict(s=0)):
        assert call(**kw) == 1, kw
    assert call(d=68) == 2 and call(b=0) == 0


def test_attend_refusals(lib):  # noqa: F811
    need = lib.sti_attn_paged_workspace_size(2, 3, 64, 512)
    assert lib.sti_attn_paged_workspace_size(0, 3, 64, 512) == 256 and need <= 4096 + 160 * 8 + 320 * 64 * 8 + 320 * 64 * 2048

    def call(q=P(FAKE), pages=P(FAKE * 512), stride=16 * 512, n=9, page=16, table=P(FAKE), ts=3, most=3, sp=P(FAKE), window=0,
             first=0, po=None, pl=None, b=2, s=3, h=64, d=512, out=P(FAKE * 4), lse=None, ws=P(FAKE * 64), wsb=need):
        return lib.sti_attn_paged(q, pages, stride, n, page, table, ts, most, sp, None, window, first, None, 0.1, po, pl, b, s,
                                  h, d, out, lse, ws, wsb, None)

    for kw in (dict(q=None), dict(q=P(FAKE + 8)), dict(pages=None), dict(pages=P(FAKE * 512 + 8)), dict(stride=16 * 512 - 8),
               dict(n=-1), dict(page=0), dict(table=None), dict(ts=2), dict(most=-1), dict(sp=None), dict(window=-1),
               dict(first=-1), dict(po=P(FAKE * 8)), dict(pl=P(FAKE * 8)), dict(b=-1), dict(s=0), dict(h=0), dict(out=None),
               dict(out=P(FAKE * 4 + 8)), dict(ws=None), dict(ws=P(FAKE * 64 + 8)), dict(wsb=need - 1), dict(out=P(FAKE)),
               dict(out=P(FAKE * 512)), dict(lse=P(FAKE * 8), po=P(FAKE * 9), pl=P(FAKE * 8))):
        assert call(**kw) == 1, kw
    for kw in (dict(h=65), dict(d=96), dict(d=576), dict(s=0x7FFFFFFF), dict(page=1 << 20, stride=512 << 20, most=1025, ts=1025)):
        assert call(**kw) == 2, kw
    assert call(b=0) == 0


@gpu
def test_python_refusals(sti):  # noqa: F811
    import torch

    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    i32 = torch.int32
    x, pos, f = z(2, 3, 4, 64), z(2, t=i32), sti.rope_freqs(32)
    for kw, err in ((dict(x=z(2, 3, 4, 64, t=torch.float16)), TypeError), (dict(x=z(2, 3, 4, 128)[..., ::2]), ValueError),
                    (dict(start_pos=z(3, t=i32)), ValueError), (dict(start_pos=z(2, t=torch.int64)), TypeError),
                    (dict(freqs=f.float()), TypeError), (dict(weight=z(65)), ValueError), (dict(n_new=z(3, t=i32)), ValueError),
                    (dict(out=z(2, 3, 4, 32)), ValueError), (dict(start_pos=pos.cpu()), ValueError), (dict(x=x.cpu()), ValueError),
                    (dict(rope_off=40), sti.StiError), (dict(out=z(1, 3, 4, 64).expand(2, 3, 4, 64)), sti.StiError)):
        with pytest.raises(err):
            sti.norm_rope(**{**dict(x=x, start_pos=pos, freqs=f), **kw})
    rows, pages, table = z(2, 3, 64), z(5, 16, 64), z(2, 4, t=i32)
    for kw, err in ((dict(x=z(2, 3, 128)), ValueError), (dict(pages=z(5, 16, 128)[..., ::2]), ValueError),
                    (dict(pages=z(5, 16, 64, t=torch.float32)), TypeError), (dict(block_table=z(3, 4, t=i32)), ValueError),
                    (dict(block_table=z(2, 4, t=torch.int64)), TypeError), (dict(ws=z(255, t=torch.uint8)), ValueError)):
        with pytest.raises(err):
            sti.kv_append_paged(**{**dict(x=rows, start_pos=pos, pages=pages, block_table=table), **kw})
    q = z(2, 3, 4, 64)
    for kw, err in ((dict(q=z(2, 3, 64)), ValueError), (dict(q=z(2, 3, 4, 128)[..., ::2]), ValueError), (dict(lse=z(2, 3, 4)), TypeError),
                    (dict(prev_out=q.clone()), sti.StiError), (dict(attn_sink=z(5, t=torch.float32)), ValueError),
                    (dict(ws=z(256, t=torch.uint8)), sti.StiError), (dict(out=q), sti.StiError), (dict(window=-1), sti.StiError)):
        with pytest.raises(err):
            sti.attn_paged(**{**dict(q=q, pages=pages, block_table=table, start_pos=pos, softmax_scale=0.1), **kw})
    assert sti.attn_paged(q[:0], pages, table[:0], pos[:0], 0.1).shape == (0, 3, 4, 64)
    torch.cuda.synchronize()
