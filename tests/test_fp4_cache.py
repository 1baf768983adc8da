"""A bounded 4-bit cache (kv_append_fp4, attn_fp4kv, kv_evict) against the fp64 oracle, and its refusals."""
import ctypes

import numpy as np
import pytest

from tests._util import bf16_out_to_f64, to_dev, to_dev_any
from workloads import bf16_bits_to_f32, rng_for, to_bf16_bits

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def sti():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sparse_top_attention_indexer_gb300 as m

    m.lib()
    return m


# ---------------------------------------------------------------------------------- inputs, tolerances


def rows_of(rng, b, rows, d):
    """fp4 rows as quantised normal values with a spread of row scales."""
    import oracle

    x = rng.standard_normal((b, rows, d)) * np.exp2(rng.integers(-2, 2, (b, rows, 1)))
    return oracle.kvfp4_quantize(x) if rows else (np.zeros((b, 0, d // 2), np.uint8), np.zeros((b, 0, d // 16), np.uint8))


def check_attention(got_out, got_lse, ref, q, codes, scales, scale, got_w=None, w0=None):
    """Element by element.  Score error ds: fp32 accumulation of d products, each step of the tensor core off
    by at most an ulp of the running sum, so at most (d / 16 + 2) 2^-23 of sum |q k| (times the scale).
    A probability is off by 2 ds (its own and the sum's) and, for the PV product, by f16 rounding (2^-11, or
    2^-25 absolute below f16's normal range, in units where the sum is at least 1); the output by bf16 rounding."""
    import oracle

    out, lse, weights, mass = ref
    d = q.shape[-1]
    n = codes.shape[1]
    kv = oracle.kvfp4_decode(codes, scales, d)
    kv = np.where(np.isnan(kv), 0.0, kv)
    sabs = 0.0
    for i in range(len(q)):
        if n:
            sabs = max(sabs, abs(scale) * float((np.abs(np.nan_to_num(q[i], posinf=0, neginf=0)).reshape(-1, d) @
                                                 np.abs(kv[i]).T).max()))
    ds = (d / 16 + 2) * 2.0 ** -23 * sabs
    fin = np.isfinite(out)
    assert np.array_equal(np.isnan(got_out), np.isnan(out))
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2 * ds + 2.0 ** -19) * mass + n * 2.0 ** -25 * np.abs(kv).max(initial=0)
    err = np.abs(got_out - out)
    assert (err[fin] <= tol[fin]).all(), f"out: {np.nanmax((err - tol)[fin]):.3g} over, worst {err[fin].max():.3g}"
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(lse)) and np.array_equal(np.isnan(got_lse), np.isnan(lse))
    f = np.isfinite(lse)
    lerr = np.abs(got_lse[f] - lse[f])
    assert (lerr <= ds + 2.0 ** -19 + 2.0 ** -21 * np.abs(lse[f])).all(), f"lse: {lerr.max():.3g}"
    if got_w is not None:
        # w0: what the weights held before (fp32)
        rel = 2 * ds + 2.0 ** -19 * (1 + np.abs(lse[f]).max(initial=0)) + 64 * q.shape[1] * 2.0 ** -24
        werr = np.abs(got_w - (w0 + weights))
        ok = werr <= rel * weights + 2.0 ** -23 * np.abs(w0 + weights)
        assert ok[np.isfinite(weights)].all(), f"row weights: {np.nanmax(werr):.3g}"


ATTEND = {
    # name: b, s, h, d, rows, start_pos, ratio, dropped, sink, prev, weights
    "one_row": (1, 1, 64, 512, 1, [0], 1, None, True, False, True),
    "one_tile_less": (2, 1, 64, 512, 127, [126, 60], 1, None, True, False, True),
    "one_tile": (2, 1, 64, 512, 128, [127, 3], 1, None, False, False, True),
    "one_tile_more": (2, 1, 64, 512, 129, [128, 127], 1, None, False, True, True),
    "ragged_empty": (5, 1, 64, 512, 700, [2799, 2, 0, 1500, 4], 4, None, True, False, True),
    "ragged_empty_prev": (5, 1, 64, 512, 700, [2799, 2, 0, 1500, 4], 4, None, True, True, True),
    "long_split": (1, 1, 64, 512, 5000, [4998], 1, None, True, True, True),
    "many_sequences": (200, 1, 64, 128, 300, None, 1, None, True, False, True),
    "few_heads": (3, 2, 5, 192, 900, [900, 333, 1], 1, None, True, True, True),
    "one_head": (2, 3, 1, 64, 260, [500, 30], 2, None, False, False, True),
    "heads_33": (2, 1, 33, 320, 400, [399, 256], 1, None, True, False, True),
    "heads_32_d448": (2, 2, 32, 448, 385, [383, 100], 1, None, True, True, True),
    "dropped": (3, 4, 64, 256, 513, [3000, 2100, 90], 4, [300, 12, 30], True, True, True),
    "causal_from_0": (2, 300, 16, 128, 300, [0, 0], 1, None, True, False, True),
    "causal_ratio_4": (1, 301, 64, 512, 76, [0], 4, None, True, True, True),
    "chunk": (2, 40, 64, 512, 400, [1200, 700], 4, None, True, True, True),
    "no_rows": (2, 3, 8, 64, 0, [5, 9], 1, None, True, True, False),
    "nothing_at_all": (2, 2, 8, 64, 0, [5, 9], 1, None, True, False, False),
    # several queries of many tiles per SM, with rows that are split between SMs
    "long_queries": (1, 400, 64, 512, 1500, [5600], 4, None, True, True, False),
    # few heads, several queries: groups of queries share their tiles
    "packed_partial_mixed": (2, 7, 20, 512, 300, [30, 2], 4, None, True, True, True),
    "packed_mixed_no_prev": (3, 9, 8, 128, 90, [0, 2, 500], 4, [0, 0, 130], True, False, True),
    "packed_split": (1, 5, 12, 256, 5000, [4990], 1, None, True, True, True),
    "packed_split_pairs": (1, 9, 32, 320, 700, [690], 1, None, False, False, True),
    "packed_kept_scores": (2, 70, 5, 64, 200, [100, 3], 2, None, True, False, True),
    "packed_two_passes": (2, 200, 3, 192, 700, [400, 0], 1, None, True, True, True),
    "packed_one_head": (3, 300, 1, 64, 4, [0, 5, 1], 4, None, True, True, True),
}


def make_attend(name):
    b, s, h, d, rows, sp, ratio, dropped, sink, prev, weights = ATTEND[name]
    rng = rng_for(9100 + len(name), d + h)
    codes, scales = rows_of(rng, b, rows, d)
    a = dict(q=to_bf16_bits(2 * rng.standard_normal((b, s, h, d))), codes=codes, scales=scales,
             start_pos=np.array(sp if sp is not None else rng.integers(0, rows, b), np.int32), ratio=ratio,
             scale=d ** -0.5, sink=rng.standard_normal(h).astype(np.float32) if sink else None,
             dropped=None if dropped is None else np.array(dropped, np.int32))
    a["prev_out"] = to_bf16_bits(rng.standard_normal((b, s, h, d))) if prev else None
    a["prev_lse"] = (4 + rng.standard_normal((b, s, h))).astype(np.float32) if prev else None
    if prev and h > 1:
        a["prev_lse"][0, 0, :2] = -np.inf      # heads for which the other rows held nothing
    a["w0"] = rng.random((b, rows)).astype(np.float32) if weights else None
    return a


def reference(orc, a):
    f = bf16_bits_to_f32
    return orc.attn_fp4kv(f(a["q"]), a["codes"], a["scales"], a["start_pos"], a["ratio"], a["scale"], a["sink"],
                          a["dropped"], None if a["prev_out"] is None else f(a["prev_out"]), a["prev_lse"])


def attend(sti, a, **kw):
    import torch

    opt = lambda v: None if v is None else to_dev_any(v)  # noqa: E731
    q = to_dev(a["q"])
    lse = torch.full(q.shape[:3], 77.0, device="cuda")
    w = opt(a["w0"])
    ws = kw.pop("ws", None)
    if ws is None:
        ws = sti.workspace(sti.attn_fp4kv_workspace_size(*q.shape, a["codes"].shape[1]))
    out = sti.attn_fp4kv(q, kw.pop("codes", None) if "codes" in kw else to_dev_any(a["codes"]),
                         kw.pop("scales", None) if "scales" in kw else to_dev_any(a["scales"]),
                         to_dev_any(a["start_pos"]), a["ratio"], a["scale"], attn_sink=opt(a["sink"]),
                         dropped=opt(a["dropped"]), prev_out=None if a["prev_out"] is None else to_dev(a["prev_out"]),
                         prev_lse=opt(a["prev_lse"]), lse=lse, row_weight=w, ws=ws, **kw)
    assert sti.read_device_status(ws) == 0
    return out, lse, w


# ---------------------------------------------------------------------------------- attention


@gpu
@pytest.mark.parametrize("name", list(ATTEND))
def test_attend(sti, orc, name):
    a = make_attend(name)
    out, lse, w = attend(sti, a)
    check_attention(bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), reference(orc, a),
                    bf16_bits_to_f32(a["q"]), a["codes"], a["scales"], a["scale"],
                    None if w is None else w.cpu().numpy().astype(np.float64), a["w0"])


@gpu
def test_attend_scores_that_climb(sti, orc):
    """Later rows score far above earlier ones, tile after tile: the running maximum moves every time; a
    second head sees the opposite order, a third all scores equal."""
    rng = rng_for(9200, 1)
    b, s, h, d, rows = 1, 1, 3, 128, 1000
    a = dict(make_attend("one_head"), q=np.zeros((b, s, h, d), np.uint16))
    x = np.zeros((b, rows, d))
    x[..., 16:] = rng.standard_normal((b, rows, d - 16))
    x[..., 0] = np.linspace(0, 600, rows)       # its own groups of 16: elements 0..15
    import oracle

    a["codes"], a["scales"] = oracle.kvfp4_quantize(x)
    q = 0.1 * rng.standard_normal((b, s, h, d))
    q[..., :16] = 0
    q[0, 0, 0, 0], q[0, 0, 1, 0], q[0, 0, 2] = 6.0, -6.0, 0.0
    a.update(q=to_bf16_bits(q), start_pos=np.array([rows - 1], np.int32), ratio=1, scale=1.0, sink=None, prev_out=None,
             prev_lse=None, dropped=None, w0=np.zeros((b, rows), np.float32))
    out, lse, w = attend(sti, a)
    check_attention(bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), reference(orc, a),
                    bf16_bits_to_f32(a["q"]), a["codes"], a["scales"], 1.0, w.cpu().numpy().astype(np.float64), a["w0"])


@gpu
@pytest.mark.parametrize("s", [1, 3])
def test_attend_garbage_past_the_visible_rows(sti, orc, s):
    """NaN scales and wild codes in rows nobody sees, in the last visible tile and behind it, change nothing."""
    a = make_attend("dropped")
    a["q"] = np.ascontiguousarray(a["q"][:, :s])
    a["prev_out"], a["prev_lse"] = np.ascontiguousarray(a["prev_out"][:, :s]), np.ascontiguousarray(a["prev_lse"][:, :s])
    clean = [x.clone() for x in attend(sti, a)]
    vis = (a["start_pos"].astype(np.int64) + s) // a["ratio"] - a["dropped"]
    for i, v in enumerate(np.clip(vis, 0, a["codes"].shape[1])):
        a["codes"][i, v:], a["scales"][i, v:] = 0xFF, 0x7F
    # the rows that only the last query sees: NaN for it, nothing for the earlier ones
    out, lse, w = attend(sti, a)
    for x, y in zip(clean, (out, lse, w)):
        assert (x == y).all()


@gpu
def test_attend_nan_row_reaches_only_its_viewers(sti):
    """A NaN row makes the queries that see it NaN and leaves the earlier queries of the step alone."""
    import torch

    a = make_attend("chunk")
    clean, _, _ = attend(sti, dict(a))
    vis = (a["start_pos"].astype(np.int64)[:, None] + np.arange(40) + 1) // 4
    a["scales"][0, vis[0, 20] - 1] = 0x7F
    out, lse, w = attend(sti, a)
    sees = torch.tensor(vis[0] >= vis[0, 20], device="cuda")
    assert sees.any() and not sees.all()
    assert torch.isnan(out[0, sees]).all() and torch.isnan(lse[0, sees]).all()
    assert (out[0, ~sees] == clean[0, ~sees]).all() and (out[1] == clean[1]).all()
    assert not torch.isnan(w[1]).any()


@gpu
@pytest.mark.parametrize("name, t", [("packed_split", 1), ("packed_split", 3), ("packed_two_passes", 100),
                                     ("packed_kept_scores", 31), ("packed_partial_mixed", 5)])
def test_attend_nan_row_in_a_group_of_queries(sti, name, t):
    """Queries that share a tile: a NaN row is NaN for those that see it only, in the weights too."""
    import torch

    a = make_attend(name)
    b, s, ratio = *a["q"].shape[:2], a["ratio"]
    vis = (a["start_pos"].astype(np.int64)[:, None] + np.arange(s) + 1) // ratio
    clean, _, _ = attend(sti, dict(a))
    bad = vis[0, t] - 1
    a["scales"][0, bad, 0] |= 0x7F
    out, lse, w = attend(sti, a)
    sees = torch.tensor(vis[0] > bad, device="cuda")
    assert sees.any() and not sees.all()
    assert torch.isnan(out[0, sees]).all() and torch.isnan(lse[0, sees]).all()
    assert (out[0, ~sees] == clean[0, ~sees]).all() and not torch.isnan(lse[0, ~sees]).any()
    seen = torch.arange(w.shape[1], device="cuda") < int(vis[0].max())
    assert (torch.isnan(w[0]) == seen).all()
    if b > 1:
        assert (out[1:] == clean[1:]).all() and not torch.isnan(w[1:]).any()


@gpu
@pytest.mark.parametrize("s, h", [(5, 12), (1, 64)])
def test_attend_scores_far_below_zero(sti, s, h):
    """Every row is all ones and every score -256 (e^256 is infinite in fp32): the average of a split query is the
    row, also for heads that see nothing of a part."""
    import torch

    d, rows = 256, 5000
    q = torch.full((1, s, h, d), -1.0, device="cuda", dtype=torch.bfloat16)
    codes = torch.full((1, rows, d // 2), 0x22, device="cuda", dtype=torch.uint8)
    scales = torch.full((1, rows, d // 16), 0x38, device="cuda", dtype=torch.uint8)
    lse = torch.empty(1, s, h, device="cuda")
    w = torch.zeros(1, rows, device="cuda")
    start = torch.tensor([4990], device="cuda", dtype=torch.int32)
    out = sti.attn_fp4kv(q, codes, scales, start, 1, 1.0, lse=lse, row_weight=w)
    assert (out == 1).all()
    n = 4991.0 + np.arange(s)
    # lse: fp32 sums and logarithms next to 256, in units of 2^-16
    np.testing.assert_allclose(lse.cpu().numpy()[0], np.repeat((np.log(n) - 256)[:, None], h, 1), atol=2.0 ** -13)
    # e^(s - lse): the error of lse and of s in log2 units (2^-15), one 2^x
    want = h * (np.arange(rows)[None] < n[:, None]).astype(float).T @ (1 / n)
    np.testing.assert_allclose(w.cpu().numpy()[0], want, rtol=2.0 ** -12)


@gpu
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_attend_bad_query_head(sti, bad):
    """A head whose query holds an infinity or NaN gets NaN; the other heads and queries are untouched."""
    import torch

    a = make_attend("few_heads")
    clean, _, _ = attend(sti, dict(a))
    q = bf16_bits_to_f32(a["q"]).copy()
    q[1, 0, 2, 7] = bad
    a["q"] = to_dev_bits(q)
    out, _, _ = attend(sti, a)
    hit = torch.zeros(out.shape[:3], dtype=torch.bool, device="cuda")
    hit[1, 0, 2] = True
    assert torch.isnan(out[hit]).all() and (out[~hit] == clean[~hit]).all()


def to_dev_bits(f32):
    """fp32 (any value) -> bf16 bits by truncation (exact for values that are bf16 already)."""
    return (np.ascontiguousarray(f32, np.float32).view(np.uint32) >> np.uint32(16)).astype(np.uint16)


@gpu
@pytest.mark.parametrize("power", [-130, -100, 100])
def test_attend_query_magnitudes(sti, orc, power):
    """Queries far from 1 (subnormal bf16 included) with a scale that brings the scores back."""
    a = make_attend("few_heads")
    q = (bf16_bits_to_f32(a["q"]).astype(np.float64) * 2.0 ** power).astype(np.float32)
    a["q"] = to_dev_bits(q)                     # below 2^-126: what bf16 keeps of it
    a["scale"] = float(a["scale"] * 2.0 ** -power) if power > -127 else float(a["scale"] * 2.0 ** 126)
    out, lse, w = attend(sti, a)
    check_attention(bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), reference(orc, a),
                    bf16_bits_to_f32(a["q"]), a["codes"], a["scales"], a["scale"], w.cpu().numpy().astype(np.float64), a["w0"])


@gpu
def test_attend_every_code_and_scale(sti, orc):
    """Rows that hold every code with every finite scale byte, negative ones included: the output over one
    visible row is that row."""
    import oracle

    d, rows = 512, 254
    byte = np.array([v for v in range(256) if v & 0x7F != 0x7F], np.uint8)
    scales = np.repeat(byte[:, None], d // 16, axis=1)[None]
    codes = np.tile(np.array([((2 * i + 1) % 16) << 4 | (2 * i) % 16 for i in range(8)], np.uint8), d // 16)
    codes = np.broadcast_to(codes, (1, rows, d // 2)).copy()
    want = oracle.kvfp4_decode(codes, scales, d)
    for j in (0, 1, 7, 8, 100, 126, 127, 128, 200, 253):
        a = dict(make_attend("one_row"), codes=codes[:, j:j + 1], scales=scales[:, j:j + 1], sink=None)
        a["w0"] = np.zeros((1, 1), np.float32)
        out, _, w = attend(sti, a)
        np.testing.assert_array_equal(bf16_out_to_f64(out)[0, 0], np.broadcast_to(want[0, j], (64, d)))
        np.testing.assert_allclose(w.cpu().numpy(), 64, rtol=2.0 ** -17)


@gpu
def test_attend_strided_cache_in_place_out_and_streams(sti, orc):
    """A slice of a larger cache (batch stride, rows behind), out = prev_out, another stream, a workspace that
    other sizes have used, and no optional outputs: the same result."""
    import torch

    a = make_attend("dropped")
    want, want_lse, want_w = attend(sti, a)
    b, rows, d2 = a["codes"].shape
    codes = torch.full((b, rows + 37, d2), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((b, rows + 37, d2 // 8), 127, dtype=torch.uint8, device="cuda")
    codes[:, :rows], scales[:, :rows] = to_dev_any(a["codes"]), to_dev_any(a["scales"])
    codes, scales = codes[:, :rows], scales[:, :rows]
    ws = sti.workspace(max(sti.attn_fp4kv_workspace_size(b, 4, 64, 256, rows),
                           sti.attn_fp4kv_workspace_size(1, 1, 64, 512, 5000)))
    attend(sti, make_attend("long_split"), ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    prev = to_dev(a["prev_out"])
    lse = torch.empty(prev.shape[:3], device="cuda")
    w = to_dev_any(a["w0"])
    args = (to_dev(a["q"]), codes, scales, to_dev_any(a["start_pos"]), a["ratio"], a["scale"])
    kw = dict(attn_sink=to_dev_any(a["sink"]), dropped=to_dev_any(a["dropped"]), prev_lse=to_dev_any(a["prev_lse"]))
    torch.cuda.synchronize()
    out = sti.attn_fp4kv(*args, prev_out=prev, out=prev, lse=lse, row_weight=w, ws=ws, stream=s, **kw)
    s.synchronize()
    assert out is prev and (out == want).all() and (lse == want_lse).all() and (w == want_w).all()
    out = sti.attn_fp4kv(*args, prev_out=to_dev(a["prev_out"]), stream=s.cuda_stream, **kw)
    w = to_dev_any(a["w0"])
    out2 = sti.attn_fp4kv(*args, prev_out=to_dev(a["prev_out"]), row_weight=w, **kw)
    torch.cuda.synchronize()
    assert (out == want).all() and (out2 == want).all() and (w == want_w).all()


@gpu
def test_attend_repeats_and_graph(sti):
    """The same call gives the same bits again, and from a captured graph replayed on new inputs."""
    import torch

    a = make_attend("long_split")
    want = attend(sti, a)
    for _ in range(3):
        for x, y in zip(want, attend(sti, a)):
            assert (x == y).all()
    q, codes, scales = torch.zeros_like(to_dev(a["q"])), to_dev_any(a["codes"]), to_dev_any(a["scales"])
    sp, lse, w = to_dev_any(a["start_pos"]) * 0, torch.zeros(1, 1, 64, device="cuda"), to_dev_any(a["w0"])
    kw = dict(attn_sink=to_dev_any(a["sink"]), prev_out=to_dev(a["prev_out"]), prev_lse=to_dev_any(a["prev_lse"]))
    ws = sti.workspace(sti.attn_fp4kv_workspace_size(1, 1, 64, 512, codes.shape[1]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sti.attn_fp4kv(q, codes, scales, sp, 1, a["scale"], lse=lse, row_weight=w, ws=ws, **kw)
    q.copy_(to_dev(a["q"]))
    sp.copy_(to_dev_any(a["start_pos"]))
    w.copy_(to_dev_any(a["w0"]))
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(want, (out, lse, w)):
        assert (x == y).all()


@gpu
def test_attend_two_streams_and_graphs_that_share_a_workspace(sti):
    """Two streams, each with its workspace, at the same time; then two graphs with one workspace, in turn."""
    import torch

    names = ("long_split", "packed_two_passes")
    cases = [make_attend(n) for n in names]
    want = [[x.clone() for x in attend(sti, a)] for a in cases]

    def call(a, ws, lse, w):
        return lambda: sti.attn_fp4kv(to_dev_q[id(a)], *dev[id(a)], a["ratio"], a["scale"], lse=lse, row_weight=w, ws=ws, **kws[id(a)])

    to_dev_q = {id(a): to_dev(a["q"]) for a in cases}
    dev = {id(a): (to_dev_any(a["codes"]), to_dev_any(a["scales"]), to_dev_any(a["start_pos"])) for a in cases}
    kws = {id(a): dict(attn_sink=to_dev_any(a["sink"]), prev_out=to_dev(a["prev_out"]), prev_lse=to_dev_any(a["prev_lse"]))
           for a in cases}
    sizes = [sti.attn_fp4kv_workspace_size(*a["q"].shape, a["codes"].shape[1]) for a in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    own = [sti.workspace(n) for n in sizes]
    shared = sti.workspace(max(sizes))
    lses = [torch.empty(a["q"].shape[:3], device="cuda") for a in cases]
    ws_ = [to_dev_any(a["w0"]) for a in cases]
    torch.cuda.synchronize()
    outs = [None, None]
    for rep in range(8):
        for w, a in zip(ws_, cases):
            w.copy_(to_dev_any(a["w0"]))
        torch.cuda.synchronize()
        for i, a in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i] = call(a, own[i], lses[i], ws_[i])()
        torch.cuda.synchronize()
        for i in range(2):
            for x, y in zip(want[i], (outs[i], lses[i], ws_[i])):
                assert (x == y).all()
    graphs = []
    for i, a in enumerate(cases):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs[i] = call(a, shared, lses[i], ws_[i])()
        graphs.append(g)
    for rep in range(4):
        for i, a in enumerate(cases):
            ws_[i].copy_(to_dev_any(a["w0"]))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for x, y in zip(want[i], (outs[i], lses[i], ws_[i])):
                assert (x == y).all()


@gpu
@pytest.mark.parametrize("budget", [100, 9000])
def test_steps_captured_and_replayed(sti, budget):
    """A decode step of a full cache (append, attend with row weights in a slice, evict) captured once and replayed
    leaves the same cache, bit for bit, as the calls made one by one."""
    import torch

    b, h, d, steps = 2, 24, 128, 12
    gen = torch.Generator(device="cuda").manual_seed(7)
    rows = budget + 2
    xs = torch.randn(steps, b, 1, d, generator=gen, device="cuda").bfloat16()
    qs = torch.randn(steps, b, 1, h, d, generator=gen, device="cuda").bfloat16()

    def fresh():
        g = torch.Generator(device="cuda").manual_seed(8)
        return dict(codes=torch.randint(0, 256, (b, rows, d // 2), generator=g, device="cuda", dtype=torch.uint8),
                    scales=torch.randint(40, 60, (b, rows, d // 16), generator=g, device="cuda", dtype=torch.uint8),
                    pos=torch.arange(rows, device="cuda", dtype=torch.int32).repeat(b, 1),
                    weight=torch.rand(b, rows + 6, generator=g, device="cuda")[:, :rows],
                    start=torch.tensor([budget, budget - 5], device="cuda", dtype=torch.int32),
                    dropped=torch.zeros(b, device="cuda", dtype=torch.int32))

    def step(c, x, q):
        sti.kv_append_fp4(x, c["start"], 1, 1, c["codes"], c["scales"], dropped=c["dropped"], row_pos=c["pos"],
                          row_weight=c["weight"])
        out = sti.attn_fp4kv(q, c["codes"], c["scales"], c["start"], 1, d ** -0.5, dropped=c["dropped"], row_weight=c["weight"])
        sti.kv_evict(c["weight"], c["pos"], c["start"], 1, 1, c["dropped"], budget, 4, 8, [c["codes"], c["scales"]])
        c["start"] += 1
        return out

    one, two = fresh(), fresh()
    want = [step(one, xs[i], qs[i]) for i in range(steps)]
    x, q = torch.zeros_like(xs[0]), torch.zeros_like(qs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(two, x, q)
    for i in range(steps):
        x.copy_(xs[i])
        q.copy_(qs[i])
        g.replay()
        assert (out == want[i]).all()
    for k in one:
        assert (one[k] == two[k]).all(), k
    assert one["dropped"].tolist() == [steps, steps - 5]


@gpu
def test_attend_matches_sparse_attention(sti):
    """Listing every visible row in sti_sparse_attn_sink_fp4kv gives the same attention (both round P: 2^-8 for
    its bf16, 2^-11 here, and the output 2^-8 each; |rows| <= 6 here and the weights add up to at most 1)."""
    import torch

    a = make_attend("ragged_empty")
    out, lse, _ = attend(sti, a)
    vis = (a["start_pos"] + 1) // 4
    idx = np.stack([np.where(np.arange(700) < v, np.arange(700), -1) for v in vis])
    idx = idx.astype(np.int32).reshape(5, 1, 700)
    q = to_dev(a["q"])
    lse2 = torch.empty(q.shape[:3], device="cuda")
    out2 = sti.sparse_attn_sink_fp4kv(q, torch.zeros(5, 0, 512, dtype=torch.bfloat16, device="cuda"),
                                      to_dev_any(a["codes"]), to_dev_any(a["scales"]), to_dev_any(a["sink"]),
                                      to_dev_any(idx), a["scale"], lse=lse2)
    top = float(out.abs().max())
    assert float((out.float() - out2.float()).abs().max()) <= (2.0 ** -8 + 2.0 ** -11) * 6 + 2 * 2.0 ** -8 * top
    fin = torch.isfinite(lse)
    assert (torch.isfinite(lse2) == fin).all() and float((lse - lse2)[fin].abs().max()) < 1e-3


# ---------------------------------------------------------------------------------- append


def special_rows(rng, shape):
    """Normal rows with groups of zeros, ties between codes, NaN, infinities, subnormal and huge values."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-20, 20, shape[:-1] + (1,)))
    f = x.reshape(-1, 64)
    if len(f) > 8:
        f[0, :32] = 0
        f[1, :16] = [6, .25, -.25, .75, -.75, 1.25, 1.75, -1.75, 2.5, 3.5, 5, -5, -6, 0, .5, 4]   # scale 1
        f[2, :32] *= 2.0 ** -130 / np.abs(f[2, :32]).max()
        f[3] = 3.0e38 * np.sign(f[3])
        f[4, :16] *= 2.0 ** -12 / np.abs(f[4, :16]).max()         # below E4M3's smallest scale
        f[5, 3], f[5, 40] = np.nan, np.inf
        f[6, 20], f[6, 63] = -np.inf, np.nan
        f[7, :16] = 6 * 2.0 ** -10                               # max / 6 halfway between scale 0 and 2^-9
    with np.errstate(over="ignore"):
        bits = to_bf16_bits(np.where(np.isnan(x), 0, x))
    return np.where(np.isnan(x), np.uint16(0x7FC0), bits)


@gpu
@pytest.mark.parametrize("fmt", ["e4m3", "e8m0"])
@pytest.mark.parametrize("b,s,ratio,dim,rows,sps,dropped", [
    (1, 1, 1, 64, 1, [0], None),
    (4, 1, 4, 512, 50, [3, 4, 7, 198], None),               # a decode step: only some complete a group
    (3, 37, 4, 512, 400, [0, 1001, 1502], [0, 250, 3]),
    (2, 700, 1, 192, 900, [5, 200], None),
    (3, 130, 2, 128, 64, [0, 200, 40], [0, 90, 20]),        # rows outside the cache are flagged and skipped
])
def test_append(sti, orc, fmt, b, s, ratio, dim, rows, sps, dropped):
    import torch

    rng = rng_for(9300 + s, dim)
    m = -(-s // ratio)
    bits = special_rows(rng, (b, m, dim))
    group = 16 if fmt == "e4m3" else 32
    codes, scales = rng.integers(0, 256, (b, rows, dim // 2), np.uint8), rng.integers(0, 256, (b, rows, dim // group), np.uint8)
    pos, weight = np.full((b, rows), -5, np.int32), np.full((b, rows), 3.0, np.float32)
    drop = np.zeros(b, np.int32) if dropped is None else np.array(dropped, np.int32)
    pad = rows + 3      # a larger cache, of which the test uses the first rows
    dev = {}
    for k, v in (("codes", codes), ("scales", scales)):
        full = torch.full((b, pad, v.shape[2]), 0xAB, dtype=torch.uint8, device="cuda")
        full[:, :rows] = to_dev_any(v)
        dev[k], dev[k + "_full"] = full[:, :rows], full
    dpos, dweight = to_dev_any(pos), to_dev_any(weight)
    ws = sti.workspace(256)
    sti.kv_append_fp4(to_dev(bits), to_dev_any(np.array(sps, np.int32)), s, ratio, dev["codes"], dev["scales"],
                      dropped=None if dropped is None else to_dev_any(drop), row_pos=dpos, row_weight=dweight, ws=ws)
    with np.errstate(invalid="ignore", over="ignore"):
        outside = orc.kv_append_fp4(bf16_bits_to_f32(bits).astype(np.float64), sps, drop, s, ratio, fmt, codes, scales, pos, weight)
    assert (sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE) == outside
    np.testing.assert_array_equal(dev["scales"].cpu().numpy(), scales)
    np.testing.assert_array_equal(dev["codes"].cpu().numpy(), codes)
    np.testing.assert_array_equal(dpos.cpu().numpy(), pos)
    np.testing.assert_array_equal(dweight.cpu().numpy(), weight)
    assert (dev["codes_full"][:, rows:] == 0xAB).all() and (dev["scales_full"][:, rows:] == 0xAB).all()


@gpu
def test_append_every_bf16(sti, orc):
    """Every finite bf16 value, beside each of several group maxima."""
    v = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    v = v[(v & 0x7F80) != 0x7F80]
    for fmt, group in (("e4m3", 16), ("e8m0", 32)):
        x = np.zeros((len(v) // (group - 1) + 1, group), np.uint16)
        x[:, 1:].reshape(-1)[:] = 0
        flat = np.resize(v, x[:, 1:].size)
        x[:, 1:] = flat.reshape(x[:, 1:].shape)
        top = np.resize(to_bf16_bits(np.array([0.1, 1, 2.9, 6, 55, 2000, 2.0 ** -9, 448 * 6, 1e30])), len(x))
        # a group's maximum is the larger of `top` and its own values: sort the values so that both occur
        x[:, 0] = top
        n = len(x) * group // 512
        bits = x.reshape(-1)[:n * 512].reshape(1, n, 512)
        import torch

        codes = torch.zeros(1, n, 256, dtype=torch.uint8, device="cuda")
        scales = torch.zeros(1, n, 512 // group, dtype=torch.uint8, device="cuda")
        sti.kv_append_fp4(to_dev(bits), torch.zeros(1, dtype=torch.int32, device="cuda"), n, 1, codes, scales)
        want_c, want_s = orc.fp4_rows(bf16_bits_to_f32(bits), fmt)
        np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
        np.testing.assert_array_equal(codes.cpu().numpy(), want_c)


# ---------------------------------------------------------------------------------- evict


def make_evict(rng, b, rows, held, weights="random"):
    w = rng.exponential(size=(b, rows)).astype(np.float32)
    if weights == "ties":
        w = rng.integers(0, 3, (b, rows)).astype(np.float32)
    elif weights == "equal":
        w[:] = 0.5
    elif weights == "special":
        w[rng.random((b, rows)) < 0.1] = np.nan
        w[rng.random((b, rows)) < 0.1] = np.inf
        w[rng.random((b, rows)) < 0.2] = 0.0
        w[rng.random((b, rows)) < 0.2] = -0.0
        w[rng.random((b, rows)) < 0.1] = -1.0
        w[rng.random((b, rows)) < 0.05] = -np.inf
    return w


EVICT = [
    # b, rows, budget, n_first, n_recent, held per sequence, seqlen, ratio, weights
    (1, 2, 1, 0, 0, [2], 1, 1, "random"),
    (3, 40, 30, 4, 8, [40, 30, 31], 10, 1, "random"),
    (4, 300, 100, 4, 32, [300, 100, 0, 199], 8, 4, "ties"),
    (2, 5000, 4000, 0, 0, [5000, 4500], 100, 1, "equal"),
    (2, 5000, 40, 10, 30, [5000, 41], 100, 1, "random"),
    (2, 8200, 8191, 4, 128, [8200, 8192], 3, 1, "special"),
    (3, 20001, 12345, 4, 128, [20001, 12346, 17000], 2002, 2, "ties"),
    (2, 70000, 65000, 4, 128, [70000, 66001], 50, 1, "special"),
    (2, 100, 0, 0, 0, [100, 7], 5, 1, "random"),
    (1, 400000, 399000, 4, 128, [399990], 50, 1, "ties"),
    # many sequences: clusters of 4, of 2, single CTAs
    (17, 20000, 19000, 4, 64, [20000 - 60 * i for i in range(17)], 5, 1, "special"),
    (40, 20000, 19900, 4, 64, [20000 - i for i in range(40)], 5, 1, "ties"),
    (150, 9000, 8990, 4, 64, [9000 - i % 12 for i in range(150)], 5, 1, "random"),
]


@gpu
@pytest.mark.parametrize("case", range(len(EVICT)))
def test_evict(sti, orc, case):
    b, rows, budget, first, recent, held, s, ratio, kind = EVICT[case]
    rng = rng_for(9400, case)
    dropped = rng.integers(0, 50, b).astype(np.int32)
    sp = np.array([max(0, (v + g) * ratio + int(rng.integers(0, ratio)) - s) for v, g in zip(held, dropped)], np.int32)
    w = make_evict(rng, b, rows, held, kind)
    pos = np.stack([rng.permutation(rows) + g for g in dropped]).astype(np.int32)
    # arrays of several row sizes and alignments
    arrays = [rng.integers(0, 256, (b, rows, 96), np.uint8), rng.integers(0, 256, (b, rows, 7), np.uint8),
              rng.integers(0, 1 << 16, (b, rows, 5), np.uint16).view(np.int16), rng.random((b, rows), np.float32)]
    dev = [to_dev_any(v) for v in (w, pos, dropped, *arrays)]
    sti.kv_evict(dev[0], dev[1], to_dev_any(sp), s, ratio, dev[2], budget, first, recent, dev[3:])
    orc.kv_evict(w, pos, sp, s, ratio, dropped, budget, first, recent, arrays)
    for x, y in zip(dev, (w, pos, dropped, *arrays)):
        np.testing.assert_array_equal(x.cpu().numpy(), y)


@gpu
def test_evict_protected_rows_beyond_the_budget(sti, orc):
    """Positions that contradict the step (every row claims to be recent): the lowest rows fill the budget."""
    rng = rng_for(9500, 0)
    w, pos = rng.random((1, 500)).astype(np.float32), np.full((1, 500), 100000, np.int32)
    sp, dropped = np.array([499], np.int32), np.zeros(1, np.int32)
    dev = [to_dev_any(v) for v in (w, pos, dropped)]
    sti.kv_evict(dev[0], dev[1], to_dev_any(sp), 1, 1, dev[2], 100, 0, 100)
    orc.kv_evict(w, pos, sp, 1, 1, dropped, 100, 0, 100)
    for x, y in zip(dev, (w, pos, dropped)):
        np.testing.assert_array_equal(x.cpu().numpy(), y)


# ---------------------------------------------------------------------------------- together


@gpu
def test_bounded_cache_steps(sti, orc):
    """A layer's steps over a cache of 160 rows: a prompt, then single tokens; every step appends the
    completed rows, attends over a window (sparse attention) joined with the whole cache, and evicts.  The oracle
    follows with its own state; the rows that stay have to be the same throughout."""
    import torch

    rng = rng_for(9600, 0)
    b, h, d, ratio, W, budget, first, recent = 3, 16, 128, 2, 16, 160, 4, 16
    prompt, n_steps = 390, 14
    rows = budget + prompt // ratio + 1
    codes, scales = np.zeros((b, rows, d // 2), np.uint8), np.zeros((b, rows, d // 16), np.uint8)
    pos, weight, dropped = np.zeros((b, rows), np.int32), np.zeros((b, rows), np.float32), np.zeros(b, np.int32)
    dcodes = torch.zeros(b, rows, d // 2, dtype=torch.uint8, device="cuda")
    dscales = torch.zeros(b, rows, d // 16, dtype=torch.uint8, device="cuda")
    dpos, dweight, ddrop = to_dev_any(pos), to_dev_any(weight), to_dev_any(dropped)
    sink = rng.standard_normal(h).astype(np.float32)
    scale = d ** -0.5
    start = np.array([0, 0, 0], np.int32)
    for step in range(n_steps):
        s = prompt if step == 0 else (1 if step % 5 else 3)
        m = -(-s // ratio)
        x = to_bf16_bits(rng.standard_normal((b, m, d)))
        q = to_bf16_bits(3 * rng.standard_normal((b, s, h, d)))
        win = to_bf16_bits(rng.standard_normal((b, W, d)))
        dsp, dq = to_dev_any(start), to_dev(q)
        sti.kv_append_fp4(to_dev(x), dsp, s, ratio, dcodes, dscales, dropped=ddrop, row_pos=dpos, row_weight=dweight)
        idx = np.broadcast_to(np.arange(W, dtype=np.int32), (b, s, W)).copy()
        idx[:, :, :3] = -1
        lse_w = torch.empty(b, s, h, device="cuda")
        o_w = sti.sparse_attn_sink(dq, to_dev(win), to_dev_any(sink), to_dev_any(idx), scale, lse=lse_w)
        lse = torch.empty(b, s, h, device="cuda")
        before = dweight.cpu().numpy()
        out = sti.attn_fp4kv(dq, dcodes, dscales, dsp, ratio, scale, dropped=ddrop, prev_out=o_w, prev_lse=lse_w, lse=lse,
                             row_weight=dweight)
        # the oracle, with the window's part as the device holds it
        assert not orc.kv_append_fp4(bf16_bits_to_f32(x), start, dropped, s, ratio, "e4m3", codes, scales, pos, weight)
        np.testing.assert_array_equal(before, weight)
        ref = orc.attn_fp4kv(bf16_bits_to_f32(q), codes, scales, start, ratio, scale, None, dropped, bf16_out_to_f64(o_w),
                             lse_w.cpu().numpy())
        got_w = dweight.cpu().numpy()
        check_attention(bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), ref, bf16_bits_to_f32(q), codes, scales,
                        scale, got_w.astype(np.float64), weight)
        weight[:] = got_w          # the eviction ranks the same numbers on both sides
        sti.kv_evict(dweight, dpos, dsp, s, ratio, ddrop, budget, first, recent, [dcodes, dscales])
        orc.kv_evict(weight, pos, start, s, ratio, dropped, budget, first, recent, [codes, scales])
        for u, v in ((dweight, weight), (dpos, pos), (ddrop, dropped), (dcodes, codes), (dscales, scales)):
            np.testing.assert_array_equal(u.cpu().numpy(), v)
        start += s
    assert (dropped > 0).all()


# ---------------------------------------------------------------------------------- refusals (no GPU)


@pytest.fixture(scope="module")
def lib():
    from sparse_top_attention_indexer_gb300 import _build

    _build.build()
    import sparse_top_attention_indexer_gb300 as m

    return m.lib()


P = ctypes.c_void_p
FAKE = 1 << 20   # an aligned address that nothing dereferences


def test_append_refusals(lib):
    def call(x=P(FAKE), xb=10 * 512, sp=P(FAKE), b=2, s=10, ratio=1, dim=512, fmt=0, codes=P(FAKE), cb=100 * 256,
             scales=P(FAKE), sb=100 * 32, rows=100, pos=None, pb=0, w=None, wb=0, ws=None):
        return lib.sti_kv_append_fp4(x, xb, sp, None, b, s, ratio, dim, fmt, codes, cb, scales, sb, rows, pos, pb, w, wb, ws,
                                     None)

    for kw in (dict(x=None), dict(x=P(FAKE + 8)), dict(xb=10 * 512 - 8), dict(xb=10 * 512 + 4), dict(sp=None),
               dict(s=0), dict(ratio=0), dict(fmt=2), dict(fmt=-1), dict(codes=None), dict(codes=P(FAKE + 8)),
               dict(cb=100 * 256 - 16), dict(cb=100 * 256 + 8), dict(scales=None), dict(sb=100 * 32 - 1),
               dict(rows=-1), dict(pos=P(FAKE), pb=99), dict(w=P(FAKE), wb=99), dict(b=-1),
               dict(ws=P(FAKE + 8)), dict(dim=0)):
        assert call(**kw) == 1, kw
    assert call(dim=96, cb=1 << 20, sb=1 << 20) == 2
    assert call(s=0x7FFFFFFF) == 2
    assert call(b=0) == 0


def test_attend_refusals(lib):
    need = lib.sti_attn_fp4kv_workspace_size(2, 3, 64, 512, 100)

    def call(q=P(FAKE), codes=P(FAKE), cb=100 * 256, scales=P(FAKE), sb=100 * 32, rows=100, sp=P(FAKE), ratio=1, po=None,
             pl=None, b=2, s=3, h=64, d=512, out=P(FAKE * 4), lse=None, w=None, wb=0, ws=P(FAKE * 64), wsb=need):
        return lib.sti_attn_fp4kv(q, codes, cb, scales, sb, rows, sp, None, ratio, None, 0.1, po, pl, b, s, h, d, out, lse, w,
                                  wb, ws, wsb, None)

    for kw in (dict(q=None), dict(q=P(FAKE + 8)), dict(out=None), dict(out=P(FAKE * 4 + 2)), dict(codes=None),
               dict(codes=P(FAKE + 4)), dict(cb=100 * 256 - 16), dict(cb=100 * 256 + 4), dict(scales=None),
               dict(scales=P(FAKE + 2)), dict(sb=100 * 32 - 4), dict(sb=100 * 32 + 2), dict(sp=None), dict(ratio=0),
               dict(s=0), dict(h=0), dict(d=0), dict(rows=-1),
               dict(po=P(FAKE * 8)), dict(pl=P(FAKE * 8)), dict(po=P(FAKE * 8 + 8), pl=P(FAKE * 16)),
               dict(w=P(FAKE), wb=99), dict(ws=None), dict(ws=P(FAKE * 64 + 8)), dict(wsb=need - 1), dict(b=-1),
               dict(out=P(FAKE)), dict(out=P(FAKE + 1024)),                                 # over q
               dict(po=P(FAKE * 4 + 1024), pl=P(FAKE * 16)),                                # out partly over prev_out
               dict(po=P(FAKE * 4), pl=P(FAKE * 16), lse=P(FAKE * 16))):                    # lse over prev_lse
        assert call(**kw) == 1, kw
    for kw in (dict(h=65), dict(d=96), dict(d=576), dict(s=0x7FFFFFFF)):
        assert call(**kw) == 2, kw
    assert call(b=0) == 0
    assert lib.sti_attn_fp4kv_workspace_size(0, 1, 64, 512, 100) == 256


def test_evict_refusals(lib):
    import sparse_top_attention_indexer_gb300 as m

    need = lib.sti_kv_evict_workspace_size(2, 100, 80)
    arr = (m.RowArray * 17)()
    for i in range(17):
        arr[i].base, arr[i].bstride, arr[i].row_bytes = FAKE, 100 * 32, 32

    def call(w=P(FAKE), wb=100, pos=P(FAKE), pb=100, sp=P(FAKE), dropped=P(FAKE), b=2, s=1, ratio=1, rows=100, budget=80,
             first=4, recent=8, arrays=arr, n=1, ws=P(FAKE * 64), wsb=need):
        return lib.sti_kv_evict(w, wb, pos, pb, sp, dropped, b, s, ratio, rows, budget, first, recent, arrays, n, ws, wsb, None)

    for kw in (dict(w=None), dict(wb=99), dict(pos=None), dict(pb=99), dict(sp=None), dict(dropped=None), dict(b=-1),
               dict(s=0), dict(ratio=0), dict(rows=-1), dict(budget=-1), dict(first=-1), dict(recent=-1),
               dict(first=40, recent=41), dict(n=17), dict(n=-1), dict(arrays=None), dict(ws=None),
               dict(ws=P(FAKE * 64 + 8)), dict(wsb=need - 1)):
        assert call(**kw) == 1, kw
    for field, value in (("base", None), ("bstride", 100 * 32 - 1), ("row_bytes", 0)):
        keep = getattr(arr[0], field)
        setattr(arr[0], field, value)
        assert call() == 1, field
        setattr(arr[0], field, keep)
    arr[0].row_bytes, arr[0].bstride = 65537, 1 << 30
    assert call() == 2
    arr[0].row_bytes, arr[0].bstride = 32, 3200
    assert call(b=0) == 0
    assert call(budget=100, w=None, ws=None) == 0      # nothing can be over the budget
    assert lib.sti_kv_evict_workspace_size(2, 100, 100) == 256


# ---------------------------------------------------------------------------------- the oracle itself


def test_oracle_evict_by_hand(orc):
    w = np.array([[5.0, 1.0, 4.0, 1.0, 3.0, 9.0, 2.0]], np.float32)
    pos = np.array([[10, 11, 12, 13, 14, 15, 16]], np.int32)
    dropped = np.array([10], np.int32)
    tag = np.arange(7)[None].copy()
    # 7 held, budget 4, the latest group (16) protected: stay 0 (5.0), 2 (4.0), 5 (9.0), 6 (recent)
    orc.kv_evict(w, pos, np.array([16]), 1, 1, dropped, 4, 0, 1, [tag])
    assert tag[0, :4].tolist() == [0, 5, 2, 6] and dropped[0] == 13
    assert w[0, :4].tolist() == [5.0, 9.0, 4.0, 2.0] and pos[0, :4].tolist() == [10, 15, 12, 16]


def test_oracle_attention_is_the_sparse_oracle(orc):
    """Over the visible rows listed as indices, the attention is the pinned sparse oracle's; the weights add up
    to one per head and query less the sink's share."""
    rng = rng_for(9700, 0)
    codes, scales = rows_of(rng, 1, 50, 64)
    q = to_bf16_bits(rng.standard_normal((1, 3, 4, 64)))
    sink = rng.standard_normal(4).astype(np.float32)
    out, lse, w, _ = orc.attn_fp4kv(bf16_bits_to_f32(q), codes, scales, [100], 4, 0.125, sink, [2])
    idx = np.stack([np.where(np.arange(50) < (100 + t + 1) // 4 - 2, np.arange(50), -1) for t in range(3)])[None]
    ref, ref_lse = orc.sparse_attn_fp4kv(q, np.zeros((1, 0, 64), np.uint16), codes, scales, sink, idx.astype(np.int32), 0.125)
    np.testing.assert_allclose(out, ref, atol=1e-12)
    np.testing.assert_allclose(lse, ref_lse, atol=1e-12)
    np.testing.assert_allclose(w.sum(), (1 - np.exp(sink - lse)).sum(), rtol=1e-12)


def test_oracle_attention_joins_parts(orc):
    """Rows attended in two parts and joined through prev_out / prev_lse are the rows attended at once."""
    rng = rng_for(9701, 0)
    codes, scales = rows_of(rng, 1, 40, 64)
    q = rng.standard_normal((1, 1, 3, 64))
    whole = orc.attn_fp4kv(q, codes, scales, [39], 1, 0.2)
    a = orc.attn_fp4kv(q, codes[:, :25], scales[:, :25], [24], 1, 0.2)
    b = orc.attn_fp4kv(q, codes[:, 25:], scales[:, 25:], [14], 1, 0.2, prev_out=a[0], prev_lse=a[1])
    np.testing.assert_allclose(b[0], whole[0], atol=1e-12)
    np.testing.assert_allclose(b[1], whole[1], atol=1e-12)
    np.testing.assert_allclose(b[2][0], whole[2][0, 25:], atol=1e-12)
