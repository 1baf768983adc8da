"""The bounded 4-bit cache: sizes of its workspaces, refusals of arguments at the edge of what fits."""
import ctypes

import pytest

from tests.test_fp4_cache import FAKE, P, attend, lib, make_attend, sti  # noqa: F401  (fixtures among them)
from tests._util import to_dev, to_dev_any

gpu = pytest.mark.gpu


def test_workspace_without_row_weights(lib):  # noqa: F811
    """The scores and sums that row weights need are not asked of a call that cannot want them: at most two partial
    outputs per CTA (160) of 64 heads, with their statistics, remain."""
    for size in ((32, 1, 64, 512, 16384), (1, 2048, 64, 512, 2048), (64, 8, 64, 64, 2048), (3, 300, 1, 64, 4), (2, 3, 8, 64, 0)):
        need = lib.sti_attn_fp4kv_noweights_workspace_size(*size)
        assert 256 <= need <= 4096 + 160 * 8 + 320 * 64 * 8 + 320 * 64 * size[3] * 4
        assert need < lib.sti_attn_fp4kv_workspace_size(*size)
    assert lib.sti_attn_fp4kv_noweights_workspace_size(0, 1, 64, 512, 100) == 256


def test_noweights_refusals(lib):  # noqa: F811
    need = lib.sti_attn_fp4kv_noweights_workspace_size(2, 3, 64, 512, 100)

    def call(q=P(FAKE), codes=P(FAKE), cb=100 * 256, scales=P(FAKE), sb=100 * 32, rows=100, sp=P(FAKE), ratio=1, po=None,
             pl=None, b=2, s=3, h=64, d=512, out=P(FAKE * 4), lse=None, ws=P(FAKE * 64), wsb=need):
        return lib.sti_attn_fp4kv_noweights(q, codes, cb, scales, sb, rows, sp, None, ratio, None, 0.1, po, pl, b, s, h, d,
                                            out, lse, ws, wsb, None)

    for kw in (dict(q=None), dict(out=None), dict(codes=None), dict(cb=100 * 256 - 16), dict(scales=P(FAKE + 2)), dict(sp=None),
               dict(ratio=0), dict(s=0), dict(rows=-1), dict(po=P(FAKE * 8)), dict(ws=None), dict(ws=P(FAKE * 64 + 8)),
               dict(wsb=need - 1), dict(b=-1), dict(out=P(FAKE))):
        assert call(**kw) == 1, kw
    for kw in (dict(h=65), dict(d=96), dict(s=0x7FFFFFFF)):
        assert call(**kw) == 2, kw
    assert call(b=0) == 0


@gpu
@pytest.mark.parametrize("name", ["long_split", "ragged_empty_prev", "few_heads", "packed_split", "packed_one_head"])
def test_attend_in_the_smaller_workspace(sti, name):  # noqa: F811
    """Without row weights: the same outputs from the smaller workspace, and no byte behind it written."""
    import torch

    a = make_attend(name)
    want, want_lse, _ = attend(sti, a)
    n = sti.attn_fp4kv_workspace_size(*a["q"].shape, a["codes"].shape[1], row_weight=False)
    room = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[:n]
    ws.zero_()
    opt = lambda v: None if v is None else to_dev_any(v)  # noqa: E731
    lse = torch.empty_like(want_lse)
    out = sti.attn_fp4kv(to_dev(a["q"]), to_dev_any(a["codes"]), to_dev_any(a["scales"]), to_dev_any(a["start_pos"]), a["ratio"],
                         a["scale"], attn_sink=opt(a["sink"]), dropped=opt(a["dropped"]),
                         prev_out=None if a["prev_out"] is None else to_dev(a["prev_out"]), prev_lse=opt(a["prev_lse"]),
                         lse=lse, ws=ws)
    assert sti.read_device_status(ws) == 0
    assert (out == want).all() and (lse == want_lse).all() and (room[n:] == 0xA5).all()
    with pytest.raises(sti.StiError):
        sti.attn_fp4kv(to_dev(a["q"]), to_dev_any(a["codes"]), to_dev_any(a["scales"]), to_dev_any(a["start_pos"]), a["ratio"],
                       a["scale"], row_weight=to_dev_any(a["w0"]), ws=ws)


def test_refuses_more_rows_than_32_bit_row_numbers_hold(lib):  # noqa: F811
    """Rows are counted in 32 bits, rounded up to tiles and to a cluster's steps: 2^30 fit, 2^31 - 1 would not."""
    rows, big = (1 << 30) + 1, 1 << 62
    for r in (rows, 0x7FFFFFFF):
        assert lib.sti_attn_fp4kv(P(FAKE), P(FAKE), r * 32, P(FAKE), r * 4, r, P(FAKE), None, 1, None, 0.1, None, None, 1, 1, 8, 64,
                                  P(FAKE * 4), None, None, 0, P(FAKE * 64), big, None) == 2
        assert lib.sti_attn_fp4kv_noweights(P(FAKE), P(FAKE), r * 32, P(FAKE), r * 4, r, P(FAKE), None, 1, None, 0.1, None, None, 1,
                                            1, 8, 64, P(FAKE * 4), None, P(FAKE * 64), big, None) == 2
        assert lib.sti_kv_evict(P(FAKE), r, P(FAKE), r, P(FAKE), P(FAKE), 1, 1, 1, r, 100, 4, 8, None, 0, P(FAKE * 64), big,
                                None) == 2


@gpu
@pytest.mark.parametrize("n", [0, 1, 255])
def test_append_refuses_a_workspace_that_is_too_small(sti, n):  # noqa: F811
    """A status word that does not fit ws would be written behind it (or, with no bytes, nowhere)."""
    import torch

    room = torch.zeros(512, dtype=torch.uint8, device="cuda")
    x = torch.ones(1, 1, 64, dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros(1, 1, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(1, 1, 4, dtype=torch.uint8, device="cuda")
    start = torch.full((1,), 7, dtype=torch.int32, device="cuda")       # row 7 of 1
    with pytest.raises(ValueError, match="ws"):
        sti.kv_append_fp4(x, start, 1, 1, codes, scales, ws=room[:n])
    assert (room == 0).all() and (codes == 0).all()
    sti.kv_append_fp4(x, start, 1, 1, codes, scales, ws=room[:256])
    assert sti.read_device_status(room[:256]) == sti.FLAG_INDEX_RANGE and (codes == 0).all()


@gpu
def test_evict_an_array_listed_twice(sti):  # noqa: F811
    """The same array twice, and row_weight and row_pos themselves, in the list: each row moves once all the same."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(3)
    b, rows, budget = 3, 300, 200
    w = torch.rand(b, rows, generator=gen, device="cuda")
    pos = torch.arange(rows, device="cuda", dtype=torch.int32).repeat(b, 1)
    tag = torch.arange(b * rows * 5, device="cuda", dtype=torch.int16).view(b, rows, 5)
    start = torch.tensor([299, 250, 100], device="cuda", dtype=torch.int32)

    def run(arrays):
        st = [w.clone(), pos.clone(), tag.clone(), torch.zeros(b, device="cuda", dtype=torch.int32)]
        sti.kv_evict(st[0], st[1], start, 1, 1, st[3], budget, 4, 8, [st[i] for i in arrays])
        return st

    for x, y in zip(run([2]), run([2, 0, 1, 2])):
        assert (x == y).all()
