"""The paged latent cache called as a serving program does: from two host threads, from graphs that share a workspace, in
place, with the same page twice."""
import numpy as np
import pytest

from tests.test_fp4_cache import sti  # noqa: F401  (the fixture)
from tests.test_fp4_cache_threads import both
from tests.test_paged_cache import attend, layer_state, layer_step, make_attend, opt, to_dev, to_dev_any

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("names", [("one_tile_less", "runs_d64"), ("parts_9_d512", "packed_padded"), ("parts_3", "ragged")])
def test_two_threads(sti, names):  # noqa: F811
    """Two threads attend on streams of their own, caches of different sizes (and kernels): what each gives alone."""
    import torch

    cases = [make_attend(n) for n in names]
    want = [attend(sti, a)[:2] for a in cases]
    jobs, outs = [], []
    for a in cases:
        t = [to_dev(a["q"]), to_dev(a["pool"]), to_dev_any(a["table"]), to_dev_any(a["start"])]
        kw = dict(window=a["window"], n_first=a["n_first"], attn_sink=opt(a["sink"]), prev_out=opt(a["prev_out"], to_dev),
                  prev_lse=opt(a["prev_lse"]), n_new=opt(a["n_new"]),
                  ws=sti.workspace(sti.attn_paged_workspace_size(*a["q"].shape)), stream=torch.cuda.Stream(),
                  out=torch.full(a["q"].shape, -7.0, dtype=torch.bfloat16, device="cuda"),
                  lse=torch.full(a["q"].shape[:3], -7.0, device="cuda"))

        def job(t=t, kw=kw, scale=a["scale"]):
            for _ in range(300):
                sti.attn_paged(*t, scale, **kw)
            kw["stream"].synchronize()

        jobs.append(job)
        outs.append(kw)
    torch.cuda.synchronize()
    errors = both(jobs)
    assert not errors, errors
    for (o, l), kw in zip(want, outs):
        assert (kw["out"] == o).all() and (kw["lse"] == l).all()


@gpu
def test_steps_of_two_layers(sti):  # noqa: F811
    """Two threads, each with its layer's step (norm, rotate, append, attend the window and the older rows, rotate back)."""
    import torch

    def layer(b, h, d, seed):
        st = layer_state(sti, b, h, d, 8, 8, 20, 3, older=300)
        xs = torch.randn(40, b, 1, (h + 1) * d, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()
        stream = torch.cuda.Stream()

        def job():
            with torch.cuda.stream(stream):
                st["out"] = torch.stack([layer_step(sti, st, x) for x in xs])
            stream.synchronize()

        return st, job

    kinds = [(3, 64, 512, 1), (5, 8, 128, 2)]
    alone, together = [layer(*k) for k in kinds], [layer(*k) for k in kinds]
    torch.cuda.synchronize()
    for _, job in alone:
        job()
    errors = both([job for _, job in together])
    assert not errors, errors
    for (one, _), (two, _) in zip(alone, together):
        assert (one["out"] == two["out"]).all() and (one["pages"].nan_to_num() == two["pages"].nan_to_num()).all()


@gpu
def test_graphs_share_a_workspace(sti):  # noqa: F811
    """Two graphs of different batches and an eager call, in turn in one stream with one workspace, lengths changed between
    the replays: each time what calls with workspaces of their own give."""
    import torch

    cases = [make_attend(n) for n in ("parts_9_d512", "parts_7_heads_33", "long_split")]
    size = max(sti.attn_paged_workspace_size(*a["q"].shape) for a in cases)
    ws = sti.workspace(size)
    runs = []
    for a in cases:
        t = [to_dev(a["q"]), to_dev(a["pool"]).nan_to_num(), to_dev_any(np.maximum(a["table"], 0)), to_dev_any(a["start"])]
        kw = dict(attn_sink=opt(a["sink"]), prev_out=opt(a["prev_out"], to_dev), prev_lse=opt(a["prev_lse"]))
        runs.append((a, t, kw, torch.empty_like(t[0]), torch.empty(a["q"].shape[:3], device="cuda")))
    torch.cuda.synchronize()
    stream, graphs = torch.cuda.Stream(), []
    with torch.cuda.stream(stream):
        for a, t, kw, out, lse in runs[:2]:
            sti.attn_paged(*t, a["scale"], out=out, lse=lse, ws=ws, **kw)
            stream.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                sti.attn_paged(*t, a["scale"], out=out, lse=lse, ws=ws, **kw)
            graphs.append(g)
        for less in (0, 1, 130, 700):
            for a, t, *_ in runs:
                t[3].copy_(to_dev_any(np.maximum(a["start"] - less, 0)))
            for _, _, _, out, lse in runs:
                out.fill_(-7)
                lse.fill_(-7)
            graphs[0].replay()
            a, t, kw, out, lse = runs[2]
            sti.attn_paged(*t, a["scale"], out=out, lse=lse, ws=ws, **kw)
            graphs[1].replay()
            stream.synchronize()
            for a, t, kw, out, lse in runs:
                lse2 = torch.empty_like(lse)
                own = sti.workspace(sti.attn_paged_workspace_size(*a["q"].shape))
                assert (sti.attn_paged(*t, a["scale"], lse=lse2, ws=own, **kw) == out).all(), less
                assert (lse2 == lse).all()
    assert sti.read_device_status(ws) == 0


@gpu
def test_pages_shared_by_sequences(sti):  # noqa: F811
    """A prefix that two sequences share, and a sequence that lists one page twice: as with copies of the pages."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(4)
    pages = torch.randn(9, 32, 128, generator=g, device="cuda").bfloat16()
    table = torch.tensor([[0, 1, 2, 3], [0, 1, 4, 5], [6, 6, 7, 6]], dtype=torch.int32, device="cuda")
    start = torch.tensor([110, 127, 100], dtype=torch.int32, device="cuda")
    q = torch.randn(3, 1, 64, 128, generator=g, device="cuda").bfloat16()
    apart = pages[table.long().flatten()].contiguous()
    other = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    for window in (0, 40):
        got = sti.attn_paged(q, pages, table, start, 0.1, window=window, n_first=window // 8)
        assert (got == sti.attn_paged(q, apart, other, start, 0.1, window=window, n_first=window // 8)).all()


@gpu
def test_rotate_in_place_of_a_strided_slice(sti):  # noqa: F811
    """The queries of a fused projection normed and rotated where they lie, on another stream than the current one, padding
    tokens and the other columns left as they were."""
    import torch

    b, s, h, d = 3, 5, 7, 64
    x = torch.randn(b, s, (h + 2) * d, generator=torch.Generator(device="cuda").manual_seed(8), device="cuda").bfloat16()
    pos = torch.tensor([0, 2 ** 20, 77], dtype=torch.int32, device="cuda")
    n_new = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    f = sti.rope_freqs(32)
    q = x[..., d:(h + 1) * d].unflatten(-1, (h, d))
    want = x.clone()
    for i in range(b):
        n = int(n_new[i])
        if n:
            want[i, :n, d:(h + 1) * d] = sti.norm_rope(q[i:i + 1, :n].contiguous(), pos[i:i + 1], f, interleaved=False).flatten(-2)[0]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    assert sti.norm_rope(q, pos, f, interleaved=False, n_new=n_new, out=q, stream=stream) is q
    stream.synchronize()
    assert (x == want).all()


@gpu
def test_nothing_to_attend(sti):  # noqa: F811
    """No sequences; a table of no pages; no pool; a long table and a batch of padding alone."""
    import torch

    q = torch.randn(3, 2, 8, 64, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    pages = torch.zeros(4, 16, 64, dtype=torch.bfloat16, device="cuda")
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    empty = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    table = torch.full((3, 4000), -1, dtype=torch.int32, device="cuda")
    lse = torch.full((3, 2, 8), -7.0, device="cuda")
    assert sti.attn_paged(q[:0], pages, table[:0], start[:0], 1.0).shape == (0, 2, 8, 64)
    sti.kv_append_paged(q[:0, :, 0], start[:0], pages, table[:0])
    prev, prev_lse = torch.ones_like(q), torch.randn(3, 2, 8, device="cuda")
    for pool, tab in ((pages, empty), (pages[:0], table)):
        ws = sti.workspace(sti.attn_paged_workspace_size(3, 2, 8, 64))
        assert (sti.attn_paged(q, pool, tab, start, 1.0, lse=lse, ws=ws) == 0).all() and (lse == float("-inf")).all()
        assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
        assert (sti.attn_paged(q, pool, tab, start, 1.0, lse=lse, prev_out=prev, prev_lse=prev_lse, ws=ws) == 1).all()
        assert (lse == prev_lse).all()
    ws = sti.workspace(sti.attn_paged_workspace_size(3, 2, 8, 64))
    out = torch.full_like(q, 5)
    lse.fill_(5)
    sti.attn_paged(q, pages, table, start + 60000, 1.0, out=out, lse=lse, n_new=start, ws=ws)
    assert (out == 5).all() and (lse == 5).all() and sti.read_device_status(ws) == 0


@gpu
@pytest.mark.parametrize("rows", [40, 3000])
def test_calls_follow_one_another(sti, rows):  # noqa: F811
    """Rows appended, attended and the outputs rotated in one stream, again and again with other inputs and no wait in between:
    each kernel sees all that the one before wrote."""
    import torch

    b, h, d, page = 5, 64, 512, 64
    g = torch.Generator(device="cuda").manual_seed(rows)
    table = torch.randperm(b * (rows // page + 1), generator=g, device="cuda").int().view(b, -1)
    f, start = sti.rope_freqs(64), torch.zeros(b, dtype=torch.int32, device="cuda")
    at = torch.full((b,), rows - 1, dtype=torch.int32, device="cuda")
    xs = [torch.randn(b, rows, d, generator=g, device="cuda").bfloat16() for _ in range(3)]
    qs = [torch.randn(b, 1, h, d, generator=g, device="cuda").bfloat16() for _ in range(3)]
    pages = torch.zeros(table.numel(), page, d, dtype=torch.bfloat16, device="cuda")
    ws = sti.workspace(sti.attn_paged_workspace_size(b, 1, h, d))

    def run(i, wait):
        steps = (lambda _: sti.norm_rope(qs[i], at, f),
                 lambda q: sti.kv_append_paged(xs[i], start, pages, table, f, norm=True) or q,
                 lambda q: sti.attn_paged(q, pages, table, at, d ** -0.5, ws=ws),
                 lambda o: sti.norm_rope(o, at, f, inverse=True, norm=False, out=o))
        v = None
        for step in steps:
            v = step(v)
            if wait:
                torch.cuda.synchronize()
        return v

    want = [run(i, True) for i in range(3)]
    got = [run(i % 3, False) for i in range(60)]
    for i, o in enumerate(got):
        assert (o == want[i % 3]).all(), i
