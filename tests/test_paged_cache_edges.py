"""The paged latent cache at its edges."""
import numpy as np
import pytest

from tests._util import bf16_out_to_f64, to_dev
from tests.test_fp4_cache import FAKE, P, lib, sti  # noqa: F401  (fixtures among them)
from tests.test_paged_cache import attend, attend_reference, check_attention, page_table, seen_by
from workloads import bf16_bits_to_f32, rng_for, to_bf16_bits

gpu = pytest.mark.gpu


def attention(b, s, h, d, page, rows, level=0.0, sink=None, prev_lse=None, seed=0):
    """Queries after `rows` rows per sequence, every score about `level`."""
    rng = rng_for(7600 + seed, b * s * h + d)
    kv = rng.standard_normal((b, rows + s, d))
    kv[..., 0] = -20 if level < 0 else 20
    q = 0.1 * rng.standard_normal((b, s, h, d))
    q[..., 0] = abs(level) * d ** 0.5 / 20
    kv, q = to_bf16_bits(kv), to_bf16_bits(q)
    table, n = page_table(rng, b, [-(-(rows + s) // page)] * b)
    pool = np.zeros((n, page, d), np.uint16)
    for i in range(b):
        for p in range(rows + s):
            pool[table[i, p // page], p % page] = kv[i, p]
    a = dict(q=q, pool=pool, table=table, start=np.full(b, rows, np.int32), count=np.full(b, s, np.int32), n_new=None, window=0,
             n_first=0, scale=d ** -0.5, kv=list(kv), sink=None if sink is None else np.full(h, sink, np.float32),
             prev_out=None, prev_lse=None)
    if prev_lse is not None:
        a["prev_out"] = to_bf16_bits(rng.standard_normal((b, s, h, d)))
        a["prev_lse"] = np.full((b, s, h), prev_lse, np.float32)
    return a


@gpu
@pytest.mark.parametrize("level", [-120.0, 0.0, 100.0])
@pytest.mark.parametrize("sink,prev_lse", [(None, None), (-200.0, None), (None, -200.0), (-118.0, -121.0)])
@pytest.mark.parametrize("b,s,h,rows", [(2, 1, 64, 200), (2, 5, 6, 250), (3, 1, 40, 5000), (3, 3, 20, 5000)])
def test_first_tile_of_bad_pages(sti, b, s, h, rows, sink, prev_lse, level):  # noqa: F811
    """Every other tile lies in pages that the pool does not have, the first among them (in the cases of 5000 rows, the first
    tile of every SM's two): the other rows' attention, however low their scores, the sink and the other part's lse are."""
    a = attention(b, s, h, 64, 64, rows, level, sink, prev_lse)
    a["table"][:, ::2] = [-1, a["pool"].shape[0]][h & 1]
    out, lse, ws = attend(sti, a)
    assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
    check_attention(a, bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64), attend_reference(a, lambda i, p: p // 64 % 2 == 0))


@gpu
@pytest.mark.parametrize("b,s,tokens_first", [(3, 1, False), (32, 1, False), (3, 5, True), (3, 1, True), (1, 4, True), (1, 1, False)])
def test_rotate_between_slices(sti, b, s, tokens_first):  # noqa: F811
    """From one part of a fused projection into another of the same tokens, for a prompt, a single token and tokens outermost."""
    import torch

    h, d = 6, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    freqs, pos = sti.rope_freqs(32), torch.arange(b, dtype=torch.int32, device="cuda")
    first, second = (s, b) if tokens_first else (b, s)
    whole = torch.randn(first, second, 3 * h * d, generator=g, device="cuda").bfloat16()
    qkv = whole.transpose(0, 1) if tokens_first else whole
    part = lambda t, i: t[..., i * h * d:(i + 1) * h * d].unflatten(-1, (h, d))  # noqa: E731
    for src, dst in ((0, 2), (0, 1), (2, 1)):
        keep = qkv.clone()
        want = sti.norm_rope(part(keep, src).contiguous(), pos, freqs)
        sti.norm_rope(part(qkv, src), pos, freqs, out=part(qkv, dst))
        assert (part(qkv, dst) == want).all()
        for i in {0, 1, 2} - {dst}:
            assert (part(qkv, i) == part(keep, i)).all()


def test_rotate_onto_itself_refused(lib):  # noqa: F811
    """Parts that share elements, by every order of the strides: refused."""
    h, d = 4, 64
    n = h * d

    def call(b, s, bs, ts, off):
        return lib.sti_norm_rope(P(FAKE), bs, ts, P(FAKE), 0, None, b, s, h, d, 1, None, 1e-6, P(FAKE), 32, 32, 0, 1.0,
                                 P(FAKE + 2 * off), bs, ts, None)

    for b, s, bs, ts in ((3, 1, 3 * n, n), (3, 5, 15 * n, 3 * n), (3, 5, 3 * n, 9 * n), (1, 5, 0, 3 * n), (1, 1, n, n),
                         (3, 2, 7 * n, 3 * n)):
        apart = {i * bs + j * ts for i in range(1 - b, b) for j in range(1 - s, s)}
        tried = 0
        for off in {at + k for at in apart for k in (8 - n, -8, 0, 8, n - 8)}:
            if off > 0:
                assert call(b, s, bs, ts, off) == 1, (b, s, bs, ts, off)
                tried += 1
        assert tried >= 2


@gpu
def test_append_to_a_table_of_no_pages(sti):  # noqa: F811
    """A table without columns: every position is past it, nothing is written, and it is reported."""
    import torch

    x = torch.randn(2, 3, 64, device="cuda").bfloat16()
    pages = torch.full((4, 16, 64), -7.0, dtype=torch.bfloat16, device="cuda")
    start, empty = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    ws = sti.workspace(256)
    sti.kv_append_paged(x, start, pages, empty, ws=ws)
    assert sti.read_device_status(ws) == sti.FLAG_INDEX_RANGE
    assert (pages == -7).all()


@gpu
@pytest.mark.parametrize("s,h", [(1, 64), (4, 4), (4, 16), (7, 9)])
def test_scores_past_fp32(sti, s, h):  # noqa: F811
    """A finite row whose scores are below fp32's range has no weight, with few heads as with many."""
    a = attention(1, s, h, 128, 16, 90, seed=1)
    q, kv = a["q"], a["kv"][0]
    q[..., 0] = to_bf16_bits(np.array([1e20]))[0]
    kv[:, 0] = 0
    kv[37, 0] = kv[70, 0] = to_bf16_bits(np.array([-1e20]))[0]
    kv[70, 1] = to_bf16_bits(np.array([3e38]))[0]
    q[..., 1] = to_bf16_bits(np.array([-2.0]))[0]
    kv[np.arange(len(kv)) != 70, 1] = 0
    for p in range(len(kv)):
        a["pool"][a["table"][0, p // 16], p % 16] = kv[p]
    out, lse, ws = attend(sti, a)
    assert sti.read_device_status(ws) == 0
    check_attention(a, bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64),
                    attend_reference(a, lambda i, p: (p == 37) | (p == 70)))


@gpu
@pytest.mark.parametrize("s,h", [(4, 4), (8, 8), (2, 32)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows_of_one_sign(sti, s, h, value):  # noqa: F811
    """Queries that share tiles with one that sees a row with an infinity or NaN, all scores with it of one sign: those that see
    it have an undefined output, every head of theirs, the others what they had without it."""
    import torch

    a = attention(1, s, h, 128, 16, 90, seed=2)
    q, pages = to_dev(a["q"]), to_dev(a["pool"])
    table, start = torch.from_numpy(a["table"]).cuda(), torch.tensor([90], dtype=torch.int32, device="cuda")
    q[..., 7] = -3.0
    want = sti.attn_paged(q, pages, table, start, a["scale"])
    at = 90 + s // 2
    pages[int(table[0, at // 16]), at % 16, 7] = value
    got = [sti.attn_paged(q, pages, table, start, a["scale"]) for _ in range(5)]
    for o in got:
        assert (o[0, :s // 2] == want[0, :s // 2]).all()
        assert o[0, s // 2:].isnan().any(-1).all()


@gpu
@pytest.mark.parametrize("tokens", [True, False])
def test_lists_of_seconds(sti, tokens):  # noqa: F811
    """As many queries as SMs, each over 268 million rows, all but the last page's the same page of zeros: two seconds of one CTA
    per query, longer than any wait for a single tile may take.  The last page has all of the weight: the others' rows have e^-40 of
    a row's there each, 2 10^-9 together."""
    import torch

    n = torch.cuda.get_device_properties(0).multi_processor_count
    b, s = (1, n) if tokens else (n, 1)
    h, d, page, most = 64, 64, 8192, 32768
    a = attention(1, s, h, d, page, 200, 40.0, seed=3)      # what is seen of the last page
    q = to_dev(a["q"]).expand(b, s, h, d).contiguous()
    pages = torch.zeros(2, page, d, dtype=torch.bfloat16, device="cuda")
    pages[1] = to_dev(a["pool"])[int(a["table"][0, 0])]
    table = torch.zeros(b, most, dtype=torch.int32, device="cuda")
    table[:, -1] = 1
    start = torch.full((b,), (most - 1) * page + 200, dtype=torch.int32, device="cuda")
    ws, lse = sti.workspace(sti.attn_paged_workspace_size(b, s, h, d)), torch.empty(b, s, h, device="cuda")
    out = sti.attn_paged(q, pages, table, start, a["scale"], lse=lse, ws=ws)
    assert sti.read_device_status(ws) == 0
    ref = attend_reference(a)
    for i in {0, b // 2, b - 1}:
        check_attention(a, bf16_out_to_f64(out[i:i + 1]), lse[i:i + 1].cpu().numpy().astype(np.float64), ref)


@gpu
@pytest.mark.parametrize("s,h", [(1, 64), (3, 10)])
def test_joined_calls_follow_one_another(sti, s, h):  # noqa: F811
    """Two parts of a context attended one after the other, the second joined with the first, again and again into the same buffers
    with other queries, lengths and pages each time and no wait in between: what calls with waits give."""
    import torch

    b, d, page = 6, 128, 64
    g = torch.Generator(device="cuda").manual_seed(s)
    pages = torch.randn(2, 60, page, d, generator=g, device="cuda").bfloat16()
    qs = [torch.randn(b, s, h, d, generator=g, device="cuda").bfloat16() for _ in range(4)]
    starts = [torch.randint(0, 600, (b,), generator=g, device="cuda", dtype=torch.int32) for _ in range(4)]
    tables = [torch.randint(0, 60, (b, 10), generator=g, device="cuda", dtype=torch.int32) for _ in range(4)]
    q, start, table = qs[0].clone(), starts[0].clone(), tables[0].clone()
    part, lse = torch.empty_like(q), torch.empty(b, s, h, device="cuda")
    ws = sti.workspace(sti.attn_paged_workspace_size(b, s, h, d))
    f = sti.rope_freqs(64)

    def step(i, wait=lambda: None):
        for to, one in ((q, qs[i]), (start, starts[i]), (table, tables[i])):
            to.copy_(one)
        wait()
        sti.norm_rope(q, start, f, out=q)
        wait()
        sti.attn_paged(q, pages[0], table, start, d ** -0.5, out=part, lse=lse, ws=ws)
        wait()
        return sti.attn_paged(q, pages[1], table, start, d ** -0.5, prev_out=part, prev_lse=lse, ws=ws)

    want = [step(i, torch.cuda.synchronize) for i in range(4)]
    got = [step(i % 4) for i in range(80)]
    for i, o in enumerate(got):
        assert (o == want[i % 4]).all(), i


def test_workspace_sizes(lib):  # noqa: F811
    """Room for a record and two parts (maximum and sum of 64 heads, outputs of the heads that share tiles) of each of the 160 CTAs
    that a call has at most, for every number of sequences, tokens and heads."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    for b in (1, 2, 7, 150, 4096):
        for s in (1, 2, 5, 63, 64, 2048):
            for h in (1, 2, 3, 5, 16, 20, 31, 32, 33, 57, 64):
                for d in (64, 192, 512):
                    heads = h * (min(64 // h, s) if h <= 32 else 1)
                    want = 256 + up(160 * 8) + up(320 * 64 * 8) + up(320 * (-(-heads // 4) * 4) * d * 4)
                    assert lib.sti_attn_paged_workspace_size(b, s, h, d) == want, (b, s, h, d)


@gpu
@pytest.mark.parametrize("b,s,h,d,window", [(3, 1, 64, 512, 128), (2, 4, 64, 128, 40), (2, 9, 16, 64, 20)])
def test_joined_with_selected_rows(sti, b, s, h, d, window):  # noqa: F811
    """A layer's attention over the rows that the indexer chose (with the sink), joined with a window of the paged cache, one query
    without any chosen row: the attention over both.  Rounded to bf16: P in both kernels (2^-8 of each row's share), the first one's
    output (2^-8 of its share) and the output; the first one's lse is off by at most 1e-4 (1 + |lse|), as its own tests hold it to."""
    import torch

    rng = rng_for(7700, b * s * h + d)
    a = attention(b, s, h, d, 16, 60, seed=4)
    a.update(window=window, n_first=2, q=to_bf16_bits(2 * rng.standard_normal((b, s, h, d))))
    sink = rng.standard_normal(h).astype(np.float32)
    rows, k = 300, 96
    chosen = to_bf16_bits(rng.standard_normal((b, rows, d)))
    idx = np.stack([[rng.permutation(rows)[:k] for _ in range(s)] for _ in range(b)]).astype(np.int32)
    idx[..., k - 5:] = -1
    idx[b - 1, s - 1] = -1
    part_lse = torch.empty(b, s, h, device="cuda")
    q = to_dev(a["q"])
    part = sti.sparse_attn_sink(q, to_dev(chosen), torch.from_numpy(sink).cuda(), torch.from_numpy(idx).cuda(), a["scale"], lse=part_lse)
    assert (part_lse[b - 1, s - 1] == float("-inf")).all()
    out, lse, ws = attend(sti, a, prev_out=part, prev_lse=part_lse)
    assert sti.read_device_status(ws) == 0
    got, got_lse = bf16_out_to_f64(out), lse.cpu().numpy().astype(np.float64)
    qf, scale = bf16_bits_to_f32(a["q"]).astype(np.float64), a["scale"]
    for i in range(b):
        for t in range(s):
            p = np.nonzero(seen_by(60 + t, window, 2))[0]
            one = idx[i, t][idx[i, t] >= 0]
            kv = bf16_bits_to_f32(np.concatenate([a["kv"][i][p], chosen[i][one]])).astype(np.float64)
            e = np.exp(scale * qf[i, t] @ kv.T)
            total = e.sum(1) + (np.exp(sink.astype(np.float64)) if len(one) else 0)
            want, mass, L = e @ kv / total[:, None], e @ np.abs(kv) / total[:, None], np.log(total)
            assert (np.abs(got_lse[i, t] - L) <= 2e-4 * (1 + np.abs(L))).all()
            off = 2.0 ** -8 * np.abs(want) + (2.0 ** -7 + 2e-4 * (1 + np.abs(L[:, None]))) * mass
            assert (np.abs(got[i, t] - want) <= off).all()
