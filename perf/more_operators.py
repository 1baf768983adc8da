"""The operators of a paged latent KV cache: per-head norm and rotation of the queries, norm, rotation and
append of the rows, attention over the pages (whole context, or a sliding window and the first tokens).

Each case is one call in its plain torch form (`own` false) or through the library (`own` true), on the same inputs.

A step brings `s` tokens to each of b sequences, the first at position start_pos [b]; n_new [b] of them are real
(a padded batch), the others leave their outputs as they were.  The cache is a pool of pages of `page` rows of
d bf16 values, one row per token, key and value of all heads; page table [b, most] says where position p lives:
row p % page of page table[b, p // page].
Rotation: `rd` of the d dims, pairs (2i, 2i + 1) ("pairs") or (i, i + rd / 2) ("halves") of them, by the angle
position * frequency_i; frequencies theta^(-2i / rd), for long contexts (`factor` > 1) divided by the factor where
they turn slowly (YaRN's ramp between 32 and 1 turns over the original length).
"""
import math

import torch

own = False

DEV = "cuda"
THETA, EPS = 10000.0, 1e-6
ORIG = 65536                    # the context that the frequencies of scaled cases were made for


# ---------------------------------------------------------------------------------- cases


def listed():
    return [
        # the queries of a decode step of 32 sequences near position 65536
        dict(name="rotate decode", op="rotate", b=32, s=1, h=64, d=512, rd=64, at="last", pairs=True, norm=True, weight=False,
             inverse=False, factor=16.0, far=65536, ragged=False),
        # the queries of a prefill chunk of 4096 tokens
        dict(name="rotate prefill", op="rotate", b=1, s=4096, h=64, d=512, rd=64, at="last", pairs=True, norm=True, weight=False,
             inverse=False, factor=16.0, far=65536, ragged=False),
        # outputs rotated back, narrow heads of the other layout, a padded batch, far positions
        dict(name="rotate back halves", op="rotate", b=4, s=301, h=20, d=128, rd=128, at="first", pairs=False, norm=False,
             weight=False, inverse=True, factor=1.0, far=1000000, ragged=True),
        # the rows that 32 decoding sequences bring in one step
        dict(name="append decode", op="append", b=32, s=1, d=512, rd=64, at="last", pairs=True, norm=True, weight=True,
             factor=16.0, page=64, ctx=2048, ragged=False),
        # the rows of a padded prefill of 8 sequences of up to 8192 tokens
        dict(name="append prefill", op="append", b=8, s=8192, d=512, rd=64, at="last", pairs=True, norm=True, weight=True,
             factor=16.0, page=64, ctx=8192, ragged=True),
        # narrow rows of the other layout into small pages
        dict(name="append odd", op="append", b=5, s=777, d=192, rd=64, at="first", pairs=False, norm=True, weight=True,
             factor=1.0, page=24, ctx=4000, ragged=True),
        # one short conversation, one token, a window layer: latency of a single call
        dict(name="attend one window", op="attend", b=1, s=1, h=64, d=512, page=64, ctx=700, window=128, first=4,
             prev=False, ragged=False),
        # the decode step of 32 sequences that attends to all of 16384 rows
        dict(name="attend decode", op="attend", b=32, s=1, h=64, d=512, page=64, ctx=16384, window=0, first=0,
             prev=False, ragged=False),
        # mixed serving: 64 sequences of up to 64k tokens, a window layer, joined with the compressed rows' attention
        dict(name="attend window mixed", op="attend", b=64, s=1, h=64, d=512, page=64, ctx=65536, window=4096, first=64,
             prev=True, ragged=True),
        # three draft tokens verified at once, few narrow heads, small pages
        dict(name="attend drafts", op="attend", b=12, s=3, h=20, d=128, page=24, ctx=4099, window=1000, first=5,
             prev=True, ragged=True),
        # a prefill chunk of 2048 queries that continues its sequence at 6144, whole context
        dict(name="attend chunk", op="attend", b=1, s=2048, h=64, d=512, page=64, ctx=8192, window=0, first=0,
             prev=False, ragged=False),
        # the same chunk in a window layer, for two sequences
        dict(name="attend chunk window", op="attend", b=2, s=2048, h=64, d=512, page=64, ctx=8192, window=128, first=4,
             prev=False, ragged=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "rotate", "append"])
    b = _log(rng, 1, 64)
    pairs = rng.random() < 0.6
    if op == "attend":
        h = rng.choice([64, 64, 32, 16, 8, 1, 5, 24, 40, 57])
        d = rng.choice([64, 128, 192, 256, 320, 512, 512, 512])
        s = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        ctx = max(s, _log(rng, 1, 65536))
        window = 0 if rng.random() < 0.4 else _log(rng, 1, 5000)
        page = rng.choice([1, 8, 16, 24, 64, 64, 100, 256])
        while b * s * ctx * 64 * 512 > 5.0e11 or b * ctx * d > 32 * 16384 * 512 or s * h * ctx > 1.08e9:
            if rng.random() < 0.5 and ctx > s:
                ctx = max(s, ctx // 2)
            elif s > 1:
                s = max(1, s // 2)
            else:
                b = max(1, b // 2)
        return dict(op=op, b=b, s=s, h=h, d=d, page=page, ctx=ctx, window=window,
                    first=rng.choice([0, 0, 4, 64, 130]) if window else 0, prev=rng.random() < 0.5,
                    ragged=rng.random() < 0.5)
    common = dict(pairs=pairs, norm=rng.random() < 0.7, factor=rng.choice([1.0, 4.0, 16.0, 40.0]),
                  at=rng.choice(["first", "last"]), ragged=rng.random() < 0.5)
    common["weight"] = common["norm"] and rng.random() < 0.5
    if op == "rotate":
        d = rng.choice([32, 64, 96, 128, 192, 256, 512, 512])
        h = rng.choice([64, 64, 32, 16, 8, 1, 5, 24, 40, 57])
        s = _log(rng, 1, 4096)
        while b * s * h * d > 4096 * 64 * 512:
            s, b = (max(1, s // 2), b) if s > 1 else (s, max(1, b // 2))
        return dict(op=op, b=b, s=s, h=h, d=d, rd=rng.choice([r for r in (16, 32, 64, 128, 512) if r <= d]),
                    inverse=rng.random() < 0.3, far=_log(rng, 100, 1000000), **common)
    d = rng.choice([64, 128, 192, 256, 320, 512, 512])
    s = _log(rng, 1, 8192)
    ctx = max(s, _log(rng, 1, 65536))
    while b * ctx * d > 8 * 8192 * 512:
        if b > 1:
            b //= 2
        else:
            s, ctx = max(1, s // 2), max(1, s // 2, ctx // 2)
    return dict(op=op, b=b, s=s, d=d, rd=rng.choice([r for r in (16, 32, 64, 512) if r <= d]),
                page=rng.choice([1, 8, 16, 24, 64, 64, 100, 256]), ctx=ctx, **common)


# ---------------------------------------------------------------------------------- inputs


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _frequencies(rd, factor):
    """Radians per position of each pair, on the host in 64 bits."""
    out = []
    if factor != 1.0:
        turn = [rd * math.log(ORIG / (beta * 2 * math.pi)) / (2 * math.log(THETA)) for beta in (32.0, 1.0)]
        low, high = max(0, math.floor(turn[0])), min(rd - 1, math.ceil(turn[1]))
    for i in range(rd // 2):
        f = THETA ** (-2 * i / rd)
        if factor != 1.0:
            ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    return out


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    b, s, d = c["b"], c["s"], c["d"]

    def pick(lo, hi):          # one whole number per sequence
        return torch.randint(lo, max(lo, hi) + 1, (b,), generator=host).tolist()

    st = dict(case=c)
    new = pick(0 if s > 1 and b > 1 else 1, s) if c["ragged"] else [s] * b
    st["n_new"] = _ints(new) if c["ragged"] else None
    if c["op"] == "rotate":
        st["start_pos"] = _ints(pick(0, c["far"] - s) if b > 1 or c["ragged"] else [max(0, c["far"] - s)])
        st["x"] = (3 * torch.randn(b, s, c["h"], d, generator=g, device=DEV)).bfloat16()
        st["out"] = torch.zeros_like(st["x"])
    else:
        held = pick(max(s, c["ctx"] // 16), c["ctx"]) if c["ragged"] else [c["ctx"]] * b      # after the step, all real
        st["start_pos"] = _ints([v - s for v in held])
        page = c["page"]
        need = [-(-v // page) for v in held]
        most = -(-c["ctx"] // page)
        n_pages = (b * most if c["op"] == "append" else sum(need)) + 3       # the pool an append returns has one size
        order = torch.randperm(n_pages, generator=host).tolist()
        table = torch.full((b, most), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        st["table"] = table.to(DEV)
        st["pages"] = torch.randn(n_pages, page, d, generator=g, device=DEV, dtype=torch.bfloat16)
        if c["op"] == "append":
            st["x"] = (3 * torch.randn(b, s, d, generator=g, device=DEV)).bfloat16()
    if c["op"] == "attend":
        h = c["h"]
        st["q"] = (2 * torch.randn(b, s, h, d, generator=g, device=DEV)).bfloat16()
        st["sink"] = torch.randn(h, generator=g, device=DEV)
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(b, s, h, device=DEV)
        if c["prev"]:          # what the attention over other rows leaves
            st["prev_out"] = (0.3 * torch.randn(b, s, h, d, generator=g, device=DEV)).bfloat16()
            st["prev_lse"] = 5.5 + torch.randn(b, s, h, generator=g, device=DEV)
        if own:                # the workspace that a serving program keeps
            import sparse_top_attention_indexer_gb300 as sti
            st["ws"] = sti.workspace(sti.attn_paged_workspace_size(b, s, h, d))
    else:
        st["weight"] = (1 + 0.2 * torch.randn(d, generator=g, device=DEV)).bfloat16() if c["weight"] else None
        st["off"] = 0 if c["at"] == "first" else d - c["rd"]
        st["freqs"] = torch.tensor(_frequencies(c["rd"], c["factor"]), dtype=torch.float64, device=DEV)
        if own:                # the table of frequencies that a model keeps
            import sparse_top_attention_indexer_gb300 as sti
            st["turns"] = sti.rope_freqs(c["rd"], THETA, factor=c["factor"], orig_len=ORIG)
    return st


# ---------------------------------------------------------------------------------- plain forms


def _norm_rotate(st, x):
    """x [b, s, h, d] normed and rotated, in fp32 (angles in fp64)."""
    c = st["case"]
    x = x.float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        if c["weight"]:
            x = x * st["weight"].float()
    rd, off = c["rd"], st["off"]
    pos = st["start_pos"][:, None] + torch.arange(c["s"], device=DEV)
    angle = pos[..., None].double() * st["freqs"]                       # [b, s, rd / 2]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    if c.get("inverse"):
        sin = -sin
    r = x[..., off:off + rd]
    u, v = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :rd // 2], r[..., rd // 2:])
    a, e = u * cos - v * sin, v * cos + u * sin
    turned = torch.stack([a, e], -1).flatten(-2) if c["pairs"] else torch.cat([a, e], -1)
    return torch.cat([x[..., :off], turned, x[..., off + rd:]], -1)


def _real(st):
    """Which tokens of the step are real: bool [b, s]."""
    c = st["case"]
    t = torch.arange(c["s"], device=DEV)
    if st["n_new"] is None:
        return torch.ones(c["b"], c["s"], dtype=torch.bool, device=DEV)
    return t < st["n_new"][:, None]


def _rotate(st):
    y = _norm_rotate(st, st["x"]).bfloat16()
    st["out"] = torch.where(_real(st)[..., None, None], y, st["out"])


def _append(st):
    c, page = st["case"], st["case"]["page"]
    y = _norm_rotate(st, st["x"][:, :, None])[:, :, 0].bfloat16()
    pos = (st["start_pos"][:, None] + torch.arange(c["s"], device=DEV)).long()
    real = _real(st)
    row = st["table"].gather(1, pos // page).long() * page + pos % page
    flat = st["pages"].view(-1, c["d"])
    flat[row[real]] = y[real]


def _attend(st):
    c = st["case"]
    b, s, h, d = st["q"].shape
    page, scale = c["page"], d ** -0.5
    pos = torch.arange(c["ctx"], device=DEV)
    for i in range(b):                                                   # one sequence at a time: the scores take GBs
        n = c["ctx"]
        kv = st["pages"][st["table"][i, :-(-n // page)].clamp_min(0).long()].view(-1, d)[:n].float()
        at = st["start_pos"][i] + torch.arange(s, device=DEV)[:, None]
        seen = pos[None] <= at
        if c["window"]:
            seen = seen & ((pos[None] > at - c["window"]) | (pos[None] < c["first"]))
        q = st["q"][i].float().view(s * h, d)
        sc = (q @ kv.T).view(s, h, -1).mul_(scale).masked_fill_(~seen[:, None], -math.inf)
        top = torch.maximum(sc.amax(-1), st["sink"])
        if c["prev"]:
            top = torch.maximum(top, st["prev_lse"][i])
        p = sc.sub_(top[..., None]).exp_()
        den = p.sum(-1) + (st["sink"] - top).exp()
        o = (p.view(s * h, -1) @ kv).view(s, h, d)
        if c["prev"]:
            carry = (st["prev_lse"][i] - top).exp()
            den = den + carry
            o = o + carry[..., None] * st["prev_out"][i].float()
        real = _real(st)[i]
        st["out"][i] = torch.where(real[:, None, None], (o / den[..., None]).bfloat16(), st["out"][i])
        st["lse"][i] = torch.where(real[:, None], top + den.log(), st["lse"][i])


def run(state):
    st, c = state, state["case"]
    if own:
        import sparse_top_attention_indexer_gb300 as sti
    if c["op"] == "rotate":
        if own:
            sti.norm_rope(st["x"], st["start_pos"], st["turns"], rope_off=st["off"], interleaved=c["pairs"],
                          inverse=c["inverse"], norm=c["norm"], weight=st["weight"], eps=EPS, n_new=st["n_new"],
                          out=st["out"])
        else:
            _rotate(st)
        return {"out": st["out"]}
    if c["op"] == "append":
        if own:
            sti.kv_append_paged(st["x"], st["start_pos"], st["pages"], st["table"], st["turns"], rope_off=st["off"],
                                interleaved=c["pairs"], norm=c["norm"], weight=st["weight"], eps=EPS, n_new=st["n_new"])
        else:
            _append(st)
        return {"pages": st["pages"]}
    if own:
        sti.attn_paged(st["q"], st["pages"], st["table"], st["start_pos"], c["d"] ** -0.5, window=c["window"],
                       n_first=c["first"], attn_sink=st["sink"], prev_out=st.get("prev_out"), prev_lse=st.get("prev_lse"),
                       n_new=st["n_new"], out=st["out"], lse=st["lse"], ws=st["ws"])
    else:
        _attend(st)
    return {"out": st["out"], "lse": st["lse"]}


def work(case):
    c = case
    b, s, d = c["b"], c["s"], c["d"]
    real = b * s * (0.5 if c["ragged"] and s > 1 else 1.0)         # tokens (mean over the seeds)
    if c["op"] == "rotate":
        return {"bytes": 4.0 * real * c["h"] * d, "flops": real * c["h"] * (3.0 * d * c["norm"] + 3.0 * c["rd"])}
    if c["op"] == "append":
        return {"bytes": 4.0 * real * d, "flops": real * (3.0 * d * c["norm"] + 3.0 * c["rd"])}
    h, held = c["h"], c["ctx"] * (17 / 32 if c["ragged"] else 1.0)
    t = real / b
    whole = max(held - (s - t / 2), 1.0)                                # rows that a query sees without a window
    per = min(whole, c["window"] + c["first"]) if c["window"] else whole
    rows = min(held, per + t) if c["window"] else max(held - (s - t), 1.0)  # rows that a sequence's queries see together
    out = 2 * real * h * d * (2 if c["prev"] else 1) + 4 * real * h * (2 if c["prev"] else 1)
    return {"bytes": 2.0 * b * rows * d + 2 * real * h * d + out, "flops": 4.0 * h * d * real * per}


# ---------------------------------------------------------------------------------- from the definitions, in 64 bits


def _exact_row(st, x, positions):
    """x [n, h, d] of tokens at `positions` (whole numbers) normed and rotated, as complex numbers in 64 bits."""
    c = st["case"]
    x = x.double()
    if c["norm"]:
        x = x / ((x * x).sum(-1, keepdim=True) / c["d"] + EPS).sqrt()
        if c["weight"]:
            x = x * st["weight"].double()
    rd, off = c["rd"], st["off"]
    first = torch.arange(rd // 2, device=DEV) * 2 if c["pairs"] else torch.arange(rd // 2, device=DEV)
    second = first + (1 if c["pairs"] else rd // 2)
    z = torch.complex(x[..., off + first], x[..., off + second])
    angle = torch.outer(positions.double(), st["freqs"]) * (-1 if c.get("inverse") else 1)
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    x[..., off + first], x[..., off + second] = z.real, z.imag
    return x


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    b, s, d = c["b"], c["s"], c["d"]
    start = st["start_pos"].tolist()
    new = st["n_new"].tolist() if st["n_new"] is not None else [s] * b
    if c["op"] == "rotate":
        out = st["out"].double()
        for i in range(b):
            out[i, :new[i]] = _exact_row(st, st["x"][i, :new[i]], start[i] + torch.arange(new[i], device=DEV))
        return {"out": out}
    page = c["page"]
    table = st["table"].tolist()
    if c["op"] == "append":
        pages = st["pages"].double()
        for i in range(b):
            y = _exact_row(st, st["x"][i, :new[i], None], start[i] + torch.arange(new[i], device=DEV))[:, 0]
            t = 0
            while t < new[i]:                                           # page by page
                p = start[i] + t
                n = min(new[i] - t, page - p % page)
                pages[table[i][p // page], p % page:p % page + n] = y[t:t + n]
                t += n
        return {"pages": pages}
    h = c["h"]
    out, lse = st["out"].double(), st["lse"].double()
    for i in range(b):
        n = start[i] + new[i]
        kv = torch.cat([st["pages"][k] for k in table[i][:-(-n // page)]] or [st["pages"][0, :0]])[:n].double()
        for t0 in range(0, new[i], 64):
            t1 = min(new[i], t0 + 64)
            at = torch.arange(start[i] + t0, start[i] + t1, device=DEV)
            # only the rows that some query of these sees
            lo = max(0, start[i] + t0 - c["window"] + 1) if c["window"] else 0
            rows = torch.cat([torch.arange(min(lo, c["first"]), device=DEV), torch.arange(lo, start[i] + t1, device=DEV)])
            x = torch.einsum("thd,nd->thn", st["q"][i, t0:t1].double(), kv[rows]) / math.sqrt(d)
            hidden = rows[None] > at[:, None]
            if c["window"]:
                hidden |= (at[:, None] - rows[None] >= c["window"]) & (rows[None] >= c["first"])
            x = x.masked_fill(hidden[:, None], -math.inf)
            parts = [torch.logsumexp(x, -1), st["sink"].double().expand(t1 - t0, h)]
            if c["prev"]:
                parts.append(st["prev_lse"][i, t0:t1].double())
            total = torch.logsumexp(torch.stack(parts), 0)
            o = torch.einsum("thn,nd->thd", (x - total[..., None]).exp(), kv[rows])
            if c["prev"]:
                o += (parts[2] - total).exp()[..., None] * st["prev_out"][i, t0:t1].double()
            out[i, t0:t1], lse[i, t0:t1] = o, total
    return {"out": out, "lse": lse}
