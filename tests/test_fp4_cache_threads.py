"""The bounded 4-bit cache called from two host threads at once, each on a stream of its own."""
import threading

import pytest

from tests.test_fp4_cache import sti  # noqa: F401  (the fixture)

gpu = pytest.mark.gpu


def both(jobs):
    """Run the jobs in threads of their own, started together; the errors they raised."""
    go, errors = threading.Barrier(len(jobs)), []

    def body(job):
        go.wait()
        try:
            job()
        except Exception as e:  # noqa: BLE001  (reported by the test)
            errors.append(e)

    threads = [threading.Thread(target=body, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def evict_job(sti, b, rows, budget, repeats):  # noqa: F811
    """A cache of the size, and a job that evicts from it and then finds it within its budget again and again.  The C
    entry is called with ready arguments: next to it nothing takes time, so the two threads' calls overlap."""
    import ctypes

    import torch

    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = torch.rand(b, rows, generator=gen, device="cuda")
    pos = torch.arange(rows, device="cuda", dtype=torch.int32).repeat(b, 1)
    start = torch.full((b,), rows - 1, device="cuda", dtype=torch.int32)
    dropped = torch.zeros(b, device="cuda", dtype=torch.int32)
    ws = sti.workspace(sti.kv_evict_workspace_size(b, rows, budget))
    stream = torch.cuda.Stream()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    args = (ptr(w), rows, ptr(pos), rows, ptr(start), ptr(dropped), b, 1, 1, rows, budget, 2, 4, None, 0, ptr(ws),
            ws.numel(), ctypes.c_void_p(stream.cuda_stream))

    def job():
        call = sti.lib().sti_kv_evict
        bad = sum(call(*args) != 0 for _ in range(repeats))
        stream.synchronize()
        if bad:
            raise RuntimeError(f"{bad} of {repeats} calls failed")

    return (w, pos, dropped, start, ws, stream), job


@gpu
@pytest.mark.parametrize("sizes", [((150, 9000), (150, 200)),        # single CTAs
                                   ((1, 60000), (1, 16000))])        # clusters of eight
def test_evict_caches_of_different_sizes(sti, sizes):  # noqa: F811
    """Neither thread's call fails because the other's asks for another amount of shared memory (it did in 1 to 8 % of
    the larger cache's calls when each call set its own amount as the kernel's limit)."""
    import torch

    alone = [evict_job(sti, b, rows, rows - 10, 1) for b, rows in sizes]
    torch.cuda.synchronize()
    for _, job in alone:
        job()
    pairs = [evict_job(sti, b, rows, rows - 10, 10000) for b, rows in sizes]
    torch.cuda.synchronize()
    errors = both([job for _, job in pairs])
    assert not errors, errors
    for (want, _), (got, _) in zip(alone, pairs):
        for x, y in zip(want[:3], got[:3]):
            assert (x == y).all()


@gpu
def test_steps_of_two_layers(sti):  # noqa: F811
    """Two threads, each with its cache: append, attend with row weights, evict, as the same steps alone leave it."""
    import torch

    def layer(b, h, d, budget, steps, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rows = budget + 1
        st = dict(codes=torch.randint(0, 256, (b, rows, d // 2), generator=gen, device="cuda", dtype=torch.uint8),
                  scales=torch.randint(40, 60, (b, rows, d // 16), generator=gen, device="cuda", dtype=torch.uint8),
                  pos=torch.arange(rows, device="cuda", dtype=torch.int32).repeat(b, 1),
                  weight=torch.rand(b, rows, generator=gen, device="cuda"),
                  start=torch.full((b,), budget, device="cuda", dtype=torch.int32),
                  dropped=torch.zeros(b, device="cuda", dtype=torch.int32))
        xs = torch.randn(steps, b, 1, d, generator=gen, device="cuda").bfloat16()
        qs = torch.randn(steps, b, 1, h, d, generator=gen, device="cuda").bfloat16()
        stream = torch.cuda.Stream()

        def job():
            outs = []
            with torch.cuda.stream(stream):
                for x, q in zip(xs, qs):
                    sti.kv_append_fp4(x, st["start"], 1, 1, st["codes"], st["scales"], dropped=st["dropped"],
                                      row_pos=st["pos"], row_weight=st["weight"])
                    outs.append(sti.attn_fp4kv(q, st["codes"], st["scales"], st["start"], 1, d ** -0.5,
                                               dropped=st["dropped"], row_weight=st["weight"]))
                    sti.kv_evict(st["weight"], st["pos"], st["start"], 1, 1, st["dropped"], budget, 4, 8,
                                 [st["codes"], st["scales"]])
                    st["start"] += 1
                st["out"] = torch.stack(outs)
            stream.synchronize()

        return st, job

    kinds = [(3, 64, 512, 3000, 40, 1), (5, 8, 128, 200, 40, 2)]
    alone = [layer(*k) for k in kinds]
    torch.cuda.synchronize()
    for _, job in alone:
        job()
    together = [layer(*k) for k in kinds]
    torch.cuda.synchronize()
    errors = both([job for _, job in together])
    assert not errors, errors
    for (want, _), (got, _) in zip(alone, together):
        for k in want:
            assert (want[k] == got[k]).all(), k
