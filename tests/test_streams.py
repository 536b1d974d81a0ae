"""Outputs that a call makes itself when it runs on another stream than the current one: their memory is neither in use
by earlier work on the current stream, nor given away before later work there has read it."""
import pytest
import torch

DEV = "cuda:0"


@pytest.fixture(scope="module")
def mkv():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    if not os.path.exists(os.path.join(root, "mixed_format_paged_gb300", "libmkv.so")):
        from mixed_format_paged_gb300 import build as b
        b.build()
    import mixed_format_paged_gb300 as m
    return m


def test_outputs_are_made_as_asked_without_a_device(mkv):
    from mixed_format_paged_gb300.rope import outputs
    a, b = outputs(5, torch.device("cpu"), lambda: torch.zeros(3), lambda: torch.ones(2))
    assert a.shape == (3,) and b.shape == (2,)
    assert outputs(None, torch.device("cpu"), lambda: 7) == [7]


def _calls(mkv):
    """name -> call(i, stream) -> outputs; i chooses one of two inputs."""
    g = torch.Generator().manual_seed(0)
    r = lambda *s: [torch.randn(*s, generator=g).to(DEV) for _ in range(2)]  # noqa: E731
    rope = mkv.Rope(128)
    q, k, pos = r(4000, 24, 256), r(4000, 4, 256), torch.arange(4000, device=DEV)
    pool = mkv.MkvPool(1, 24, 4, 256, 64, 40, 4, max_seqs=2, max_pages_per_seq=20, device=DEV)
    pool.extend([0, 1], [700, 300])
    pk, pv, pq, dq = r(1000, 4, 256), r(1000, 4, 256), r(1000, 24, 256), r(2, 24, 256)
    pool.append(0, [0, 1], [700, 300], pk[0], pv[0])
    b8 = mkv.Blk8Cache(1, 8, 2, 128, 64, 20, 2, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    lens, table = i32([600, 100]), torch.arange(20, dtype=torch.int32).reshape(2, 10).to(DEV)
    bk, bq = r(700, 2, 128), [x.bfloat16() for x in r(2, 1, 8, 128)]
    b8.append(0, bk[0], bk[1], i32([0, 600, 700]), lens, table)
    _, lse = pool.decode(0, [0, 1], dq[0])
    torch.cuda.synchronize()
    return {
        "rope": lambda i, s: rope(q[i], k[i], pos, stream=s),
        "append_rope": lambda i, s: (pool.append_rope(0, [0, 1], [700, 300], pq[i], pk[0], pv[0], rope, stream=s),),
        "attention": lambda i, s: b8.attention(0, bq[i], lens, table, stream=s),
        "decode": lambda i, s: pool.decode(0, [0, 1], dq[i], stream=s),
        "relevance": lambda i, s: (pool.relevance(0, [0, 1], dq[i], lse, stream=s),),
        "dequantize": lambda i, s: pool.dequantize(0, i, 0, 2, stream=s),
    }


SLEEP = 100_000_000      # cycles: some 50 ms


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", ["rope", "append_rope", "attention", "decode", "relevance", "dequantize"])
def test_outputs_on_another_stream_disturb_nothing_and_last(mkv, name, handle):
    call = _calls(mkv)[name]
    want = [[x.clone() for x in call(i, None)] for i in range(2)]
    side = torch.cuda.Stream()
    s = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    # tensors of the outputs' sizes, freed while the current stream has yet to read them
    mine = [torch.full_like(x, 3.0) for x in want[0]]
    copies = [torch.empty_like(x) for x in want[0]]
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    for c, x in zip(copies, mine):
        c.copy_(x)
    del mine, x
    got = call(0, s)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    torch.cuda.synchronize()
    assert all((c == 3.0).all() for c in copies)
    # outputs freed while the current stream has yet to read them, and another call at once
    got = call(0, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(SLEEP)
    for c, x in zip(copies, got):
        c.copy_(x)
    del got, x
    again = call(1, s)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, want[1]))
    torch.cuda.synchronize()
    assert all(torch.equal(c, w) for c, w in zip(copies, want[0]))
    # the default stream's handle, with another one current
    with torch.cuda.stream(side):
        got = call(1, 0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
