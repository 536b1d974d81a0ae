"""Forking, truncating and copying sequences of the pool: bookkeeping and refusals on the CPU (host-only pools), page
contents on the GPU."""
import numpy as np
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


def _host(mkv, **kw):
    a = dict(num_layers=2, num_q_heads=24, num_kv_heads=4, head_dim=256, page_size=64, fp8_slots=12, tq3_slots=6,
             max_seqs=6, max_pages_per_seq=16, rotation_seed=9)
    a.update(kw)
    return mkv.MkvPool(host_only=True, **a)


def _refused(mkv, status, fn, *args):
    with pytest.raises(mkv.MkvError) as e:
        fn(*args)
    assert e.value.status == status, e.value


def _slots(p, r):
    return [p.page_info(r, i) for i in range(p.seq_info(r)[1])]


# ------------------------------------------------------------------ CPU
def test_fork_shares_full_pages_and_copies_the_tail(mkv):
    p = _host(mkv)
    p.extend([0], [64 * 3 + 5])
    p.set_tier(0, 0, 2)
    p.demote([0], [1])
    p.fork([0, 0], [1, 2])
    a, b, c = (_slots(p, r) for r in range(3))
    assert a[:3] == b[:3] == c[:3] and [t for t, _ in b] == [2, 3, 1, 1]
    assert len({a[3], b[3], c[3]}) == 3
    st = p.stats()
    assert st.fp8_slots_free == 12 - 5 and st.tq3_slots_free == 5
    assert st.fp8_bytes == 2 * 5 * 132096 and st.tq3_bytes == 2 * 50176      # shared pages count once
    assert (st.recent_pages, st.anchor_pages, st.stale_pages) == (6, 3, 3)   # logical pages
    p.release(0)
    assert p.stats().fp8_slots_free == 12 - 4 and p.stats().tq3_slots_free == 5
    p.release(2)
    p.release(1)
    assert p.stats().fp8_slots_free == 12 and p.stats().tq3_slots_free == 6


def test_forks_demote_and_extend_apart(mkv):
    p = _host(mkv)
    p.extend([0], [64 * 2])                              # no partial page: nothing is copied
    p.fork([0], [1])
    assert _slots(p, 0) == _slots(p, 1) and p.stats().fp8_slots_free == 10
    p.extend([0, 1], [1, 1])
    assert _slots(p, 0)[2] != _slots(p, 1)[2]
    p.demote([0], [0])
    assert _slots(p, 0)[0][0] == 3 and _slots(p, 1)[0][0] == 1
    p.demote([1], [0])                                   # the last sequence to let go frees the FP8 slot
    assert p.stats().fp8_slots_free == 12 - 1 - 2 and p.stats().tq3_slots_free == 4
    p.fork([1], [2])                                     # a TQ3 page is shared too
    assert _slots(p, 2)[0] == _slots(p, 1)[0] and p.stats().tq3_slots_free == 4


def test_fork_refusals_leave_everything_unchanged(mkv):
    p = _host(mkv, fp8_slots=4)
    p.extend([0, 1], [64 + 3, 64 + 3])
    before = _slots(p, 0), p.stats().fp8_slots_free
    _refused(mkv, 1, p.fork, [0], [9])
    _refused(mkv, 1, p.fork, [-1], [2])
    _refused(mkv, 1, p.fork, [0], [1])                   # not empty
    _refused(mkv, 1, p.fork, [3], [3])
    _refused(mkv, 1, p.fork, [0, 0], [2, 2])
    _refused(mkv, 1, p.fork, [2, 0], [3, 2])             # 2 is both
    _refused(mkv, 3, p.fork, [0], [2])                   # no slot for the tail
    assert (_slots(p, 0), p.stats().fp8_slots_free) == before and p.seq_info(2) == (0, 0)
    p.fork([4], [5])                                     # an empty source gives an empty sequence
    p.fork([], [])
    with pytest.raises(ValueError):
        p.fork([0], [])


def test_truncate_frees_pages_and_unshares_a_cut_page(mkv):
    p = _host(mkv)
    p.extend([0], [64 * 4 + 9])
    p.fork([0], [1])
    free = p.stats().fp8_slots_free
    p.truncate([1], [64 * 2 + 7])                        # page 2 was shared and becomes partial: a copy of its own
    assert p.seq_info(1) == (135, 3) and _slots(p, 1)[:2] == _slots(p, 0)[:2] and _slots(p, 1)[2] != _slots(p, 0)[2]
    assert p.stats().fp8_slots_free == free - 1 + 1      # its own tail went, a copy came
    p.truncate([1], [64])
    assert _slots(p, 1) == _slots(p, 0)[:1]
    p.truncate([1, 0], [0, 64 * 4 + 1])
    assert p.seq_info(1) == (0, 0) and p.seq_info(0) == (257, 5)
    p.truncate([0], [257])
    assert p.stats().fp8_slots_free == 12 - 5


def test_truncating_both_owners_of_a_shared_page(mkv):
    p = _host(mkv)
    p.extend([0], [64 * 2])
    p.fork([0], [1])
    p.truncate([0, 1], [70, 80])
    assert _slots(p, 0)[0] == _slots(p, 1)[0] and _slots(p, 0)[1] != _slots(p, 1)[1]
    p.release(0)
    p.release(1)
    assert p.stats().fp8_slots_free == 12


def test_truncate_refusals(mkv):
    p = _host(mkv, fp8_slots=3)
    p.extend([0], [64 * 3])
    _refused(mkv, 1, p.truncate, [0], [193])
    _refused(mkv, 1, p.truncate, [0], [-1])
    _refused(mkv, 1, p.truncate, [7], [0])
    _refused(mkv, 1, p.truncate, [0, 0], [1, 1])
    p.demote([0], [1])
    _refused(mkv, 4, p.truncate, [0], [100])             # inside a TQ3 page
    p.truncate([0], [128])                               # at its end
    p.extend([0], [64])
    p.fork([0], [1])
    p.extend([1], [64])
    _refused(mkv, 3, p.truncate, [0], [150])             # shared, and no slot is free
    assert p.seq_info(0) == (192, 3)


def test_shared_pages_are_not_written(mkv):
    p = _host(mkv)
    p.extend([0], [64])
    p.fork([0], [1])                                     # before the page was appended
    B = mkv.binding
    rope = mkv.Rope(2).table
    for r in (0, 1):
        _refused(mkv, 4, B.mkv_append_tokens, p.handle, 0, [r], [64], 0x1000, 0x1000, 0)
        _refused(mkv, 4, B.mkv_append_rope, p.handle, 0, [r], [1], rope, None, None, 0x1000, 0x1000, 0)
        _refused(mkv, 4, B.mkv_append_decode, p.handle, 0, [r], 0x1000, 0x1000, 0, 0x1000, 0, 0x1000, 0x1000)
    p.extend([0], [1])
    B.mkv_append_tokens(p.handle, 0, [0], [1], 0x1000, 0x1000, 0)
    p.release(1)
    B.mkv_append_tokens(p.handle, 0, [0], [65], 0x1000, 0x1000, 0)


def test_copy_between_pools_keeps_tiers_and_sharing(mkv):
    a, b = _host(mkv), _host(mkv, fp8_slots=5, tq3_slots=1, max_seqs=3)
    a.extend([0], [64 * 3 + 1])
    a.set_tier(0, 2, 2)
    a.demote([0], [0])
    a.fork([0], [3])
    a.extend([3], [1])
    b.copy_from(a, [0, 3], [2, 0])
    x, y = _slots(b, 2), _slots(b, 0)
    assert [t for t, _ in x] == [3, 1, 2, 1] and x[:3] == y[:3] and x[3] != y[3]
    assert [s for _, s in x] == [0, 0, 1, 2] and y[3][1] == 3
    assert b.seq_info(2) == (193, 4) and b.seq_info(0) == (194, 4)
    assert b.stats().fp8_slots_free == 1 and b.stats().tq3_slots_free == 0
    b.release(2)
    b.release(0)
    assert b.stats().fp8_slots_free == 5 and b.stats().tq3_slots_free == 1
    a.copy_from(a, [0], [5])                             # within a pool: pages of its own
    assert not set(_slots(a, 5)) & set(_slots(a, 0))


def test_copy_refusals(mkv):
    a, b = _host(mkv), _host(mkv, fp8_slots=2, max_seqs=2, max_pages_per_seq=3)
    a.extend([0, 1], [64 * 3, 64 * 4])
    _refused(mkv, 3, b.copy_from, a, [0], [0])
    _refused(mkv, 1, b.copy_from, a, [1], [0])           # longer than the destination allows
    _refused(mkv, 1, b.copy_from, a, [0], [2])
    _refused(mkv, 1, b.copy_from, a, [9], [0])
    _refused(mkv, 1, b.copy_from, a, [0, 0], [1, 1])
    _refused(mkv, 1, a.copy_from, a, [0], [0])
    _refused(mkv, 1, a.copy_from, a, [0], [1])
    for kw in (dict(rotation_seed=1), dict(num_layers=1), dict(page_size=128), dict(num_kv_heads=6)):
        _refused(mkv, 1, _host(mkv, **kw).copy_from, a, [0], [0])
    assert b.seq_info(0) == (0, 0) and b.stats().fp8_slots_free == 2


def test_random_forks_truncations_and_copies_keep_the_slots_balanced(mkv):
    rng = np.random.default_rng(4)
    p, q = (_host(mkv, fp8_slots=60, tq3_slots=30, max_seqs=8) for _ in range(2))
    for _ in range(600):
        pool, other = (p, q) if rng.random() < 0.5 else (q, p)
        r, t = (int(x) for x in rng.integers(0, 8, 2))
        op = rng.integers(0, 6)
        try:
            if op == 0:
                pool.extend([r], [int(rng.integers(0, 200))])
            elif op == 1:
                pool.fork([r], [t])
            elif op == 2:
                pool.truncate([r], [int(rng.integers(0, pool.seq_info(r)[0] + 1))])
            elif op == 3:
                pool.copy_from(other, [r], [t])
            elif op == 4:
                pool.release(r)
            else:
                pool.demote([r], [int(rng.integers(0, 4))])
        except mkv.MkvError:
            pass
        for x in (p, q):
            used = [{s for i in range(8) for tier, s in _slots(x, i) if (tier == 3) == f} for f in (False, True)]
            st = x.stats()
            assert len(used[0]) == 60 - st.fp8_slots_free and len(used[1]) == 30 - st.tq3_slots_free
            owners = {}
            for i in range(8):                           # a page that is not full has one owner
                n, npg = x.seq_info(i)
                if n % 64:
                    tier, s = x.page_info(i, npg - 1)
                    assert tier != 3
                    owners.setdefault(s, []).append(i)
            for s, who in owners.items():
                assert sum(s in [b for t, b in _slots(x, i) if t != 3] for i in range(8)) == 1 == len(who)


# ------------------------------------------------------------------ GPU
def _fill(mkv, P=64, layers=3, fp8=40, tq3=20, seqs=8, lens=(5 * 64 + 17, 130), seed=2):
    g = torch.Generator().manual_seed(seed)
    pool = mkv.MkvPool(layers, 24, 4, 256, P, fp8, tq3, max_seqs=seqs, max_pages_per_seq=16, rotation_seed=5, device=DEV)
    for r, n in enumerate(lens):
        pool.extend([r], [n])
        for layer in range(layers):
            k, v = (torch.randn(n, 4, 256, generator=g).to(DEV) for _ in range(2))
            pool.append(layer, [r], [n], k, v)
    return pool, g


def _pages(pool, layer, r):
    return [pool.export_page(layer, r, i) for i in range(pool.seq_info(r)[1])]


def _dense(pool, layer, r):
    n = pool.seq_info(r)[0]
    return [x[:n].clone() for x in pool.dequantize(layer, r, 0, pool.seq_info(r)[1])]


@pytest.mark.gpu
@pytest.mark.parametrize("P", [64, 128])
def test_forks_hold_the_parents_values_and_go_on_alone(mkv, P):
    pool, g = _fill(mkv, P, lens=(5 * P + 17, P + 1, 2 * P))
    pool.demote([0, 0], [1, 2])
    want = {(l, r): _dense(pool, l, r) for l in range(3) for r in range(3)}
    q = torch.randn(3, 24, 256, generator=g).to(DEV)
    o, lse = pool.decode(1, [0, 1, 2], q)
    pool.fork([0, 1, 2, 0], [4, 5, 6, 7])
    o2, lse2 = pool.decode(1, [4, 5, 6], q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # the children extend, the first child's page 3 goes to TQ3: parents keep every bit
    pool.extend([4, 5, 6], [3, 200, 1])
    for layer in range(3):
        k, v = (torch.randn(204, 4, 256, generator=g).to(DEV) for _ in range(2))
        pool.append(layer, [4, 5, 6], [3, 200, 1], k, v)
    pool.demote([4], [3])
    for (layer, r), kv in want.items():
        for x, y in zip(kv, _dense(pool, layer, r)):
            assert torch.equal(x, y)
        n = kv[0].shape[0]
        m = n if r else 3 * P                            # the child's page 3 changed its format
        for x, y in zip(kv, _dense(pool, layer, 4 + r)):
            assert torch.equal(x[:m], y[:m])
        for x, y in zip(want[layer, 0], _dense(pool, layer, 7)):
            assert torch.equal(x, y)
    for r in (0, 4, 5):
        pool.release(r)
    for x, y in zip(want[2, 0], _dense(pool, 2, 7)):     # still referred to by 7
        assert torch.equal(x, y)
    pool.check_device_errors()


@pytest.mark.gpu
@pytest.mark.parametrize("tail", [1, 2, 7, 63])
def test_tail_copy_moves_the_rows_of_its_tokens_only(mkv, tail):
    pool, g = _fill(mkv, lens=(64 + tail,))
    pool.extend([3], [64])                               # a slot with other contents, freed again, becomes the child's
    other = torch.randn(64, 4, 256, generator=g).to(DEV)
    for layer in range(3):
        pool.append(layer, [3], [64], other, other)
    old = [pool.export_page(layer, 3, 0)[0] for layer in range(3)]
    slot = pool.page_info(3, 0)[1]
    pool.release(3)
    pool.fork([0], [1])
    assert pool.page_info(1, 1)[1] == slot
    for layer in range(3):
        a = np.frombuffer(pool.export_page(layer, 0, 1)[0], np.uint8).reshape(4, 2, -1)
        b = np.frombuffer(pool.export_page(layer, 1, 1)[0], np.uint8).reshape(4, 2, -1)
        c = np.frombuffer(old[layer], np.uint8).reshape(4, 2, -1)
        for kv, rows in ((0, tail), (1, tail + tail % 2)):
            at = rows * 256
            assert (a[:, kv, :at] == b[:, kv, :at]).all() and (b[:, kv, at:64 * 256] == c[:, kv, at:64 * 256]).all()
            s = 64 * 256 + 2 * tail
            assert (a[:, kv, 64 * 256:s] == b[:, kv, 64 * 256:s]).all() and (b[:, kv, s:] == c[:, kv, s:]).all()


@pytest.mark.gpu
def test_truncate_rolls_speculative_tokens_back(mkv):
    pool, g = _fill(mkv, lens=(64 * 3 + 60, 64 * 3))
    before = [_dense(pool, l, 0) for l in range(3)]
    pool.fork([0], [2])
    pool.extend([0], [8])                                # runs into a new page
    for layer in range(3):
        x = torch.randn(8, 4, 256, generator=g).to(DEV)
        pool.append(layer, [0], [8], x, x)
    pool.truncate([0], [64 * 3 + 60])
    pool.truncate([2], [64 + 5])                         # a shared page is cut: its rows come along
    for layer in range(3):
        for x, y, z in zip(before[layer], _dense(pool, layer, 0), _dense(pool, layer, 2)):
            assert torch.equal(x, y) and torch.equal(x[:64 + 5], z)
    pool.extend([2], [1])
    x = torch.randn(1, 4, 256, generator=g).to(DEV)
    pool.append(0, [2], [1], x, x)
    assert torch.equal(before[0][0], _dense(pool, 0, 0)[0])


@pytest.mark.gpu
def test_step_graph_goes_on_after_a_fork_and_a_truncation(mkv):
    pool, g = _fill(mkv, lens=(200, 64 * 4), seqs=6)
    q, k, v = ([torch.randn(2, h, 256, generator=g).to(DEV) for _ in range(3)] for h in (24, 4, 4))
    out, lse = [torch.zeros(2, 24, 256, device=DEV) for _ in range(3)], [torch.zeros(2, 24, device=DEV) for _ in range(3)]
    pool.extend([0, 1], [1, 1])
    graph = pool.step_graph([0, 1], q, out, lse, k, v)
    graph.launch()
    pool.fork([0, 1], [4, 5])
    first = [x.clone() for x in out]
    pool.truncate([0, 1], [200, 256])                    # the step again, from the same state
    pool.extend([0, 1], [1, 1])
    graph.launch()
    for x, y in zip(first, out):
        assert torch.equal(x, y)
    o, _ = pool.decode(2, [4, 5], q[2])
    assert torch.equal(o, first[2])


@pytest.mark.gpu
@pytest.mark.parametrize("P", [64, 128])
def test_copy_moves_every_page_of_every_layer(mkv, P):
    a, g = _fill(mkv, P, lens=(6 * P + 3, P - 1, 2 * P))
    a.set_tier(0, 0, 2)
    a.demote([0, 0, 2], [1, 3, 0])
    a.fork([0], [5])
    b = mkv.MkvPool(3, 24, 4, 256, P, 12, 5, max_seqs=8, max_pages_per_seq=16, rotation_seed=5, device=DEV)
    b.extend([7], [1])                                   # the destination is not empty
    b.copy_from(a, [0, 1, 2, 5], [1, 2, 3, 4])
    for layer in range(3):
        for r, s in ((0, 1), (1, 2), (2, 3), (5, 4)):
            for x, y in zip(_pages(a, layer, r), _pages(b, layer, s)):
                assert x[1:] == y[1:]
                full = x[2] == P or x[1] == 3
                assert x[0] == y[0] if full else True
            for x, y in zip(_dense(a, layer, r), _dense(b, layer, s)):
                assert torch.equal(x, y)
    q = torch.randn(4, 24, 256, generator=g).to(DEV)
    assert torch.equal(a.decode(0, [0, 1, 2, 5], q)[0], b.decode(0, [1, 2, 3, 4], q)[0])


@pytest.mark.gpu
def test_more_copies_than_one_launch_takes(mkv):
    n = 1030                                             # 1,024 page copies travel with one launch
    pool = mkv.MkvPool(1, 8, 1, 256, 64, n + 4, 1, max_seqs=n + 2, max_pages_per_seq=2, device=DEV)
    pool.extend([0], [3])
    x = torch.randn(3, 1, 256, device=DEV)
    pool.append(0, [0], [3], x, x)
    pool.fork([0] * n, list(range(1, n + 1)))
    want = pool.dequantize(0, 0, 0, 1)[1][:3]
    for r in (1, 2, 511, 1023, 1024, 1025, n):
        assert torch.equal(pool.dequantize(0, r, 0, 1)[1][:3], want)


@pytest.mark.gpu
def test_calls_that_the_host_plans_refuse_a_capture(mkv):
    """A replay would write where the pages were: the calls refuse, and pool and capture go on."""
    pool, g = _fill(mkv)
    other, _ = _fill(mkv)
    rope = mkv.Rope(64)
    want = [_dense(pool, 0, r) for r in range(2)]
    pool.extend([1], [1])
    k, v = (torch.randn(1, 4, 256, generator=g).to(DEV) for _ in range(2))
    q = torch.randn(1, 24, 256, generator=g).to(DEV)
    a = torch.zeros(4, device=DEV)
    pool.append_rope(0, [1], [1], q, k, v, rope)         # (destinations uploaded: a cached call is refused as well)
    torch.cuda.synchronize()
    before = [pool.seq_info(r) for r in range(8)], pool.stats().fp8_slots_free
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a += 1
        for call in (lambda: pool.append_rope(0, [1], [1], None, k, v, rope), lambda: pool.fork([0], [5]),
                     lambda: pool.truncate([0], [17]), lambda: other.copy_from(pool, [0], [5])):
            with pytest.raises(mkv.MkvError) as e:
                call()
            assert e.value.status == 4
    graph.replay()
    torch.cuda.synchronize()
    assert (a == 1).all()
    assert before == ([pool.seq_info(r) for r in range(8)], pool.stats().fp8_slots_free)
    pool.fork([0], [5])
    pool.truncate([1], [130])
    for r in range(2):
        assert all(torch.equal(x, y) for x, y in zip(want[r], _dense(pool, 0, r)))


# ------------------------------------------------------------------ several owners of shared pages in one truncation
def _cut_rows(mkv, pool, ids, lens):
    """Truncate and check the page records: full pages stay where they were, and a page that was shared and became
    partial lies in a slot that was free before the call, one that nobody else has."""
    n = pool.cfg.max_seqs
    before = {i: _slots(pool, i) for i in range(n)}
    P = pool.cfg.page_size
    in_use = {s for i in range(n) for t, s in before[i] if t != 3}
    owners = {s: sum(s == b for i in range(n) for t, b in before[i] if t != 3) for s in in_use}
    pool.truncate(ids, lens)
    for i in range(n):
        after = _slots(pool, i)
        if i not in ids:
            assert after == before[i]
            continue
        m = lens[ids.index(i)]
        assert after[:m // P] == before[i][:m // P] and len(after) == -(-m // P)
        if m % P:
            was, now = before[i][m // P][1], after[m // P][1]
            if owners[was] > 1:
                assert now not in in_use, f"sequence {i}: slot {now} held another page when its rows were copied"
            else:
                assert now == was
    used = [s for i in range(n) for t, s in _slots(pool, i) if t != 3]
    assert len(set(used)) == pool.cfg.fp8_slots - pool.stats().fp8_slots_free
    tails = [_slots(pool, i)[-1][1] for i in range(n) if pool.seq_info(i)[0] % P]
    assert all(used.count(s) == 1 for s in tails)


@pytest.mark.parametrize("order", [[0, 1, 2], [0, 2, 1], [1, 0, 3, 2], [0, 1, 2, 3], [3, 2, 1, 0]])
def test_truncating_all_owners_of_several_shared_pages(mkv, order):
    p = _host(mkv)
    p.extend([0, 2], [128, 128])
    p.fork([0, 2], [1, 3])
    _cut_rows(mkv, p, order, [69] * len(order))
    for i in range(4):
        p.release(i)
    assert p.stats().fp8_slots_free == 12


def test_random_truncations_of_several_sequences_a_call(mkv):
    rng = np.random.default_rng(11)
    cut = 0
    for _ in range(60):
        p = _host(mkv, fp8_slots=60, max_seqs=12)
        roots = [int(x) for x in rng.permutation(12)[:3]]
        p.extend(roots, [int(x) for x in rng.integers(1, 64 * 5, 3)])
        for i in range(12):
            if i not in roots and rng.random() < 0.8:
                p.fork([roots[int(rng.integers(0, 3))]], [i])
        for _ in range(4):
            ids = [int(x) for x in rng.permutation(12)[:int(rng.integers(1, 13))]]
            lens = [int(rng.integers(0, p.seq_info(i)[0] + 1)) for i in ids]
            try:
                _cut_rows(mkv, p, ids, lens)
            except mkv.MkvError as e:
                assert e.status == 3
                continue
            cut += 1
    assert cut > 100


@pytest.mark.gpu
@pytest.mark.parametrize("order", [[0, 1, 2, 3, 4, 5], [1, 0, 3, 2, 5, 4], [0, 2, 4, 1, 3, 5]])
def test_truncated_owners_of_several_shared_pages_hold_their_own_rows(mkv, order):
    pool, _ = _fill(mkv, lens=(3 * 64, 2 * 64, 2 * 64 + 9))
    want = {(l, r): _dense(pool, l, r) for l in range(3) for r in range(3)}
    pool.fork([0, 1, 2], [3, 4, 5])
    lens = [64 + 7 + 3 * r for r in range(6)]
    pool.truncate([(i % 3) + 3 * (i // 3) for i in order], [lens[i] for i in order])
    for layer in range(3):
        for r in range(6):
            for a, b in zip(_dense(pool, layer, r), want[layer, r % 3]):
                assert torch.equal(a, b[:lens[r]]), (layer, r)


@pytest.mark.gpu
def test_random_forks_and_batched_truncations_keep_every_sequences_rows(mkv):
    """A model of the contents: each sequence's rows are a prefix of its ancestor's followed by rows of its own."""
    rng = np.random.default_rng(5)
    pool, g = _fill(mkv, layers=2, fp8=64, lens=(200, 150, 128), seqs=8)
    rows = {r: [_dense(pool, layer, r) for layer in range(2)] for r in range(3)}
    for step in range(40):
        live = [r for r in range(8) if pool.seq_info(r)[0]]
        empty = [r for r in range(8) if not pool.seq_info(r)[0]]
        op = int(rng.integers(0, 4))
        if op == 0 and live and empty:
            src = [live[int(rng.integers(0, len(live)))] for _ in empty]
            pool.fork(src, empty)
            for s, d in zip(src, empty):
                rows[d] = [list(x) for x in rows[s]]
        elif op == 1 and live:
            ids = [int(x) for x in rng.permutation(live)[:4]]
            add = [int(x) for x in rng.integers(1, 40, len(ids))]
            if any(pool.seq_info(i)[0] + n > 64 * 8 for i, n in zip(ids, add)):
                continue
            pool.extend(ids, add)
            for layer in range(2):
                k, v = (torch.randn(sum(add), 4, 256, generator=g).to(DEV) for _ in range(2))
                pool.append(layer, ids, add, k, v)
                for i, n in zip(ids, add):
                    new = _dense(pool, layer, i)
                    for old, x in zip(rows[i][layer], new):
                        assert torch.equal(x[:old.shape[0]], old), (step, layer, i)
                    rows[i][layer] = new
        elif live:
            ids = [int(x) for x in rng.permutation(live)]
            lens = [int(rng.integers(1, pool.seq_info(i)[0] + 1)) for i in ids]
            pool.truncate(ids, lens)
            for i, n in zip(ids, lens):
                rows[i] = [[x[:n] for x in kv] for kv in rows[i]]
        for r in range(8):
            if pool.seq_info(r)[0]:
                for layer in range(2):
                    for a, b in zip(_dense(pool, layer, r), rows[r][layer]):
                        assert torch.equal(a, b), (step, layer, r)


# ------------------------------------------------------------------ ids and counts as one-shot iterators
def test_iterators_and_arrays_name_the_same_batches_as_lists(mkv):
    forms = [list, tuple, iter, lambda x: (i for i in x), lambda x: map(int, x), np.array, torch.tensor]
    for form in forms:
        p = _host(mkv)
        p.extend(form([0, 1]), form([70, 64]))
        assert p.seq_info(0) == (70, 2) and p.seq_info(1) == (64, 1), form
        p.fork(form([0, 0]), form([2, 3]))
        assert p.seq_info(3) == (70, 2)
        p.truncate(form([2, 3]), form([3, 65]))
        assert p.seq_info(2) == (3, 1) and p.seq_info(3) == (65, 2)
        q = _host(mkv)
        q.copy_from(p, form([3]), form([5]))
        assert q.seq_info(5) == (65, 2)
        p.demote(form([0]), form([0]))
        assert p.page_info(0, 0)[0] == 3


@pytest.mark.gpu
def test_appends_of_iterators_write_what_lists_write(mkv):
    from mixed_format_paged_gb300 import Rope
    rope, got = Rope(128), []
    for form in (list, iter):
        pool, g = _fill(mkv, lens=())
        q, k, v = (torch.randn(75, h, 256, generator=g).to(DEV) for h in (24, 4, 4))
        pool.extend(form([0, 1]), form([70, 5]))
        pool.append(0, form([0, 1]), form([70, 5]), k, v)
        out = pool.append_rope(1, form([0, 1]), form([70, 5]), q, k, v, rope)
        got.append([out] + [x for layer in range(2) for r in range(2) for x in _dense(pool, layer, r)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ------------------------------------------------------------------ demotions of shared pages
def test_a_demotion_of_all_owners_keeps_a_page_shared(mkv):
    p = _host(mkv, tq3_slots=2)
    p.extend([0], [64 * 3 + 1])
    p.fork([0, 0, 0], [1, 2, 3])
    free = p.stats().fp8_slots_free
    before = p.stats().fp8_bytes + p.stats().tq3_bytes
    p.demote([0, 1, 2, 3, 1, 0], [0, 0, 0, 0, 2, 2])     # page 2 for two of its owners
    assert len({_slots(p, r)[0] for r in range(4)}) == 1 and _slots(p, 0)[0][0] == 3
    assert _slots(p, 0)[2] == _slots(p, 1)[2] != _slots(p, 2)[2] == _slots(p, 3)[2]
    st = p.stats()
    assert st.tq3_slots_free == 0 and st.fp8_slots_free == free + 1
    assert st.fp8_bytes + st.tq3_bytes == before - 2 * 132096 + 2 * 2 * 50176
    _refused(mkv, 3, p.demote, [2, 3], [2, 2])           # one more slot is needed, and nothing changes
    assert _slots(p, 2)[2][0] == 1
    for r in (1, 3, 0, 2):
        p.release(r)
    st = p.stats()
    assert st.tq3_slots_free == 2 and st.fp8_slots_free == 12


@pytest.mark.gpu
def test_a_shared_demoted_page_holds_what_an_unshared_one_does(mkv):
    pool, g = _fill(mkv, lens=(5 * 64 + 17, 130))
    alone, _ = _fill(mkv, lens=(5 * 64 + 17, 130))
    for x in (pool, alone):
        x.fork([0, 1, 0], [2, 3, 4])
    pages = [([0, 2, 4, 1, 3], [1, 1, 1, 0, 0]), ([0, 2, 4], [3, 3, 3])]
    for ids, pgs in pages:
        pool.demote(ids, pgs)
        for r, pg in zip(ids, pgs):                       # one by one: a copy each
            alone.demote([r], [pg])
    assert pool.stats().tq3_slots_free == 20 - 3 and alone.stats().tq3_slots_free == 20 - 8
    q = torch.randn(5, 24, 256, generator=g).to(DEV)
    for layer in range(3):
        for r in range(5):
            for a, b in zip(_dense(pool, layer, r), _dense(alone, layer, r)):
                assert torch.equal(a, b)
        for a, b in zip(pool.decode(layer, range(5), q), alone.decode(layer, range(5), q)):     # the same plan
            assert torch.equal(a, b)
    pool.check_device_errors()


# ------------------------------------------------------------------ what lies behind a sequence's end
@pytest.mark.gpu
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("P,keep", [(64, 66), (64, 65), (128, 143), (64, 3)])
def test_rows_behind_the_end_of_a_sequence_reach_nobody(mkv, P, keep, bad):
    """Rows with NaNs and infinities are cut off (or their sequence is released): the shorter sequence, its fork, and the
    next one in the freed pages decode as they do in a pool that never held such rows."""
    H, D, n = 4, 256, keep + 7
    g = torch.Generator().manual_seed(keep)
    k, v = (torch.randn(n, H, D, generator=g).to(DEV) for _ in range(2))
    kb, vb = k.clone(), v.clone()
    for x in (kb, vb):
        x[keep:, :, 11] = float(bad)
        x[keep + 1:, :, 200] = -float(bad)
    pools = []
    for rows in ((k, v), (kb, vb)):
        pool = mkv.MkvPool(1, 24, H, D, P, 8, 2, max_seqs=6, max_pages_per_seq=8, device=DEV)
        pool.extend([0], [n])
        pool.append(0, [0], [n], *rows)
        pool.truncate([0], [keep])
        pool.fork([0], [1])
        pools.append(pool)
    q = torch.randn(2, 24, D, generator=g).to(DEV)
    qm = torch.randn(2, 3, 24, D, generator=g).to(DEV)

    def same(fn):
        for a, b in zip(*(fn(p) for p in pools)):
            assert torch.isfinite(a).all() and torch.equal(a, b)
    same(lambda p: p.decode(0, [0, 1], q))
    same(lambda p: p.decode_multi(0, [0, 1], qm[:, :min(3, keep)].contiguous()))
    same(lambda p: p.decode_multi(0, [0, 1], qm[:, :2].contiguous()))
    one = [torch.randn(2, H, D, generator=g).to(DEV) for _ in range(2)]
    for p in pools:
        p.extend([0, 1], [1, 1])
    same(lambda p: p.append_decode(0, [0, 1], *one, q))
    same(lambda p: p.dequantize(0, 1, 0, p.seq_info(1)[1]))
    # the freed pages' next owner
    few = [torch.randn(5, H, D, generator=g).to(DEV) for _ in range(2)]
    for p in pools:
        p.extend([0], [6])                                # the rows of old values come into use again: written anew
        p.append(0, [0], [6], *(torch.cat([x, x[:1]]) for x in few))
        p.release(0)
        p.release(1)
        p.extend([2], [P + 5])
        p.append(0, [2], [P + 5], torch.cat([k[:1].expand(P, H, D), few[0]]), torch.cat([v[:1].expand(P, H, D), few[1]]))
    same(lambda p: p.decode(0, [2], q[:1]))
    for p in pools:
        p.check_device_errors()
