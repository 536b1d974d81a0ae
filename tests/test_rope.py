"""Rotary positions (mkv_rope) and the append fused with them (mkv_append_rope): frequencies and refusals on the
CPU; values, gradients, layouts and strides on the GPU against the formula in extended precision."""
import itertools
import math

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


# ------------------------------------------------------------------ CPU
def test_frequencies_without_scaling_and_linear(mkv):
    r = mkv.Rope(64, base=10000.0)
    want = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    assert np.allclose(r.inv_freq, want, rtol=1e-14) and r.mscale == 1.0
    r = mkv.Rope(64, base=10000.0, scaling="linear", factor=8.0)
    assert np.allclose(r.inv_freq, np.array(want) / 8, rtol=1e-14)


def test_turns_are_the_frequencies_over_two_pi(mkv):
    # 2^-53 of the frequency's own rounding in w / 2 pi, 2^-65 of the table's
    for w in (1.0, 0.37, 1e-9, 7.5, -0.2, 0.0):
        t = mkv.Rope(2, inv_freq=[w]).table.turns[0]
        exact = (np.longdouble(w) / (2 * np.longdouble(math.pi))) % 1
        d = abs(np.longdouble(t) / np.longdouble(2) ** 64 - exact)
        assert min(d, 1 - d) <= 2.0 ** -52 * max(abs(w), 2.0 ** -11), w


def test_ntk_keeps_the_fastest_pair_and_stretches_the_slowest_by_the_factor(mkv):
    plain, ntk = mkv.Rope(128, base=1e6), mkv.Rope(128, base=1e6, scaling="ntk", factor=4.0)
    assert ntk.inv_freq[0] == plain.inv_freq[0] == 1.0
    assert np.isclose(ntk.inv_freq[-1], plain.inv_freq[-1] / 4.0, rtol=1e-12)


def test_yarn_keeps_fast_pairs_divides_slow_ones_and_scales(mkv):
    L, f = 32768, 4.0
    plain = mkv.Rope(128, base=1e6)
    yarn = mkv.Rope(128, base=1e6, scaling="yarn", factor=f, original_length=L, beta_fast=32, beta_slow=1)
    for a, b in zip(plain.inv_freq, yarn.inv_freq):
        turns = L * a / (2 * math.pi)
        if turns > 32 * 1.3:        # the ramp's ends are rounded to whole pairs: base^(2/128) = 1.24 apart
            assert b == a
        elif turns < 1 / 1.3:
            assert np.isclose(b, a / f, rtol=1e-14)
        else:
            assert a / f <= b * (1 + 1e-14) and b <= a * (1 + 1e-14)
    assert np.isclose(yarn.mscale, 0.1 * math.log(f) + 1, rtol=1e-7)


@pytest.mark.parametrize("rot,base,L,f", [
    (128, 1e4, 131072, 4.0), (128, 1e4, 65536, 4.0), (64, 1e4, 131072, 8.0), (256, 1e4, 262144, 2.0), (4, 1e6, 32768, 4.0),
    (2, 1e4, 4096, 4.0), (128, 500.0, 1 << 20, 4.0), (6, 100.0, 1e9, 4.0), (128, 1e6, 32768, 4.0), (64, 1e4, 100, 2.0),
])
def test_yarn_ramp_may_end_past_the_last_pair(mkv, rot, base, L, f):
    # in 64-bit numpy; the library's own fp64 differs by a few roundings (2^-53 each) of logs, powers and products
    fast, slow = 32.0, 1.0
    w = base ** (-np.arange(0, rot, 2) / rot)
    index = lambda turns: rot / 2 * math.log(L / (2 * math.pi * turns)) / math.log(base)    # pair of that many turns
    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rot - 1)
    ramp = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
    got = mkv.Rope(rot, base=base, scaling="yarn", factor=f, original_length=L, beta_fast=fast, beta_slow=slow).inv_freq
    assert np.allclose(got, w * (1 - ramp) + w / f * ramp, rtol=1e-12, atol=0)
    for a, b in zip(w, got):        # only pairs of fewer than beta_slow turns take the whole factor
        if L * a / (2 * math.pi) > slow and index(slow) < rot - 1:
            assert b > a / f * (1 + 1e-9)


def test_wavelength_scaling_blends_by_turns(mkv):
    L, f, lo, hi = 8192, 8.0, 1.0, 4.0
    plain = mkv.Rope(128, base=5e5)
    w = mkv.Rope(128, base=5e5, scaling="wavelength", factor=f, original_length=L, low_freq=lo, high_freq=hi)
    for a, b in zip(plain.inv_freq, w.inv_freq):
        t = L * a / (2 * math.pi)
        s = min(max((t - lo) / (hi - lo), 0), 1)
        assert np.isclose(b, a * s + a / f * (1 - s), rtol=1e-13)


@pytest.mark.parametrize("kw", [
    dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=258), dict(rot_dim=8, base=1.0), dict(rot_dim=8, base=float("nan")),
    dict(rot_dim=8, scaling="linear", factor=0.5), dict(rot_dim=8, scaling="ntk", factor=float("inf")),
    dict(rot_dim=8, scaling="yarn", factor=2.0, original_length=0), dict(rot_dim=8, scaling="yarn", factor=2.0, beta_slow=0.0),
    dict(rot_dim=8, scaling="yarn", factor=2.0, beta_fast=0.5), dict(rot_dim=8, scaling="wavelength", factor=2.0, high_freq=1.0),
    dict(rot_dim=4, inv_freq=[1.0, float("nan")]), dict(rot_dim=4, inv_freq=[1.0, 2.0], mscale=float("inf")),
])
def test_bad_tables_are_refused(mkv, kw):
    with pytest.raises(mkv.MkvError) as e:
        mkv.Rope(**kw)
    assert e.value.status == 1


def test_bad_table_arguments_in_python(mkv):
    with pytest.raises(ValueError):
        mkv.Rope(8, scaling="other")
    with pytest.raises(ValueError):
        mkv.Rope(8, inv_freq=[1.0])


def test_tensors_that_autograd_would_record_are_refused(mkv):
    rope, pos = mkv.Rope(16), torch.zeros(3, dtype=torch.int64)
    x, w = torch.zeros(3, 2, 16), torch.zeros(3, 2, 16, requires_grad=True)
    for args, kw in (((w, None, pos), {}), ((x, w, pos), {}), ((w * 2, x, pos), {}), ((x, x, pos), dict(q_out=w)),
                     ((x, x, pos), dict(k_out=w)), ((w, w, pos), dict(inverse=True))):
        with pytest.raises(RuntimeError, match="autograd"):
            rope(*args, **kw)
        with torch.no_grad(), pytest.raises(TypeError, match="CUDA"):        # past that check, to the next (no device here)
            rope(*args, **kw)
    with pytest.raises(TypeError, match="CUDA"):
        rope(x, x, pos)


@pytest.mark.gpu
def test_rope_inside_an_autograd_function_has_the_formulas_gradient(mkv):
    rope = mkv.Rope(32, interleaved=True)

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, pos):
            ctx.save_for_backward(pos)
            return rope(x, None, pos)[0]

        @staticmethod
        def backward(ctx, grad):
            return rope(grad.contiguous(), None, ctx.saved_tensors[0], inverse=True)[0], None

    g = torch.Generator().manual_seed(1)
    pos = torch.arange(9).to(DEV)
    x = torch.randn(9, 3, 48, generator=g).to(DEV).requires_grad_()
    up = torch.randn(9, 3, 48, generator=g).to(DEV)
    Rotate.apply(x, pos).backward(up)
    ref, size = _reference(up.double().cpu().numpy(), pos.cpu().numpy(), rope.inv_freq, rope.mscale, True, transpose=True)
    _close(x.grad, ref, size, pos.cpu().numpy(), rope.inv_freq, torch.float32)


def _rows(mkv, heads=2, d=16, ptr=0x1000, out=0x100000, **kw):
    a = dict(inp=ptr, out=out, heads=heads, reserved=0, in_token=heads * d, in_head=d, out_token=heads * d, out_head=d)
    a.update(kw)
    return mkv.binding.RopeRows(*(a[n] for n, _ in mkv.binding.RopeRows._fields_))


@pytest.mark.parametrize("bad", [
    dict(d=8), dict(d=5000), dict(nbytes=2), dict(dtype=7), dict(tokens=-1), dict(pos=None), dict(pos=0x1002),
    dict(row=dict(inp=None)), dict(row=dict(out=0x100001)), dict(row=dict(in_token=-32)), dict(row=dict(out_head=8)),
    dict(row=dict(out_token=0)), dict(row=dict(out=0x1000, in_token=64)), dict(row=dict(heads=-1)), dict(row=dict(reserved=1)),
])
def test_rope_refuses_before_any_launch(mkv, bad):
    t = mkv.Rope(16).table
    row = _rows(mkv, **bad.get("row", {}))
    with pytest.raises(mkv.MkvError) as e:
        mkv.binding.mkv_rope(t, bad.get("tokens", 4), bad.get("d", 16), bad.get("pos", 0x2000), bad.get("nbytes", 8), row,
                             None, bad.get("dtype", 0))
    assert e.value.status == 1


@pytest.mark.parametrize("row", [dict(heads=4, out_token=1, out_head=2 ** 62), dict(heads=4, out_token=2 ** 62, out_head=1)])
def test_rope_refuses_overlaps_past_64_bits(mkv, row):
    with pytest.raises(mkv.MkvError) as e:
        mkv.binding.mkv_rope(mkv.Rope(16).table, 8, 16, 0x2000, 8, _rows(mkv, **row), None, 0)
    assert e.value.status == 1


def test_append_rope_refuses_on_a_host_only_pool(mkv):
    pool = mkv.MkvPool(2, 24, 4, 256, 64, fp8_slots=12, tq3_slots=6, max_seqs=4, max_pages_per_seq=16, host_only=True)
    rope = mkv.Rope(128)
    pool.extend([0, 1], [64 * 3, 10])
    B = mkv.binding
    ok = dict(layer=0, ids=[0], new=[4], q=0x1000, qo=0x1000, k=0x2000, v=0x3000, dtype=0)

    def call(**kw):
        a = {**ok, **kw}
        B.mkv_append_rope(pool.handle, a["layer"], a["ids"], a["new"], kw.get("table", rope.table), a["q"], a["qo"], a["k"],
                          a["v"], a["dtype"])
    call()
    call(new=[0], k=None, v=None)
    broken = mkv.Rope(128).table
    broken.rot_dim = 300
    for bad, status in ((dict(layer=2), 1), (dict(ids=[9]), 1), (dict(new=[200]), 1), (dict(k=None), 1), (dict(q=None), 1),
                        (dict(qo=None), 1), (dict(k=0x2008), 1), (dict(dtype=2), 1), (dict(table=broken), 1),
                        (dict(ids=[0, 0], new=[1, 1]), 1)):
        with pytest.raises(mkv.MkvError) as e:
            call(**bad)
        assert e.value.status == status, bad
    pool.demote([0], [1])
    with pytest.raises(mkv.MkvError) as e:
        call(new=[100])                                  # reaches into the TQ3 page
    assert e.value.status == 4
    with pytest.raises(ValueError):
        B.mkv_append_rope(pool.handle, 0, [0], [1, 2], rope.table, None, None, 0x1000, 0x1000, 0)


# ------------------------------------------------------------------ GPU
def _reference(x, pos, w, m, interleaved, transpose=False):
    """Extended precision: (rotated, |pair| bound per element).  x [T, H, d] float64 numpy."""
    half = len(w)
    ang = pos.astype(np.longdouble)[:, None] * np.asarray(w, np.longdouble)
    c, s = (np.cos(ang) * m).astype(np.float64)[:, None], (np.sin(ang) * m).astype(np.float64)[:, None]
    if transpose:
        s = -s
    y, size = x.copy(), np.zeros_like(x)
    a = np.s_[..., 0:2 * half:2] if interleaved else np.s_[..., :half]
    b = np.s_[..., 1:2 * half:2] if interleaved else np.s_[..., half:2 * half]
    y[a], y[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    size[a] = size[b] = (np.abs(x[a]) + np.abs(x[b])) * abs(m)
    return y, size


def _close(got, ref, size, pos, w, dtype):
    # angle: 2^-25 turns from the fp32 turn, 2^-51 of pos w from the table and the reference; sincospif 2^-23;
    # three fp32 roundings; then half a step of the output type
    ang = 2 * math.pi * 2.0 ** -25 + 2.0 ** -51 * float(np.abs(pos).max()) * max(abs(x) for x in w)
    tol = size * (ang + 2.0 ** -23 + 3 * 2.0 ** -24) + np.abs(ref) * torch.finfo(dtype).eps / 2
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25                           # half a step of the subnormals
    d = np.abs(got.double().cpu().numpy() - ref)
    assert (d <= tol * 1.01).all(), (d / np.maximum(tol, 1e-300)).max()


CASES = [(T, hq, hk, d, rot) for (T, hq, hk, d, rot) in [
    (1, 1, 1, 2, 2), (1, 24, 4, 256, 256), (3, 5, 0, 64, 64), (64, 24, 4, 256, 128), (129, 7, 1, 96, 34), (33, 2, 2, 66, 10),
    (1000, 16, 4, 128, 128), (700, 24, 4, 256, 64)]]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", CASES, ids=str)
def test_rope_matches_the_formula(mkv, shape, interleaved, dtype):
    T, hq, hk, d, rot = shape
    g = torch.Generator().manual_seed(T * 7 + rot)
    q, k = (torch.randn(T, h, d, generator=g).to(dtype) for h in (hq, max(hk, 1)))
    pos = torch.randint(0, 2 ** 31 - 1, (T,), generator=g)
    pos[0] = 0
    rope = mkv.Rope(rot, base=10000.0, interleaved=interleaved, scaling="yarn", factor=2.0, original_length=2048)
    idx = pos.to(torch.int32) if T % 2 else pos
    yq, yk = rope(q.to(DEV), k.to(DEV) if hk else None, idx.to(DEV))
    for x, y in ((q, yq), (k, yk))[:2 if hk else 1]:
        ref, size = _reference(x.double().numpy(), pos.numpy(), rope.inv_freq, rope.mscale, interleaved)
        _close(y, ref, size, pos.numpy(), rope.inv_freq, dtype)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_strides_in_place_and_shared_buffer(mkv, interleaved):
    # q, k and v as slices of one projection, an odd offset, the heads outermost, a head repeated by stride 0
    g = torch.Generator().manual_seed(5)
    T, hq, hk, d = 37, 6, 2, 64
    rope = mkv.Rope(32, interleaved=interleaved)
    pos = torch.arange(T) * 1001
    qkv = torch.randn(T, (hq + 2 * hk) * d + 3, generator=g)
    buf = qkv.to(DEV)
    view = buf[:, 3:].unflatten(1, (hq + 2 * hk, d))     # 12 bytes off: the scalar path
    q, k = view[:, :hq], view[:, hq:hq + hk]
    rq, sq = _reference(q.double().cpu().numpy(), pos.numpy(), rope.inv_freq, 1.0, interleaved)
    rk, sk = _reference(k.double().cpu().numpy(), pos.numpy(), rope.inv_freq, 1.0, interleaved)
    oq, ok = rope(q, k, pos.to(DEV))
    hm = torch.full((hq, T, d), 9.0, device=DEV)         # heads outermost
    rope(q, None, pos.to(DEV), q_out=hm.transpose(0, 1))
    rope(q, k, pos.to(DEV), q_out=q, k_out=k)
    for got, ref, size in ((oq, rq, sq), (ok, rk, sk), (q, rq, sq), (k, rk, sk), (hm.transpose(0, 1), rq, sq)):
        _close(got, ref, size, pos.numpy(), rope.inv_freq, torch.float32)
    assert torch.equal(buf[:, :3].cpu(), qkv[:, :3]) and torch.equal(view[:, hq + hk:].cpu(), qkv[:, 3:].unflatten(1, (hq + 2 * hk, d))[:, hq + hk:])
    one = torch.randn(T, 1, d, generator=g).to(DEV)
    wide, _ = rope(one.expand(T, 4, d), None, pos.to(DEV))
    assert all(torch.equal(wide[:, 0], wide[:, i]) for i in range(4))
    with pytest.raises(mkv.MkvError):
        rope(q, None, pos.to(DEV), q_out=one.expand(T, hq, d))       # an output whose heads overlap


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved,rot", [(False, 64), (True, 64), (False, 30), (True, 30)])
def test_rope_gradient_is_the_transpose(mkv, interleaved, rot):
    g = torch.Generator().manual_seed(8)
    T, h, d = 50, 3, 64
    rope = mkv.Rope(rot, interleaved=interleaved, scaling="yarn", factor=3.0, original_length=100)
    pos = torch.randint(-5000, 5000, (T,), generator=g)
    grad = torch.randn(T, h, d, generator=g)
    gx, _ = rope(grad.to(DEV), None, pos.to(DEV), inverse=True)
    ref, size = _reference(grad.double().numpy(), pos.numpy(), rope.inv_freq, rope.mscale, interleaved, transpose=True)
    _close(gx, ref, size, pos.numpy(), rope.inv_freq, torch.float32)
    # differences: the map is linear, so a step along v changes <grad, R x> by <R^T grad, v> up to rounding:
    # 3 h d T terms, each within a few 2^-23
    x, v = (torch.randn(T, h, d, generator=g) for _ in range(2))
    f = lambda z: float((rope(z.to(DEV), None, pos.to(DEV))[0].double().cpu() * grad.double()).sum())  # noqa: E731
    diff = (f(x + 0.5 * v) - f(x - 0.5 * v))
    want = float((gx.double().cpu() * v.double()).sum())
    bound = 2.0 ** -20 * float(((x.abs() + v.abs()) * 4 * (grad.abs().amax() + 1)).sum())
    assert abs(diff - want) <= bound
    # mscale 1: the transpose is the inverse
    plain = mkv.Rope(rot, interleaved=interleaved)
    back, _ = plain(plain(x.to(DEV), None, pos.to(DEV))[0], None, pos.to(DEV), inverse=True)
    assert (back.cpu() - x).abs().max() <= 4e-6 * x.abs().max()


@pytest.mark.gpu
def test_rope_without_tokens_on_a_side_stream_and_captured(mkv):
    rope = mkv.Rope(64)
    e = torch.empty(0, 4, 64, device=DEV)
    q, k = rope(e, e, torch.empty(0, dtype=torch.int64, device=DEV))
    assert q.shape == k.shape == (0, 4, 64)
    x = torch.randn(40, 4, 64, device=DEV)
    pos = torch.arange(40, device=DEV)
    want, _ = rope(x, None, pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, _ = rope(x, None, pos)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope(x, None, pos, q_out=out)
    x.copy_(torch.randn_like(x))
    pos.add_(17)
    graph.replay()
    assert torch.equal(out, rope(x, None, pos)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rot,interleaved", [(256, False), (128, True), (64, False), (2, False), (34, True), (250, False)])
@pytest.mark.parametrize("P,new", [(64, [1, 1, 1]), (64, [67, 1, 130]), (128, [0, 129, 3]), (64, [900, 5, 64])])
def test_append_rope_is_rope_then_append(mkv, P, new, rot, interleaved, dtype):
    g = torch.Generator().manual_seed(sum(new) + rot)
    rope = mkv.Rope(rot, base=10000.0, interleaved=interleaved)
    old = [37, 64, 0]
    pools = [mkv.MkvPool(2, 24, 4, 256, P, 40, 4, max_seqs=3, max_pages_per_seq=20, device=DEV) for _ in range(2)]
    pos = torch.cat([torch.arange(a) + b for a, b in zip(new, old)]).to(DEV)
    for pool in pools:
        pool.extend([0, 1, 2], old)
        pool.extend([0, 1, 2], new)
    T = sum(new)
    for layer in (1, 0):
        q = torch.randn(T, 24, 256, generator=g).to(dtype).to(DEV)
        k, v = (torch.randn(T, 4, 256, generator=g).to(dtype).to(DEV) for _ in range(2))
        k[0, 0] = 0                                      # a row of zeros
        qr, _ = rope(q, None, pos)
        kr, _ = rope(k.float(), None, pos)               # K is not rounded between the two
        pools[0].append(layer, [0, 1, 2], new, kr, v.float())
        got = pools[1].append_rope(layer, [0, 1, 2], new, q, k, v, rope)
        assert torch.equal(got, qr)
        again = pools[1].append_rope(layer, [0, 1, 2], new, None, k, v, rope)    # the cached destinations, no q
        assert again is None
        for r in range(3):
            for pg in range(pools[0].seq_info(r)[1]):
                a, b = pools[0].export_page(layer, r, pg), pools[1].export_page(layer, r, pg)
                assert a[0] == b[0], (layer, r, pg)
    # in place, and mixed with plain appends of the same tokens
    q2 = q.clone()
    pools[1].append_rope(0, [0, 1, 2], new, q2, k, v, rope, q_out=q2)
    assert torch.equal(q2, qr)
    pools[1].append(0, [0, 1, 2], new, kr, v.float())
    pools[1].append_rope(0, [0, 1, 2], new, q, k, v, rope)
    assert pools[0].export_page(0, 1, 0)[0] == pools[1].export_page(0, 1, 0)[0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_append_rope_quantises_as_append_does_at_every_magnitude(mkv, dtype):
    """The quotients by reciprocal are the divisions: rows whose values span the exponents, subnormal and vanishing
    scales, scales past fp16's range, values next to code borders, signed zeros."""
    g = torch.Generator().manual_seed(9)
    n = 640
    k = torch.randn(n, 4, 256, generator=g) * torch.exp2(torch.randint(-140, 24, (n, 4, 1), generator=g).float())
    k[:64] *= torch.exp2(torch.randint(-60, 1, (64, 4, 256), generator=g).float())
    steps = torch.arange(256).float() / 16                # multiples of half a step of the codes, and their neighbours
    k[64:128] = (1 + steps) * torch.exp2(torch.arange(64).float() - 32)[:, None, None]
    k[128:192] = torch.nextafter(k[64:128], torch.tensor(0.0))
    k[192] = 0
    k[193] = -0.0
    k[194] = 3e38
    k, v = k.to(dtype).to(DEV), k.flip(0).to(dtype).contiguous().to(DEV)
    rope = mkv.Rope(2, inv_freq=[0.0])                    # the identity
    pools = [mkv.MkvPool(1, 24, 4, 256, 64, 12, 1, max_seqs=1, max_pages_per_seq=12, device=DEV) for _ in range(2)]
    for pool in pools:
        pool.extend([0], [n])
    pools[0].append(0, [0], [n], k, v)
    pools[1].append_rope(0, [0], [n], None, k, v, rope)
    for pg in range(10):
        a, b = (np.frombuffer(p.export_page(0, 0, pg)[0], np.uint8) for p in pools)
        # the rotated first pair loses the sign of a zero (0 * x is added): compare values there, bits elsewhere
        bad = np.flatnonzero(a != b)
        assert all(a[i] & 0x7F == 0 and b[i] & 0x7F == 0 for i in bad), (pg, bad[:5], a[bad[:5]], b[bad[:5]])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [70, 3000])
def test_append_rope_quantises_infinities_and_nans_as_append_does(mkv, n, dtype):
    """Rows with an infinity (scale infinity), with a NaN (the scale of the others), with both, at both launch shapes."""
    g = torch.Generator().manual_seed(10)
    k = torch.randn(n, 4, 256, generator=g)
    k[3, 0, 7] = math.inf                                 # (not in the rotated pair, whose other value it would reach)
    k[5, 1, 255] = -math.inf
    k[6, 2, 100] = math.nan
    k[7, 3, 9], k[7, 3, 200] = math.inf, math.nan
    k[8, 0, 2:] = math.inf
    k[9, 1, 2:] = math.nan
    k, v = k.to(dtype).to(DEV), k.flip(0).to(dtype).contiguous().to(DEV)
    rope = mkv.Rope(2, inv_freq=[0.0])                    # the identity
    pools = [mkv.MkvPool(1, 24, 4, 256, 64, 60, 1, max_seqs=1, max_pages_per_seq=60, device=DEV) for _ in range(2)]
    for pool in pools:
        pool.extend([0], [n])
    pools[0].append(0, [0], [n], k, v)
    pools[1].append_rope(0, [0], [n], None, k, v, rope)
    for pg in range(pools[0].seq_info(0)[1]):
        a, b = (np.frombuffer(p.export_page(0, 0, pg)[0], np.uint8).reshape(4, 2, 64 * 258) for p in pools)
        scales = [x[:, :, 64 * 256:].copy().view(np.uint16) for x in (a, b)]
        assert (scales[0] == scales[1]).all(), pg
        # codes: bits, but for the sign of a zero (see above) and of a NaN
        bad = np.flatnonzero(a != b)
        a, b = a.reshape(-1)[bad], b.reshape(-1)[bad]
        assert ((a & 0x7F) == (b & 0x7F)).all() and np.isin(a & 0x7F, [0, 0x7F]).all(), pg


@pytest.mark.gpu
def test_append_rope_decode_step_against_the_definition(mkv):
    """Rotate, append and attend, as a decode loop does, against fp64 attention over the exported pages' values and
    the formula's q."""
    g = torch.Generator().manual_seed(3)
    rope = mkv.Rope(256, base=1e6, scaling="yarn", factor=4.0, original_length=128)
    pool = mkv.MkvPool(1, 24, 4, 256, 64, 40, 20, max_seqs=2, max_pages_per_seq=20, device=DEV)
    pool.extend([0, 1], [300, 70])
    k, v = (torch.randn(370, 4, 256, generator=g).to(DEV) for _ in range(2))
    pool.append_rope(0, [0, 1], [300, 70], None, k, v, rope)
    pool.demote([0, 0], [1, 2])
    pool.extend([0, 1], [1, 1])
    q = torch.randn(2, 24, 256, generator=g).to(DEV)
    k1, v1 = (torch.randn(2, 4, 256, generator=g).to(DEV) for _ in range(2))
    qr = pool.append_rope(0, [0, 1], [1, 1], q, k1, v1, rope)
    out, lse = pool.decode(0, [0, 1], qr)
    for r, n in ((0, 301), (1, 71)):
        kd, vd = pool.dequantize(0, r, 0, pool.seq_info(r)[1])
        kd, vd = kd[:n].double().cpu().numpy(), vd[:n].double().cpu().numpy()
        rq, _ = _reference(q[r:r + 1].double().cpu().numpy(), np.array([n - 1]), rope.inv_freq, rope.mscale, False)
        for h in range(24):
            s = kd[:, h // 6] @ rq[0, h] / 16.0
            w = np.exp(s - s.max())
            ref = w @ vd[:, h // 6] / w.sum()
            assert np.abs(out[r, h].double().cpu().numpy() - ref).max() <= 2e-3 * np.abs(ref).max()
            assert abs(float(lse[r, h]) - (s.max() + math.log(w.sum()))) <= 1e-4
    # the appended K row is the formula's, quantised: half a step of e4m3, of the fp16 scale, and of the subnormals
    kd, _ = pool.dequantize(0, 1, 1, 1)
    ref, _ = _reference(k1[1:].double().cpu().numpy(), np.array([70]), rope.inv_freq, rope.mscale, False)
    d = np.abs(kd[70 - 64].double().cpu().numpy() - ref[0])
    amax = np.abs(ref[0]).max(-1, keepdims=True)
    assert (d <= np.abs(ref[0]) * (2.0 ** -4 + 2.0 ** -11) + amax / 448 * 2.0 ** -10 + 1e-6).all()
    pool.check_device_errors()


@pytest.mark.gpu
def test_append_rope_wants_tensors_of_the_pools_device(mkv):
    pool = mkv.MkvPool(1, 8, 1, 256, 64, 4, 1, max_seqs=2, max_pages_per_seq=2, device=DEV)
    pool.extend([0], [3])
    q, k = torch.zeros(3, 8, 256), torch.zeros(3, 1, 256)
    for args in ((q.to(DEV), k.to(DEV), k), (q.to(DEV), k, k.to(DEV)), (q, k.to(DEV), k.to(DEV))):
        with pytest.raises(ValueError):
            pool.append_rope(0, [0], [3], *args, mkv.Rope(16))
    with pytest.raises(ValueError):
        pool.append_rope(0, [0], [3], q.to(DEV), k.to(DEV), k.to(DEV), mkv.Rope(16), q_out=q.clone())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hk,d,rot", [(50, 24, 4, 256, 250), (4001, 24, 4, 256, 100), (2000, 5, 0, 64, 6), (77, 3, 1, 72, 66),
                                           (1, 1, 1, 256, 2), (3000, 16, 4, 128, 120), (31, 2, 1, 20, 12)])
def test_dims_past_the_rotated_ones_keep_their_bits(mkv, T, hq, hk, d, rot, interleaved, dtype):
    """Whatever they hold (infinities, NaN, -0), in place and not; chunks that end inside the rotated part or past it."""
    g = torch.Generator().manual_seed(T + rot)
    rope = mkv.Rope(rot, interleaved=interleaved)
    pos = torch.randint(0, 100000, (T,), generator=g)
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 0.0, 1.5])
    x = torch.randn(T, hq + hk, d, generator=g).to(dtype)
    x[..., rot:] = odd[torch.randint(0, 6, (T, hq + hk, d - rot), generator=g)].to(dtype)
    x[..., :rot:3] = -0.0
    bits = torch.int32 if dtype == torch.float32 else torch.int16
    y = x.to(DEV)
    q, k = y[:, :hq], y[:, hq:] if hk else None
    q1, k1 = rope(q, k, pos.to(DEV))
    rope(q, k, pos.to(DEV), q_out=q, k_out=k)            # in place
    got = torch.cat([q1, k1], 1) if hk else q1
    assert torch.equal(got.view(bits), y.view(bits))
    assert torch.equal(y[..., rot:].cpu().view(bits), x[..., rot:].contiguous().view(bits))
    ref, size = _reference(x[..., :rot].double().numpy(), pos.numpy(), rope.inv_freq, rope.mscale, interleaved)
    _close(y[..., :rot], ref, size, pos.numpy(), rope.inv_freq, dtype)
