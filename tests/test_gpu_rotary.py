"""Head norms and rotation by position against the formulas in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from agent_shared_context_gb300 import kvc  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _frequencies(rot, base):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def _reference(x, pos, rot, base, interleaved, norm, w, amplitude=1.0):
    """(value, size of the terms that it is a sum of) of every element, in 64 bits."""
    x = x.double().cpu()
    d = x.shape[-1]
    if norm:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        if w is not None:
            x = x * w.double().cpu()
    y, size = x.clone(), x.abs()
    ang = torch.outer(pos.double().cpu(), torch.tensor(_frequencies(rot, base), dtype=torch.float64))
    c, s = (amplitude * f(ang)[:, None] for f in (torch.cos, torch.sin))
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = amplitude * (a.abs() + b.abs())
    assert y.shape[-1] == d
    return y, size


def _check(got, want, size, dtype):
    """The result is rounded once, by half a step at most; in fp32 the cosine is off by
    (1.6 + 2) 2^-24 (angle of 2^-25 half turns, two units of sincospi), the norm by less
    than 20 2^-24 (sum of 256 squares by 16 + 5 levels, halved, root, two products), the
    two products and the sum by 3 2^-24, each of the terms: 32 2^-24 in all."""
    got = got.double().cpu()
    half = torch.finfo(dtype).eps / 2
    bound = half * want.abs() * (1 + 2 ** -10) + (1 + half) * 32 * 2.0 ** -24 * size + 1e-38
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() - bound)[bad].max()))


def _run(N, Hq, H, d, rot, dtype, interleaved=False, norm=False, weights=True, layout="plain",
         base=10000.0, far=100000, seed=0, stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dt)  # noqa: E731
    if layout == "packed":                     # parts of one projection's rows
        x = rnd(N, Hq + 2 * H, d)
        q, k = x[:, :Hq], x[:, Hq:Hq + H]
    elif layout == "odd":                      # nothing on a 16-byte boundary
        q, k = (rnd(N, h, d + 3)[:, :, 1:d + 1] for h in (Hq, H))
    elif layout == "heads":                    # heads outermost
        q, k = (rnd(h, N, d).transpose(0, 1) for h in (Hq, H))
    else:
        q, k = rnd(N, Hq, d), rnd(N, H, d)
    pos = torch.randint(0, far, (N,), generator=g, device="cuda", dtype=torch.int32)
    w = [(1 + 0.3 * rnd(d).float()).to(dt) if norm and weights else None for _ in "qk"]
    turns, amp = kvc.rotary_turns(rot, base)
    turns = turns.cuda()
    out = [torch.full_like(t, 7) for t in (q, k)] if layout != "packed" else [q.clone(), k.clone()]
    rp = kvc.rotary_params(q if Hq else None, k if H else None, out[0] if Hq else None,
                           out[1] if H else None, rot, interleaved, norm, EPS, amp)
    kvc.kvc_rotate_heads(rp, q, k, pos, turns, out[0], out[1], *w)
    torch.cuda.synchronize()
    for x, y, wt in zip((q, k), out, w):
        if x.shape[1]:
            _check(y, *_reference(x, pos, rot, base, interleaved, norm, wt), dt)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("N,Hq,H,d,rot,layout", [
    (1, 32, 8, 128, 128, "plain"), (37, 28, 4, 128, 128, "packed"), (5, 8, 2, 64, 64, "heads"),
    (300, 3, 1, 80, 20, "plain"), (9, 8, 8, 256, 256, "plain"), (4, 2, 2, 256, 250, "odd"),
    (7, 5, 0, 96, 48, "plain"), (7, 0, 5, 40, 40, "plain"), (2, 1, 1, 2, 2, "plain"),
    (3, 7, 1, 6, 4, "odd"), (11, 130, 3, 32, 32, "packed"), (2, 4, 4, 64, 0, "plain"),
    (6, 4, 2, 24, 8, "packed"), (3, 600, 600, 16, 16, "plain"),
])
def test_against_the_formula(N, Hq, H, d, rot, layout, norm, interleaved, dtype):
    _run(N, Hq, H, d, rot, dtype, interleaved, norm, layout=layout)


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(far):
    """In 64 bits p f has an error of 2^-53 2^31 of its own: far below the bound."""
    _run(200, 2, 1, 128, 128, "f32", far=far, base=500000.0, seed=3)


def test_norm_without_weights():
    _run(20, 4, 2, 128, 64, "bf16", norm=True, weights=False)


def test_amplitude_goes_to_the_rotated_part():
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn((6, 3, 64), generator=g, device="cuda")
    pos = torch.arange(6, device="cuda", dtype=torch.int32) * 1000
    turns, _ = kvc.rotary_turns(32, 10000.0)
    out = torch.empty_like(q)
    rp = kvc.rotary_params(q, None, out, None, 32, amplitude=1.25)
    kvc.kvc_rotate_heads(rp, q, None, pos, turns.cuda(), out, None)
    _check(out, *_reference(q, pos, 32, 10000.0, False, False, None, 1.25), torch.float32)
    assert torch.equal(out[..., 32:], q[..., 32:])


@pytest.mark.parametrize("layout", ["packed", "odd"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_in_place_is_the_same(layout, interleaved, norm):
    g = torch.Generator(device="cuda").manual_seed(1)
    d, pad = 64, 3 if layout == "odd" else 0
    x = torch.randn((50, 6 + 2 + 2, d + pad), generator=g, device="cuda").to(torch.bfloat16)
    before = x.clone()
    q, k = x[:, :6, pad:], x[:, 6:8, pad:]
    pos = torch.randint(0, 5000, (50,), generator=g, device="cuda", dtype=torch.int32)
    turns = kvc.rotary_turns(48)[0].cuda()
    out = [torch.empty(t.shape, dtype=t.dtype, device="cuda") for t in (q, k)]
    rp = kvc.rotary_params(q, k, out[0], out[1], 48, interleaved, norm)
    kvc.kvc_rotate_heads(rp, q, k, pos, turns, out[0], out[1])
    rp = kvc.rotary_params(q, k, q, k, 48, interleaved, norm)
    kvc.kvc_rotate_heads(rp, q, k, pos, turns, q, k)
    assert torch.equal(q, out[0]) and torch.equal(k, out[1])
    assert torch.equal(x[:, 8:], before[:, 8:]) and torch.equal(x[..., :pad], before[..., :pad])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("planes", [False, True])
def test_in_place_where_heads_alternate(planes, dtype):
    """Queries, keys and values of a head beside each other, in tokens' rows or in planes."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N, H, d = 45, 5, 64
    x = torch.randn((H, 3, N, d) if planes else (N, H, 3, d), generator=g, device="cuda").to(DT[dtype])
    before = x.clone()
    q, k, v = ((x[:, i].transpose(0, 1) if planes else x[:, :, i]) for i in range(3))
    q0, k0 = q.clone(), k.clone()
    pos = torch.randint(0, 5000, (N,), generator=g, device="cuda", dtype=torch.int32)
    turns = kvc.rotary_turns(d)[0].cuda()
    kvc.kvc_rotate_heads(kvc.rotary_params(q, k, q, k, d), q, k, pos, turns, q, k)
    torch.cuda.synchronize()
    for a, b in ((q, q0), (k, k0)):
        _check(a, *_reference(b, pos, d, 10000.0, False, False, None), DT[dtype])
    assert torch.equal(v, before[:, 2].transpose(0, 1) if planes else before[:, :, 2])


def test_rows_of_no_token_stay():
    q = torch.randn((8, 3, 128), device="cuda").to(torch.bfloat16)
    q[2] = math.nan
    pos = torch.tensor([5, -1, -1, 7, -2147483648, 0, 1, -1], dtype=torch.int32, device="cuda")
    turns = kvc.rotary_turns(128)[0].cuda()
    out = torch.full_like(q, 9)
    kvc.kvc_rotate_heads(kvc.rotary_params(q, None, out, None, 128), q, None, pos, turns, out, None)
    live = pos >= 0
    assert bool((out[~live] == 9).all())
    _check(out[live], *_reference(q[live], pos[live], 128, 10000.0, False, False, None),
           torch.bfloat16)


def test_one_row_does_not_reach_another():
    """An infinity or NaN stays in its own head; zero heads stay zero under the norm."""
    q = torch.randn((4, 6, 64), device="cuda")
    ref = q.clone()
    q[1, 2, 5], q[2, 3, 60], q[3, 4] = math.inf, math.nan, 0.0
    pos = torch.arange(4, device="cuda", dtype=torch.int32)
    turns = kvc.rotary_turns(64)[0].cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    for x, y in ((q, a), (ref, b)):
        rp = kvc.rotary_params(x, None, y, None, 64, norm=True)
        kvc.kvc_rotate_heads(rp, x, None, pos, turns, y, None)
    same = torch.ones((4, 6), dtype=torch.bool, device="cuda")
    same[1, 2] = same[2, 3] = same[3, 4] = False
    assert torch.equal(a[same], b[same]) and bool((a[3, 4] == 0).all())
    assert not bool(torch.isfinite(a[2, 3]).any())


def test_no_tokens_and_a_replayed_graph():
    turns = kvc.rotary_turns(64)[0].cuda()
    e = torch.empty((0, 4, 64), device="cuda")
    kvc.kvc_rotate_heads(kvc.rotary_params(e, None, e, None, 64), e, None, None, turns, e, None)
    q = torch.randn((16, 4, 64), device="cuda")
    pos = torch.arange(16, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    rp = kvc.rotary_params(q, None, out, None, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kvc.kvc_rotate_heads(rp, q, None, pos, turns, out, None)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvc.kvc_rotate_heads(rp, q, None, pos, turns, out, None)
    pos += 31                                   # read at replay
    graph.replay()
    torch.cuda.synchronize()
    _check(out, *_reference(q, pos, 64, 10000.0, False, False, None), torch.float32)


def test_many_tokens():
    """As many as a context has, and a slice of them looked at."""
    N = 20000
    q = torch.randn((N, 4, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(N, device="cuda", dtype=torch.int32)
    turns = kvc.rotary_turns(64)[0].cuda()
    out = torch.empty_like(q)
    kvc.kvc_rotate_heads(kvc.rotary_params(q, None, out, None, 64), q, None, pos, turns, out, None)
    at = slice(N - 700, N)
    _check(out[at], *_reference(q[at], pos[at], 64, 10000.0, False, False, None), torch.bfloat16)
