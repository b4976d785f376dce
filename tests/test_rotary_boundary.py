"""The rotation's table of frequencies, and what the call refuses.  No GPU: the device
addresses are fake and never dereferenced, so those tests only run where none is visible."""
import math
from fractions import Fraction

import pytest

torch = pytest.importorskip("torch")

from agent_shared_context_gb300 import kvc  # noqa: E402

FAKE = 0x7F0000000000
FAR = 1 << 34
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake device addresses are only passed where no GPU exists")


def _share(i, rot, base, mode, factor, low, high, original):
    """Share of the frequency that is kept, out of the definition."""
    turns = original * base ** (-2 * i / rot) / (2 * math.pi)
    if mode == "linear":
        return 0.0
    if mode == "bands":
        return min(max((turns - low) / (high - low), 0.0), 1.0)
    if mode == "ramp":
        at = lambda t: rot / 2 * math.log(original / (2 * math.pi * t), base)  # noqa: E731
        lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
        return 1 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
    return 1.0


@pytest.mark.parametrize("mode", ["none", "linear", "bands", "ramp"])
@pytest.mark.parametrize("rot,base", [(2, 1e4), (20, 1e4), (64, 1e6), (128, 500000.0), (256, 1e4)])
def test_table(mode, rot, base):
    factor, low, high, original = 8.0, 1.0, 32.0 if mode == "ramp" else 4.0, 8192.0
    turns, amp = kvc.rotary_turns(rot, base, mode, factor, low, high, original)
    assert turns.dtype == torch.int64 and turns.shape == (rot // 2,)
    for i, t in enumerate(turns.tolist()):
        keep = _share(i, rot, base, mode, factor, low, high, original)
        f = base ** (-2 * i / rot) * (keep + (1 - keep) / factor) / (2 * math.pi)
        # pow, the share and the division: a few units of 2^-53 each; the unit of the table
        assert abs(Fraction(t, 1 << 64) - Fraction(f)) <= Fraction(f) * Fraction(1, 1 << 47) + Fraction(1, 1 << 64)
    assert amp == pytest.approx(0.1 * math.log(factor) + 1 if mode == "ramp" else 1.0, rel=1e-6)


def test_table_refusals():
    for kw in (dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=258), dict(base=1.0), dict(base=math.nan),
               dict(base=math.inf), dict(scaling="linear", factor=0.5),
               dict(scaling="bands", factor=math.inf), dict(scaling="bands", factor=8.0, low=0.0),
               dict(scaling="ramp", factor=8.0, low=4.0, high=4.0),
               dict(scaling="ramp", factor=8.0, original=0.0),
               dict(scaling="bands", factor=8.0, original=math.nan)):
        a = dict(rot_dim=64, base=10000.0)
        a.update(kw)
        with pytest.raises(kvc.KvcError):
            kvc.rotary_turns(**a)
    with pytest.raises(ValueError):
        kvc.rotary_turns(64, scaling="other")
    assert kvc.rotary_turns(0)[0].numel() == 0


def _rp(**over):
    a = dict(n_tokens=10, n_q_heads=4, n_kv_heads=2, d=64, rot_dim=64, interleaved=0, norm=0, eps=1e-6,
             amplitude=1.0, dtype=kvc.KVC_BF16, q_s_tok=256, q_s_head=64, k_s_tok=128, k_s_head=64,
             q_out_s_tok=256, q_out_s_head=64, k_out_s_tok=128, k_out_s_head=64)
    a.update(over)
    return kvc.kvc_rotary_params(**a)


def _call(rp=None, **over):
    a = dict(q=FAKE, k=FAKE + FAR, positions=FAKE + 2 * FAR, turns=FAKE + 3 * FAR,
             q_out=FAKE + 4 * FAR, k_out=FAKE + 5 * FAR)
    a.update(over)
    return kvc.kvc_rotate_heads(rp or _rp(), stream=0, check=False, **a)


@no_gpu
@pytest.mark.parametrize("over,status", [
    (dict(dtype=7), "DTYPE"), (dict(n_tokens=-1), "SHAPE"), (dict(n_tokens=(1 << 30) + 1), "SHAPE"),
    (dict(n_q_heads=-1), "SHAPE"), (dict(n_q_heads=0, n_kv_heads=0), "SHAPE"),
    (dict(n_q_heads=65536), "SHAPE"), (dict(d=63), "UNSUPPORTED"), (dict(d=258), "UNSUPPORTED"),
    (dict(d=0), "UNSUPPORTED"), (dict(rot_dim=66), "SHAPE"), (dict(rot_dim=5), "SHAPE"),
    (dict(rot_dim=-2), "SHAPE"), (dict(interleaved=2), "INVALID_ARGUMENT"),
    (dict(norm=-1), "INVALID_ARGUMENT"), (dict(norm=1, eps=-1.0), "INVALID_ARGUMENT"),
    (dict(norm=1, eps=math.nan), "INVALID_ARGUMENT"), (dict(amplitude=math.inf), "INVALID_ARGUMENT"),
    (dict(q_s_head=63), "SHAPE"), (dict(k_s_tok=60), "SHAPE"), (dict(k_out_s_tok=-128), "SHAPE"),
    (dict(q_out_s_tok=1 << 40), "UNSUPPORTED"),
])
def test_descriptor_refusals(over, status):
    assert _call(_rp(**over)) == getattr(kvc, "KVC_ERR_" + status)


@no_gpu
def test_pointer_refusals():
    for n in ("q", "k", "positions", "turns", "q_out", "k_out"):
        assert _call(**{n: None}) == kvc.KVC_ERR_INVALID_ARGUMENT, n
        assert n in kvc.lib.kvc_last_error().decode()
        assert _call(**{n: FAKE + 20 * FAR + 1}) == kvc.KVC_ERR_ALIGNMENT, n
    assert _call(turns=FAKE + 3 * FAR + 4) == kvc.KVC_ERR_ALIGNMENT
    assert _call(w_q=FAKE + 6 * FAR) == kvc.KVC_ERR_INVALID_ARGUMENT          # no norm
    assert _call(_rp(norm=1), w_k=FAKE + 6 * FAR + 1) == kvc.KVC_ERR_ALIGNMENT
    assert kvc.lib.kvc_rotate_heads(None, *[None] * 9) == kvc.KVC_ERR_INVALID_ARGUMENT
    assert _call(_rp(n_tokens=0), q=None, positions=None) == kvc.KVC_OK


@no_gpu
def test_overlaps():
    for over in (dict(q_out=FAKE + 128), dict(k_out=FAKE + FAR - 128), dict(q_out=FAKE + FAR),
                 dict(k_out=FAKE + 4 * FAR + 64), dict(q_out=FAKE + 2 * FAR + 36),
                 dict(k_out=FAKE + 3 * FAR + 248)):
        assert _call(**over) == kvc.KVC_ERR_ALIAS, over
    # the same address with other strides is not in place
    assert _call(_rp(q_out_s_tok=512), q_out=FAKE) == kvc.KVC_ERR_ALIAS
    # parts of one projection: outputs over the values are other elements, over the keys not
    p = _rp(q_s_tok=512, k_s_tok=512, q_out_s_tok=512, k_out_s_tok=512, n_q_heads=4)
    at = lambda head: FAKE + 2 * 64 * head  # noqa: E731
    assert _call(p, q=at(0), k=at(4), q_out=at(1), k_out=FAKE + 5 * FAR) == kvc.KVC_ERR_ALIAS
    assert _call(p, q=at(0), k=at(4), q_out=FAKE + 4 * FAR, k_out=at(5)) == kvc.KVC_ERR_ALIAS
    assert _call(p, q=at(0), k=at(4), q_out=at(0), k_out=at(3)) == kvc.KVC_ERR_ALIAS
    # shifted by a token the last rows would be the next token's
    assert _call(p, q=at(0), k=at(4), q_out=FAKE + 4 * FAR, k_out=at(7)) == kvc.KVC_ERR_ALIAS


def _shared(a, b, row, N):
    """Whether two of a byte's rows are the same one, by looking at all of them."""
    (p, heads, s_tok, s_head), (p2, heads2, s_tok2, s_head2) = a, b
    mine = {p + t * s_tok + h * s_head + i for t in range(N) for h in range(heads) for i in range(row)}
    return any(p2 + t * s_tok2 + h * s_head2 + i in mine
               for t in range(N) for h in range(heads2) for i in range(row))


@no_gpu
@pytest.mark.parametrize("N", [1, 2, 5])
def test_heads_that_alternate(N):
    """In place where the heads of queries, keys and values take turns in a token's row, or in
    planes of their own with the tokens inside."""
    def try_(q, k, q_tok, q_head, k_tok, k_head, heads=4, kv=4, **out):
        p = _rp(n_tokens=N, n_q_heads=heads, n_kv_heads=kv, q_s_tok=q_tok, q_s_head=q_head, k_s_tok=k_tok,
                k_s_head=k_head, q_out_s_tok=q_tok, q_out_s_head=q_head, k_out_s_tok=k_tok, k_out_s_head=k_head)
        a = dict(q=FAKE + 2 * q, k=FAKE + 2 * k, q_out=FAKE + 2 * q, k_out=FAKE + 2 * k)
        a.update(out)
        return _call(p, **a)
    went_on = kvc.KVC_ERR_CUDA                               # to the launch, which finds no GPU
    assert try_(0, 64, 768, 192, 768, 192) == went_on        # [N, heads, 3, d]
    assert try_(64, 0, 768, 192, 768, 192) == went_on
    assert try_(0, 7 * 64, 4 * 576, 576, 4 * 576, 576) == went_on          # [N, H, group + 2, d]
    assert try_(0, 64, 64, 3 * 64 * N, 64, 3 * 64 * N) == (went_on if N == 1 else kvc.KVC_ERR_ALIAS)
    assert try_(0, 64 * N, 64, 3 * 64 * N, 64, 3 * 64 * N) == went_on      # [heads, 3, N, d]
    assert try_(0, 64, 768, 192, 768, 768, kv=1) == went_on  # one key head beside many
    assert try_(0, 128, 768, 192, 768, 768, kv=1) == went_on
    # keys in every second gap; at the queries' places; half a row off
    assert try_(0, 64, 768, 192, 768, 384, kv=2) == went_on
    assert try_(0, 192, 768, 192, 768, 384, kv=2) == kvc.KVC_ERR_ALIAS
    assert try_(0, 96, 768, 192, 768, 192, kv=3) == went_on
    assert try_(0, 32, 768, 192, 768, 192) == kvc.KVC_ERR_ALIAS
    assert try_(0, 160, 768, 192, 768, 192, kv=3) == kvc.KVC_ERR_ALIAS


@no_gpu
def test_overlaps_of_all_small_layouts():
    """No call that shares a byte passes, and none without one is refused where the heads'
    strides are alike or the tokens' rows apart."""
    import itertools
    N, row = 3, 4                                            # bytes: 2 elements of bf16
    refused = passed = 0
    for q_tok, q_head, k_tok, k_head, off, (hq, hk) in itertools.product(
            (2, 6, 14), (2, 4, 8), (2, 6, 14), (2, 4, 8), range(-16, 18, 1), ((2, 2), (1, 2), (3, 1))):
        p = _rp(n_tokens=N, n_q_heads=hq, n_kv_heads=hk, d=2, rot_dim=2, q_s_tok=64, q_s_head=8, k_s_tok=k_tok,
                k_s_head=k_head, q_out_s_tok=q_tok, q_out_s_head=q_head, k_out_s_tok=64, k_out_s_head=8)
        st = _call(p, q=FAKE + FAR, k=FAKE + 2 * off, q_out=FAKE, k_out=FAKE + 6 * FAR)
        a, b = (0, hq, 2 * q_tok, 2 * q_head), (2 * off, hk, 2 * k_tok, 2 * k_head)
        own = len({x + t * q_tok + h * q_head for t in range(N) for h in range(hq) for x in range(2)}) < 2 * N * hq
        if own:                                              # rows of the output itself
            continue
        if _shared(a, b, row, N):
            assert st == kvc.KVC_ERR_ALIAS, (a, b)
            refused += 1
        elif q_tok == k_tok and ((hq - 1) * q_head < q_tok - 1 and (hk - 1) * k_head < k_tok - 1):
            assert st == kvc.KVC_ERR_CUDA, (a, b)
            passed += 1
    assert refused > 100 and passed > 100


@no_gpu
def test_outputs_whose_rows_overlap():
    """Two rows of an output at the same bytes would be written by two CTAs."""
    N, heads, d = 3, 3, 4
    seen = set()
    for s_tok in range(d, 30):
        for s_head in range(d, 30):
            rows = sorted(t * s_tok + h * s_head for t in range(N) for h in range(heads))
            want = kvc.KVC_ERR_CUDA if all(b - a >= d for a, b in zip(rows, rows[1:])) else kvc.KVC_ERR_ALIAS
            for x in "qk":
                p = _rp(n_tokens=N, n_q_heads=heads, n_kv_heads=heads, d=d, rot_dim=d, q_s_tok=12, q_s_head=4,
                        k_s_tok=12, k_s_head=4, q_out_s_tok=12, q_out_s_head=4, k_out_s_tok=12, k_out_s_head=4)
                setattr(p, x + "_out_s_tok", s_tok)
                setattr(p, x + "_out_s_head", s_head)
                assert _call(p) == want, (s_tok, s_head)
            seen.add(want)
    assert len(seen) == 2
    # one token or one head: nothing to fold; the inputs may
    assert _call(_rp(n_tokens=1, q_out_s_tok=64)) == _call(_rp(n_q_heads=1, q_out_s_head=0)) == kvc.KVC_ERR_CUDA
    assert _call(_rp(q_s_tok=64)) == kvc.KVC_ERR_CUDA
    assert _call(_rp(q_out_s_tok=64)) == kvc.KVC_ERR_ALIAS
    # tokens within heads
    assert _call(_rp(q_out_s_head=640, q_out_s_tok=64)) == kvc.KVC_ERR_CUDA


def test_binding_refusals():
    q, k = torch.zeros((5, 4, 64)), torch.zeros((5, 2, 64))
    ok = kvc.rotary_params(q, k, q, k, 64)
    assert (ok.n_q_heads, ok.n_kv_heads, ok.q_s_tok, ok.k_out_s_tok, ok.dtype) == (4, 2, 256, 128, kvc.KVC_F32)
    for a in ((q, k, q, None), (None, None, None, None), (q, k, q[:4], k), (q, k[:4], q, k[:4]),
              (q, k[..., :32], q, k[..., :32]), (q.half(), None, q.half(), None),
              (q, k.double(), q, k.double()), (q[0], None, q[0], None),
              (q.transpose(1, 2), None, q.transpose(1, 2), None), (q, k, q.to("meta"), k)):
        with pytest.raises(ValueError):
            kvc.rotary_params(*a, 32)
