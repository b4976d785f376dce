"""Paged attention where the values, the mask or the table are at a limit of what a
call takes, against the float64 oracle (tolerances: test_gpu_paged).

A value row with an infinity gives every row that sees it the infinity of the formula,
sum_j p_j v_j with p_j > 0: its sign in that column, NaN where infinities of both signs
are seen.  The scores here are within 30 of one another, so that no p_j underflows."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

from .test_gpu_paged import FEW, Batch

pytestmark = pytest.mark.gpu

CHUNKS = [(40, 200), (1, 77), (130, 131), (3, 3), (1, 1), (0, 9)]


def _key(b, r, j):
    """(page, row) of key j of request r."""
    return b.table[r, j // b.B], j % b.B


def _sees(b, r, j, causal, window):
    """[N] bool: the rows that see key j of request r."""
    seen = np.zeros(b.N, dtype=bool)
    n, kv = b.lens[r]
    for i in range(n):
        p = kv - n + i
        seen[b.q_start[r] + i] = (not causal or j <= p) and (not window or j > p - window)
    return seen


@pytest.mark.parametrize("lens", [FEW, CHUNKS], ids=["few", "chunks"])
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("G", [1, 2, 12])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 30)])
def test_infinite_values_in_sight(lens, dtype, d, G, causal, window):
    b = Batch(lens, 2 * G, 2, d, 20, dtype, seed=G)
    want = np.zeros((b.N, 2 * G, d))               # infinities of each sign that a row sees
    minus = np.zeros_like(want)
    for r, (_, kv) in enumerate(b.lens):
        for j, head, col, sign in [(0, 0, 0, 1), (kv // 2, 0, 3, -1), (kv - 1, 0, d - 1, 1),
                                   (kv // 3, 1, 7, 1), (2 * kv // 3, 1, 7, -1),
                                   (kv - 1, 1, 8, -1)]:
            if not 0 <= j < kv:
                continue
            page, row = _key(b, r, j)
            b.host[1][page, 0, head, row, col] = 0.0
            if not b.V[page, 0, head, row, col].isinf():
                b.V[page, 0, head, row, col] = sign * float("inf")
                seen = _sees(b, r, j, causal, window)
                to = want if sign > 0 else minus
                to[seen, head * G:head * G + G, col] = 1
    plus, minus = torch.from_numpy(want).cuda() > 0, torch.from_numpy(minus).cuda() > 0
    b.run(causal, window)
    got = b.out.clone()
    assert got[plus & minus].isnan().all()
    assert (got[plus & ~minus] == float("inf")).all()
    assert (got[minus & ~plus] == float("-inf")).all()
    b.V.copy_(b.host[1])
    b.run(causal, window)
    b.out.copy_(torch.where(plus | minus, b.out, got))   # the rest is what it is without them
    b.check(causal, window)


@pytest.mark.parametrize("lens", [FEW, CHUNKS], ids=["few", "chunks"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_odd_keys_in_sight(lens, d, value):
    """A score of -inf has no weight, one of +inf or NaN no softmax."""
    G = 2
    b = Batch(lens, 2 * G, 2, d, 20, "bf16", seed=5)
    r, j = 1, 0
    page, row = _key(b, r, j)
    b.K[page, 0, 0, row, 2] = value
    b.run()
    got = b.out.clone()
    rows = torch.from_numpy(_sees(b, r, j, True, 0)).cuda()
    up = b.q[:, :G, 2].float() * value
    bad = torch.zeros(b.N, 2 * G, dtype=torch.bool, device="cuda")
    bad[:, :G] = rows[:, None] & ~(up == float("-inf"))
    assert got[bad].isnan().all() and got[~bad].isfinite().all()
    other = ~rows[:, None].expand(-1, 2 * G).clone()     # what does not see it
    other[:, G:] = True
    b.K.copy_(b.host[0])
    b.run()
    b.out.copy_(torch.where(other[:, :, None], got, b.out))
    b.check()


@pytest.mark.parametrize("dtype,d,G", [("bf16", 64, 1), ("bf16", 128, 1), ("bf16", 128, 4),
                                       ("bf16", 64, 12), ("f32", 64, 1), ("f32", 80, 4)])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 300, 2 ** 30, 2 ** 30 - 1])
@pytest.mark.parametrize("lens", [[(9, 4), (6, 2), (1, 700)] + [(0, 3)] * 20,
                                  [(9, 4), (300, 10), (700, 200), (1, 700), (40, 400)]],
                         ids=["few", "chunks"])
def test_windows_longer_than_any_context(dtype, d, G, window, lens):
    """Also with more new tokens than keys, whose first positions are negative."""
    b = Batch(lens, 2 * G, 2, d, 16, dtype, seed=G)
    b.run(True, window)
    b.check(True, window)


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("B", [8, 16, 48, 130])
@pytest.mark.parametrize("lens", [[(1, 900), (2, 700), (0, 5), (1, 50)],
                                  [(40, 900), (1, 700), (150, 800), (3, 40)]],
                         ids=["few", "chunks"])
def test_pages_behind_the_window_are_not_in_use(dtype, d, B, lens):
    """A serving program may give them back: their entries mean nothing."""
    window = 100
    b = Batch(lens, 4, 2, d, B, dtype, seed=B)
    gone = 0
    for r, (n, kv) in enumerate(lens):
        first = max(0, kv - n - window + 1) if n else kv          # the first key that a row sees
        for k, junk in zip(range(first // B), [-1, b.P, 2 ** 31 - 1, -2 ** 31] * 30):
            b.d_table[r, k] = junk
            gone += 1
    assert gone > 5
    b.run(True, window)
    b.check(True, window)                          # with the status
    # an entry in sight is reported
    b.d_table[0, (lens[0][1] - 1) // B] = b.P
    b.run(True, window)
    torch.cuda.synchronize()
    from agent_shared_context_gb300 import kvc
    assert int(b.status.item()) == kvc.KVC_ERR_SHAPE


@pytest.mark.parametrize("d,B", [(64, 16), (128, 16), (128, 48), (64, 130)])
@pytest.mark.parametrize("window", [130, 400])
def test_infinities_along_a_window(d, B, window):
    """One key in thirty holds an infinity, so that most tiles at the edges of sight have
    value rows that some rows see and others do not; call after call with the same bits."""
    lens = [(700, 3000), (150, 900), (33, 300), (1, 500)]
    G = 4
    b = Batch(lens, 2 * G, 2, d, B, "bf16", seed=B)
    rng = np.random.RandomState(d + B)
    plus = np.zeros((b.N, 2 * G, d), dtype=bool)
    for r, (n, kv) in enumerate(lens):
        for j in np.flatnonzero(rng.rand(kv) < 1 / 30):
            page, row = _key(b, r, j)
            head, col = rng.randint(2), rng.randint(d)
            b.host[1][page, 0, head, row, col] = 0.0
            b.V[page, 0, head, row, col] = float("inf")
            plus[_sees(b, r, j, True, window), head * G:head * G + G, col] = True
    plus = torch.from_numpy(plus).cuda()
    assert 0.01 < plus.float().mean() < 0.5
    b.run(True, window)
    got = b.out.clone()
    assert (got[plus] == float("inf")).all()
    for _ in range(20):
        b.run(True, window)
        assert torch.equal(got, b.out)
    b.V.copy_(b.host[1])
    b.run(True, window)
    b.out.copy_(torch.where(plus, b.out, got))
    b.check(True, window)


@pytest.mark.parametrize("lens", [FEW, CHUNKS], ids=["few", "chunks"])
@pytest.mark.parametrize("low,high", [(-125, -116), (-149, -127)])
def test_f32_tiny_factors(lens, low, high):
    """Keys of 2^low .. 2^high.  From 2^-126 on a product is off by at most 2^-10 of
    itself, and smaller factors may count as zeros: a score is off by 2^-10 E, or by E,
    besides what it is off by elsewhere."""
    b = Batch(lens, 4, 2, 64, 16, "f32", seed=8)
    g = torch.Generator().manual_seed(2)
    K, q = b.host[0], b.host[2]
    size = torch.exp2(torch.rand(K.shape, generator=g, dtype=torch.float64) * (high - low) + low)
    K.copy_(torch.where(K.isnan(), K, torch.copysign(size.float(), K)))
    q.mul_(2.0 ** 119)
    b.K.copy_(K), b.q.copy_(q)
    b.run()
    n64 = lambda t: t.double().numpy()  # noqa: E731
    o, z, A, E = PO.paged_attention(n64(q), n64(K), n64(b.host[1]), b.table, b.q_start,
                                    [kv for _, kv in lens], 64 ** -0.5)
    torch.cuda.synchronize()
    n = max(kv for _, kv in lens)
    ds = ((2.0 ** -10 if low >= -126 else 1.0) + (64 + 16) * 2.0 ** -24) * E
    off = np.abs(b.out.cpu().double().numpy() - o)
    assert (off <= (np.expm1(2 * ds[:, :, None]) + (n + 4) * 2.0 ** -24) * A
            + 2.0 ** -23 * np.abs(o)).all()
    off = np.abs(b.lse.cpu().double().numpy() - z)
    assert (off <= ds + (n + 4) * 2.0 ** -24 + 2.0 ** -23 * np.abs(z)).all()
