"""Paged caches on the GPU against the float64 oracle: the plan (whole
numbers, exact), the write (bit-exact) and the attention.

Attention tolerances, per output element.  With A = sum_j p_j |v_j| and
E = max_j scale sum_i |q_i k_ij| (both from the oracle) and n keys in sight:
  * a score is a sum of d products in fp32, off by at most (d + 16) 2^-24 E
    =: s (16 covers the scale, the shift by the maximum and exp2), so every
    p_j is off by a factor exp(2 s) at most and lse by s + (n + 4) 2^-24;
  * sums over the keys run in fp32: (n + 4) 2^-24 A;
  * bf16 only: probabilities rounded for the product with V, 2^-9 A, and the
    result rounded once, 2^-9 |out|; f32 rounds the result by 2^-24.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _kvc():
    from agent_shared_context_gb300 import kvc
    return kvc


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _np(t):
    return t.detach().cpu().double().numpy()


class Batch:
    """Pools, tables and queries of a batch of requests ``lens`` = [(new, kv)]."""

    def __init__(self, lens, Hq, H, d, B, dtype="bf16", seed=0, L=1, layer=0, stale=float("nan"),
                 layout="plain", spare=2, qscale=2.0):
        g = torch.Generator().manual_seed(seed)
        dt = DT[dtype]
        self.lens, self.Hq, self.H, self.d, self.B, self.dtype = lens, Hq, H, d, B, dtype
        self.layer, self.L = layer, L
        R = len(lens)
        blocks = [-(-kv // B) for _, kv in lens]
        self.P = sum(blocks) + spare
        self.width = max(max(blocks), 1)
        perm = torch.randperm(self.P, generator=g).tolist()
        table = np.full((R, self.width), -7, dtype=np.int64)      # entries beyond a row mean nothing
        pools = []
        for _ in "KV":
            x = torch.randn((self.P, L, H, B, d), generator=g).to(dt)
            pools.append(x)
        used = torch.zeros((self.P, B), dtype=torch.bool)
        at = 0
        for r, (_, kv) in enumerate(lens):
            for b in range(blocks[r]):
                table[r, b] = perm[at]
                used[perm[at], :max(0, min(B, kv - b * B))] = True
                at += 1
        for x in pools:                                            # rows that no request holds
            x.masked_fill_(~used[:, None, None, :, None], stale)
        self.table = table
        self.q_start = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
        self.N = int(self.q_start[-1])
        q = (qscale * torch.randn((self.N, Hq, d), generator=g)).to(dt)
        self.host = (pools[0], pools[1], q)
        if layout == "plain":
            self.K, self.V = pools[0].cuda(), pools[1].cuda()
            self.q = q.cuda()
            self.out = torch.full_like(self.q, 3.0)
        else:
            # token-major pages with K and V side by side, q a slice of a fused projection,
            # out in a head-major buffer
            both = torch.stack([p.permute(0, 3, 1, 2, 4) for p in pools], dim=1).contiguous().cuda()
            self.K = both[:, 0].permute(0, 2, 3, 1, 4)
            self.V = both[:, 1].permute(0, 2, 3, 1, 4)
            fused = torch.zeros((self.N, Hq + 2 * H, d), dtype=dt, device="cuda")
            fused[:, H:H + Hq] = q.cuda()
            self.q = fused[:, H:H + Hq]
            self.out = torch.full((Hq, self.N, d), 3.0, dtype=dt, device="cuda").permute(1, 0, 2)
        self.lse = torch.full((self.N, Hq), 3.0, device="cuda")
        self.d_table = torch.from_numpy(table).to(torch.int32).cuda()
        self.d_start = _i32(self.q_start.tolist())
        self.d_kv = _i32([kv for _, kv in lens])
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kvc = _kvc()
        self.pg = kvc.paged(self.P, B, L, H, d, dtype, R, self.width)
        at_ = kvc.attn_params(self.q, self.out, layer)
        n = kvc.kvc_paged_attention_workspace(self.pg, at_)
        self.ws = torch.zeros(n, dtype=torch.uint8, device="cuda")

    def run(self, causal=True, window=0, scale=None, lse=True, stream=None):
        kvc = _kvc()
        at = kvc.attn_params(self.q, self.out, self.layer, scale=scale or self.d ** -0.5,
                             causal=causal, window=window)
        kvc.kvc_paged_attention(self.pg, at, self.q, self.K, self.V, self.d_table, self.d_start,
                                self.d_kv, self.out, self.ws, self.status,
                                lse=self.lse if lse else None, stream=stream)

    def check(self, causal=True, window=0, scale=None, lse=True):
        K, V, q = (_np(t) for t in self.host)
        s = scale or self.d ** -0.5
        o, z, A, E = PO.paged_attention(q, K, V, self.table, self.q_start, [kv for _, kv in self.lens],
                                        s, self.layer, causal, window)
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        assert not self.ws[:8192].any(), "the counters are left at zero"
        got = _np(self.out)
        n = max([kv for _, kv in self.lens] + [1])
        ds = (self.d + 16) * 2.0 ** -24 * E[:, :, None]
        tol = (np.expm1(2 * ds) + (n + 4) * 2.0 ** -24) * A
        tol += 2.0 ** -9 * (1.01 * A + 1.01 * np.abs(o)) if self.dtype == "bf16" else 2.0 ** -23 * np.abs(o)
        bad = ~(np.abs(got - o) <= tol)
        assert not bad.any(), "%d of %d rows, first %s: %s against %s, off by %g of the tolerance" % (
            bad.any(-1).sum(), bad.shape[0] * bad.shape[1], np.argwhere(bad)[0],
            got[bad][:3], o[bad][:3], np.nanmax(np.abs(got - o)[bad] / np.maximum(tol[bad], 1e-30)))
        if lse:
            gl = _np(self.lse)
            empty = np.isneginf(z)
            assert np.array_equal(np.isneginf(gl), empty)
            off = np.abs(np.where(empty, 0, gl) - np.where(empty, 0, z))
            assert (off <= ds[:, :, 0] + (n + 4) * 2.0 ** -24
                    + 2.0 ** -23 * np.abs(np.where(empty, 0, z))).all()


RAGGED = [(1, 1), (0, 0), (3, 130), (1, 259), (0, 40), (17, 17), (70, 333), (2, 64), (1, 128)]


@pytest.mark.parametrize("B", [1, 7, 8, 16, 20, 48, 64, 100, 128, 130, 256, 1000])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_attention_page_sizes(dtype, d, B):
    b = Batch(RAGGED, 8, 2, d, B, dtype, seed=B)
    b.run()
    b.check()


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8, 16, 33, 64])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_head_groups(dtype, G):
    b = Batch([(40, 200), (1, 150), (5, 5), (2, 129)], 2 * G, 2, 64, 16, dtype, seed=G)
    b.run()
    b.check()


@pytest.mark.parametrize("d", [4, 20, 64, 68, 80, 128, 132, 192, 256])
def test_attention_f32_head_dims(d):
    b = Batch([(40, 200), (1, 150), (5, 70)], 4, 2, d, 16, "f32", seed=d)
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 80)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 17), (True, 128), (True, 300)])
def test_attention_masks(dtype, d, causal, window):
    b = Batch(RAGGED + [(300, 700), (1, 900)], 8, 2, d, 32, dtype, seed=window)
    b.run(causal, window)
    b.check(causal, window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rows_that_see_nothing(dtype):
    """More new tokens than keys: the first rows have negative positions."""
    lens = [(5, 0), (9, 4), (300, 10), (1, 0), (200, 199)]
    for causal in (True, False):
        b = Batch(lens, 4, 1, 64, 16, dtype, seed=5)
        b.run(causal)
        b.check(causal)


@pytest.mark.parametrize("dtype,d,layout", [("bf16", 128, "fused"), ("bf16", 64, "fused"), ("f32", 64, "fused")])
def test_attention_strides_and_layers(dtype, d, layout):
    b = Batch(RAGGED + [(150, 600)], 12, 4, d, 24, dtype, seed=3, L=3, layer=2, layout=layout)
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("lens", [
    [(1, 5000)],                                  # one decode, divided over many CTAs
    [(2, 4097), (1, 1)],
    [(700, 3000)],                                # a chunk, several row tiles
    [(1, 50 + 37 * i) for i in range(40)],        # ragged decodes
    [(1, 400)] * 300 + [(0, 0)] * 20 + [(33, 90)],
])
def test_attention_divided_work(dtype, d, lens):
    b = Batch(lens, 4, 2, d, 64, dtype, seed=len(lens))
    b.run()
    b.check()
    first = b.out.clone(), b.lse.clone()
    b.out.zero_()
    b.run()                                       # the same bits again: no order of arrival in them
    torch.cuda.synchronize()
    assert torch.equal(first[0], b.out) and torch.equal(first[1], b.lse)


# at most one new token per request on average: the decoding kernel
DECODE = [(1, 1), (0, 70), (1, 33), (3, 130), (0, 0), (1, 259), (0, 5), (1, 128), (2, 700), (0, 1),
          (0, 0), (1, 1025)]


@pytest.mark.parametrize("B", [1, 7, 16, 48, 64, 128, 130, 1000])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 100)])
def test_decode_page_sizes_and_masks(d, B, causal, window):
    b = Batch(DECODE, 8, 2, d, B, "bf16", seed=B + window)
    b.run(causal, window)
    b.check(causal, window)


@pytest.mark.parametrize("G", [1, 3, 4, 7, 8, 16])
def test_decode_head_groups(G):
    b = Batch(DECODE, 3 * G, 3, 128, 32, "bf16", seed=G, L=2, layer=1, layout="fused")
    b.run()
    b.check()


def test_decode_one_request_among_idle_ones():
    """A chunk of 60 tokens and 70 requests without any: many row tiles of the same request."""
    b = Batch([(60, 500)] + [(0, 9)] * 70, 8, 2, 64, 16, "bf16", seed=2)
    b.run()
    b.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_decode_values_out_of_sight(d, value):
    """As test_attention_values_out_of_sight, for a request with four tokens."""
    b = Batch([(4, 200), (0, 0), (0, 3), (1, 77)], 4, 2, d, 16, "bf16", seed=4)
    page, off = b.table[0, 199 // b.B], 199 % b.B
    b.V[page, 0, :, off] = value
    b.run()
    torch.cuda.synchronize()
    assert not b.out[3].isfinite().any()          # the last token sees it
    b.V.copy_(b.host[1])
    got = b.out.clone()
    b.run()
    torch.cuda.synchronize()
    got[3] = b.out[3]
    b.out.copy_(got)
    b.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_large_and_shifted_scores(dtype):
    """Scores of +-100 that grow along the keys: the running maximum moves in every tile."""
    b = Batch([(1, 1000), (130, 900)], 4, 2, 64, 16, dtype, seed=9)
    ramp = torch.linspace(-1, 1, b.P * b.B).view(b.P, 1, 1, b.B, 1)
    K = b.host[0]
    q = b.host[2]
    K[..., 0] = torch.where(K[..., 0].isnan(), K[..., 0], (100 * ramp[..., 0]).to(K.dtype))
    q[..., 0] = 8.0
    b.K.copy_(K)
    b.q.copy_(q)
    b.run()
    b.check()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attention_values_out_of_sight(dtype, d, value):
    """A key beyond a row's sight adds nothing, whatever its key and value rows hold."""
    lens = [(40, 200), (1, 77), (130, 131)]
    b = Batch(lens, 4, 2, d, 16, dtype, seed=4)
    r, last = 0, 199                              # the last token of request 0
    page, off = b.table[r, last // b.B], last % b.B
    for x, host in ((b.K, b.host[0]), (b.V, b.host[1])):
        x[page, 0, :, off] = value
    b.run()
    torch.cuda.synchronize()
    sees = int(b.q_start[1]) - 1                  # only the last row of the request sees it
    got = b.out.clone()
    assert not got[sees].isfinite().all()
    keep = b.out[sees].clone()
    for x, host in ((b.K, b.host[0]), (b.V, b.host[1])):
        x.copy_(host)
    b.out.fill_(3.0)
    b.run()
    torch.cuda.synchronize()
    got[sees] = b.out[sees]
    b.out.copy_(got)
    b.lse[sees] = b.lse[sees]
    b.check()
    assert not keep.isfinite().all()


def test_attention_offsets_beyond_32_bits():
    """Pages whose elements lie more than 2^31 elements into the pool."""
    kvc = _kvc()
    H, d, B, L = 2, 128, 128, 8
    P = (1 << 32) // (L * H * B * d) + 5          # over 2^32 elements, 8.6 GB a pool
    b = Batch([(3, 300), (1, 513)], 8, H, d, B, "bf16", seed=1)
    big = [torch.empty((P, L, H, B, d), dtype=torch.bfloat16, device="cuda") for _ in "KV"]
    move = np.array([P - 1 - 7 * p for p in range(b.P)])
    for x, y in zip(big, (b.K, b.V)):
        for p in range(b.P):
            x[move[p], L - 1] = y[p, 0]
    b.K, b.V, b.layer, b.L, b.P = big[0], big[1], L - 1, L, P
    b.d_table = torch.from_numpy(np.where(b.table >= 0, move[b.table.clip(0)], -7)).to(torch.int32).cuda()
    b.pg = kvc.paged(P, B, L, H, d, "bf16", 2, b.width)
    b.run()
    b.layer = 0
    b.check()
    slots = torch.tensor([[int(move[0]) * B + 5, (P - 1) * B + B - 1]], device="cuda")
    src = [torch.randn((1, L, H, 2, d), device="cuda").bfloat16() for _ in "KV"]
    kvc.kvc_page_write(b.pg, src[0], src[1], slots, big[0], big[1])
    for x, s in zip(big, src):
        assert torch.equal(x[move[0], :, :, 5], s[0, :, :, 0])
        assert torch.equal(x[P - 1, :, :, B - 1], s[0, :, :, 1])


def test_attention_rows_of_no_request_stay():
    b = Batch([(3, 30), (2, 90)], 4, 2, 64, 16, "bf16", seed=8)
    b.d_start = _i32([0, 3, 4])                   # the last row belongs to nobody
    b.run()
    torch.cuda.synchronize()
    assert (b.out[4] == 3).all() and (b.lse[4] == 3).all()
    assert not (b.out[:4] == 3).all(-1).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_reports_tables_out_of_range(dtype):
    kvc = _kvc()
    for what in ("page", "kv", "start"):
        b = Batch([(3, 30), (2, 90)], 4, 2, 64, 16, dtype, seed=8, stale=0.0)
        if what == "page":
            b.d_table[1, 2] = b.P
        elif what == "kv":
            b.d_kv[1] = b.width * b.B + 1
            b.d_table.clamp_(min=0)
        else:
            b.d_start[2] = b.N + 1
        b.run()
        torch.cuda.synchronize()
        assert int(b.status.item()) == kvc.KVC_ERR_SHAPE, what
        assert not b.ws[:8192].any()


def test_attention_on_a_side_stream_and_in_a_graph():
    b = Batch([(1, 600), (1, 90), (4, 333)], 8, 2, 128, 16, "bf16", seed=12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run()
    side.synchronize()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run()
    b.lens = [(1, 512), (1, 17), (4, 200)]        # other lengths, the same captured call
    b.d_kv.copy_(_i32([kv for _, kv in b.lens]))
    b.out.zero_()
    graph.replay()
    b.check()


def test_attention_without_tokens_or_requests():
    kvc = _kvc()
    b = Batch([(0, 30), (0, 0)], 4, 2, 64, 16, "bf16", seed=8)
    b.run()
    torch.cuda.synchronize()
    assert int(b.status.item()) == 0
    assert kvc.KVC_OK == 0


# -------------------------------------------------------------------- plan
def _plan(B, new, kv, table, free, n_free, max_tokens, P):
    kvc = _kvc()
    R, width = table.shape
    d_table = torch.from_numpy(table).to(torch.int32).cuda()
    d_free = torch.from_numpy(free).to(torch.int32).cuda()
    e = lambda n, dt=torch.int32: torch.full((n,), 99, dtype=dt, device="cuda")  # noqa: E731
    out = dict(kv_lens=e(R), n_free=e(1), q_start=e(R + 1), slots=e(max_tokens, torch.int64),
               positions=e(max_tokens), status=e(R))
    d_new, d_kv, d_n = _i32(new), _i32(kv), _i32([n_free])
    pg = kvc.paged(P, B, 1, 1, 64, "bf16", R, width)
    res = []
    for _ in range(2):                            # repeating the call repeats its result
        kvc.kvc_page_plan(pg, d_new, d_kv, out["kv_lens"], d_table, d_free, d_n, out["n_free"],
                          out["q_start"], out["slots"], out["positions"], out["status"])
        torch.cuda.synchronize()
        res.append({k: v.cpu().numpy().copy() for k, v in
                    dict(out, block_table=d_table, free_pages=d_free).items()})
    for k in res[0]:
        assert np.array_equal(res[0][k], res[1][k]), k
    assert torch.equal(d_new, _i32(new)) and torch.equal(d_kv, _i32(kv))
    return res[0]


def _check_plan(B, new, kv, table, free, n_free, max_tokens, P):
    got = _plan(B, new, kv, table, free, n_free, max_tokens, P)
    want = PO.page_plan(B, new, kv, table, free, n_free, max_tokens)
    for k, v in want.items():
        assert np.array_equal(got[k].reshape(np.shape(v)), v), k
    return want


@pytest.mark.parametrize("R", [1, 2, 31, 33, 512, 513, 1025, 4096])
@pytest.mark.parametrize("B", [1, 16, 20, 128])
def test_plan_random(R, B):
    rng = np.random.RandomState(R + B)
    refused = set()
    for trial in range(4):
        kv = rng.randint(0, 6 * B + 2, R)
        new = rng.randint(0, 3 * B + 2, R)
        new[rng.rand(R) < 0.2] = -1
        new[rng.rand(R) < 0.1] = 0
        width = -(-(int(kv.max()) + int(new.max()) + 1) // B) - (trial == 1)
        if trial == 3:
            width = width // 2                    # many rows full
        kv = np.minimum(kv, width * B)
        if trial == 1 and R > 3:
            new[R // 2] = -2
            kv[R // 3] = -1
            kv[R // 4] = width * B + 1
        table = np.full((R, max(width, 1)), -9, dtype=np.int64)
        held = [-(-int(c) // B) if 0 <= c <= width * B else 0 for c in kv]
        need = sum(max(0, -(-(int(c) + max(int(n), 0)) // B) - h) for c, n, h in zip(kv, new, held))
        back = sum(h for h, n in zip(held, new) if n == -1)
        n_free = max(0, need - back + (3 if trial < 2 else -(need // 4 + 1)))
        P = sum(held) + n_free + 2
        perm = rng.permutation(P)
        at = 0
        for r in range(R):
            table[r, :held[r]] = perm[at:at + held[r]]
            at += held[r]
        free = np.full(P, -5, dtype=np.int64)
        free[:n_free] = perm[at:at + n_free]
        total = int(sum(max(0, n) for n in new))
        want = _check_plan(B, new.tolist(), kv.tolist(), table, free, n_free,
                           total + 5 if trial == 0 else max(0, total - total // 7), P)
        refused |= set(want["status"].tolist())
    if R > 500:
        assert refused == {0, 1, 2, 3, 4}


def test_plan_edges():
    z = np.zeros((1, 4), dtype=np.int64)
    f = np.arange(10, 18)
    _check_plan(16, [0], [0], z, f, 8, 0, 8)                    # nothing to do, no token buffers
    _check_plan(16, [64], [0], z, f, 4, 64, 8)                  # a row filled to its last slot
    _check_plan(16, [65], [0], z, f, 8, 65, 8)                  # one token too many
    _check_plan(16, [-1], [64], np.array([[3, 2, 1, 0]]), f, 0, 4, 8)
    two = np.array([[3, 2, 1, 0], [-1, -1, -1, -1]])
    _check_plan(16, [-1, 60], [50, 0], two, f, 0, 60, 8)        # the returned pages serve the next
    _check_plan(1 << 20, [1000000], [5], z[:, :2], f, 1, 1000000, 8)
    # lengths whose sum runs over 31 bits: only the requests that they belong to are refused
    huge = 2 ** 31 - 1
    four = np.full((4, 4), -1)
    _check_plan(16, [5, huge, huge, 0], [0, 0, 0, 0], four, f, 8, 40, 8)
    _check_plan(16, [5, 40, huge, 3], [0, 0, 0, 0], four, f, 8, 45, 8)
    _check_plan(16, [huge] * 600 + [3], [0] * 601, np.full((601, 2), -1), f, 8, 45, 8)
    _check_plan(16, [3] + [huge] * 600, [0] * 601, np.full((601, 2), -1), f, 8, 45, 8)


def test_plan_without_requests():
    kvc = _kvc()
    pg = kvc.paged(4, 16, 1, 1, 64, "bf16", 0, 4)
    n, n2, qs, free = _i32([3]), _i32([0]), _i32([7]), _i32([0, 1, 2, 3])
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    pos = _i32([0, 0, 0])
    kvc.kvc_page_plan(pg, None, None, None, None, free, n, n2, qs, slots, pos, None)
    torch.cuda.synchronize()
    assert n2.item() == 3 and qs.item() == 0
    assert slots.tolist() == [-1] * 3 and pos.tolist() == [-1] * 3


# ------------------------------------------------------------------- write
@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f32", 4), ("f32", 80), ("f32", 256)])
@pytest.mark.parametrize("n,T,nl,H,B", [(1, 1, 1, 1, 16), (3, 50, 2, 3, 7), (2, 129, 1, 8, 64), (1, 700, 3, 1, 1)])
def test_write_rows(dtype, d, n, T, nl, H, B):
    kvc = _kvc()
    g = torch.Generator().manual_seed(d + T)
    dt = DT[dtype]
    L, layer = nl + 2, 1
    P = -(-n * T // B) + 2
    pools = [torch.randn((P, L, H, B, d), generator=g).to(dt) for _ in "KV"]
    slots = torch.randperm(P * B, generator=g)[:n * T].view(n, T)
    slots[torch.rand((n, T), generator=g) < 0.2] = -1
    slots[0, 0] = P * B                            # out of the pool: skipped
    for packed in (False, True):
        src = [torch.randn((n, nl, T, H, d), generator=g).to(dt).permute(0, 1, 3, 2, 4) if packed
               else torch.randn((n, nl, H, T, d), generator=g).to(dt) for _ in "KV"]
        dev = [p.cuda() for p in pools]
        pg = kvc.paged(P, B, L, H, d, dtype, n, 1)
        kvc.kvc_page_write(pg, src[0].cuda() if not packed else src[0].permute(0, 1, 3, 2, 4).contiguous().cuda().permute(0, 1, 3, 2, 4),
                           src[1].cuda() if not packed else src[1].permute(0, 1, 3, 2, 4).contiguous().cuda().permute(0, 1, 3, 2, 4),
                           slots.cuda(), dev[0], dev[1], layer=layer)
        torch.cuda.synchronize()
        for p, s, x in zip(pools, src, dev):
            want = PO.page_write(s.float().numpy(), slots.numpy(), p.float().numpy(), layer)
            assert np.array_equal(x.float().cpu().numpy(), want)


def test_write_slots_beyond_31_bits():
    """Rows of 16 bytes: over 2^31 slots in 34 GB a pool."""
    kvc = _kvc()
    P, B = (1 << 24) + 9, 128
    pools = [torch.empty((P, 1, 1, B, 4), device="cuda") for _ in "KV"]
    slots = torch.tensor([[0, P * B - 1, (1 << 31) + 77, P * B, -1, 1 << 31, (1 << 31) - 1]], device="cuda")
    src = [torch.randn((1, 1, 1, 7, 4), device="cuda") for _ in "KV"]
    kvc.kvc_page_write(kvc.paged(P, B, 1, 1, 4, "f32", 1, 1), src[0], src[1], slots, pools[0], pools[1])
    for pool, s in zip(pools, src):
        for i in (0, 1, 2, 5, 6):
            at = int(slots[0, i])
            assert torch.equal(pool[at // B, 0, 0, at % B], s[0, 0, 0, i])


def test_write_into_token_major_pools():
    kvc = _kvc()
    both = torch.zeros((6, 2, 16, 2, 4, 64), dtype=torch.bfloat16, device="cuda")   # [P, K|V, B, L, H, d]
    K, V = (both[:, i].permute(0, 2, 3, 1, 4) for i in range(2))
    src = [torch.randn((1, 2, 4, 5, 64), device="cuda").bfloat16() for _ in "KV"]
    slots = torch.tensor([[3, 95, 16, 17, 40]], device="cuda")
    pg = kvc.paged(6, 16, 2, 4, 64, "bf16", 1, 1)
    kvc.kvc_page_write(pg, src[0], src[1], slots, K, V)
    for x, s in ((K, src[0]), (V, src[1])):
        want = PO.page_write(s.float().cpu().numpy(), slots.cpu().numpy(), np.zeros(x.shape), 0)
        assert np.array_equal(x.float().cpu().numpy(), want)


FEW = [(1, 1), (1, 300), (0, 7), (2, 1030), (0, 0), (1, 128)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [2, 9, 12, 16])
def test_decode_few_requests_head_groups(d, G):
    b = Batch(FEW, 2 * G, 2, d, 20, "bf16", seed=G)
    b.run()
    b.check()


def test_decode_thirty_tokens_of_one_request():
    b = Batch([(30, 500)] + [(0, 9)] * 40, 8, 2, 128, 16, "bf16", seed=2)
    b.run()
    b.check()


@pytest.mark.parametrize("d", [4, 20, 64, 80, 96, 128, 132, 256])
@pytest.mark.parametrize("G", [1, 3, 16])
def test_f32_decode(d, G):
    b = Batch(FEW + [(1, 700)], 2 * G, 2, d, 17, "f32", seed=d + G)
    b.run()
    b.check()


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 50), (True, 200)])
def test_f32_decode_masks(causal, window):
    b = Batch(FEW, 8, 2, 64, 16, "f32", seed=window)
    b.run(causal, window)
    b.check(causal, window)


@pytest.mark.parametrize("lens", [FEW, [(40, 200), (1, 77), (130, 131)]])
@pytest.mark.parametrize("d", [64, 128, 192])
@pytest.mark.parametrize("where", ["K", "V", "q"])
def test_f32_infinities_in_sight(lens, d, where):
    """Rows that see an infinite value (or a value near the type's largest) get what
    the formula says; the rest what they got before."""
    b = Batch(lens, 4, 2, d, 16, "f32", seed=6)
    at = (b.table[1, 0], 0, 0, 0) if where != "q" else (int(b.q_start[1]), 0)
    x = {"K": b.K, "V": b.V, "q": b.q}[where]
    x[at][d - 1] = float("inf")
    b.run()
    torch.cuda.synchronize()
    r0, r1 = int(b.q_start[1]), int(b.q_start[2])
    heads = slice(0, 1) if where == "q" else slice(0, 2)
    if where == "K":                              # a score of -inf has no weight, +inf no softmax
        up = b.q[r0:r1, :2, d - 1] > 0
        assert torch.equal(b.out[r0:r1, :2].isnan().all(-1), up)
        assert torch.equal(b.out[r0:r1, :2].isfinite().all(-1), ~up)
    else:
        assert not b.out[r0:r1, heads].isfinite().all()
    if where == "V":                              # only the last column of the first KV head
        assert b.out[r0:r1, :2, :d - 1].isfinite().all()
        assert (b.out[r0:r1, :2, d - 1] == float("inf")).all()
    # what does not see it is as it would be without
    x[at][d - 1] = 3.4e38 if where == "V" else 0.5
    hx = {"K": b.host[0], "V": b.host[1], "q": b.host[2]}[where]
    hx[at][d - 1] = 3.4e38 if where == "V" else 0.5
    got = b.out.clone()
    b.run()
    b.check()
    torch.cuda.synchronize()
    same = torch.ones(b.N, 4, dtype=torch.bool)
    same[r0:r1, heads] = False
    assert torch.allclose(got[same.cuda()], b.out[same.cuda()], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("lens", [FEW, [(40, 200), (1, 77), (130, 131)]])
def test_f32_large_and_small_numbers(lens):
    b = Batch(lens, 4, 2, 64, 16, "f32", seed=8)
    for x, h, f in ((b.K, b.host[0], 1e18), (b.V, b.host[1], 1e30), (b.q, b.host[2], 1e-18)):
        h.mul_(f)
        x.copy_(h)
    b.run()
    b.check()
