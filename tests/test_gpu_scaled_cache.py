"""A chain's corrected caches served from pages of 8-bit numbers: chain, pages, a prompt whose
heads are normalised and turned by position, decoding in a replayed graph.  The attention is
held against float64 over the elements that the pages stand for, the elements against the
rows that went in."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from agent_shared_context_gb300 import paged, synth  # noqa: E402
from oracle import scaled_oracle as SO  # noqa: E402
from tests.test_gpu_paged_scaled import Batch  # noqa: E402
from tests.test_gpu_rotary import _check as check_rotated, _reference as rotated  # noqa: E402


def _chain(**over):
    from agent_shared_context_gb300.chain import ChainRunner
    wl = synth.scaled(synth.workload("llama2k"), **dict(dict(L=2, H=2, R=3, seg_len=[64, 72], pf=24), **over))
    runner = ChainRunner(wl, synth.generate(wl, device="cuda"))
    runner.run()
    return wl, runner


def _attention(pc, layer, q, out, n):
    """`out` of n new tokens per request against the elements in the pages."""
    torch.cuda.synchronize()
    b = Batch.__new__(Batch)
    kv = pc.kv_lens.tolist()
    b.lens, b.B, b.block, b.d, b.layer = [(n, t) for t in kv], pc.pg.page_size, pc.sc.block, pc.pg.d, layer
    b.table, b.q_start = pc.table.cpu().numpy().astype(np.int64), np.arange(len(kv) + 1) * n
    b.bytes, b.exps = [[x.cpu().numpy() for x in y] for y in ((pc.pool_K, pc.pool_V), (pc.exp_K, pc.exp_V))]
    b.host_q, b.out, b.status, b.ws = q.double().cpu().numpy(), out, pc.dev_status, pc.workspace
    b.check(lse=False)


def _elements(pc, which, r, n):
    """[L, H, n, d] of request r, and the powers of two of the rows' blocks."""
    pool, exps = ((pc.pool_K, pc.exp_K), (pc.pool_V, pc.exp_V))[which]
    B = pc.pg.page_size
    pages = pc.table[r, :-(-n // B)].long().cpu().numpy()
    x, e = pool.cpu().numpy()[pages], exps.cpu().numpy()[pages]
    v = SO.values(x, e, pc.sc.block)
    s = np.repeat(2.0 ** (e.astype(np.int64) - 127), pc.sc.block, -1)[..., :B, None]
    cut = lambda y: np.broadcast_to(y, v.shape).transpose(1, 2, 0, 3, 4).reshape(  # noqa: E731
        *v.shape[1:3], -1, v.shape[-1])[:, :, :n]
    return cut(v), cut(s)


def _near(v, s, x):
    """Half a step of a number, 2^-4 of it or 2^-10 beside a power of two of 1; once more for
    a block that grew, whose earlier rounding was to a smaller step."""
    x = x.double().cpu().numpy()
    assert (np.abs(v - x) <= (2.0 ** -4 * np.abs(x) + 2.0 ** -10 * s) * (1 + 2.0 ** -4) + 2.0 ** -10 * s).all()


@pytest.mark.parametrize("page,block", [(16, 16), (20, 8)])
def test_served_chain(page, block):
    wl, runner = _chain()
    agent, prompt = wl.n_agents - 1, 37
    R, L, H, d, T, Hq = wl.R, wl.L, wl.H, wl.d, wl.T, wl.H * 4
    pc = paged.from_chain(runner, agent, Hq, prompt + 4, page, "e4m3", block)
    held = runner.held(agent)
    for r in range(R):
        for which in range(2):
            _near(*_elements(pc, which, r, T), held[which][r])
    g = torch.Generator(device="cuda").manual_seed(5)
    rows = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    rotary, w = paged.Rotary(d, 500000.0, eps=1e-6), [rows(d), rows(d)]
    pc.plan([prompt] * R, R * prompt)
    pos = T + torch.arange(prompt).repeat(R)
    for i in range(L):
        q, k, v = rows(R * prompt, Hq, d), rows(R * prompt, H, d), rows(R * prompt, H, d)
        before = q.clone(), k.clone()
        assert pc.rotate(rotary, q, k, *w)[0] is q
        for y, x, wt in zip((q, k), before, w):
            check_rotated(y, *rotated(x, pos, d, 500000.0, False, True, wt), torch.bfloat16)
        pc.write(i, k, v)
        _attention(pc, i, q, pc.attend(i, q), prompt)
    q, k, v = rows(2, L, R, Hq, d), rows(2, L, R, H, d), rows(2, L, R, H, d)
    out = torch.full_like(q, float("nan"))
    turn = paged.Rotary(64, 10000.0, interleaved=True)
    graph = paged.decode_graph(pc, torch.ones(R, dtype=torch.int32, device="cuda"), q, k, v, out, turn)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    kv = T + prompt + 4
    assert pc.kv_lens.tolist() == [kv] * R and pc.positions[:R].tolist() == [kv - 1] * R
    for i in range(L):
        last = rotated(q[1, i], torch.full((R,), kv - 1), 64, 10000.0, True, False, None)[0]
        _attention(pc, i, last.to(torch.bfloat16), out[1, i], 1)
    for r in range(R):                                    # the last token's keys and values
        x = rotated(k[1, :, r], torch.full((L,), kv - 1), 64, 10000.0, True, False, None)[0]
        for which, y in ((0, x), (1, v[1, :, r])):
            e, s = _elements(pc, which, r, kv)
            _near(e[:, :, -1], s[:, :, -1], y)
    assert not pc.plan_status.any() and not int(pc.dev_status)


def test_own_stream_and_recycled_pages():
    """A cache on a stream of its own gives what one on the current stream does, and pages that
    come back hold nothing of their last use."""
    g = torch.Generator(device="cuda").manual_seed(6)
    R, L, H, d, T, Hq = 2, 1, 2, 128, 45, 8
    big = [(1000 * torch.randn((R, L, H, T, d), generator=g, device="cuda")).bfloat16() for _ in "KV"]
    small = [torch.randn((R, L, H, T, d), generator=g, device="cuda").bfloat16() for _ in "KV"]
    q = torch.randn((R, Hq, d), generator=g, device="cuda").bfloat16()
    outs = []
    for stream, first in ((None, big), (torch.cuda.Stream(), big), (None, None)):
        pc = paged.PagedCache(L, H, d, "e4m3", Hq, 8, 16, R, 4, R * T, stream=stream, scale_block=8)
        if first is not None:
            pc.plan([T] * R)
            pc.load(*first)
            pc.plan([-1] * R, 0)
        pc.plan([T] * R)
        pc.load(*small)
        pc.plan([1] * R, R)
        pc.write(0, small[0][:, 0, :, 0].contiguous(), small[1][:, 0, :, 0].contiguous())
        outs.append(pc.attend(0, q))
        torch.cuda.synchronize()
        assert not pc.plan_status.any() and not int(pc.dev_status)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_rows_that_replace_others():
    g = torch.Generator(device="cuda").manual_seed(7)
    R, L, H, d, T = 2, 2, 2, 64, 50
    a, b = ([torch.randn((R, L, H, T, d), generator=g, device="cuda").bfloat16() * f for _ in "KV"]
            for f in (1.0, 3.0))
    rows = torch.rand((R, T), generator=g, device="cuda") < 0.5
    pc = paged.PagedCache(L, H, d, "e4m3", 4, 8, 16, R, 4, R * T, scale_block=8)
    pc.plan([T] * R)
    pc.load(*a)
    pc.load(*b, rows)
    torch.cuda.synchronize()
    for r in range(R):
        for which in range(2):
            want = torch.where(rows[r][None, None, :, None], b[which][r], a[which][r])
            _near(*_elements(pc, which, r, T), want)


def test_demonstration(capsys):
    paged.main(["--workload", "llama2k", "--layers", "1", "--prompt", "20", "--steps", "4", "--cache", "e4m3",
                "--rotary"])
    assert "e4m3" in capsys.readouterr().out


@pytest.mark.parametrize("own_stream", [False, True])
def test_pages_of_a_chain_that_reuses_its_buffers(own_stream):
    """The agent's rows are rounded once: as if its whole cache had been written, with nothing
    left of the agent whose buffer it took over."""
    from agent_shared_context_gb300.chain import ChainRunner
    wl = synth.scaled(synth.workload("llama2k"), L=2, H=2, R=3, seg_len=[64, 72], pf=24)
    inp = synth.generate(wl, device="cuda")
    agent = wl.n_agents - 1
    for x in (inp.exact_K[agent - 2], inp.exact_V[agent - 2]):    # whose buffer that is
        x.mul_(64.0)
    torch.cuda.synchronize()
    runner = ChainRunner(wl, inp, keep_outputs=False, stream=torch.cuda.Stream() if own_stream else None)
    torch.cuda.synchronize()                              # its buffers are made on this stream
    runner.run()
    assert not runner.own_prefix(agent)
    pc = paged.from_chain(runner, agent, 8, 4, 16, "e4m3", 16)
    torch.cuda.synchronize()
    mask = runner.ph_rows[:, None, None, :, None]
    whole = [torch.where(mask, x, y) for x, y in zip(runner.held(agent), (inp.exact_K[agent], inp.exact_V[agent]))]
    want = paged.PagedCache(wl.L, wl.H, wl.d, "e4m3", 8, pc.pg.n_pages, 16, wl.R, pc.pg.max_blocks,
                            wl.R * wl.T, scale_block=16)
    want.plan([wl.T] * wl.R)
    want.load(*whole)
    torch.cuda.synchronize()
    assert torch.equal(pc.table, want.table) and torch.equal(pc.kv_lens, want.kv_lens)
    for name in ("pool_K", "pool_V", "exp_K", "exp_V"):
        assert torch.equal(getattr(pc, name), getattr(want, name)), name
