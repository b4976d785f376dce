"""PagedCache on the GPU: what a captured step keeps, contexts of memory-lean chains,
steps without tokens, and a cache whose calls run on a stream of its own."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _cache(dtype="bf16", stream=None, requests=3):
    from agent_shared_context_gb300 import paged
    return paged.PagedCache(2, 2, 64, dtype, 8, 64, 16, requests, 12, 200, stream=stream)


def test_captured_steps_keep_their_tensors():
    """The caller drops everything but the graph and the cache; what it allocates next
    must not be read as the steps' lengths and tokens."""
    from agent_shared_context_gb300 import paged
    pc = _cache()
    g = torch.Generator(device="cuda").manual_seed(1)

    def tokens(heads):
        return torch.randn((2, 2, 3, heads, 64), generator=g, device="cuda").bfloat16()

    graph = paged.decode_graph(pc, torch.ones(3, dtype=torch.int32, device="cuda"), tokens(8),
                               tokens(2), tokens(2), torch.zeros_like(tokens(8)))
    junk = [torch.full((n,), 77, dtype=torch.int32, device="cuda")
            for n in (3, 6144, 1536) for _ in range(40)]
    for step in (2, 4):
        graph.replay()
        torch.cuda.synchronize()
        assert pc.kv_lens.tolist() == [step] * 3 and not pc.plan_status.any()
    assert all((x == 77).all() for x in junk)


def _rows(pc, K, r, T):
    """[L, H, T, d]: the first T rows of request r out of the pool ``K``."""
    B = pc.pg.page_size
    pages = K[pc.table[r, :-(-T // B)].long()]                    # [n, L, H, B, d]
    return pages.permute(1, 2, 0, 3, 4).flatten(2, 3)[:, :, :T]


def _runners(**kw):
    from agent_shared_context_gb300 import synth
    from agent_shared_context_gb300.chain import ChainRunner
    wl = synth.scaled(synth.workload("llama2k"), L=2, H=2, R=2, seg_len=[64, 72], pf=24, **kw)
    inp = synth.generate(wl, device="cuda")
    return wl, ChainRunner(wl, inp), ChainRunner(wl, inp, keep_outputs=False)


def test_context_of_a_memory_lean_chain():
    """A chain that alternates between two buffers hands out the same context as one that
    keeps them all: an agent's own tokens are its own."""
    from agent_shared_context_gb300 import paged
    wl, full, lean = _runners()
    assert wl.edges == 3
    full.run(), lean.run()
    for agent in (0, 2, 3):
        a, b = (paged.from_chain(x, agent, 8, 5, 16) for x in (full, lean))
        for r in range(wl.R):
            for x, y, held in zip((a.pool_K, a.pool_V), (b.pool_K, b.pool_V), full.held(agent)):
                assert torch.equal(_rows(a, x, r, wl.T), held[r])
                assert torch.equal(_rows(b, y, r, wl.T), held[r]), agent
    with pytest.raises(ValueError):
        paged.from_chain(lean, 1, 8, 5, 16)                       # agent 3's rows are there


def test_context_of_a_memory_lean_chain_between_its_edges():
    from agent_shared_context_gb300 import paged
    wl, full, lean = _runners()
    for j in range(1, wl.edges + 1):
        full.run_edge(j), lean.run_edge(j)
        b = paged.from_chain(lean, j, 8, 5, 16)
        for r in range(wl.R):
            for x, held in zip((b.pool_K, b.pool_V), full.held(j)):
                assert torch.equal(_rows(b, x, r, wl.T), held[r]), j
        for other in range(j + 1, wl.edges + 1):
            if other > 2:
                with pytest.raises(ValueError):
                    paged.from_chain(lean, other, 8, 5, 16)       # its edge has not run


def _steps(stream, busy, lists):
    """Steps of a cache with and without a stream of its own; every input is made on the
    current stream behind a pause, dropped or overwritten after its call, and the
    outputs' memory is handed on at once."""
    from agent_shared_context_gb300 import paged
    g = torch.Generator(device="cuda").manual_seed(9)
    pause = (lambda: torch.cuda._sleep(4_000_000)) if busy else (lambda: None)
    pause()
    pc = paged.PagedCache(2, 2, 64, "bf16", 8, 64, 16, 3, 12, 200, stream=stream)
    kept, dropped = [], []
    for lens in [[40, 3, 0], [1, 5, 30], [1, 1, 1], [0, -1, 2], [2, 7, 1]] * 2:
        if stream is not None and busy:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(4_000_000)
        pause()
        N = sum(max(n, 0) for n in lens)
        pc.plan(lens if lists else torch.tensor(lens, dtype=torch.int32).pin_memory().to(
            "cuda", non_blocking=True), N)
        for i in range(2):
            rows = lambda h: torch.randn((N, h, 64), generator=g, device="cuda").bfloat16()  # noqa: E731
            q, k, v, lse = rows(8), rows(2), rows(2), torch.empty((N, 8), device="cuda")
            pc.write(i, k, v)
            kept.append((pc.attend(i, q, lse=lse), lse))
            pc.attend(i, q)                        # dropped: its memory is the next one's
            dropped.append(torch.full_like(q, 7.0))
            del q, k, v
            junk = [torch.full((N, h, 64), 9.0, dtype=torch.bfloat16, device="cuda") for h in (8, 2, 2)]
            del junk
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    assert all((x == 7).all() for x in dropped)
    assert not int(pc.dev_status) and not pc.plan_status.any()
    return kept, pc


@pytest.mark.parametrize("lists", [False, True])
def test_cache_on_a_stream_of_its_own(lists):
    want, a = _steps(None, False, lists)
    for _ in range(3):
        got, b = _steps(torch.cuda.Stream(), True, lists)
        for (x, s), (y, t) in zip(want, got):
            assert torch.equal(x, y) and torch.equal(s, t)
        assert a.kv_lens.tolist() == b.kv_lens.tolist() == [88, 7, 68]   # 1 ends twice
        assert torch.equal(a.pool_K, b.pool_K) and torch.equal(a.pool_V, b.pool_V)
        assert torch.equal(a.table, b.table) and int(a.n_free) == int(b.n_free)


def test_context_of_a_chain_on_a_stream_of_its_own():
    from agent_shared_context_gb300 import paged, synth
    from agent_shared_context_gb300.chain import ChainRunner
    wl = synth.scaled(synth.workload("llama2k"), L=2, H=2, R=2, seg_len=[64, 72], pf=24)
    inp = synth.generate(wl, device="cuda")
    side = torch.cuda.Stream()
    want = ChainRunner(wl, inp)
    want.run()
    for keep in (True, False):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            runner = ChainRunner(wl, inp, stream=side, keep_outputs=keep)
            torch.cuda._sleep(20_000_000)
        runner.run()
        pc = paged.from_chain(runner, 3, 8, 5, 16)             # the current stream is idle
        side.synchronize()
        for r in range(wl.R):
            for x, held in zip((pc.pool_K, pc.pool_V), want.held(3)):
                assert torch.equal(_rows(pc, x, r, wl.T), held[r])


def test_captured_steps_take_no_list():
    pc = _cache()
    pc.plan([1, 1, 1], 3)
    graph = torch.cuda.CUDAGraph()
    x = torch.zeros(4, device="cuda")
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(ValueError):
            pc.plan([1, 1, 1], 3)
    graph.replay()
    torch.cuda.synchronize()
    assert x.tolist() == [1] * 4 and pc.kv_lens.tolist() == [1] * 3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_without_tokens(dtype):
    pc = _cache(dtype)
    dt = pc.pool_K.dtype
    pc.plan([5, 0, 3], 8)
    q = torch.randn((8, 8, 64), device="cuda").to(dt)
    pc.write(1, q[:, :2], q[:, 2:4])
    K = pc.pool_K.clone()
    pc.plan([0, 0, 0], 0)
    pc.write(1, q[:0, :2], q[:0, 2:4])
    assert pc.attend(1, q[:0]).shape == (0, 8, 64)
    torch.cuda.synchronize()
    assert torch.equal(K, pc.pool_K) and pc.kv_lens.tolist() == [5, 0, 3]
    assert pc.q_start.tolist() == [0] * 4
    assert not int(pc.dev_status) and not pc.plan_status.any()
