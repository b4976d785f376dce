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
