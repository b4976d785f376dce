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
