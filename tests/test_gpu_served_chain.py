"""A chain's corrected caches served from pages: chain, pages, a prompt that
attends to them, decoding in a replayed graph; against float64 attention over
the same dense caches.  Tolerances per element as in test_gpu_paged."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


def _check(got, q, K, V, kv, n, dtype):
    """Rows of ``n`` new tokens per request over dense caches [R, H, T, d]."""
    R, H, _, d = K.shape
    o, _, A, E = PO.paged_attention(q, K[:, None], V[:, None], [[r] for r in range(R)],
                                    np.arange(R + 1) * n, [kv] * R, d ** -0.5)
    ds = (d + 16) * 2.0 ** -24 * E[:, :, None]
    tol = (np.expm1(2 * ds) + (kv + 4) * 2.0 ** -24) * A
    tol += 2.0 ** -9 * (1.01 * A + 1.01 * np.abs(o)) if dtype == "bf16" else 2.0 ** -23 * np.abs(o)
    assert (np.abs(got - o) <= tol).all()


@pytest.mark.parametrize("name,over", [
    ("tiny", {}),
    ("llama2k", dict(L=2, H=2, R=3, seg_len=[64, 72], pf=24)),
])
def test_served_chain(name, over):
    from agent_shared_context_gb300 import paged, synth
    from agent_shared_context_gb300.chain import ChainRunner
    wl = synth.workload(name)
    if over:
        wl = synth.scaled(wl, **over)
    runner = ChainRunner(wl, synth.generate(wl, device="cuda"))
    runner.run()
    agent, group, prompt, page = wl.n_agents - 1, 4, 37, 16
    R, L, H, d, T, Hq = wl.R, wl.L, wl.H, wl.d, wl.T, wl.H * group
    pc = paged.from_chain(runner, agent, Hq, prompt + 4, page)
    dt = pc.pool_K.dtype
    g = torch.Generator(device="cuda").manual_seed(5)

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    dense = [torch.cat([x, torch.zeros((R, L, H, prompt + 4, d), dtype=dt, device="cuda")], 3)
             for x in runner.held(agent)]
    f64 = lambda x: x.detach().cpu().double().numpy()  # noqa: E731

    def put(layer, at, k, v):
        n = k.shape[0] // R
        for x, y in zip(dense, (k, v)):
            x[:, layer, :, at:at + n] = y.reshape(R, n, H, d).transpose(1, 2)

    pc.plan([prompt] * R, R * prompt)
    for i in range(L):
        q, k, v = rows(R * prompt, Hq, d), rows(R * prompt, H, d), rows(R * prompt, H, d)
        pc.write(i, k, v)
        put(i, T, k, v)
        out = pc.attend(i, q)
        _check(f64(out), f64(q), f64(dense[0][:, i]), f64(dense[1][:, i]), T + prompt, prompt,
               wl.dtype)

    q, k, v = rows(2, L, R, Hq, d), rows(2, L, R, H, d), rows(2, L, R, H, d)
    out = torch.full_like(q, float("nan"))
    graph = paged.decode_graph(pc, torch.ones(R, dtype=torch.int32, device="cuda"), q, k, v, out)
    kv = T + prompt
    for replay in range(2):                              # the second with other tokens
        if replay:
            q.copy_(rows(*q.shape)), k.copy_(rows(*k.shape)), v.copy_(rows(*v.shape))
        graph.replay()
        torch.cuda.synchronize()
        for s in range(2):
            kv += 1
            for i in range(L):
                put(i, kv - 1, k[s, i], v[s, i])
                _check(f64(out[s, i]), f64(q[s, i]), f64(dense[0][:, i]), f64(dense[1][:, i]), kv,
                       1, wl.dtype)
    assert pc.kv_lens.tolist() == [kv] * R and kv == T + prompt + 4
    assert pc.positions[:R].tolist() == [kv - 1] * R
    assert int(pc.n_free) == pc.pg.n_pages - R * (-(-kv // page))
    assert not pc.plan_status.any() and not int(pc.dev_status) and not int(runner.dev_status)

    pc.plan([-1] * R, 0)                                 # the requests end
    assert int(pc.n_free) == pc.pg.n_pages and not pc.kv_lens.any()


def test_served_chain_refusals():
    from agent_shared_context_gb300 import kvc, paged
    pc = paged.PagedCache(1, 2, 64, "bf16", 8, 4, 16, 2, 3, 32)
    q = torch.zeros((8, 8, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        pc.attend(0, q)                                  # nothing planned
    with pytest.raises(ValueError):
        pc.plan([1, 1], 33)
    with pytest.raises(ValueError):
        pc.plan([1, 1, 1])
    pc.plan([4, 4], 8)
    with pytest.raises(ValueError):
        pc.attend(0, q.float())
    with pytest.raises(ValueError):
        pc.write(0, q[:, :2], q[:, :1])
    with pytest.raises(ValueError):
        pc.load(q[None, None], q[None, None])
    with pytest.raises(kvc.KvcError):
        pc.attend(1, q)                                  # no such layer
    with pytest.raises(ValueError):
        paged.PagedCache(1, 2, 96, "bf16", 8, 4, 16, 2, 3, 32)   # bf16 heads are 64 or 128
    pc.plan([40, 8], 32)
    assert pc.plan_status.tolist()[0] != 0 and pc.kv_lens.tolist()[0] == 4


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_steps_that_follow_one_another(dtype, d):
    """Plan, write and attention of many small steps without a pause between them (each
    kernel is launched while the one before ends) give the bits of steps that wait."""
    from agent_shared_context_gb300 import paged
    R, H, Hq, B = 5, 2, 8, 16
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    g = torch.Generator(device="cuda").manual_seed(3)
    steps = [[1] * R if i % 3 else [(7 * i + 3 * r) % 40 for r in range(R)] for i in range(30)]
    lens = [torch.tensor(s, dtype=torch.int32, device="cuda") for s in steps]
    rows = [[torch.randn((sum(s), h, d), generator=g, device="cuda").to(dt) for h in (Hq, H, H)]
            for s in steps]
    blocks = sum(max(s) for s in steps) // B + 1

    def run(wait):
        pc = paged.PagedCache(1, H, d, dtype, Hq, R * blocks, B, R, blocks, 40 * R)
        outs = []
        torch.cuda.synchronize()
        for s, n, (q, k, v) in zip(steps, lens, rows):
            pc.plan(n, sum(s))
            if wait:
                torch.cuda.synchronize()
            pc.write(0, k, v)
            if wait:
                torch.cuda.synchronize()
            outs.append(pc.attend(0, q))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert not pc.plan_status.any() and not int(pc.dev_status)
        return outs, pc.kv_lens.tolist()

    want, kv = run(True)
    assert kv == [sum(s[r] for s in steps) for r in range(R)]
    for _ in range(5):
        got, _ = run(False)
        assert all(torch.equal(x, y) for x, y in zip(want, got))
