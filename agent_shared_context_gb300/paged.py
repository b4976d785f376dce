"""Serving from corrected caches: page pools, their tables and a step's calls.

``PagedCache`` owns the pools of one model's K and V, the block tables, the
stack of free pages and the workspaces, and drives the library for a step of
serving: ``plan`` (pages, slots and positions of the step's new tokens), then
per layer ``write`` (their K and V rows) and ``attend`` (their attention over
the cache).  ``load`` puts dense caches, such as the corrected caches of a
``ChainRunner``, into the pages of the tokens just planned.  ``from_chain``
does all of that for one agent of a chain: the agent's held cache (corrected
PH rows, its own PF rows; KVCMAS listing, Figure 1(c)) becomes the context
that its new tokens attend to.

Nothing here waits for the device: lengths, tables and the stack of free pages
live on the GPU, and a captured CUDA graph replays with new ones.  ``plan``
reads one pair of state buffers and writes the other, so a graph that is to be
replayed holds an even number of steps.

    python -m agent_shared_context_gb300.paged --workload llama2k --layers 4

runs a chain, takes the last agent's caches into pages, lets a prompt attend
to them and then decodes (synthetic queries, keys and values: the library
holds no model weights).
"""
from __future__ import annotations

import argparse
from typing import Optional, Sequence, Union

import torch

from . import kvc, synth
from .chain import ChainRunner

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


class PagedCache:
    """Pools [n_pages, L, H, page_size, d] and the state of up to ``requests``
    requests of at most ``max_blocks`` pages; a step brings at most
    ``max_tokens`` new tokens with ``n_q_heads`` query heads.

    With a ``stream`` the state above is made on it and every call runs on it,
    behind what the current stream was given before the call; who reads state
    or results elsewhere waits for ``stream``."""

    def __init__(self, L: int, H: int, d: int, dtype: str, n_q_heads: int, n_pages: int,
                 page_size: int, requests: int, max_blocks: int, max_tokens: int,
                 device="cuda", stream: Optional[torch.cuda.Stream] = None):
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.n_q_heads, self.max_tokens = n_q_heads, max_tokens
        self.device, self.stream = dev, stream
        self.pg = kvc.paged(n_pages, page_size, L, H, d, dtype, requests, max_blocks)
        with torch.cuda.stream(stream):
            self.pool_K = torch.zeros((n_pages, L, H, page_size, d), dtype=_DTYPES[dtype],
                                      device=dev)
            self.pool_V = torch.zeros_like(self.pool_K)
            self.table = torch.zeros((requests, max_blocks), **i32)
            self.free_pages = torch.arange(n_pages - 1, -1, -1, **i32)   # page 0 is taken first
            self._n_free = [torch.full((1,), n_pages, **i32), torch.zeros(1, **i32)]
            self._kv_lens = [torch.zeros(requests, **i32) for _ in range(2)]
            self._now = self._planned = 0
            self.q_start = torch.zeros(requests + 1, **i32)
            self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=dev)
            self.positions = torch.full((max_tokens,), -1, **i32)
            self.plan_status = torch.zeros(requests, **i32)
            self.dev_status = torch.zeros(1, **i32)
            # the largest step's size serves every step: it does not shrink with fewer tokens
            q = torch.empty((max_tokens, n_q_heads, d), dtype=_DTYPES[dtype], device="meta")
            ws = kvc.kvc_paged_attention_workspace(self.pg, kvc.attn_params(q, q))
            if ws == 0:
                raise ValueError("no attention of this shape: head dims are 64 or 128 in bf16, "
                                 "multiples of 4 up to 256 in f32, at most 64 query heads a KV "
                                 "head")
            self.workspace = torch.zeros(ws, dtype=torch.uint8, device=dev)

    @property
    def kv_lens(self) -> torch.Tensor:
        """[requests] int32 on the device: tokens in the cache."""
        return self._kv_lens[self._now]

    @property
    def n_free(self) -> torch.Tensor:
        """[1] int32 on the device: pages that no request holds."""
        return self._n_free[self._now]

    def plan(self, new_lens: Union[torch.Tensor, Sequence[int]],
             tokens: Optional[int] = None) -> None:
        """Pages, slots and positions of the step's new tokens (-1: the
        request is finished), of which there are at most ``tokens``
        (``max_tokens`` if not given).  ``plan_status`` tells what was refused."""
        tokens = self.max_tokens if tokens is None else tokens
        if not 0 <= tokens <= self.max_tokens:
            raise ValueError("a step brings at most max_tokens tokens")
        if not isinstance(new_lens, torch.Tensor):
            with torch.cuda.stream(self.stream):
                if torch.cuda.is_current_stream_capturing():
                    raise ValueError("the lengths of a captured step are a tensor")
                # out of pinned memory: the copy takes its turn, and nothing waits for it
                host = torch.tensor(new_lens, dtype=torch.int32, pin_memory=True)
                new_lens = host.to(self.device, non_blocking=True)
        if (new_lens.dtype != torch.int32 or new_lens.shape != (self.pg.R,)
                or new_lens.device != self.table.device):
            raise ValueError("new_lens is [requests] int32, on the pools' device")
        new_lens = new_lens.contiguous()
        self._take(new_lens)
        old, new = self._now, 1 - self._now
        kvc.kvc_page_plan(self.pg, new_lens, self._kv_lens[old], self._kv_lens[new],
                          self.table, self.free_pages, self._n_free[old], self._n_free[new],
                          self.q_start, self.slots, self.positions, self.plan_status,
                          stream=self.stream, max_tokens=tokens)
        self._now, self._planned = new, tokens

    def write(self, layer: int, K: torch.Tensor, V: torch.Tensor) -> None:
        """The planned tokens' rows [N, H, d] into their pages of a layer."""
        self._tokens(K)
        self._tokens(V)
        if K.shape[1] != self.pg.H or V.shape != K.shape:
            raise ValueError("K and V are [N, H, d] with the pools' heads")
        self._take(K, V)
        view = lambda x: x.permute(1, 0, 2)[None, None]  # noqa: E731   [1, 1, H, N, d]
        kvc.kvc_page_write(self.pg, view(K), view(V), self.slots, self.pool_K, self.pool_V, layer,
                           stream=self.stream)

    def load(self, K: torch.Tensor, V: torch.Tensor, rows: Optional[torch.Tensor] = None) -> None:
        """All layers of dense caches [requests, L, H, T, d] into the pages of
        the tokens just planned (T of each request); of those, where ``rows``
        ([requests, T] bool) is given, only the ones that it names."""
        if (K.dim() != 5 or V.shape != K.shape or K.shape[4] != self.pg.d
                or K.shape[:3] != (self.pg.R, self.pg.L, self.pg.H)):
            raise ValueError("dense caches are [requests, L, H, T, d]")
        self._like_pools(K)
        self._like_pools(V)
        if rows is not None and (rows.shape != (K.shape[0], K.shape[3]) or rows.dtype != torch.bool
                                 or rows.device != K.device):
            raise ValueError("rows is [requests, T] bool")
        if K.shape[0] * K.shape[3] > self._planned:
            raise ValueError("more tokens than were planned")
        self._take(K, V, rows)
        with torch.cuda.stream(self.stream):
            slots = self.slots
            if rows is not None:
                slots = torch.where(rows.reshape(-1), slots[:rows.numel()], -1)
            kvc.kvc_page_write(self.pg, K, V, slots, self.pool_K, self.pool_V, 0,
                               stream=self.stream)

    def attend(self, layer: int, q: torch.Tensor, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, causal: bool = True, window: int = 0,
               scale: float = 0.0) -> torch.Tensor:
        """Attention of the planned tokens' queries [N, n_q_heads, d]; ``lse``
        [N, n_q_heads] float32 gets the logarithms of the softmax's sums."""
        self._tokens(q)
        if q.shape[1] > self.n_q_heads:
            raise ValueError("more query heads than n_q_heads")
        out = torch.empty_like(q) if out is None else out
        self._like_pools(out)
        if lse is not None and (lse.shape != q.shape[:2] or lse.dtype != torch.float32
                                or lse.device != q.device or not lse.is_contiguous()):
            raise ValueError("lse is [N, n_q_heads] float32, contiguous")
        self._take(q, out, lse)
        at = kvc.attn_params(q, out, layer, scale, causal, window)
        kvc.kvc_paged_attention(self.pg, at, q, self.pool_K, self.pool_V, self.table, self.q_start,
                                self.kv_lens, out, self.workspace, self.dev_status, lse=lse,
                                stream=self.stream)
        return out

    def _take(self, *tensors: Optional[torch.Tensor]) -> None:
        """A call's tensors belong to the current stream: the cache's own waits for
        what was given to it, and their memory is not reused before it is done."""
        if self.stream is None:
            return
        current = torch.cuda.current_stream(self.pool_K.device)
        if current == self.stream:
            return
        self.stream.wait_stream(current)
        for x in tensors:
            if x is not None:
                x.record_stream(self.stream)

    def _tokens(self, x: torch.Tensor) -> None:
        if x.dim() != 3 or x.shape[0] > self._planned or x.shape[2] != self.pg.d:
            raise ValueError("a step's rows are [N, heads, d], no more than were planned")
        self._like_pools(x)

    def _like_pools(self, x: torch.Tensor) -> None:
        if x.dtype != self.pool_K.dtype or x.device != self.pool_K.device:
            raise ValueError("what goes with the pools has their type and is on their device")


def from_chain(runner: ChainRunner, agent: int, n_q_heads: int, new_tokens: int,
               page_size: int = 16) -> PagedCache:
    """Pages that hold agent ``agent``'s held caches of every request, with
    room for ``new_tokens`` more per request.  A chain that reuses its output
    buffers hands out the agents whose rows are still there."""
    if not runner.holds(agent):
        raise ValueError("agent %d's cache is not in its buffer: the chain reuses them "
                         "(keep_outputs=False)" % agent)
    K, V = runner.held(agent)
    R, L, H, T, d = K.shape
    blocks = -(-(T + new_tokens) // page_size)
    pc = PagedCache(L, H, d, runner.wl.dtype, n_q_heads, R * blocks, page_size, R, blocks,
                    R * max(T, new_tokens), device=K.device, stream=runner.stream)
    pc.plan([T] * R, R * T)
    pc.load(K, V)
    if not runner.own_prefix(agent):
        pc.load(runner.inp.exact_K[agent], runner.inp.exact_V[agent], ~runner.ph_rows)
    return pc


def decode_graph(pc: PagedCache, new_lens: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                 v: torch.Tensor, out: torch.Tensor) -> torch.cuda.CUDAGraph:
    """Two steps over all layers as a CUDA graph: tokens ``q``, ``out``
    [2, L, N, n_q_heads, d] and ``k``, ``v`` [2, L, N, H, d], read at replay.
    The graph keeps them, ``new_lens`` and the cache for as long as it lives."""
    if pc.stream is not None:
        raise ValueError("a captured step runs on the capturing stream: stream=None")

    def two_steps(lens):
        for s in range(2):
            pc.plan(lens, q.shape[2])
            for i in range(pc.pg.L):
                pc.write(i, k[s, i], v[s, i])
                pc.attend(i, q[s, i], out[s, i])

    two_steps(torch.zeros_like(new_lens))                # loads the kernels, changes nothing
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two_steps(new_lens)
    graph.buffers = (pc, new_lens, q, k, v, out)         # which a replay reads and writes
    return graph


def main(argv: Optional[Sequence[str]] = None) -> None:
    ap = argparse.ArgumentParser(description="decode from the corrected caches of a chain")
    ap.add_argument("--workload", default="tiny")
    ap.add_argument("--layers", type=int, default=None, help="shrink the workload to these layers")
    ap.add_argument("--group", type=int, default=4, help="query heads per KV head")
    ap.add_argument("--prompt", type=int, default=128, help="tokens of the agent's prompt")
    ap.add_argument("--steps", type=int, default=64, help="tokens to decode, an even number")
    ap.add_argument("--page-size", type=int, default=16)
    a = ap.parse_args(argv)
    if a.steps < 2 or a.steps % 2 or a.prompt < 1:
        ap.error("--steps is even and at least 2, --prompt at least 1")
    wl = synth.workload(a.workload)
    if a.layers is not None:
        wl = synth.scaled(wl, L=a.layers)
    runner = ChainRunner(wl, synth.generate(wl, device="cuda"))
    runner.run()
    Hq = wl.H * a.group
    pc = from_chain(runner, wl.n_agents - 1, Hq, a.prompt + a.steps + 2, a.page_size)

    def rows(*shape):
        return torch.randn(shape, device="cuda").to(_DTYPES[wl.dtype])

    N = wl.R * a.prompt
    pc.plan([a.prompt] * wl.R, N)
    for i in range(wl.L):
        pc.write(i, rows(N, wl.H, wl.d), rows(N, wl.H, wl.d))
        pc.attend(i, rows(N, Hq, wl.d))

    ones = torch.ones(wl.R, dtype=torch.int32, device="cuda")
    q, k, v = rows(2, wl.L, wl.R, Hq, wl.d), *(rows(2, wl.L, wl.R, wl.H, wl.d) for _ in "kv")
    out = torch.empty_like(q)
    graph = decode_graph(pc, ones, q, k, v, out)
    graph.replay()                                       # two tokens more than are timed
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda.synchronize()
    ev[0].record()
    for _ in range(a.steps // 2):
        graph.replay()
    ev[1].record()
    torch.cuda.synchronize()
    status = int(pc.dev_status) or int(runner.dev_status) or int(pc.plan_status.abs().max())
    if status or not bool(torch.isfinite(out.float()).all()):
        raise RuntimeError(f"decoding failed (status {status})")
    ms = ev[0].elapsed_time(ev[1]) / a.steps
    print(f"{a.workload}: {wl.R} requests of {int(pc.kv_lens.max())} tokens, {wl.L} layers, "
          f"{Hq}/{wl.H} heads of {wl.d}, {wl.dtype}: {1e3 * ms:.1f} us per decoded step "
          f"({1e3 * ms / wl.L:.1f} per layer), {wl.R / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
