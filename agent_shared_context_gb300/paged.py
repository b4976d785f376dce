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

With dtype "e4m3" the pools hold bytes, numbers of 8 bits with a power of two for each
block of tokens and head: half of bf16's memory; decoding with up to 128 rows of queries a
KV head takes 0.64 to 0.71 of bf16's time, with more of them 1.7 times (64 requests of
4,000 tokens, 32 heads on 8), prompts 1.25 to 1.4 times.  Rows go in and queries attend as bf16.  ``rotate`` turns a step's queries and keys by the positions that
``plan`` gave them, with the heads' norms where the model has some.

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

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}       # of a step's rows
_POOLS = dict(_DTYPES, e4m3=torch.uint8)


class Rotary:
    """How a model turns its heads by position: frequencies base^(-2 i / rot_dim), scaled for
    long contexts as ``kvc.rotary_turns`` says, pairs of neighbours or of halves; with an
    ``eps`` every head is divided by its root mean square first."""

    def __init__(self, rot_dim: int, base: float = 10000.0, scaling: str = "none",
                 interleaved: bool = False, eps: Optional[float] = None, device="cuda", **scaled):
        turns, self.amplitude = kvc.rotary_turns(rot_dim, base, scaling, **scaled)
        self.turns = turns.to(device)
        self.rot_dim, self.interleaved, self.eps = rot_dim, interleaved, eps


class PagedCache:
    """Pools [n_pages, L, H, page_size, d] and the state of up to ``requests``
    requests of at most ``max_blocks`` pages; a step brings at most
    ``max_tokens`` new tokens with ``n_q_heads`` query heads.  ``dtype`` is "bf16", "f32" or
    "e4m3" (scaled pools: rows, queries and outputs are bf16, ``scale_block`` rows of a page
    share a power of two, ``exp_K`` and ``exp_V`` hold its exponent + 127).

    With a ``stream`` the state above is made on it and every call runs on it,
    behind what the current stream was given before the call; who reads state
    or results elsewhere waits for ``stream``."""

    def __init__(self, L: int, H: int, d: int, dtype: str, n_q_heads: int, n_pages: int,
                 page_size: int, requests: int, max_blocks: int, max_tokens: int,
                 device="cuda", stream: Optional[torch.cuda.Stream] = None, scale_block: int = 16):
        dev = torch.device(device)
        i32 = dict(dtype=torch.int32, device=dev)
        self.n_q_heads, self.max_tokens = n_q_heads, max_tokens
        self.device, self.stream = dev, stream
        self.pg = kvc.paged(n_pages, page_size, L, H, d, dtype, requests, max_blocks)
        self.scaled = dtype == "e4m3"
        self.row_dtype = torch.bfloat16 if self.scaled else _DTYPES[dtype]
        with torch.cuda.stream(stream):
            self.pool_K = torch.zeros((n_pages, L, H, page_size, d), dtype=_POOLS[dtype],
                                      device=dev)
            self.pool_V = torch.zeros_like(self.pool_K)
            if self.scaled:
                if not 1 <= scale_block <= 128:
                    raise ValueError("scale_block is 1 to 128 rows")
                block = min(scale_block, page_size)
                self.exp_K = torch.full((n_pages, L, H, -(-page_size // block)), 27,
                                        dtype=torch.uint8, device=dev)       # 2^-100
                self.exp_V = self.exp_K.clone()
                self.sc = kvc.scales(self.exp_K, self.exp_V, block)
            self.table = torch.zeros((requests, max_blocks), **i32)
            self.free_pages = torch.arange(n_pages - 1, -1, -1, **i32)   # page 0 is taken first
            self._n_free = [torch.full((1,), n_pages, **i32), torch.zeros(1, **i32)]
            self._kv_lens = [torch.zeros(requests, **i32) for _ in range(2)]
            self._now = self._planned = 0
            self._loaded = None                  # tokens a request of whole caches since the last plan
            self.q_start = torch.zeros(requests + 1, **i32)
            self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=dev)
            self.positions = torch.full((max_tokens,), -1, **i32)
            self.plan_status = torch.zeros(requests, **i32)
            self.dev_status = torch.zeros(1, **i32)
            # the largest step's size serves every step: it does not shrink with fewer tokens
            q = torch.empty((max_tokens, n_q_heads, d), dtype=self.row_dtype, device="meta")
            at = kvc.attn_params(q, q)
            ws = (kvc.kvc_paged_attention_scaled_workspace(self.pg, at, self.sc) if self.scaled
                  else kvc.kvc_paged_attention_workspace(self.pg, at))
            if ws == 0:
                raise ValueError("no attention of this shape: head dims are 64 or 128 in bf16 "
                                 "and e4m3, multiples of 4 up to 256 in f32, at most 64 query "
                                 "heads a KV head")
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
        self._now, self._planned, self._loaded = new, tokens, None

    def write(self, layer: int, K: torch.Tensor, V: torch.Tensor) -> None:
        """The planned tokens' rows [N, H, d] into their pages of a layer."""
        self._tokens(K)
        self._tokens(V)
        if K.shape[1] != self.pg.H or V.shape != K.shape:
            raise ValueError("K and V are [N, H, d] with the pools' heads")
        self._take(K, V)
        view = lambda x: x.permute(1, 0, 2)[None, None]  # noqa: E731   [1, 1, H, N, d]
        self._put(view(K), view(V), self.slots, layer, False)

    def load(self, K: torch.Tensor, V: torch.Tensor, rows: Optional[torch.Tensor] = None) -> None:
        """All layers of dense caches [requests, L, H, T, d] into the pages of
        the tokens just planned (T of each request); of those, where ``rows``
        ([requests, T] bool) is given, only the ones that it names.  Over scaled pools rows
        replace some of caches of the same T that were loaded whole since the plan."""
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
        if self.scaled and rows is not None and self._loaded != K.shape[3]:
            # the blocks' exponents would be those of the pages' last use
            raise ValueError("scaled pools take rows of caches once the caches were loaded whole")
        self._take(K, V, rows)
        with torch.cuda.stream(self.stream):
            slots = self.slots
            if rows is not None:
                slots = torch.where(rows.reshape(-1), slots[:rows.numel()], -1)
            self._put(K, V, slots, 0, rows is not None)
        if rows is None:
            self._loaded = K.shape[3]

    def _load_merged(self, K: torch.Tensor, V: torch.Tensor, own_K: torch.Tensor,
                     own_V: torch.Tensor, rows: torch.Tensor) -> None:
        """``load`` of K and V with ``rows`` out of own_K and own_V, in one write, a layer at a
        time: written over, the blocks would keep the exponents of the rows replaced and round
        the others a second time."""
        self._take(K, V, own_K, own_V, rows)
        with torch.cuda.stream(self.stream):
            mine = rows[:, None, None, :, None]
            for i in range(self.pg.L):
                k, v = (torch.where(mine, x[:, i:i + 1], y[:, i:i + 1])
                        for x, y in ((own_K, K), (own_V, V)))
                self._put(k, v, self.slots, i, False)
        self._loaded = K.shape[3]

    def rotate(self, rotary: Rotary, q: torch.Tensor, k: torch.Tensor,
               w_q: Optional[torch.Tensor] = None, w_k: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None):
        """The planned tokens' queries [N, heads, d] and keys [N, H, d] turned by their
        positions, with weights [d] of the norms where ``rotary`` has one, in place or into
        outputs; (queries, keys).  Rows of tokens that the plan refused stay as they are."""
        self._tokens(q)
        self._tokens(k)
        q_out, k_out = q if q_out is None else q_out, k if k_out is None else k_out
        for x, y in ((q, q_out), (k, k_out)):
            self._like_pools(y)
            if y.shape != x.shape or x.shape[0] != q.shape[0]:
                raise ValueError("queries, keys and outputs are of the same tokens and heads")
        for w in (w_q, w_k):
            if w is not None:
                self._like_pools(w)
                if w.shape != (self.pg.d,) or not w.is_contiguous() or rotary.eps is None:
                    raise ValueError("weights are [d], contiguous, and go with a norm's eps")
        if rotary.turns.device != q.device:
            raise ValueError("the rotation's table is on the pools' device")
        self._take(q, k, w_q, w_k, q_out, k_out, rotary.turns)
        rp = kvc.rotary_params(q, k, q_out, k_out, rotary.rot_dim, rotary.interleaved,
                               rotary.eps is not None, rotary.eps or 0.0, rotary.amplitude)
        kvc.kvc_rotate_heads(rp, q, k, self.positions, rotary.turns, q_out, k_out, w_q, w_k,
                             stream=self.stream)
        return q_out, k_out

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
        args = (q, self.pool_K, self.pool_V, self.table, self.q_start, self.kv_lens, out,
                self.workspace, self.dev_status)
        if self.scaled:
            kvc.kvc_paged_attention_scaled(self.pg, at, self.sc, *args, lse=lse, stream=self.stream)
        else:
            kvc.kvc_paged_attention(self.pg, at, *args, lse=lse, stream=self.stream)
        return out

    def _put(self, K: torch.Tensor, V: torch.Tensor, slots: torch.Tensor, layer: int,
             keep: bool) -> None:
        if self.scaled:
            kvc.kvc_page_write_scaled(self.pg, self.sc, K, V, slots, self.pool_K, self.pool_V,
                                      layer, keep, stream=self.stream)
        else:
            kvc.kvc_page_write(self.pg, K, V, slots, self.pool_K, self.pool_V, layer,
                               stream=self.stream)

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
        if x.dtype != self.row_dtype or x.device != self.pool_K.device:
            raise ValueError("what goes with the pools has their type (bf16 with e4m3) and is on "
                             "their device")


def from_chain(runner: ChainRunner, agent: int, n_q_heads: int, new_tokens: int,
               page_size: int = 16, dtype: Optional[str] = None,
               scale_block: int = 16) -> PagedCache:
    """Pages that hold agent ``agent``'s held caches of every request, with
    room for ``new_tokens`` more per request, in the chain's type or, of a bf16
    chain, as "e4m3".  A chain that reuses its output
    buffers hands out the agents whose rows are still there."""
    if not runner.holds(agent):
        raise ValueError("agent %d's cache is not in its buffer: the chain reuses them "
                         "(keep_outputs=False)" % agent)
    dtype = runner.wl.dtype if dtype is None else dtype
    if dtype != runner.wl.dtype and (dtype, runner.wl.dtype) != ("e4m3", "bf16"):
        raise ValueError("the pages of a %s chain are not %s" % (runner.wl.dtype, dtype))
    K, V = runner.held(agent)
    R, L, H, T, d = K.shape
    blocks = -(-(T + new_tokens) // page_size)
    pc = PagedCache(L, H, d, dtype, n_q_heads, R * blocks, page_size, R, blocks,
                    R * max(T, new_tokens), device=K.device, stream=runner.stream,
                    scale_block=scale_block)
    pc.plan([T] * R, R * T)
    if runner.own_prefix(agent):
        pc.load(K, V)
    elif pc.scaled:
        pc._load_merged(K, V, runner.inp.exact_K[agent], runner.inp.exact_V[agent], ~runner.ph_rows)
    else:
        pc.load(K, V)
        pc.load(runner.inp.exact_K[agent], runner.inp.exact_V[agent], ~runner.ph_rows)
    return pc


def decode_graph(pc: PagedCache, new_lens: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                 v: torch.Tensor, out: torch.Tensor,
                 rotary: Optional[Rotary] = None) -> torch.cuda.CUDAGraph:
    """Two steps over all layers as a CUDA graph: tokens ``q``, ``out``
    [2, L, N, n_q_heads, d] and ``k``, ``v`` [2, L, N, H, d], read at replay,
    queries and keys turned by their positions on the way if there is a ``rotary``.
    The graph keeps them, ``new_lens`` and the cache for as long as it lives."""
    if pc.stream is not None:
        raise ValueError("a captured step runs on the capturing stream: stream=None")
    turned = (torch.empty_like(q[0, 0]), torch.empty_like(k[0, 0])) if rotary else None

    def two_steps(lens):
        for s in range(2):
            pc.plan(lens, q.shape[2])
            for i in range(pc.pg.L):
                qi, ki = q[s, i], k[s, i]
                if rotary is not None:
                    qi, ki = pc.rotate(rotary, qi, ki, q_out=turned[0], k_out=turned[1])
                pc.write(i, ki, v[s, i])
                pc.attend(i, qi, out[s, i])

    two_steps(torch.zeros_like(new_lens))                # loads the kernels, changes nothing
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        two_steps(new_lens)
    graph.buffers = (pc, new_lens, q, k, v, out, rotary, turned)   # which a replay reads and writes
    return graph


def main(argv: Optional[Sequence[str]] = None) -> None:
    ap = argparse.ArgumentParser(description="decode from the corrected caches of a chain")
    ap.add_argument("--workload", default="tiny")
    ap.add_argument("--layers", type=int, default=None, help="shrink the workload to these layers")
    ap.add_argument("--group", type=int, default=4, help="query heads per KV head")
    ap.add_argument("--prompt", type=int, default=128, help="tokens of the agent's prompt")
    ap.add_argument("--steps", type=int, default=64, help="tokens to decode, an even number")
    ap.add_argument("--page-size", type=int, default=16)
    ap.add_argument("--cache", choices=["bf16", "f32", "e4m3"], default=None,
                    help="type of the pages (default: the chain's)")
    ap.add_argument("--scale-block", type=int, default=16, help="rows of a power of two (e4m3)")
    ap.add_argument("--rotary", action="store_true", help="norms and rotation of the new tokens' heads")
    a = ap.parse_args(argv)
    if a.steps < 2 or a.steps % 2 or a.prompt < 1:
        ap.error("--steps is even and at least 2, --prompt at least 1")
    wl = synth.workload(a.workload)
    if a.layers is not None:
        wl = synth.scaled(wl, L=a.layers)
    runner = ChainRunner(wl, synth.generate(wl, device="cuda"))
    runner.run()
    Hq = wl.H * a.group
    pc = from_chain(runner, wl.n_agents - 1, Hq, a.prompt + a.steps + 2, a.page_size, a.cache,
                    a.scale_block)
    rotary = Rotary(wl.d, 500000.0, eps=1e-6) if a.rotary else None

    def rows(*shape):
        return torch.randn(shape, device="cuda").to(_DTYPES[wl.dtype])

    N = wl.R * a.prompt
    pc.plan([a.prompt] * wl.R, N)
    for i in range(wl.L):
        q, k = rows(N, Hq, wl.d), rows(N, wl.H, wl.d)
        if rotary is not None:
            pc.rotate(rotary, q, k)
        pc.write(i, k, rows(N, wl.H, wl.d))
        pc.attend(i, q)

    ones = torch.ones(wl.R, dtype=torch.int32, device="cuda")
    q, k, v = rows(2, wl.L, wl.R, Hq, wl.d), *(rows(2, wl.L, wl.R, wl.H, wl.d) for _ in "kv")
    out = torch.empty_like(q)
    graph = decode_graph(pc, ones, q, k, v, out, rotary)
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
          f"{Hq}/{wl.H} heads of {wl.d}, {a.cache or wl.dtype}: {1e3 * ms:.1f} us per decoded step "
          f"({1e3 * ms / wl.L:.1f} per layer), {wl.R / ms * 1e3:.0f} tokens/s")


if __name__ == "__main__":
    main()
