"""C-ABI boundary of the paged-cache calls, without a GPU: every malformed call
is refused with its documented status before anything is launched.  As in
test_boundary.py the device addresses are fake and never dereferenced, so the
file only runs where no GPU is visible."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake device addresses are only passed where no GPU exists")

from agent_shared_context_gb300 import kvc  # noqa: E402

FAKE = 0x7F0000000000
FAR = 1 << 34                                   # spacing of the fake buffers


def _pg(**over):
    a = dict(n_pages=64, page_size=16, L=2, H=2, d=128, dtype="bf16", R=3, max_blocks=20)
    a.update(over)
    return kvc.paged(**a)


def _pool(i, pg, **over):
    s_tok = pg.d
    s_head = pg.page_size * s_tok
    st = [pg.L * pg.H * s_head, pg.H * s_head, s_head, s_tok]
    for k, v in over.items():
        st[["s_req", "s_layer", "s_head", "s_tok"].index(k)] = v
    return kvc.cache_view(FAKE + i * FAR, st)


def _plan(pg=None, max_tokens=100, **over):
    names = ("new_lens", "kv_lens", "kv_lens_out", "block_table", "free_pages", "n_free", "n_free_out",
             "q_start", "slot_map", "positions", "plan_status")
    a = {n: FAKE + i * FAR for i, n in enumerate(names)}
    a.update(over)
    return kvc.kvc_page_plan(pg or _pg(), stream=0, max_tokens=max_tokens, check=False, **a)


def test_plan_refusals():
    for n in ("new_lens", "kv_lens", "kv_lens_out", "block_table", "free_pages", "n_free", "n_free_out",
              "q_start", "slot_map", "positions", "plan_status"):
        assert _plan(**{n: None}) == kvc.KVC_ERR_INVALID_ARGUMENT, n
        assert n in kvc.lib.kvc_last_error().decode()
        assert _plan(**{n: FAKE + 30 * FAR + 2}) == kvc.KVC_ERR_ALIGNMENT, n
    assert _plan(slot_map=FAKE + 30 * FAR + 4) == kvc.KVC_ERR_ALIGNMENT
    assert _plan(_pg(R=4097)) == kvc.KVC_ERR_UNSUPPORTED
    assert _plan(max_tokens=-1) == kvc.KVC_ERR_SHAPE
    # the state comes out in other buffers than it went in by
    assert _plan(kv_lens_out=FAKE + 1 * FAR) == kvc.KVC_ERR_ALIAS
    assert _plan(n_free_out=FAKE + 5 * FAR) == kvc.KVC_ERR_ALIAS
    assert _plan(positions=FAKE + 8 * FAR + 8 * 100 - 4) == kvc.KVC_ERR_ALIAS
    assert _plan(new_lens=FAKE + 3 * FAR + 4 * 59) == kvc.KVC_ERR_ALIAS    # inside the table


@pytest.mark.parametrize("over,status", [
    (dict(n_pages=0), "SHAPE"), (dict(page_size=0), "SHAPE"), (dict(L=0), "SHAPE"), (dict(H=0), "SHAPE"),
    (dict(max_blocks=0), "SHAPE"), (dict(R=-1), "SHAPE"), (dict(dtype=7), "DTYPE"),
    (dict(n_pages=(1 << 30) + 1), "UNSUPPORTED"), (dict(max_blocks=1 << 27), "UNSUPPORTED"),
])
def test_descriptor_refusals(over, status):
    want = getattr(kvc, "KVC_ERR_" + status)
    assert _plan(_pg(**over)) == want
    assert _write(_pg(**over)) == want
    assert _attend(_pg(**over)) == want


def _write(pg=None, shape=(1, 1, 50), **over):
    pg = pg or _pg()
    src = lambda i: kvc.cache_view(FAKE + i * FAR, (1 << 20, 1 << 18, 128, 256))  # noqa: E731
    a = dict(src_K=src(10), src_V=src(11), slot_map=FAKE + 12 * FAR, pool_K=_pool(13, pg), pool_V=_pool(14, pg))
    a.update(over)
    return kvc.kvc_page_write(pg, stream=0, shape=shape, check=False, **a)


def test_write_refusals():
    null = kvc.cache_view(None)
    for n in ("src_K", "src_V", "pool_K", "pool_V"):
        assert _write(**{n: null}) == kvc.KVC_ERR_INVALID_ARGUMENT, n
        odd = kvc.cache_view(FAKE + 20 * FAR + 8, (1 << 20, 1 << 18, 2048, 128))
        assert _write(**{n: odd}) == kvc.KVC_ERR_ALIGNMENT, n
        row = kvc.cache_view(FAKE + 20 * FAR, (1 << 20, 1 << 18, 2048, 132))
        assert _write(**{n: row}) == kvc.KVC_ERR_ALIGNMENT, n
        short = kvc.cache_view(FAKE + 20 * FAR, (1 << 20, 1 << 18, 2048, 64))
        assert _write(**{n: short}) == kvc.KVC_ERR_SHAPE, n
        wide = kvc.cache_view(FAKE + 20 * FAR, (1 << 40, 1 << 18, 2048, 128))
        assert _write(**{n: wide}) == kvc.KVC_ERR_UNSUPPORTED, n
    assert _write(slot_map=None) == kvc.KVC_ERR_INVALID_ARGUMENT
    assert _write(slot_map=FAKE + 4) == kvc.KVC_ERR_ALIGNMENT
    assert _write(shape=(1, 3, 50)) == kvc.KVC_ERR_SHAPE                 # three layers of two
    assert _write(layer=2) == kvc.KVC_ERR_SHAPE
    assert _write(layer=-1) == kvc.KVC_ERR_SHAPE
    assert _write(shape=(-1, 1, 50)) == kvc.KVC_ERR_SHAPE
    assert _write(_pg(d=96)) == kvc.KVC_ERR_UNSUPPORTED
    assert _write(_pg(d=6, dtype="f32")) == kvc.KVC_ERR_UNSUPPORTED
    big = _pg(L=40000)
    assert _write(big, shape=(1, 40000, 1)) == kvc.KVC_ERR_UNSUPPORTED
    pg = _pg()
    inside = kvc.cache_view(FAKE + 14 * FAR + 4096, (1 << 20, 1 << 18, 128, 256))
    assert _write(pg, src_V=inside) == kvc.KVC_ERR_ALIAS
    assert _write(shape=(0, 1, 50)) == kvc.KVC_OK                         # nothing to write
    assert _write(shape=(1, 1, 0), slot_map=None) == kvc.KVC_OK


def _att(pg, **over):
    a = dict(n_q_heads=8, n_tokens=30, layer=1, causal=1, window=0, scale=0.1, q_s_tok=8 * pg.d,
             q_s_head=pg.d, out_s_tok=8 * pg.d, out_s_head=pg.d)
    a.update(over)
    return kvc.kvc_attn_params(**a)


def _attend(pg=None, at=None, ws=None, **over):
    pg = pg or _pg()
    at = at or _att(pg)
    a = dict(q=FAKE, pool_K=_pool(1, pg), pool_V=_pool(2, pg), block_table=FAKE + 3 * FAR,
             q_start=FAKE + 4 * FAR, kv_lens=FAKE + 5 * FAR, out=FAKE + 6 * FAR, lse=FAKE + 7 * FAR,
             workspace=FAKE + 8 * FAR, dev_status=FAKE + 9 * FAR)
    a.update(over)
    return kvc.kvc_paged_attention(pg, at, stream=0, workspace_bytes=1 << 33 if ws is None else ws,
                                   check=False, **a)


def test_attention_refusals():
    pg = _pg()
    for n in ("q", "out", "block_table", "q_start", "kv_lens", "dev_status"):
        assert _attend(**{n: None}) == kvc.KVC_ERR_INVALID_ARGUMENT, n
    for n in ("pool_K", "pool_V"):
        assert _attend(**{n: kvc.cache_view(None)}) == kvc.KVC_ERR_INVALID_ARGUMENT, n
        assert _attend(**{n: _pool(20, pg, s_tok=132)}) == kvc.KVC_ERR_ALIGNMENT, n
        assert _attend(**{n: _pool(20, pg, s_tok=64)}) == kvc.KVC_ERR_SHAPE, n
    for over, st in [(dict(n_q_heads=7), "SHAPE"), (dict(n_q_heads=0), "SHAPE"),
                     (dict(n_q_heads=130), "UNSUPPORTED"), (dict(n_tokens=-1), "SHAPE"),
                     (dict(layer=2), "SHAPE"), (dict(layer=-1), "SHAPE"),
                     (dict(causal=2), "INVALID_ARGUMENT"), (dict(window=-1), "INVALID_ARGUMENT"),
                     (dict(causal=0, window=5), "INVALID_ARGUMENT"), (dict(scale=0.0), "INVALID_ARGUMENT"),
                     (dict(scale=float("inf")), "INVALID_ARGUMENT"), (dict(scale=float("nan")), "INVALID_ARGUMENT"),
                     (dict(q_s_head=64), "SHAPE"), (dict(out_s_head=-128), "SHAPE"),
                     (dict(out_s_tok=0), "SHAPE"), (dict(q_s_tok=1028), "ALIGNMENT"),
                     (dict(out_s_head=132), "ALIGNMENT"), (dict(q_s_tok=1 << 40), "UNSUPPORTED")]:
        assert _attend(pg, _att(pg, **over)) == getattr(kvc, "KVC_ERR_" + st), over
        if not any(k.endswith(("tok", "head")) for k in over):
            assert kvc.kvc_paged_attention_workspace(pg, _att(pg, **over)) == 0
    assert _attend(_pg(d=96)) == kvc.KVC_ERR_UNSUPPORTED
    assert _attend(q=FAKE + 8) == kvc.KVC_ERR_ALIGNMENT
    assert _attend(lse=FAKE + 30 * FAR + 2) == kvc.KVC_ERR_ALIGNMENT
    need = kvc.kvc_paged_attention_workspace(pg, _att(pg))
    assert need > 8192
    assert _attend(ws=need - 1) == kvc.KVC_ERR_WORKSPACE
    assert _attend(workspace=None) == kvc.KVC_ERR_WORKSPACE
    assert _attend(workspace=FAKE + 30 * FAR + 128) == kvc.KVC_ERR_ALIGNMENT
    assert _attend(out=FAKE) == kvc.KVC_ERR_ALIAS                          # over the queries
    assert _attend(out=FAKE + 2 * FAR) == kvc.KVC_ERR_ALIAS                # over the values
    assert _attend(lse=FAKE + 6 * FAR) == kvc.KVC_ERR_ALIAS                # over the output
    assert _attend(workspace=FAKE + 7 * FAR) == kvc.KVC_ERR_ALIAS          # over lse


def test_attention_with_nothing_to_do_is_a_no_op():
    pg = _pg()
    assert _attend(pg, _att(pg, n_tokens=0), q=None, out=None) == kvc.KVC_OK
    assert _attend(_pg(R=0), block_table=None, q_start=None, kv_lens=None) == kvc.KVC_OK


def test_binding_takes_strided_tensors_and_checks_shapes():
    q = torch.zeros(5, 12, 64)[:, 2:10]
    out = torch.zeros(8, 5, 64).permute(1, 0, 2)
    a = kvc.attn_params(q, out)
    assert (a.n_q_heads, a.n_tokens, a.q_s_tok, a.q_s_head) == (8, 5, 768, 64)
    assert (a.out_s_tok, a.out_s_head) == (64, 320)
    assert abs(a.scale - 0.125) < 1e-9
    with pytest.raises(ValueError):
        kvc.attn_params(q, out[:, :4])
    with pytest.raises(ValueError):
        kvc.attn_params(q.transpose(1, 2), q.transpose(1, 2))
    with pytest.raises(kvc.KvcError) as e:
        kvc.kvc_page_plan(_pg(), None, *[FAKE + i * FAR for i in range(7)], 1 << 20, 1 << 21, 1 << 22,
                          stream=0, max_tokens=4)
    assert e.value.status == kvc.KVC_ERR_INVALID_ARGUMENT and "new_lens" in str(e.value)


def test_struct_sizes():
    assert ctypes.sizeof(kvc.kvc_paged) == 32
    assert ctypes.sizeof(kvc.kvc_attn_params) == 56
