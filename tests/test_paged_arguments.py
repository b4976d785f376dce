"""PagedCache refuses tensors that do not fit its pools before anything is launched.
The tensors lie in host memory, so that no launch could take them: no GPU is needed."""
import pytest

torch = pytest.importorskip("torch")

from agent_shared_context_gb300 import paged  # noqa: E402

OTHER = {"bf16": torch.float32, "f32": torch.bfloat16}


def _cache(dtype, planned=6, device="cpu"):
    """2 layers, 4 KV heads of 64, 8 query heads, 2 requests; `planned` tokens."""
    pc = paged.PagedCache(2, 4, 64, dtype, 8, 16, 8, 2, 4, 12, device=device)
    pc._planned = planned
    return pc


@pytest.fixture(params=["bf16", "f32"])
def pc(request):
    return _cache(request.param)


def _other(pc):
    return torch.float32 if pc.pool_K.dtype == torch.bfloat16 else torch.bfloat16


def _refused(call, *args, **kw):
    with pytest.raises(ValueError) as e:
        call(*args, **kw)
    return str(e.value)


def test_write_refuses_rows_that_do_not_fit(pc):
    dt = pc.pool_K.dtype
    good = torch.zeros((6, 4, 64), dtype=dt)
    for heads in (1, 3, 5, 8):                     # fewer would be read past their end
        bad = torch.zeros((6, heads, 64), dtype=dt)
        assert "heads" in _refused(pc.write, 0, bad, bad)
    for bad in (good.to(_other(pc)), good[:5], good[:, :3], good[:, :, :32],
                torch.zeros((6, 4, 64), dtype=dt, device="meta")):
        _refused(pc.write, 0, good, bad)
        _refused(pc.write, 0, bad, good)
    _refused(pc.write, 0, torch.zeros((7, 4, 64), dtype=dt), torch.zeros((7, 4, 64), dtype=dt))


def test_load_refuses_caches_that_do_not_fit(pc):
    dt = pc.pool_K.dtype
    good = torch.zeros((2, 2, 4, 3, 64), dtype=dt)
    for bad in (good.to(_other(pc)), good[..., :32], good[:, :, :3], good[:, :1], good[:1],
                torch.zeros((2, 2, 4, 3, 128), dtype=dt), good[:, :, :, :2],
                torch.zeros((2, 2, 4, 3, 64), dtype=dt, device="meta")):
        _refused(pc.load, good, bad)
        _refused(pc.load, bad, good)
    for bad in (good.to(_other(pc)), good[..., :32],
                torch.zeros((2, 2, 4, 4, 64), dtype=dt)):           # more than was planned
        _refused(pc.load, bad, bad)
    for rows in (torch.ones((2, 4), dtype=torch.bool), torch.ones((2, 3)),
                 torch.ones(6, dtype=torch.bool), torch.ones((2, 3), dtype=torch.bool, device="meta")):
        _refused(pc.load, good, good, rows)


def test_attend_refuses_outputs_that_do_not_fit(pc):
    dt = pc.pool_K.dtype
    q = torch.zeros((6, 8, 64), dtype=dt)
    for bad in (q.to(_other(pc)), q[:5], q[:, :4], torch.zeros((6, 8, 128), dtype=dt),
                torch.zeros((6, 8, 64), dtype=dt, device="meta"),
                torch.zeros((6, 64, 8), dtype=dt).transpose(1, 2)):
        _refused(pc.attend, 0, q, bad)
    for bad in (torch.zeros((6, 8), dtype=torch.float16), torch.zeros((6, 8), dtype=torch.float64),
                torch.zeros((5, 8)), torch.zeros((6, 4)), torch.zeros(48), torch.zeros((8, 6)).T,
                torch.zeros((6, 8), device="meta")):
        assert "lse" in _refused(pc.attend, 0, q, lse=bad)
    for bad in (torch.zeros((6, 8, 64), dtype=dt, device="meta"), q.to(_other(pc))):
        _refused(pc.attend, 0, bad)


def test_plan_refuses_lengths_elsewhere(pc):
    for bad in (torch.zeros(2, dtype=torch.int32, device="meta"), torch.zeros(2, dtype=torch.int64),
                torch.zeros((2, 1), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)):
        _refused(pc.plan, bad)


def test_writing_nothing_takes_empty_tensors():
    """An empty tensor has no address."""
    from agent_shared_context_gb300 import kvc
    pg = kvc.paged(16, 8, 2, 4, 64, "bf16", 2, 4)
    pool = kvc.cache_view(0x7F0000000000, (2 * 4 * 8 * 64, 4 * 8 * 64, 8 * 64, 64))
    for shape in ((0, 2, 4, 3, 64), (2, 2, 4, 0, 64)):
        x = torch.zeros(shape, dtype=torch.bfloat16)
        assert kvc.kvc_page_write(pg, x, x, None, pool, pool, stream=0) == kvc.KVC_OK
        with pytest.raises(kvc.KvcError):          # the rest is looked at all the same
            kvc.kvc_page_write(pg, x, x, None, kvc.cache_view(None), pool, stream=0)
        with pytest.raises(kvc.KvcError):
            kvc.kvc_page_write(pg, x, x, None, pool, pool, layer=1, stream=0)
