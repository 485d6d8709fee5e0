"""Debug mode RLT_VALIDATE=1 of the 8-bit cache's calls: a batch that breaks the rules of slots, pages or
lengths is refused with a status and nothing is launched; a valid one runs as without the mode."""
import pytest

from test_gpu_kv8_append import dev, make_pool      # noqa: F401  (dev: fixture)
from test_gpu_kv8_decode import Case

pytestmark = pytest.mark.gpu

OUT_OF_RANGE = 2


@pytest.fixture(autouse=True)
def validate(monkeypatch):
    monkeypatch.setenv("RLT_VALIDATE", "1")


@pytest.mark.parametrize("slots,status", [([5, -1, 9, 0], None), ([5, -1, 48, 0], OUT_OF_RANGE), ([5, -1, 9, 5], 1)])
def test_append_slots(dev, slots, status):          # noqa: F811
    import torch
    import paged_kv_looped_gb300 as rlt
    pool = make_pool(rlt, torch, dev, 1, 3, 2, 16, 64, 1)
    before = pool.k.view(torch.uint8).clone(), pool.k_exp.clone()
    k, v = (torch.randn(4, 2, 64, device=dev).bfloat16() for _ in range(2))
    out = torch.full_like(k, 7.0)
    where = torch.tensor(slots, device=dev)
    run = lambda: rlt.rlt_kv8_append_rope(pool, 0, k, v, torch.arange(4, device=dev), where, 64, 10000.0,
                                          k_out=out)  # noqa: E731
    rlt.rlt_get_device_error()
    if status is None:
        run()
        assert rlt.rlt_get_device_error() == 0
        assert not torch.equal(out, torch.full_like(k, 7.0))
        assert not torch.equal(pool.k.view(torch.uint8), before[0])
    else:
        with pytest.raises(rlt.RltError) as e:
            run()
        assert e.value.status == status
        assert rlt.rlt_get_device_error() == 0
        assert torch.all(out == 7.0)
        assert torch.equal(pool.k.view(torch.uint8), before[0]) and torch.equal(pool.k_exp, before[1])


@pytest.mark.parametrize("page,length,status", [(None, None, None), (10 ** 6, None, OUT_OF_RANGE), (None, 10 ** 6, OUT_OF_RANGE)])
def test_decode_batch(dev, page, length, status):   # noqa: F811
    import paged_kv_looped_gb300 as rlt
    c = Case(dev, [40, 3, 17], 4, 2, 64, 16)
    ref = c.reference()
    if page is not None:
        c.table[1, 0] = page
    if length is not None:
        c.seq[2] = length
    rlt.rlt_get_device_error()
    if status is None:
        c.check(*c.run(), ref)
    else:
        with pytest.raises(rlt.RltError) as e:
            c.run()
        assert e.value.status == status
    assert rlt.rlt_get_device_error() == 0
