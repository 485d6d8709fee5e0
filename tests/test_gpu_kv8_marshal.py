"""The C marshaller of the 8-bit cache's and the prompts' calls: a call in the plain form goes through it and does what
the binding's Python path does; anything else is left to that path (which refuses or makes it)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rlt(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return rlt


class Nothing:
    """A marshaller that takes no call."""

    def __init__(self):
        self.append = self.decode = self.prefill = lambda *a: None


class Watch:
    """The marshaller, counting the calls it took."""

    def __init__(self, m):
        self.took = 0
        for name in ("append", "decode", "prefill"):
            def call(*a, f=getattr(m, name)):
                r = f(*a)
                self.took += r is not None
                return r
            setattr(self, name, call)


def inputs(rlt, n=37, hq=6, hkv=2, d=64):
    import torch
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g).bfloat16().cuda()
    s = {"q": x[:, :hq], "k": x[:, hq:hq + hkv], "v": x[:, hq + hkv:], "pos": torch.arange(n).cuda(),
         "slots": torch.arange(n).cuda(), "table": torch.arange(3, dtype=torch.int32).cuda()[None],
         "lens": torch.tensor([n], dtype=torch.int32).cuda(), "n": n}
    s["plan"] = rlt.rlt_plan_prefill([20, 17], hq // hkv).to("cuda")
    return s


def chain(rlt, s, **kw):
    """Append, prompts and one request's decode; every output."""
    import torch
    n, hq, d = s["q"].shape
    pool = rlt.KV8Pool(*(torch.zeros(1, 3, s["k"].shape[1], 16, d, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                         for _ in range(2)),
                       *(torch.full((1, 3, s["k"].shape[1], 16), 127, dtype=torch.uint8, device="cuda") for _ in range(2)))
    qo, ko, vo = (torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"], s["v"]))
    rlt.rlt_kv8_append_rope(pool, 0, s["k"], s["v"], s["pos"], s["slots"], d, 1e4, q=s["q"], q_out=qo, k_out=ko, v_out=vo, **kw)
    out, lse = torch.empty_like(qo), torch.empty(n, hq, device="cuda")
    rlt.rlt_prefill_attn(qo, ko, vo, s["plan"], out=out, lse_out=lse, **kw)
    one, one_lse = torch.empty_like(qo[:1]), torch.empty(1, hq, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    rlt.rlt_paged_decode_attn_kv8(pool, 0, qo[-1:], s["table"], s["lens"], n, out=one, lse_out=one_lse, workspace=ws,
                                  split_tokens=16, **kw)
    torch.cuda.synchronize()
    return [qo, ko, vo, out, lse, one, one_lse, pool.k.view(torch.uint8), pool.v.view(torch.uint8), pool.k_exp, pool.v_exp]


@pytest.mark.parametrize("stream", ["current", "object", "handle"])
def test_both_paths_agree(rlt, monkeypatch, stream):
    import torch
    s = inputs(rlt)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    kw = {} if stream == "current" else {"stream": other if stream == "object" else other.cuda_stream}
    watch = Watch(rlt._plain())
    monkeypatch.setattr(rlt, "_bound", watch)
    got = chain(rlt, s, **kw)
    assert watch.took == 3
    monkeypatch.setattr(rlt, "_bound", Nothing())
    want = chain(rlt, s, **kw)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert rlt.rlt_get_device_error() == 0


def test_other_forms_are_left_alone(rlt):
    import torch
    s, m, d = inputs(rlt), rlt._plain(), 64
    n, hkv = s["n"], 2
    pool = rlt.KV8Pool.empty(1, 3, hkv, 16, d)
    good = [pool.address, pool.device_index, hkv, d, 0, s["k"], s["v"], s["pos"], s["slots"], d, 1e4, None, None, None, None, None]
    bad = {1: 7, 5: s["k"].float(), 6: s["v"].cpu(), 7: s["pos"].int(), 8: s["slots"][:-1], 9: 64.0, 10: "1e4", 11: s["q"],
           12: s["q"], 13: s["k"], 14: torch.empty(n, hkv, d, device="cuda"), 15: "stream", 4: 1 << 40}
    for i, x in bad.items():
        call = list(good)
        call[i] = x
        assert m.append(*call) is None, i
    assert m.append(*good[:-1]) is None and m.append() is None
    call = list(good)
    call[5] = s["k"].transpose(0, 2).contiguous().transpose(0, 2)     # heads of a token apart
    assert m.append(*call) is None
    # a status of the library is handed on: a bank outside the pool
    call = list(good)
    call[4] = 3
    assert m.append(*call) == 2                 # RLT_ERR_OUT_OF_RANGE
    q = torch.randn(1, 6, d, device="cuda").bfloat16()
    out, ws = torch.empty_like(q), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    good = [pool.address, pool.device_index, d, 0, q, s["table"], s["lens"], n, out, None, ws, 0.0, 0, 0, None]
    bad = {2: 128, 4: q[:, ::2], 5: s["table"].long(), 6: s["lens"].repeat(2), 7: 3.5, 8: None, 9: out, 10: None, 14: 1.5}
    for i, x in bad.items():
        call = list(good)
        call[i] = x
        assert m.decode(*call) is None, i
    full = torch.empty(n, 6, d, dtype=torch.bfloat16, device="cuda")
    p = s["plan"]
    good = [s["q"], s["k"], s["v"], p.dev, p.num_items, p.num_rows, p.max_key_tiles, p.total_key_tiles, 3, full, None, 0.0, 0, None]
    bad = {0: s["q"][:30], 1: s["k"][:30], 2: s["q"], 3: None, 4: p.num_items + 1, 5: n + 1, 8: 2, 9: None, 10: full, 13: []}
    for i, x in bad.items():
        call = list(good)
        call[i] = x
        assert m.prefill(*call) is None, i
    torch.cuda.synchronize()
    assert rlt.rlt_get_device_error() == 0


def test_no_reference_is_lost_or_kept(rlt):
    import sys
    import torch
    s, m = inputs(rlt), rlt._plain()
    pool = rlt.KV8Pool.empty(1, 3, 2, 16, 64)
    watched = [s["q"], s["k"], s["v"], s["pos"], s["slots"], torch.bfloat16, torch.int64]
    qo = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    call = [pool.address, pool.device_index, 2, 64, 0, s["k"], s["v"], s["pos"], s["slots"], 64, 1e4, s["q"], qo, None, None, None]
    assert m.append(*call) == 0
    before = [sys.getrefcount(x) for x in watched]
    for _ in range(50):
        assert m.append(*call) == 0
        assert m.append(*call[:9], "x", *call[10:]) is None
    assert [sys.getrefcount(x) for x in watched] == before
    torch.cuda.synchronize()
