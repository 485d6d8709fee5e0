"""Paged decode attention over the 8-bit cache, against the 64-bit reference."""
import numpy as np
import pytest

import kv8_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    return cuda_device


class Case:
    """A filled pool, page tables in random order and queries; everything no request maps (rows behind
    a request's end among it) holds NaN with the largest exponent."""

    def __init__(self, dev, lens, hq, hkv, d, ps, seed=0, spread=0.1, banks=2, bank=1, q_scale=1.0):
        import torch
        import paged_kv_looped_gb300 as rlt
        rng = np.random.default_rng(seed)
        B = len(lens)
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages)
        width = max(max(need), 1) + 1
        self.tables = np.full((B, width), -7, np.int32)
        k8 = np.full((banks, pages, hkv, ps, d), 0x7F, np.uint8)
        v8, ke, ve = k8.copy(), np.full((banks, pages, hkv, ps), 255, np.uint8), None
        ve = ke.copy()
        at = 0
        for b, n in enumerate(lens):
            self.tables[b, : need[b]] = order[at: at + need[b]]
            at += need[b]
            for i in range(need[b]):
                m = min(ps, n - i * ps)
                pg = self.tables[b, i]
                for x8, xe in ((k8, ke), (v8, ve)):
                    rows = rng.standard_normal((hkv, m, d)) * np.exp2(np.round(rng.standard_normal((hkv, m, 1)) * spread * 4))
                    e = R.row_exponent(rows)
                    val = torch.from_numpy(R.e4m3(rows * np.exp2(-e)[..., None])).float().to(torch.float8_e4m3fn)
                    x8[bank, pg, :, :m] = val.view(torch.uint8).numpy()
                    xe[bank, pg, :, :m] = (e + 127).astype(np.uint8)
        t = lambda a: torch.from_numpy(a).to(dev)              # noqa: E731
        self.pool = rlt.KV8Pool(t(k8).view(torch.float8_e4m3fn), t(v8).view(torch.float8_e4m3fn), t(ke), t(ve))
        self.bank, self.lens, self.ps = bank, np.array(lens, np.int32), ps
        self.q = (torch.from_numpy(rng.standard_normal((B, hq, d))) * q_scale).bfloat16().to(dev)
        self.table, self.seq = t(self.tables), t(self.lens)
        dec = lambda x8, xe: (torch.from_numpy(x8[bank]).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)  # noqa: E731
                              * np.exp2(xe[bank].astype(np.float64) - 127)[..., None])
        self.k, self.v = dec(k8, ke), dec(v8, ve)
        self.scale = 1 / np.sqrt(d)

    def reference(self):
        return R.decode(self.q.float().cpu().numpy().astype(np.float64), self.k, self.v, self.tables, self.lens, self.ps,
                        self.scale)

    def run(self, **kw):
        import torch
        import paged_kv_looped_gb300 as rlt
        lse = torch.full(self.q.shape[:2], 5.0, device=self.q.device)
        out = rlt.rlt_paged_decode_attn_kv8(self.pool, self.bank, self.q, self.table, self.seq,
                                            kw.pop("max_seq_len", int(self.lens.max(initial=0))), lse_out=lse, **kw)
        return out, lse

    def check(self, out, lse, ref=None):
        import torch
        torch.cuda.synchronize()
        o, l, mag, terms = self.reference() if ref is None else ref
        go, gl = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        assert np.isfinite(go).all()
        assert np.array_equal(np.isneginf(gl), np.isneginf(l))
        fin = np.isfinite(l)
        assert np.all(np.abs(gl[fin] - l[fin]) <= R.lse_bound(l, terms, o.shape[-1])[fin]), np.abs(gl[fin] - l[fin]).max(initial=0)
        assert np.all(np.abs(go - o) <= R.attention_bound(o, mag, terms, 2.0 ** -11)), np.abs(go - o).max()


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 300]


@pytest.mark.parametrize("hq,hkv,d,ps", [(2, 2, 64, 16), (4, 2, 64, 32), (6, 2, 128, 16), (4, 1, 128, 64),
                                         (5, 1, 64, 256), (12, 2, 128, 128), (7, 1, 128, 16), (8, 1, 128, 16),
                                         (16, 2, 64, 48), (3, 3, 128, 16)])
@pytest.mark.parametrize("split", [0, 16, 48, 128])
def test_lengths_around_tiles(dev, hq, hkv, d, ps, split):
    import paged_kv_looped_gb300 as rlt
    c = Case(dev, EDGES, hq, hkv, d, ps, seed=hq + d)
    c.check(*c.run(split_tokens=split))
    assert rlt.rlt_get_device_error() == 0


@pytest.mark.parametrize("lens,hq,hkv,d,ps", [([5000, 1, 0, 777], 8, 2, 128, 16), ([9001], 4, 4, 64, 64),
                                              ([4096, 4097, 2047], 8, 1, 128, 256), ([0, 0], 4, 2, 128, 16)])
@pytest.mark.parametrize("split", [0, 2048, 512])
def test_long_and_empty(dev, lens, hq, hkv, d, ps, split):
    c = Case(dev, lens, hq, hkv, d, ps, seed=7)
    c.check(*c.run(split_tokens=split))


@pytest.mark.parametrize("d", [64, 128])
def test_scales_far_apart(dev, d):
    """Rows whose scales span 2^40: one-hot weights, tiny values under large weights and the reverse."""
    c = Case(dev, [100, 513, 40], 8, 2, d, 16, seed=11, spread=2.5, q_scale=0.05)
    c.check(*c.run(split_tokens=64))
    c.check(*c.run())


def test_query_scales_zero_heads_and_nan(dev):
    import torch
    c = Case(dev, [70, 33], 8, 2, 128, 16, seed=12)
    c.q[0, 0] = 0.0
    c.q[0, 1] *= 2.0 ** -120
    c.q[0, 2, :64] *= 2.0 ** -20
    c.q[1, 3] = c.q[1, 3] * 2.0 ** -130
    c.check(*c.run())
    for split in (0, 32):
        c.q[1, 6, 5] = 1.0
        ref, _ = c.run(split_tokens=split)
        c.q[1, 6, 5] = float("nan")                             # one head's NaN stays its own
        out, lse = c.run(split_tokens=split)
        torch.cuda.synchronize()
        assert torch.isnan(out[1, 6]).all() and torch.isnan(lse[1, 6])
        keep = torch.ones(2, 8, dtype=torch.bool)
        keep[1, 6] = False
        assert torch.equal(out[keep], ref[keep])


def test_bad_pages_and_lengths(dev):
    import paged_kv_looped_gb300 as rlt
    c = Case(dev, [100, 60, 200], 8, 2, 128, 16, seed=13)
    c.tables[0, 2] = 1 << 20
    c.tables[1, 0] = -1
    c.tables[2, :] = 99999                                      # nothing of this request is in the pool
    c.table.copy_(__import__("torch").from_numpy(c.tables))
    for split in (0, 32):
        c.check(*c.run(split_tokens=split))
        assert rlt.rlt_get_device_error() == rlt.DEVERR_BAD_PAGE
    c = Case(dev, [30, 60], 8, 2, 128, 16, seed=14)
    c.seq[0] = -4
    c.seq[1] = 1 << 30                                          # clamped to the table's pages
    c.run(max_seq_len=60)
    assert rlt.rlt_get_device_error() & rlt.DEVERR_BAD_LEN


def test_streams_graph_and_workspaces(dev):
    import torch
    import paged_kv_looped_gb300 as rlt
    a, b = Case(dev, [600, 50, 0, 999], 8, 2, 128, 16, seed=15), Case(dev, [900, 77, 300], 8, 1, 128, 64, seed=16)
    ra, rb = a.reference(), b.reference()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for _ in range(5):                                          # two calls at once, workspaces of their own
        res.append((a.run(split_tokens=64, stream=s1), b.run(split_tokens=128, stream=s2)))
    torch.cuda.synchronize()
    for x, y in res:
        a.check(*x, ra)
        b.check(*y, rb)
        assert torch.equal(x[0], res[0][0][0])                  # the same bits every time
    # captured and replayed with other queries and lengths, early start included
    ws = torch.empty(rlt.rlt_paged_decode_kv8_workspace_size(4, 8, 2, 128, 999, 64), dtype=torch.uint8, device=dev)
    out, lse = torch.empty_like(a.q), torch.empty(4, 8, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for early in (False, True, True):
            rlt.rlt_paged_decode_attn_kv8(a.pool, 1, a.q, a.table, a.seq, 999, out=out, lse_out=lse, workspace=ws,
                                          split_tokens=64, early_start=early)
    a.q.neg_()
    a.lens[:] = [599, 1, 33, 0]
    a.tables[2, :3] = a.tables[3, :3]
    a.seq.copy_(torch.from_numpy(a.lens))
    a.table.copy_(torch.from_numpy(a.tables))
    graph.replay()
    a.check(out, lse)


def test_guards(dev):
    """Nothing around out, lse and the workspace is written."""
    import torch
    import paged_kv_looped_gb300 as rlt
    c = Case(dev, [600, 50, 0], 6, 2, 128, 16, seed=17)
    need = rlt.rlt_paged_decode_kv8_workspace_size(3, 6, 2, 128, 600, 64)
    buf = torch.full((need + 512,), 0xAB, dtype=torch.uint8, device=dev)
    o = torch.full((3 * 6 * 128 + 256,), 9.0, dtype=torch.bfloat16, device=dev)
    l = torch.full((3 * 6 + 64,), 9.0, device=dev)
    out, lse = o[128:-128].view(3, 6, 128), l[32:-32].view(3, 6)
    before = [t.view(torch.uint8).clone() for t in (c.pool.k, c.pool.v, c.pool.k_exp, c.pool.v_exp)]
    rlt.rlt_paged_decode_attn_kv8(c.pool, 1, c.q, c.table, c.seq, 600, out=out, lse_out=lse, workspace=buf[256:-256],
                                  split_tokens=64)
    c.check(out, lse)
    assert (o[:128] == 9).all() and (o[-128:] == 9).all() and (l[:32] == 9).all() and (l[-32:] == 9).all()
    assert (buf[:256] == 0xAB).all() and (buf[-256:] == 0xAB).all()
    for t, x in zip((c.pool.k, c.pool.v, c.pool.k_exp, c.pool.v_exp), before):
        assert torch.equal(t.view(torch.uint8), x)


def test_rows_past_32_bits(dev):
    """A bank far into a pool: byte offsets past 2^31 and 2^32."""
    import torch
    import paged_kv_looped_gb300 as rlt
    hkv, ps, d, pages = 8, 256, 128, 8500                       # 2.2 GB a side and bank
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("not enough free device memory")
    pool = rlt.KV8Pool.empty(2, pages, hkv, ps, d, dev)
    for t in (pool.k, pool.v):
        t.view(torch.uint8).fill_(0x7F)
    pool.k_exp.fill_(255), pool.v_exp.fill_(255)
    n = 300
    k, v = (torch.randn(n, hkv, d, device=dev).bfloat16() for _ in range(2))
    table = torch.tensor([[8499, 8200]], dtype=torch.int32, device=dev)
    at = torch.arange(n, device=dev)
    slots = table[0].long()[at // ps] * ps + at % ps
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    q = torch.randn(1, 16, d, device=dev).bfloat16()
    rlt.rlt_kv8_append_rope(pool, 1, k, v, at, slots, d, 10000.0, k_out=ko, v_out=vo)
    lse = torch.empty(1, 16, device=dev)
    out = rlt.rlt_paged_decode_attn_kv8(pool, 1, q, table, torch.tensor([n], dtype=torch.int32, device=dev), n, lse_out=lse)
    torch.cuda.synchronize()
    kk, vv = (x.double().cpu().numpy() for x in (ko, vo))
    qq = q.double().cpu().numpy()
    for h in range(16):
        o, l, m = R.softmax_rows(qq[0, h][None] @ kk[:, h // 2].T / np.sqrt(d), vv[:, h // 2])
        terms = (np.abs(qq[0, h]) @ np.abs(kk[:, h // 2]).T).max() / np.sqrt(d)
        assert np.all(np.abs(out[0, h].double().cpu().numpy() - o[0]) <=
                      R.attention_bound(o[0], m[0], np.array(terms), 2.0 ** -11))
        assert abs(float(lse[0, h]) - l[0]) <= R.lse_bound(l[0], terms, d)
