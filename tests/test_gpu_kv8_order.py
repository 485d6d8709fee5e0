"""The 8-bit cache's and the prompts' calls start while the kernel ahead of them ends and read nothing before it has:
runs of calls that write what the next one reads, eagerly and captured, give what they give one at a time."""
import pytest

pytestmark = pytest.mark.gpu

STEPS = 12


class Model:
    """Two requests; each step appends a token per request, attends, and feeds the output back into the next
    step's rows.  Lengths, positions, slots and plans change on the device between the calls."""

    def __init__(self, rlt, between):
        import torch
        self.rlt, self.between = rlt, between
        g = torch.Generator().manual_seed(3)
        self.hq, self.hkv, self.d, self.ps, self.n = 8, 2, 128, 16, 700
        pages = 2 * 64
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")        # noqa: E731
        self.pool = rlt.KV8Pool(*(u8(1, pages, self.hkv, self.ps, self.d).view(torch.float8_e4m3fn) for _ in range(2)),
                                *(u8(1, pages, self.hkv, self.ps) for _ in range(2)))
        self.table = torch.arange(pages, dtype=torch.int32).view(2, 64).cuda()
        self.prompt = torch.randn(2 * self.n, self.hq + 2 * self.hkv, self.d, generator=g).bfloat16().cuda()
        self.plans = [rlt.rlt_plan_prefill(x, self.hq // self.hkv) for x in ([self.n, self.n], [self.n + 44, self.n - 44])]
        assert self.plans[0].num_items == self.plans[1].num_items
        self.items = [torch.from_numpy(p.items).cuda() for p in self.plans]
        self.plan = self.plans[0].to("cuda")
        self.plan.max_key_tiles = max(p.max_key_tiles for p in self.plans)
        self.plan.total_key_tiles = max(p.total_key_tiles for p in self.plans)
        self.pos = torch.arange(self.n).repeat(2).cuda()
        at = torch.arange(self.n)
        self.slots = torch.cat([at, 64 * self.ps + at]).cuda()
        new = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")    # noqa: E731
        self.qo, self.ko, self.vo = (new(2 * self.n, h, self.d) for h in (self.hq, self.hkv, self.hkv))
        self.out = new(2 * self.n, self.hq, self.d)
        self.rows, self.q1 = new(2, self.hq + 2 * self.hkv, self.d), new(2, self.hq, self.d)
        self.one, self.lse = new(2, self.hq, self.d), torch.zeros(2, self.hq, device="cuda")
        self.lens = torch.full((2,), self.n, dtype=torch.int32, device="cuda")
        self.pos1 = torch.full((2,), self.n, device="cuda")
        self.slot1 = torch.tensor([self.n, 64 * self.ps + self.n], device="cuda")
        self.ws = u8(1 << 22)
        self.kept = torch.zeros(2 * STEPS + 2, 2, self.hq, self.d, dtype=torch.bfloat16, device="cuda")

    def reset(self):
        for x in (self.pool.k, self.pool.v):
            x.view(__import__("torch").uint8).zero_()
        for x in (self.pool.k_exp, self.pool.v_exp, self.kept):
            x.zero_()
        self.lens.fill_(self.n)
        self.pos1.fill_(self.n)
        self.slot1.copy_(self.lens.long() + self.table[:, 0].long() * self.ps)

    def run(self):
        rlt, hq, hkv, x = self.rlt, self.hq, self.hkv, self.prompt
        go = self.between
        rlt.rlt_kv8_append_rope(self.pool, 0, x[:, hq:hq + hkv], x[:, hq + hkv:], self.pos, self.slots, self.d, 1e4,
                                q=x[:, :hq], q_out=self.qo, k_out=self.ko, v_out=self.vo)
        go()
        for i in (1, 0):                         # the plan changes between two calls on the same rows
            self.plan.dev.copy_(self.items[i])
            go()
            rlt.rlt_prefill_attn(self.qo, self.ko, self.vo, self.plan, out=self.out)
            go()
            self.kept[2 * STEPS + i].copy_(self.out[self.n - 1::self.n])
        for step in range(STEPS):
            # the next token's rows from the last output; its place one further
            self.rows[:, :hq].copy_(self.out[-2:] if step == 0 else self.one)
            self.rows[:, hq:].copy_(self.rows[:, :2 * hkv] + self.prompt[2 * step:2 * step + 2, hq:])
            go()
            rlt.rlt_kv8_append_rope(self.pool, 0, self.rows[:, hq:hq + hkv], self.rows[:, hq + hkv:], self.pos1, self.slot1,
                                    self.d, 1e4, q=self.rows[:, :hq], q_out=self.q1)
            self.lens.add_(1)
            go()
            rlt.rlt_paged_decode_attn_kv8(self.pool, 0, self.q1, self.table, self.lens, self.n + STEPS, out=self.one,
                                          lse_out=self.lse, workspace=self.ws, split_tokens=64)
            go()
            self.kept[2 * step].copy_(self.one)
            # the same rows once more, straight behind: a decode of the decode's output
            rlt.rlt_paged_decode_attn_kv8(self.pool, 0, self.one, self.table, self.lens, self.n + STEPS, out=self.q1,
                                          workspace=self.ws, split_tokens=64)
            go()
            self.kept[2 * step + 1].copy_(self.q1)
            self.pos1.add_(1)
            self.slot1.add_(1)
        return self.kept


@pytest.fixture(scope="module")
def want(cuda_device):
    import torch
    import paged_kv_looped_gb300 as rlt
    rlt.load()
    rlt.rlt_get_device_error()
    m = Model(rlt, torch.cuda.synchronize)
    m.reset()
    k = m.run().clone()
    assert torch.isfinite(k.float()).all() and k.abs().amax() > 0.1 and rlt.rlt_get_device_error() == 0
    return k


def test_eager(want):
    import torch
    import paged_kv_looped_gb300 as rlt
    m = Model(rlt, lambda: None)
    for _ in range(3):
        m.reset()
        assert torch.equal(m.run(), want)


def test_captured(want):
    import torch
    import paged_kv_looped_gb300 as rlt
    m = Model(rlt, lambda: None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.reset()
        m.run()
    for _ in range(3):
        g.replay()
        assert torch.equal(m.kept, want)


def test_captured_across_streams(want):
    # every call behind a join: its kernel has two nodes ahead of it, one of them a copy
    import torch
    import paged_kv_looped_gb300 as rlt
    side = torch.cuda.Stream()
    a, b = torch.zeros(1 << 22, device="cuda"), torch.zeros(1 << 22, device="cuda")

    def fork():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            b.copy_(a)
        here.wait_stream(side)

    m = Model(rlt, fork)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.reset()
        m.run()
    for _ in range(2):
        g.replay()
        assert torch.equal(m.kept, want)
    m.reset()
    assert torch.equal(m.run(), want)
