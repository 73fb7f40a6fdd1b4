"""The operators as a serving loop runs them together: rotate and append,
block bounds, then attention (shared-prefix, and sparse over chosen blocks),
eagerly, on another stream, and replayed from CUDA graphs."""
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu
D, HQ, HKV = 128, 32, 8


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_464_b200 import capi
    capi.get_device_error(clear=True)
    yield capi
    code, detail = capi.get_device_error(clear=True)
    assert code == 0, (code, detail)


class Loop:
    """A batch of 12 sequences over one 320-token prefix that grows by a token a step."""

    def __init__(self, pa, seed):
        self.pa, self.n, self.prefix = pa, 12, 320
        lens = [320 + (11 * b) % 37 for b in range(self.n)]
        room = [x + 8 for x in lens]
        k, v, tables, _ = ref.make_cache(room, HKV, "bf16", seed=seed, shared=[(0, self.n, 320)])
        for b in range(self.n):       # no token yet behind a sequence's length
            for t in range(lens[b], room[b]):
                k[tables[b, t // 16], t % 16] = v[tables[b, t // 16], t % 16] = float("nan")
        self.tables_host, self.lens_host = tables, torch.tensor(lens, dtype=torch.int32)
        self.k, self.v, self.tables, self.lens = k.cuda(), v.cuda(), tables.cuda(), self.lens_host.cuda()
        self.table = pa.rope_table(512, D, 500000.0)
        self.gs = torch.tensor([0, self.n], dtype=torch.int32, device="cuda")
        self.pl = torch.tensor([self.prefix], dtype=torch.int32, device="cuda")
        self.bounds = torch.zeros((k.shape[0], 2, HKV, D), dtype=k.dtype, device="cuda")
        pa.update_block_bounds(self.k, self.bounds, self.tables, self.lens, self.lens, max_new_len=512)
        self.ones = torch.ones(self.n, dtype=torch.int32, device="cuda")
        T = self.n + 4                # rows of a padded batch
        self.qkv = torch.zeros((T, HQ + 2 * HKV, D), dtype=torch.bfloat16, device="cuda")
        self.pos = torch.full((T,), -1, dtype=torch.int64, device="cuda")
        self.slot = torch.full((T,), -1, dtype=torch.int64, device="cuda")
        self.q = torch.zeros((T, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.chosen = torch.zeros((self.n, HKV, 6), dtype=torch.int32, device="cuda")
        self.dense = torch.zeros((self.n, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.sparse = torch.zeros_like(self.dense)
        size = max(pa.decode_shared_prefix_workspace_bytes(self.n, 1, HQ, HKV, D, self.prefix, 64, self.n),
                   pa.select_blocks_workspace_bytes(self.n, HKV, 512),
                   pa.decode_selected_workspace_bytes(self.n, HQ, HKV, D, 6))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def feed(self, seed):
        """The next token of every sequence (host side of a step)."""
        g = torch.Generator().manual_seed(seed)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g).bfloat16())
        at = self.lens_host.long()
        self.pos[:self.n] = at.cuda()
        block = self.tables_host[torch.arange(self.n), at // 16].long()
        self.slot[:self.n] = (block * 16 + at % 16).cuda()
        self.lens_host = self.lens_host + 1
        self.lens.copy_(self.lens_host)

    def step(self, stream=None):
        pa = self.pa
        q, key, val = self.qkv[:, :HQ], self.qkv[:, HQ:HQ + HKV], self.qkv[:, HQ + HKV:]
        pa.rope_and_cache(q, key, val, self.pos, self.table, self.k, self.v, self.slot, self.q, stream=stream)
        pa.update_block_bounds(self.k, self.bounds, self.tables, self.lens, self.ones, max_new_len=1, stream=stream)
        q = self.q[:self.n]
        pa.decode_shared_prefix(q, self.k, self.v, self.tables, self.lens, self.gs, self.pl, 0.088, self.dense,
                                max_prefix_len=self.prefix, max_suffix_len=64, max_group_size=self.n,
                                workspace=self.ws, stream=stream)
        pa.select_blocks(q, self.bounds, self.tables, self.lens, self.chosen, max_context_len=512, workspace=self.ws,
                         stream=stream)
        pa.decode_selected(q, self.k, self.v, self.tables, self.lens, self.chosen, 0.088, self.sparse,
                           workspace=self.ws, stream=stream)

    def check(self):
        torch.cuda.synchronize()
        q = self.q.cpu()
        k, v, lens = self.k.cpu(), self.v.cpu(), self.lens_host
        want_q, _ = ref.rotate(self.qkv[:self.n, :HQ].cpu().double(), self.pos[:self.n].cpu(), self.table.cpu(), False)
        assert ((q[:self.n].double() - want_q).abs() <= 2.0 ** -8 * want_q.abs() + 1e-5).all()
        assert (q[self.n:] == 0).all()                        # rows behind the last sequence
        want_b = ref.block_bounds(k, self.bounds.cpu(), self.tables_host, lens, lens)
        assert torch.equal(self.bounds.cpu(), want_b)
        want_c = ref.choose(q[:self.n], want_b, self.tables_host, lens, 6, 1, 1)
        assert torch.equal(self.chosen.cpu(), want_c)
        for out, chosen in ((self.dense, None), (self.sparse, want_c)):
            want, weight = ref.attention(q[:self.n], k, v, self.tables_host, lens, 0.088, chosen)
            tol = ref.attention_tolerance(want, weight, "bf16", 16)
            assert ((out.cpu().double() - want).abs() <= tol).all()


def test_eager_steps(pa):
    loop = Loop(pa, 1)
    for i in range(3):
        loop.feed(i)
        loop.step()
        loop.check()


def test_on_another_stream(pa):
    loop = Loop(pa, 2)
    s = torch.cuda.Stream()
    loop.feed(7)
    s.wait_stream(torch.cuda.current_stream())
    loop.step(stream=s)
    torch.cuda.current_stream().wait_stream(s)
    loop.check()
    # workspace and outputs allocated by the call live on that stream too
    q = loop.q[:loop.n]
    s.wait_stream(torch.cuda.current_stream())
    out = pa.decode_shared_prefix(q, loop.k, loop.v, loop.tables, loop.lens, loop.gs, loop.pl, 0.088, stream=s)
    chosen = pa.select_blocks(q, loop.bounds, loop.tables, loop.lens, 6, stream=s)
    sparse = pa.decode_selected(q, loop.k, loop.v, loop.tables, loop.lens, chosen, 0.088, stream=s)
    s.synchronize()
    assert torch.equal(out, loop.dense) or ((out - loop.dense).abs() <= 0.02).all()   # another split of the suffix
    assert torch.equal(chosen, loop.chosen) and torch.equal(sparse, loop.sparse)


def test_replayed_from_a_graph(pa):
    """One capture, three replays with new tokens: every buffer is the caller's, so nothing is bound to the capture."""
    loop, eager = Loop(pa, 3), Loop(pa, 3)
    loop.feed(0), eager.feed(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        loop.step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    eager.step()
    for i in range(1, 4):
        loop.feed(i), eager.feed(i)
        loop.dense.fill_(float("nan")), loop.sparse.fill_(float("nan"))
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        for name in ("q", "k", "v", "bounds", "chosen", "dense", "sparse"):
            a, b = getattr(loop, name), getattr(eager, name)
            a, b = (a.view(torch.int16), b.view(torch.int16)) if a.dtype == torch.bfloat16 else (a, b)
            assert torch.equal(a, b), (i, name)
    loop.check()


def test_two_graphs_that_share_a_workspace(pa):
    """Replayed one after the other on one stream."""
    loops = [Loop(pa, 4), Loop(pa, 5)]
    loops[1].ws = loops[0].ws
    graphs = []
    for loop in loops:
        loop.feed(1)
        loop.step()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            loop.step()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    for loop in loops:
        loop.check()


def test_sizes_of_nothing(pa):
    """No sequences, no tokens: no-ops."""
    e = dict(device="cuda")
    k = torch.zeros((2, 16, 1, D), dtype=torch.bfloat16, **e)
    q = torch.zeros((0, 4, D), dtype=torch.bfloat16, **e)
    kv = torch.zeros((0, 1, D), dtype=torch.bfloat16, **e)
    i32, i64 = torch.zeros(0, dtype=torch.int32, **e), torch.zeros(0, dtype=torch.int64, **e)
    t = torch.zeros((0, 3), dtype=torch.int32, **e)
    b = torch.zeros((2, 2, 1, D), dtype=torch.bfloat16, **e)
    assert pa.rope_and_cache(q, kv, kv, i64, pa.rope_table(4, D), k, k.clone(), i64).shape == q.shape
    gs = torch.zeros(1, dtype=torch.int32, **e)
    assert pa.decode_shared_prefix(q, k, k, t, i32, gs, i32, 0.1).shape == q.shape
    pa.update_block_bounds(k, b, t, i32, i32)
    chosen = pa.select_blocks(q, b, t, i32, 3)
    assert chosen.shape == (0, 1, 3)
    assert pa.decode_selected(q, k, k, t, i32, chosen, 0.1).shape == q.shape


class LongPrefix:
    """480 rows over 65536 tokens of one KV head, and one sequence with 1100 tokens of its own: the walk over the
    sequences' own tokens is split (a third launch joins), runs on the SMs that the prefix kernel leaves, and is
    through long before it."""

    def __init__(self, seed):
        n, prefix = 60, 65536
        lens = [prefix + (1100 if b == 17 else b % 7) for b in range(n)]
        self.k, self.v, self.tables, self.lens = ref.make_cache(lens, 1, "bf16", seed=seed, shared=[(0, n, prefix)])
        self.q = [ref.make_q(n, 8, "bf16", seed=seed + i) for i in range(2)]
        self.device = [t.cuda() for t in (self.k, self.v, self.tables, self.lens)]
        self.groups = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [prefix])]
        self.q_device = [x.cuda() for x in self.q]

    def call(self, pa, i, out, workspace):
        return pa.decode_shared_prefix(self.q_device[i], *self.device, *self.groups, 0.088, out, max_prefix_len=65536,
                                       max_suffix_len=1100, max_group_size=60, workspace=workspace)


@pytest.fixture(scope="module")
def long_prefix():
    return LongPrefix(1)


def test_prefix_that_outlasts_the_suffix_walk(pa, long_prefix):
    """Calls one after the other with one workspace, eager and replayed: each gives what it gives alone."""
    x = long_prefix
    need = pa.decode_shared_prefix_workspace_bytes(60, 1, 8, 1, 128, 65536, 1100, 60)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    alone = []
    for i in range(2):
        ws.fill_(0xFF)      # NaN in every partial
        alone.append(torch.empty_like(x.q_device[i]))
        torch.cuda.synchronize()
        x.call(pa, i, alone[i], ws)
        torch.cuda.synchronize()
        want, weight = ref.attention(x.q[i], x.k, x.v, x.tables, x.lens, 0.088)
        assert ((alone[i].cpu().double() - want).abs() <= ref.attention_tolerance(want, weight, "bf16", 15)).all()
    outs = [torch.full_like(alone[0], float("nan")) for _ in range(40)]
    ws.fill_(0xFF)
    for i, out in enumerate(outs):
        x.call(pa, i % 2, out, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(out, alone[i % 2]) for i, out in enumerate(outs))
    ws.fill_(0xFF)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(6):
            x.call(pa, i % 2, outs[i], ws)
    for _ in range(10):
        for out in outs[:6]:
            out.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i], alone[i % 2]) for i in range(6))


def test_what_follows_a_shared_prefix_call_waits_for_it(pa, long_prefix):
    """The next call overwrites what the prefix kernel still reads, the workspace at once: nothing of it is seen early."""
    x = long_prefix
    need = pa.decode_shared_prefix_workspace_bytes(60, 1, 8, 1, 128, 65536, 1100, 60)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = x.call(pa, 0, None, ws).clone()
    k, v = x.device[0].clone(), x.device[1].clone()
    T, D = 512, 128
    rows = torch.full((T, 3, D), 9.0, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    table = pa.rope_table(8, D)
    slots = [(x.tables[0, 4096 - 32:4096].long()[:, None] * 16 + torch.arange(16)).flatten().cuda()]   # the prefix's end
    q_out = torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda")
    for _ in range(10):
        out = torch.empty_like(want)
        x.device[0].copy_(k), x.device[1].copy_(v)
        x.call(pa, 0, out, ws)
        pa.rope_and_cache(rows[:, :1], rows[:, 1:2], rows[:, 2:], pos, table, x.device[0], x.device[1], slots[0], q_out)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    x.device[0].copy_(k), x.device[1].copy_(v)
