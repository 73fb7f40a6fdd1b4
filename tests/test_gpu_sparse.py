"""Block bounds (bit-exact), block choice (equal, ties to the lowest block) and
decode over chosen blocks (within rounding) against plain 64-bit forms."""
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_464_b200 import capi
    capi.get_device_error(clear=True)
    yield capi
    code, detail = capi.get_device_error(clear=True)
    assert code == 0, (code, detail)


def cuda(*ts):
    return [t.cuda() for t in ts]


LENS = [1, 0, 15, 16, 17, 33, 250, 31, 64, 129]


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("new", ["one", "all", "some"])
def test_bounds(pa, ty, hkv, new):
    k, _, tables, lens = ref.make_cache(LENS, hkv, ty, seed=hkv)
    n = {"one": lens.clamp(max=1), "all": lens, "some": torch.tensor([0, 0, 15, 2, 2, 20, 100, 16, 33, 1], dtype=torch.int32)}[new]
    bounds = torch.full((k.shape[0], 2, hkv, k.shape[3]), 9.0, dtype=k.dtype)
    want = ref.block_bounds(k, bounds, tables, lens, n)
    kd, bd, td, ld, nd = cuda(k, bounds, tables, lens, n)
    pa.update_block_bounds(kd, bd, td, ld, nd, max_new_len=int(n.max()))
    assert torch.equal(bd.cpu(), want)
    bd2 = bounds.cuda()
    pa.update_block_bounds(kd, bd2, td, ld, nd)         # the maximum read from the device
    assert torch.equal(bd2, bd)


@pytest.mark.parametrize("most", [1000, 1 << 30, (1 << 31) - 1])
def test_bounds_with_a_generous_maximum(pa, most):
    """Only an upper bound: the rows' last blocks are found all the same."""
    k, _, tables, lens = ref.make_cache(LENS, 2, "bf16", seed=6)
    n = lens.clamp(max=1)
    bounds = torch.full((k.shape[0], 2, 2, 128), 9.0, dtype=k.dtype)
    kd, bd, td, ld, nd = cuda(k, bounds, tables, lens, n)
    pa.update_block_bounds(kd, bd, td, ld, nd, max_new_len=most)
    assert torch.equal(bd.cpu(), ref.block_bounds(k, bounds, tables, lens, n))
    none = torch.empty((len(LENS), 0), dtype=torch.int32, device="cuda")     # no table, no token
    pa.update_block_bounds(kd, bd, none, torch.zeros_like(ld), torch.zeros_like(nd), max_new_len=most)


def test_bounds_keep_nan_and_infinity(pa):
    k, _, tables, lens = ref.make_cache([40], 2, "bf16", seed=1)
    k[tables[0, 0], 3, 0, 5] = float("nan")
    k[tables[0, 1], 2, 1, 7] = float("-inf")
    kd, td, ld = cuda(k, tables, lens)
    bd = torch.zeros((k.shape[0], 2, 2, 128), dtype=k.dtype, device="cuda")
    pa.update_block_bounds(kd, bd, td, ld, ld, max_new_len=40)
    b = bd.cpu()
    assert b[tables[0, 0], :, 0, 5].isnan().all() and int(b.isnan().sum()) == 2
    assert b[tables[0, 1], 0, 1, 7] == float("-inf") and b[tables[0, 1], 1, 1, 7].isfinite()


@pytest.mark.expects_device_error
def test_bounds_report_bad_input(pa):
    k, _, tables, lens = ref.make_cache([40, 40, 40], 1, "bf16", seed=2)
    good = ref.block_bounds(k, torch.zeros((k.shape[0], 2, 1, 128), dtype=k.dtype), tables, lens, lens)
    kd, ld = cuda(k, lens)

    def call(tables, new, lens=ld, most=40):
        bd = torch.zeros((k.shape[0], 2, 1, 128), dtype=k.dtype, device="cuda")
        pa.update_block_bounds(kd, bd, tables.cuda(), lens, torch.tensor(new, dtype=torch.int32, device="cuda"), max_new_len=most)
        return bd.cpu(), pa.get_device_error(clear=True)

    for new, seq in (([40, 41, 40], 1), ([40, 40, -1], 2)):
        b, err = call(tables, new)
        assert err == (4, seq)
        for s in range(3):
            same = torch.equal(b[tables[s, :3].long()], good[tables[s, :3].long()])
            assert same == (s != seq)
    assert call(tables, [40, 40, 40], most=39)[1][0] == 4
    t = tables.clone()
    t[1, 1] = k.shape[0]
    assert call(t, [40, 40, 40])[1] == (1, k.shape[0])
    long = ld.clone()
    long[0] = tables.shape[1] * 16 + 1
    assert call(tables, [1, 1, 1], lens=long)[1] == (4, 0)


def bounds_of(k, tables, lens):
    return ref.block_bounds(k, torch.zeros((k.shape[0], 2, *k.shape[2:]), dtype=k.dtype), tables, lens, lens)


SELECT_LENS = [0, 1, 16, 17, 63, 64, 65, 333, 1024, 4097]


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hkv,G", [(1, 1), (3, 2), (2, 4), (2, 8)])
@pytest.mark.parametrize("K,sink,recent", [(1, 0, 1), (4, 1, 1), (5, 2, 3), (37, 0, 0), (300, 1, 4)])
def test_choice(pa, ty, hkv, G, K, sink, recent):
    k, _, tables, lens = ref.make_cache(SELECT_LENS, hkv, ty, seed=hkv * 10 + G)
    q = ref.make_q(len(lens), hkv * G, ty, seed=K)
    bounds = bounds_of(k, tables, lens)
    want = ref.choose(q, bounds, tables, lens, K, sink, recent)
    got = pa.select_blocks(*cuda(q, bounds, tables, lens), K, sink_blocks=sink, recent_blocks=recent)
    assert torch.equal(got.cpu(), want)


def test_choice_ties_go_to_the_lowest_block(pa):
    """Blocks with the same bounds, all of them or in turn, and whole-number scores."""
    hkv, G, n = 2, 4, 400
    lens = torch.tensor([n * 16], dtype=torch.int32)
    tables = torch.arange(n, dtype=torch.int32)[None]
    g = torch.Generator().manual_seed(1)
    q = torch.randint(-2, 3, (1, hkv * G, 128), generator=g).bfloat16()
    for kinds in (1, 2, 7):
        base = torch.randint(-2, 3, (kinds, 2, hkv, 128), generator=g)
        base = torch.stack([base.amin(1), base.amax(1)], 1)
        bounds = base[torch.arange(n) % kinds].bfloat16()
        for K, sink, recent in ((3, 0, 0), (9, 1, 1), (150, 2, 5), (399, 0, 1), (6, 3, 3)):
            want = ref.choose(q, bounds, tables, lens, K, sink, recent)
            got = pa.select_blocks(*cuda(q, bounds, tables, lens), K, sink_blocks=sink, recent_blocks=recent)
            assert torch.equal(got.cpu(), want), (kinds, K)


def test_choice_near_ties_are_ordered_in_64_bits(pa):
    """Scores of about 2^12 that differ by 2^-14: 26 bits apart, which no fp32 sum can order."""
    n = 64
    lens = torch.tensor([n * 16], dtype=torch.int32)
    tables = torch.arange(n, dtype=torch.int32)[None]
    q = torch.ones((1, 1, 128), dtype=torch.float32)[..., :64].contiguous()
    q[0, 0, 0] = 2.0 ** -20
    hi = torch.full((n, 64), 64.0)
    step = torch.randperm(n, generator=torch.Generator().manual_seed(4))
    hi[:, 0] = step.float() * 64          # adds step * 2^-14
    bounds = torch.stack([-hi, hi], 1)[:, :, None].contiguous()
    got = pa.select_blocks(*cuda(q, bounds, tables, lens), 8, sink_blocks=0, recent_blocks=0)
    want = torch.argsort(step, descending=True)[:8].sort().values.int()
    assert torch.equal(got.cpu()[0, 0], want)


def test_choice_takes_nan_blocks_first(pa):
    k, _, tables, lens = ref.make_cache([1000], 1, "bf16", seed=4)
    bounds = bounds_of(k, tables, lens)
    for j in (11, 40):
        bounds[tables[0, j], 0, 0, 9] = bounds[tables[0, j], 1, 0, 9] = float("nan")
    bounds[tables[0, 20], 1, 0, 3] = float("inf")
    q = ref.make_q(1, 8, "bf16", seed=1)
    want = ref.choose(q, bounds, tables, lens, 5, 0, 0)
    got = pa.select_blocks(*cuda(q, bounds, tables, lens), 5, sink_blocks=0, recent_blocks=0).cpu()
    assert torch.equal(got, want) and {11, 20, 40} <= set(got[0, 0].tolist())


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("n,kinds,K", [(3000, 2, 700), (5000, 1, 1500), (70000, 3, 40), (70000, 70000, 40)])
def test_choice_of_many_blocks_and_ties(pa, ty, n, kinds, K):
    """More ties than the fast path takes, more blocks than its cache (4096) and its bits (65536) hold."""
    d = ref.HEAD_DIM[ty]
    lens = torch.tensor([n * 16], dtype=torch.int32)
    g = torch.Generator().manual_seed(n + kinds)
    base = torch.randn((min(kinds, 1000), 2, 1, d), generator=g).to(ref.TYPES[ty])
    base = torch.stack([base.amin(1), base.amax(1)], 1)
    tables = (torch.arange(n) % base.shape[0])[None].int()       # blocks of equal content are one block
    q = ref.make_q(1, 2, ty, seed=n)
    x = q[0].double()[:, None]
    rows = base[:, :, 0].double()
    score = (x * torch.where(x >= 0, rows[:, 1], rows[:, 0])).sum(-1).amax(0)[torch.arange(n) % base.shape[0]]
    score[0] = score[-2:] = float("inf")
    want = torch.argsort(score, descending=True, stable=True)[:K].sort().values.int()
    got = pa.select_blocks(*cuda(q, base, tables, lens), K, sink_blocks=1, recent_blocks=2)
    assert torch.equal(got.cpu()[0, 0], want)


def test_choice_with_scores_that_overflow_fp32(pa):
    """Products beyond fp32: their blocks are ranked in 64 bits like the others."""
    n = 300
    lens = torch.tensor([n * 16], dtype=torch.int32)
    tables = torch.arange(n, dtype=torch.int32)[None]
    g = torch.Generator().manual_seed(2)
    bounds = torch.randn((n, 2, 1, 128), generator=g).bfloat16()
    bounds = torch.stack([bounds.amin(1), bounds.amax(1)], 1)
    bounds[::7] *= 2.0 ** 120
    q = (torch.randn((1, 4, 128), generator=g) * 2.0 ** 20).bfloat16()
    for K in (5, 43, 44, 60):
        want = ref.choose(q, bounds, tables, lens, K, 0, 1)
        got = pa.select_blocks(*cuda(q, bounds, tables, lens), K, sink_blocks=0, recent_blocks=1)
        assert torch.equal(got.cpu(), want), K


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_choice_with_scores_below_fp32(pa, ty):
    """Products under the smallest fp32 number (f16: its subnormals): the order is still that of the 64-bit scores."""
    n, d = 200, ref.HEAD_DIM[ty]
    lens = torch.tensor([n * 16], dtype=torch.int32)
    tables = torch.arange(n, dtype=torch.int32)[None]
    g = torch.Generator().manual_seed(12)
    small = 2.0 ** -20 if ty == "f16" else 2.0 ** -80
    bounds = (torch.randn((n, 2, 1, d), generator=g) * small).to(ref.TYPES[ty])
    bounds = torch.stack([bounds.amin(1), bounds.amax(1)], 1)
    q = (torch.randn((1, 4, d), generator=g) * small).to(ref.TYPES[ty])
    for K in (1, 8, 77):
        want = ref.choose(q, bounds, tables, lens, K, 0, 1)
        got = pa.select_blocks(*cuda(q, bounds, tables, lens), K, sink_blocks=0, recent_blocks=1)
        assert torch.equal(got.cpu(), want), K


@pytest.mark.expects_device_error
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_choice_puts_bad_blocks_last(pa, ty):
    k, _, tables, lens = ref.make_cache([640], 1, ty, seed=4)
    bounds = bounds_of(k, tables, lens)
    bounds[0] = bounds.abs().nan_to_num(1.0).amax() * torch.tensor([-1.0, 1.0])[:, None, None].to(bounds.dtype)   # block 0 above all
    q = ref.make_q(1, 4, ty, seed=1)
    t = tables.clone()
    t[0, 7], t[0, 21] = -7, k.shape[0]
    got = pa.select_blocks(*cuda(q, bounds, t, lens), 38, sink_blocks=0, recent_blocks=0).cpu()
    assert pa.get_device_error(clear=True)[0] == 1
    assert got[0, 0].tolist() == [j for j in range(40) if j not in (7, 21)]


@pytest.mark.expects_device_error
def test_choice_reports_bad_input(pa):
    k, _, tables, lens = ref.make_cache([200, 300], 1, "bf16", seed=4)
    bounds = bounds_of(k, tables, lens)
    q = ref.make_q(2, 4, "bf16", seed=1)
    want = ref.choose(q, bounds, tables, lens, 5, 1, 1)
    qd, bd, td = cuda(q, bounds, tables)
    for bad in (-1, 301):
        l2 = lens.clone()
        l2[0] = bad
        got = pa.select_blocks(qd, bd, td, l2.cuda(), 5, max_context_len=300).cpu()
        assert pa.get_device_error(clear=True) == (4, 0)
        assert (got[0] == -1).all() and torch.equal(got[1], want[1])
    t = tables.clone()
    t[1, 2] = -7
    pa.select_blocks(qd, bd, t.cuda(), lens.cuda(), 5, max_context_len=300)
    assert pa.get_device_error(clear=True) == (1, -7)


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hkv,G", [(1, 1), (3, 2), (2, 4), (2, 8)])
@pytest.mark.parametrize("K", [1, 4, 9, 70])
def test_decode_over_chosen_blocks(pa, ty, hkv, G, K):
    lens = [0, 1, 16, 17, 63, 333, 1024, 40]
    k, v, tables, lens = ref.make_cache(lens, hkv, ty, seed=K)
    q = ref.make_q(len(lens), hkv * G, ty, seed=K)
    g = torch.Generator().manual_seed(K)
    chosen = torch.full((len(lens), hkv, K), -1, dtype=torch.int32)
    for b in range(len(lens)):
        n = -(-int(lens[b]) // 16)
        for h in range(hkv):
            m = min(K, n)
            if b == 7 and h == 0:
                m = 0                      # a list that names no block
            pick = torch.randperm(n, generator=g)[:m].int()     # any order, holes between
            at = torch.randperm(K, generator=g)[:m]
            chosen[b, h, at] = pick
    scale = q.shape[2] ** -0.5
    want, weight = ref.attention(q, k, v, tables, lens, scale, chosen)
    out = torch.full_like(q, 4.0).cuda()
    qd, kd, vd, td, ld, cd = cuda(q, k, v, tables, lens, chosen)
    pa.decode_selected(qd, kd, vd, td, ld, cd, scale, out)
    err = (out.cpu().double() - want).abs()
    # 16-bit grouped heads: P in two parts of bf16 (2^-16 and less); fp32: none
    tol = ref.attention_tolerance(want, weight, ty, 16)
    assert (err <= tol).all(), (err - tol).max()
    assert (out.cpu()[0] == 0).all() and (out.cpu()[7, :G] == 0).all()
    again = pa.decode_selected(qd, kd, vd, td, ld, cd, scale)
    assert torch.equal(again, out)


def test_every_block_chosen_is_decode(pa):
    k, v, tables, lens = ref.make_cache([700, 33, 1500], 8, "bf16", seed=3)
    q = ref.make_q(3, 32, "bf16", seed=3)
    qd, kd, vd, td, ld = cuda(q, k, v, tables, lens)
    bd = torch.zeros((k.shape[0], 2, 8, 128), dtype=k.dtype, device="cuda")
    pa.update_block_bounds(kd, bd, td, ld, ld, max_new_len=1500)
    chosen = pa.select_blocks(qd, bd, td, ld, 100, max_context_len=1500)
    out = pa.decode_selected(qd, kd, vd, td, ld, chosen, 0.088)
    dense = pa.decode(qd, kd, vd, td, ld, 0.088, max_context_len=1500)
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    tol = ref.attention_tolerance(want, weight, "bf16", 16)
    assert ((out.cpu().double() - want).abs() <= tol).all() and ((dense.cpu().double() - want).abs() <= tol).all()


def test_live_nan_reaches_the_output(pa):
    k, v, tables, lens = ref.make_cache([200], 1, "bf16", seed=3)
    v[tables[0, 5], 2, 0, 17] = float("nan")
    k2 = k.clone()
    k2[tables[0, 5]] = float("nan")
    q = ref.make_q(1, 4, "bf16", seed=3)
    chosen = torch.tensor([[[2, 5, -1]]], dtype=torch.int32)
    out = pa.decode_selected(*cuda(q, k, v, tables, lens, chosen), 0.088).cpu()
    assert out[0, :, 17].isnan().all() and int(out.isnan().sum()) == 4
    assert pa.decode_selected(*cuda(q, k2, v, tables, lens, chosen), 0.088).isnan().all()
    only = torch.tensor([[[5, -1, -1]]], dtype=torch.int32)
    assert pa.decode_selected(*cuda(q, k2, v, tables, lens, only), 0.088).isnan().all()
    apart = torch.tensor([[[2, 7, -1]]], dtype=torch.int32)     # the NaN block is not named
    assert pa.decode_selected(*cuda(q, k2, v, tables, lens, apart), 0.088).isfinite().all()


@pytest.mark.expects_device_error
def test_decode_selected_reports_bad_entries(pa):
    k, v, tables, lens = ref.make_cache([100, 64], 1, "bf16", seed=3)
    q = ref.make_q(2, 4, "bf16", seed=3)
    good = torch.tensor([[[0, 3, 6]], [[1, 2, -1]]], dtype=torch.int32)
    want, weight = ref.attention(q, k, v, tables, lens, 0.088, good)
    tol = ref.attention_tolerance(want, weight, "bf16", 16)
    qd, kd, vd, td, ld = cuda(q, k, v, tables, lens)
    bad = good.clone()
    bad[1, 0, 2] = 4                   # the sequence has four blocks: 0 .. 3
    out = pa.decode_selected(qd, kd, vd, td, ld, bad.cuda(), 0.088).cpu()
    assert pa.get_device_error(clear=True) == (1, 4)
    assert ((out.double() - want).abs() <= tol).all()       # the entry counts for nothing
    t = tables.clone()
    t[0, 3] = 10 ** 6
    pa.decode_selected(qd, kd, vd, t.cuda(), ld, good.cuda(), 0.088)
    assert pa.get_device_error(clear=True) == (1, 10 ** 6)
    l2 = ld.clone()
    l2[0] = -3
    out = torch.full_like(qd, 2.0)
    pa.decode_selected(qd, kd, vd, td, l2, good.cuda(), 0.088, out)
    assert pa.get_device_error(clear=True) == (4, 0)
    assert (out[0] == 2.0).all() and ((out[1].cpu().double() - want[1]).abs() <= tol[1]).all()


def test_blocks_past_four_gigabytes(pa):
    blocks, hkv = (1 << 17) + 40, 8
    k = torch.zeros((blocks, 16, hkv, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    bounds = torch.zeros((blocks, 2, hkv, 128), dtype=torch.bfloat16, device="cuda")
    ks, vs, tables, lens = ref.make_cache([500], hkv, "bf16", seed=8)
    far = tables.clone()
    n = ks.shape[0]
    far[far >= 0] += blocks - n
    k[blocks - n:], v[blocks - n:] = ks.cuda(), vs.cuda()
    q = ref.make_q(1, 32, "bf16", seed=8)
    fd, ld, qd = cuda(far, lens, q)
    pa.update_block_bounds(k, bounds, fd, ld, ld, max_new_len=500)
    want_b = bounds_of(ks, tables, lens)
    assert torch.equal(bounds[blocks - n:].cpu(), want_b)
    assert int((bounds[:blocks - n] != 0).sum()) == 0
    chosen = pa.select_blocks(qd, bounds, fd, ld, 7, max_context_len=500)
    assert torch.equal(chosen.cpu(), ref.choose(q, want_b, tables, lens, 7, 1, 1))
    out = pa.decode_selected(qd, k, v, fd, ld, chosen, 0.088)
    want, weight = ref.attention(q, ks, vs, tables, lens, 0.088, chosen.cpu())
    assert ((out.cpu().double() - want).abs() <= ref.attention_tolerance(want, weight, "bf16", 16)).all()


@pytest.mark.parametrize("ty,hkv,G,S,K", [("bf16", 8, 2, 64, 9), ("f16", 8, 4, 64, 21), ("bf16", 8, 8, 61, 33),
                                          ("f16", 3, 8, 100, 70), ("bf16", 3, 4, 100, 70), ("f32", 8, 2, 64, 9)])
def test_decode_of_large_batches(pa, ty, hkv, G, S, K):
    """More CTAs than a wave of four-warp ones: two-warp CTAs for 16-bit grouped heads; lists with holes, of every
    length from none, whole and in partitions that are joined (100 sequences of 3 heads)."""
    g = torch.Generator().manual_seed(S + K)
    lens = [0, 1, 16, 17] + [int(x) for x in torch.randint(1, 1200, (S - 4,), generator=g)]
    k, v, tables, lens = ref.make_cache(lens, hkv, ty, seed=K)
    q = ref.make_q(S, hkv * G, ty, seed=K)
    chosen = torch.full((S, hkv, K), -1, dtype=torch.int32)
    for b in range(S):
        n = -(-int(lens[b]) // 16)
        for h in range(hkv):
            m = min(n, int(torch.randint(0, K + 1, (1,), generator=g)))
            at = torch.randperm(K, generator=g)[:m]
            chosen[b, h, at] = torch.randperm(n, generator=g)[:m].int()
    scale = q.shape[2] ** -0.5
    want, weight = ref.attention(q, k, v, tables, lens, scale, chosen)
    out = torch.full_like(q, 4.0).cuda()
    args = cuda(q, k, v, tables, lens, chosen)
    pa.decode_selected(*args, scale, out)
    err = (out.cpu().double() - want).abs()
    tol = ref.attention_tolerance(want, weight, ty, 16)
    assert (err <= tol).all(), (err - tol).max()
    empty = ((chosen >= 0).sum(2) == 0).repeat_interleave(G, 1)
    assert (out.cpu()[empty] == 0).all()
    assert torch.equal(pa.decode_selected(*args, scale), out)


@pytest.mark.parametrize("ty,G", [("bf16", 8), ("f16", 1), ("f32", 2)])
@pytest.mark.parametrize("K,sink,recent", [(64, 1, 4), (520, 0, 0)])
def test_choice_of_many_long_lists(pa, ty, G, K, sink, recent):
    """More than two lists an SM: 256 threads a list, with blocks in registers (512), in shared memory (4096) and read
    again behind those.  Blocks are drawn from 3000, so that ties are frequent."""
    S, hkv, d, pool = 40, 8, ref.HEAD_DIM[ty], 3000
    g = torch.Generator(device="cuda").manual_seed(K + G)
    blocks = [0, 1, K, K + 1, 511, 512, 513, 600, 1025, 4095, 4096, 4097, 4099, 4607, 4608, 4609, 5000, 9000] + \
        [400 + 37 * i for i in range(S - 18)]
    lens = torch.tensor([max(0, 16 * n - n % 16) for n in blocks], dtype=torch.int32, device="cuda")
    n = (lens + 15) // 16
    tables = torch.randint(0, pool, (S, 9001), generator=g, device="cuda").int()
    x = torch.randn((pool, 2, hkv, d), generator=g, device="cuda").to(ref.TYPES[ty])
    bounds = torch.stack([x.amin(1), x.amax(1)], 1)
    q = torch.randn((S, hkv * G, d), generator=g, device="cuda").to(ref.TYPES[ty])
    got = pa.select_blocks(q, bounds, tables, lens, K, sink_blocks=sink, recent_blocks=recent)
    rows = q.double().view(S, hkv, G, d)
    score = (torch.einsum("bhgd,phd->bhgp", rows.clamp(min=0), bounds[:, 1].double())
             + torch.einsum("bhgd,phd->bhgp", rows.clamp(max=0), bounds[:, 0].double())).amax(2)
    for b in range(S):
        m = int(n[b])
        want = torch.full((hkv, K), -1, dtype=torch.int32, device="cuda")
        if m:
            s = score[b][:, tables[b, :m].long()].clone()     # the same block has the same score: ties are exact
            s[:, :sink] = float("inf")
            s[:, m - recent:] = float("inf") if recent else s[:, m:]
            best = torch.sort(s, dim=1, descending=True, stable=True).indices[:, :K].sort(1).values
            want[:, :best.shape[1]] = best.int()
        assert torch.equal(got[b], want), b


def test_bounds_of_a_block_copied_to_be_written(pa):
    """Copy-on-write copies no bounds; the ordinary call for the token that is then written covers the copy."""
    k, v, tables, lens = ref.make_cache([40, 40], 2, "bf16", seed=9)
    tables[1] = tables[0]                                        # one request forked into two
    spare = [i for i in range(k.shape[0]) if i not in tables[0].tolist()][0]
    kd, vd = cuda(k, v)
    bounds = torch.full((k.shape[0], 2, 2, 128), 9.0, dtype=k.dtype, device="cuda")
    pa.update_block_bounds(kd, bounds, *cuda(tables, lens, lens))
    pa.copy_blocks(kd, vd, torch.tensor([[int(tables[0, 2]), spare]], device="cuda"))
    tables[1, 2] = spare
    lens[1] = 41
    new = torch.randn((1, 2, 128), generator=torch.Generator().manual_seed(1)).bfloat16().cuda() * 3
    pa.reshape_and_cache(new, new, kd, vd, torch.tensor([spare * 16 + 8], device="cuda"))
    pa.update_block_bounds(kd, bounds, *cuda(tables, lens, torch.tensor([0, 1], dtype=torch.int32)))
    want = ref.block_bounds(kd.cpu(), torch.full(bounds.shape, 9.0, dtype=k.dtype), tables, lens, lens)
    assert torch.equal(bounds.cpu(), want)
