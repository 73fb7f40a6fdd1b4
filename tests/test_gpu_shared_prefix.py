"""Shared-prefix decode against the plain 64-bit attention, over group sizes
around the 128-row tiles, prefixes around the 128-token tiles, ragged and empty
suffixes, and its error paths."""
import math

import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu
# The prefix's softmax weights: one fp16 part (half a step, 2^-11), or two bf16 parts: the upper 16 bits leave less
# than 2^-7 of the weight, which is rounded to bf16 (2^-8 of that): 2^-15.
P_BITS = {"f16": 11, "bf16": 15}


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_464_b200 import capi
    capi.get_device_error(clear=True)
    yield capi
    code, detail = capi.get_device_error(clear=True)
    assert code == 0, (code, detail)


def make(sizes, prefixes, suffix, hkv, G, ty, seed):
    starts, lens, shared = [0], [], []
    for size, prefix in zip(sizes, prefixes):
        first = starts[-1]
        lens += [prefix + suffix(first + i) for i in range(size)]
        shared.append((first, first + size, prefix))
        starts.append(first + size)
    k, v, tables, lens = ref.make_cache(lens, hkv, ty, seed=seed, shared=shared)
    q = ref.make_q(len(lens), hkv * G, ty, seed=seed)
    gs, pl = torch.tensor(starts, dtype=torch.int32), torch.tensor(prefixes, dtype=torch.int32)
    # the prefix entries of a group's other rows are not read
    blind = tables.clone()
    for first, last, prefix in shared:
        blind[first + 1:last, :prefix // 16] = -5
    return q, k, v, tables, blind, lens, gs, pl


def check(pa, sizes, prefixes, suffix, hkv, G, ty, seed, scale=0.088):
    q, k, v, tables, blind, lens, gs, pl = make(sizes, prefixes, suffix, hkv, G, ty, seed)
    want, weight = ref.attention(q, k, v, tables, lens, scale)
    args = [t.cuda() for t in (q, k, v, blind, lens, gs, pl)]
    out = torch.full_like(args[0], float("nan"))
    pa.decode_shared_prefix(*args, scale, out)
    err = (out.cpu().double() - want).abs()
    tol = ref.attention_tolerance(want, weight, ty, P_BITS[ty])
    assert (err <= tol).all(), (err - tol).max()
    assert torch.equal(pa.decode_shared_prefix(*args, scale), out)      # the same bits again


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("size", [1, 2, 16, 17, 33])
def test_group_sizes(pa, ty, G, size):
    check(pa, [size], [272], lambda b: (7 * b) % 40, 2, G, ty, seed=size + G)


@pytest.mark.parametrize("ty,G,size", [("bf16", 8, 31), ("bf16", 8, 32), ("bf16", 8, 48), ("bf16", 8, 49),
                                       ("f16", 1, 127), ("f16", 1, 129), ("f16", 1, 256), ("f16", 1, 257),
                                       ("bf16", 2, 193)])
def test_row_tile_edges(pa, ty, G, size):
    """Rows 128, 256 and 384 are where a CTA's warpgroups change from sharing rows to sharing tiles."""
    check(pa, [size], [400], lambda b: 1 + b % 5, 1, G, ty, seed=size)


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("prefix", [0, 16, 112, 128, 144, 256, 272, 640, 2048, 5008])
@pytest.mark.parametrize("size", [3, 40])
def test_prefix_lengths(pa, ty, prefix, size):
    check(pa, [size], [prefix], lambda b: b % 18, 1, 4, ty, seed=prefix + size)


def test_suffix_longer_than_a_partition(pa):
    check(pa, [5], [160], lambda b: [0, 1, 1024, 1025, 2300][b], 2, 4, "bf16", seed=1)


def test_several_groups(pa):
    """Unequal groups, an empty one, one without a prefix, one of a single sequence, rows without any token."""
    check(pa, [9, 0, 70, 1, 4], [128, 512, 336, 1040, 0], lambda b: [0, 3, 16, 55][b % 4], 2, 4, "bf16", seed=2)


def test_many_groups(pa):
    check(pa, [1 + i % 3 for i in range(70)], [16 * (i % 5) for i in range(70)], lambda b: b % 21, 1, 2, "f16", seed=3)


def test_growing_maxima_rescale(pa):
    """Keys that grow along the prefix: every tile's maximum is far above the last one's."""
    for ty in ("bf16", "f16"):
        for size in (3, 60):
            q, k, v, tables, _, lens, gs, pl = make([size], [1536], lambda b: 20, 1, 4, ty, seed=4)
            grow = (torch.arange(96) // 8 + 1).to(k.dtype)
            k[tables[0, :96].long()] *= grow[:, None, None, None]
            want, weight = ref.attention(q, k, v, tables, lens, 0.088)
            out = pa.decode_shared_prefix(*[t.cuda() for t in (q, k, v, tables, lens, gs, pl)], 0.088).cpu()
            # scores up to 12 times larger than attention_tolerance counts on
            tol = ref.attention_tolerance(want, 12 * weight, ty, P_BITS[ty])
            assert ((out.double() - want).abs() <= tol).all()


def test_no_range_limit_on_values(pa):
    """bf16 values far outside what fp16 holds."""
    q, k, v, tables, _, lens, gs, pl = make([40], [256], lambda b: 9, 1, 4, "bf16", seed=5)
    for factor in (2.0 ** 60, 2.0 ** -60):
        x = v * factor
        want, weight = ref.attention(q, k, x, tables, lens, 0.088)
        out = pa.decode_shared_prefix(*[t.cuda() for t in (q, k, x, tables, lens, gs, pl)], 0.088).cpu()
        tol = ref.attention_tolerance(want, weight, "bf16", 16) - 1e-7     # relative alone
        assert ((out.double() - want).abs() <= tol).all()


def test_live_nan_reaches_its_group_only(pa):
    q, k, v, tables, _, lens, gs, pl = make([5, 6], [256, 256], lambda b: 9, 1, 4, "bf16", seed=5)
    v[tables[0, 3], 2, 0, 17] = float("nan")
    out = pa.decode_shared_prefix(*[t.cuda() for t in (q, k, v, tables, lens, gs, pl)], 0.088).cpu()
    assert out[:5, :, 17].isnan().all() and int(out.isnan().sum()) == 5 * 4


def test_agrees_with_decode(pa):
    from paged_kv_cache_464_b200 import inputs
    case = inputs.make_case("shared_prefix", lens=[1040, 1300, 1536, 1100, 1025] * 7)
    d = "cuda"
    # the workload's copy-on-write destinations hold what the shared block holds
    args = [case.q.to(d), case.k_cache_post.to(d), case.v_cache_post.to(d), case.block_tables.to(d),
            case.context_lens.to(d)]
    gs = torch.tensor([0, 35], dtype=torch.int32, device=d)
    pl = torch.tensor([1024], dtype=torch.int32, device=d)
    out = pa.decode_shared_prefix(*args, gs, pl, case.scale).double()
    dense = pa.decode(*args, case.scale, max_context_len=case.max_context_len).double()
    assert ((out - dense).abs() <= 2e-3 + 1e-2 * dense.abs()).all()


@pytest.mark.expects_device_error
def test_bad_groups_and_lengths_are_reported(pa):
    q, k, v, tables, _, lens, gs, pl = make([3, 4], [128, 160], lambda b: 9, 1, 4, "bf16", seed=6)
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    tol = ref.attention_tolerance(want, weight, "bf16", 16)

    def call(gs=gs, pl=pl, lens=lens, tables=tables, mp=160, ms=9, mg=4):
        out = torch.full_like(q, 6.0).cuda()
        pa.decode_shared_prefix(*[t.cuda() for t in (q, k, v, tables, lens, gs, pl)], 0.088, out, max_prefix_len=mp,
                                max_suffix_len=ms, max_group_size=mg)
        out = out.cpu()
        kept = [b for b in range(7) if (out[b] == 6.0).all()]
        fine = [b for b in range(7) if ((out[b].double() - want[b]).abs() <= tol[b]).all()]
        return kept, fine, pa.get_device_error(clear=True)

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32)

    first, second = [0, 1, 2], [3, 4, 5, 6]
    assert call() == ([], first + second, (0, 0))
    assert call(pl=i32(128, 150)) == (second, first, (8, 1))         # not a multiple of 16
    assert call(pl=i32(-16, 160)) == (first, second, (8, 0))
    assert call(mp=144) == (second, first, (8, 1))                   # beyond the bound
    assert call(mg=3) == (second, first, (8, 1))
    assert call(gs=i32(0, 3, 8)) == (second, first, (8, 1))          # past the batch
    kept, fine, err = call(gs=i32(1, 3, 7))                          # sequence 0 is in no group
    assert kept == [0] and err == (8, -1) and set(second) <= set(fine)
    short = lens.clone()
    short[1], short[5] = 100, -2                                     # shorter than the prefix
    kept, fine, err = call(lens=short)
    assert kept == [1, 5] and fine == [0, 2, 3, 4, 6] and err[0] == 4 and err[1] in (1, 5)
    assert call(ms=8)[0] == first + second
    t = tables.clone()
    t[0, 2] = 10 ** 6
    kept, fine, err = call(tables=t)
    assert kept == [] and err == (1, 10 ** 6) and set(second) <= set(fine)


@pytest.mark.expects_device_error
def test_wait_that_runs_out_is_reported(pa):
    """One CTA of the prefix kernel leaves its first K tile unissued: it gives up, the context stays usable."""
    for size in (4, 60):
        q, k, v, tables, _, lens, gs, pl = make([size], [1024], lambda b: 9, 1, 4, "bf16", seed=7)
        args = [t.cuda() for t in (q, k, v, tables, lens, gs, pl)]
        pa.test_stall_next_launch("shared_prefix", 1)
        pa.decode_shared_prefix(*args, 0.088)
        assert pa.get_device_error(clear=True) == (5, 1)
        want, weight = ref.attention(q, k, v, tables, lens, 0.088)
        out = pa.decode_shared_prefix(*args, 0.088).cpu()
        assert ((out.double() - want).abs() <= ref.attention_tolerance(want, weight, "bf16", 16)).all()


def test_guard_bands(pa):
    """Nothing is written outside out and the workspace."""
    q, k, v, tables, blind, lens, gs, pl = make([33, 5], [272, 144], lambda b: b % 20, 2, 4, "f16", seed=8)
    S, hq, d = q.shape
    qd, kd, vd, td, ld, gd, pd = [t.cuda() for t in (q, k, v, blind, lens, gs, pl)]
    need = pa.decode_shared_prefix_workspace_bytes(S, 2, hq, 2, d, 272, 19, 33)
    pad = 4096
    buf = torch.full((need + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
    room = torch.full((S * hq * d + 2 * pad,), 11.0, dtype=torch.half, device="cuda")
    out = room[pad:-pad].view(S, hq, d)
    kb, vb = kd.clone(), vd.clone()
    pa.decode_shared_prefix(qd, kd, vd, td, ld, gd, pd, 0.088, out, max_prefix_len=272, max_suffix_len=19,
                            max_group_size=33, workspace=buf[pad:pad + need])
    assert (buf[:pad] == 0xA5).all() and (buf[pad + need:] == 0xA5).all()
    assert (room[:pad] == 11.0).all() and (room[-pad:] == 11.0).all()
    assert torch.equal(kb.view(torch.int16), kd.view(torch.int16)) and torch.equal(vb.view(torch.int16), vd.view(torch.int16))
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    assert ((out.cpu().double() - want).abs() <= ref.attention_tolerance(want, weight, "f16", 11)).all()


def test_blocks_past_four_gigabytes(pa):
    blocks, hkv = (1 << 17) + 60, 8
    k = torch.zeros((blocks, 16, hkv, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    q, ks, vs, tables, _, lens, gs, pl = make([6], [256], lambda b: 30, hkv, 4, "bf16", seed=9)
    n = ks.shape[0]
    far = tables.clone()
    far[far >= 0] += blocks - n
    k[blocks - n:], v[blocks - n:] = ks.cuda(), vs.cuda()
    out = pa.decode_shared_prefix(q.cuda(), k, v, far.cuda(), lens.cuda(), gs.cuda(), pl.cuda(), 0.088).cpu()
    want, weight = ref.attention(q, ks, vs, tables, lens, 0.088)
    assert ((out.double() - want).abs() <= ref.attention_tolerance(want, weight, "bf16", 16)).all()


@pytest.mark.parametrize("size", [3, 60])
@pytest.mark.parametrize("ty", ["f16", "bf16"])
@pytest.mark.parametrize("level", [12.0, 19.6, 24.4, 25.7])
def test_tail_under_a_dominant_key(pa, ty, level, size):
    """One key that outweighs every other by 2^level and has no value: the output is the rest of the prefix alone."""
    q, k, v, tables, _, lens, gs, pl = make([size], [8192], lambda b: 0, 1, 4, ty, seed=11)
    ids = tables[0, :512].long()
    k[ids] = 0.0
    k[ids[100], 5, 0, 0] = level * math.log(2.0) / (0.088 * 8)
    q[:], q[..., 0] = 0.0, 8.0
    v[ids] = v[ids].abs() + 0.5
    v[ids[100], 5] = 0.0
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    args = [t.cuda() for t in (q, k, v, tables, lens, gs, pl)]
    err = (pa.decode_shared_prefix(*args, 0.088).cpu().double() - want).abs()
    # the largest score, 25.7 ln 2 = 17.9 at scale, is a single product: attention_tolerance's 2^-13 covers it; each of
    # the 8192 weights is off by 2^-31 of the largest beside its relative error (fp16), |V| is at most weight's own mean
    # of it times 8 (0.5 + |N(0, 1)|, mean 1.3, largest of a million 5.4); half a step of a subnormal fp16 output is 2^-25
    tol = ref.attention_tolerance(want, weight, ty, P_BITS[ty]) - 1e-7 + 8192 * 2.0 ** -31 * 8 * 1.3 * 2.0 ** -13 + 2.0 ** -25
    assert (err <= tol).all(), ((err - tol).max(), err.max(), want.abs().max())


@pytest.mark.parametrize("ty,bits", [("f16", 20), ("bf16", 15)])
@pytest.mark.parametrize("size", [3, 60])
def test_weights_of_two_kinds_that_nearly_cancel(pa, ty, bits, size):
    """Half of the tokens of weight 1 and value 1, half of weight 0.5 + 2^-12 (halfway between two fp16 numbers) and
    value -2: what is left is 1/2000 of either half."""
    q, k, v, tables, _, lens, gs, pl = make([size], [2048], lambda b: 0, 1, 4, ty, seed=12)
    ids = tables[0, :128].long()
    score = math.log(0.5 + 2.0 ** -12) / 0.088
    first = torch.tensor(score / 8).to(k.dtype)
    q[:] = 0.0
    q[..., 0], q[..., 1] = 8.0, 2.0 ** -6
    k[ids], v[ids] = 0.0, 1.0
    k[ids, 1::2, 0, 0], k[ids, 1::2, 0, 1] = first, ((score - 8 * first.double()) * 2 ** 6).to(k.dtype)
    v[ids, 1::2] = -2.0
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    assert (want.abs() < 2.0 ** -10 * weight).all() and (want.abs() > 2.0 ** -13 * weight).all()
    out = pa.decode_shared_prefix(*[t.cuda() for t in (q, k, v, tables, lens, gs, pl)], 0.088).cpu()
    # the weights' relative error; a score of two products below 8 (2^-24 each) times scale, the exponential (2^-22),
    # and sums of 2048 products over 16 steps of 128 tokens each: below 2^-18 together
    tol = ref.HALF_STEP[ty] * want.abs() + (2.0 ** -bits + 2.0 ** -18) * weight + 2.0 ** -25
    assert ((out.double() - want).abs() <= tol).all(), ((out.double() - want).abs() / weight).max()


@pytest.mark.parametrize("at", [0, 1, 31, 32, 40, 65])
def test_one_long_prefix_among_many_groups(pa, at):
    """The group with the prefix stands anywhere among sequences that share nothing, some groups empty."""
    sizes = [i % 3 % 2 for i in range(66)]
    prefixes = [0] * 66
    sizes[at], prefixes[at] = 37, 4000
    sizes[50], prefixes[50] = 5, 272
    check(pa, sizes, prefixes, lambda b: 1 + (13 * b) % 60, 2, 4, "bf16", seed=20 + at)


@pytest.mark.parametrize("G,ty", [(1, "f16"), (8, "bf16")])
def test_groups_of_every_kind(pa, G, ty):
    """More and fewer rows than a CTA takes, long and short prefixes, split suffixes in one of them (a third launch)."""
    sizes, prefixes = [70, 1, 300 // G, 0, 2, 33], [640, 3008, 144, 512, 0, 1040]
    check(pa, sizes, prefixes, lambda b: 2 + b % 30, 1, G, ty, seed=30)
    check(pa, sizes, prefixes, lambda b: 1100 if b == 73 else 2 + b % 30, 1, G, ty, seed=31)


def test_groups_without_a_prefix_leave_the_split_of_the_others(pa):
    """A group of 64 over a long prefix, alone and beside 50 sequences that share nothing: the added rows' own work is
    small, so the call must not take several times as long (nine times, when every group was planned as a long one)."""
    prefix, hq, hkv = 32768, 32, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    blocks = prefix // 16
    k = torch.randn((blocks + 114 * 8, 16, hkv, 128), generator=g, device="cuda").bfloat16()
    v = torch.randn(k.shape, generator=g, device="cuda").bfloat16()
    q = torch.randn((114, hq, 128), generator=g, device="cuda").bfloat16()
    tables = torch.zeros((114, blocks + 8), dtype=torch.int32, device="cuda")
    tables[:64, :blocks] = torch.randperm(blocks, generator=g, device="cuda").int()
    own = blocks + torch.arange(114 * 8, device="cuda").int().view(114, 8)
    tables[:64, blocks:], tables[64:, :8] = own[:64], own[64:]
    lens = torch.tensor([prefix + 100] * 64 + [120] * 50, dtype=torch.int32, device="cuda")

    def run(n):
        gs = torch.tensor([0] + list(range(64, n + 1)), dtype=torch.int32, device="cuda")
        pl = torch.tensor([prefix] + [0] * (n - 64), dtype=torch.int32, device="cuda")
        out = torch.empty_like(q[:n])
        need = pa.decode_shared_prefix_workspace_bytes(n, n - 63, hq, hkv, 128, prefix, 120, 64)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        best = 1e9
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(200_000)      # the call's host side passes behind it
            a.record()
            pa.decode_shared_prefix(q[:n], k, v, tables[:n], lens[:n], gs, pl, 0.088, out, max_prefix_len=prefix,
                                    max_suffix_len=120, max_group_size=64, workspace=ws)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return out, best

    alone, t_alone = run(64)
    mixed, t_mixed = run(114)
    assert ((alone.float() - mixed[:64].float()).abs() <= 2.0 ** -12 + 2.0 ** -7 * alone.float().abs()).all()
    rest = pa.decode(q[64:], k, v, tables[64:], lens[64:], 0.088, max_context_len=120)
    assert ((mixed[64:].float() - rest.float()).abs() <= 2.0 ** -12 + 2.0 ** -7 * rest.float().abs()).all()
    assert t_mixed < 2.5 * t_alone, (t_mixed, t_alone)


@pytest.mark.parametrize("sizes,prefixes", [([7], [272]), ([9, 1, 0, 40, 3], [128, 0, 256, 336, 0]),
                                            ([i % 3 for i in range(70)], [16 * (i % 9) for i in range(70)])])
def test_generous_maxima(pa, sizes, prefixes):
    """Upper bounds far above what the batch has, as a graph captured for any batch is given."""
    q, k, v, tables, _, lens, gs, pl = make(sizes, prefixes, lambda b: 3 + b % 19, 2, 4, "bf16", seed=40)
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    args = [t.cuda() for t in (q, k, v, tables, lens, gs, pl)]
    tol = ref.attention_tolerance(want, weight, "bf16", 15)
    for mp, ms, mg in ((65536, 21, 4096), (2048, 5000, 64), (1 << 20, 40, 64)):
        out = pa.decode_shared_prefix(*args, 0.088, max_prefix_len=mp, max_suffix_len=ms, max_group_size=mg).cpu()
        assert ((out.double() - want).abs() <= tol).all(), (mp, ms, mg)


@pytest.mark.expects_device_error
@pytest.mark.parametrize("bad", [0, 31, 32, 45, 65])
def test_a_bad_group_among_many(pa, bad):
    """Its rows are left as they were, the others are right, and its index is reported."""
    sizes, prefixes = [1 + i % 2 for i in range(66)], [16 * (i % 7) + 16 for i in range(66)]
    q, k, v, tables, _, lens, gs, pl = make(sizes, prefixes, lambda b: 2 + b % 9, 1, 4, "bf16", seed=41)
    want, weight = ref.attention(q, k, v, tables, lens, 0.088)
    tol = ref.attention_tolerance(want, weight, "bf16", 15)
    wrong = pl.clone()
    wrong[bad] += 8
    out = torch.full_like(q, 6.0).cuda()
    pa.decode_shared_prefix(*[t.cuda() for t in (q, k, v, tables, lens, gs, wrong)], 0.088, out, max_prefix_len=128,
                            max_suffix_len=200, max_group_size=2)
    assert pa.get_device_error(clear=True) == (8, bad)
    out, rows = out.cpu(), range(int(gs[bad]), int(gs[bad + 1]))
    for b in range(len(lens)):
        if b in rows:
            assert (out[b] == 6.0).all()
        else:
            assert ((out[b].double() - want[b]).abs() <= tol[b]).all(), b


def test_two_streams_at_once(pa):
    """Calls that overlap, each with its own workspace: every one gives what it gives alone."""
    work = []
    for i, (size, prefix, suffix) in enumerate([(60, 8192, 30), (9, 20000, 2100)]):
        q, k, v, tables, _, lens, gs, pl = make([size], [prefix], lambda b: suffix - b % 7, 2, 4, "bf16", seed=50 + i)
        args = [t.cuda() for t in (q, k, v, tables, lens, gs, pl)]
        maxima = dict(max_prefix_len=prefix, max_suffix_len=suffix, max_group_size=size)
        need = pa.decode_shared_prefix_workspace_bytes(size, 1, 8, 2, 128, prefix, suffix, size)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        work.append((args, maxima, ws, pa.decode_shared_prefix(*args, 0.088, workspace=ws, **maxima), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[torch.empty_like(w[3]) for _ in range(30)] for w in work]
    for i in range(30):
        for (args, maxima, ws, _, stream), out in zip(work, outs):
            pa.decode_shared_prefix(*args, 0.088, out[i], workspace=ws, stream=stream, **maxima)
    torch.cuda.synchronize()
    for w, out in zip(work, outs):
        assert all(torch.equal(o, w[3]) for o in out)
