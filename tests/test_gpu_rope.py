"""Rotate-and-append against the formula in 64 bits, and bit by bit against the
same fp32 products and sums in torch.

Tolerance of a rotated element a c - b s: two fp32 products and a sum, each off by
at most 2^-24 relative (together below 2 * 2^-24 * (|a c| + |b s|)), then half a
step of the stored type."""
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


def make(T, hq, hkv, ty, rotary, max_position, seed, padding=()):
    g = torch.Generator().manual_seed(seed)
    d, t = ref.HEAD_DIM[ty], ref.TYPES[ty]
    qkv = torch.randn((T, hq + 2 * hkv, d), generator=g).to(t)
    pos = torch.randint(0, max_position, (T,), generator=g)
    blocks = -(-max(T, 1) // 16) + 3
    slot = torch.randperm(blocks * 16, generator=g)[:T].clone()
    for i in padding:
        pos[i], slot[i] = -1 - i, -1
    return qkv, pos, slot, blocks


def plain_fp32(x, positions, cos_sin, interleaved):
    """The same elementary fp32 operations in torch."""
    r = cos_sin.shape[1]
    cs = cos_sin[positions.clamp(min=0)][:, None]
    c, s = cs[..., :r // 2], cs[..., r // 2:]
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,part", [(1, 1, 1, 1), (3, 8, 8, 2), (17, 32, 8, 1), (130, 5, 3, 4), (257, 64, 8, 1)])
def test_matches_the_formula(pa, ty, interleaved, T, hq, hkv, part):
    d = ref.HEAD_DIM[ty]
    r = d // part
    qkv, pos, slot, blocks = make(T, hq, hkv, ty, r, 4096, seed=T + hq, padding=[T - 1] if T > 1 else [])
    table = pa.rope_table(4096, r, 10000.0)
    dev = qkv.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    kc = torch.full((blocks, 16, hkv, d), 7.0, dtype=qkv.dtype, device="cuda")
    vc = torch.full_like(kc, 7.0)
    q_out = torch.full((T, hq, d), 3.0, dtype=qkv.dtype, device="cuda")
    res = pa.rope_and_cache(q, k, v, pos.cuda(), table, kc, vc, slot.cuda(), q_out, interleaved=interleaved)
    assert res is q_out
    torch.cuda.synchronize()
    cs = table.cpu()
    live = pos >= 0
    for got, x in ((q_out.cpu()[live], qkv[live][:, :hq]),
                   (kc.cpu().view(-1, hkv, d)[slot[live]], qkv[live][:, hq:hq + hkv])):
        want, mag = ref.rotate(x.double(), pos[live], cs, interleaved)
        err = (got.double() - want).abs()
        tol = ref.HALF_STEP[ty] * want.abs() + (2 + 2 * ref.HALF_STEP[ty]) * 2.0 ** -24 * mag + 2.0 ** -25 * (ty == "f16")
        assert (err <= tol).all(), (err - tol).max()
        assert torch.equal(got, plain_fp32(x, pos[live], cs, interleaved).to(got.dtype))
    assert torch.equal(vc.cpu().view(-1, hkv, d)[slot[live]], qkv[live][:, hq + hkv:])
    # padding rows and every other slot stay as they were
    assert (q_out.cpu()[~live].float() == 3.0).all()
    rest = torch.ones(blocks * 16, dtype=torch.bool)
    rest[slot[live]] = False
    assert (kc.cpu().view(-1, hkv, d)[rest].float() == 7.0).all() and (vc.cpu().view(-1, hkv, d)[rest].float() == 7.0).all()


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved,part", [(False, 1), (True, 2)])
def test_fp8_cache(pa, ty, interleaved, part):
    T, hq, hkv, d = 75, 8, 2, 128
    r = d // part
    qkv, pos, slot, blocks = make(T, hq, hkv, ty, r, 512, seed=5, padding=[4, 74])
    qkv[0, hq:] *= 1000     # saturates
    table = pa.rope_table(512, r, 500000.0)
    dev = qkv.cuda()
    kc = torch.zeros((blocks, 16, hkv, d), dtype=torch.uint8, device="cuda")
    vc, vc2 = torch.zeros_like(kc), torch.zeros_like(kc)
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    q_out = pa.rope_and_cache_fp8(q, k, v, pos.cuda(), table, kc, vc, slot.cuda(), 0.0125, 0.02,
                                  interleaved=interleaved)
    live = pos >= 0
    kx = plain_fp32(qkv[live][:, hq:hq + hkv], pos[live], table.cpu(), interleaved)
    codes = (kx / torch.tensor(0.0125)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(kc.cpu().view(-1, hkv, d)[slot[live]], codes)
    want, _ = ref.rotate(qkv[live][:, hq:hq + hkv].double(), pos[live], table.cpu(), interleaved)
    want = (want / float(torch.tensor(0.0125))).clamp(-448, 448)
    got = codes.view(torch.float8_e4m3fn).double()
    # half a step: 2^-4 relative, 2^-10 absolute below the smallest normal 2^-6; the fp32 quotient 2^-22 more
    assert ((got - want).abs() <= want.abs().clamp(min=2.0 ** -6) * (2.0 ** -4 + 2.0 ** -21)).all()
    # the values' codes are those of the plain quantising write
    pa.reshape_and_cache_fp8(k.contiguous(), v.contiguous(), torch.zeros_like(kc), vc2, slot.cuda(), 0.0125, 0.02)
    assert torch.equal(vc, vc2)
    assert torch.equal(q_out.cpu()[live], plain_fp32(qkv[live][:, :hq], pos[live], table.cpu(), interleaved).to(q.dtype))


def boundary_values(scale, g):
    """32768 fp32 numbers: next to every rounding boundary of E4M3 times the scale, small, large, zero, not finite."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    ties = torch.cat([codes, (codes[1:] + codes[:-1]) / 2, torch.tensor([464.0, 512.0, 2.0 ** -12])])
    near = (ties * float(scale)).float()
    near = torch.cat([near] + [(near.view(torch.int32) + k).clamp(min=0).view(torch.float32) for k in (-3, -2, -1, 1, 2, 3)])
    wide = torch.exp2(torch.rand(8000, generator=g) * 250 - 125)
    x = torch.cat([near, wide, torch.tensor([0.0, float("inf"), 1e-45, 3e38])])
    rest = torch.rand(16384 - x.numel(), generator=g) * 500 * float(scale)
    x = torch.cat([x, rest])
    return torch.cat([x, -x])


@pytest.mark.parametrize("ty", ["bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_fp8_codes_are_those_of_the_fp32_quotient(pa, ty, interleaved):
    """Bit by bit, at every rounding boundary and for every 16-bit value: K elements are made arbitrary fp32 numbers
    by pairs (1, 0) and cosines of any size."""
    T, d = 512, 128
    g = torch.Generator().manual_seed(3)
    step = 2.0 ** -23
    scales = [1.0, 0.0125, 1 + step, 1 + 3 * step, 2 - step, 1.5 + step, 2.0 ** -60, 2.0 ** -61, 2.0 ** 60, 2.0 ** 61,
              1e-30, 1e30, 1e-45, 1e-38, 3e38] + (torch.rand(12, generator=g) + 0.5).tolist()
    x = torch.zeros((T, 3, d), dtype=ref.TYPES[ty])
    x[:, 1, 0::2 if interleaved else 1] = 1.0
    if not interleaved:
        x[:, 1, 64:] = 0.0
    x[:, 2] = torch.arange(65536).view(T, d).to(torch.uint16).view(x.dtype)
    dev = x.cuda()
    at = torch.arange(T, device="cuda")
    for scale in scales:
        scale = torch.tensor(scale, dtype=torch.float32)
        table = torch.zeros((T, d))
        table[:, :64] = boundary_values(scale, g).view(T, 64)
        kc = torch.zeros((T // 16, 16, 1, d), dtype=torch.uint8, device="cuda")
        vc, vc2 = torch.zeros_like(kc), torch.zeros_like(kc)
        pa.rope_and_cache_fp8(dev[:, :1], dev[:, 1:2], dev[:, 2:], at, table.cuda(), kc, vc, at, float(scale), float(scale),
                              interleaved=interleaved)
        got = kc.cpu().view(T, d)
        got = got[:, 0::2] if interleaved else got[:, :64]
        want = (table[:, :64] / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        nan = table[:, :64].isnan()       # (the neighbours of an infinity; a NaN's sign is not a value)
        assert torch.equal(got[~nan], want[~nan]) and ((got[nan] & 0x7f) == 0x7f).all(), float(scale)
        pa.reshape_and_cache_fp8(dev[:, 1:2].contiguous(), dev[:, 2:].contiguous(), torch.zeros_like(kc), vc2, at,
                                 float(scale), float(scale))
        assert torch.equal(vc, vc2), float(scale)


def test_table(pa):
    for n, r, base in ((1, 2, 10000.0), (1000, 128, 10000.0), (131072, 64, 500000.0)):
        table = pa.rope_table(n, r, base).cpu().double()
        want = ref.rope_table(n, r, base)
        # an fp64 angle below 2^17 is off by less than 2^-33 whatever pow's last bits are; then half an fp32 step
        assert ((table - want).abs() <= 2.0 ** -24 * want.abs() + 2.0 ** -33).all()


def test_q_in_place_and_no_cache_write(pa):
    T, hq, hkv, d = 33, 8, 2, 128
    qkv, pos, slot, blocks = make(T, hq, hkv, "bf16", d, 256, seed=9)
    slot[::3] = -1          # rotated, not cached (their blocks are shared already)
    table = pa.rope_table(256, d)
    dev = qkv.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    kc = torch.zeros((blocks, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pa.rope_and_cache(q, k, v, pos.cuda(), table, kc, vc, slot.cuda(), q)
    want = plain_fp32(qkv[:, :hq], pos, table.cpu(), False).bfloat16()
    assert torch.equal(q.cpu(), want)
    assert torch.equal(dev.cpu()[:, hq:], qkv[:, hq:])          # key and value rows are not written
    used = slot[slot >= 0]
    assert (kc.cpu().view(-1, hkv, d)[used].float().abs().sum((1, 2)) > 0).all()
    assert int((kc.cpu().view(-1, hkv, d).float().abs().sum((1, 2)) > 0).sum()) == used.numel()


def test_nan_and_infinity_pass_through(pa):
    T, hq, hkv, d = 2, 1, 1, 128
    x = torch.randn(T, 3, d).half()
    x[0, 1, 3], x[1, 1, 70], x[0, 2, 5] = float("nan"), float("inf"), float("-inf")
    table = pa.rope_table(8, d)
    kc = torch.zeros((1, 16, 1, d), dtype=torch.half, device="cuda")
    vc = torch.zeros_like(kc)
    dev = x.cuda()
    pa.rope_and_cache(dev[:, :1], dev[:, 1:2], dev[:, 2:], torch.tensor([1, 2], device="cuda"), table, kc, vc,
                      torch.tensor([0, 1], device="cuda"))
    want = plain_fp32(x[:, 1:2], torch.tensor([1, 2]), table.cpu(), False).half()
    assert torch.equal(kc[0, :2].cpu().isnan(), want.isnan())
    assert torch.equal(kc[0, :2].cpu().nan_to_num(1.0, 2.0, 3.0), want.nan_to_num(1.0, 2.0, 3.0))
    assert torch.equal(vc[0, :2].cpu(), x[:, 2:])


@pytest.mark.expects_device_error
def test_bad_positions_and_slots_are_skipped(pa):
    T, hq, hkv, d = 4, 2, 1, 128
    qkv, pos, slot, blocks = make(T, hq, hkv, "bf16", d, 64, seed=3)
    table = pa.rope_table(64, d)
    dev = qkv.cuda()
    kc = torch.zeros((blocks, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)

    def call(pos, slot):
        out = torch.full((T, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
        kc.zero_(), vc.zero_()
        pa.rope_and_cache(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], pos.cuda(), table, kc, vc, slot.cuda(), out)
        return out.cpu(), pa.get_device_error(clear=True)

    bad = pos.clone()
    bad[2] = 64
    out, err = call(bad, slot)
    assert err == (7, 64) and (out[2].float() == 5.0).all()
    assert (kc.view(-1, hkv, d)[slot[2]] == 0).all() and (kc.view(-1, hkv, d)[slot[1]] != 0).any()
    bad = slot.clone()
    bad[1] = blocks * 16
    out, err = call(pos, bad)
    assert err == (2, blocks * 16)
    assert torch.equal(out[1], plain_fp32(qkv[:, :hq], pos, table.cpu(), False).bfloat16()[1])   # q is rotated


def test_slots_past_four_gigabytes(pa):
    """The last slot of a cache of 2^17 + 5 blocks of 8 heads (4 GiB and more each)."""
    hq, hkv, d = 8, 8, 128
    blocks = (1 << 17) + 5
    kc = torch.zeros((blocks, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    qkv, pos, _, _ = make(3, hq, hkv, "bf16", d, 64, seed=1)
    slot = torch.tensor([blocks * 16 - 1, 0, (1 << 21) + 3])
    table = pa.rope_table(64, d)
    dev = qkv.cuda()
    pa.rope_and_cache(dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:], pos.cuda(), table, kc, vc, slot.cuda())
    want = plain_fp32(qkv[:, hq:hq + hkv], pos, table.cpu(), False).bfloat16()
    assert torch.equal(kc.view(-1, hkv, d)[slot.cuda()].cpu(), want)
    assert torch.equal(vc.view(-1, hkv, d)[slot.cuda()].cpu(), qkv[:, hq + hkv:])
    assert int((kc.view(-1, hkv * d).abs().amax(1) > 0).sum()) == 3


def test_binding_refusals(pa):
    d = 128
    dev = torch.zeros((4, 4, d), dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros((2, 16, 1, d), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int64, device="cuda")
    table = torch.zeros((8, d), device="cuda")
    q, k, v = dev[:, :2], dev[:, 2:3], dev[:, 3:]

    def call(q=q, k=k, v=v, pos=pos, table=table, kc=kc, slot=pos, out=None):
        return pa.rope_and_cache(q, k, v, pos, table, kc, kc.clone(), slot, out)

    for bad in (dict(q=q.half()), dict(k=k.float()), dict(pos=pos.int()), dict(pos=pos[:3]), dict(slot=pos.int()),
                dict(table=table.double()), dict(k=dev[:, 1:3]), dict(q=dev.transpose(1, 2)), dict(pos=pos.cpu()),
                dict(out=torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")),
                dict(q=torch.zeros((4, 2, 2 * d), dtype=torch.bfloat16, device="cuda")[..., ::2])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(pa.PaError):
        call(out=dev[:, 1:3])        # overlaps q
    with pytest.raises(pa.PaError):
        call(table=torch.zeros((8, 24), device="cuda"))


@pytest.mark.parametrize("order", ["oqkv", "qkvo", "qokv"])
@pytest.mark.parametrize("T", [1, 2, 37])
def test_rotated_q_beside_its_inputs(pa, order, T):
    """q_out as other columns of the buffer that holds q, key and value: slices of the same rows, none in common."""
    hq, hkv, d = 8, 2, 128
    qkv, pos, slot, blocks = make(T, hq, hkv, "bf16", d, 256, seed=T)
    heads = {"q": hq, "k": hkv, "v": hkv, "o": hq}
    at, wide = {}, torch.full((T, 2 * hq + 2 * hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
    n = 0
    for name in order:
        at[name] = wide[:, n:n + heads[name]]
        n += heads[name]
    for name, part in (("q", qkv[:, :hq]), ("k", qkv[:, hq:hq + hkv]), ("v", qkv[:, hq + hkv:])):
        at[name].copy_(part)
    table = pa.rope_table(256, d)
    kc = torch.zeros((blocks, 16, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    pa.rope_and_cache(at["q"], at["k"], at["v"], pos.cuda(), table, kc, vc, slot.cuda(), at["o"])
    assert torch.equal(at["o"].cpu(), plain_fp32(qkv[:, :hq], pos, table.cpu(), False).bfloat16())
    assert torch.equal(torch.cat([at["q"], at["k"], at["v"]], 1).cpu(), qkv)
    assert torch.equal(vc.view(-1, hkv, d)[slot.cuda()].cpu(), qkv[:, hq + hkv:])
    first = sum(heads[c] for c in order[:order.index("q")])
    for lo in (first - hq + 1, first + hq - 1):      # a head in common with q
        if 0 <= lo and lo + hq <= wide.shape[1]:
            with pytest.raises(pa.PaError):
                pa.rope_and_cache(at["q"], at["k"], at["v"], pos.cuda(), table, kc, vc, slot.cuda(), wide[:, lo:lo + hq])


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (30, 3), (4, 20)])
def test_large_batches(pa, ty, interleaved, hq, hkv):
    """More than a wave of CTAs: three heads a thread, with a last one that 36, 44 or 48 rows leave in part without."""
    T, d = 2999, ref.HEAD_DIM[ty]
    part = 2 if hq == 30 else 1
    qkv, pos, slot, blocks = make(T, hq, hkv, ty, d // part, 5000, seed=hq, padding=[0, 1501, 2998])
    table = pa.rope_table(5000, d // part, 10000.0)
    dev, pos, slot = qkv.cuda(), pos.cuda(), slot.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    live = pos >= 0
    want_q, want_k = (plain_fp32(x, pos, table, interleaved) for x in (q, k))    # (elementary operations, on the device)

    def caches(dtype):
        kc = torch.full((blocks, 16, hkv, d), 7.0, device="cuda").to(dtype)
        return kc, kc.clone()

    kinds = ["same"] if ty == "f32" else ["same", "fp8"]
    for kind in kinds:
        kc, vc = caches(torch.float8_e4m3fn if kind == "fp8" else dev.dtype)
        q_out = torch.full((T, hq, d), 3.0, dtype=dev.dtype, device="cuda")
        if kind == "fp8":
            pa.rope_and_cache_fp8(q, k, v, pos, table, kc, vc, slot, 0.0125, 0.02, q_out, interleaved=interleaved)
            # (by a tensor: torch divides a CUDA tensor by a number as a product with its reciprocal)
            rows_k = (want_k / torch.full_like(want_k, 0.0125)).clamp(-448, 448).to(kc.dtype)
            rows_v = (v.float() / torch.full_like(v.float(), 0.02)).clamp(-448, 448).to(kc.dtype)
        else:
            pa.rope_and_cache(q, k, v, pos, table, kc, vc, slot, q_out, interleaved=interleaved)
            rows_k, rows_v = want_k.to(dev.dtype), v
        rows_q = torch.where(live[:, None, None], want_q.to(dev.dtype), torch.full_like(q_out, 3.0))
        assert torch.equal(q_out, rows_q)
        for cache, rows in ((kc, rows_k), (vc, rows_v)):
            want = caches(cache.dtype)[0].view(torch.uint8).view(-1, hkv, d * cache.element_size())
            want[slot[live]] = rows[live].contiguous().view(torch.uint8)
            assert torch.equal(cache.view(torch.uint8).view(want.shape), want)
