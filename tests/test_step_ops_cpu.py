"""Host checks of rotate-and-append, shared-prefix decode and block-sparse
decode: every refusal comes back before any CUDA call (16 is a dummy device
address, never dereferenced), and the binding refuses what it can see."""
import pytest
import torch

NULL, DTYPE, SHAPE, WORKSPACE, ALIGN = 1, 2, 3, 4, 6
F32, F16, BF16, FP8 = 0, 1, 2, 3
BIG = 1 << 32


@pytest.fixture(scope="module")
def capi():
    from paged_kv_cache_464_b200 import build
    build.build()
    from paged_kv_cache_464_b200 import capi
    return capi


def test_rope_table_refusals(capi):
    r = capi.raw.pa_rope_table
    assert r(None, 8, 64, 1e4, None) == NULL
    assert r(16, 0, 64, 1e4, None) == SHAPE and r(16, 8, 63, 1e4, None) == SHAPE and r(16, 8, 0, 1e4, None) == SHAPE
    assert r(16, 8, 64, 0.0, None) == SHAPE and r(16, 8, 64, float("nan"), None) == SHAPE
    assert r(8, 8, 64, 1e4, None) == ALIGN


def _rope(capi, fp8=False, **k):
    # q_out, q, key and value far apart: their rows must not overlap
    a = dict(qo=BIG, q=2 * BIG, key=3 * BIG, val=4 * BIG, kc=16, vc=16, pos=16, cs=16, slot=16, T=4, so=1024, sq=1024,
             sk=256, sv=256, maxp=64, rot=128, il=0, NB=8, bs=16, Hq=8, Hkv=2, D=128, dt=BF16, ks=0.1, vs=0.1)
    a.update(k)
    args = [a[x] for x in ("qo", "q", "key", "val", "kc", "vc", "pos", "cs", "slot", "T", "so", "sq", "sk", "sv", "maxp",
                           "rot", "il", "NB", "bs", "Hq", "Hkv", "D", "dt")]
    if fp8:
        return capi.raw.pa_rope_and_cache_fp8(*args, a["ks"], a["vs"], None)
    return capi.raw.pa_rope_and_cache(*args, None)


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_refusals(capi, fp8):
    def rope(**k):
        return _rope(capi, fp8, **k)
    assert rope(T=0) == 0
    assert rope(T=-1) == SHAPE and rope(NB=0) == SHAPE and rope(bs=32) == SHAPE and rope(D=64) == SHAPE
    assert rope(dt=7) == DTYPE and rope(dt=FP8) == DTYPE
    if fp8:
        assert rope(dt=F32) == DTYPE
        assert rope(ks=0.0) == SHAPE and rope(vs=float("inf")) == SHAPE
    assert rope(Hq=0) == SHAPE and rope(maxp=0) == SHAPE
    assert rope(rot=0) == SHAPE and rope(rot=8) == SHAPE and rope(rot=144) == SHAPE
    assert rope(sq=1016) == SHAPE and rope(so=1016) == SHAPE and rope(sk=248) == SHAPE and rope(sv=248) == SHAPE
    assert rope(sq=1 << 31) == SHAPE
    assert rope(sq=1028) == ALIGN and rope(sk=260) == ALIGN and rope(so=1028) == ALIGN
    for name in ("qo", "q", "key", "val", "kc", "vc", "pos", "cs", "slot"):
        assert rope(**{name: None}) == NULL, name
        assert rope(**{name: 4}) == ALIGN, name
    # q_out: q itself, or apart from every input
    assert rope(qo=2 * BIG, so=2048) == SHAPE            # q's pointer with another stride
    assert rope(qo=2 * BIG + 16) == SHAPE
    assert rope(qo=3 * BIG - 16) == SHAPE and rope(qo=4 * BIG + 512) == SHAPE


def test_rope_refusals_f32(capi):
    assert _rope(capi, dt=F32, D=64, rot=64, so=512, sq=512, sk=128, sv=128, T=0) == 0
    assert _rope(capi, dt=F32, D=64, rot=60, so=512, sq=512, sk=128, sv=128) == SHAPE


def _shared(capi, **k):
    a = dict(out=16, q=16, kc=16, vc=16, bt=16, mbs=64, cl=16, gs=16, pl=16, S=4, n=1, Hq=32, mp=512, ms=64, mg=4,
             scale=0.088, ws=None, wsb=0, NB=8, bs=16, Hkv=8, D=128, dt=BF16)
    a.update(k)
    return capi.raw.pa_decode_shared_prefix(*[a[x] for x in (
        "out", "q", "kc", "vc", "bt", "mbs", "cl", "gs", "pl", "S", "n", "Hq", "mp", "ms", "mg", "scale", "ws", "wsb",
        "NB", "bs", "Hkv", "D", "dt")], None)


def test_shared_prefix_refusals(capi):
    def f(**k):
        return _shared(capi, **k)
    assert f(S=0, n=0, mg=0) == 0
    assert f(dt=F32, D=64) == DTYPE and f(dt=FP8) == DTYPE and f(dt=9) == DTYPE
    assert f(D=64) == SHAPE and f(bs=8) == SHAPE and f(NB=0) == SHAPE
    assert f(S=-1) == SHAPE and f(n=-1) == SHAPE and f(n=0) == SHAPE and f(mg=0) == SHAPE and f(mg=-1) == SHAPE
    assert f(Hq=30) == SHAPE and f(Hq=48) == SHAPE and f(Hq=128) == SHAPE and f(Hq=0) == SHAPE
    assert f(mp=-16) == SHAPE and f(mp=500) == SHAPE and f(ms=-1) == SHAPE
    assert f(mbs=-1) == SHAPE and f(mbs=1 << 28) == SHAPE
    assert f(scale=0.0) == SHAPE and f(scale=-1.0) == SHAPE and f(scale=float("nan")) == SHAPE
    assert f(n=(1 << 31) - 1, mg=1 << 24, Hq=1 << 19, Hkv=1 << 16) == SHAPE   # a grid past 2^63
    assert f(S=1 << 20, Hq=1 << 14, Hkv=1 << 14) == SHAPE
    for name in ("out", "q", "kc", "vc", "bt", "cl", "gs", "pl"):
        assert f(**{name: None}) == NULL, name
    for name in ("out", "q", "kc", "vc"):
        assert f(**{name: 8}) == ALIGN, name
    for name in ("bt", "cl", "gs", "pl"):
        assert f(**{name: 2}) == ALIGN, name
    need = capi.decode_shared_prefix_workspace_bytes(4, 1, 32, 8, 128, 512, 64, 4)
    assert need >= 4 * 32 * 2 * (128 + 2) * 4      # a prefix and a suffix partial a row at least
    assert f() == WORKSPACE and f(ws=256, wsb=need - 1) == WORKSPACE
    assert f(ws=128, wsb=need) == ALIGN


def test_shared_prefix_workspace_sizes(capi):
    size = capi.decode_shared_prefix_workspace_bytes
    assert size(0, 0, 32, 8, 128, 512, 64, 0) == 0
    assert size(4, 1, 32, 8, 64, 512, 64, 4) == 0 and size(4, 0, 32, 8, 128, 512, 64, 4) == 0
    assert size(4, 1, 32, 8, 128, 500, 64, 4) == 0
    assert size(4, 1, 32, 8, 128, 0, 64, 4) > 0             # nothing shared: the suffix partials
    assert size(4, 1, 32, 8, 128, 512, 0, 4) > 0
    assert size(64, 1, 32, 8, 128, 32768, 512, 64) < 1 << 28


def _bounds(capi, **k):
    a = dict(kc=16, bb=16, bt=16, mbs=4, cl=16, nl=16, S=2, mn=1, NB=8, bs=16, Hkv=2, D=128, dt=BF16)
    a.update(k)
    return capi.raw.pa_update_block_bounds(*[a[x] for x in ("kc", "bb", "bt", "mbs", "cl", "nl", "S", "mn", "NB", "bs",
                                                            "Hkv", "D", "dt")], None)


def test_block_bounds_refusals(capi):
    def f(**k):
        return _bounds(capi, **k)
    assert f(S=0) == 0 and f(mn=0) == 0
    assert f(dt=FP8) == DTYPE and f(dt=7) == DTYPE and f(D=64) == SHAPE and f(bs=8) == SHAPE
    assert f(S=-1) == SHAPE and f(mn=-1) == SHAPE and f(mbs=-1) == SHAPE
    for name in ("kc", "bb", "bt", "cl", "nl"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: 2}) == ALIGN, name


def _select(capi, **k):
    a = dict(sel=16, q=16, bb=16, bt=16, mbs=64, cl=16, S=2, Hq=8, ml=512, K=4, sink=1, rec=1, ws=None, wsb=0, NB=8,
             bs=16, Hkv=2, D=128, dt=BF16)
    a.update(k)
    return capi.raw.pa_select_blocks(*[a[x] for x in ("sel", "q", "bb", "bt", "mbs", "cl", "S", "Hq", "ml", "K", "sink",
                                                      "rec", "ws", "wsb", "NB", "bs", "Hkv", "D", "dt")], None)


def test_select_blocks_refusals(capi):
    def f(**k):
        return _select(capi, **k)
    assert f(S=0) == 0
    assert f(dt=FP8) == DTYPE and f(dt=7) == DTYPE and f(D=64) == SHAPE
    assert f(K=0) == SHAPE and f(K=-1) == SHAPE and f(sink=-1) == SHAPE and f(rec=-1) == SHAPE
    assert f(K=(1 << 26) + 1) == SHAPE
    assert f(sink=3, rec=2) == SHAPE and f(ml=-1) == SHAPE and f(Hq=6) == SHAPE and f(Hq=7) == SHAPE
    for name in ("sel", "q", "bb", "bt", "cl"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: 2}) == ALIGN, name
    need = capi.select_blocks_workspace_bytes(2, 2, 512)
    assert need >= 2 * 2 * 32 * 8
    assert f() == WORKSPACE and f(ws=256, wsb=need - 1) == WORKSPACE and f(ws=64, wsb=need) == ALIGN
    assert capi.select_blocks_workspace_bytes(0, 2, 512) == 0


def _selected(capi, **k):
    a = dict(out=16, q=16, kc=16, vc=16, bt=16, mbs=64, cl=16, sel=16, S=2, Hq=8, K=400, scale=0.088, ws=None, wsb=0,
             NB=8, bs=16, Hkv=2, D=128, dt=BF16)
    a.update(k)
    return capi.raw.pa_decode_selected(*[a[x] for x in ("out", "q", "kc", "vc", "bt", "mbs", "cl", "sel", "S", "Hq", "K",
                                                        "scale", "ws", "wsb", "NB", "bs", "Hkv", "D", "dt")], None)


def test_decode_selected_refusals(capi):
    def f(**k):
        return _selected(capi, **k)
    assert f(S=0) == 0
    assert f(dt=FP8) == DTYPE and f(dt=7) == DTYPE and f(D=64) == SHAPE
    assert f(K=(1 << 26) + 1) == SHAPE and capi.decode_selected_workspace_bytes(2, 8, 2, 128, (1 << 26) + 1) == 0
    assert f(K=0) == SHAPE and f(K=-3) == SHAPE and f(Hq=6) == SHAPE and f(S=-1) == SHAPE
    assert f(scale=float("inf")) == SHAPE and f(mbs=-1) == SHAPE and f(mbs=1 << 28) == SHAPE
    for name in ("out", "q", "kc", "vc", "bt", "cl", "sel"):
        assert f(**{name: None}) == NULL, name
        assert f(**{name: 2}) == ALIGN, name
    need = capi.decode_selected_workspace_bytes(2, 8, 2, 128, 400)
    assert need > 0
    assert f() == WORKSPACE and f(ws=256, wsb=need - 1) == WORKSPACE and f(ws=64, wsb=need) == ALIGN


def test_binding_refuses_host_tensors(capi):
    bf = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    kv = torch.zeros((2, 1, 128), dtype=torch.bfloat16)
    cache = torch.zeros((4, 16, 1, 128), dtype=torch.bfloat16)
    i64 = torch.zeros(2, dtype=torch.int64)
    i32 = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        capi.rope_and_cache(bf, kv, kv, i64, torch.zeros((8, 128)), cache, cache, i64)
    with pytest.raises(ValueError):
        capi.rope_and_cache_fp8(bf, kv, kv, i64, torch.zeros((8, 128)), cache, cache, i64, 1.0, 1.0)
    with pytest.raises(ValueError):
        capi.decode_shared_prefix(bf, cache, cache, table, i32, i32, i32[:1], 0.1)
    with pytest.raises(ValueError):
        capi.update_block_bounds(cache, torch.zeros((4, 2, 1, 128), dtype=torch.bfloat16), table, i32, i32)
    with pytest.raises(ValueError):
        capi.select_blocks(bf, torch.zeros((4, 2, 1, 128), dtype=torch.bfloat16), table, i32, 2)
    with pytest.raises(ValueError):
        capi.decode_selected(bf, cache, cache, table, i32, torch.zeros((2, 1, 3), dtype=torch.int32), 0.1)
    with pytest.raises(ValueError):
        capi.rope_table(8, 64, device="cpu")


def test_stall_hook_takes_the_prefix_kernel(capi):
    assert capi.raw.pa_test_stall_next_launch(3, -1) == 0
    assert capi.raw.pa_test_stall_next_launch(4, 0) == SHAPE


def test_shared_prefix_plan_of_a_mixed_batch(capi):
    """Sequences that share nothing (groups of one without a prefix) leave a long prefix its partitions: the workspace
    has room for a group's partials as if it were alone.  (Its rows' share grows with the batch, so fewer may be best.)"""
    size = capi.decode_shared_prefix_workspace_bytes
    alone = size(64, 1, 32, 8, 128, 32768, 512, 64) / 64
    for n in (1, 8, 20, 50):
        assert size(64 + n, 1 + n, 32, 8, 128, 32768, 512, 64) / (64 + n) >= 0.6 * alone


def test_rope_refuses_rows_that_share_columns(capi):
    """q_out in the same wide rows as q, key and value (rows of 1024, 256 and 256 elements, 2560 apart): any element in
    common, in the same row or a neighbouring one, is refused."""
    wide, row, kv = 2560 * 2, 1024 * 2, 256 * 2
    a = dict(so=2560, sq=2560, sk=2560, sv=2560, T=4, q=BIG, key=BIG + row, val=BIG + row + kv)
    for shift in (16, row - 16, 16 - row):
        for turn in (-wide, 0, wide):
            assert _rope(capi, **a, qo=BIG + shift + turn) == SHAPE, (shift, turn)
    free = row + 2 * kv                                   # the columns behind value
    for shift in (-16, 16):                               # into value, and around into the next row's q
        assert _rope(capi, **a, qo=BIG + free + shift) == SHAPE, shift
    # other strides are compared as whole ranges
    assert _rope(capi, **{**a, "so": 5120}, qo=BIG + free) == SHAPE


def test_shared_prefix_refuses_more_groups_than_its_loops_count(capi):
    """The kernels walk the groups 32 at a time in 32 bits: without a bound, 2^31 - 1 groups would never end."""
    for mp in (0, 512):
        assert _shared(capi, n=(1 << 24) + 1, mp=mp) == SHAPE and _shared(capi, n=(1 << 31) - 1, mp=mp) == SHAPE
    assert _shared(capi, n=1 << 24, mp=0) == WORKSPACE
    assert capi.decode_shared_prefix_workspace_bytes(4, (1 << 24) + 1, 32, 8, 128, 0, 64, 4) == 0
