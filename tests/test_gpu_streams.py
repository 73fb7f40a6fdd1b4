"""Calls given a stream: lengths written on that stream a moment before the call
are the ones that the call goes by when it reads its maxima itself, and what it
allocates belongs to that stream."""
import pytest
import torch

import step_reference as ref

pytestmark = pytest.mark.gpu
HQ, HKV, D = 8, 2, 128
LATE = [700, 1200, 33]      # written on the side stream behind a wait of some 50 ms
EARLY = [16, 16, 16]        # what the tensors hold before


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_464_b200 import capi
    capi.get_device_error(clear=True)
    yield capi
    code, detail = capi.get_device_error(clear=True)
    assert code == 0, (code, detail)


class Batch:
    def __init__(self, pa, fp8=False):
        k, v, tables, _ = ref.make_cache(LATE, HKV, "bf16", seed=3)
        k, v = k.nan_to_num(0.0), v.nan_to_num(0.0)
        self.k, self.v, self.tables = k.cuda(), v.cuda(), tables.cuda()
        self.q = ref.make_q(3, HQ, "bf16", seed=3).cuda()
        self.key, self.value = (torch.zeros((3, HKV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if fp8:
            self.k, self.v = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (self.k, self.v))
        self.bounds = torch.zeros((k.shape[0], 2, HKV, D), dtype=torch.bfloat16, device="cuda")
        pa.update_block_bounds(k.cuda(), self.bounds, self.tables, *[torch.tensor(LATE, dtype=torch.int32, device="cuda")] * 2)
        self.lens = torch.tensor(EARLY, dtype=torch.int32, device="cuda")
        self.new = torch.ones(3, dtype=torch.int32, device="cuda")
        self.gs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
        self.prefix = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
        self.starts = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
        self.chunk = ref.make_q(40, HQ, "bf16", seed=4).cuda()

    def finish(self):
        """The lengths and the groups that the step is about."""
        self.lens.copy_(self.late["lens"], non_blocking=True)
        self.new.copy_(self.late["new"], non_blocking=True)
        self.gs.copy_(self.late["gs"], non_blocking=True)
        self.starts.copy_(self.late["starts"], non_blocking=True)

    late = {"lens": torch.tensor(LATE, dtype=torch.int32), "new": torch.tensor([40, 500, 33], dtype=torch.int32),
            "gs": torch.tensor([0, 2, 3], dtype=torch.int32), "starts": torch.tensor([0, 1, 30, 40], dtype=torch.int32)}


def bounds(pa, b, stream):
    out = torch.full_like(b.bounds, 5.0)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    pa.update_block_bounds(b.k, out, b.tables, b.lens, b.new, stream=stream)
    return out


CALLS = {
    "shared_prefix": lambda pa, b, s: pa.decode_shared_prefix(b.q, b.k, b.v, b.tables, b.lens, b.gs, b.prefix, 0.088, stream=s),
    "bounds": bounds,
    "select": lambda pa, b, s: pa.select_blocks(b.q, b.bounds, b.tables, b.lens, 5, stream=s),
    "decode": lambda pa, b, s: pa.decode(b.q, b.k, b.v, b.tables, b.lens, 0.088, stream=s),
    "decode_append": lambda pa, b, s: pa.decode_append(b.q, b.key, b.value, b.k, b.v, b.tables, b.lens, 0.088, stream=s),
    "decode_fp8": lambda pa, b, s: pa.decode_fp8(b.q, b.k, b.v, 0.5, 0.5, b.tables, b.lens, 0.088, stream=s),
    "prefill": lambda pa, b, s: pa.prefill(b.chunk, b.k, b.v, b.tables, b.lens, b.starts, 0.088, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_maxima_are_those_of_the_calls_stream(pa, name):
    call = CALLS[name]
    b = Batch(pa, fp8=name == "decode_fp8")
    b.finish()
    torch.cuda.synchronize()
    want = call(pa, b, None).clone()
    b = Batch(pa, fp8=name == "decode_fp8")
    b.late = {key: x.pin_memory() for key, x in b.late.items()}    # so that the copies do not wait
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
        b.finish()
    got = call(pa, b, s)
    s.synchronize()
    assert pa.get_device_error(clear=True) == (0, 0)
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", CALLS)
def test_what_a_call_allocates_is_its_streams(pa, name, monkeypatch):
    """(Scratch of another stream could be handed out again while the call still runs.)"""
    b = Batch(pa, fp8=name == "decode_fp8")
    b.finish()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    seen = []
    for make in ("empty", "empty_like"):
        real = getattr(torch, make)

        def watched(*args, real=real, **kwargs):
            t = real(*args, **kwargs)
            if t.is_cuda:
                seen.append(torch.cuda.current_stream())
            return t
        monkeypatch.setattr(pa.torch, make, watched)
    CALLS[name](pa, b, s)
    monkeypatch.undo()
    s.synchronize()
    assert all(x == s for x in seen) and (seen or name == "bounds")
