"""The measured cases of perf/operators.py, and some more of their ranges: the
kernels' outputs beside the plain forms' and the definitions' in 64 bits."""
import random

import pytest
import torch

from perf import operators

pytestmark = pytest.mark.gpu

DRAWS = 24


def cases():
    rng = random.Random(20)
    drawn = [operators.draw(rng) for _ in range(DRAWS)]
    return operators.listed() + [dict(c, name=f"drawn {i} {c['op']}") for i, c in enumerate(drawn)]


def outputs(case, own):
    state = operators.prepare(case, 3)
    operators.own = own
    try:
        out = operators.run(state)
    finally:
        operators.own = False
    out = out if isinstance(out, dict) else {"out": out}
    return {k: v.clone() for k, v in out.items()}


@pytest.fixture(scope="module", autouse=True)
def no_device_error():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_464_b200 import capi
    capi.get_device_error(clear=True)
    yield
    assert capi.get_device_error(clear=True) == (0, 0)


@pytest.mark.parametrize("case", cases(), ids=lambda c: c["name"].replace(" ", "_"))
def test_case(case):
    got, plain = outputs(case, True), outputs(case, False)
    exact = operators.exact(case, 3)
    for name in got:
        if name == "out" and case["op"] != "bounds":
            continue
        if got[name].dtype == torch.float8_e4m3fn:
            # (the plain form's quotient is a product with the scale's reciprocal, at times another code)  Half a step:
            # 2^-4 relative, 2^-10 absolute below the smallest normal 2^-6; the quotient 2^-24 relative.  The rotation
            # a c - b s of |a|, |b| < 6 may cancel: its products are off by 6 * 2^-24 each, the sum (below 8.5) by
            # 8.5 * 2^-24, together less than 2^-19, which the scale divides.
            err, want = (got[name].double() - exact[name]).abs(), exact[name].abs()
            tol = want.clamp(min=2.0 ** -6) * (2.0 ** -4 + 2.0 ** -20) + 2.0 ** -19 / 0.0125
            assert (err <= tol).all(), name
            continue
        # rotated rows, caches, bounds, chosen blocks: the same bits (-0 and 0 are one bound)
        a, b = got[name], plain[name]
        if case["op"] == "bounds":
            assert torch.equal(a, b)
        else:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    if case["op"] in ("shared", "sparse"):
        exact = exact["out"] if isinstance(exact, dict) else exact
        norm = exact.norm()
        if norm == 0:
            assert (got["out"] == 0).all()
            return
        own, theirs = ((x["out"].double() - exact).norm() / norm for x in (got, plain))
        # The plain form sums in 32 bits and rounds once.  The kernels' weights are off by up to 2^-15 more (bf16),
        # 2^-20 (fp16) or nothing (fp32) of the mean of |V|, whose sums over n_eff tokens of either sign shrink the
        # result by as much as the errors, each of its own sign: the same 2^-15 of the result, in quadrature, and the
        # fp32 sums' order (2^-22 over the few hundred steps of a walk).
        weights = {"bf16": 2.0 ** -15, "f16": 2.0 ** -20, "f32": 0.0}[case["type"]]
        assert own <= (theirs ** 2 + (8 * weights) ** 2) ** 0.5 + 2.0 ** -20, (own, theirs)
