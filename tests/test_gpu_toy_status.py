"""ToyTarget in 8 bits reports what its norms and products record on the device."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300.verify_pass import ToyTarget, VerifyPass

pytestmark = pytest.mark.gpu
DEV = "cuda"
R, G, V = 4, 3, 512


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _target(eight_bit=True):
    vp = VerifyPass(R, G, 2, 4, 2, 64, capacity=64, page_size=16, device=DEV)
    target = ToyTarget(vp, V, 256, seed=5, eight_bit=eight_bit)
    return vp, target


def _pass(vp, target):
    vp.assemble(_i32([3, 0, 2, 3]), _i32([1, 2, 3, 4]), _i32([[7, 8, 9]] * R))
    out = torch.zeros((R, G + 1, V), dtype=torch.bfloat16, device=DEV)
    target.logits(out)
    return out


@pytest.mark.parametrize("eight_bit", [False, True])
def test_nothing_is_reported_where_all_is_well(eight_bit):
    vp, target = _target(eight_bit)
    target.prompt(torch.arange(70, device=DEV), [30, 1, 9, 30])
    out = _pass(vp, target)
    assert vp.check() == 0 and target.check() == 0 and bool(torch.isfinite(out).all())


def test_a_row_that_is_not_finite_is_reported_once():
    vp, target = _target()
    target.embed[8] = float("inf")
    _pass(vp, target)
    vp.check()
    assert target.check() == ds.ERR_NONFINITE_INPUT and target.check() == 0
    # weights too
    target.embed[8] = 0
    target._codes(torch.full((256, 256), float("nan"), dtype=torch.bfloat16, device=DEV))
    assert target.check() == ds.ERR_NONFINITE_INPUT


def test_a_wait_that_runs_out_in_a_projection_is_reported():
    vp, target = _target()
    want = _pass(vp, target).clone()
    assert vp.check() == 0 and target.check() == 0
    ds.set_wait_limit(1)
    try:
        _pass(vp, target)
        torch.cuda.synchronize()
    finally:
        ds.set_wait_limit(0)
    assert target.check() == ds.ERR_TIMEOUT
    vp.check()
    got = _pass(vp, target)
    assert target.check() == 0 and vp.check() == 0 and torch.equal(got, want)


def test_prompts_longer_than_the_batch_have_room_and_captured_passes_keep_theirs():
    vp, target = _target()
    want = _pass(vp, target).clone()
    out = torch.zeros_like(want)
    vp.assemble(_i32([3, 0, 2, 3]), _i32([1, 2, 3, 4]), _i32([[7, 8, 9]] * R))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        target.logits(out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        target.logits(out)
    small = len(target.works)
    other = VerifyPass(R, G, 2, 4, 2, 64, capacity=64, page_size=16, device=DEV)
    target.vp, kept = other, target.vp
    target.prompt(torch.arange(200, device=DEV), [50, 50, 50, 50])        # more rows than a verify batch
    target.vp = kept
    assert len(target.works) > small and all(w.numel() for w in target.works)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert target.check() == 0 and torch.equal(out, want)
