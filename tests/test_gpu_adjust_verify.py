"""Verification right behind the kernel that writes its target gives what it gives once that kernel has ended."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import pass_ref as ref
import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300 import workloads as wl

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _round(R, G, V, dtype):
    rnd = wl.make_round("adjust_verify", R, G, V, 64, 96, dtype, seed=6, device=DEV, u_std=1.0)
    rnd.temperature[::3] = 0.0          # a third of the requests decode greedily
    return rnd


def _verified(rnd, runner, write, apart):
    """The outcome of rounds whose target write() makes, with the kernels' ends awaited between them or not."""
    got = []
    for i in range(4):
        runner.set_round(i)
        runner.run_draft()
        torch.cuda.synchronize()
        write()
        if apart:
            torch.cuda.synchronize()
        ds._call("dspark_verify", ds.C.byref(runner.va), runner.vws.data_ptr(), runner.vws.numel(), ds._stream(None))
        torch.cuda.synchronize()
        got.append([runner.vout[k].cpu().numpy().copy() for k in ("accepted", "next_token", "resampled")])
    assert runner.check() == 0
    return got


@pytest.mark.parametrize("R,G,V,dtype", [(64, 4, 151936, "bf16"), (24, 2, 100003, "bf16"), (24, 2, 65536, "f32")])
def test_behind_an_adjustment_in_place(R, G, V, dtype):
    """A mask leaves the last ids only: a row read too early holds others."""
    rnd = _round(R, G, V, dtype)
    given = rnd.target.clone()
    allowed = np.zeros((1, V), bool)
    allowed[0, V - 200:V - 50] = True
    mask = torch.as_tensor(ref.pack_bits(allowed), device=DEV)
    state = torch.zeros((R, G + 1), dtype=torch.int32, device=DEV)
    runner = ds.RoundRunner(rnd)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out = {"out": rnd.target}

    def write():
        rnd.target.copy_(given)
        ds.adjust_logits(rnd.target, mask=mask, mask_row=state, out=out, workspace=ws)

    apart, together = (_verified(rnd, runner, write, x) for x in (True, False))
    for a, b in zip(apart, together):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
        assert np.all((b[1] >= V - 200) & (b[1] < V - 50))
    assert ds.check(ws) == 0


@pytest.mark.parametrize("path", [ds.PATH_CUDA_CORE, ds.PATH_TENSOR_CORE])
def test_behind_the_head(path):
    """The head's product straight into the target, another one each time."""
    R, G, V, K = 32, 3, 20000, 256
    rnd = _round(R, G, V, "bf16")
    runner = ds.RoundRunner(rnd)
    g = torch.Generator(device=DEV).manual_seed(1)
    w = ds.add_norm_quant(torch.randn((V, K), device=DEV, generator=g), norm=False)
    x = ds.add_norm_quant(torch.randn((R * (G + 1), K), device=DEV, generator=g), norm=False)
    scale = x["scale"].clone()
    a, out = ds.linear_i8_args(x["codes"], scale, w["codes"], w["scale"], path=path, out={"out": rnd.target})
    work = torch.zeros(ds.workspace_bytes("linear_i8", a), dtype=torch.uint8, device=DEV)

    def write():
        # what was there before would come out otherwise: the largest logits at the lowest ids
        rnd.target.zero_()
        rnd.target[..., :7] = 1000.0
        ds.linear_i8(x["codes"], scale, w["codes"], w["scale"], path=path, out=out, workspace=work)

    apart, together = (_verified(rnd, runner, write, x) for x in (True, False))
    for a, b in zip(apart, together):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))
    assert ds.check(work) == 0


def test_rounds_that_adjust_are_the_same_in_a_row():
    """RoundRunner(adjust=...) with nothing awaited between its kernels, against the same rounds in steps."""
    R, G, V = 32, 4, 151936

    def rounds(apart):
        rnd = _round(R, G, V, "bf16")
        given = rnd.target.clone()
        seen = ds.seen_table(R, V)
        runner = ds.RoundRunner(rnd, adjust=dict(seen=seen, repetition=torch.full((R,), 1.7, device=DEV),
                                                 frequency=torch.full((R,), 0.5, device=DEV)))
        got = []
        for i in range(5):
            rnd.target.copy_(given)
            runner.set_round(i)
            if apart:
                runner.run_draft()
                torch.cuda.synchronize()
                ds._call("dspark_adjust_logits", ds.C.byref(runner.ja), runner.jws.data_ptr(), 256, ds._stream(None))
                torch.cuda.synchronize()
                ds._call("dspark_verify", ds.C.byref(runner.va), runner.vws.data_ptr(), runner.vws.numel(), ds._stream(None))
                torch.cuda.synchronize()
                ds._call("dspark_seen_add", ds.C.byref(runner.na), runner.jws.data_ptr(), 256, ds._stream(None))
            else:
                runner.run()
            got.append([runner.results()[k].cpu().numpy().copy() for k in ("accepted", "next_token", "resampled")])
            rnd.anchor.copy_(runner.results()["next_token"])
        assert runner.check() == 0
        return got + [[seen.cpu().numpy()]]

    for a, b in zip(rounds(True), rounds(False)):
        assert all(np.array_equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("V", [600, 5003])
def test_masks_that_leave_nothing(V):
    """Token 0 comes out, recorded where the request samples; the other requests are not touched by it."""
    R, G = 8, 3
    for greedy in (False, True):
        got = []
        for empty in (False, True):
            rnd = wl.make_round("nothing_left", R, G, V, 32, 48, "bf16", seed=4, device=DEV, u_std=1.0)
            rnd.temperature.fill_(0.0 if greedy else 1.0)
            mask = torch.zeros((2, -(-V // 32)), dtype=torch.int32, device=DEV)
            mask[1] = -1
            state = torch.ones((R, G + 1), dtype=torch.int32, device=DEV)
            if empty:
                state[0], state[3, 1:] = 0, 0
            runner = ds.RoundRunner(rnd, adjust=dict(mask=mask, mask_row=state))
            runner.run()
            assert runner.check() == (ds.ERR_DEVICE_INPUT if empty and not greedy else 0)
            got.append([runner.results()[k].cpu().numpy().copy() for k in ("accepted", "next_token")])
        (_, plain), (accepted, masked) = got
        assert accepted[0] == 0 and masked[0] == 0
        others = [1, 2, 4, 5, 6, 7]
        assert np.array_equal(plain[others], masked[others]) and 0 <= masked[3] < V


@pytest.mark.parametrize("path", [ds.PATH_AUTO, ds.PATH_CUDA_CORE, ds.PATH_RESIDENT])
def test_a_draft_right_behind_the_adjustment_of_its_logits(path):
    """The backbone's logits adjusted in place and drafted from at once, and with the adjustment's end awaited."""
    R, G, V = 64, 4, 65536
    rnd = wl.make_round("adjust_draft", R, G, V, 256, 96, "bf16", seed=6, device=DEV, u_std=1.0)
    given = rnd.U.clone()
    allowed = np.zeros((1, V), bool)
    allowed[0, V - 200:V - 50] = True
    mask = torch.as_tensor(ref.pack_bits(allowed), device=DEV)
    state = torch.zeros((R, G), dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    runner = ds.RoundRunner(rnd, path=path)
    got = []
    for apart in (True, False):
        for i in range(3):
            runner.set_round(i)
            rnd.U.copy_(given)
            torch.cuda.synchronize()
            ds.adjust_logits(rnd.U, mask=mask, mask_row=state, out={"out": rnd.U}, workspace=ws)
            if apart:
                torch.cuda.synchronize()
            runner.run_draft()
            torch.cuda.synchronize()
            got.append({k: runner.sout[k].cpu().numpy().copy() for k in ("tokens", "draft_lse", "draft_logit", "surv")})
    assert runner.check() == 0 and ds.check(ws) == 0
    for a, b in zip(got[:3], got[3:]):
        assert all(np.array_equal(a[k], b[k]) for k in a)
        assert np.all((b["tokens"] >= V - 200) & (b["tokens"] < V - 50))
