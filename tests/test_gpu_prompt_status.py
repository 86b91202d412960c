"""What VerifyPass.check says of prompts: the status of their attention, which has a workspace apart from the other calls',
is kept until it is asked for, on every stream and in graphs."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds
import test_gpu_layer as layer
from speculative_decoding_draft_round_gb300.verify_pass import ToyTarget, VerifyPass

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ds.lib()


def _prompt(n, dtype=torch.bfloat16, D=64, **kw):
    vp = VerifyPass(len(n), 4, 1, 8, 2, D, capacity=256, dtype=dtype, device=DEV, **kw)
    request, position, offsets = (layer._i32(x) for x in layer._flat(n))
    g = torch.Generator(device=DEV).manual_seed(len(n))
    qkv = torch.randn((sum(n), vp.qkv.shape[1]), device=DEV, generator=g).to(dtype)
    return vp, qkv, lambda max_q, **s: vp.prompt(0, qkv, request, position, offsets, max_q, **s)


# 4 rows a key head take the kernel of few rows, 100 that of many, heads of 96 that of CUDA cores
@pytest.mark.parametrize("n,D", [([3, 1], 64), ([100, 9], 64), ([100, 9], 128), ([5, 2], 96)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_max_q_are_reported(n, D, dtype):
    vp, _, prompt = _prompt(n, dtype, D)
    prompt(n[0])
    assert vp.check() == 0
    prompt(n[0] - 1)
    prompt(n[0])                                     # a good call after it does not hide it
    assert vp.check() == ds.ERR_DEVICE_INPUT
    assert vp.check() == 0


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("n", [[3, 1], [100, 9]])
def test_a_nan_in_the_queries_is_reported(n, norm):
    vp, qkv, prompt = _prompt(n, norm=norm)
    qkv[1, 70] = float("nan")                        # in the second query head
    out = prompt(n[0])
    assert vp.check() == ds.ERR_NONFINITE_INPUT
    assert torch.isnan(out[1, 1]).all() and not torch.isnan(out[0]).any()


def test_prompts_on_two_streams_have_workspaces_of_their_own():
    vp, _, prompt = _prompt([100, 9])
    want = prompt(100).clone()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    short = prompt(99, stream=a)
    full = prompt(100, stream=b)
    assert vp.check() == ds.ERR_DEVICE_INPUT         # waits for both
    assert torch.equal(full, want) and torch.equal(short[:99], want[:99])
    assert len({w.data_ptr() for w in vp._prompt_ws.values()}) == 3


def test_prompts_of_one_stream_share_a_workspace():
    vp, _, prompt = _prompt([100, 9])
    first = prompt(100).clone()
    for _ in range(3):
        assert torch.equal(prompt(100), first)
    assert len(vp._prompt_ws) == 1 and vp.check() == 0


def test_status_of_a_captured_prompt():
    """Each replay's status is there until the next check; its inputs are the buffers it was captured with."""
    vp, qkv, prompt = _prompt([100, 9], norm=False)
    want = prompt(100).clone()
    assert vp.check() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = [prompt(100) for _ in range(2)]
    qkv[0, 3] = float("inf")
    g.replay()
    assert vp.check() == ds.ERR_NONFINITE_INPUT
    qkv[0, 3] = 1.0
    g.replay()
    assert vp.check() == 0
    rows = np.r_[100:109]                            # of the request whose rows are as they were
    for o in out:
        assert torch.equal(o[rows], want[rows])


def test_a_prompt_of_no_rows():
    """Requests that start with nothing: no row a request, alone or as a model's prompt."""
    vp, qkv, _ = _prompt([3, 1])
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    out = vp.prompt(0, qkv[:0], none, none, torch.zeros(3, dtype=torch.int32, device=DEV), 0)
    assert out.shape == (0, 8, 64) and vp.check() == 0
    target = ToyTarget(vp, 50, 32)
    target.prompt(none, [0, 0])
    assert vp.check() == 0 and vp.ctx_len.tolist() == [0, 0]
