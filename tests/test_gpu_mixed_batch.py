"""cache_attend for a long prompt among many single rows, in tables far wider than their contexts: the matrix kernels take
it, and offsets that repeat rows more often than their counters hold leave no row computed."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds
import test_gpu_layer as layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
R, LONG, PAGE, WIDTH = 2047, 512, 64, 16384   # 2^20 tokens of room a request


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ds.lib()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_long_prompt_among_single_rows(dtype):
    rng = np.random.default_rng(2)
    ctx, each = rng.integers(0, 40, R).tolist(), [1] * R
    each[R // 3], each[5] = LONG, 0
    D, Hq, Hkv = 64, 4, 4
    pool, narrow, keys, values = layer._filled(ctx, each, PAGE, Hkv, D, 11)
    table = torch.full((R, WIDTH), -1, dtype=torch.int32, device=DEV)
    table[:, :narrow.shape[1]] = layer._i32(narrow)
    _, _, offsets = layer._flat(each)
    g = torch.Generator(device=DEV).manual_seed(3)
    q = torch.randn((int(offsets[-1]), Hq, D), device=DEV, generator=g).to(layer.TYPES[dtype])
    out = ds.cache_attend(q, pool, table, layer._i32(offsets), layer._i32(ctx), max_q=LONG, path=ds.PATH_TENSOR_CORE)
    assert ds.check(out["workspace"]) == 0
    want = ref.attend(layer._f64(q), keys, values, ctx, offsets, 1 / math.sqrt(D), 0, 0)
    layer._check_attend(layer._f64(out["out"]), layer._f64(out["lse"]), want, dtype, values, 40 + LONG)


@pytest.mark.parametrize("dtype,Hq", [("f32", 4), ("bf16", 128)])   # blocks of 16 rows, and of 128
def test_offsets_that_repeat_rows(dtype, Hq):
    """1024 requests claim the same 512 rows after a million keys: more than 2^32 tiles."""
    T, D, Hkv = LONG, 64, 4
    q = torch.ones((T, Hq, D), device=DEV, dtype=layer.TYPES[dtype])
    pool = ds.cache_pool(1, Hkv, PAGE, D)
    table = torch.zeros((R, WIDTH), dtype=torch.int32, device=DEV)
    offsets = np.zeros(R + 1, np.int64)
    offsets[1::2] = T
    ctx = np.full(R, WIDTH * PAGE - T)
    out = {"out": torch.full_like(q, 7), "lse": torch.full((T, Hq), 7.0, device=DEV)}
    got = ds.cache_attend(q, pool, table, layer._i32(offsets), layer._i32(ctx), max_q=LONG, path=ds.PATH_TENSOR_CORE, out=out)
    assert ds.check(got["workspace"]) == ds.ERR_DEVICE_INPUT
    assert torch.all(got["out"] == 7) and torch.all(got["lse"] == 7)
