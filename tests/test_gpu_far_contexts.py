"""cache_attend at the end of the longest context that a table can have, 2^31 - 16 tokens: what the window reaches lies in the
last pages, and the counts of keys and tiles end just below what an int holds."""
import math

import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds
import test_gpu_layer as layer

pytestmark = pytest.mark.gpu
DEV = "cuda"
PAGE, SHIFT = 16, (1 << 31) - 256     # the tokens before those that are there
CTX, EACH = 235, 5                    # of the tokens that are: 240, to the table's end


@pytest.fixture(scope="module")
def wide():
    ds.lib()
    return torch.full((1, (1 << 27) - 1), -1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("window", [1, 64, 100])
@pytest.mark.parametrize("D,dtype,max_q,path", [(64, "f32", 5, "auto"), (128, "bf16", 5, "auto"), (64, "bf16", 512, "auto"),
                                                (128, "bf16", 512, "auto"), (96, "f32", 5, "auto"), (64, "bf16", 5, "cuda")])
def test_the_last_rows_of_the_longest_context(wide, D, dtype, max_q, path, window):
    pool, table, keys, values = layer._filled([CTX], [EACH], PAGE, 1, D, D + window)
    n = (CTX + EACH) // PAGE
    wide[0, SHIFT // PAGE:] = layer._i32(table[0, :n])
    g = torch.Generator(device=DEV).manual_seed(window)
    q = torch.randn((EACH, 2, D), device=DEV, generator=g).to(layer.TYPES[dtype])
    out = ds.cache_attend(q, pool, wide, layer._i32([0, EACH]), layer._i32([SHIFT + CTX]), window=window, max_q=max_q,
                          path=layer.PATHS[path])
    assert ds.check(out["workspace"]) == 0
    want = ref.attend(layer._f64(q), keys, values, [CTX], [0, EACH], 1 / math.sqrt(D), window, 0)
    layer._check_attend(layer._f64(out["out"]), layer._f64(out["lse"]), want, dtype, values, CTX + EACH)
