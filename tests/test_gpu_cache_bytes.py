"""The cache's bytes for batches of thousands of tokens, where a CTA has several: what cache_append writes against blocks
packed on the host, and what cache_read makes of blocks that the host packed. And attention with heads of 32, 96 and 256,
which have no matrix kernel, in windows, other pages and prompts."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds
import test_gpu_layer as layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ds.lib()


def _batch(T, page, seed, pad=0.05):
    """T flat tokens of 7 requests in any order, some of them padding, in scattered pages: request, position, contexts,
    table, pages, and for each token its page and slot."""
    rng = np.random.default_rng(seed)
    R = 7
    ctx = rng.integers(0, 3 * page, R)
    request = rng.integers(0, R, T)
    request[rng.random(T) < pad] = -rng.integers(1, 5)
    position = np.zeros(T, np.int64)
    for r in range(R):
        mine = np.flatnonzero(request == r)
        position[mine] = rng.permutation(len(mine))
    width = -(-int((ctx + np.bincount(request[request >= 0], minlength=R)).max()) // page)
    table = rng.permutation(R * width + 3)[:R * width].reshape(R, width)
    at = np.where(request >= 0, ctx[request.clip(0)] + position, 0)
    return request, position, ctx, table, R * width + 3, table[request.clip(0), at // page], at % page


def _pack(blocks, x, where, slot, page, half):
    """Rows x [N][Hkv][D] into the blocks [pages][Hkv][bytes] of their pages."""
    N, H, D = x.shape
    vc, ks, vs, _ = ref.block_parts(page, D)
    s = ref.scales_of(x)
    u = (ref.codes_of(x, s) + 8).astype(np.uint8)
    n, h = np.arange(N)[:, None], np.arange(H)[None, :]
    first = (0 if half == 0 else vc) + slot * (D // 2)
    blocks[where[n][..., None], h[..., None], first[:, None, None] + np.arange(D // 2)] = u[..., 0::2] | u[..., 1::2] << 4
    G = D // 32
    g = np.arange(G)
    to = ks + 2 * (slot[:, None] * G + g) if half == 0 else vs + 2 * (((slot // 16)[:, None] * G + g) * 16 + (slot % 16)[:, None])
    raw = s.astype(np.float16).view(np.uint8).reshape(N, H, G, 2)
    blocks[where[n][..., None, None], h[..., None, None], (to[:, :, None] + np.arange(2))[:, None]] = raw


SIZES = [(1217, 64, 3, 16), (5003, 64, 3, 16), (60001, 32, 1, 256), (5003, 128, 8, 48), (20011, 96, 5, 32), (9001, 256, 2, 64),
         (3001, 64, 40, 16)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,Hkv,page", SIZES)
def test_append_of_many_tokens(T, D, Hkv, page, dtype):
    request, position, ctx, table, n_pages, where, slot = _batch(T, page, T)
    g = torch.Generator(device=DEV).manual_seed(T)
    rows = torch.randn((T, 2 * Hkv * D), device=DEV, generator=g)
    rows = (rows * torch.exp(torch.empty((T, 1), device=DEV).uniform_(-6, 6, generator=g))).to(layer.TYPES[dtype])
    k, v = rows[:, :Hkv * D].unflatten(1, (Hkv, D)), rows[:, Hkv * D:].unflatten(1, (Hkv, D))
    pool = ds.cache_pool(n_pages, Hkv, page, D)
    pool.fill_(0xA5)
    out = ds.cache_append(k, v, pool, *(layer._i32(x) for x in (table, request, position, ctx)))
    assert ds.check(out["workspace"]) == 0
    want = np.full(tuple(pool.shape), 0xA5, np.uint8)
    live = request >= 0
    for half, x in ((0, k), (1, v)):
        _pack(want, x.float().cpu().numpy()[live], where[live], slot[live], page, half)
    got = pool.cpu().numpy()
    assert np.array_equal(got, want), np.argwhere(got != want)[:5]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,D,Hkv,page", SIZES)
def test_read_of_many_tokens(T, D, Hkv, page, dtype):
    request, position, ctx, table, n_pages, where, slot = _batch(T, page, T + 1)
    rng = np.random.default_rng(T)
    vc, ks, _, end = ref.block_parts(page, D)
    blocks = rng.integers(0, 256, (n_pages, Hkv, end), dtype=np.uint8)
    scales = (rng.random((n_pages, Hkv, (end - ks) // 2)) * np.exp2(rng.integers(-20, 10, (n_pages, Hkv, 1)))).astype(np.float16)
    blocks[..., ks:] = scales.view(np.uint8)
    # the values of all of it, by page and slot
    G = D // 32
    u = [blocks[..., a:a + vc].reshape(n_pages, Hkv, page, D // 2) for a in (0, vc)]
    s = [scales[..., :page * G].reshape(n_pages, Hkv, page, G),
         scales[..., page * G:].reshape(n_pages, Hkv, page // 16, G, 16).swapaxes(3, 4).reshape(n_pages, Hkv, page, G)]
    back = ds.cache_read(torch.as_tensor(blocks, device=DEV), *(layer._i32(x) for x in (table, request, position, ctx)), D=D,
                         dtype=layer.TYPES[dtype])
    assert ds.check(back["workspace"]) == 0
    for half, name in enumerate("kv"):
        code = np.stack([u[half] & 15, u[half] >> 4], -1).reshape(n_pages, Hkv, page, D).astype(np.float32) - 8
        value = code * np.repeat(s[half].astype(np.float32), 32, -1)        # exact in fp32
        want = torch.as_tensor(value[where, :, slot]).to(layer.TYPES[dtype])
        want[request < 0] = 0
        assert torch.equal(back[name].cpu(), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,Hq,Hkv", [(32, 6, 2), (96, 5, 1), (256, 4, 2)])
@pytest.mark.parametrize("page,window,sinks", [(16, 17, 5), (48, 100, 0), (256, 64, 130), (80, 0, 0)])
def test_heads_without_a_matrix_kernel(D, Hq, Hkv, page, window, sinks, dtype):
    layer._attend_case([0, 3, page, 700], [5, 0, 17, 9], Hq, Hkv, D, page, dtype, window, sinks, seed=D + page)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [32, 96, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_prompts_of_heads_without_a_matrix_kernel(D, window, sinks, dtype):
    layer._attend_case([130, 5], [211, 1], 4, 2, D, 64, dtype, window, sinks, seed=D)
