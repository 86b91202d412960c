"""Channels from rot on pass qk_norm_rope as they are, whatever their neighbours hold: an infinity stays in its channel (or,
turned, in its pair)."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_draft_round_gb300 as ds

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 0), (64, 2), (64, 10), (64, 16), (128, 46), (256, 250), (24, 14), (63 * 2, 46)])
def test_an_infinity_stays_in_its_channel(D, rot, inter, dtype):
    ds.lib()
    T, pairs = 3, rot // 2
    g = torch.Generator(device=DEV).manual_seed(D + rot)
    x = torch.randn((T, 2, D), device=DEV, generator=g).to(dtype)
    where = [c for c in (rot, rot + 1, rot + 5, D - 1, 1) if c < D]
    freq = ds.rope_frequencies(rot) if rot else None
    pos = torch.tensor([0, 1, 77], dtype=torch.int32, device=DEV)
    run = lambda y: ds.qk_norm_rope(y, y[:, :1], freq, pos, norm=False, interleaved=inter)["q"]
    clean = run(x)
    assert torch.equal(clean[..., rot:], x[..., rot:])
    for c in where:
        y = x.clone()
        y[:, 1, c] = float("inf")
        out = run(y)
        mine = {c} if c >= rot else {c, c ^ 1} if inter else {c % pairs, c % pairs + pairs}
        rest = [k for k in range(D) if k not in mine]
        assert torch.equal(out[:, 0], clean[:, 0])
        assert torch.equal(out[:, 1, rest], clean[:, 1, rest]), c
        assert not torch.isfinite(out[:, 1, c]).any() and (c < rot or torch.isinf(out[:, 1, c]).all())
