"""VerifyPass: rounds of random projections through the pass against the 64-bit formula on the history that was
accepted, and whole rounds of drafting and verification with a small random target."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds
import test_gpu_layer as layer
from speculative_decoding_draft_round_gb300 import workloads as wl
from speculative_decoding_draft_round_gb300.verify_pass import ToyTarget, VerifyPass

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ds.lib()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
@pytest.mark.parametrize("R,G,Hq,Hkv,D", [(3, 4, 4, 2, 64), (2, 16, 8, 2, 128)])
def test_rounds_of_a_pass(R, G, Hq, Hkv, D, window, sinks, dtype):
    """Each round's rows attend to the tokens accepted before and to their own: rejected ones leave no trace."""
    layers, rng = 2, np.random.default_rng(R + window)
    vp = VerifyPass(R, G, layers, Hq, Hkv, D, capacity=4 * (G + 1) + 33, page_size=16, dtype=layer.TYPES[dtype],
                    norm=False, window=window, sinks=sinks, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    past = [33, 0, 7][:R]
    request, position, offsets = layer._flat(past)
    for l in range(layers):
        qkv = torch.randn((len(request), vp.qkv.shape[1]), device=DEV, generator=g).to(vp.qkv.dtype)
        vp.prompt(l, qkv, layer._i32(request), layer._i32(position), layer._i32(offsets), max(past))
    vp.advance_by(layer._i32(past))
    for _ in range(3):
        keep = rng.integers(0, G + 1, R)
        tokens = layer._i32(rng.integers(0, 99, (R, G)))
        b = vp.assemble(layer._i32(keep), tokens[:, 0].contiguous(), tokens)
        offsets = b["offsets"].cpu().numpy()
        assert offsets.tolist() == np.concatenate([[0], np.cumsum(keep + 1)]).tolist()
        ctx = vp.ctx_len.cpu().numpy()
        for l in range(layers):
            vp.qkv.normal_(generator=g)
            out = vp.layer(l).clone()
            # all that is in the cache for these queries, as the values it stands for
            n = (ctx + keep + 1).tolist()
            rq, ps, _ = layer._flat(n)
            kv = ds.cache_read(vp.pools[l], vp.table, layer._i32(rq), layer._i32(ps), layer._i32(np.zeros(R)), D=D,
                               dtype=torch.float32)
            edge = np.concatenate([[0], np.cumsum(n)])
            keys, values = ([layer._f64(kv[x][edge[r]:edge[r + 1]]) for r in range(R)] for x in "kv")
            want = ref.attend(layer._f64(vp.turned["q"]), keys, values, ctx.tolist(), offsets, 1 / math.sqrt(D),
                              window, sinks)
            layer._check_attend(layer._f64(out), want[1], want, dtype, values, max(n))
            # this round's own rows are the batch's, after the tokens that were accepted before
            own = np.concatenate([np.arange(edge[r] + ctx[r], edge[r + 1]) for r in range(R)])
            again = ds.cache_pool(len(own), Hkv, 16, D)
            one = (again, layer._i32(np.arange(len(own))[:, None]), layer._i32(np.arange(len(own))),
                   layer._i32(np.zeros(len(own))), layer._i32(np.zeros(len(own))))
            v = vp.qkv[:len(own)].unflatten(1, (-1, D))[:, Hq + Hkv:]
            ds.cache_append(vp.turned["k"][:len(own)], v, *one)
            alone = ds.cache_read(*one, D=D, dtype=torch.float32)
            for x in "kv":
                assert torch.equal(kv[x][torch.as_tensor(own, device=DEV)], alone[x])
        assert vp.check() == 0
        accepted = rng.integers(0, keep + 1)
        vp.advance(layer._i32(accepted))
        assert vp.ctx_len.cpu().tolist() == (ctx + accepted + 1).tolist()


def test_a_prompt_in_pieces_is_the_prompt():
    """Row by row, the outputs of a prompt that comes in two pieces are close to those of the whole one."""
    R, Hq, Hkv, D = 2, 8, 2, 64
    n = np.array([150, 41])
    g = torch.Generator(device=DEV).manual_seed(8)
    make = lambda: VerifyPass(R, 4, 1, Hq, Hkv, D, capacity=256, device=DEV)
    a, b = make(), make()
    qkv = torch.randn((int(n.sum()), a.qkv.shape[1]), device=DEV, generator=g).bfloat16()
    request, position, offsets = layer._flat(n.tolist())
    whole = a.prompt(0, qkv, layer._i32(request), layer._i32(position), layer._i32(offsets), int(n.max()))
    got = torch.empty_like(whole)
    done = np.zeros(2, dtype=int)
    for piece in (np.array([64, 40]), np.array([86, 1])):
        rows = np.concatenate([offsets[r] + done[r] + np.arange(piece[r]) for r in range(R)])
        rq, ps, of = layer._flat(piece.tolist())
        at = torch.as_tensor(rows, device=DEV)
        got[at] = b.prompt(0, qkv[at], layer._i32(rq), layer._i32(ps), layer._i32(of), int(piece.max()))
        b.advance_by(layer._i32(piece))
        done += piece
    assert a.check() == 0 and b.check() == 0
    assert torch.equal(a.pools[0], b.pools[0])
    # two results within one rounding to bf16 and a weight's rounding to fp16 each of the same sums
    err, top = (got.float() - whole.float()).abs(), 6.0
    assert float(whole.abs().max()) <= top and float(err.max()) <= 2 * (2 * 2.0 ** -11 + 2.0 ** -8) * top


def test_rounds_with_a_target():
    """Draft, verify pass and acceptance for some rounds, twice with the same outcome; contexts grow as accepted."""
    def rounds():
        R, G, V = 6, 5, 1000
        rnd = wl.make_round("verify_pass_test", R, G, V, 64, 96, "bf16", seed=3, device=DEV, u_std=1.0)
        runner = ds.RoundRunner(rnd)
        vp = VerifyPass(R, G, 2, 8, 2, 64, capacity=128, page_size=16, device=DEV)
        target = ToyTarget(vp, V, 128, seed=2)
        lengths = [1, 30, 16, 17, 2, 5]
        g = torch.Generator(device=DEV).manual_seed(1)
        target.prompt(torch.randint(0, V, (sum(lengths),), device=DEV, generator=g), lengths)
        ctx, history = np.array(lengths), []
        for i in range(4):
            runner.set_round(i)
            runner.run_draft()
            vp.assemble(runner.cout["keep"], rnd.anchor, runner.sout["tokens"])
            target.logits(rnd.target)
            runner.run_verify()
            assert runner.check() == 0 and vp.check() == 0
            out = runner.results()
            assert torch.isfinite(rnd.target.float()).all()
            accepted = out["accepted"].cpu().numpy()
            assert np.all(accepted <= out["keep"].cpu().numpy())
            vp.advance(out["accepted"])
            ctx = ctx + accepted + 1
            assert vp.ctx_len.cpu().tolist() == ctx.tolist()
            rnd.anchor.copy_(out["next_token"])
            history.append((out["next_token"].cpu().tolist(), accepted.tolist()))
        return history

    assert rounds() == rounds()


def test_a_full_cache_is_reported():
    """Tokens past a request's pages are not written anywhere, and the status says so."""
    vp = VerifyPass(2, 3, 1, 2, 1, 64, capacity=16, page_size=16, device=DEV)
    vp.advance_by(layer._i32([14, 0]))
    tokens = layer._i32(np.zeros((2, 3)))
    vp.assemble(layer._i32([3, 3]), tokens[:, 0].contiguous(), tokens)
    vp.qkv.normal_()
    vp.layer(0)
    assert vp.check() == ds.ERR_DEVICE_INPUT
