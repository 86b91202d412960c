"""The rest of the target's pass as it is used: norm, 8-bit head scattered to its rows and the logits' adjustment in place,
on streams and in a graph; rounds with an 8-bit target; a RoundRunner that adjusts what it verifies."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import pass_ref as ref
import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300 import workloads as wl
from speculative_decoding_draft_round_gb300.verify_pass import ToyTarget, VerifyPass

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Chain:
    """Inputs and buffers of norm -> head -> adjustment for R requests of up to S rows."""

    def __init__(self, R, S, K, V, seed):
        rng = self.rng = np.random.default_rng(seed)
        self.R, self.S, self.K, self.V = R, S, K, V
        self.w, self.ws = rng.integers(-127, 128, (V, K)).astype(np.int8), (np.exp(rng.standard_normal(V)) / 500).astype(np.float32)
        self.dw, self.dws = torch.as_tensor(self.w, device=DEV), torch.as_tensor(self.ws, device=DEV)
        self.x, self.res = (torch.empty((R * S, K), device=DEV) for _ in range(2))
        self.place, self.rows, self.keep = _i32(np.zeros(R * S)), _i32([0]), _i32(np.zeros(R))
        self.tokens, self.rep = _i32(np.zeros((R, S - 1))), torch.ones(R, device=DEV)
        self.seen = ds.seen_table(R, V)
        self.target = torch.zeros((R, S, V), device=DEV)
        self.work = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)

    def fill(self):
        rng, R, S, K, V = self.rng, self.R, self.S, self.K, self.V
        self.h = {n: rng.standard_normal((R * S, K)).astype(np.float32) for n in ("x", "res")}
        keep = rng.integers(0, S, R)
        place = np.full(R * S, -1)
        place[:(keep + 1).sum()] = np.concatenate([r * S + np.arange(keep[r] + 1) for r in range(R)])
        self.h.update(keep=keep, place=place, tokens=rng.integers(0, V, (R, S - 1)), rep=(1 + rng.random(R)).astype(np.float32),
                      seen=np.where(rng.random((R, self.seen.shape[1])) < .1, 3, 0).astype(np.int16))
        for n, v in self.h.items():
            t = getattr(self, n)
            t.copy_(torch.as_tensor(v).to(t.dtype))
        self.rows.fill_(int((keep + 1).sum()))

    def run(self, stream=None):
        q = ds.add_norm_quant(self.x, residual=self.res, n_rows=self.rows, workspace=self.work, stream=stream)
        ds.linear_i8(q["codes"], q["scale"], self.dw, self.dws, out_row=self.place, n_rows=self.rows, workspace=self.work,
                     out={"out": self.target}, stream=stream)
        ds.adjust_logits(self.target, seen=self.seen, repetition=self.rep, tokens=self.tokens, keep=self.keep,
                         out={"out": self.target}, workspace=self.work, stream=stream)

    def compare(self):
        h, n = self.h, int((self.h["keep"] + 1).sum())
        _, _, codes, scale = ref.norm_quant(h["x"][:n], h["res"][:n], None, True, 1e-6, False)
        z, _, _ = ref.linear(codes.astype(np.int8), scale.astype(np.float32), self.w, self.ws, None)
        full = np.zeros((self.R * self.S, self.V))
        full[h["place"][:n]] = z
        want, mag = ref.adjust(full.reshape(self.R, self.S, self.V), h["seen"], h["rep"], None, None, h["tokens"], None, None,
                               None, h["keep"])
        live = np.arange(self.S) <= h["keep"][:, None]
        got = self.target.double().cpu().numpy()
        # the scale's 2^-17, twice the rounding of a product and what follows; nothing else is near that
        assert np.all(np.abs(got - want)[live] <= 2.0 ** -16 * mag[live])


@pytest.mark.parametrize("R,S,K,V", [(3, 5, 100, 1003), (20, 17, 512, 2048), (1, 1, 64, 300)])
def test_norm_head_and_adjustment(R, S, K, V):
    c = Chain(R, S, K, V, 1)
    c.fill()
    c.run()
    c.compare()
    assert ds.check(c.work) == 0


def test_in_a_graph_and_on_two_streams():
    a, b = Chain(9, 9, 256, 3000, 2), Chain(5, 17, 384, 1000, 3)
    for c in (a, b):
        c.fill()
        c.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run()
    side = torch.cuda.Stream()
    for _ in range(3):
        a.fill()
        b.fill()
        torch.cuda.synchronize()
        g.replay()
        b.run(side)
        torch.cuda.synchronize()
        a.compare()
        b.compare()
    assert ds.check(a.work) == 0 and ds.check(b.work) == 0


def test_rounds_with_an_eight_bit_target():
    """Draft, verify pass through 8-bit layers and acceptance, twice with the same outcome; the table counts what came out."""
    def rounds():
        R, G, V = 6, 5, 1000
        rnd = wl.make_round("eight_bit_test", R, G, V, 64, 96, "bf16", seed=3, device=DEV, u_std=1.0)
        vp = VerifyPass(R, G, 2, 8, 2, 64, capacity=128, page_size=16, device=DEV)
        target = ToyTarget(vp, V, 128, seed=2, eight_bit=True)
        seen = ds.seen_table(R, V)
        runner = ds.RoundRunner(rnd, adjust=dict(seen=seen, repetition=torch.full((R,), 1.3, device=DEV)))
        lengths = [1, 30, 16, 17, 2, 5]
        g = torch.Generator(device=DEV).manual_seed(1)
        target.prompt(torch.randint(0, V, (sum(lengths),), device=DEV, generator=g), lengths)
        want = np.zeros((R, seen.shape[1]), np.int16)
        history = []
        for i in range(4):
            runner.set_round(i)
            runner.run_draft()
            vp.assemble(runner.cout["keep"], rnd.anchor, runner.sout["tokens"])
            target.logits(rnd.target)
            runner.run_verify()
            assert runner.check() == 0 and vp.check() == 0
            out = {k: v.cpu().numpy() for k, v in runner.results().items() if k in ("accepted", "next_token", "tokens", "keep")}
            assert np.all(out["accepted"] <= out["keep"])
            want = ref.seen_add(want, V, out["tokens"], out["accepted"], out["next_token"], None, False)
            assert np.array_equal(seen.cpu().numpy(), want)
            vp.advance(runner.results()["accepted"])
            rnd.anchor.copy_(runner.results()["next_token"])
            history.append((out["next_token"].tolist(), out["accepted"].tolist()))
        return history

    assert rounds() == rounds()


def test_an_eight_bit_layer_is_near_the_plain_one():
    """The same weights in bf16 and in 8 bits give logits of the same rows that go the same way."""
    R, G, V, width = 4, 3, 512, 256
    outs = []
    for eight in (False, True):
        vp = VerifyPass(R, G, 1, 4, 2, 64, capacity=64, page_size=16, device=DEV)
        target = ToyTarget(vp, V, width, seed=5, eight_bit=eight)
        vp.assemble(_i32([3, 0, 2, 3]), _i32([1, 2, 3, 4]), _i32([[7, 8, 9]] * R))
        out = torch.zeros((R, G + 1, V), dtype=torch.bfloat16, device=DEV)
        target.logits(out)
        assert vp.check() == 0
        outs.append(out.float())
    for r, n in enumerate((4, 1, 3, 4)):
        a, b = outs[0][r, :n], outs[1][r, :n]
        assert torch.nn.functional.cosine_similarity(a, b, dim=-1).min() > 0.9
    assert not outs[1][1, 1:].any()                    # rows behind the last stay as they were


def test_what_a_mask_forbids_does_not_come_out():
    R, G, V = 16, 4, 600
    rnd = wl.make_round("masked", R, G, V, 32, 48, "bf16", seed=4, device=DEV, u_std=1.0)
    allowed = np.zeros((1, V), bool)
    allowed[0, 100:140] = True
    given = rnd.target.clone()
    runner = ds.RoundRunner(rnd, adjust=dict(mask=torch.as_tensor(ref.pack_bits(allowed), device=DEV),
                                             mask_row=_i32(np.zeros((R, G + 1)))))
    plain = ds.RoundRunner(rnd)
    for i in range(5):
        rnd.target.copy_(given)
        runner.set_round(i)
        runner.run()
        assert runner.check() == 0
        out = runner.results()
        nxt, tok, acc = (out[k].cpu().numpy() for k in ("next_token", "tokens", "accepted"))
        assert np.all((nxt >= 100) & (nxt < 140))
        for r in range(R):
            assert np.all((tok[r, :acc[r]] >= 100) & (tok[r, :acc[r]] < 140))
    # a runner without adjustments leaves the target as it is
    rnd.target.copy_(given)
    plain.run()
    assert plain.check() == 0 and torch.equal(rnd.target, given)
