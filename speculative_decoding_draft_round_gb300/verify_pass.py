"""The verify batch through a target model's attention: assemble -> (qk_norm_rope -> cache_append -> cache_attend)
for every layer, and the caches moved on by what was accepted.

VerifyPass keeps the paged 4-bit caches of all layers and the calls' arguments, outputs and workspace, as
RoundRunner does for the draft round. A round is

    runner.run_draft()                      # tokens, keep
    batch = vp.assemble(keep, anchor, tokens)
    for l in range(layers):
        vp.qkv.copy_(...)                   # the layer's projection of the flat tokens, [T][(Hq + 2 Hkv) D]
        attended = vp.layer(l)              # [T][Hq][D]
        ...                                 # its output projection and the rest of the layer
    runner.run_verify()                     # accepted
    vp.advance(accepted)

Rows of rejected tokens stay where they are: the next round's tokens are appended at ctx_len and so over them, and no
query looks past its own position. ToyTarget and main() below run rounds of a small random target that way.
"""
from __future__ import annotations

import torch

from . import (_launch, _on, assemble, assemble_args, cache_append, cache_append_args, cache_attend_args, cache_pool, check,
               lib, qk_norm_rope, qk_norm_rope_args, rope_frequencies, workspace_bytes)


class VerifyPass:
    """R requests of at most gamma_max drafted tokens, `capacity` tokens of cache each. gains: [layers] pairs
    (q_gain, k_gain) of fp32 [D] tensors, or None for norms without them; norm=False leaves the heads as they are."""

    def __init__(self, R, gamma_max, layers, Hq, Hkv, D, *, capacity, page_size=32, dtype=torch.bfloat16, rot=None,
                 base=10000.0, interleaved=False, norm=True, gains=None, eps=1e-6, window=0, sinks=0, device="cuda"):
        self.R, self.gamma_max, self.layers, self.Hq, self.Hkv, self.D = R, gamma_max, layers, Hq, Hkv, D
        self.T = T = R * (gamma_max + 1)
        self.window, self.sinks = window, sinks
        width = -(-capacity // page_size)
        self.capacity = width * page_size
        i32 = dict(dtype=torch.int32, device=device)
        self.pools = [cache_pool(R * width, Hkv, page_size, D, device=device) for _ in range(layers)]
        self.table = torch.arange(R * width, **i32).view(R, width)
        self.ctx_len = torch.zeros(R, **i32)
        self.batch = {n: torch.full((T,), -1, **i32) for n in ("flat_tokens", "flat_request", "flat_position")}
        self.batch["offsets"] = torch.zeros(R + 1, **i32)
        self.qkv = torch.zeros((T, (Hq + 2 * Hkv) * D), dtype=dtype, device=device)
        self.turned = {"q": torch.empty((T, Hq, D), dtype=dtype, device=device),
                       "k": torch.empty((T, Hkv, D), dtype=dtype, device=device)}
        self.attended = {"out": torch.empty((T, Hq, D), dtype=dtype, device=device)}
        freq = rope_frequencies(D if rot is None else rot, base, device=device)
        gains = gains or [(None, None)] * layers
        self._rope = [dict(freq=freq, ctx_len=self.ctx_len, q_gain=g, k_gain=h, eps=eps, norm=norm,
                           interleaved=interleaved) for g, h in gains]
        b = self.batch
        q, k, v = self._heads(self.qkv)
        self._calls = []
        for l, pool in enumerate(self.pools):
            at = (pool, self.table, b["flat_request"], b["flat_position"], self.ctx_len)
            self._calls.append((
                qk_norm_rope_args(q, k, position=b["flat_position"], request=b["flat_request"], out=self.turned,
                                  **self._rope[l])[0],
                cache_append_args(self.turned["k"], v, *at),
                cache_attend_args(self.turned["q"], pool, self.table, b["offsets"], self.ctx_len, window=window,
                                  sinks=sinks, max_q=gamma_max + 1, out=self.attended)[0]))
        size = workspace_bytes("assemble", assemble_args(self.ctx_len, self.ctx_len, torch.zeros((R, gamma_max), **i32),
                                                         out=self.batch)[0])
        self.batch["workspace"] = torch.zeros(size, dtype=torch.uint8, device=device)
        self.ws = torch.zeros(max(workspace_bytes("cache_attend", self._calls[0][2]), 256), dtype=torch.uint8,
                              device=device)
        self._prompt_ws = {}                        # of the prompts' attention, by stream and size
        self._captured = torch.zeros(1, **i32)      # the status of prompts in graphs

    def _heads(self, qkv):
        """Views of the projection's rows: q [T][Hq][D], k and v [T][Hkv][D]."""
        D = self.D
        return (x.unflatten(1, (-1, D)) for x in qkv.split([self.Hq * D, self.Hkv * D, self.Hkv * D], 1))

    def assemble(self, keep, anchor, tokens, stream=None):
        """The admitted prefixes as this pass's flat batch; returns it (flat_tokens, flat_request, flat_position,
        offsets)."""
        assemble(keep, anchor, tokens, out=self.batch, workspace=self.batch["workspace"], stream=stream)
        return self.batch

    def layer(self, l, stream=None):
        """Layer l's attention for the batch, from self.qkv; returns [T][Hq][D] (zeros in padding), valid until
        the next layer's."""
        a, b, c = self._calls[l]
        _launch("dspark_qk_norm_rope", lib().dspark_qk_norm_rope, a, self.ws, stream)
        _launch("dspark_cache_append", lib().dspark_cache_append, b, self.ws, stream)
        _launch("dspark_cache_attend", lib().dspark_cache_attend, c, self.ws, stream)
        return self.attended["out"]

    def prompt(self, l, qkv, request, position, offsets, max_q, stream=None):
        """The same for the rows of prompts: qkv [T][(Hq + 2 Hkv) D] of any T, laid out as request, position [T] and
        offsets [R + 1] (int32, on the device), at most max_q rows a request (0 where none has a row). A prompt that
        comes in pieces is moved on with advance_by between them."""
        q, k, v = self._heads(qkv)
        turned = qk_norm_rope(q, k, position=position, request=request, workspace=self.ws, stream=stream,
                              **self._rope[l])
        cache_append(turned["k"], v, self.pools[l], self.table, request, position, self.ctx_len, workspace=self.ws,
                     stream=stream)
        with _on(stream):
            a, out = cache_attend_args(turned["q"], self.pools[l], self.table, offsets, self.ctx_len, window=self.window,
                                       sinks=self.sinks, max_q=max(1, max_q), lse=False)
            ws = self._prompt_workspace(a)
            _launch("dspark_cache_attend", lib().dspark_cache_attend, a, ws, None)
            if torch.cuda.is_current_stream_capturing():
                torch.maximum(self._captured, ws[:4].view(torch.int32), out=self._captured)
        return out["out"]

    def _prompt_workspace(self, args):
        """The current stream's workspace for a prompt's attention. Its status word has to last until check(), so
        workspaces stay: one for each size (a kernel has one size, whatever the prompt) and stream (prompts on two
        streams may run at the same time). A captured call has one of the graph's own, and its status is kept apart."""
        size, here = max(workspace_bytes("cache_attend", args), 256), torch.cuda.current_stream(self.qkv.device)
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(size, dtype=torch.uint8, device=self.qkv.device)
        ws = self._prompt_ws.get((here, size))
        if ws is None:
            ws = self._prompt_ws[here, size] = torch.zeros(size, dtype=torch.uint8, device=self.qkv.device)
        return ws

    def advance_by(self, tokens, stream=None):
        """ctx_len += tokens ([R] int32 on the device)."""
        with _on(stream):
            self.ctx_len += tokens

    def advance(self, accepted, stream=None):
        """After verify: the anchor and the accepted tokens are in the caches."""
        with _on(stream):
            self.ctx_len += accepted + 1

    def check(self, stream=None) -> int:
        """The first device status recorded since the last check, the prompts' among them. Waits for `stream`, by
        default the current one, where graphs with prompts have been replayed, and for the prompts' own streams."""
        prompts = [check(w, s) for (s, _), w in self._prompt_ws.items()]
        codes = [check(w, stream) for w in (self.ws, self.batch["workspace"], self._captured)]
        return next((c for c in codes + prompts if c), 0)


class ToyTarget:
    """A small random target model around VerifyPass: embedding, layers of attention with a residual, logits."""

    def __init__(self, vp, V, width, *, seed=0):
        g = torch.Generator(device=vp.qkv.device).manual_seed(seed)
        dt, dev = vp.qkv.dtype, vp.qkv.device
        draw = lambda n, m: (torch.randn((n, m), device=dev, generator=g) / n ** 0.5).to(dt)
        self.vp = vp
        self.embed = (draw(V, width).float() * V ** 0.5).to(dt)
        self.w_qkv = [draw(width, vp.qkv.shape[1]) for _ in range(vp.layers)]
        self.w_out = [draw(vp.Hq * vp.D, width) for _ in range(vp.layers)]
        self.w_logits = draw(width, V)

    def prompt(self, tokens, lengths):
        """tokens: the prompts one after the other on the device, lengths: a list of R."""
        vp, dev = self.vp, self.embed.device
        n = torch.tensor(lengths, dtype=torch.int32)
        offsets = torch.zeros(len(lengths) + 1, dtype=torch.int32)
        offsets[1:] = n.cumsum(0)
        request = torch.repeat_interleave(torch.arange(len(lengths), dtype=torch.int32), n.long())
        position = torch.arange(len(request), dtype=torch.int32) - offsets[request.long()]
        request, position, offsets, n = (x.to(dev) for x in (request, position, offsets, n))
        x = self.embed[tokens.long()]
        for l in range(vp.layers):
            x = x + vp.prompt(l, x @ self.w_qkv[l], request, position, offsets, max(lengths)).flatten(1) @ self.w_out[l]
        vp.advance_by(n)

    def logits(self, out):
        """The batch that was assembled through all layers; row (r, j) of out [R][gamma_max + 1][V] becomes the
        logits after request r's token j (rows past its last admitted token: anything)."""
        vp, b = self.vp, self.vp.batch
        x = self.embed[b["flat_tokens"].clamp(min=0).long()]
        for l in range(vp.layers):
            torch.mm(x, self.w_qkv[l], out=vp.qkv)
            x = x + vp.layer(l).flatten(1) @ self.w_out[l]
        at = b["offsets"][:-1, None].long() + torch.arange(vp.gamma_max + 1, device=x.device)
        out.copy_((x @ self.w_logits)[at.clamp(max=vp.T - 1).flatten()].view(out.shape))


def main():
    """Rounds of drafting, a verify pass through a random four-layer target, and acceptance."""
    from . import RoundRunner
    from .workloads import make_round

    R, G, V, rounds = 32, 7, 4096, 6
    rnd = make_round("verify_pass", R, G, V, 256, 512, "bf16", seed=1, device="cuda", u_std=1.0)
    runner = RoundRunner(rnd)
    vp = VerifyPass(R, G, 4, 16, 4, 128, capacity=1024)
    target = ToyTarget(vp, V, 512)
    lengths = [100 + 17 * r for r in range(R)]
    target.prompt(torch.randint(0, V, (sum(lengths),), device="cuda"), lengths)
    for i in range(rounds):
        runner.set_round(i)
        runner.run_draft()
        vp.assemble(runner.cout["keep"], rnd.anchor, runner.sout["tokens"])
        target.logits(rnd.target)
        runner.run_verify()
        out = runner.results()
        vp.advance(out["accepted"])
        rnd.anchor.copy_(out["next_token"])
        assert runner.check() == 0 and vp.check() == 0
        print("round %d: %d tokens admitted, %d accepted, longest context %d" % (
            i, int(out["keep"].sum()), int(out["accepted"].sum()), int(vp.ctx_len.max())))


if __name__ == "__main__":
    main()
