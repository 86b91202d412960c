"""The entry points of the rest of the target's pass without a GPU: struct layouts, refusals before any launch, the
binding's own checks, and pins of the 64-bit reference the GPU tests compare with."""
import ctypes as C
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import pass_ref as ref
import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300 import build as dsbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    dsbuild.build()
    return ds.lib()


def test_struct_layouts_match_c(L, tmp_path):
    structs = {"dspark_add_norm_quant_args": ds.AddNormQuantArgs, "dspark_linear_i8_args": ds.LinearI8Args,
               "dspark_seen_add_args": ds.SeenAddArgs, "dspark_adjust_logits_args": ds.AdjustLogitsArgs}
    lines = ['  printf("%%zu\\n", sizeof(%s));' % n for n in structs]
    want = [C.sizeof(s) for s in structs.values()]
    for n, s in structs.items():
        for f, _ in s._fields_:
            lines.append('  printf("%%zu\\n", offsetof(%s, %s));' % (n, f))
            want.append(getattr(s, f).offset)
    src, exe = tmp_path / "t.c", tmp_path / "t"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"dspark.h\"\nint main(void) {\n%s\n  return 0;\n}\n"
                   % "\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == want


def _make(cls, values, pointers, kw):
    a = cls()
    a.struct_size = C.sizeof(a)
    for k, v in values.items():
        setattr(a, k, v)
    for f in pointers:
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _norm(**kw):
    return _make(ds.AddNormQuantArgs, dict(T=5, N=64, norm=1, eps=1e-6, x_stride=64, residual_stride=64, sum_stride=64,
                                           y_stride=64, codes_stride=64),
                 ("x", "residual", "gain", "n_rows", "sum", "codes", "scale"), kw)


def _linear(**kw):
    return _make(ds.LinearI8Args, dict(T=5, K=64, N=32, out_rows=5, x_stride=64, w_stride=64, out_stride=32),
                 ("x", "x_scale", "w", "w_scale", "bias", "n_rows", "out"), kw)


def _seen(**kw):
    return _make(ds.SeenAddArgs, dict(R=3, W=4, V=100, seen_stride=104, tokens_stride=4),
                 ("seen", "tokens", "n", "extra", "fresh"), kw)


def _adjust(**kw):
    return _make(ds.AdjustLogitsArgs, dict(R=3, S=5, V=100, n_masks=15, n_bias=4, seen_stride=104, mask_stride=4),
                 ("logits", "out", "seen", "repetition", "presence", "frequency", "tokens", "bias_offsets", "bias_token",
                  "bias_value", "mask", "keep"), kw)


CALLS = {
    "add_norm_quant": (_norm, [(1, dict(struct_size=8)), (1, dict(T=-1)), (1, dict(N=0)), (1, dict(dtype=2)),
                               (1, dict(norm=2)), (1, dict(eps=-1.0)), (1, dict(eps=math.nan)), (1, dict(eps=math.inf)),
                               (1, dict(x=None)), (1, dict(scale=None)), (1, dict(codes=None)),
                               (1, dict(codes=None, scale=None)), (1, dict(residual=None)), (1, dict(y=FAKE)),
                               (1, dict(sum_stride=63)), (1, dict(codes_stride=0)), (1, dict(y=2 * FAKE, y_stride=8)),
                               (1, dict(x_stride=-64)), (1, dict(residual_stride=-1)), (2, dict(N=32769))]),
    "linear_i8": (_linear, [(1, dict(struct_size=8)), (1, dict(T=-1)), (1, dict(K=0)), (1, dict(N=0)), (1, dict(dtype=2)),
                            (1, dict(path=3)), (1, dict(path=-1)), (1, dict(out_rows=4)), (1, dict(out_rows=-1, out_row=FAKE)),
                            (1, dict(reserved=1)), (1, dict(x=None)), (1, dict(x_scale=None)), (1, dict(w=None)),
                            (1, dict(w_scale=None)), (1, dict(out=None)), (1, dict(x_stride=-1)), (1, dict(w_stride=-1)),
                            (1, dict(out_stride=31)), (2, dict(K=131072)), (2, dict(N=(1 << 24) + 1))]),
    "seen_add": (_seen, [(1, dict(struct_size=8)), (1, dict(R=0)), (1, dict(W=-1)), (1, dict(V=0)), (1, dict(prompt=2)),
                         (1, dict(reserved=1)), (1, dict(seen=None)), (1, dict(seen=FAKE + 8)), (1, dict(seen_stride=100)),
                         (1, dict(seen_stride=96)), (1, dict(tokens=None)), (1, dict(tokens_stride=-4)),
                         (2, dict(R=8193)), (2, dict(V=(1 << 24) + 1))]),
    "adjust_logits": (_adjust, [(1, dict(struct_size=8)), (1, dict(R=0)), (1, dict(S=0)), (1, dict(V=0)), (1, dict(dtype=2)),
                                (1, dict(n_masks=-1)), (1, dict(n_bias=-1)), (1, dict(reserved=1)), (1, dict(logits=None)),
                                (1, dict(out=None)), (1, dict(seen=FAKE + 2)), (1, dict(seen_stride=96)),
                                (1, dict(seen_stride=101)), (1, dict(bias_token=None)), (1, dict(bias_value=None)),
                                (1, dict(mask_stride=3)), (1, dict(n_masks=14)), (1, dict(mask=None, mask_row=FAKE)),
                                (2, dict(R=8193)), (2, dict(S=34)), (2, dict(V=(1 << 24) + 1))]),
}


@pytest.mark.parametrize("call", sorted(CALLS))
def test_refusals_come_before_any_launch(L, call):
    make, bad = CALLS[call]
    size, run = getattr(L, "dspark_%s_workspace_size" % call), getattr(L, "dspark_" + call)
    n = C.c_size_t(0)
    before = ds.launch_count()
    assert size(C.byref(make()), C.byref(n)) == 0 and n.value >= 256
    assert size(C.byref(make()), None) == 1
    assert size(None, C.byref(n)) == 1
    for code, kw in bad:
        assert size(C.byref(make(**kw)), C.byref(n)) == code, kw
        assert run(C.byref(make(**kw)), FAKE, 1 << 30, None) == code, kw
    assert run(C.byref(make()), None, 1 << 20, None) == 3
    assert run(C.byref(make()), FAKE, 16, None) == 3
    assert run(C.byref(make()), FAKE + 2, 1 << 30, None) == 1
    if call in ("add_norm_quant", "linear_i8"):
        assert run(C.byref(make(T=0)), FAKE, 1 << 30, None) == 0   # nothing to do: no launch
    assert ds.launch_count() == before


def test_binding_refuses_what_it_cannot_marshal():
    x = torch.zeros((3, 64))
    with pytest.raises(TypeError):
        ds.add_norm_quant(x)
    with pytest.raises(TypeError):
        ds.linear_i8(x.to(torch.int8), x, x, x)
    with pytest.raises(TypeError):
        ds.seen_add(x, None, V=3)
    with pytest.raises(TypeError):
        ds.adjust_logits(x[None])


# ------------------------------------------------------------------ pins of the reference

def test_reference_codes_by_hand():
    x = np.array([[2.54, -1.27, 0.01, 0.0]], np.float32)
    s, y, c, scale = ref.norm_quant(x, None, None, False, 0.0, False)
    assert np.array_equal(s, x) and c.tolist() == [[127, -64, 0, 0]]     # -63.5 goes to the even one
    assert abs(scale[0] - 0.02) < 1e-8
    s, y, c, scale = ref.norm_quant(x, x, np.array([1, 2, 1, 1], np.float32), True, 0.0, False)
    assert np.array_equal(s, 2 * x) and c.tolist() == [[127, -127, 0, 0]]
    assert abs((y[0] / [1, 2, 1, 1] ** np.ones(4)) @ (y[0] / [1, 2, 1, 1] ** np.ones(4)) - 4) < 1e-12


def test_reference_table_and_logits_by_hand():
    t = np.zeros((1, 8), np.int16)
    t = ref.seen_add(t, 5, [[1, 1, 9]], [3], [2], None, False)
    t = ref.seen_add(t, 5, [[2, 3]], [1], None, None, True)
    assert t.view(np.uint16)[0].tolist() == [0, 2, 0x8001, 0, 0, 0, 0, 0]
    z = np.array([[[4.0, 4.0, -4.0, 1.0, 0.0]] * 2])
    out, _ = ref.adjust(z, t, [2.0], [0.5], [0.25], [[3]], [[(4, 1.0), (4, 2.0)]],
                        np.array([[True, True, True, True, False]]), [[-1, 0]], None)
    assert out[0, 0].tolist() == [4.0, 4 / 2 - 0.5 - 0.5, -8 - 0.25 - 0.5, 1.0, 3.0]
    assert out[0, 1].tolist() == [4.0, 1.0, -8.75, 0.5 - 0.25 - 0.5, -np.inf]
    assert ref.pack_bits(np.arange(40)[None] % 2 == 1).view(np.uint32).tolist() == [[0xAAAAAAAA, 0xAA]]
