"""The target layer's entry points without a GPU: struct layouts, refusals before any launch, the
binding's own checks, and the pins of the 64-bit reference the GPU tests compare with."""
import ctypes as C
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import layer_ref as ref
import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300 import build as dsbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    dsbuild.build()
    return ds.lib()


def test_struct_layouts_match_c(L, tmp_path):
    structs = {"dspark_cache": ds.Cache, "dspark_qk_norm_rope_args": ds.QkNormRopeArgs,
               "dspark_cache_append_args": ds.CacheAppendArgs, "dspark_cache_read_args": ds.CacheReadArgs,
               "dspark_cache_attend_args": ds.CacheAttendArgs}
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


def test_block_bytes(L):
    assert ds.cache_block_bytes(16, 32) == 16 * 32 * 9 // 8
    assert ds.cache_block_bytes(64, 128) == 9216
    assert ds.cache_block_bytes(256, 256) == 73728
    for page, D in ((0, 128), (8, 128), (17, 128), (272, 128), (16, 0), (16, 16), (16, 48), (16, 288), (-16, 64)):
        with pytest.raises(ds.DsparkError) as e:
            ds.cache_block_bytes(page, D)
        assert e.value.code == 2


def _cache(**kw):
    c = ds.Cache()
    c.pages, c.n_pages, c.page_size, c.Hkv, c.D, c.R, c.table_width = FAKE, 8, 16, 2, 64, 3, 4
    c.table = c.ctx_len = FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _rope(**kw):
    a = ds.QkNormRopeArgs()
    a.struct_size = C.sizeof(a)
    a.T, a.Hq, a.Hkv, a.D, a.rot, a.R, a.norm, a.eps = 5, 4, 2, 64, 32, 3, 1, 1e-6
    for f in ("q", "k", "freq", "position", "request", "ctx_len", "q_out", "k_out"):
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _append(cache=None, **kw):
    a = ds.CacheAppendArgs()
    a.struct_size, a.T, a.cache = C.sizeof(a), 5, cache or _cache()
    for f in ("k", "v", "request", "position"):
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _read(cache=None, **kw):
    a = ds.CacheReadArgs()
    a.struct_size, a.T, a.cache = C.sizeof(a), 5, cache or _cache()
    for f in ("k_out", "v_out", "request", "position"):
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _attend(cache=None, **kw):
    a = ds.CacheAttendArgs()
    a.struct_size, a.T, a.Hq, a.max_q, a.scale, a.cache = C.sizeof(a), 5, 4, 5, 0.125, cache or _cache()
    for f in ("q", "offsets", "out", "lse"):
        setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD_CACHE = [(1, dict(pages=None)), (1, dict(pages=FAKE + 8)), (1, dict(n_pages=0)), (1, dict(n_pages=1 << 31)),
             (1, dict(table=None)), (1, dict(ctx_len=None)), (1, dict(table_width=0)), (1, dict(R=0)),
             (1, dict(Hkv=0)), (1, dict(reserved=1)), (2, dict(page_size=24)), (2, dict(page_size=0)),
             (2, dict(D=40)), (2, dict(D=512)), (2, dict(R=8193)), (2, dict(Hkv=1025)),
             (2, dict(table_width=1 << 27))]
CALLS = {
    "qk_norm_rope": (_rope, [(1, dict(struct_size=8)), (1, dict(T=-1)), (1, dict(Hq=0)), (1, dict(Hkv=0)),
                             (1, dict(D=63)), (1, dict(D=0)), (1, dict(D=1026)), (1, dict(rot=66)), (1, dict(rot=31)),
                             (1, dict(rot=-2)), (1, dict(dtype=2)), (1, dict(norm=2)), (1, dict(interleaved=-1)),
                             (1, dict(eps=-1.0)), (1, dict(eps=math.nan)), (1, dict(eps=math.inf)),
                             (1, dict(R=0)), (1, dict(request=None)), (1, dict(q=None)), (1, dict(k_out=None)),
                             (1, dict(position=None)), (1, dict(freq=None)), (1, dict(reserved=4))]),
    "cache_append": (_append, [(1, dict(struct_size=8)), (1, dict(T=-1)), (1, dict(dtype=2)), (1, dict(k=None)),
                               (1, dict(v=None)), (1, dict(request=None)), (1, dict(position=None)),
                               (1, dict(reserved=1))]),
    "cache_read": (_read, [(1, dict(struct_size=8)), (1, dict(T=-1)), (1, dict(dtype=2)), (1, dict(k_out=None)),
                           (1, dict(v_out=FAKE + 8)), (1, dict(request=None)), (1, dict(position=None))]),
    "cache_attend": (_attend, [(1, dict(struct_size=8)), (1, dict(T=-1)), (1, dict(Hq=3)), (1, dict(Hq=0)),
                               (1, dict(dtype=2)), (1, dict(path=3)), (1, dict(path=-1)), (1, dict(max_q=0)),
                               (1, dict(window=-1)), (1, dict(sinks=-1)), (1, dict(scale=0.0)),
                               (1, dict(scale=-1.0)), (1, dict(scale=math.nan)), (1, dict(scale=math.inf)),
                               (1, dict(q=None)), (1, dict(offsets=None)), (1, dict(out=None)),
                               (1, dict(out=FAKE + 8)), (2, dict(Hq=2 * 1025))]),
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
    if call != "qk_norm_rope":
        for code, kw in BAD_CACHE:
            assert run(C.byref(make(cache=_cache(**kw))), FAKE, 1 << 30, None) == code, kw
    assert run(C.byref(make()), None, 1 << 20, None) == 3
    assert run(C.byref(make()), FAKE, 16, None) == 3
    assert run(C.byref(make(T=0)), FAKE, 1 << 30, None) == 0   # nothing to do: no launch
    assert ds.launch_count() == before


def test_binding_refuses_what_it_cannot_marshal():
    q = torch.zeros((3, 4, 64))
    with pytest.raises(TypeError):
        ds.qk_norm_rope(q, q, None, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        ds.cache_attend(q, q, q, q, q)
    with pytest.raises(ValueError):
        ds.rope_frequencies(31, device="cpu")


def test_frequencies_are_fractions_of_a_turn():
    f = ds.rope_frequencies(8, base=100.0, device="cpu").tolist()
    for i, x in enumerate(f):
        assert abs(x / 2.0 ** 64 - 100.0 ** (-2 * i / 8) / (2 * math.pi)) < 2.0 ** -52
    assert ds.rope_frequencies(0, device="cpu").numel() == 0


# ------------------------------------------------------------------ pins of the reference

def test_reference_scale_has_eight_bits_and_codes_are_nearest():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 64)) * np.exp(rng.uniform(-8, 8, (50, 1)))).astype(np.float32)
    s = ref.scales_of(x)
    m, _ = np.frexp(s)
    assert np.all(m * 256 == np.rint(m * 256))
    v = ref.stored(x)
    prod = (v.astype(np.float32)).astype(np.float16).astype(np.float64)
    assert np.array_equal(prod, v)                       # code * scale is exact in fp16
    step = np.repeat(s, 32, -1)
    # within half a step, but for what the scale's rounding (2^-9) leaves above 7 steps
    assert np.all(np.abs(v - x) <= step / 2 + 7 * step * 2.0 ** -8)


def test_reference_attention_by_hand():
    # one head, two keys of width 32; the query sees both, then only itself in a window of 1
    k = np.zeros((2, 1, 32))
    v = np.zeros((2, 1, 32))
    k[0, 0, 0], k[1, 0, 0], v[0, 0, 5], v[1, 0, 5] = 1.0, 3.0, 2.0, 4.0
    q = np.zeros((1, 1, 32))
    q[0, 0, 0] = 1.0
    out, lse, _ = ref.attend(q, [k], [v], [1], [0, 1], 1.0, 0, 0)
    w = math.exp(1) / (math.exp(1) + math.exp(3))
    assert abs(out[0, 0, 5] - (2 * w + 4 * (1 - w))) < 1e-14
    assert abs(lse[0, 0] - math.log(math.exp(1) + math.exp(3))) < 1e-14
    out, lse, _ = ref.attend(q, [k], [v], [1], [0, 1], 1.0, 1, 0)
    assert out[0, 0, 5] == 4.0 and lse[0, 0] == 3.0
    out, _, _ = ref.attend(q, [k], [v], [1], [0, 1], 1.0, 1, 1)   # the first token stays visible
    assert abs(out[0, 0, 5] - (2 * w + 4 * (1 - w))) < 1e-14


def test_reference_rotation_keeps_lengths_and_far_positions():
    x = np.random.default_rng(0).standard_normal((2, 1, 8))
    f = [int(0.25 * 2 ** 64), int(2 ** 64 / 3)]
    y = ref.norm_rope(x, None, [1, (1 << 31) - 1], f, False, 0.0, True)
    np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-13)
    np.testing.assert_allclose(y[0, 0, :2], [-x[0, 0, 1], x[0, 0, 0]], atol=1e-12)       # a quarter turn
    assert ((1 << 31) - 1) % 4 == 3
    np.testing.assert_allclose(y[1, 0, :2], [x[1, 0, 1], -x[1, 0, 0]], atol=1e-12)       # three quarters
