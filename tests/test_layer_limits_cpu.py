"""Which batches the matrix kernels of cache_attend count in 32 bits: by the rows that there are, not by as many for every
request as one of them may have. No launch: a workspace that is too small says that the kernel would have been taken."""
import ctypes as C

import pytest

import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300 import build as dsbuild

FAKE = 0x10000
WORKSPACE, UNSUPPORTED = 3, 2


@pytest.fixture(scope="module")
def run():
    dsbuild.build()
    before = ds.launch_count()

    def code(T, R, max_q, Hq, Hkv, width, dtype, D=128, page=64):
        a = ds.CacheAttendArgs()
        a.struct_size, a.T, a.Hq, a.max_q, a.scale, a.dtype = C.sizeof(a), T, Hq, max_q, 0.1, dtype
        a.path = ds.PATH_TENSOR_CORE
        a.q = a.offsets = a.out = a.lse = FAKE
        c = a.cache
        c.pages = c.table = c.ctx_len = FAKE
        c.n_pages, c.page_size, c.Hkv, c.D, c.R, c.table_width = 1, page, Hkv, D, R, width
        return ds.lib().dspark_cache_attend(C.byref(a), FAKE, 256, None)

    yield code
    assert ds.launch_count() == before


@pytest.mark.parametrize("dtype", [ds.F32, ds.BF16])
@pytest.mark.parametrize("T,R,max_q,tokens", [(8192 + 127, 128, 8192, 32768), (65536, 64, 65536, 131072),
                                              (8192, 8192, 8192, 32768), (20000, 4, 20000, 1 << 20)])
def test_one_long_prompt_among_single_rows(run, T, R, max_q, tokens, dtype):
    assert run(T, R, max_q, 32, 8, tokens // 64, dtype) == WORKSPACE


def test_batches_past_the_counters_are_refused(run):
    assert run(1 << 20, 1, 1 << 20, 32, 8, (1 << 20) // 64, ds.F32) == UNSUPPORTED
    assert run(1 << 22, 1, 1 << 22, 64, 8, (1 << 22) // 64, ds.BF16) == UNSUPPORTED
    assert run(1 << 28, 1, 1 << 28, 32, 8, 1, ds.BF16) == UNSUPPORTED   # rows of a request and key head


def test_blocks_of_128_rows_are_counted_as_such(run):
    """More blocks of 16 rows than can be counted, but not of 128."""
    assert run(1 << 18, 1, 1 << 18, 32, 8, (1 << 18) // 64, ds.F32) == UNSUPPORTED
    assert run(1 << 18, 1, 1 << 18, 32, 8, (1 << 18) // 64, ds.BF16) == WORKSPACE


@pytest.mark.parametrize("D", [128, 96])   # the matrix kernels' workspace, and a status word alone
def test_workspaces_off_their_boundaries_are_refused(run, D):
    a = ds.CacheAttendArgs()
    a.struct_size, a.T, a.Hq, a.max_q, a.scale, a.dtype = C.sizeof(a), 0, 8, 4, 0.1, ds.BF16
    c = a.cache
    c.pages = c.table = c.ctx_len = FAKE
    c.n_pages, c.page_size, c.Hkv, c.D, c.R, c.table_width = 1, 16, 2, D, 3, 4
    n = C.c_size_t(0)
    assert ds.lib().dspark_cache_attend_workspace_size(C.byref(a), C.byref(n)) == 0 and (n.value > 256) == (D == 128)
    for off in range(17):
        ok = off % (16 if D == 128 else 4) == 0
        assert ds.lib().dspark_cache_attend(C.byref(a), FAKE + off, n.value, None) == (0 if ok else 1), off
    assert ds.lib().dspark_cache_attend(C.byref(a), FAKE, n.value - 1, None) == WORKSPACE


@pytest.mark.parametrize("call,args", [("qk_norm_rope", ds.QkNormRopeArgs), ("cache_append", ds.CacheAppendArgs),
                                       ("cache_read", ds.CacheReadArgs)])
def test_status_words_off_their_boundaries_are_refused(run, call, args):
    a = args()
    a.struct_size = C.sizeof(a)
    if call == "qk_norm_rope":
        a.Hq, a.Hkv, a.D = 2, 1, 64
    else:
        c = a.cache
        c.pages = c.table = c.ctx_len = FAKE
        c.n_pages, c.page_size, c.Hkv, c.D, c.R, c.table_width = 1, 16, 2, 64, 3, 4
    for off in range(9):
        assert getattr(ds.lib(), "dspark_" + call)(C.byref(a), FAKE + off, 256, None) == (1 if off % 4 else 0), off


def test_empty_batches_need_no_pointers(run):
    """An empty tensor's address is 0."""
    a = ds.QkNormRopeArgs()
    a.struct_size = C.sizeof(a)
    a.Hq, a.Hkv, a.D, a.rot, a.R, a.ctx_len, a.freq = 2, 1, 64, 64, 3, FAKE, FAKE
    assert ds.lib().dspark_qk_norm_rope(C.byref(a), FAKE, 256, None) == 0
