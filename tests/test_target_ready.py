"""When verification may read the target's first rows: only where the caller states that they were written before the
scheduler began (target_ready). No GPU needed."""
import ctypes as C
import os
import re
import types

import pytest

import speculative_decoding_draft_round_gb300 as ds
from speculative_decoding_draft_round_gb300 import build as dsbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_nothing_of_the_target_is_read_before_the_wait_unless_it_is_ready():
    """The kernel before dspark_verify may be the one that writes the target (dspark_adjust_logits in place)."""
    text = open(os.path.join(ROOT, "speculative_decoding_draft_round_gb300", "csrc", "verify.cu"), encoding="utf-8").read()
    body = text[text.index("verify_rows_kernel(VerifyParams p)"):]
    before = body[:body.index("pdl_enter()")]
    # the only items formed there come from pre_item, which has none without target_ready
    assert re.search(r"const int pre = p\.target_ready \? kRowPre : 0;", before)
    assert re.search(r"if \(k >= pre \|\| it >= n0\) return RowItem\{-1, 0, 0\};", before)
    items = re.findall(r"RowItem (\w+) = (\w+)\(", before)
    assert items and all(made == "pre_item" for _, made in items)
    # and rows are read by plain loads, not by those for data that nothing writes while the kernel runs
    load = text[text.index("void row_load8("):]
    assert "__ldg" not in load[:load.index("\n}\n")]


def _args(**kw):
    a = ds.VerifyArgs()
    a.struct_size = C.sizeof(ds.VerifyArgs)
    a.R, a.gamma_max, a.V, a.r, a.dtype = 8, 4, 100, 16, ds.BF16
    for f in ("target", "U", "E", "W", "anchor", "tokens", "draft_lse", "draft_logit", "keep", "temperature", "accepted",
              "next_token", "resampled"):
        setattr(a, f, 0x10000)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_values_and_the_struct_without_it():
    dsbuild.build()
    size, n = ds.lib().dspark_verify_workspace_size, C.c_size_t(0)
    short = ds.VerifyArgs.target_ready.offset
    for kw in (dict(), dict(target_ready=1), dict(struct_size=short), dict(struct_size=short, target_ready=7, reserved=9)):
        assert size(C.byref(_args(**kw)), C.byref(n)) == 0, kw
    for kw in (dict(target_ready=2), dict(target_ready=-1), dict(reserved=1), dict(struct_size=short - 8),
               dict(struct_size=short + 4)):
        assert size(C.byref(_args(**kw)), C.byref(n)) == 1, kw


@pytest.mark.parametrize("adjusts", [False, True])
def test_a_runner_says_so_for_whole_rounds_only(monkeypatch, adjusts):
    calls = []
    monkeypatch.setattr(ds, "_call", lambda name, *a: calls.append((name, runner.va.target_ready)))
    monkeypatch.setattr(ds, "_stream", lambda s: None)
    runner = object.__new__(ds.RoundRunner)
    ws = types.SimpleNamespace(data_ptr=lambda: 0, numel=lambda: 0)
    runner.sws = runner.cws = runner.vws = runner.jws = ws
    runner.sa, runner.ca, runner.va = ds.SampleArgs(), ds.ScheduleArgs(), ds.VerifyArgs()
    runner.ja, runner.na = (ds.AdjustLogitsArgs(), ds.SeenAddArgs()) if adjusts else (None, None)
    runner.run()
    runner.run_draft()
    runner.run_verify()
    assert [r for name, r in calls if name == "dspark_verify"] == [0 if adjusts else 1, 0]
    assert [name for name, _ in calls].count("dspark_adjust_logits") == (2 if adjusts else 0)
