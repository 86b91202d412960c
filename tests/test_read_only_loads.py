"""Source rule: a kernel that may start while the one before it still runs takes what that one writes by plain loads.
Loads through the read-only path (__ldg) are for data that nothing writes while the kernel runs."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_draft_round_gb300", "csrc")


def _body(name, start):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    text = text[text.index(start):]
    return re.sub(r"//[^\n]*", "", text[:text.index("\n}\n")])


@pytest.mark.parametrize("name,start", [
    ("logits.cu", "adjust_kernel(AdjustParams p)"),              # the table, masks, logits
    ("logits.cu", "seen_add_kernel(SeenParams p)"),              # verification's outcome
    ("verify.cu", "void row_load8("),                            # the target's rows
    ("linear_i8.cu", "linear_simt_kernel(LinearParams p)"),      # codes and scales
    ("linear_i8_tc.cu", "linear_layout_kernel("),
    ("linear_i8_tc.cu", "void pad_bytes("),
])
def test_no_read_only_loads_of_what_the_kernel_before_writes(name, start):
    assert "__ldg" not in _body(name, start)
