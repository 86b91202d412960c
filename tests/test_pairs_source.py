"""Source rules for kernels whose CTAs work in pairs on tensor memory, where a fault would be a stop of the GPU: tensor
memory is asked for when both CTAs stand, and no CTA leaves while arrivals at its barriers are under way."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_draft_round_gb300", "csrc")


def _kernels():
    """The kernels that allocate for both CTAs of a pair, without comments."""
    found = {}
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(f, encoding="utf-8").read())
        for m in re.finditer(r"\n__global__ .*?\n}\n", text, flags=re.S):
            if "pair_alloc(" in m.group(0):
                found[os.path.basename(f)] = m.group(0)
    return found


def test_a_pair_stands_before_it_allocates_and_after():
    kernels = _kernels()
    assert kernels
    for name, body in kernels.items():
        at = body.index("pair_alloc(")
        assert "cluster_wait();" in body[body.index("cluster_arrive();"):at], name
        after = body[at:]
        first_use = after.index("const uint32_t tmem")
        assert "cluster_sync();" in after[:first_use], name


def test_a_pair_leaves_after_its_last_arrivals():
    for name, body in _kernels().items():
        end = body[body.rindex("pair_commit(bar(kFin), both)"):]
        drain, freed = end.index("drain(bar(kFin), 0u)"), end.index("pair_dealloc(")
        assert "__syncthreads();" in end[:drain], name                  # its limit counts from when all warps are through
        assert "cluster_sync();" in end[drain:freed], name
        # the widening warps of either CTA see the release of every step
        assert re.search(r"for \(int left = min\(n, g\.slots\); left > 0 && ok; --left\) \{\s*ok = wait\.warp\(bar\(kDone \+ back\)",
                         end), name
