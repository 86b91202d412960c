"""Source rule for the waits in the CUDA kernels, in every form their loops take: a loop that tries a barrier or looks at
a count has a bound by the global timer, and the bound's start is taken for this wait, right before the loop."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_draft_round_gb300", "csrc")
SPIN = re.compile(r"while\s*\((\s*true\s*\)|.*(try_wait|test_wait|try_for)\s*\(|.*\*\s*(done|count)\b|.*volatile)")


def unbounded(name, lines):
    """The loops of a file that break the rule, and how many loops there are."""
    hits, loops = [], 0
    for i, line in enumerate(lines):
        if not SPIN.search(line):
            continue
        loops += 1
        if "globaltimer() - t0" not in "\n".join(lines[i:i + 8]):
            hits.append("%s:%d has no bound" % (name, i + 1))
        elif "t0 = globaltimer()" not in "\n".join(lines[max(0, i - 4):i]):
            hits.append("%s:%d is not timed from its own start" % (name, i + 1))
    return hits, loops


def test_every_wait_has_a_bound_of_its_own():
    hits, loops = [], 0
    for f in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        h, n = unbounded(os.path.basename(f), open(f, encoding="utf-8").read().splitlines())
        hits += h
        loops += n
    assert loops >= 13 and hits == []


def test_the_rule_sees_what_breaks_it():
    good = ["const unsigned long long t0 = globaltimer();", "while (!try_for(bar, parity, nap)) {",
            "    if (globaltimer() - t0 > limit_ns) return false;", "}"]
    assert unbounded("a", good) == ([], 1)
    assert unbounded("a", good[1:2] + good[3:])[0] == ["a:1 has no bound"]
    once = good[:1] + ["for (int n = 0; n < tiles; ++n) {"] + ["    work();"] * 5 + \
        ["    while (ok && n - *done > 4) {", "        if (globaltimer() - t0 > 4 * limit_ns) ok = false;", "    }", "}"]
    assert unbounded("a", once)[0] == ["a:8 is not timed from its own start"]
