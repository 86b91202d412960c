"""Source rule: where a product's rounding error is taken by a fused multiply-add, the product and the differences around it
are spelt out, so that the compiler fuses none of them."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_draft_round_gb300", "csrc")


def test_remainders_of_products_in_add_norm_quant():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "add_norm_quant.cu"), encoding="utf-8").read())
    for name in ("int settled(", "int remainder_at("):
        body = text[text.index(name):]
        body = body[:body.index("\n}\n")]
        assert "__fmaf_rn(" in body and not re.search(r"\bfmaf\(", body)
        # whatever enters a remainder is a spelt product: no operator between its operands
        for product in re.findall(r"__fmaf_rn\(([^()]*(?:\([^()]*\))?[^()]*), -(\w)\)", body):
            factors, head = product
            assert "%s = __fmul_rn(%s)" % (head, factors) in body, (name, product)
        assert not re.search(r"\bd = .*[-+*] ", body[body.index("__fmaf_rn("):])
