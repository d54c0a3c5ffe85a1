"""The beam selection's promise that logits of a beam at -inf are not read, on the CPU: what such a
read returns has no effect, so no result shows it, and memory that must not be read is not for a test.
So this looks at the kernel's order: it loads no logit before it knows that the beam counts."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decoding_verification_65_gb300", "csrc")


def test_no_logit_before_the_beam_is_known_to_count():
    with open(os.path.join(CSRC, "spec_beam.cu")) as f:
        text = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    kernel = text[text.index("beam_kernel(const __grid_constant__ BeamParams P)"):]
    before, after = kernel.split("if (counts)", 1)
    assert "counts = " in before and "A.scores[row]" in before and "A.finished[row]" in before
    assert not re.search(r"\bfetch\(|\bedge\(|\bload1\(|A\.logits", before)
    assert "fetch(" in after and "edge(" in after
