"""Direct loads to LDS in inline assembly (CPU): the compiler counts wait states
for its own instructions only, so each block that writes M0 has to hold the one
that a load to LDS needs after it."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_int8_gemm_amd", "csrc")


def test_a_wait_state_between_the_write_of_m0_and_the_load():
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*")):
        for text in re.findall(r"asm\s*(?:volatile)?\s*\(\s*((?:\"[^\"]*\"\s*)+)", open(path).read()):
            lines = re.split(r"\\n|\\t|;", "".join(re.findall(r"\"([^\"]*)\"", text)))
            lines = [x.strip() for x in lines if x.strip()]
            for i, x in enumerate(lines):
                if re.match(r"(buffer|global|scratch)_load.*\blds$", x):
                    found += 1
                    assert i >= 2 and lines[i - 1].startswith("s_nop") and re.match(r"s_\w+ m0,", lines[i - 2]), (path, lines)
    assert found >= 2
