"""Every function of the attention kernels' sources has a caller."""
import glob
import os
import re

SOURCES = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "invariant_deterministic_gemm_gb300", "csrc_ops")


def test_no_function_without_a_caller():
    texts = {f: re.sub(r"//[^\n]*", "", open(f).read()) for f in glob.glob(os.path.join(SOURCES, "*"))}
    everything = "\n".join(texts.values())
    found = 0
    for f, text in texts.items():
        if not os.path.basename(f).startswith(("attn", "rope")):
            continue
        for name in re.findall(r"(?:__device__|__global__|inline)[^;{}()=\n]*(?:\([^)]*\)[^;{}()=\n]*?)?\b(\w+)\(", text):
            found += 1
            assert len(re.findall(r"\b%s\b" % name, everything)) > 1, (os.path.basename(f), name)
    assert found > 60
