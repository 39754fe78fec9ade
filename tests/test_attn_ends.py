"""The ends of the attention kernels' CTAs, in their sources: copies and products that are under way when a role gives up (a wait's
limit) are awaited once all roles are over, before shared memory and TMEM go back. A role that looks for itself may end before
another one gives up. No GPU needed, and none could show it without a fault."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = {"attn_fwd.cu": 1, "attn_bwd.cu": 2, "attn_decode.cu": 1}      # those with copies and products of their own


def bodies(text, pattern):
    for m in re.finditer(pattern, text):
        start = text.index("{", m.end())
        yield text[start:text.index("\n}\n", start)]


@pytest.mark.parametrize("name", KERNELS)
def test_copies_and_products_are_awaited_when_all_roles_are_over(name):
    text = open(os.path.join(ROOT, "invariant_deterministic_gemm_gb300", "csrc_ops", name)).read()
    roles = list(bodies(text, r"__device__ void \w*(copy|issue|math|softmax|join|page)\w*\("))
    assert len(roles) >= 3
    copying = [b for b in roles if re.search(r"load_tile<|cp\.async\.bulk", b)]
    assert len(copying) == KERNELS[name]
    for body in copying:
        assert "copies.add(" in body and re.search(r"\n {4,8}S\.copies(\[kind\])? = copies;\n", body + "\n")
    kernels = [b for b in bodies(text, r"__global__ void __launch_bounds__\([^)]*\) \w+\(") if "tcgen05.dealloc" in b]
    assert len(kernels) == KERNELS[name]
    for body in kernels:
        assert "S.copies" in body[:body.index("__syncthreads()")]        # none are under way at first
        end = body[body.rindex("if (*wait.abort_flag) {"):]
        before = body[:body.rindex("if (*wait.abort_flag) {")].rstrip()
        assert before.endswith("__syncthreads();\n    tc_fence_after();")
        places = [end.index(x) for x in ("drain_copies(", "drain_products(", "__syncthreads();", "tcgen05.dealloc")]
        assert places == sorted(places)
