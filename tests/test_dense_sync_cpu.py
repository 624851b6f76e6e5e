"""The dense products' waits in csrc/moe_dense.cuh, read from their source. A run's
bounded waits may not begin before the work that it depends on has ended: launches
overlap, and however long the kernels before it take, a run whose copies wait for
them has not failed."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def kernel(name):
    text = open(os.path.join(ROOT, "sparse_expert_gemv_gb300", "csrc", "moe_dense.cuh")).read()
    text = re.sub(r"//[^\n]*", "", text)
    start = re.search(r"__global__[^;{]*\b%s\(" % name, text).end()
    return text[start:text.index("\n}\n", start)]


# each role's first and, where it ends before the next one's, last text
ROLES = {"moe_dense_tiles": ["if (warp == 0) {", "} else if (warp == 1) {", "} else if (FLOAT && warp >= 4) {",
                             "} else if (!FLOAT && warp >= 4) {"],
         "moe_dense_split": ["if (warp == 8) {", "} else if (warp == 9) {", "if (warp < 8) {"]}


@pytest.mark.parametrize("name,role", [(k, i) for k, v in ROLES.items() for i in range(len(v))])
def test_every_role_waits_for_the_kernels_before_it_first(name, role):
    text, starts = kernel(name), ROLES[name]
    first = [text.index(starts[0])]
    for s in starts[1:]:
        first.append(text.index(s, first[-1] + 1))
    body = text[first[role]:first[role + 1] if role + 1 < len(first) else len(text)]
    waits = [m.start() for m in re.finditer(r"(dense_wait<|prod_wait_end\()", body)]
    assert waits and "pdl_wait();" in body
    before = body[:body.index("pdl_wait();")]
    assert body.index("pdl_wait();") < min(waits)
    # and does so under no condition that its waits are not under
    depth = before.count("{") - before.count("}")
    wait_depth = body[:min(waits)].count("{") - body[:min(waits)].count("}")
    assert depth <= wait_depth


@pytest.mark.parametrize("name", ROLES)
def test_no_output_is_touched_before_the_kernels_before_it_end(name):
    # every role that writes passes pdl_wait above; the waits in front of the roles are
    # for what the pair itself does
    text = kernel(name)
    front = text[:text.index(ROLES[name][0])]
    assert "dense_wait" not in front and "p.out" not in re.sub(r"p\.out_float|prefetch_tmap\(&p\.tm_out\)", "", front)
