"""What the kernels' sources promise the compiler, read from their signatures:
no `__restrict__` on a pointer that a documented call may alias, or whose data
the preceding grid still writes when the kernel starts."""
import os
import re

import pytest

from mixed_precision_int8_b200 import build


def signature(source, kernel):
    """{parameter: its declaration} of a kernel."""
    text = open(os.path.join(build.CSRC, source)).read()
    at = re.search(r"\b%s\(" % kernel, text).end()
    end, depth = at, 1
    while depth:
        depth += {"(": 1, ")": -1}.get(text[end], 0)
        end += 1
    return {re.search(r"(\w+)$", p.strip()).group(1): " ".join(p.split())
            for p in text[at:end - 1].split(",")}


# layer norm works in place: y on x, dx on x or dy
IN_PLACE = [("layernorm.cuh", "k_ln_forward", ("x", "y")),
            ("layernorm.cuh", "k_ln_forward_long", ("x", "y")),
            ("layernorm.cuh", "k_ln_backward", ("dy", "x", "dx")),
            ("layernorm.cuh", "k_ln_backward_long", ("dy", "x", "dx")),
            ("adapters.cuh", "k_rows_expand", ("base", "out"))]


@pytest.mark.parametrize("source,kernel,names", IN_PLACE)
def test_pointers_that_may_be_the_same_are_not_restrict(source, kernel, names):
    params = signature(source, kernel)
    for name in names:
        assert "*" in params[name] and "__restrict__" not in params[name], params[name]


# what the preceding grid still writes while a programmatic dependent starts:
# a read through `const __restrict__` may take the read-only path, or move
# before the wait for that grid
WRITTEN_BY_THE_PRECEDING_GRID = [("adapters.cuh", "k_rows_expand", ("part",)),
                                 ("layernorm.cuh", "k_ln_reduce", ("part",)),
                                 ("grad_clip.cuh", "k_clip_scale", ("partial",))]


@pytest.mark.parametrize("source,kernel,names", WRITTEN_BY_THE_PRECEDING_GRID)
def test_results_of_a_grid_still_running_are_not_restrict(source, kernel, names):
    test_pointers_that_may_be_the_same_are_not_restrict(source, kernel, names)
