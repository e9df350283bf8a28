"""What the kernels' sources promise the compiler, read from their signatures:
no `__restrict__` on a pointer that a documented call may alias, or whose data
the preceding grid still writes when the kernel starts; and the scopes of the
signals between the CTAs of a pair."""
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


def test_arrivals_in_the_other_cta_release_at_cluster_scope():
    """An arrival without a scope has that of its own CTA: it would not order
    its thread's writes for a waiter in the other one."""
    seen = 0
    for name in sorted(os.listdir(build.CSRC)):
        text = open(os.path.join(build.CSRC, name)).read()
        for op in re.finditer(r"mbarrier\.arrive[\w.:]*shared::cluster[\w.:]*", text):
            before = text[text.rindex("asm", 0, op.start()):op.start()]
            assert (".release.cluster" in op[0] or ".relaxed.cluster" in op[0] and
                    "fence.release.sync_restrict::shared::cta.cluster;" in before), (name, op[0])
            seen += 1
    assert seen  # k_input_grad's


def test_the_input_gradient_s_issuer_acquires_what_the_other_cta_released():
    text = open(os.path.join(build.CSRC, "input_grad_sm100.cuh")).read()
    issuer = text[text.index("- MMA issuer"):text.index("- TMA producer of the codes")]
    waits = re.findall(r"mbar_wait\w*\((\w+)", issuer)
    assert {w: f for f, w in re.findall(r"(mbar_wait\w*)\((\w+)", issuer)} == {
        "full_bar": "mbar_wait_bounded_cluster", "tempty_bar": "mbar_wait_bounded_cluster",
        "drain_bar": "mbar_wait_bounded"}  # drain: this thread's own commit
    assert len(waits) == 4
