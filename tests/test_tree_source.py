"""What csrc/tree.cuh has to do in every path, read from its source: orders that neither a result nor the
model of its barriers would show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_int4_tma_gb300", "csrc")


def source():
    with open(os.path.join(CSRC, "tree.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def order(text, taken):
    """The events of straight code with one kind of branch, `if (a.head_dim < DP) {`, taken or not: accesses to the
    memory at `base` by ordinary instructions, fences between them and the copies, barriers of all threads."""
    events, skip, depth = [], None, 0
    for m in re.finditer(r"if \(a\.head_dim < DP\) \{|\{|\}|locate\(seg\)|prefix\[|tree_store16\(base|"
                         r"fence_proxy_async_smem\(\)|__syncthreads\(\)", text):
        word = m.group()
        if word.endswith("{"):
            if word != "{" and not taken and skip is None:
                skip = depth
            depth += 1
        elif word == "}":
            depth -= 1
            if skip == depth:
                skip = None
        elif skip is None:
            events.append({"f": "fence", "_": "barrier"}.get(word[0], "access"))
    return events


def ready(events):
    """A copy by another thread may write there: since the last access every thread has fenced and then met the
    others."""
    state = "clean"
    for e in events:
        if e == "access":
            state = "touched"
        elif e == "fence" and state == "touched":
            state = "fenced"
        elif e == "barrier" and state == "fenced":
            state = "clean"
    return state == "clean"


@pytest.mark.parametrize("taken", [False, True])
def test_prefix_sums_give_way_to_the_queries(taken):
    """The prefix sums of the split stand where the first queries will; the tensor copies that bring those write
    through the async proxy, which only a fence orders behind ordinary accesses."""
    text = source()
    begin = text.index("bool more = locate(seg);")
    events = order(text[begin: text.index("if (warp >= S::LOADERS", begin)], taken)
    assert events[0] == "access" and ready(events), events


def test_the_check_of_order_finds_what_is_missing():
    assert ready(["access", "fence", "barrier"]) and ready(["access", "barrier", "access", "fence", "barrier"])
    for bad in (["access", "barrier"], ["access", "fence"], ["fence", "access", "barrier"],
                ["access", "fence", "barrier", "access", "barrier"], ["access", "barrier", "fence"]):
        assert not ready(bad), bad


def test_no_copy_is_issued_after_a_wait_that_ran_out():
    """Every place that issues tensor copies looks at the flag of a wait that gave up between its last wait, or its
    beginning, and the copies: what is under way when the kernel ends is what was issued before."""
    text = source()
    places = [m.start() for m in re.finditer(r"auto (issue|ask_queries) = ", text)]
    copies = [m.start() for m in re.finditer(r"tma_tensor_4d_g2s\(", text)]
    assert len(places) == len(copies) == 2
    for place, copy in zip(places, copies):
        assert place < copy
        waited = max(place, text.rfind("wait(", place, copy))
        assert "abort_flag" in text[waited: copy], text[place: copy]


def test_only_tensor_maps_that_were_made_are_prefetched():
    """Without boxes the kernel is given zeros in a map's place."""
    text = source()
    for name, boxes in (("kmap", "box_rows"), ("vmap", "box_rows"), ("qmap", "q_box")):
        at = text.index(f"prefetch_tensormap(&{name})")
        begin = text.rindex(f"if ({boxes} > 0)", 0, at)
        assert "}" not in text[begin: at], text[begin: at]
