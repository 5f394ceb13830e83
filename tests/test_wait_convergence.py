"""Waits of the kernels and lanes that leave their warp, read from the sources (no GPU needed).

mbar_wait answers each thread for itself, so the lanes of a warp may leave one
at the end of its limit with different answers. The instructions that follow in
a warp (elect.sync, tcgen05.ld, __syncwarp) wait for all lanes without a limit:
a warp therefore waits by mbar_wait_warp, whose answer is the same for every
lane, or by mbar_wait_lanes, which leaves every lane on the warp's path, and
mbar_wait stands only where one thread runs or as the argument of a vote."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "video_diffusion_transformer_fwd_b200", "csrc")
SOURCES = sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu")))
ONE_THREAD = re.compile(r"\blane == 0\b|\bthreadIdx\.x == 0\b|\belect_one\(\)")
SINGLE = re.compile(r"\bmbar_wait\(")
VOTE = re.compile(r"__all_sync\(0xffffffffu, [^;]*$")


def plain(text):
    text = re.sub(r"/\*.*?\*/", lambda m: re.sub(r"[^\n]", " ", m[0]), text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def waits_of_several_threads(text):
    """Lines of the calls of mbar_wait that no block or condition around them
    leaves to one thread, and no vote takes."""
    text, heads, start, found = plain(text), [], 0, []
    calls = {m.start() for m in SINGLE.finditer(text)}
    for i, c in enumerate(text):
        if i in calls and not VOTE.search(text[start:i]) and not any(ONE_THREAD.search(h) for h in heads + [text[start:i]]):
            found.append(text.count("\n", 0, i) + 1)
        if c == "{":
            heads.append(text[start:i])
            start = i + 1
        elif c == "}":
            heads.pop()
            start = i + 1
        elif c == ";" and text.count("(", start, i) == text.count(")", start, i):    # not inside a for's head
            start = i + 1
    assert not heads
    return found


def test_the_reader_tells_the_two_apart():
    one = "void f() { if (lane == 0 && n) { for (int i = 0; i < n; ++i) { if (!mbar_wait(b, 0)) break; } } }"
    warp = "void f() { if (lane == 0) { g(); }\n for (int i = 0; i < n; ++i) {\n if (!mbar_wait(b, 0)) break; // lane == 0\n } }"
    assert waits_of_several_threads(one) == [] and waits_of_several_threads(warp) == [3]
    vote = "void f() { ok = __all_sync(0xffffffffu, ok && mbar_wait(b, 0)); mbar_wait_warp(b, 0); mbar_wait_lanes(ok, b, 0); }"
    assert waits_of_several_threads(vote) == []


@pytest.mark.parametrize("name", SOURCES)
def test_warps_wait_with_one_answer(name):
    with open(os.path.join(CSRC, name)) as f:
        assert waits_of_several_threads(f.read()) == []


@pytest.mark.parametrize("name", SOURCES)
def test_no_lane_leaves_its_warp(name):
    """No return, break or continue that a lane takes for itself: what comes
    after it in the warp is executed by all lanes or by none."""
    with open(os.path.join(CSRC, name)) as f:
        text = plain(f.read())
    assert re.findall(r"if \([^;{}]*\b(?:lane|threadIdx\.x)\b[^;{}]*\) (?:return|break|continue)\b", text) == []


def test_no_cta_waits_for_tmem_of_another():
    """Kernels that take more of TMEM than a share take the shared memory that
    keeps other CTAs off their SM."""
    for name in SOURCES:
        with open(os.path.join(CSRC, name)) as f:
            text = plain(f.read())
        if "tmem_alloc" in text:
            assert "SMEM_ALONE" in text, name
