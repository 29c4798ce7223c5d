"""Waits that run out end their kernel (no GPU needed; nothing here makes one run out)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ordered_merge_gb300", "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_the_beam_selection_heeds_its_waits():
    """The ring's wait is asked whether it ran out; nothing is copied after that, and other waits then do not spin."""
    code = _code("beam_kernels.cuh")
    calls = re.findall(r"(\w*\s*\(?!?)mbar_wait_(\w+)\(", code)
    assert [kind for _, kind in calls] == ["bounded", "or_stop"]
    ran_out = re.search(r"if \(!mbar_wait_or_stop\(&s\.full\[stage\], phase, a\.err, &s\.stop\) && threadIdx\.x == 0\) \{(.*?)\}", code, re.S)
    assert "ring_stops(a, stage, phase, s);" in ran_out[1] and "copies = 0, next_slice = live;" in ran_out[1]
    assert re.search(r"if \(copies == 0\) \{\s*if \(next_slice >= live\) return;", code)  # (fill)
    spin = _code("om_ptx.cuh").split("bool mbar_wait_or_stop")[1].split("\n}")[0]
    assert spin.index("if (*stop) return false;") < spin.index("global_timer_ns() - t0") < spin.index("*stop = 1;")


def test_the_phases_of_the_stages_under_way():
    """Chunk k lies in stage k % n, in its phase k // n: those of the next n - 1 chunks, as the end of a wait names them."""
    for n in (2, 4):
        for k in range(64):
            stage, phase = k % n, k // n & 1
            for i in range(1, n):
                assert ((stage + i) % n, phase ^ (stage + i >= n)) == ((k + i) % n, (k + i) // n & 1)
