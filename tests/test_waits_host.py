"""A bounded wait ends for every lane by itself, so its answer may differ
within a warp when a phase completes at the time limit.  Lanes that go on to
the warp's collective instructions (tcgen05.ld / st, votes, exchanges) without
the others hang, which no test can show on a device: read from the sources
instead.  A wait of one lane stands in a branch of one thread, any other in a
form that votes."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sequence_parallelism_striped_gb300",
                    "csrc")
LANE_WAIT = re.compile(r"\b(mbar_try_wait|mbar_wait_timed|mbar_wait|win_wait_timed|win_wait|bwd_wait)\s*(<\w+>)?\s*\(")
ONE_THREAD = re.compile(r"\blane == 0\b|\bthreadIdx\.x == 0\b")
REST_RETURNS = re.compile(r"if \(threadIdx\.x != \w+\) return;")
WAIT_FUNCTION = re.compile(r"\bbool \w*wait\w*\([^()]*$|\bbool \w*wait\w*\([^()]*\)\s*$")


def lane_waits_of_many(text):
    """Lines of waits whose lanes may part: (line, source)."""
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), text)
    stack, header, bad = [], 0, []  # open blocks: (header text, where the block begins)
    for m in re.finditer(r"[{};]|" + LANE_WAIT.pattern, text):
        c = m.group()
        if c == "{":
            stack.append((text[header:m.start()], m.end()))
        elif c == "}":
            if stack:
                stack.pop()
        if c in "{};":
            # the ';' of a for's header does not end the header
            if c != ";" or text[header:m.start()].count("(") == text[header:m.start()].count(")"):
                header = m.end()
            continue
        if text[:m.start()].endswith("bool "):
            continue  # a definition
        if any(WAIT_FUNCTION.search(h.strip()) or ONE_THREAD.search(h) for h, _ in stack):
            continue
        if any(REST_RETURNS.search(text[b:m.start()]) for _, b in stack[1:]):
            continue
        if re.search(r"__all_sync\(0xffffffffu, $", text[:m.start()]):
            continue
        line = text.count("\n", 0, m.start())
        bad.append((line + 1, text.split("\n")[line].strip()))
    return bad


def test_the_reader_of_sources():
    src = """namespace striped {
bool mbar_wait(int a);
__device__ __forceinline__ bool x_wait(uint32_t bar, const WaitCtl &w) { return mbar_wait(bar); }
__global__ void k(int n) {
    if (warp == 0 && lane == 0) {
        for (int i = 0; i < n; ++i) mbar_wait(a);  // mbar_wait(
    } else if (warp == 1) {
        ok = __all_sync(0xffffffffu, mbar_wait(a));
    } else {
        for (int i = 0; i < n; ++i)
            if (!bwd_wait(a)) break;
        auto f = [&](int i) -> bool {
            if (!win_wait<HD>(a)) return false;
        };
    }
}
}"""
    assert [n for n, _ in lane_waits_of_many(src)] == [11, 13]


@pytest.mark.parametrize("name", ["attn_window_fwd.cu", "attn_window_bwd.cu", "attn_decode.cu", "norm_rope.cu",
                                  "common.cuh", "attn_fwd_tc.cu", "attn_fwd_pair.cu", "attn_bwd_tc.cu"])
def test_warps_wait_as_one(name):
    with open(os.path.join(CSRC, name)) as f:
        bad = lane_waits_of_many(f.read())
    assert not bad, "\n".join(f"{name}:{n}: {s}" for n, s in bad)
