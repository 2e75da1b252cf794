"""The tensor-core scan's decay vectors arrive by an asynchronous copy of their own, which other copies of the same
chunk may overtake.  Whether a missing wait shows on a GPU is a matter of timing, so the wait is looked for in the
source: the vectors' place in shared memory is known to two places only, the copy and the accessor that waits for it,
and every role takes them from that accessor before it reads one."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_18_b200",
                      "csrc", "ssm_scan_tc.cuh")


def kernel():
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    start = text.index("scan_kernel(const __grid_constant__")
    return text[start:text.index("inline PFN_cuTensorMapEncodeTiled")]


def test_the_vectors_are_reached_through_their_wait_only():
    lines = [l.strip() for l in kernel().splitlines() if "Lay::vec " in l]
    assert len(lines) == 2, lines
    assert any("bulk_load(" in l and "bar(VR + cc % kV)" in l for l in lines)
    body = re.search(r"auto vectors = \[&\]\(int cc\) \{(.*?)\};", kernel(), re.S)
    assert body and "Lay::vec " in body.group(1)
    first, second = [l.strip() for l in body.group(1).strip().splitlines()]
    assert first == "wait(VR + cc % kV, cc / kV);" and second.startswith("return ")


def test_every_role_takes_the_vectors_before_it_reads_them():
    use = re.compile(r"\[V[UWEPTD]\b|\bvec \+ V[UWEPTD]\b")
    roles = re.split(r"regs_(?:dec|inc)<\d+>\(\);", kernel())     # each warpgroup's part starts with its registers
    readers = [r for r in roles if use.search(r)]
    assert len(readers) == 3                                 # X'; P and the state; y
    for r in readers:
        taken = r.index("vectors(cc)")
        assert taken <= use.search(r).start()
        assert r.index("for (int c = 0; c < it.nc") < taken   # in every chunk
