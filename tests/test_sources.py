"""Rules of the CUDA sources that no run shows reliably (no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gate_up_swiglu_gb300", "csrc")


def asm_statements(text):
    """(line, statement) of every inline assembly statement."""
    text = re.sub(r"//[^\n]*", "", text)
    for m in re.finditer(r"\basm\b(\s+volatile)?\s*\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text.count("\n", 0, m.start()) + 1, text[m.start():at]


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_shared_memory_loads_stay_behind_their_barriers(path):
    """What another thread or CTA wrote to shared memory is read by assembly that the
    compiler may neither drop, repeat nor move over a barrier."""
    for line, s in asm_statements(open(path).read()):
        if re.search(r"\bld\.shared\b", s):
            assert re.match(r"asm\s+volatile", s) and '"memory"' in s, f"{os.path.basename(path)}:{line}"


@pytest.mark.parametrize("name,kernel_name,roles,sites", [
    # scheduler: slot, answer, bad answer; producer: tile, stage, landing; MMA: tile, its two, the last commit
    ("grouped_mm.cu", "grouped_mm_kernel", ("if (warp == kScheduler)", "// ---- epilogue"), 7),
    ("fc1_swiglu.cu", "fc1_swiglu_pair_kernel", ("// ---- producer", "// ---- epilogue"), 10)])
def test_a_pair_that_gave_up_stays_until_its_loads_have_landed(name, kernel_name, roles, sites):
    """The threads of a pair that issue work tell both CTAs that a wait ran out, and after
    their last meeting one thread of each waits for what is in flight."""
    text = open(os.path.join(CSRC, name)).read()
    kernel = text[text.index(kernel_name + "(const __grid_constant__"):]
    kernel = kernel[:kernel.index("\n}\n")]
    last = kernel[kernel.rindex("cluster_sync();"):]
    assert "if (threadIdx.x == 0 && *abort_flag) settle();" in last
    part = kernel[kernel.index(roles[0]):kernel.index(roles[1])]
    assert part.count("give_up();") == sites and "*abort_flag = 1" not in part
    assert re.search(r"void settle\(\) \{[^}]*kSettleNs", open(os.path.join(CSRC, "tc_pair.cuh")).read())


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_shuffles_name_their_lanes(path):
    """No mask of the lanes that happen to be converged."""
    assert "__activemask" not in open(path).read()


def test_columns_of_an_accumulator_are_given_free_after_its_products():
    """The 4-bit pair kernel's epilogue warps arrive for a tile once each, behind their wait for
    the tile's products: ahead of it a warp could arrive twice for one tile, in the place of one
    that has still to read the columns that the next tile overwrites."""
    text = open(os.path.join(CSRC, "mx4_mm.cu")).read()
    kernel = text[text.index("mx4_pair_kernel(const __grid_constant__"):]
    loop = kernel[kernel.index("// ---- epilogue"):kernel.index("\n}\n")]
    wait = loop.index("wait(acc_full0")
    assert "(acc_empty_leader)" in loop[wait:] and "(acc_empty_leader)" not in loop[:wait]
    assert loop.count("(acc_empty_leader)") == 1 and loop.index("if (!sharing) read();") < loop.index("if (sharing) read();")
