"""Rules that the kernels' sources keep, read from the sources themselves (no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_298_gb300", "csrc")
SOURCES = sorted(sum((glob.glob(os.path.join(CSRC, p)) for p in ("*.cu", "*.cuh", "*.h", "*.cpp")), []))


def code_of(path):
    """The file without its comments."""
    with open(path) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_to_several_ctas(path):
    """The library is what every replica of a run on several GPUs loads, and the addresses that its kernels copy from are the
    caller's: no copy is sent to more than one CTA."""
    assert "multicast" not in code_of(path)


@pytest.mark.parametrize("path", [p for p in SOURCES if "tcgen05.alloc" in code_of(p)], ids=os.path.basename)
def test_dependents_launch_after_tensor_memory_is_held(path):
    """A kernel's next one may become resident once every CTA has let it, and may take tensor memory before it waits for the
    kernel's end.  So a CTA lets it from the warp that allocates, after the allocation (which waits until it succeeds): else a
    CTA that still waits for its columns and the one that took them would wait for each other."""
    code = code_of(path)
    allocs = [m.start() for m in re.finditer(r"tcgen05\.alloc\.", code)]
    assert allocs
    for at in allocs:
        guard = code.rfind("if (", 0, at)
        assert re.match(r"if \(warp == 0\) \{\s*asm", code[guard:]), "one warp allocates"
        trigger = code.find("griddepcontrol.launch_dependents", at)
        assert trigger > 0
        line = code[code.rfind("\n", 0, trigger):trigger]
        assert line.strip() == 'if (warp == 0) asm volatile("', "the allocating warp lets the dependents launch"
        assert code.find("griddepcontrol.launch_dependents", 0, at) < 0 or "__global__" in code[
            code.find("griddepcontrol.launch_dependents"):at], "not before the allocation"


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_the_device_says_how_many_sms_it_has(path):
    assert not re.search(r"\b1(48|52)(LL|L|u)?\b", code_of(path))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_load_that_a_running_kernel_may_outdate(path):
    """A kernel may be resident while the one before it still writes block tables, slots, boundaries, codes or factors (each lets
    its dependents start early).  A load through the read-only path is only defined for what nobody writes while its kernel
    lives, from before its wait on, and may be moved in front of that wait: no kernel has one, nor gives the compiler leave
    to make one."""
    code = code_of(path)
    assert not re.search(r"__ldg\b|__ldlu\b|\.nc\b|__restrict__", code)
