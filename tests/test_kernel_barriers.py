"""Order of a kernel's set-up, read from its source: mbarriers are initialised, made visible and handed to the block's other
warps by a barrier of the block before anything uses them.  (On a GPU the loads behind it usually hide a missing one.)"""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "coalesced_packed_attention_gb300", "csrc")
USES = r"\bmbar_(?:arrive|wait|try_wait|arrive_expect_tx)\(|\bbulk_load\(|\btma_load_\w+\(|\bmma_commit\w*\(|cp\.async\.bulk|\bproduce = "


def body(text, at):
    """From the brace that opens behind `at` to the one that closes it."""
    start = text.index("{", text.index(")", text.index("zl_", at)))
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError("a kernel without an end")


def kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"__global__", text):
            b = body(text, m.start())
            if "mbar_init(" in b:
                yield pytest.param(b, id=f"{os.path.basename(path)}:{re.search(r'zl_[a-z0-9_]+kernel', text[m.start():]).group()}")


def test_there_are_such_kernels():
    assert len(list(kernels())) >= 6


@pytest.mark.parametrize("text", list(kernels()))
def test_barriers_are_initialised_before_any_warp_uses_them(text):
    last = max(m.end() for m in re.finditer(r"\bmbar_init\(", text))
    assert not re.search(USES, text[:last])
    fence, sync = text.find("fence_mbar_init();", last), text.find("__syncthreads();", last)
    use = re.search(USES, text[last:]).start() + last
    assert last < fence < sync < use
    # one thread initialises them all, and fences behind that
    block = text[text.rindex("== 0) {", 0, text.index("mbar_init(")) + len("== 0) "):fence]
    assert block.count("{") == block.count("}") + 1


def test_aligned_instructions_come_behind_a_whole_warp():
    """Barriers of a cluster and loads from tensor memory are .aligned: all lanes of a warp execute them together."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"barrier\.cluster\.arrive[a-z.]*aligned", text):
            assert "__syncwarp();" in text[text.rindex("{", 0, text.rindex("asm", 0, m.start())):m.start()], path
        # where lanes leave a loop's body early, they wait for one another ahead of the next load
        for m in re.finditer(r"(.*)\s*tmem_ld\w+\([^;]*;\s*tmem_ld_wait\(\);\s*if \([^;]*\) continue;", text):
            assert m.group(1).strip() == "__syncwarp();", path
