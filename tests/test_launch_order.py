"""Kernels launched with programmatic dependent launch start while the kernel
in front of them may still run: only what stands behind griddepcontrol.wait
sees that kernel's writes, whether it was one of the library's or the
caller's.  So every kernel waits before it reads or writes global memory, and
before any of its threads leaves (a grid that is through without having waited
says nothing about the grid in front of it).  Checked on the sources."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_424_b200", "csrc")
# device functions that read the call's arrays
READERS = r"\b(scheduled_seq|seq_split|int4_seq|checked_len|checked_block|row_range|query_row|load_\w*q\w*|flag_error)\s*\("
# fields of the parameter structures that point to global memory
FIELDS = r"\bp\.(out|q|k|v|q_out|k_out|k_cache|v_cache|block_tables|context_lens|ws_o|ws_lse|seq_order|slots|positions|inv_freq|key|value)\b"


def matching(text, at, opening="{", closing="}"):
    """Index behind the bracket that closes the one at `at`."""
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == opening) - (text[i] == closing)
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced source")


def kernels():
    found = []
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        launched = set(re.findall(r"launch_pdl\(\s*(\w+)", text)) | set(re.findall(r"kern = (\w+)", text))
        for m in re.finditer(r"__global__\s+void\s+(?:__launch_bounds__\()?", text):
            at = m.end()
            if m.group().endswith("("):
                at = matching(text, at - 1, "(", ")")
            name = re.match(r"\s*(\w+)\s*\(", text[at:])
            start = text.index("(", at)
            end = matching(text, start, "(", ")")
            body = text.index("{", end)
            if name and text[end:body].strip() == "":
                found.append((os.path.basename(path), name.group(1), name.group(1) in launched, text[start:end],
                              text[body:matching(text, body)]))
    return found


def before_wait(body):
    """What a kernel does before its wait: the text up to it, without the bodies of functions that are only defined there."""
    text = body[:body.index("pdl_wait();")]
    while True:
        m = re.search(r"auto \w+ = \[&\]\s*\([^)]*\)[^{]*\{", text)
        if not m:
            return text
        text = text[:m.start()] + text[matching(text, m.end() - 1):]


def test_the_sources_kernels_are_found():
    names = {k[1] for k in kernels() if k[2]}
    assert {"decode_tc_kernel", "decode_part_kernel", "merge_part_kernel", "decode_int4_kernel", "decode_int4_balanced_kernel", "merge_int4_kernel",
            "rope_kernel", "write_int4_kernel", "gather_kernel", "copy_blocks_kernel", "swap_blocks_kernel"} <= names


@pytest.mark.parametrize("path,name,launched,params,body", kernels(), ids=[k[1] for k in kernels()])
def test_kernels_wait_before_they_touch_memory_or_leave(path, name, launched, params, body):
    if not launched:
        pytest.skip("not launched while another kernel may run")
    assert "pdl_wait();" in body, f"{path}: {name} does not wait for the kernel in front of it"
    text = before_wait(body)
    assert not re.search(r"\breturn\b", text), f"{path}: {name} may leave without having waited"
    assert not re.search(READERS, text), f"{path}: {name} reads its inputs before it waits"
    reads = re.sub(r"= reinterpret_cast<[^>]*>\(" + FIELDS + r"\);", "", text)  # a pointer kept for later
    assert not re.search(FIELDS, reads), f"{path}: {name} takes an array before it waits"
    for pointer in re.findall(r"\*\s*(?:__restrict__\s*)?(\w+)\s*[,)]", params):
        assert not re.search(r"\b%s\s*\[|\*\s*%s\b" % (pointer, pointer), text), f"{path}: {name} reads {pointer} before it waits"
