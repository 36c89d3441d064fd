"""Rules of the kernel sources that no run can show to be kept: breaking them is undefined, and may
still give the right values.  CPU only."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_decode_ls_b200", "csrc")

ALIGNED = re.compile(r"\b(?:tmem_ld32|tmem_ld64|tmem_st32)\(|\"bar\.sync ")
WHOLE = re.compile(r"__syncwarp\(\)|__(?:all|any)_sync\(0xffffffffu")


def code(name):
    """The file without comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def innermost_loop(text, at):
    """Start and end of the body of the innermost `for (...) {` around offset `at`."""
    found = None
    for m in re.finditer(r"\bfor \([^{};]*;[^{};]*;[^{};]*\) \{", text[:at]):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        if i > at:
            found = (m.end(), i)
    return found


def test_aligned_instructions_come_behind_a_point_where_the_warp_is_whole():
    """tcgen05.ld / st and bar.sync are .aligned: all lanes of a warp have to execute them together.  In a
    loop some of whose lanes take a branch of their own (rows that are not live), nothing brings
    the lanes together again before its next pass but a barrier of the warp."""
    text = code("prefix_attn.cuh")
    seen = 0
    for m in ALIGNED.finditer(text):
        loop = innermost_loop(text, m.start())
        if loop is None:
            continue
        body = text[loop[0]: loop[1]]
        if not re.search(r"\bif \((?:!)?(?:live|lane|nv)\b|\bcontinue;", body):
            continue
        seen += 1
        before = text[loop[0]: m.start()]
        at = max([w.end() for w in WHOLE.finditer(before)], default=None)
        assert at is not None, text[m.start() - 200: m.end()]
        # and no lane leaves the others between that point and the instruction
        assert not re.search(r"\bif \((?:!)?(?:live|lane|nv)\b", before[at:]), before[at:]
    assert seen >= 3  # the S tiles, the epilogue's columns, the barrier before them
