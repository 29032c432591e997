"""The device code's inline assembly says which fixed registers it writes."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_ep_get_dispatch_amd", "csrc")


def statements(text):
    """Every asm statement of ``text``, from its opening bracket to its closing one."""
    for m in re.finditer(r"\basm\s+volatile\s*\(", text):
        depth, i = 1, m.end()
        quoted = False
        while depth:
            c = text[i]
            if c == '"' and text[i - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            i += 1
        yield text[m.end():i - 1]


def test_every_block_that_writes_m0_clobbers_it():
    """The compiler may hold a value of its own in M0 (an index, the place of a load
    to LDS), which a block that writes it without saying so would replace."""
    writes = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            for s in statements(f.read()):
                if re.search(r"s_mov_b32 m0\b", s):
                    writes += 1
                    clobbers = s.rsplit(":", 1)[1]
                    assert '"m0"' in clobbers, (os.path.basename(path), s)
    assert writes
