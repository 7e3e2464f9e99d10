"""Facts about the block operators' sources that no call can show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "stream_compaction_gb300", "csrc")


def code(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def blocks_around(text, at):
    """What stands before each brace that is open at a position."""
    opened = []
    for m in re.finditer(r"[{}]", text[:at]):
        if m.group() == "{":
            opened.append(text[max(text.rfind(c, 0, m.start()) for c in ";{}") + 1:m.start()].strip())
        else:
            opened.pop()
    return opened


def test_a_stage_is_written_only_for_a_tile_that_is_there():
    """A stage's results leave by copies that are waited for where it is filled again.  A warp
    without a tile in the last round fills none, so it must not write to the stage either:
    the copy of earlier results may still be reading it."""
    text = code("sc_gated.cuh")
    puts = [m.start() for m in re.finditer(r"\b[xg]r\.put\(", text)]
    assert len(puts) == 3  # y; dx and dgate
    for at in puts:
        assert any(b.endswith("if (valid > 0)") for b in blocks_around(text, at)), text[at - 200:at]
    stores = [m.start() for m in re.finditer(r"\btma_store_3d\(&maps", text)]
    assert len(stores) == 3
    for at in stores:
        assert any(b.endswith("if (valid > 0)") for b in blocks_around(text, at)), text[at - 200:at]
