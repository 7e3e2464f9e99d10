"""Facts about the sequence operators' sources that no call can show on one kind of GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "stream_compaction_gb300", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if re.match(r"sc_(seq|embed|conv|ssm)", f))


def code(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_the_device_is_asked_for_its_multiprocessors():
    """Splits of the work follow the device in use: no count of one GPU's multiprocessors in them."""
    assert len(FILES) > 10
    for name in FILES:
        assert not re.search(r"\b152(ll)?\b", code(name)), name
    assert any("seq_sms()" in code(name) for name in FILES)
