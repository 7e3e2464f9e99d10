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


def test_the_common_convolutions_do_not_spill():
    """Registers of the forward kernel for aligned rows of up to four taps, as the
    assembler reports them: a bound that one element type can live with made another
    keep its elements in memory (152 bytes a thread)."""
    import subprocess
    from stream_compaction_gb300 import build
    cmd = [build.nvcc()] + build.NVCC_FLAGS + ["-Xptxas", "-v", "-c", os.path.join(CSRC, "sc_conv.cu"), "-o", os.devnull]
    log = subprocess.run(cmd, capture_output=True, text=True, check=True).stderr
    found = re.findall(r"Compiling entry function '(\w*conv_kernelI\w*?Li4ELb1ELb0E\w*)'.*?(\d+) bytes spill stores", log, re.S)
    assert len(found) == 3, found
    assert all(int(spilled) <= 16 for _, spilled in found), found
