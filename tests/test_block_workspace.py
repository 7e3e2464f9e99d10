"""What the norm's gradient asks of the stream's workspace."""
import pytest

import stream_compaction_gb300 as sc


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_gb300 import build
    build.build()
    return sc.load()


@pytest.mark.parametrize("dtype", [sc.SC_F32, sc.SC_BF16])
@pytest.mark.parametrize("channels", [8193, 16384, 131072])
def test_wide_rows_ask_for_what_their_sums_fill(lib, channels, dtype):
    """Rows of more than 8192 channels have at most 32 partial sums of dweight and dbias."""
    ask = lambda rows: lib.sc_layer_norm_grad_workspace_bytes(rows, 1, channels, dtype)  # noqa: E731
    row = 2 * channels * 4
    for rows in (2, 31, 32):
        assert ask(rows) == ask(1) + (rows - 1) * row
    for rows in (33, 1000, 1 << 20):
        assert ask(rows) == ask(32)
    assert lib.sc_layer_norm_grad_workspace_bytes(4, 1 << 18, channels, dtype) == ask(32)


@pytest.mark.parametrize("channels", [1, 4096, 8192])
def test_other_rows_have_one_a_cta(lib, channels):
    ask = lambda rows: lib.sc_layer_norm_grad_workspace_bytes(rows, 1, channels, sc.SC_F32)  # noqa: E731
    assert ask(400) == ask(1) + 399 * 2 * channels * 4 and ask(1 << 20) >= ask(400)
