"""New tensors of the sequence operators come from torch where somebody asks for that."""
import pytest

torch = pytest.importorskip("torch")

import stream_compaction_gb300 as sc  # noqa: E402


def _lib():
    from stream_compaction_gb300 import build
    build.build()
    sc.load()


def test_a_buffer_for_a_host_tensor():
    """selective_scan_saved takes its tensor's device, whichever that is."""
    _lib()
    saved = sc.selective_scan_saved(torch.zeros(1, 20, 4), torch.zeros(4, 3))
    assert saved.device.type == "cpu" and saved.dtype == torch.float32 and saved.shape == (1, 2, 2, 4, 4)


def _calls():
    x = torch.zeros(2, 20, 8, device="cuda")
    A, B = -torch.ones(8, 3, device="cuda"), torch.zeros(2, 20, 1, 3, device="cuda")
    ids = torch.zeros(5, dtype=torch.int64, device="cuda")
    order = sc.expert_sort(ids[:, None], 3)
    return {
        "embed": lambda: sc.embed(ids, x[0]),
        "causal_conv": lambda: sc.causal_conv(x, torch.zeros(8, 4, device="cuda")),
        "selective_scan": lambda: sc.selective_scan(x, x, A, B, B),
        "selective_scan_saved": lambda: sc.selective_scan_saved(x, A),
        "gated_scan": lambda: sc.gated_scan(x, x.clone()),
        "layer_norm": lambda: sc.layer_norm(x, residual=x),
        "expert_gather": lambda: sc.expert_gather(x[0, :5], order),
    }


@pytest.mark.gpu
def test_dispatch_modes_see_them():
    from torch.utils._python_dispatch import TorchDispatchMode

    class Seen(TorchDispatchMode):
        made = 0

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.made += func is torch.ops.aten.empty.memory_format
            return func(*args, **(kwargs or {}))

    _lib()
    for name, call in _calls().items():
        want = call()
        with Seen() as seen:
            before = seen.made
            got = call()
        assert seen.made > before, name
        for a, b in zip(*((t,) if torch.is_tensor(t) else t for t in (got, want))):
            assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device, name


@pytest.mark.gpu
def test_deterministic_algorithms_fill_them():
    _lib()
    x = torch.zeros(2, 20, 8, device="cuda")
    torch.use_deterministic_algorithms(True)
    try:
        saved = [sc.selective_scan_saved(x, torch.zeros(8, 3, device="cuda")), sc.gated_scan_saved(x), sc.layer_norm_saved(x)]
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(t.isnan().all() for t in saved)
