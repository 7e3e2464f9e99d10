"""The block operators from several host threads, a stream each: the results of one thread."""
import threading

import pytest
import torch

import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


def _inputs(n):
    gen = torch.Generator(device="cuda").manual_seed(n)
    rand = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return {"x": rand(2, 300 + 40 * n, 512 + 8 * n).bfloat16(), "g": rand(2, 300 + 40 * n, 512 + 8 * n).bfloat16(),
            "w": rand(512 + 8 * n), "ids": torch.randint(-1, 9, (2 * (300 + 40 * n), 2), generator=gen, device="cuda"),
            "share": torch.rand(2 * (300 + 40 * n), 2, generator=gen, device="cuda")}


def _all(c):
    saved, kept = sc.layer_norm_saved(c["x"]), sc.gated_scan_saved(c["x"])
    y, s = sc.layer_norm(c["x"], c["w"], residual=c["g"], saved=saved)
    grads = sc.layer_norm_grad(c["g"], s, c["w"], saved=saved, dsum=c["x"])
    h = sc.gated_scan(y, c["g"], saved=kept)
    back = sc.gated_scan_grad(s, y, c["g"], saved=kept)
    order = sc.expert_sort(c["ids"], 9)
    rows = sc.expert_gather(h.flatten(0, 1), order)
    out = sc.expert_combine(rows, order, c["share"])
    last = sc.expert_combine_grad(out, rows, order, c["share"])
    return [y, s, h, rows, out, *order, *grads.values(), *back.values(), *last.values()]


def test_threads():
    ensure_lib()
    inputs = [_inputs(n) for n in range(4)]
    want = [_all(c) for c in inputs]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = _all(inputs[n])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                        wrong.append(n)
            sc.sc_release_stream(int(stream.cuda_stream))
        except Exception as e:  # noqa: BLE001  (shown below, in the test's thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong, (errors, wrong)
