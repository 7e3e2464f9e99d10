"""Host threads that call the sequence operators at the same time, each on a stream of
its own, as include/sc_scan.h allows."""
import threading

import pytest
import torch

import stream_compaction_gb300 as sc
from gpu_helpers import ensure_lib

pytestmark = pytest.mark.gpu


def test_embedding_gradients_of_different_tables():
    """Tables whose sorts need different amounts of shared memory (digits of 10 and of 9
    bits): neither call may see the other's.  Through the C ABI, which ctypes calls
    without the interpreter's lock."""
    lib = ensure_lib()
    tokens, dim, calls = 500, 8, 3000
    work = []
    for vocab in (1000, 131072):
        gen = torch.Generator(device="cuda").manual_seed(vocab)
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device="cuda")
        dout = torch.randn(tokens, dim, generator=gen, device="cuda")
        work.append((vocab, ids, dout, torch.empty(vocab, dim, device="cuda"), torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    start = threading.Barrier(2)

    def call(vocab, ids, dout, out, stream, statuses):
        start.wait()
        for _ in range(calls):
            statuses.append(lib.sc_embed_grad(ids.data_ptr(), 1, tokens, sc.SC_F32, dout.data_ptr(), dim, vocab, dim, 1.0,
                                              sc.SC_F32, out.data_ptr(), dim, 0, stream.cuda_stream))

    threads = [threading.Thread(target=call, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for vocab, ids, dout, out, stream, statuses in work:
        assert len(statuses) == calls and set(statuses) == {sc.SC_OK}, (vocab, calls - statuses.count(sc.SC_OK))
        want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, ids, dout.double())
        assert torch.allclose(out.double(), want, rtol=1e-6, atol=1e-5)  # few terms of O(1) a row
        assert sc.sc_release_stream(stream.cuda_stream) == sc.SC_OK
