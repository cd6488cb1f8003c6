"""Calls that answer with a quantized model, from several host threads at once."""
import threading

import pytest
import torch

from tests.test_gemv_gpu import BF, FP, U  # noqa: F401

pytestmark = pytest.mark.gpu


def test_products_from_two_threads(U):  # noqa: F811
    """Products of one kernel that take differing amounts of shared memory
    (few and many chunks of a row), each thread on a stream of its own: every
    call runs, and gives what it gives alone."""
    sizes = [(1, 2048), (8, 2048), (4, 64), (8, 640)]
    w = {k: U.ufp4_quantize(torch.randn(256, k, device="cuda"), U.UFP4_E1M2) for _, k in sizes}
    x = [torch.randn(t, k, device="cuda").to(BF) for t, k in sizes]
    want = [U.ufp4_gemv(a, w[a.shape[1]], dtype=BF) for a in x]
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(4), []

    def run(i):
        s, a = torch.cuda.Stream(), x[i]
        start.wait()
        try:
            for _ in range(3000):
                y = U.ufp4_gemv(a, w[a.shape[1]], dtype=BF, stream=s)
            s.synchronize()
            if not torch.equal(y, want[i]):
                wrong.append((i, "other results"))
        except U.UFP4Error as e:
            wrong.append((i, str(e)))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
