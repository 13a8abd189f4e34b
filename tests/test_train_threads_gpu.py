"""Several host threads on one stream, none with a workspace of its own: every result is the
one of a call alone."""

import threading

import pytest
import torch

from gpu_util import DEV
from train_util import normal
from test_train_gpu import weight, w  # noqa: F401

pytestmark = pytest.mark.gpu


def test_threads_on_one_stream(w):  # noqa: F811
    K, F, V = 256, 512, 2000
    up, head = weight(w, K, 2 * F, "bf16", 128).packed, weight(w, K, V, "bf16", 128).packed
    work, want = [], []
    for i, M in enumerate((3, 20, 40, 130, 300, 700)):                # needs of different sizes
        x, _ = normal(500 + i, (M, K), "bf16")
        dh, _ = normal(600 + i, (M, F), "bf16")
        lab = torch.arange(M, dtype=torch.int32, device=DEV) * 2
        ids = (lab[:, None] + torch.arange(4, dtype=torch.int32, device=DEV)[None, :]).to(torch.int32).contiguous()
        top = torch.zeros((M, 4), device=DEV)

        def call(x=x, dh=dh, lab=lab, ids=ids, top=top):
            return (*w.w4a16_cross_entropy(x, lab, head, V, grad=True), *w.w4a16_distill(x, ids, top, head, V, grad=True),
                    w.w4a16_gated_grad(x, dh, up, F))
        work.append(call)
        want.append(call())
    torch.cuda.synchronize()
    wrong = []

    def thread(first):
        for n in range(30):
            i = (first + n) % len(work)
            got = work[i]()
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want[i])):
                wrong.append(i)
    threads = [threading.Thread(target=thread, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
