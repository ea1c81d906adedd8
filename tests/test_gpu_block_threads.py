"""The norms around a block and the clipping called from several threads at once, each on its own
stream with its own sizes: the results of the calls alone."""

import threading

import torch
import pytest

import permute_grouped_gemm_gb300 as pgg
import test_gpu_block_norm as norm
import test_gpu_clip as clip
from test_gpu_block_norm import built  # noqa: F401

pytestmark = pytest.mark.gpu


def norm_call(**kw):
    s = norm.case(**kw)

    def run():
        r, h = pgg.block_norm(s["x"], s["y"], **norm.kwargs(s))
        got, _ = pgg.block_norm_grad(s["d_r"], s["d_h"], r, s["y"], **norm.kwargs(s))
        return [r, h] + [t for t in got.values() if t is not None]
    return run


def clip_call(sizes, seed):
    grads = clip.grads_of(sizes, seed=seed)
    return lambda: list(pgg.clip_grads(grads, 0.5, out=[torch.empty_like(g) for g in grads])[1])


def test_threads():
    calls = [norm_call(T=300, H=1024, post="layer", pre="layer", gate="full"),
             norm_call(T=40, H=7168, params="bf16", bias=False), norm_call(T=90, H=333, gate="token"),
             clip_call([100000, 7, 33], 1), clip_call([50 + i for i in range(600)], 2)]
    want = [run() for run in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = calls[i]()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
