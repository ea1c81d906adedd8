"""Host threads that call the operators at the same time, each on a stream of its own: what one
call sets for a kernel does not reach another's launch."""

import threading

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def side_by_side(calls, repeats):
    """Every call `repeats` times, each in a thread and on a stream of its own; the threads start
    together. Returns the last results."""
    torch.cuda.synchronize()
    start = threading.Barrier(len(calls))
    last, errors = [None] * len(calls), []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for _ in range(repeats):
                    last[i] = calls[i]()
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append((i, e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]
    return last


def test_routers_of_one_block_with_few_and_many_experts():
    # one token a warp: the counters of 1024 experts take 70 KB, those of 600 two thirds of that. The C
    # calls alone, so that the threads meet in them.
    kept, calls, want = [], [], []
    execute = pgg.load().pgg_route_execute
    for t, g in [(64, 1024), (64, 600)] * 4:
        logits = torch.randn(t, g, device="cuda")
        want.append([x.clone() for x in pgg.route(logits, 10)[:4]])
        out = [torch.empty_like(x) for x in want[-1]]
        ws = torch.empty(pgg.pgg_route_workspace_size(t, g, 10), dtype=torch.uint8, device="cuda")
        kept.append((logits, out, ws))
        stream = torch.cuda.Stream()
        args = (logits.data_ptr(), None, t, g, 10, 0, pgg.PGG_F32, 0, 1, 1.0, ws.data_ptr(),
                ws.numel(), *(x.data_ptr() for x in out), stream.cuda_stream)

        def call(args=args, out=out):
            rc = execute(*args)
            if rc != 0:
                raise pgg.PggError(rc, "pgg_route_execute")
            return out

        calls.append(call)
    got = side_by_side(calls, 20000)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_adapter_calls_with_few_and_many_adapters():
    calls, want = [], []
    for T, A in ((300, 1000), (700, 600), (5000, 300), (300, 900)):
        x = torch.randn(T, 64, device="cuda").bfloat16()
        w = torch.randn(64, 64, device="cuda").bfloat16() / 8
        a = torch.randn(A, 64, 8, device="cuda").bfloat16() / 8
        b = torch.randn(A, 64, 8, device="cuda").bfloat16() / 3
        ad = torch.randint(-1, A, (T,), device="cuda")
        out = torch.empty(T, 64, device="cuda", dtype=torch.bfloat16)
        ws = torch.empty(pgg.pgg_adapters_workspace_size(T, 64, 64, 8, A, pgg.PGG_BF16),
                         dtype=torch.uint8, device="cuda")
        args = (x, w, a, b, ad)
        calls.append(lambda args=args, out=out, ws=ws: pgg.adapters(*args, out=out, workspace=ws))
        want.append(pgg.adapters(*args)[0].clone())
    got = side_by_side(calls, 1500)
    for (y, ws), w in zip(got, want):
        assert pgg.status(ws) == 0
        assert torch.equal(y.view(torch.int16), w.view(torch.int16))
