"""The global norm of a list of gradients and the clipping by it, against 64 bits.

Bounds, u = 2^-24: 32 squares are summed in fp32 (at most 10 u of the sum), the rest in fp64; the
norm is rounded once, so 8 u of it; c is two quotients and products (4 u), and an output is rounded
once more, by half a step of its type.
"""

import math

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = (torch.bfloat16, torch.float32, torch.float16)


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from permute_grouped_gemm_gb300 import build as pbuild
    pbuild.build()
    pgg.load()


def grads_of(sizes, types=TYPES, std=0.1, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * std).to(types[i % len(types)])
            for i, n in enumerate(sizes)]


def exact_norm(grads, scale=1.0):
    return abs(scale) * math.sqrt(math.fsum(float(g.double().square().sum()) for g in grads))


def check(grads, max_norm=1.0, scale=1.0, eps=1e-6, **kw):
    kept = [g.clone() for g in grads]
    norm, out, ws = pgg.clip_grads(grads, max_norm, eps=eps, scale=scale, **kw)
    assert pgg.status(ws) == 0
    want = exact_norm(kept, scale)
    assert abs(float(norm) - want) <= 8 * U * want
    assert float(pgg.grad_norm(kept, scale=scale)[0]) == float(norm)
    c = scale * min(1.0, max_norm / (want + eps))
    for g, o in zip(kept, out):
        half = torch.finfo(o.dtype).eps / 2
        x = g.double() * c
        bound = x.abs() * (half + 16 * U) + torch.finfo(o.dtype).smallest_normal * half * 2
        assert o.dtype == g.dtype and o.shape == g.shape
        assert bool(((o.double() - x).abs() <= bound).all())
    return float(norm), out


@pytest.mark.parametrize("sizes", [
    [1], [7], [31, 1, 0, 5], [16384], [16385, 16383], [1 << 20, 3, 100000], [0, 0, 4],
    [(37 * i) % 97 + 1 for i in range(40)], [5000 + i for i in range(600)], [20_000_003]])
@pytest.mark.parametrize("scale", [1.0, 1 / 1024, -2.0])
def test_lists(sizes, scale):
    check(grads_of(sizes, std=0.1), scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("max_norm", [0.0, 0.3, 1e9, float("inf")])
def test_types_and_limits(dtype, max_norm):
    check(grads_of([3000, 70000, 11], (dtype,)), max_norm)


def test_out_of_place_and_in_place():
    grads = grads_of([40000, 9, 333])
    kept = [g.clone() for g in grads]
    out = [torch.full_like(g, 5) for g in grads]
    _, got = check(grads, 0.5, out=out)
    assert got is out and all(torch.equal(a, b) for a, b in zip(grads, kept))
    _, got = check(grads, 0.5)
    assert got is grads and all(torch.equal(a, b) for a, b in zip(grads, out))
    # a norm below the limit leaves what is its own output, and copies the rest
    now = [g.clone() for g in grads]
    check(grads, 10.0)
    assert all(torch.equal(a, b) for a, b in zip(grads, now))
    check(grads, 10.0, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, now))


def test_shapes_and_an_empty_list():
    grads = [g.view(s) for g, s in zip(grads_of([60, 1, 24]), ((3, 4, 5), (), (24, 1)))]
    check(grads)
    norm = torch.full((), 7.0, device="cuda")
    got, out, _ = pgg.clip_grads([], 1.0, norm=norm)
    assert got is norm and float(norm) == 0.0 and out == []
    check([torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_clips_nothing(bad):
    grads = grads_of([5000, 20000])
    grads[1][777] = bad
    kept = [g.clone() for g in grads]
    norm, out, _ = pgg.clip_grads(grads, 0.1)
    assert not math.isfinite(float(norm)) and math.isnan(float(norm)) == math.isnan(bad)
    assert all(torch.equal(torch.nan_to_num(a.float(), 9), torch.nan_to_num(b.float(), 9))
               for a, b in zip(out, kept))


@pytest.mark.parametrize("size", [1e-44, 1e-38, 1e-30, 1e-20, 1e18, 1e25, 1e33])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_squares_outside_the_range(size, dtype):
    """Gradients whose squares fp32 does not hold; below 2^-126 the norm's own step is coarser."""
    grads = [(g.float() * size).to(dtype) for g in grads_of([50000, 3], (torch.float32,), std=1.0)]
    want = exact_norm(grads)
    norm = float(pgg.grad_norm(grads)[0])
    assert abs(norm - want) <= 8 * U * want + 2.0 ** -150
    if want > 1e-30:
        check(grads, max_norm=want / 3, eps=0.0)


def test_large_and_small_side_by_side():
    grads = [torch.full((100,), 1e30, device="cuda"), torch.full((100000,), 1e-30, device="cuda"),
             torch.randn(1000, device="cuda")]
    check(grads, 1e29)


def test_any_alignment_and_nothing_beside_written():
    for dtype in TYPES:
        for n in (5, 16384, 40001):
            buf = torch.randn(n + 2, device="cuda").to(dtype)
            ends = buf[0].clone(), buf[-1].clone()
            check([buf[1:-1], torch.randn(10, device="cuda")], 0.25)
            assert buf[0] == ends[0] and buf[-1] == ends[1]


def test_repeatable_in_a_graph():
    grads = grads_of([30000 + 17 * i for i in range(530)])
    out = [torch.empty_like(g) for g in grads]
    norm, _, ws = pgg.clip_grads(grads, 1.0, out=out)
    want = float(norm), [o.clone() for o in out]
    ws.fill_(0xEE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            norm, _, _ = pgg.clip_grads(grads, 1.0, out=out, workspace=ws)
    for o in out:
        o.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert float(norm) == want[0] and all(torch.equal(a, b) for a, b in zip(out, want[1]))


def test_more_elements_than_32_bits_count():
    n = 2**32 + 12345
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 2.0
    norm, _, _ = pgg.clip_grads([g], 1.0, eps=0.0)
    assert abs(float(norm) - math.sqrt(12)) <= 8 * U * 4
    assert bool((g[-3:].float() == torch.tensor(2 / math.sqrt(12)).bfloat16().item()).all())
    assert not bool(g[:100].any())


def test_wrapper_refusals():
    g = grads_of([10, 20])
    with pytest.raises(ValueError):
        pgg.clip_grads([g[0], g[1].cpu()], 1.0)
    with pytest.raises(ValueError):
        pgg.clip_grads([g[0][::2]], 1.0)
    with pytest.raises(ValueError):
        pgg.clip_grads(g, 1.0, out=[g[0], g[1].float().half()[:5]])
    with pytest.raises(pgg.PggError):
        pgg.clip_grads(g, 1.0, out=g[:1])
    with pytest.raises(pgg.PggError):
        pgg.clip_grads(g, -1.0)
    with pytest.raises(pgg.PggError):
        pgg.clip_grads([g[0].double()], 1.0)
    with pytest.raises(pgg.PggError):
        pgg.grad_norm(g, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
