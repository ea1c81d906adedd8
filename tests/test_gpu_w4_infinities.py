"""Infinities and NaN of x in the 4-bit products: every form gives what the definition gives, an
infinity of the weights' sign or NaN, whatever its other operands and arithmetic are."""

import pytest
import torch

import permute_grouped_gemm_gb300 as pgg
from test_gpu_w4 import PRODUCTS, built, call, case, weights  # noqa: F401
from test_gpu_w4_forms import form  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def want(s):
    """The results in 64 bits, term by term (a library product need not keep inf 0 = NaN apart)."""
    rows = torch.arange(s["idx"].numel(), device="cuda") if s["product"] == "combined" \
        else s["gather"] // s["top_k"]
    x, w = s["x"].double()[rows], weights(s)
    y = torch.stack([(x[i] * w[int(s["pick"][i])]).sum(1) for i in range(x.shape[0])])
    if s["product"] == "gated":
        gate, up = y[:, :s["N"]], y[:, s["N"]:]
        p = s["probs"].double().reshape(-1)[s["gather"]][:, None]
        y = p * (gate / (1 + (-gate).exp())) * up
    if s["product"] == "combined":
        y = y[torch.argsort(s["gather"])].view(s["T"], s["top_k"], -1).sum(1)
    return y


def check(s, clean):
    got, ws = call(s, out=torch.full_like(clean, 3.0))
    assert pgg.status(ws) == 0
    y = want(s)
    bad = ~torch.isfinite(y)
    assert bool(bad.any()) and bool((~bad).any())
    assert torch.equal(torch.isnan(got), torch.isnan(y))
    assert torch.equal(got[torch.isinf(y)].double(), y[torch.isinf(y)])
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("zeros,scales,group,out", [
    (False, "bf16", 128, None), (True, "bf16", 64, None), (True, "fp32", 32, "fp32"),
    (False, "fp32", 96, "fp32")])
@pytest.mark.parametrize("product", PRODUCTS)
def test_infinities_have_the_weights_signs(form, product, zeros, scales, group, out):  # noqa: F811
    if product == "gated":
        out = None
    s = case(product, T=40, G=3, top_k=2, K=544, N=72, group=group, zeros=zeros, scales=scales,
             out=out, seed=group)
    clean = call(s)[0]
    x = s["x"].clone()
    x[1, 0] = INF            # one element, of either sign
    x[4, 543] = -INF
    x[7, 31], x[7, 500] = INF, INF      # weights of one sign, or NaN
    x[11, 128], x[11, 129] = INF, -INF
    x[13, 77] = NAN
    x[17, 5], x[17, 6] = INF, NAN
    x[20] = INF
    check(dict(s, x=x), clean)


@pytest.mark.parametrize("zeros", [False, True])
def test_whole_rows_of_infinities(form, zeros):  # noqa: F811
    """More of them in a row than a block keeps positions of, weights of one sign."""
    s = case("rows", T=12, G=2, top_k=1, K=1056, N=40, group=32, zeros=zeros)
    s["codes"].fill_(0xFE)
    if zeros:
        s["zeros"].fill_(3)
    s["codes"][1, 5, 7] = 0x33 if zeros else 0x88  # a weight of 0: NaN in its column
    s["scales"][:, 1::3] *= -1
    clean = call(s)[0]
    x = s["x"].clone()
    x[3] = INF
    x[8] = -INF
    x[5, ::2] = INF
    check(dict(s, x=x), clean)


def test_fp16(form):  # noqa: F811
    s = case("gated", T=20, G=2, K=256, N=33, group=128, dtype="fp16", scales="fp16", zeros=True)
    clean = call(s)[0]
    x = s["x"].clone()
    x[2, 9], x[6, 255] = INF, -INF
    check(dict(s, x=x), clean)


@pytest.mark.parametrize("zeros,scales", [(True, "bf16"), (False, "bf16"), (False, "fp32")])
@pytest.mark.parametrize("product", PRODUCTS)
def test_a_scale_that_is_not_finite_stays_with_its_column(form, product, zeros, scales):  # noqa: F811
    s = case(product, T=20, G=3, K=256, N=48, group=64, zeros=zeros, scales=scales)
    clean = call(s)[0]
    bad = s["scales"].clone()
    bad[1, 7, 2], bad[1, 20, 0] = INF, NAN
    got = call(dict(s, scales=bad))[0]
    keep = torch.ones_like(clean, dtype=torch.bool)
    rows = s["pick"] == 1
    if product == "combined":
        rows = (s["gather"] // s["top_k"])[rows]
    for c in (7, 20):
        keep[rows, c] = False
    assert torch.equal(got[keep], clean[keep]) and not bool(torch.isfinite(got[~keep]).any())


@pytest.mark.parametrize("name,zeros,out", [("idx", True, None), ("groups", False, None),
                                            ("idx", False, "fp32")])
@pytest.mark.parametrize("product", PRODUCTS)
def test_bad_routing_gives_zeros_in_every_form(form, product, name, zeros, out):  # noqa: F811
    out = None if product == "gated" else out
    s = case(product, T=30, G=3, K=256, N=72, group=128, zeros=zeros, out=out)
    clean, _ = call(s)
    s[name] = s[name].clone()
    s[name][0] = s[name][1] if name == "idx" else s[name][0] + 1
    got, ws = call(s, out=torch.full_like(clean, 3.0))
    status = "PGG_ERR_NOT_PERM" if name == "idx" else "PGG_ERR_GROUPSUM"
    assert pgg.STATUS[pgg.status(ws)] == status and not bool(got.any())
