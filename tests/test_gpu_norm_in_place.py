"""The norm in place where rows are not whole 16-byte vectors, so that neighbouring rows share vectors: the sum written
over x or over the residual, dx over d_sum, the same bits as into buffers of their own."""
import pytest
import torch

from dropless_mixture_experts_top_gb300 import moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _build():
    from dropless_mixture_experts_top_gb300 import _build as B
    B.build()


# rows shorter than a vector, of every phase, of a block each, of 1024 threads; more rows than run at once
@pytest.mark.parametrize("T,H", [(5, 3), (40000, 5), (30000, 33), (9000, 250), (3000, 1001), (700, 4097), (600, 8191)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_in_place(T, H, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    x, r, dy, ds = (torch.randn(T, H, generator=gen, device="cuda").to(dt) for _ in range(4))
    w, b = (torch.randn(H, generator=gen, device="cuda").to(dt) for _ in range(2))
    n = moe.Norm(T, H, dtype=dtype)
    want = n.forward(x, w, b, residual=r)
    grads = n.backward(dy, want["sum"], w, want["stats"], d_sum=ds)
    for over in ("x", "r"):
        xx, rr = x.clone(), r.clone()
        out = {"y": torch.empty_like(x), "sum": xx if over == "x" else rr, "stats": torch.empty_like(want["stats"])}
        n.forward(xx, w, b, residual=rr, out=out)
        assert all(torch.equal(out[k], want[k]) for k in want), over
    dd = ds.clone()
    got = n.backward(dy, want["sum"], w, want["stats"], d_sum=dd,
                     grads={"dx": dd, "dweight": torch.empty_like(grads["dweight"]),
                            "dbias": torch.empty_like(grads["dbias"])})
    assert all(torch.equal(got[k], grads[k]) for k in grads)
