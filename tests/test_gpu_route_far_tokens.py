"""The router with more tokens than a launch of its gradient takes (2^32 threads)."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def test_route_gradient_of_more_tokens_than_a_launch():
    """2^26 tokens and 5 of padding, in one call and in 16: the same bits, since T is a power of two
    either way and the losses' gradients are scaled by others."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    note("route, 2^26 + 5 tokens of 129 experts")
    T, pad, E, k, parts = 1 << 26, 5, 129, 2, 16
    torch.manual_seed(0)
    some = torch.randn(100003, E, device="cuda", dtype=torch.bfloat16)      # repeated: T is no multiple
    x = torch.empty(T + pad, E, device="cuda", dtype=torch.bfloat16)
    for at in range(0, T + pad, len(some)):
        x[at:at + len(some)] = some[:min(len(some), T + pad - at)]
    x[T:] = float("nan")
    idx, w, lse, counts, losses = m.fp8_moe_route(x, k, tokens_valid=T)
    assert (idx[T:] == -1).all() and (w[T:] == 0).all() and counts.sum().item() == T * k
    dw = torch.randn(T + pad, k, device="cuda")
    dl = torch.tensor([0.75, -0.5], device="cuda") * T
    d = m.fp8_moe_route_bwd(x, lse, idx, w, counts, dw, dl, tokens_valid=T)
    assert (d[T:] == 0).all()
    n = T // parts
    for p in range(parts):
        s = slice(p * n, (p + 1) * n)
        want = m.fp8_moe_route_bwd(x[s], lse[s], idx[s], w[s], counts, dw[s],
                                   dl / torch.tensor([parts * parts, parts], device="cuda"))
        assert torch.equal(d[s], want), p
    assert (d[T - 1] != 0).any()
