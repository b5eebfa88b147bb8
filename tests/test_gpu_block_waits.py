"""The cross-attention kernels' bounded waits: with a wait limit of 0 the first wait that is not already satisfied runs
out, the call reports BSA_EDEVICE through the plan's error word (no trap, no hang), and the next call with the default
limit gives the bits it gave before."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_top_b200 import build
    build.build()
    import block_sparse_attention_top_b200 as m
    return m


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_expired_wait_is_reported_then_recovers(bsa, d, masked):
    B, N, H, M = 2, 700, 3, 300
    g = torch.Generator().manual_seed(d)
    q, k, v, do = (torch.randn(B, n, H, d, generator=g).bfloat16().cuda() for n in (N, M, M, N))
    kw = dict(key_mask=(torch.rand(B, M, generator=g) > 0.3).cuda()) if masked else {}
    plan = bsa.Plan(B, H, 1, 1, N, d, 64, bsa.BSA_ORDER_IDENTITY)

    def step():
        o, lse = bsa.cross_attn(plan, q, k, v, return_lse=True, **kw)
        first = bsa.bsa_last_device_error(plan)
        grads = bsa.cross_attn_backward(plan, do, q, k, v, o, lse, **kw)
        return (o, lse, *grads), (first, bsa.bsa_last_device_error(plan))

    want, errors = step()
    assert errors == (bsa.BSA_OK, bsa.BSA_OK)
    plan.set_wait_limit(0)
    _, errors = step()
    assert errors == (bsa.BSA_EDEVICE, bsa.BSA_EDEVICE)
    assert bsa.bsa_last_device_error(plan) == bsa.BSA_OK                # reading clears the word
    plan.set_wait_limit(4_000_000_000)
    got, errors = step()
    assert errors == (bsa.BSA_OK, bsa.BSA_OK)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
