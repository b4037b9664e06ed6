"""4-bit products whose waits run out, where the copier of the ring has long finished by then."""
import pytest
import torch

import newton_schulz_12_b200 as nsb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,n,k", [(4100, 4200, 96), (4100, 4200, 256), (2100, 2300, 250), (300, 200, 200), (1000, 777, 256),
                                   (100, 60, 250), (16, 4096, 512), (7, 300, 4096)])
def test_everything_has_landed_before_the_kernel_ends(m, n, k):
    """No more stages than the ring holds: the copier starts them all and leaves its loop before the wait for
    the withheld copy runs out.  The call reports, what is outside the result is as it was, and the calls
    after it are right."""
    g = torch.Generator().manual_seed(m + k)
    a, b = nsb.muon_mx_quantize([torch.randn(m, k, generator=g).cuda(), torch.randn(n, k, generator=g).cuda()])
    want = nsb.muon_mx_product(a, b)
    wide = torch.full((m + 2, n + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    assert nsb.muon_get_status() == 0
    nsb.muon_set_wait_timeout_ms(100)
    try:
        nsb.muon_set_fault_injection(1)
        nsb.muon_mx_product(a, b, out=wide[1:-1, 8:8 + n])
        assert nsb.muon_get_status() == -5
    finally:
        nsb.muon_set_fault_injection(0)
        nsb.muon_set_wait_timeout_ms(2000)
    wide[1:-1, 8:8 + n] = 7.0
    assert (wide == 7.0).all()
    for _ in range(3):
        assert torch.equal(nsb.muon_mx_product(a, b), want)
    assert nsb.muon_get_status() == 0
