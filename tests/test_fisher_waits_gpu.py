"""Fisher builds whose waits give up (needs a B200): the next build, started right behind one that gave
up, is whole; its tiles reuse the shared memory that the other's copies were meant for."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("guided", [True, False])
@pytest.mark.parametrize("n,d_in,groups", [(64, 128, 1), (512, 256, 2), (2048, 1024, 2)])
def test_the_build_behind_one_that_gave_up_is_whole(guided, n, d_in, groups):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from post_weight_quantization_guided_b200 import binding as b, workloads as wl
    layer = wl.scaled(wl.TINY, n=n, d_in=d_in, d_out=8, groups=groups)
    X, G, _ = wl.make_layer(layer, torch.device("cuda:0"))
    G, groups = (G, groups) if guided else (None, 1)
    want = b.lnq_build_fisher(X, G, groups)
    d_out = G.shape[1] if guided else groups
    ws = [b.workspace(b.LNQ_OP_BUILD_FISHER, n, d_in, d_out, groups) for _ in range(2)]
    torch.cuda.synchronize()
    for limit in (0, 0, 300, 1500, 5000):
        b.lnq_set_wait_limit(limit)
        try:
            b.lnq_build_fisher(X, G, groups, ws=ws[0])
        finally:
            b.lnq_set_wait_limit(-1)
        F = b.lnq_build_fisher(X, G, groups, ws=ws[1])
        status = b.lnq_workspace_check(ws[0])
        assert status == b.LNQ_ERR_TIMEOUT if limit == 0 else status in (b.LNQ_OK, b.LNQ_ERR_TIMEOUT)
        assert b.lnq_workspace_check(ws[1]) == b.LNQ_OK
        assert torch.equal(F, want)
