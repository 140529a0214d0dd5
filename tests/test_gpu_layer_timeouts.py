"""Waits that give up, in the streamed recurrence and the 8-bit product: a copy is
left out, the wait for it runs out after about a second, the status says so, and
the context goes on (needs a B200)."""
import numpy as np
import pytest
import torch

from kalman_filter_linear_b200 import kdn
from oracle import fp8_ref, linear_scan_ref
from gpu_util import f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,D,tile", [(2, 1500, 128, 0), (2, 1500, 128, 5), (40, 900, 64, 1),
                                        (3, 1500, 100, 2)])
def test_scan(B, T, D, tile):
    g = torch.Generator().manual_seed(T)
    a, x = torch.sigmoid(torch.randn(B, T, D, generator=g)).cuda(), torch.randn(B, T, D, generator=g).cuda()
    ws = torch.empty(kdn.kdn_linear_scan_workspace_size(B, T, D), dtype=torch.uint8, device='cuda')
    kdn.kdn_testing_linear_scan_skip_copy(a, x, tile, ws)
    assert kdn.kdn_read_workspace_status(ws) == kdn.KDN_ERR_TIMEOUT
    y, h = kdn.kdn_linear_scan_forward(a, x, workspace=ws)
    assert kdn.kdn_read_workspace_status(ws) == kdn.KDN_OK
    for i in range(B):
        want, hT = linear_scan_ref.forward(f64(a[i]), f64(x[i]))
        tol, tol_end = linear_scan_ref.forward_bound(f64(a[i]), f64(x[i]))
        assert (np.abs(f64(y[i]) - want) <= 2.0 ** -24 * tol).all()
        assert (np.abs(f64(h[i]) - hT) <= 2.0 ** -24 * tol_end).all()


@pytest.mark.parametrize("M,N,K,block", [(8, 2048, 2048, 0), (8, 300, 2048, 1), (60, 500, 2048, 3),
                                         (600, 1000, 2048, 0), (600, 1000, 2048, 9),
                                         (2100, 2312, 1400, 7)])
@pytest.mark.parametrize("tile", [False, True])
def test_product(M, N, K, block, tile):
    g = torch.Generator().manual_seed(M)
    x = kdn.kdn_fp8_quantize(torch.randn(M, K, generator=g).cuda())
    w = kdn.kdn_fp8_quantize(torch.randn(N, K, generator=g).cuda(), tile=tile)
    status = torch.zeros(1, dtype=torch.int32, device='cuda')
    kdn.kdn_testing_fp8_matmul_skip_copy(*x, *w, block, status)
    assert kdn.kdn_read_workspace_status(status.view(torch.uint8)) == kdn.KDN_ERR_TIMEOUT
    status.zero_()
    got = kdn.kdn_fp8_matmul(*x, *w, out_dtype=torch.float32, status=status)
    assert kdn.kdn_read_workspace_status(status.view(torch.uint8)) == kdn.KDN_OK
    want, size = fp8_ref.matmul(f64(x[0].float()), f64(x[1]), f64(w[0].float()), f64(w[1]), tile)
    assert (np.abs(f64(got) - want) <= (128 + 3 * -(-K // 128) + 8) * 2.0 ** -23 * size).all()
