"""The norm gradient's workspace: one sized for the largest shape serves every
smaller one."""
import numpy as np
import pytest
import torch

import mx_reference as R
import quantized_int8_gemm_amd as q
from quantized_int8_gemm_amd import _binding as b
from gpu_util import case, dev

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("M,n,larger", [(8192, 100, (8193, 100)), (2048, 400, (2049, 400)), (4096, 8192, (4096, 8193)),
                                        (600, 1000, (600, 1025)), (37, 100, (16384, 16384))])
def test_a_larger_shapes_workspace_serves(M, n, larger):
    case(f"rms_norm_grad {M}x{n} with the workspace of {larger}")
    d = dev()
    g = torch.Generator(device=d).manual_seed(n)
    h, dy = (torch.randn(M, n, generator=g, device=d) for _ in range(2))
    w = torch.ones(n, device=d)
    _, r = q.rms_norm(h, w)
    full = q.rms_norm_grad(dy, h, w, r)
    need = b.lib.rms_norm_grad_workspace_bytes(*larger)
    ws = torch.full((need + 64,), 77, dtype=torch.uint8, device=d)
    got = []
    for _ in range(2):
        dx, dw = torch.empty_like(h), torch.empty_like(w)
        st = b.lib.rms_norm_grad(M, n, dy.data_ptr(), b.QG_FP32, n, h.data_ptr(), n, w.data_ptr(), b.QG_FP32, r.data_ptr(),
                                 None, 0, dx.data_ptr(), n, dw.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == b.QG_OK
        got.append((dx, dw))
    assert torch.equal(got[0][0], full[0]) and torch.equal(got[0][1], got[1][1])   # dx does not depend on it, dw repeats
    assert (ws[need:] == 77).all()
    want = R.grad(*(t.cpu().double().numpy() for t in (dy, h, w, r)))[1]
    size = (dy.double() * h.double() * r.double()[:, None]).abs().sum(0).cpu().numpy()
    # 256 workgroups at least: ceil(M / 256) rows in a lane, 32 groups, 16 partial rows, 10 sums, 4 steps a term
    assert np.all(np.abs(got[0][1].cpu().double().numpy() - want) <= (-(-M // 256) + 62) * U * size)
