"""int8 form of rows and blocks that hold a NaN of any bits: codes 0, scale NaN."""
import numpy as np
import pytest
import torch

import quantized_int8_gemm_amd as q
from gpu_util import case, dev

pytestmark = pytest.mark.gpu

NANS = [0x7fc00000, 0x7fc00001, 0xffc0ffff, 0x7f800001, 0xffffffff, 0x7fffff7f]


def row(n, bits, at):
    x = np.random.default_rng(n).normal(size=n).astype(np.float32)
    x.view(np.uint32)[at] = bits
    return x


@pytest.mark.parametrize("n", [1, 5, 33, 96, 500, 3000])
def test_quantiser(n):
    for bits in NANS:
        case(f"int8 of a NaN {bits:#x} among {n}")
        x = torch.from_numpy(np.stack([row(n, 0x3f800000, n // 2), row(n, bits, n // 2)])).to(dev())
        codes, scale = q.int8_quantize(x)
        assert not codes[1].any() and scale[1].isnan() and not scale[0].isnan() and codes[0].abs().max() == 127
        codes, scale = q.int8_quantize(x, 32)
        b = n // 2 // 32
        assert not codes[1, 32 * b:32 * b + 32].any() and scale.isnan().sum() == 1 and scale[1, b].isnan()
        keep = torch.ones(n, dtype=torch.bool, device=dev())
        keep[32 * b:32 * b + 32] = False
        assert torch.equal(codes[0, keep], codes[1, keep])


@pytest.mark.parametrize("kind", [0, 3, 4, 6])
def test_checkpoints(kind, monkeypatch):
    """A NaN that comes in by the bias stays in its block; one by a row's scale takes the row."""
    monkeypatch.setenv("QGEMM_FUSED", str(kind))
    m, n, k = 20, 130, 64
    r = np.random.default_rng(4)
    a, w = (torch.from_numpy(r.integers(-128, 128, s, dtype=np.int8)).to(dev()) for s in ((m, k), (n, k)))
    for bits in NANS:
        case(f"checkpoint with a NaN {bits:#x}, kind {kind}")
        sa, bias = row(m, bits, 7), row(n, bits, 70)
        _, (codes, scale) = q.qgemm_a8w8_linear(a, w, torch.from_numpy(sa).to(dev()), torch.ones(n, device=dev()), activation="silu",
                                                bias=torch.from_numpy(bias).to(dev()), b_trans=True, checkpoint=True)
        bad = torch.zeros(m, 5, dtype=torch.bool, device=dev())
        bad[7], bad[:, 2] = True, True
        assert torch.equal(scale.isnan(), bad)
        assert not codes[bad.repeat_interleave(32, 1)[:, :n]].any() and codes[0, :64].abs().max() == 127
        _, (codes, scale) = q.qgemm_a8w8_gated(a, w, w, torch.from_numpy(sa).to(dev()), torch.ones(n, device=dev()),
                                               torch.ones(n, device=dev()), b_trans=True, checkpoint=True)
        assert not codes[:, 7].any() and scale[:, 7].isnan().all() and not scale[:, :7].isnan().any()
