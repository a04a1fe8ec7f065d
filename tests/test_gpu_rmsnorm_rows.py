"""fp4_rmsnorm_backward where a workgroup walks over several rows: the next row's
loads, the alternating buffers of the joins and the sum of dw over rows, in each
of its kernels, against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import _mx_ref as R
import fp4_precision_gemms_amd as F
from _util import need_gpu, say
from test_gpu_rmsnorm import U32, back_reference, bf, inputs

pytestmark = pytest.mark.gpu

# three rows a workgroup and a remainder: 1024 workgroups up to 1024 columns, 512
# up to 2048, else 256
SHAPES = [(3100, 1024), (1100, 1056), (1600, 2048), (700, 2080), (800, 4096), (700, 4128), (800, 8192), (520, 8224),
          (600, 16384), (520, 16416), (600, 32768)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("with_dh", [True, False])
def test_backward_of_several_rows_a_workgroup(rows, cols, with_dh):
    need_gpu()
    say("rmsnorm back, several rows", rows, cols, with_dh)
    assert rows > 2 * (F.fp4_rmsnorm_workspace_bytes(rows, cols) // (4 * cols))
    rng = np.random.default_rng(rows + cols)
    x, r, w = inputs(rows, cols, rows * 3 + cols)
    h, rstd, _ = R.rmsnorm(x, r, w, 1e-5)
    dy = R.to_bf16(rng.standard_normal((rows, cols)) * 1e-3)
    dh = R.to_bf16(rng.standard_normal((rows, cols)) * 1e-3) if with_dh else None
    args = (bf(dy), bf(h), bf(w), torch.from_numpy(rstd).cuda())
    dx, dw = F.fp4_rmsnorm_backward(*args, None if dh is None else bf(dh))
    torch.cuda.synchronize()
    ref, near, dwref, dwsize = back_reference(dy, h, w, rstd, dh)
    assert (np.abs(dx.double().cpu().numpy() - ref) <= near).all()
    # rows of a workgroup one after another, then 32 slices of the parts; three
    # roundings of a term
    parts = F.fp4_rmsnorm_workspace_bytes(rows, cols) // (4 * cols)
    depth = -(-rows // parts) + -(-parts // 32) + 32 + 3
    assert (np.abs(dw.double().cpu().numpy() - dwref) <= depth * U32 * dwsize).all()


def test_dw_of_a_tensor_beyond_32_bits():
    need_gpu()
    rows, cols = 65600, 32768
    say("rmsnorm back, dw beyond 32 bits")
    g = torch.Generator(device="cuda").manual_seed(0)
    h, dy = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_(0, 1, generator=g) for _ in range(2))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(rows, device="cuda").uniform_(0.5, 2, generator=g)
    _, dw = F.fp4_rmsnorm_backward(dy, h, w, rstd)
    ref, size = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
    for lo in range(0, rows, 4100):
        t = dy[lo:lo + 4100].double() * h[lo:lo + 4100].double() * rstd[lo:lo + 4100, None].double()
        ref += t.sum(0)
        size += t.abs().sum(0)
    assert ((dw.double() - ref).abs() <= (-(-rows // 256) + 8 + 32 + 3) * U32 * size).all()
