"""Every instance of the norm: 1, 2, 4, 8 and 16 pieces of 8 values a thread, up to 1024 threads a row."""
import pytest
import torch

import f8_util as f8
from gpu_util import DEV
from test_gpu_f8_rows import rows
from tensor_matmul_collective_gb300 import coc

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16

# rows, hidden.  On 152 SMs: 1 piece up to 1024 threads (64 rows of 8192, 8 of 6144); 2 (few rows of 8208 to 16384, short rows in
# numbers); 4 (many rows); 8 (16400 to 32768); 16 above
SIZES = [(64, 8192), (8, 6144), (5, 12304), (16, 16384), (64, 12288), (400, 400), (700, 512), (400, 8208), (200, 16384), (3, 16400), (3, 20000), (153, 20000),
         (160, 24576), (153, 32768), (1, 32768), (2, 32784), (200, 40000)]


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("n,h", SIZES)
def test_norm(n, h, res):
    dt = BF if (n + h // 16) % 2 else HF
    x, r = rows(1, n, h, dt, n + h)[0], rows(1, n, h, dt, n + h + 1, 2.0)[0]
    w = (1.0 + 0.3 * torch.randn(h, generator=torch.Generator().manual_seed(h))).to(dt)
    codes, scales, sums = coc.add_rms_norm_f8([x.to(DEV)], w.to(DEV), residuals=[r.to(DEV)] if res else None, eps=1e-5)
    if res:
        assert torch.equal(sums[0].cpu().view(torch.int16), (x.float() + r.float()).to(dt).view(torch.int16))
    s = x.double() + (r.double() if res else 0.0)
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + float(torch.tensor(1e-5))) * w.double()
    # the squares' sum: 128 values a thread, 5 shuffles and 32 warps, 2**-24 an addition, halved by the root: 2**-17.6; the values, the
    # reciprocal root and the products 2**-20 more
    f8.check_codes(codes[0], scales[0], y, 2.0 ** -17 * y.abs())


@pytest.mark.parametrize("h", [1024, 8192, 12288, 20000, 40000])
def test_rows_that_overflow_among_others(h):
    """Squares beyond fp32 take the second sum, behind its barriers, in blocks of every width."""
    x = rows(1, 7, h, BF, h)[0]
    x[2] *= 2.0 ** 100
    x[5, 3] = 2.0 ** 70
    codes, scales, _ = coc.add_rms_norm_f8([x.to(DEV)], torch.ones(h, dtype=BF, device=DEV), eps=1e-5)
    s = x.double()
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + float(torch.tensor(1e-5)))
    f8.check_codes(codes[0], scales[0], y, 2.0 ** -17 * y.abs() + 2.0 ** -110)
