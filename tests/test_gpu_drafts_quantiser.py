"""GPU: the quantiser inside qsa_prep_batched against qsa_prep_quantize on the same fp16 rows, bit for bit: rows of
every magnitude that fp16 holds, zero blocks, infinities and NaN."""
import numpy as np
import pytest
import torch

from int8_kv_top_gb300 import qsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rd", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("n", [300, 4000])  # seven warps a token; one
@pytest.mark.parametrize("odd", ["plain", "nan", "inf", "zeros"])
def test_same_codes_and_scales(odd, n, rd):
    rng = np.random.default_rng(rd + n)
    x = rng.standard_normal((n, 4, 256)) * 2.0 ** rng.uniform(-27, 13, (n, 4, 4)).repeat(64, -1)
    x = np.clip(x, -65504, 65504).astype(np.float16)
    if odd != "plain":
        x[rng.random(x.shape) < (0.01 if odd != "zeros" else 0.9)] = {"nan": np.nan, "inf": np.inf, "zeros": 0}[odd]
        x[:, :, 64:128][rng.random((n, 4, 64)) < 0.5] *= -1
        x[: n // 4, :, :64] = 0  # blocks of zeros with one odd element, or none
        x[: n // 8, :, 5] = {"nan": np.nan, "inf": -np.inf, "zeros": -0.0}[odd]
    raw = torch.from_numpy(x).cuda()
    q = torch.zeros(n, 24, 256, dtype=torch.float16, device="cuda")
    one = torch.ones(256, device="cuda")
    kq = torch.full((n, 2, 256), 99, dtype=torch.int8, device="cuda")
    ksc = torch.full((n, 2, 4), 7, dtype=torch.float16, device="cuda")
    vq, vsc, kcur, qcur = kq.clone(), ksc.clone(), torch.empty(n, 2, 256, dtype=torch.float16, device="cuda"), q.clone()
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    qsa.qsa_prep_batched(q, raw[:, :2], raw[:, 2:], one, one, at, at, n, n, qcur, kcur, kq, ksc, vq, vsc,
                         rope=(10000.0, rd, 1e-6, (rd // 2, 0, 0)))
    for rows, codes, scales in ((kcur, kq, ksc), (raw[:, 2:].contiguous(), vq, vsc)):
        want_q, want_s = torch.empty_like(codes), torch.empty_like(scales)
        qsa.qsa_prep_quantize(rows, want_q, want_s)
        assert torch.equal(codes, want_q)
        assert torch.equal(scales.view(torch.int16), want_s.view(torch.int16))
    qsa.qsa_check_device_status()
