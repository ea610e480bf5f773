"""Many adapters over as many short rows as 32-bit offsets hold."""
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_nf4_quantized_17_amd as q  # noqa: E402


def test_a_nan_at_the_end_of_short_rows_reaches_no_other():
    """dY of 8 columns, 16 bytes a row, a little under 2 GiB: what a row reads
    behind its last column is zeros, not a row near the buffer's end (whose
    product with the weight's zeros there would still be NaN)."""
    M, N, K, r = 2**27 - 321, 8, 64, 1
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB")
    log(f"[multi short rows] M={M}")
    gen = torch.Generator(device="cuda").manual_seed(0)
    w = q.nf4_quantize(torch.randn(N, K, device="cuda", generator=gen) * 0.02)
    W = q.nf4_dequantize(w).double()
    ad = q.AdapterSet(torch.zeros(1, r, K, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(1, N, r, dtype=torch.bfloat16, device="cuda"), torch.ones(1, device="cuda"))
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    dY = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    dY[:2000] = torch.randn(2000, N, device="cuda", generator=gen).bfloat16()
    dY[-1800:] = float("nan")
    ids = torch.full((M,), -1, dtype=torch.int32, device="cuda")
    T = torch.zeros(M, r, device="cuda")
    dX, dA, dB = q.qlora_multi_bwd(w, X, dY, ad, ids, T=T)
    torch.cuda.synchronize()
    want = dY[:2000].double() @ W
    # eight products, their sum and the rounding to bf16
    bound = 2.0**-8 * want.abs() + 9 * 2.0**-24 * (dY[:2000].double().abs() @ W.abs()) + 1e-30
    assert torch.isfinite(dX[:2000]).all()
    assert ((dX[:2000].double() - want).abs() <= bound * 1.01).all()
    assert torch.isnan(dX[-1800:]).all() and torch.isfinite(dX[-3000:-1800]).all()
    assert not dA.any() and not dB.any()
