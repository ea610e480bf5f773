"""Many adapters on every tile of the fused kernel: 64, 128 and 256 rows, the
contraction whole and in parts, against the 64-bit forms and their bounds.
Each case states the tile it is there for."""
import pytest

import multi_ref as ref
from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_nf4_quantized_17_amd as q  # noqa: E402


class Case:
    def __init__(self, M, N, K, r, count, pattern, rows, split, backward):
        gen = torch.Generator(device="cuda").manual_seed(M + 7 * N + 13 * K + 101 * r)
        rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.w = q.nf4_quantize(rn(N, K) * 0.02)
        kernel, got, parts = q.qlora_multi_plan(self.w, M, r, backward)
        assert (kernel, got, parts > 1) == ("fused", rows, split)
        self.W = q.nf4_dequantize(self.w).double()
        self.X, self.dY = rn(M, K).bfloat16(), rn(M, N).bfloat16()
        self.A, self.B = (rn(count, r, K) / r).bfloat16(), (rn(count, N, r) * 0.05).bfloat16()
        self.scale = torch.rand(count, device="cuda", generator=gen) * 2 - 0.25
        if pattern == "distinct":    # neighbours never share an adapter, a tile's run table is long
            ids = torch.arange(M, device="cuda") % count
        else:
            ids = torch.randint(-1, count, (M,), device="cuda", generator=gen)
        self.ids = (ids.sort().values.roll(M // 3) if pattern == "runs" else ids).int()
        self.ids[M // 2] = 0
        log(f"[multi tiles] M={M} N={N} K={K} r={r} count={count} {pattern} {rows} rows, parts {parts}, backward {backward}")

    def fwd(self):
        return q.qlora_multi_fwd(self.w, self.X, q.AdapterSet(self.A, self.B, self.scale), self.ids)

    def bwd(self, T):
        return q.qlora_multi_bwd(self.w, self.X, self.dY, q.AdapterSet(self.A, self.B, self.scale), self.ids, T=T)


FWD = [
    # M, N, K, r, count, pattern, rows, split
    (1030, 8000, 64, 64, 6, "mixed", 256, False),
    (1030, 8003, 128, 37, 9, "runs", 256, False),
    (700, 11008, 64, 100, 3, "mixed", 256, False),
    (1030, 8000, 64, 8, 300, "distinct", 256, False),
    (1030, 8001, 64, 9, 300, "distinct", 256, False),
    (1030, 8000, 64, 8, 1030, "distinct", 256, False),   # every row its own run
    (129, 11008, 2048, 128, 3, "mixed", 256, True),
    (129, 11007, 2048, 12, 60, "distinct", 256, True),
    (513, 8000, 64, 64, 5, "mixed", 128, False),
    (385, 11007, 64, 20, 200, "distinct", 128, False),
    (65, 11008, 2048, 16, 4, "mixed", 128, True),
    (129, 7999, 2048, 100, 40, "distinct", 128, True),
    (200, 250, 64, 77, 4, "runs", 64, False),
    (200, 256, 1024, 128, 80, "distinct", 64, True),
]
BWD = [
    (1030, 72, 8000, 64, 6, "mixed", 256, False),
    (1030, 65, 8064, 9, 300, "distinct", 256, False),
    (129, 2048, 11008, 128, 3, "runs", 256, True),
    (129, 2047, 11008, 9, 60, "distinct", 256, True),
    (513, 72, 8000, 100, 5, "mixed", 128, False),
    (65, 2041, 11008, 16, 4, "mixed", 128, True),
    (200, 60, 256, 33, 4, "runs", 64, False),
    (200, 1024, 256, 128, 80, "distinct", 64, True),
]


@pytest.mark.parametrize("M,N,K,r,count,pattern,rows,split", FWD)
def test_forward(M, N, K, r, count, pattern, rows, split):
    c = Case(M, N, K, r, count, pattern, rows, split, False)
    Y, T = c.fwd()
    torch.cuda.synchronize()
    rY, rT, eY, eT = ref.forward(c.W, c.X, c.A, c.B, c.scale, c.ids)
    log(f"  error of bound: T, Y = {ref.check(T, rT, eT, 'T'):.3g}, {ref.check(Y, rY, eY, 'Y'):.3g}")


@pytest.mark.parametrize("M,N,K,r,count,pattern,rows,split", BWD)
def test_backward(M, N, K, r, count, pattern, rows, split):
    c = Case(M, N, K, r, count, pattern, rows, split, True)
    _, T = c.fwd()
    got = c.bwd(T)
    torch.cuda.synchronize()
    want = ref.backward(c.W, c.X, c.dY, c.A, c.B, c.scale, c.ids, T)
    worst = [ref.check(g, x, e, what) for g, x, e, what in zip(got, want[:3], want[3:], ("dX", "dA", "dB"))]
    log(f"  error of bound: dX, dA, dB = {worst}")


@pytest.mark.parametrize("backward,case", [(b, c) for b, cs in ((False, FWD), (True, BWD)) for c in cs])
def test_a_broken_request_reaches_no_other(backward, case):
    """NaN and infinity in one adapter and in its tokens' rows leave every
    other row and gradient as it was, bit for bit."""
    c = Case(*case, backward)
    bad = case[4] - 1
    hit = c.ids == bad
    assert hit.any() and not hit.all()
    before = c.bwd(None) if backward else c.fwd()
    for t in (c.A, c.B):
        t[bad, ::2], t[bad, 1::2] = float("nan"), float("inf")
    c.X[hit], c.dY[hit] = float("nan"), float("-inf")
    after = c.bwd(None) if backward else c.fwd()
    torch.cuda.synchronize()
    rows, grads = ((0,), (1, 2)) if backward else ((0, 1), ())
    for i in rows:
        assert torch.equal(before[i][~hit], after[i][~hit])
        assert not torch.isfinite(after[i][hit].float()).any()
    for i in grads:
        assert torch.equal(before[i][:bad], after[i][:bad])
