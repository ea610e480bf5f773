"""The many-adapter layer on whole numbers: with a weight of zeros the outputs
are the LoRA terms alone, every product and sum of which is exact in fp32
where scale T and scale U are not rounded to bf16.  So Y and dX are the bf16
roundings of the exact sums, bit for bit.

The numbers: T and U are sums of products of small integers, under 2^16 in
magnitude, and a scale is a power of two, so two bf16 terms (8 significant bits
each) hold scale T exactly; sums over the rank stay under 2^24."""
import pytest

import multi_ref as ref
from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_nf4_quantized_17_amd as q  # noqa: E402


def _whole(gen, top, *shape):
    return torch.randint(-top, top + 1, shape, device="cuda", generator=gen, dtype=torch.int32).bfloat16()


def _case(M, N, K, r, count):
    gen = torch.Generator(device="cuda").manual_seed(M + 3 * N + 5 * K + 7 * r)
    w = q.nf4_quantize(torch.zeros(N, K, device="cuda"))
    A, B = _whole(gen, 8, count, r, K), _whole(gen, 3, count, N, r)
    scale = torch.tensor([1.0, -2.0, 0.5, 4.0], device="cuda").repeat(-(-count // 4))[:count].contiguous()
    ids = torch.randint(-1, count, (M,), device="cuda", generator=gen, dtype=torch.int32)
    ids[0] = 0
    return w, A, B, scale, ids, _whole(gen, 8, M, K), _whole(gen, 8, M, N)


def _usable(t):
    assert t.abs().max() < 2**16
    assert (t.bfloat16().double() != t.double()).any()   # one bf16 term would not do


FWD = [
    # M, N, K, r, count
    (1, 256, 1024, 16, 2),         # weight stream
    (7, 300, 1088, 33, 3),
    (16, 520, 1024, 128, 5),
    (17, 256, 512, 64, 9),         # T from the ids, 64-row tile
    (40, 300, 320, 20, 5),
    (64, 1000, 256, 128, 30),
    (65, 256, 128, 16, 3),         # sorted, 64-row tiles
    (100, 333, 1024, 100, 7),
    (513, 8000, 64, 64, 5),        # 128-row tiles
    (500, 7999, 128, 12, 5),
    (65, 11008, 2048, 16, 4),
    (1030, 8000, 64, 64, 6),       # 256-row tiles
    (1030, 8003, 64, 37, 6),
    (129, 11008, 2048, 128, 3),
    (129, 11007, 2048, 12, 3),
]


@pytest.mark.parametrize("M,N,K,r,count", FWD)
def test_forward_is_the_rounded_sum(M, N, K, r, count):
    log(f"[multi whole numbers, forward] M={M} N={N} K={K} r={r} count={count}")
    w, A, B, scale, ids, X, _ = _case(M, N, K, r, count)
    Y, T = q.qlora_multi_fwd(w, X, q.AdapterSet(A, B, scale), ids)
    torch.cuda.synchronize()
    rY, rT, *_ = ref.forward(torch.zeros(N, K, dtype=torch.float64, device="cuda"), X, A, B, scale, ids)
    _usable(rT)
    assert torch.equal(T.double(), rT)
    assert torch.equal(Y, rY.bfloat16()), f"{int((Y != rY.bfloat16()).sum())} of {Y.numel()} differ"


BWD = [
    (1, 1000, 64, 16, 2),
    (40, 1003, 320, 20, 5),
    (100, 520, 320, 100, 7),
    (513, 1000, 8000, 64, 5),
    (65, 2048, 11008, 16, 4),
    (1030, 520, 8000, 37, 6),
    (129, 2048, 11008, 128, 3),
]


@pytest.mark.parametrize("M,N,K,r,count", BWD)
def test_input_gradient_is_the_rounded_sum(M, N, K, r, count):
    log(f"[multi whole numbers, dX] M={M} N={N} K={K} r={r} count={count}")
    w, A, B, scale, ids, X, dY = _case(M, N, K, r, count)
    dX, _, _ = q.qlora_multi_bwd(w, X, dY, q.AdapterSet(A, B, scale), ids)
    torch.cuda.synchronize()
    U = torch.zeros(M, r, dtype=torch.float64, device="cuda")
    want = torch.zeros(M, K, dtype=torch.float64, device="cuda")
    for a in range(count):
        at = (ids == a).nonzero()[:, 0]
        U[at] = dY[at].double() @ B[a].double()
        want[at] = scale[a].double() * (U[at] @ A[a].double())
    _usable(U)
    assert torch.equal(dX, want.bfloat16()), f"{int((dX != want.bfloat16()).sum())} of {dX.numel()} differ"


@pytest.mark.parametrize("direction", ["forward", "backward"])
def test_activations_past_32_bit_offsets(direction):
    """2 GiB of activations: the kernels with 64-bit addresses."""
    M, r, count = 270000, 12, 3
    N, K = (64, 4096) if direction == "forward" else (4096, 64)
    log(f"[multi whole numbers, 2 GiB, {direction}]")
    w, A, B, scale, ids, X, dY = _case(M, N, K, r, count)
    ad = q.AdapterSet(A, B, scale)
    at = torch.cat((torch.arange(300, device="cuda"), torch.arange(M - 300, M, device="cuda")))
    if direction == "forward":
        got = q.qlora_multi_fwd(w, X, ad, ids)[0][at]
        P, F, G = X, A.transpose(1, 2), B.transpose(1, 2)
    else:
        got = q.qlora_multi_bwd(w, X, dY, ad, ids)[0][at]
        P, F, G = dY, B, A
    torch.cuda.synchronize()
    want = torch.zeros(got.shape, dtype=torch.float64, device="cuda")
    for a in range(count):
        own = ids[at] == a
        t = P[at][own].double() @ F[a].double()
        _usable(t)
        want[own] = scale[a].double() * (t @ G[a].double())
    assert torch.equal(got, want.bfloat16())
