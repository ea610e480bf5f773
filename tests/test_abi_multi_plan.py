"""The host query for a many-adapter call's kernel (CPU: fake addresses, never
dereferenced)."""
import ctypes

import bit_nf4_quantized_17_amd as q

FAKE = 0x7f0000000000
STREAM, FUSED, GENERIC = 0, 1, 2


def _plan(M, N, K, r=16, backward=0, dq=256):
    w = q._Weight(FAKE, FAKE if dq else None, FAKE, N, K, 64, dq)
    out = (ctypes.c_int * 3)()
    assert q.lib().qlora_multi_plan(ctypes.byref(w), M, r, backward, ctypes.byref(out)) == 0, q.lib().qlora_last_error()
    return tuple(out)


def test_kernels_by_size():
    assert _plan(1, 4096, 4096)[0] == STREAM and _plan(16, 333, 192)[0] == STREAM
    assert _plan(16, 4096, 4096, dq=0)[0] == FUSED           # fp32 scales: tiles
    assert _plan(17, 4096, 4096)[0] == FUSED and _plan(16, 4096, 4096, backward=1)[0] == FUSED
    assert _plan(270000, 64, 4096)[0] == GENERIC and _plan(270000, 64, 4096, backward=1)[0] == FUSED
    assert _plan(270000, 4096, 64, backward=1)[0] == GENERIC
    # short rows of dY, up to what 32-bit offsets hold
    assert _plan(2**27 - 321, 8, 64, backward=1)[0] == FUSED and _plan(2**27 - 320, 8, 64, backward=1)[0] == GENERIC


def test_tiles_are_of_64_128_or_256_rows_and_parts_take_four_steps():
    seen = set()
    for M in (17, 64, 129, 513, 1030, 4096):
        for N in (8, 1000, 11008):
            for K in (64, 2048, 8192):
                for b in (0, 1):
                    kernel, rows, parts = _plan(M, N, K, backward=b)
                    steps = -(-(N if b else K) // 64)
                    assert kernel == FUSED and rows in (64, 128, 256) and 1 <= parts <= 16
                    assert parts == 1 or 4 * (parts - 1) < steps
                    seen.add((rows, parts > 1))
    assert len(seen) == 6


def test_refusals():
    w, out = q._Weight(FAKE, FAKE, FAKE, 256, 256, 64, 256), (ctypes.c_int * 3)()
    call = lambda w, M, r, o: q.lib().qlora_multi_plan(ctypes.byref(w) if w else None, M, r, 0, ctypes.byref(o) if o else None)  # noqa: E731
    assert call(None, 4, 8, out) == -1 and call(w, 4, 8, None) == -1
    assert call(w, 0, 8, out) == -2 and call(w, 4, 0, out) == -3 and call(w, 4, 129, out) == -3
