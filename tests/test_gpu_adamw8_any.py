"""The 8-bit AdamW step on gradients that are not finite or whose squares are
not: bit for bit adamw8_any_ref, and nothing of one element in another."""
import numpy as np
import pytest

import adamw8_any_ref as ra
import adamw8_ref as r8
from helpers import log

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_nf4_quantized_17_amd as q  # noqa: E402

F = np.float32
TOP = 2.0**127 * (2 - 2.0**-7)   # bf16's largest


def _same(got, want, what):
    got = got.float().cpu().numpy() if got.dtype == torch.bfloat16 else got.cpu().numpy()
    want = want.float().numpy() if isinstance(want, torch.Tensor) else want
    if want.dtype == F:   # (any NaN is one)
        assert np.array_equal(np.isnan(got), np.isnan(want)), what
        got, want = (np.where(np.isnan(x), F(0), x).view(np.uint32) for x in (got, want))
    assert np.array_equal(got, want), f"{what}: {int((got != want).sum())} of {got.size} differ"


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("kind", ["nan", "inf", "large", "mixed"])
def test_bits_and_neighbours(kind, master):
    log(f"[adamw8 any gradient] {kind} master={master}")
    n = 256 * 20 + 100 + 3
    rng = np.random.default_rng(5)
    theta = r8.bf16(rng.normal(size=n) * 0.05).float().numpy()
    p, w = r8.bf16(theta).cuda(), torch.from_numpy(theta.copy()).cuda() if master else None
    nb = -(-n // 256)
    host = [np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(nb, F), np.zeros(nb, F)]
    state = q.AdamW8State.zeros(p)
    values = {"nan": [np.nan], "inf": [np.inf, -np.inf], "large": [2.0**70, -(2.0**100), TOP],
              "mixed": [np.nan, np.inf, -np.inf, 2.0**70, -TOP]}[kind]
    hit = np.zeros(n, bool)
    for t in range(1, 6):
        g = r8.bf16(rng.normal(size=n) * 1e-3).float().numpy()
        if t in (2, 4):
            at = np.concatenate([rng.choice(n, 9, replace=False), [n - 1, 300]])
            g[at] = np.resize(values, at.size)
            hit[at[~np.isfinite(g[at])]] = True
        q.qlora_adamw8_step([p], [torch.from_numpy(g).bfloat16().cuda()], [state], lr=1e-3, weight_decay=0.01, step=t,
                            masters=[w])
        torch.cuda.synchronize()
        theta, *host = ra.step(theta, g, *host, 0, t, 1e-3, 0.9, 0.999, 1e-8, 0.01, t)
        _same(p, r8.bf16(theta), f"param step {t}")
        if master:
            _same(w, theta, f"master step {t}")
        else:
            theta = r8.bf16(theta).float().numpy()
        for got, want, what in zip((state.exp_avg, state.exp_root, state.exp_avg_scale, state.exp_root_scale), host,
                                   ("exp_avg", "exp_root", "exp_avg_scale", "exp_root_scale")):
            _same(got, want, f"{what} step {t}")
    assert torch.isfinite(state.exp_avg_scale).all() and torch.isfinite(state.exp_root_scale).all()
    assert np.array_equal(torch.isnan(p).cpu().numpy(), hit)
    for v in state.moments():
        bad = torch.isnan(v).cpu().numpy()
        assert np.array_equal(bad, hit)


def test_a_nan_code_stays_one_element():
    """A state read from elsewhere, with a NaN code in the first moment alone."""
    rng = np.random.default_rng(6)
    n = 700
    host = [rng.integers(0, 127, n).astype(np.uint8), rng.integers(0, 127, n).astype(np.uint8),
            (rng.random(3) * 1e-5).astype(F), (rng.random(3) * 1e-5).astype(F)]
    host[0][[5, 300]] = 0x7F, 0xFF
    state = q.AdamW8State(*(torch.from_numpy(x.copy()).cuda() for x in host))
    theta, g = r8.bf16(rng.normal(size=n)), r8.bf16(rng.normal(size=n) * 1e-3)
    p = theta.cuda()
    q.qlora_adamw8_step([p], [g.cuda()], [state], lr=1e-3, step=4)
    torch.cuda.synchronize()
    th, *host = ra.step(theta.float().numpy(), g.float().numpy(), *host, 0, 4, 1e-3, 0.9, 0.999, 1e-8, 0.0, 4)
    _same(p, r8.bf16(th), "param")
    for got, want in zip((state.exp_avg, state.exp_root, state.exp_avg_scale, state.exp_root_scale), host):
        _same(got, want, "state")
    assert torch.isnan(p).nonzero()[:, 0].tolist() == [5, 300]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_one_adapter_leaves_the_others(bad):
    """Adapters of 96 elements share blocks of 256: the gradients of one are
    not finite, and the rest step as they do beside zeros."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    g = torch.randn(8, 2, 48, device="cuda", generator=gen).bfloat16()
    out = []
    for x in (bad, 0.0):
        p = torch.ones_like(g)
        s = q.AdamW8State.zeros(p)
        for t in (1, 2, 3):
            gt = g * t
            gt[2] = x
            q.qlora_adamw8_step([p], [gt], [s], lr=1e-2, step=t)
        out.append((p, s.exp_avg.view(g.shape), s.exp_root.view(g.shape)))
    torch.cuda.synchronize()
    keep = torch.arange(8, device="cuda") != 2
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(*out))
    assert torch.isnan(out[0][0][2]).all()
