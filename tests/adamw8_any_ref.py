"""The 8-bit AdamW step of adamw8_ref for any gradient: numbers whose squares
leave fp32's range, infinities and NaN.  On gradients under 2^60 it is
adamw8_ref.step bit for bit; an element that is not finite keeps to itself."""
import numpy as np

import adamw8_ref as r8

F = np.float32
NAN_CODE = 0x7F


def step(theta, g, cm, cu, dm, du, first_block, seed, lr, b1, b2, eps, wd, t):
    n, nb = theta.size, -(-theta.size // r8.BLOCK)
    rep = lambda d: np.repeat(d, r8.BLOCK)[:n]  # noqa: E731
    decay, size = F(1.0 - lr * wd), F(lr / (1.0 - b1**t))
    inv, c1, c2, b1, b2 = F(1.0 / np.sqrt(1.0 - b2**t)), F(1.0 - b1), F(1.0 - b2), F(b1), F(b2)
    with np.errstate(all="ignore"):
        m = b1 * (r8.decode(cm) * rep(dm)) + c1 * g
        uo = r8.decode(cu) * rep(du)
        v = b2 * (uo * uo) + c2 * (g * g)
        s = F(2.0**-64)
        scaled = np.sqrt(b2 * ((uo * s) * (uo * s)) + c2 * ((g * s) * (g * s))) * F(2.0**64)
        u = np.where(v < np.inf, np.sqrt(v), scaled)
        theta = theta * decay - size * (m / (u * inv + F(eps)))
        fm, fu = np.isfinite(m), np.isfinite(u)

        def largest(x, finite):
            out = np.zeros(nb * r8.BLOCK, F)
            out[:n] = np.where(finite, np.abs(x), F(0))
            return out.reshape(nb, r8.BLOCK).max(1)
        am, au = largest(m, fm), largest(u, fu)
        am = np.where(am >= F(2.0**-117), am, F(0))
        im, iu = (np.where(a > 0, F(448.0) / a, F(0)).astype(F) for a in (am, au))
        zm, zu = np.where(fm, m, F(0)), np.where(fu, u, F(0))
        cm = np.where(fm, r8.encode_nearest(zm * rep(im)), NAN_CODE).astype(np.uint8)
        cu = np.where(fu, r8.encode_stochastic(zu * rep(iu), r8.low_bits(first_block, n, seed)), NAN_CODE).astype(np.uint8)
    k = F(1.0) / F(448.0)
    assert theta.dtype == m.dtype == u.dtype == F
    return theta, cm, cu, am * k, au * k
