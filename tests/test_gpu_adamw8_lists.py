"""Lists of the 8-bit AdamW step that name the same memory twice: two blocks of
threads would write it, so the call is refused before any launch."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

import bit_nf4_quantized_17_amd as q  # noqa: E402


def _two(n=600):
    p = [torch.ones(n, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    return p, [torch.ones_like(x) for x in p], [q.AdamW8State.zeros(x) for x in p]


@pytest.mark.parametrize("field", ["exp_avg", "exp_root", "exp_avg_scale", "exp_root_scale"])
def test_a_state_buffer_of_two_tensors(field):
    p, g, s = _two()
    setattr(s[1], field, getattr(s[0], field))
    with pytest.raises(ValueError, match=r"states\[1\]: the same tensor twice"):
        q.qlora_adamw8_step(p, g, s, lr=1e-3)


@pytest.mark.parametrize("a,b", [("exp_avg", "exp_root"), ("exp_avg_scale", "exp_root_scale")])
def test_one_buffer_for_both_moments(a, b):
    p, g, s = _two()
    setattr(s[0], b, getattr(s[0], a))
    with pytest.raises(ValueError, match=r"states\[0\]: the same tensor twice"):
        q.qlora_adamw8_step(p, g, s, lr=1e-3)


def test_overlapping_slices():
    p, g, s = _two()
    buf = torch.ones(1200, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match=r"params\[1\]: shares memory with params\[0\]"):
        q.qlora_adamw8_step([buf[:600], buf[592:1192]], g, s, lr=1e-3)
    codes = torch.zeros(1200, dtype=torch.uint8, device="cuda")
    s[0].exp_avg, s[1].exp_root = codes[496:1096], codes[:600]
    with pytest.raises(ValueError, match=r"states\[0\]: shares memory with states\[1\]"):
        q.qlora_adamw8_step(p, g, s, lr=1e-3)
    torch.cuda.synchronize()
    assert (p[0] == 1).all() and (buf == 1).all() and not codes.any()


def test_neighbouring_slices_and_shared_gradients_are_taken():
    p, g, s = _two(608)
    buf = torch.ones(1216, dtype=torch.bfloat16, device="cuda")
    empty = torch.empty(0, dtype=torch.bfloat16, device="cuda")
    e = q.AdamW8State.zeros(empty)
    q.qlora_adamw8_step([buf[608:], empty, buf[:608], empty], [g[0], empty, g[0], empty], [s[0], e, s[1], e], lr=1e-3, seed=1)
    q.qlora_adamw8_step([p[0]], [g[0]], [q.AdamW8State.zeros(p[0])], lr=1e-3, seed=1)
    torch.cuda.synchronize()
    assert torch.equal(buf[608:], p[0]) and torch.equal(buf[:608], p[0])
