"""CPU checks of the 8-bit AdamW step's argument lists."""
import warnings

import pytest

import bit_nf4_quantized_17_amd as q

torch = pytest.importorskip("torch")


def test_a_tracers_tensors_are_refused_without_asking_for_their_address():
    """torch warns where a tensor without memory is asked for its address, and
    will raise: the refusal comes before."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("error")
        new = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda:0")  # noqa: E731
        p = new(300)
        for master in (None, new(300, dtype=torch.float32)):
            with pytest.raises(ValueError, match="plain tensors"):
                q.qlora_adamw8_step([p], [new(300)], [q.AdamW8State.zeros(p)], lr=1e-3, masters=[master])
        w = q.NF4Weight(new(256 * 32, dtype=torch.uint8), new(256, dtype=torch.uint8), new(1, dtype=torch.float32), 256, 64)
        ad = q.AdapterSet(new(2, 4, 64), new(2, 256, 4), new(2, dtype=torch.float32))
        ids = new(3, dtype=torch.int32)
        with pytest.raises(ValueError, match="plain tensors"):
            q.qlora_multi_fwd(w, new(3, 64), ad, ids)
        with pytest.raises(ValueError, match="plain tensors"):
            q.qlora_multi_bwd(w, new(3, 64), new(3, 256), ad, ids)


def test_what_has_memory():
    native = q._native()
    assert native.has_memory(torch.zeros(3)) and native.has_memory(torch.nn.Parameter(torch.zeros(3)))
    assert not native.has_memory(None) and not native.has_memory([1]) and not native.has_memory()
    assert not native.has_memory(torch.zeros(3).to_sparse())
