"""The binding of the layers around RMA attention, without a GPU."""
import ctypes
from types import SimpleNamespace

import pytest


@pytest.fixture(scope="module")
def rma():
    import bounded_memory_attention_b200
    return bounded_memory_attention_b200


@pytest.mark.parametrize("field", ["batch", "n_layers", "n_k_heads", "n_v_heads", "head_dim", "conv_width"])
@pytest.mark.parametrize("times", [1, -1])
def test_sizes_beyond_32_bits_are_refused_and_not_cut(rma, field, times):
    """ctypes keeps the low 32 bits: 2^32 + 1 sequences were laid out as one."""
    cfg = rma.GdnConfig()
    setattr(cfg, field, getattr(cfg, field) + times * 2 ** 32)
    with pytest.raises(ValueError, match=field):
        rma.gdn_state_bytes(cfg)


def test_an_eps_beyond_its_range_is_refused(rma):
    """Beside 3e38 a key of 2^-56 is normed to 2^-120, and with its decay it leaves FP32's normal numbers in a chunk."""
    assert rma.gdn_state_bytes(rma.GdnConfig(l2_eps=3e38)) == 0 and "l2_eps" in rma.lib.rma_last_error().decode()
    assert rma.gdn_state_bytes(rma.GdnConfig(l2_eps=1e30)) > 0


@pytest.mark.parametrize("layer", [2 ** 32, 2 ** 31, -2 ** 32, 2 ** 63])
def test_layers_beyond_32_bits_are_refused_and_not_cut(rma, layer):
    from bounded_memory_attention_b200 import layers
    called = []
    with pytest.raises(ValueError, match="layer"):
        layers._call(lambda *a: called.append(a) or 0, "f", 0, SimpleNamespace(cuda_stream=0),
                     ctypes.c_void_p(), layer, 1)
    assert not called


def test_tokens_beyond_32_bits_are_refused_and_not_cut(rma):
    state = SimpleNamespace(_h=ctypes.c_void_p())
    with pytest.raises(ValueError, match="n_tok"):
        rma.GdnState.workspace_bytes(state, 2 ** 32 + 1)
