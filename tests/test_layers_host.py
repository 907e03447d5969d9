"""The layers around RMA attention without a GPU: sizes, layouts and refusals found on the host."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def rma():
    import bounded_memory_attention_b200
    return bounded_memory_attention_b200


def test_state_bytes_are_the_recurrent_and_convolution_states(rma):
    """The pages' model: 24 layers of 32 heads of 128 x 128 (24 MiB at two bytes a value, 48 MiB here in FP32)
    and three rows of 8,192 channels a layer."""
    n = rma.gdn_state_bytes(rma.GdnConfig(batch=1, n_layers=24))
    delta, conv = 24 * 32 * 128 * 128 * 4, 24 * 3 * 8192 * 2
    assert delta == 48 * 2 ** 20
    assert delta + conv + 4 <= n <= delta + conv + 3 * 256
    assert rma.GdnConfig().channels == 8192


@pytest.mark.parametrize("field,value,code", [
    ("head_dim", 64, "RMA_ERR_UNSUPPORTED"), ("conv_width", 3, "RMA_ERR_UNSUPPORTED"),
    ("batch", 0, "RMA_ERR_INVALID_ARG"), ("n_layers", 0, "RMA_ERR_INVALID_ARG"),
    ("n_k_heads", 0, "RMA_ERR_INVALID_ARG"), ("n_v_heads", 0, "RMA_ERR_INVALID_ARG"),
    ("n_v_heads", 24, "RMA_ERR_INVALID_ARG"), ("qk_l2norm", 2, "RMA_ERR_INVALID_ARG"),
    ("l2_eps", -1.0, "RMA_ERR_INVALID_ARG"), ("l2_eps", float("nan"), "RMA_ERR_INVALID_ARG"),
    ("scale", float("inf"), "RMA_ERR_INVALID_ARG"), ("batch", 1 << 20, "RMA_ERR_UNSUPPORTED"),
    ("n_v_heads", 1 << 14, "RMA_ERR_UNSUPPORTED")])
def test_bad_configs_are_refused(rma, field, value, code):
    cfg = rma.GdnConfig(**{field: value})
    assert rma.gdn_state_bytes(cfg) == 0
    assert rma.lib.rma_last_error().decode() != ""
    h = ctypes.c_void_p()
    rc = rma.lib.rma_gdn_state_alloc(ctypes.byref(cfg._c()), 256, 1 << 40, None, ctypes.byref(h))
    assert rma.ERRORS[rc] == code and not h.value
    with pytest.raises(ValueError):
        rma.GdnState(cfg, device="cpu")


def test_state_alloc_refuses_bad_buffers(rma):
    cfg = rma.GdnConfig()
    n = rma.gdn_state_bytes(cfg)
    h = ctypes.c_void_p()
    c = ctypes.byref(cfg._c())
    assert rma.lib.rma_gdn_state_alloc(c, None, n, None, ctypes.byref(h)) == -1
    assert rma.lib.rma_gdn_state_alloc(c, 256, n, None, None) == -1
    assert rma.lib.rma_gdn_state_alloc(c, 128, n, None, ctypes.byref(h)) == -5
    assert rma.lib.rma_gdn_state_alloc(c, 256, n - 1, None, ctypes.byref(h)) == -3
    assert rma.lib.rma_gdn_state_alloc(None, 256, n, None, ctypes.byref(h)) == -1
    rma.lib.rma_gdn_state_free(None)


def test_null_states_are_refused(rma):
    L = rma.lib
    assert L.rma_qk_norm_rope(None, 0, 1, 256, 8, 256, 8, 256, 256, 0.0, 256, 2, 0, None, 256, 256, None) == -1
    assert L.rma_gdn_conv(None, 0, 1, 256, 8, 256, None, None, 256, None) == -1
    assert L.rma_gdn_decode_step(None, 0, 256, 256, 256, 8, 256, 256, 256, None) == -1
    assert L.rma_gdn_prefill(None, 0, 1, 256, 256, 256, 8, 256, 256, None, 256, 256, 256, None) == -1
    out = ctypes.c_size_t()
    assert L.rma_gdn_workspace_bytes(None, 1, ctypes.byref(out)) == -1
    assert L.rma_gdn_get_status(None, None, ctypes.byref(ctypes.c_uint32())) == -1
    assert L.rma_gdn_state_layout(None, None) == -1


def test_token_strides_of_views():
    """The rows a call takes: contiguous tokens, evenly spaced over the whole batch."""
    from bounded_memory_attention_b200 import layers

    class OnDevice(torch.Tensor):   # a CPU tensor that says it is on a GPU: only shapes and strides are read
        is_cuda = True

    def rows(t, batch, n, inner):
        t = t.as_subclass(OnDevice)
        return layers._rows(t, torch.bfloat16, batch, n, inner, "x", t.get_device())[1]

    wide = torch.zeros(2, 3, 640, dtype=torch.bfloat16)
    assert rows(wide[..., :512].view(2, 3, 2, 256), 2, 3, (2, 256)) == 640
    assert rows(wide[..., 128:], 2, 3, (512,)) == 640
    assert rows(wide[:, 0, :512], 2, 1, (512,)) == 3 * 640
    assert rows(wide[:, :1, :512], 2, 1, (512,)) == 3 * 640
    assert rows(wide[:1, 1:, :512], 1, 2, (512,)) == 640
    assert rows(torch.zeros(1, 1, 512, dtype=torch.bfloat16), 1, 1, (512,)) == 512
    for bad in (lambda: rows(wide[:, :2, :512], 2, 2, (512,)),            # a gap between the sequences
                lambda: rows(wide[..., ::2], 2, 3, (320,)),               # values apart
                lambda: rows(wide.transpose(0, 1), 3, 2, (640,)),         # order of tokens and batch
                lambda: rows(wide, 2, 3, (512,)),
                lambda: rows(wide[0], 2, 3, (640,))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        layers._rows(wide, torch.bfloat16, 2, 3, (640,), "x", 0)   # on the CPU
    with pytest.raises(TypeError):
        rows(wide.float(), 2, 3, (640,))
