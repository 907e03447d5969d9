"""How near the layers around RMA attention come to FP32 arithmetic, against the FP64 oracle.

Beside the elementwise bounds, a share: how many BF16 outputs are not the rounding of the oracle's value.  A value
whose error before the rounding is e is rounded to a neighbour with probability 2 e / step, the step between BF16 values
being 2^-8 to 2^-7 of the value.  FP32 arithmetic, or factors carried in 22 bits (a pair of FP16 or TF32 values without
lo x lo, 2^-22), leaves errors of a few 2^-22 of the terms, taken together less than 2^-20 of the sum of the absolute
terms since they are of either sign.  That sum is about 2^4 of the value for sums of 128 and more terms of either sign:
2 * 2^-20 * 2^4 / 2^-8 = 2^-7 of the outputs, a hundredth at most.  One factor of 11 bits (2^-12 of each term, of either
sign: 2^-15 to 2^-16 of their sum) makes it a tenth and more.
"""
import numpy as np
import pytest
import torch

import oracle
from _gpu import lib  # noqa: F401
from test_gpu_layers import BF, _device, close, delta_case, f64, rope_case, rope_check  # noqa: F401

pytestmark = pytest.mark.gpu


def share_off(got, ref):
    """Share of the finite entries of `ref` whose BF16 rounding `got` is not."""
    live = ~np.isnan(ref)
    want = torch.from_numpy(np.where(live, ref, 0.0)).to(torch.float32).to(BF).double().numpy()
    return (f64(got).reshape(ref.shape) != want)[live].mean()


def delta_reference(x, hk, **more):
    return oracle.delta_rule(*[f64(x[k]) for k in ("qkv", "a", "b", "a_log", "dt_bias", "state")], hk, **more)


@pytest.mark.parametrize("batch,n,hk,hv,fresh", [(1, 100, 4, 8, True), (2, 64, 1, 4, False), (3, 130, 2, 2, False),
                                                 (40, 70, 1, 5, False), (1, 2050, 1, 2, True)])
def test_block_outputs_are_of_fp32_arithmetic(batch, n, hk, hv, fresh):
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=300 + n, fresh=fresh)
    out = torch.empty(batch, n, hv, 128, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
    ref, S, osize, _ = delta_reference(x, hk)
    # sums of 128 terms and more in accumulators of 23 bits: at most 2^-16 of their absolute sum, in the updates and again here
    close(out, ref, 2.0 ** -15 * osize, "out")
    assert share_off(out, ref) <= 0.01


# Keys, values and states far outside the range whose squares and products FP32 holds: (queries and keys, values, state)
FAR = [(2.0 ** 70, 1.0, 1.0), (2.0 ** 100, 2.0 ** -50, 2.0 ** -70), (2.0 ** -80, 2.0 ** 40, 1.0), (2.0 ** -100, 1.0, 2.0 ** 60)]


@pytest.mark.parametrize("n", [1, 5, 70])
@pytest.mark.parametrize("k_scale,v_scale,s_scale", FAR)
def test_normed_rows_of_any_magnitude(n, k_scale, v_scale, s_scale):
    """l2_eps = 0, rows of every finite magnitude: the token form (alone and in a short block) and the chunks agree with
    the oracle, whose squares have 64 bits."""
    rma, _, _, x = delta_case(2, n, 2, 4, seed=310)
    spread = 2.0 ** torch.randint(-4, 5, x["qkv"].shape, generator=torch.Generator().manual_seed(11)).float()
    scale = torch.cat((torch.full((512,), k_scale), torch.full((512,), v_scale)))
    x["qkv"] = (x["qkv"].float() * spread * scale).to(BF)
    x["state"] = x["state"] * s_scale
    d = {k: v.cuda() for k, v in x.items()}
    st = rma.GdnState(rma.GdnConfig(batch=2, n_k_heads=2, n_v_heads=4, l2_eps=0.0))
    st.delta[0].copy_(d["state"])
    out = torch.empty(2, n, 4, 128, dtype=BF, device="cuda")
    if n == 1:
        rma.gdn_decode_step(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out)
    else:
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
    ref, S, osize, size = delta_reference(x, 2, l2_eps=0.0)
    # The bounds of the test above; value columns do not meet, so each is held to its own size.  In a chunk a column's
    # factors are pairs of FP16 under one power of two: what bounds them comes to lie below 2^15, and the smallest step
    # is 2^-24, an error of 2^-40 of that bound in each of the 64 factors of an output (2^-34 in all, |q| |k| scale < 1).
    # The bound is a sum of absolute values where the column's largest is about its root: 16 times as large.  2^-30, of
    # the largest up to this chunk, as the state hands it on: case four has a state of 2^60 that fades to 2^32 meanwhile.
    chunks = n > 8
    floor, sfloor = np.zeros_like(osize), 0.0
    for lo in range(0, n if chunks else 0, 64):
        floor[:, lo:lo + 64] = 2.0 ** -30 * osize[:, :lo + 64].max(1, keepdims=True)
        sfloor = 2.0 ** -30 * np.maximum(np.abs(f64(x["state"])).max(-2, keepdims=True), size.max(-2, keepdims=True))
    close(out, ref, 2.0 ** -15 * osize + floor + 2.0 ** -120, "out")
    assert (np.abs(f64(st.delta[0]) - S) <= 2.0 ** -15 * size.max(-2, keepdims=True) + sfloor + 2.0 ** -120).all()


@pytest.mark.parametrize("n", [1, 5, 70])
def test_an_update_of_zero_adds_nothing_however_large_its_key(n):
    """Without the norm, b = -inf: u is 0, and k.q, beyond FP32, multiplies it.  The output is the old state's."""
    rma, _, _, x = delta_case(1, n, 1, 2, seed=311, l2norm=False)
    x["qkv"][..., :256] = (x["qkv"][..., :256].float() * 2.0 ** 68).to(BF)
    x["b"][:] = -float("inf")
    x["state"] = x["state"] * 2.0 ** -10
    d = {k: v.cuda() for k, v in x.items()}
    st = rma.GdnState(rma.GdnConfig(n_k_heads=1, n_v_heads=2, qk_l2norm=False))
    st.delta[0].copy_(d["state"])
    out = torch.empty(1, n, 2, 128, dtype=BF, device="cuda")
    if n == 1:
        rma.gdn_decode_step(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out)
    else:
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
    ref, S, osize, size = delta_reference(x, 1, l2norm=False)
    close(out, ref, 2.0 ** -15 * osize, "out")
    assert (np.abs(f64(st.delta[0]) - S) <= 2.0 ** -15 * size.max((-1, -2), keepdims=True)).all()


@pytest.mark.parametrize("n", [3, 2050])
@pytest.mark.parametrize("scale,eps", [(2.0 ** 70, 1e-6), (2.0 ** 110, 0.0), (2.0 ** -80, 0.0), (2.0 ** -110, 0.0), (2.0 ** -80, 1e-6),
                                       (2.0 ** -60, 2.0 ** -120)])
def test_rotated_rows_of_any_magnitude(n, scale, eps):
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(1, n, 2, 32, seed=320)
    q, k = ((t.float() * scale).to(BF) for t in (q, k))
    pos = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    rma.qk_norm_rope(st, 0, q, k, w_q, w_k, f, q_out, k_out, positions=pos, eps=eps)
    p = pos.cpu().numpy()
    rope_check(q, k, w_q, w_k, f, q_out, k_out, p, p, eps=float(np.float32(eps)))


@pytest.mark.parametrize("where", ["a", "b", "q", "k", "v", "overflow"])
@pytest.mark.parametrize("t", [66, 101, 127])
def test_what_is_not_finite_is_seen_from_its_token_on(where, t):
    """A NaN, or unnormed keys whose products exceed FP32, at token t of head 1's: every output of that head from there on
    and its state are not finite; the tokens of earlier chunks, the other head and the other sequence keep their bits."""
    rma, _, _, x = delta_case(2, 160, 2, 2, seed=330, l2norm=where != "overflow")
    st = rma.GdnState(rma.GdnConfig(batch=2, n_k_heads=2, n_v_heads=2, qk_l2norm=where != "overflow"))

    def call():
        d = {k: v.cuda() for k, v in x.items()}
        st.delta[0].copy_(d["state"])
        out = torch.empty(2, 160, 2, 128, dtype=BF, device="cuda")
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(160))
        return out, st.delta[0].clone()

    want, want_state = call()
    row = x["qkv"][1, t].view(6, 128)
    if where in "ab":
        x[where][1, t, 1] = float("nan")
    elif where == "overflow":
        x["qkv"][1, t - 1:t + 1, 384:512] = torch.full((128,), 2.0 ** 66, dtype=BF)
    else:
        row["qkv".index(where) * 2 + 1, 3] = float("nan")
    out, state = call()
    assert torch.equal(out[0], want[0]) and torch.equal(state[0], want_state[0])
    assert torch.equal(out[1, :, 0], want[1, :, 0]) and torch.equal(state[1, 0], want_state[1, 0])
    assert torch.equal(out[1, :64, 1], want[1, :64, 1])
    lost = ~torch.isfinite(out[1, :, 1].float())
    if where == "q":
        assert lost[t].all()
    else:
        # (a NaN in v is in its own value column alone)
        lost, bad = (lost[:, 3], ~torch.isfinite(state[1, 1, :, 3])) if where == "v" else (lost.all(-1), ~torch.isfinite(state[1, 1]))
        assert lost[t:].all() and bad.all()


@pytest.mark.parametrize("what", ["a", "b", "zero key"])
def test_how_far_back_a_chunk_is_spoilt(what):
    """The reach that the header states: of a NaN gate, or of a key of zeros without eps, no token before the chunk's first
    (at most 63 before it) is touched, in a block of chunks, and none before the token itself in a short block."""
    for n, t, first in ((130, 100, 64), (6, 4, 4)):
        rma, _, _, x = delta_case(1, n, 1, 1, seed=340)
        st = rma.GdnState(rma.GdnConfig(n_k_heads=1, n_v_heads=1, l2_eps=0.0))
        if what == "zero key":
            x["qkv"][0, t, 128:256] = 0
        else:
            x[what][0, t] = float("nan")
        d = {k: v.cuda() for k, v in x.items()}
        st.delta[0].copy_(d["state"])
        out = torch.empty(1, n, 1, 128, dtype=BF, device="cuda")
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
        fine = torch.isfinite(out.float()).flatten(2).all(-1)[0]
        assert fine[:first].all() and not fine[t:].any() and not torch.isfinite(st.delta).any()


@pytest.mark.parametrize("n", [1, 5, 70])
@pytest.mark.parametrize("eps", [3.0, 1e12, 1e30])
@pytest.mark.parametrize("scale", [2.0 ** -56, 1.0, 2.0 ** 60])
def test_rows_beside_a_large_eps(n, eps, scale):
    """Any l2_eps that is not refused: rows far below it become x / sqrt(eps), tiny but not 0, in both forms."""
    rma, _, _, x = delta_case(1, n, 1, 2, seed=350, fresh=True)
    x["qkv"][..., :256] = (x["qkv"][..., :256].float() * scale).to(BF)
    x["qkv"][..., 256:] = (x["qkv"][..., 256:].float() * 2.0 ** 60).to(BF)
    d = {k: v.cuda() for k, v in x.items()}
    st = rma.GdnState(rma.GdnConfig(n_k_heads=1, n_v_heads=2, l2_eps=eps))
    out = torch.empty(1, n, 2, 128, dtype=BF, device="cuda")
    if n == 1:
        rma.gdn_decode_step(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out)
    else:
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
    _, S, _, size = delta_reference(x, 1, l2_eps=float(np.float32(eps)))
    assert np.abs(S).max() > 2.0 ** -90   # not lost in FP32
    assert (np.abs(f64(st.delta[0]) - S) <= 2.0 ** -15 * size.max((-1, -2), keepdims=True)).all()
