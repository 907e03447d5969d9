"""The layers around RMA attention at the sizes that choose their kernels, and at random ones, held to FP32 arithmetic.

Slacks beside the half step of the BF16 rounding (2^-8 of the value):
  rotation     the norm's sum of 256 squares, five factors and one product: 2^-18 of the head's largest value;
  convolution  five FP32 operations, 5 x 2^-24 of the sum of absolute terms, and SiLU, whose exponential has an argument
               rounded to 2^-24 of |z| < 16 and two approximations of 2^-22: 2^-20; together below 2^-19 of the sum;
  delta rule   token by token: FP32 sums of 128 terms in a row and its update, 2 x 128 x 2^-24 = 2^-16 of the sum of
               absolute terms if all erred one way, which those of eight tokens stay within;
               chunks: as derived in test_gpu_layers_precision.py, 2^-15; states 2^-18 of their largest value, four
               times what the header states.
"""
import random

import numpy as np
import pytest
import torch

import oracle
import synth_inputs as si
from _gpu import lib  # noqa: F401
from test_gpu_layers import BF, _device, close, delta_case, f64, rope_case  # noqa: F401
from test_gpu_layers_precision import delta_reference, share_off

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- rotation: two tokens a CTA from 4,096 group-tokens on

def rope_exact(q, k, w_q, w_k, f, q_out, k_out, pos_q, pos_k, interleaved=False):
    for x, w, out, pos in ((q, w_q, q_out, pos_q), (k, w_k, k_out, pos_k)):
        ref = oracle.norm_rope(f64(x), f64(w), pos, f64(f), 1e-6, interleaved)
        big = np.abs(oracle.norm_rope(f64(x), f64(w), pos, [], 1e-6)).max(-1, keepdims=True)
        close(out, ref, 2.0 ** -18 * big, "norm_rope")


@pytest.mark.parametrize("batch,n,groups,pairs,interleaved", [
    (8, 129, 4, 128, False),     # halves of whole eights
    (1, 1367, 3, 33, False),     # an odd last token; partners through shared memory, twice in a CTA
    (1, 4097, 1, 32, True),      # neighbours, an odd last token
    (5, 205, 4, 100, False), (3, 459, 3, 0, False)])
def test_rotation_of_blocks_with_two_tokens_a_cta(batch, n, groups, pairs, interleaved):
    assert batch * n * groups >= 4096
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(batch, n, groups, pairs, seed=400 + n)
    pos = si.uniform_int((batch, n), 0, 1 << 18, 3).to(torch.int32)
    rma.qk_norm_rope(st, 1, q, k, w_q, w_k, f if pairs else None, q_out, k_out, positions=pos.cuda(), interleaved=interleaved)
    p = pos.numpy()
    rope_exact(q, k, w_q, w_k, f, q_out, k_out, p, p, interleaved)
    assert rma.get_status(st) == 0


@pytest.mark.parametrize("batch,n,groups,pairs", [(1367, 1, 3, 32), (457, 3, 3, 33)])
def test_rotation_from_counters_where_two_sequences_share_a_cta(batch, n, groups, pairs):
    """Odd token counts: a CTA's two tokens are of two sequences, each at its own group's place; one counter is corrupted."""
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(batch, n, groups, pairs, seed=410 + n)
    at = si.uniform_int((2, batch, groups), 0, 1 << 18, 4).to(torch.int32)
    st.counters[..., 0] = at.cuda()
    st.counters[1, 7, groups - 1, 0] = -9
    at[1, 7, groups - 1] = 0
    rma.qk_norm_rope(st, 1, q, k, w_q, w_k, f, q_out, k_out)
    pk = at[1].numpy()[:, None, :] + np.arange(n)[None, :, None]
    rope_exact(q, k, w_q, w_k, f, q_out, k_out, np.repeat(pk, 4, 2), pk)
    assert rma.get_status(st) == rma.STATUS_BAD_COUNTERS


@pytest.mark.parametrize("pairs,interleaved", [(128, False), (33, False), (100, True)])
def test_rotation_of_blocks_in_place_and_as_single_tokens(pairs, interleaved):
    """Two tokens a CTA, in place or not, and one: the same bits; a NaN stays in its head."""
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(2, 1025, 2, pairs, seed=420)
    q, k = q.contiguous(), k.contiguous()
    q[1, 1024, 3, 17] = float("nan")
    pos = si.uniform_int((2, 1025), 0, 1 << 18, 5).to(torch.int32).cuda()
    rma.qk_norm_rope(st, 0, q, k, w_q, w_k, f, q_out, k_out, positions=pos, interleaved=interleaved)
    bad = torch.isnan(q_out.float())
    assert bad[1, 1024, 3].all() and bad.sum() == 256 and not torch.isnan(k_out.float()).any()
    for at in (0, 511, 512, 1024):
        one_q, one_k = torch.empty_like(q[:, at]), torch.empty_like(k[:, at])
        rma.qk_norm_rope(st, 0, q[:, at].contiguous(), k[:, at].contiguous(), w_q, w_k, f, one_q, one_k,
                         positions=pos[:, at].contiguous(), interleaved=interleaved)
        assert torch.equal(torch.nan_to_num(one_q.float(), 9.0), torch.nan_to_num(q_out[:, at].float(), 9.0))
        assert torch.equal(one_k, k_out[:, at])
    rma.qk_norm_rope(st, 0, q, k, w_q, w_k, f, q, k, positions=pos, interleaved=interleaved)
    assert torch.equal(torch.nan_to_num(q.float(), 9.0), torch.nan_to_num(q_out.float(), 9.0)) and torch.equal(k, k_out)


# ---------------------------------------------------------------- convolution

def conv_exact(out, x, old, w, bias, lens):
    ref, new = oracle.conv_silu(f64(x), f64(old), f64(w), None if bias is None else f64(bias), lens)
    xs, ws = np.abs(f64(x)), np.abs(f64(w)).T
    seen = np.concatenate((np.abs(f64(old)), xs), 1)
    size = sum(seen[:, j:j + xs.shape[1]] * ws[j] for j in range(4)) + (0 if bias is None else np.abs(f64(bias)))
    past = np.isnan(ref)
    close(torch.where(torch.from_numpy(past).cuda(), 0.0, out.float()), np.where(past, 0.0, ref),
          2.0 ** -19 * np.where(past, 0.0, size), "conv")
    return past, new


# ---------------------------------------------------------------- delta rule

def fp32_check(out, state, x, hk, chunks, l2norm=True, lens=None):
    ref, S, osize, size = delta_reference(x, hk, l2norm=l2norm, lens=lens)
    past = np.isnan(ref)
    got = out.float().view(ref.shape)
    close(torch.where(torch.from_numpy(past).cuda(), 0.0, got), np.where(past, 0.0, ref),
          (2.0 ** -15 if chunks else 2.0 ** -16) * osize, "out")
    off, big = np.abs(f64(state) - S).max((-1, -2)), np.abs(S).max((-1, -2))
    assert (off <= 2.0 ** -18 * big).all(), f"state: {(off / big).max()} of its largest value"
    return past, ref


@pytest.mark.parametrize("batch,hk,hv,l2norm", [(1, 16, 32, True), (40, 4, 8, True), (5, 3, 3, False), (400, 1, 1, True)])
def test_a_step_is_of_fp32_arithmetic(batch, hk, hv, l2norm):
    """Four CTAs a head, and from 296 heads on one."""
    rma, st, d, x = delta_case(batch, 1, hk, hv, seed=430, l2norm=l2norm)
    out = torch.empty(batch, hv, 128, dtype=BF, device="cuda")
    rma.gdn_decode_step(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out)
    _, ref = fp32_check(out, st.delta[0], x, hk, False, l2norm=l2norm)
    assert share_off(out, ref) <= 0.01


@pytest.mark.parametrize("batch,n,hk,hv,lens", [(3, 8, 1, 2, None), (2, 12, 2, 4, [12, 5]), (10, 8, 16, 32, None),
                                                (150, 7, 1, 2, "random"), (37, 5, 4, 8, "random")])
def test_short_blocks_token_by_token(batch, n, hk, hv, lens):
    """Blocks below the chunks, a CTA a head or four: FP32 arithmetic, rows past a length untouched."""
    if lens == "random":
        lens = si.uniform_int((batch,), 0, n, 31).tolist()
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=440 + n)
    ln = None
    if lens is not None:
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        for b, m in enumerate(lens):
            for key in ("qkv", "a", "b"):
                d[key][b, m:] = float("nan")
    out = torch.full((batch, n, hv, 128), 7.0, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n), lens=ln)
    past, ref = fp32_check(out, st.delta[0], x, hk, False, lens=lens)
    assert (f64(out)[past] == 7.0).all() and share_off(out, ref) <= 0.01
    for b, m in enumerate(lens or []):
        if m == 0:
            assert torch.equal(st.delta[0, b].cpu(), x["state"][b])
    assert rma.gdn_get_status(st) == 0


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes_through_a_delta_layer(seed):
    """Convolution and delta rule over random batches, lengths, heads and forms: padding of NaN, gates as columns of wider
    rows, a poisoned workspace; nothing else of the state changes, and no status is left."""
    r = random.Random(seed)
    rma = lib()
    hk = r.choice([1, 2, 3, 5])
    hv = hk * r.choice([1, 2, 3, 4, 9])
    n = r.choice([1, 2, r.randint(3, 12), r.randint(13, 64), r.randint(65, 200), r.randint(200, 420)])
    batch = r.randint(1, max(1, min(40, 600 // (n * hv) if n > 1 else 40)))
    layer, lens = r.randrange(2), None
    if r.random() < 0.6:
        lens = [r.choice([0, 1, n, r.randint(0, n), r.randint(0, n)]) for _ in range(batch)]
    st = rma.GdnState(rma.GdnConfig(batch=batch, n_layers=2, n_k_heads=hk, n_v_heads=hv))
    x = si.gdn_inputs(batch, n, hk, hv, seed=500 + seed)
    st.conv.copy_(si.bf16_normal(tuple(st.conv.shape), 501 + seed).cuda())
    st.delta[0], st.delta[1] = 3.0, 5.0
    st.delta[layer].copy_(x["state"].cuda())
    other = (st.conv[1 - layer].clone(), st.delta[1 - layer].clone())
    d = {k: v.cuda() for k, v in x.items()}
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    raw = si.bf16_normal((batch, n, st.cfg.channels + 16), 502 + seed).cuda()[..., 8:-8]
    for b, m in enumerate(lens or []):
        raw[b, m:] = float("nan")
    w = si.f32_normal((st.cfg.channels, 4), 503 + seed, std=0.5).cuda()
    bias = si.f32_normal((st.cfg.channels,), 504 + seed).cuda() if r.random() < 0.5 else None
    y, old = torch.full((batch, n, st.cfg.channels), 7.0, dtype=BF, device="cuda"), st.conv[layer].clone()
    rma.gdn_conv(st, layer, raw, w, y, bias=bias, lens=ln)
    past, new = conv_exact(y, raw, old, w, bias, lens)
    assert (f64(y)[past] == 7.0).all() and np.array_equal(f64(st.conv[layer]), new)
    for b, m in enumerate(lens or []):
        y[b, m:] = float("nan")
    ab = torch.cat((d["b"], torch.zeros_like(d["b"][..., :1]), d["a"]), -1)
    for b, m in enumerate(lens or []):
        ab[b, m:] = float("nan")
    ws = st.workspace(n)
    ws.fill_(r.choice([0, 255, 127]))
    out = torch.full((batch, n, hv, 128), 7.0, dtype=BF, device="cuda")
    rma.gdn_prefill(st, layer, y, ab[..., hv + 1:], ab[..., :hv], d["a_log"], d["dt_bias"], out, ws, lens=ln)
    seen = x | {"qkv": torch.nan_to_num(y.float())}
    past, ref = fp32_check(out, st.delta[layer], seen, hk, n > 8, lens=lens)
    assert (f64(out)[past] == 7.0).all()
    assert torch.equal(st.conv[1 - layer], other[0]) and torch.equal(st.delta[1 - layer], other[1])
    assert rma.gdn_get_status(st) == 0


@pytest.mark.parametrize("batch,hk,hv,n,lens", [(1, 16, 16, 2049, None), (2, 7, 7, 2070, [2070, 1999]), (3, 4, 8, 2500, [2500, 0, 77]),
                                                (1, 4, 12, 7200, None)])
def test_blocks_of_few_heads_in_one_launch(batch, hk, hv, n, lens):
    """More items than the first launch runs at once, few heads: one cooperative launch, whatever the workspace held, the
    same bits every time and the bits of the two launches that a sequence alone takes."""
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=600 + batch)
    assert -(-n // 64) * batch * hk > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, m in enumerate(lens or []):
        d["qkv"][b, m:] = float("nan")
    ws, first = st.workspace(n), None
    for fill in (1, 255, 0, None):
        out = torch.full((batch, n, hv, 128), 7.0, dtype=BF, device="cuda")
        if fill is not None:
            ws.fill_(fill)
        st.delta[0].copy_(d["state"])
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws, lens=ln)
        first = first or (out.clone(), st.delta.clone())
        assert torch.equal(out, first[0]) and torch.equal(st.delta, first[1])
    past, _ = fp32_check(out, st.delta[0], x, hk, True, lens=lens)
    assert (f64(out)[past] == 7.0).all() and rma.gdn_get_status(st) == 0
    # one key head's value heads alone go in two launches
    r = hv // hk
    few = rma.GdnState(rma.GdnConfig(batch=batch, n_k_heads=1, n_v_heads=r))
    few.delta[0].copy_(d["state"][:, -r:])
    q = torch.cat((d["qkv"][..., (hk - 1) * 128:hk * 128], d["qkv"][..., (2 * hk - 1) * 128:2 * hk * 128], d["qkv"][..., -r * 128:]), -1)
    one = torch.full((batch, n, r, 128), 7.0, dtype=BF, device="cuda")
    rma.gdn_prefill(few, 0, q.contiguous(), d["a"][..., -r:].contiguous(), d["b"][..., -r:].contiguous(), d["a_log"][-r:].contiguous(),
                    d["dt_bias"][-r:].contiguous(), one, few.workspace(n), lens=ln)
    assert torch.equal(one, out[:, :, -r:]) and torch.equal(few.delta[0], st.delta[0, :, -r:])


def test_two_cooperative_launches_at_once_and_replayed():
    """Two such blocks of two states on two streams at once, then both replayed from graphs at once, among calls of the other
    kinds: the bits of the calls alone."""
    rma, sides = lib(), []
    for side in range(2):
        _, st, d, _ = delta_case(1, 2048, 16, 16, seed=610 + side)
        w = si.f32_normal((st.cfg.channels, 4), 612 + side, std=0.5).cuda()
        ws, out = st.workspace(2048), torch.empty(1, 2048, 16, 128, dtype=BF, device="cuda")
        y, one = torch.empty_like(d["qkv"]), torch.empty(1, 16, 128, dtype=BF, device="cuda")

        def call(st=st, d=d, w=w, ws=ws, out=out, y=y, one=one):
            rma.gdn_conv(st, 0, d["qkv"], w, y)
            rma.gdn_prefill(st, 0, y, d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws)
            rma.gdn_decode_step(st, 0, y[:, 99].contiguous(), d["a"][:, 99], d["b"][:, 99], d["a_log"], d["dt_bias"], one)

        call()
        torch.cuda.synchronize()
        sides.append((st, d, out, one, (out.clone(), one.clone(), st.buffer.clone()), call, torch.cuda.Stream(), torch.cuda.CUDAGraph()))

    def at_once(run):
        for st, d, out, *_ in sides:
            st.conv.zero_()
            st.delta[0].copy_(d["state"])
            out.fill_(3.0)
        torch.cuda.synchronize()
        for side in sides:
            with torch.cuda.stream(side[6]):
                run(side)
        torch.cuda.synchronize()
        for st, d, out, one, want, *_ in sides:
            assert torch.equal(out, want[0]) and torch.equal(one, want[1]) and torch.equal(st.buffer, want[2])
            assert rma.gdn_get_status(st) == 0

    for _ in range(3):
        at_once(lambda side: side[5]())
    for side in sides:
        with torch.cuda.graph(side[7], stream=side[6]):
            side[5]()
    for _ in range(3):
        at_once(lambda side: side[7].replay())
