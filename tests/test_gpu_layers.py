"""GPU parity of the layers around RMA attention against the FP64 oracle.

Tolerances.  A BF16 output carries half a step, 2^-8 of its value, plus the error of the arithmetic
before the rounding:
  rotation, convolution   FP32 sums of at most 256 terms of the row: 2^-15 of the largest term;
  delta rule, outputs     the chunked form rounds three factors of its products (state, weights, updates)
                          to FP16, half a step 2^-11 each, so 4 x 2^-11 of the sum of absolute terms
                          covers them and the FP32 sums;
  delta rule, state       FP32 sums of at most 192 terms a chunk, 192 x 2^-24 < 2^-16 of the sum of
                          absolute terms, factors carried to 2^-21: 2^-15 of the largest such sum.
The convolution state is a copy and has to be equal.
"""
import numpy as np
import pytest
import torch

import oracle
import synth_inputs as si
from _gpu import TOL, lib, make_pair, output_error
from _util import to_np

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def f64(t):
    return t.detach().cpu().double().numpy()


def close(got, ref, slack, what=""):
    got = f64(got)
    ok = np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + slack
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {(~ok).sum()} of {ok.size} off, first {i}: {got[i]} for {ref[i]}")


# ---------------------------------------------------------------- norm and rotation

def rope_case(batch, n, groups, pairs, seed, slots=8):
    rma = lib()
    st = rma.State(rma.Config(batch=batch, n_layers=2, n_groups=groups, ring_slots=slots, bank_slots=slots, pend_slots=slots))
    qk = si.bf16_normal((batch, n, 5 * groups * 256 + 64), seed).cuda()   # queries, keys, and 64 values of something else
    q = qk[..., :4 * groups * 256].view(batch, n, 4 * groups, 256)
    k = qk[..., 4 * groups * 256:5 * groups * 256].view(batch, n, groups, 256)
    w_q, w_k = 1 + si.f32_normal((256,), seed + 1, std=0.2).cuda(), 1 + si.f32_normal((256,), seed + 2, std=0.2).cuda()
    f = 1e6 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    q_out, k_out = (torch.full((batch, n, h, 256), 7.0, dtype=BF, device="cuda") for h in (4 * groups, groups))
    return rma, st, q, k, w_q, w_k, f.cuda(), q_out, k_out


def rope_check(q, k, w_q, w_k, f, q_out, k_out, pos_q, pos_k, eps=1e-6, interleaved=False):
    for x, w, out, pos in ((q, w_q, q_out, pos_q), (k, w_k, k_out, pos_k)):
        ref = oracle.norm_rope(f64(x), f64(w), pos, f64(f), eps, interleaved)
        big = np.abs(oracle.norm_rope(f64(x), f64(w), pos, [], eps)).max(-1, keepdims=True)
        close(out, ref, 2.0 ** -15 * big, "norm_rope")


@pytest.mark.parametrize("batch,n,groups,pairs,interleaved", [
    (1, 1, 4, 32, False), (1, 1, 1, 128, True), (3, 5, 4, 128, False), (2, 7, 3, 33, False), (2, 7, 3, 33, True),
    (5, 1, 2, 1, False), (2, 3, 2, 0, False), (1, 300, 1, 100, True)])
def test_norm_rope_at_given_positions(batch, n, groups, pairs, interleaved):
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(batch, n, groups, pairs, seed=10 + n)
    pos = si.uniform_int((batch, n), 0, 1 << 18, 3).to(torch.int32)
    pos[0, 0] = 2 ** 31 - 1
    pos[-1, -1] = -5
    rma.qk_norm_rope(st, 1, q, k, w_q, w_k, f if pairs else None, q_out, k_out, positions=pos.cuda(), interleaved=interleaved)
    p = pos.numpy()
    rope_check(q, k, w_q, w_k, f, q_out, k_out, p, p, interleaved=interleaved)
    assert rma.get_status(st) == 0


def test_norm_rope_takes_the_counters_places_of_each_group():
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(3, 4, 2, 32, seed=20)
    at = torch.tensor([[[131072, 5], [0, 77], [9, 9]]] * 2, dtype=torch.int32)
    at[0] += 1000
    st.counters[..., 0] = at.cuda()
    rma.qk_norm_rope(st, 1, q, k, w_q, w_k, f, q_out, k_out)
    pk = at[1].numpy()[:, None, :] + np.arange(4)[None, :, None]
    rope_check(q, k, w_q, w_k, f, q_out, k_out, np.repeat(pk, 4, 2), pk)
    assert rma.get_status(st) == 0
    st.counters[1, 1, 1, 0] = -3   # a corrupted counter counts as 0
    rma.qk_norm_rope(st, 1, q, k, w_q, w_k, f, q_out, k_out)
    pk[1, :, 1] = np.arange(4)
    rope_check(q, k, w_q, w_k, f, q_out, k_out, np.repeat(pk, 4, 2), pk)
    assert rma.get_status(st) == rma.STATUS_BAD_COUNTERS


def test_norm_rope_in_place_and_special_rows():
    """In place gives the same bits; a NaN stays in its head; zero rows stay zero; q and k of one token may be
    [B, heads, 256]."""
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(2, 3, 2, 64, seed=30)
    q, k = q.contiguous(), k.contiguous()
    q[1, 2, 3, 17] = float("nan")
    q[0, 0, 0] = 0
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    rma.qk_norm_rope(st, 0, q, k, w_q, w_k, f, q_out, k_out, positions=pos)
    bad = torch.isnan(q_out.float()).all(-1)
    assert bad[1, 2, 3] and bad.sum() == 1 and not torch.isnan(k_out.float()).any()
    assert (q_out[0, 0, 0] == 0).all()
    q1, k1 = q[:, 0].contiguous(), k[:, 0].contiguous()
    one_q, one_k = torch.empty_like(q1), torch.empty_like(k1)
    rma.qk_norm_rope(st, 0, q1, k1, w_q, w_k, f, one_q, one_k, positions=pos[:, 0].contiguous())
    assert torch.equal(one_q, q_out[:, 0]) and torch.equal(one_k, k_out[:, 0])
    rma.qk_norm_rope(st, 0, q, k, w_q, w_k, f, q, k, positions=pos)
    assert torch.equal(torch.nan_to_num(q.float(), 9.0), torch.nan_to_num(q_out.float(), 9.0)) and torch.equal(k, k_out)


def test_norm_rope_refusals():
    rma, st, q, k, w_q, w_k, f, q_out, k_out = rope_case(2, 3, 2, 64, seed=40)

    def refused(error, code=None, **change):
        a = dict(layer=0, q=q, k=k, w_q=w_q, w_k=w_k, inv_freq=f, q_out=q_out, k_out=k_out) | change
        with pytest.raises(error) as e:
            rma.qk_norm_rope(st, **a)
        if code is not None:
            assert e.value.code == code, str(e.value)

    refused(rma.RmaError, -1, layer=2)
    refused(rma.RmaError, -1, eps=-1.0)
    refused(rma.RmaError, -1, eps=float("nan"))
    refused(rma.RmaError, -1, inv_freq=torch.ones(129, dtype=torch.float64, device="cuda"))
    dense_q, dense_k = q.contiguous(), k.contiguous()
    refused(rma.RmaError, -1, q=dense_q, q_out=dense_q, k=dense_k, k_out=dense_q.view(-1)[:dense_k.numel()].view_as(k_out))
    flat = torch.zeros(q_out.numel() + 8, dtype=BF, device="cuda")
    flat[:q.numel()] = dense_q.view(-1)
    refused(rma.RmaError, -1, q=flat[:-8].view_as(dense_q), q_out=flat[8:].view_as(q_out))   # shifted by 8 values
    refused(rma.RmaError, -5, q_out=torch.zeros(q_out.numel() + 1, dtype=BF, device="cuda")[1:].view_as(q_out))
    refused(TypeError, inv_freq=f.float())
    refused(TypeError, q=q.float())
    refused(TypeError, q=q.cpu())
    refused(ValueError, k=k[:, :2])
    refused(ValueError, q=q[..., ::2])
    refused(ValueError, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))
    odd = torch.zeros(2, 3, 8 * 256 + 4, dtype=BF, device="cuda")[..., :2048].view(2, 3, 8, 256)
    refused(rma.RmaError, -1, q=odd)   # a stride that is no multiple of 8


# ---------------------------------------------------------------- convolution

@pytest.mark.parametrize("batch,n,hk,hv,bias,lens", [
    (1, 1, 1, 1, False, None), (3, 1, 2, 4, True, None), (300, 1, 1, 1, False, [1, 0] * 150),
    (2, 2, 1, 3, True, [2, 1]), (2, 33, 1, 1, False, None), (4, 70, 1, 2, True, [70, 0, 3, 65]), (1, 200, 2, 2, False, None)])
def test_convolution(batch, n, hk, hv, bias, lens):
    rma = lib()
    st = rma.GdnState(rma.GdnConfig(batch=batch, n_layers=2, n_k_heads=hk, n_v_heads=hv))
    C = st.cfg.channels
    st.conv.copy_(si.bf16_normal(tuple(st.conv.shape), 1).cuda())
    before = st.buffer.clone()
    x = si.bf16_normal((batch, n, C + 24), 2).cuda()[..., 8:C + 8]   # a view of wider rows
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:
        for b, m in enumerate(lens):
            x[b, m:] = float("nan")
    w, bs = si.f32_normal((C, 4), 3, std=0.5).cuda(), (si.f32_normal((C,), 4).cuda() if bias else None)
    out = torch.full((batch, n, C), 7.0, dtype=BF, device="cuda")
    old = st.conv[1].clone()
    rma.gdn_conv(st, 1, x, w, out, bias=bs, lens=ln)
    ref, new = oracle.conv_silu(f64(x), f64(old), f64(w), None if bs is None else f64(bs), lens)
    past = np.isnan(ref)
    assert (f64(out)[past] == 7.0).all()
    size = 5 * 8.0   # five terms, |w| < 2.5 and |x| < 5 wherever these seeds go: slack 2^-15 of them
    close(torch.where(torch.from_numpy(past).cuda(), 0.0, out.float()), np.where(past, 0.0, ref), 2.0 ** -15 * size, "conv")
    assert np.array_equal(f64(st.conv[1]), new)
    st.conv[1].copy_(old)
    assert torch.equal(st.buffer, before)   # nothing else of the state changed
    assert rma.gdn_get_status(st) == 0


def test_convolution_in_pieces_gives_the_same_bits():
    rma = lib()
    cfg = rma.GdnConfig(batch=2, n_k_heads=1, n_v_heads=2)
    x = si.bf16_normal((2, 103, cfg.channels), 5).cuda()
    w = si.f32_normal((cfg.channels, 4), 6).cuda()
    one, many = rma.GdnState(cfg), rma.GdnState(cfg)
    whole = torch.empty_like(x)
    rma.gdn_conv(one, 0, x, w, whole)
    at = 0
    for m in (1, 2, 1, 64, 3, 32):
        piece = torch.empty(2, m, cfg.channels, dtype=BF, device="cuda")
        rma.gdn_conv(many, 0, x[:, at:at + m].contiguous(), w, piece)
        assert torch.equal(piece, whole[:, at:at + m])
        at += m
    assert at == 103 and torch.equal(one.conv, many.conv)


# ---------------------------------------------------------------- delta rule

def delta_case(batch, n, hk, hv, seed, l2norm=True, fresh=False, lens=None, layers=1):
    rma = lib()
    x = si.gdn_inputs(batch, n, hk, hv, seed=seed)
    if not l2norm:
        x["qkv"] = (x["qkv"].float() * 0.08).to(BF)   # keys of norm about 1: the recurrence stays bounded
    if fresh:
        x["state"].zero_()
    st = rma.GdnState(rma.GdnConfig(batch=batch, n_layers=layers, n_k_heads=hk, n_v_heads=hv, qk_l2norm=l2norm))
    st.delta[-1].copy_(x["state"].cuda())
    d = {k: v.cuda() for k, v in x.items()}
    return rma, st, d, x


def delta_check(out, state, x, hk, lens=None, l2norm=True, what=""):
    ref, S, osize, size = oracle.delta_rule(*[f64(x[k]) for k in ("qkv", "a", "b", "a_log", "dt_bias", "state")], hk,
                                            l2norm=l2norm, lens=lens)
    past = np.isnan(ref)
    close(torch.where(torch.from_numpy(past).cuda(), 0.0, out.float().view(ref.shape)), np.where(past, 0.0, ref),
          4 * 2.0 ** -11 * osize, what + " out")
    off = np.abs(f64(state) - S)
    lim = 2.0 ** -15 * size.max((-1, -2), keepdims=True)
    assert (off <= lim).all(), f"{what} state: {(off / lim).max()} times the tolerance"
    return past


@pytest.mark.parametrize("batch,hk,hv,l2norm", [(1, 1, 1, True), (1, 16, 32, True), (3, 2, 6, True), (40, 4, 8, True),
                                                (5, 3, 3, False), (400, 1, 1, True)])
def test_step(batch, hk, hv, l2norm):
    rma, st, d, x = delta_case(batch, 1, hk, hv, seed=50, l2norm=l2norm, layers=2)
    zero = st.delta[0].clone()
    ab = torch.cat((d["b"][:, 0], d["a"][:, 0]), -1)   # one projection's rows
    out = torch.empty(batch, hv, 128, dtype=BF, device="cuda")
    rma.gdn_decode_step(st, 1, d["qkv"], ab[:, hv:], ab[:, :hv], d["a_log"], d["dt_bias"], out)
    delta_check(out, st.delta[1], x, hk, l2norm=l2norm)
    assert torch.equal(st.delta[0], zero)


def test_step_with_infinite_gates():
    """a = inf forgets, a = -inf keeps; b = -inf writes nothing, b = inf replaces."""
    rma, st, d, x = delta_case(1, 1, 1, 4, seed=51)
    inf = float("inf")
    x["a"][0, 0] = torch.tensor([inf, -inf, -inf, inf])
    x["b"][0, 0] = torch.tensor([inf, -inf, inf, -inf])
    out = torch.empty(1, 4, 128, dtype=BF, device="cuda")
    rma.gdn_decode_step(st, 0, d["qkv"], x["a"].cuda(), x["b"].cuda(), d["a_log"], d["dt_bias"], out)
    delta_check(out, st.delta[0], x, 1)
    assert torch.equal(st.delta[0, 0, 1].cpu(), x["state"][0, 1]) and (st.delta[0, 0, 3] == 0).all()


@pytest.mark.parametrize("batch,n,hk,hv,fresh,l2norm", [
    (1, 1, 1, 1, False, True), (1, 2, 2, 4, True, True), (2, 17, 1, 3, False, True), (1, 63, 1, 1, False, True),
    (1, 64, 1, 2, False, True), (1, 65, 1, 1, True, True), (3, 100, 2, 2, False, False), (2, 128, 1, 1, False, True),
    (1, 129, 2, 6, True, True), (1, 100, 16, 32, True, True), (2, 333, 1, 2, False, True), (70, 70, 1, 2, True, True),
    (1, 700, 1, 1, False, False)])
def test_block(batch, n, hk, hv, fresh, l2norm):
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=60 + n, l2norm=l2norm, fresh=fresh, layers=2)
    zero = st.delta[0].clone()
    out = torch.empty(batch, n, hv, 128, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 1, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n))
    delta_check(out, st.delta[1], x, hk, l2norm=l2norm)
    assert torch.equal(st.delta[0], zero) and rma.gdn_get_status(st) == 0


@pytest.mark.parametrize("n,lens", [(5, [5, 0, 1]), (64, [64, 63, 1]), (130, [0, 130, 65]), (200, [128, 127, 200]),
                                    (66, [0, 0, 0])])
def test_block_of_lengths(n, lens):
    """Rows past a length hold NaN and are neither read nor written; a length of 0 keeps every bit of the state."""
    rma, st, d, x = delta_case(3, n, 2, 4, seed=70 + n)
    for b, m in enumerate(lens):
        for k in ("qkv", "a", "b"):
            d[k][b, m:] = float("nan")
    wide = torch.full((3 * n + 2, 4, 128), 7.0, dtype=BF, device="cuda")
    out = wide[1:-1].view(3, n, 4, 128)
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n),
                    lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    past = delta_check(out, st.delta[0], x, 2, lens=lens)
    assert (f64(out)[past] == 7.0).all() and (wide[0] == 7).all() and (wide[-1] == 7).all()
    for b, m in enumerate(lens):
        if m == 0:
            assert torch.equal(st.delta[0, b].cpu(), x["state"][b])
    assert rma.gdn_get_status(st) == 0


def test_block_of_more_heads_than_multiprocessors():
    """180 (sequence, head) pairs of very different lengths: a multiprocessor takes several, one after another."""
    B, n = 60, 70
    lens = si.uniform_int((B,), 0, n, 71).to(torch.int32)
    lens[:6] = torch.tensor([n, 0, 64, 65, 1, 0])
    rma, st, d, x = delta_case(B, n, 1, 3, seed=72)
    out = torch.full((B, n, 3, 128), 7.0, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(n), lens=lens.cuda())
    past = delta_check(out, st.delta[0], x, 1, lens=lens.numpy())
    assert (f64(out)[past] == 7.0).all() and torch.equal(st.delta[0, 1].cpu(), x["state"][1])
    again = torch.full_like(out, 7.0)   # without lengths of 0, in the batch's own order
    few = rma.GdnState(rma.GdnConfig(batch=1, n_k_heads=1, n_v_heads=3))
    for b in (0, 2, 3):
        few.delta[0].copy_(d["state"][b:b + 1])
        m = int(lens[b])
        o = torch.empty(1, m, 3, 128, dtype=BF, device="cuda")
        p = {k: d[k][b:b + 1, :m].contiguous() for k in ("qkv", "a", "b")}
        rma.gdn_prefill(few, 0, p["qkv"], p["a"], p["b"], d["a_log"], d["dt_bias"], o, few.workspace(m))
        again[b, :m] = o[0]
        assert torch.equal(again[b], out[b]) and torch.equal(few.delta[0, 0], st.delta[0, b])


@pytest.mark.parametrize("batch,hk,hv,n,lens", [(1, 1, 2, 1700, None), (3, 2, 4, 1601, [1601, 500, 40]), (2, 2, 20, 1540, [0, 1537])])
def test_long_blocks_of_few_heads(batch, hk, hv, n, lens):
    """Prompts of many chunks, back to back on one workspace; sequences end in any chunk."""
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=73 + batch)
    out = torch.full((batch, n, hv, 128), 7.0, dtype=BF, device="cuda")
    ws = st.workspace(n)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(3):
        st.delta[0].copy_(d["state"])
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws, lens=ln)
        if first is None:
            first = (out.clone(), st.delta.clone())
        assert torch.equal(out, first[0]) and torch.equal(st.delta, first[1])
    past = delta_check(out, st.delta[0], x, hk, lens=lens)
    assert (f64(out)[past] == 7.0).all() and rma.gdn_get_status(st) == 0


@pytest.mark.parametrize("batch,hk,hv,n,lens", [(1, 1, 2, 2049, None), (3, 2, 4, 2100, [2100, 0, 1990]), (2, 3, 9, 2050, [777, 2050]),
                                                (1, 5, 5, 1985, None), (1, 1, 9, 2000, [1999])])
def test_blocks_long_enough_for_one_launch(batch, hk, hv, n, lens):
    """32 chunks and more of few heads go in one launch: against the oracle, whatever the workspace held (its flags
    among it), with NaN in the padding, and the same bits every time."""
    rma, st, d, x = delta_case(batch, n, hk, hv, seed=173 + batch)
    ln = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    if lens is not None:
        for b, m in enumerate(lens):
            d["qkv"][b, m:] = float("nan")
    ws = st.workspace(n)
    first = None
    for fill in (1, 255, 0, None):
        out = torch.full((batch, n, hv, 128), 7.0, dtype=BF, device="cuda")
        if fill is not None:
            ws.fill_(fill)
        st.delta[0].copy_(d["state"])
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws, lens=ln)
        if first is None:
            first = (out.clone(), st.delta.clone())
        assert torch.equal(out, first[0]) and torch.equal(st.delta, first[1])
    past = delta_check(out, st.delta[0], x, hk, lens=lens)
    assert (f64(out)[past] == 7.0).all() and rma.gdn_get_status(st) == 0


def test_long_blocks_at_once_and_replayed():
    """Two long blocks of two states on two streams at once, then both replayed from graphs at once, between calls of
    the other kinds: the bits of the calls alone."""
    rma = lib()
    sides = []
    for side in range(2):
        rma, st, d, x = delta_case(1, 2048, 2, 4, seed=180 + side)
        w = si.f32_normal((st.cfg.channels, 4), 182 + side, std=0.5).cuda()
        ws, out = st.workspace(2048), torch.empty(1, 2048, 4, 128, dtype=BF, device="cuda")
        y, one = torch.empty_like(d["qkv"]), torch.empty(1, 4, 128, dtype=BF, device="cuda")

        def call(st=st, d=d, w=w, ws=ws, out=out, y=y, one=one):
            rma.gdn_conv(st, 0, d["qkv"], w, y)
            rma.gdn_prefill(st, 0, y, d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws)
            rma.gdn_decode_step(st, 0, y[:, 99].contiguous(), d["a"][:, 99], d["b"][:, 99], d["a_log"], d["dt_bias"], one)

        call()
        torch.cuda.synchronize()
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        sides.append((st, d, out, one, (out.clone(), one.clone(), st.buffer.clone()), call, stream, graph))

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


def test_lengths_out_of_range_are_clamped_and_reported():
    rma, st, d, x = delta_case(2, 70, 1, 2, seed=80)
    out = torch.full((2, 70, 2, 128), 7.0, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(70),
                    lens=torch.tensor([1000, -4], dtype=torch.int32, device="cuda"))
    delta_check(out, st.delta[0], x, 1, lens=[70, 0])
    assert rma.gdn_get_status(st) == rma.STATUS_BAD_LENGTH and rma.gdn_get_status(st) == 0
    y = torch.empty_like(d["qkv"])
    rma.gdn_conv(st, 0, d["qkv"], torch.zeros(st.cfg.channels, 4, device="cuda"), y,
                 lens=torch.tensor([71, 3], dtype=torch.int32, device="cuda"))
    assert rma.gdn_get_status(st) == rma.STATUS_BAD_LENGTH


def test_block_of_one_repeated_key():
    """The same key again and again, written fully and never forgotten: every weight between the tokens of a
    chunk is 1, the triangular system at its stiffest."""
    rma, st, d, x = delta_case(1, 150, 1, 2, seed=81)
    x["qkv"][:, :, 128:256] = x["qkv"][:, :1, 128:256]
    x["a"][:] = -30.0
    x["b"][:] = 30.0
    d = {k: v.cuda() for k, v in x.items()}
    out = torch.empty(1, 150, 2, 128, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(150))
    delta_check(out, st.delta[0], x, 1)


def test_block_with_strong_decays_among_weak_ones():
    """Tokens that forget all (also by a = inf) next to ones that forget nothing: a weak decay after a strong one
    keeps its precision, and the updates before it are gone."""
    rma, st, d, x = delta_case(2, 140, 1, 2, seed=82)
    x["a"][:] = -6.0
    for t, v in ((3, 1000.0), (20, float("inf")), (21, 50.0), (64, 300.0), (100, float("inf")), (127, 2000.0)):
        x["a"][:, t] = v
    x["b"][:, 5] = -float("inf")
    x["b"][:, 6] = float("inf")
    d = {k: v.cuda() for k, v in x.items()}
    out = torch.empty(2, 140, 2, 128, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(140))
    delta_check(out, st.delta[0], x, 1)


@pytest.mark.parametrize("k_scale,v_scale,s_scale", [(2.0 ** -60, 2.0 ** 40, 1.0), (2.0 ** 50, 2.0 ** -50, 2.0 ** -70),
                                                     (1.0, 2.0 ** 90, 2.0 ** 60), (2.0 ** -20, 0.0, 0.0)])
def test_block_of_extreme_magnitudes(k_scale, v_scale, s_scale):
    """Keys, values and states far outside FP16's range, spread over eight binades within a head and by column."""
    rma, st, d, x = delta_case(1, 100, 1, 1, seed=83)
    spread = 2.0 ** si.uniform_int((1, 100, 384), -4, 4, 9).float()
    scale = torch.cat((torch.full((256,), k_scale), torch.full((128,), v_scale)))
    x["qkv"] = (x["qkv"].float() * spread * scale).to(BF)
    x["state"] = x["state"] * s_scale * 2.0 ** si.uniform_int((128,), -20, 20, 10).float()
    d = {k: v.cuda() for k, v in x.items()}
    st = rma.GdnState(rma.GdnConfig(n_k_heads=1, n_v_heads=1, l2_eps=0.0))
    st.delta[0].copy_(d["state"])
    out = torch.empty(1, 100, 1, 128, dtype=BF, device="cuda")
    rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(100))
    ref, S, osize, size = oracle.delta_rule(*[f64(x[k]) for k in ("qkv", "a", "b", "a_log", "dt_bias", "state")], 1, l2_eps=0.0)
    # value columns do not meet, so each is held to its own size
    close(out, ref, 4 * 2.0 ** -11 * osize + 2.0 ** -120, "out")
    lim = 2.0 ** -15 * size.max(-2, keepdims=True) + 2.0 ** -120
    assert (np.abs(f64(st.delta[0]) - S) <= lim).all()


def test_blocks_and_steps_follow_one_another():
    """A prompt in two blocks, then three tokens: the state carries over between the forms and the calls."""
    rma, st, d, x = delta_case(2, 203, 2, 4, seed=84)
    out = torch.empty(2, 203, 4, 128, dtype=BF, device="cuda")
    for lo, hi in ((0, 130), (130, 200)):
        o = torch.empty(2, hi - lo, 4, 128, dtype=BF, device="cuda")
        p = {k: d[k][:, lo:hi].contiguous() for k in ("qkv", "a", "b")}
        rma.gdn_prefill(st, 0, p["qkv"], p["a"], p["b"], d["a_log"], d["dt_bias"], o, st.workspace(hi - lo))
        out[:, lo:hi] = o
    for t in range(200, 203):
        o = torch.empty(2, 4, 128, dtype=BF, device="cuda")
        rma.gdn_decode_step(st, 0, d["qkv"][:, t].contiguous(), d["a"][:, t], d["b"][:, t], d["a_log"], d["dt_bias"], o)
        out[:, t] = o
    delta_check(out, st.delta[0], x, 2)


def test_block_repeats_to_the_bit():
    rma, st, d, x = delta_case(3, 150, 2, 4, seed=85)
    outs, states = [], []
    ws = st.workspace(150)
    for fill in (0, 255, 77):
        ws.fill_(fill)   # what a workspace holds does not matter
        st.delta[0].copy_(d["state"])
        out = torch.empty(3, 150, 4, 128, dtype=BF, device="cuda")
        rma.gdn_prefill(st, 0, d["qkv"], d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws)
        outs.append(out)
        states.append(st.delta.clone())
    assert all(torch.equal(outs[0], o) for o in outs) and all(torch.equal(states[0], s) for s in states)


def test_gdn_calls_replayed_from_graphs_on_two_streams():
    """Two states' block and token calls captured on two streams, replayed at once over their own workspaces."""
    rma = lib()
    sides = []
    for side in range(2):
        rma, st, d, x = delta_case(2, 100, 2, 4, seed=86 + side)
        w = si.f32_normal((st.cfg.channels, 4), 90 + side, std=0.5).cuda()
        ws, out = st.workspace(100), torch.empty(2, 100, 4, 128, dtype=BF, device="cuda")
        y, one = torch.empty_like(d["qkv"]), torch.empty(2, 4, 128, dtype=BF, device="cuda")

        def call(st=st, d=d, w=w, ws=ws, out=out, y=y, one=one):
            rma.gdn_conv(st, 0, d["qkv"], w, y)
            rma.gdn_prefill(st, 0, y, d["a"], d["b"], d["a_log"], d["dt_bias"], out, ws)
            rma.gdn_decode_step(st, 0, y[:, 99].contiguous(), d["a"][:, 99], d["b"][:, 99], d["a_log"], d["dt_bias"], one)

        call()
        torch.cuda.synchronize()
        want = (out.clone(), one.clone(), st.buffer.clone())
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            call()
        sides.append((st, d, out, one, want, call, stream, graph))   # call keeps the captured buffers alive
    for _ in range(3):
        for st, d, out, one, want, call, stream, graph in sides:
            st.conv.zero_()
            st.delta[0].copy_(d["state"])
            out.fill_(3.0)
        torch.cuda.synchronize()
        for *_, stream, graph in sides:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for st, d, out, one, want, call, stream, graph in sides:
            assert torch.equal(out, want[0]) and torch.equal(one, want[1]) and torch.equal(st.buffer, want[2])


def test_large_state_offsets():
    """More than 2^31 values of state: the last sequences give what they give alone."""
    rma = lib()
    B = 4100
    x = si.gdn_inputs(4, 1, 16, 32, seed=91, device="cuda")
    st, few = (rma.GdnState(rma.GdnConfig(batch=b)) for b in (B, 4))
    few.delta[0].copy_(x["state"])
    st.delta[0, B - 4:].copy_(x["state"])
    qkv = torch.zeros(B, 8192, dtype=BF, device="cuda")
    a = torch.zeros(B, 32, dtype=BF, device="cuda")
    b = torch.zeros_like(a)
    qkv[B - 4:], a[B - 4:], b[B - 4:] = x["qkv"][:, 0], x["a"][:, 0], x["b"][:, 0]
    out, out4 = torch.empty(B, 32, 128, dtype=BF, device="cuda"), torch.empty(4, 32, 128, dtype=BF, device="cuda")
    assert st.delta.numel() > 2 ** 31
    rma.gdn_decode_step(st, 0, qkv, a, b, x["a_log"], x["dt_bias"], out)
    rma.gdn_decode_step(few, 0, x["qkv"], x["a"], x["b"], x["a_log"], x["dt_bias"], out4)
    # the two batches may split a head's columns differently over CTAs: sums in another order
    torch.testing.assert_close(out[B - 4:].float(), out4.float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(st.delta[0, B - 4:], few.delta[0], rtol=1e-5, atol=1e-6)
    assert (out[:B - 4] == 0).all() and (st.delta[0, :B - 4] == 0).all()


def test_gdn_refusals():
    rma, st, d, x = delta_case(2, 70, 1, 2, seed=92)
    ws = st.workspace(70)
    out = torch.empty(2, 70, 2, 128, dtype=BF, device="cuda")
    before = st.buffer.clone()

    def refused(error, code=None, call="gdn_prefill", **change):
        a = dict(layer=0, qkv=d["qkv"], a=d["a"], b=d["b"], a_log=d["a_log"], dt_bias=d["dt_bias"], out=out, ws=ws)
        if call == "gdn_conv":
            a = dict(layer=0, x=d["qkv"], w=torch.zeros(512, 4, device="cuda"), out=torch.empty_like(d["qkv"]))
        with pytest.raises(error) as e:
            getattr(rma, call)(st, **(a | change))
        if code is not None:
            assert e.value.code == code, str(e.value)

    refused(rma.RmaError, -1, layer=1)
    refused(rma.RmaError, -1, layer=-1)
    refused(rma.RmaError, -1, out=d["qkv"].view(-1)[:out.numel()].view_as(out))
    refused(rma.RmaError, -3, ws=ws[:ws.numel() - 1])
    refused(rma.RmaError, -5, ws=ws[16:])
    big = torch.zeros(ws.numel() + 2 * d["qkv"].numel(), dtype=torch.uint8, device="cuda")
    inside = big[1024:1024 + 2 * d["qkv"].numel()].view(BF).view_as(d["qkv"])
    refused(rma.RmaError, -1, ws=big, qkv=inside)
    refused(ValueError, b=torch.zeros(2, 70, 4, dtype=BF, device="cuda")[..., :2])   # not the spacing of a
    refused(ValueError, a=d["a"][:, :69])
    refused(ValueError, qkv=d["qkv"][..., :256])
    refused(TypeError, a_log=d["a_log"].double())
    refused(TypeError, lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    refused(ValueError, lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    shifted = torch.zeros(d["qkv"].numel() + 1, dtype=BF, device="cuda")[1:].view_as(d["qkv"])
    refused(rma.RmaError, -5, qkv=shifted)
    refused(rma.RmaError, -1, call="gdn_conv", out=d["qkv"])
    refused(rma.RmaError, -5, call="gdn_conv", out=shifted)
    refused(rma.RmaError, -1, call="gdn_conv", x=torch.zeros(2, 70, 516, dtype=BF, device="cuda")[..., :512])
    refused(ValueError, call="gdn_conv", w=torch.zeros(512, 3, device="cuda"))
    with pytest.raises(rma.RmaError):
        st.workspace(0)
    with pytest.raises(rma.RmaError):
        st.workspace(1 << 24)
    torch.cuda.synchronize()
    assert torch.equal(before, st.buffer)


def test_gdn_inputs_inside_the_state_are_refused():
    """A call updates its state while it reads its inputs, so none may lie there."""
    rma, st, d, x = delta_case(2, 1, 1, 2, seed=93)
    out, y = torch.empty(2, 2, 128, dtype=BF, device="cuda"), torch.empty(2, 512, dtype=BF, device="cuda")
    w = torch.zeros(512, 4, device="cuda")
    flat = st.delta.view(-1)
    gates = flat[:2].view(BF).view(2, 2)
    good = dict(qkv=d["qkv"], a=d["a"], b=d["b"], a_log=d["a_log"], dt_bias=d["dt_bias"], out=out)
    before = st.buffer.clone()
    for change in (dict(qkv=st.conv.view(-1)[:1024].view(2, 512)),
                   dict(a=gates), dict(b=gates), dict(a_log=flat[:2]), dict(dt_bias=flat[2:4]), dict(out=flat[:256].view(BF).view(2, 2, 128))):
        for call, more in (("gdn_decode_step", {}), ("gdn_prefill", dict(ws=st.workspace(1)))):
            with pytest.raises(rma.RmaError) as e:
                getattr(rma, call)(st, 0, **(good | change | more))
            assert e.value.code == -1
    for change in (dict(x=st.conv.view(-1)[:1024].view(2, 512)), dict(w=flat[:2048].view(512, 4)), dict(bias=flat[:512]),
                   dict(lens=flat[:2].view(torch.int32))):
        with pytest.raises(rma.RmaError) as e:
            rma.gdn_conv(st, 0, **(dict(x=d["qkv"], w=w, out=y) | change))
        assert e.value.code == -1
    torch.cuda.synchronize()
    assert torch.equal(before, st.buffer)


# ---------------------------------------------------------------- together

def test_a_prompt_and_tokens_through_a_delta_layer():
    """conv then delta rule over a padded batch of two prompts, then two tokens, against the oracle fed with the
    convolution's own BF16 outputs."""
    rma, st, d, x = delta_case(2, 90, 2, 4, seed=95, fresh=True)
    lens = [90, 41]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    w = si.f32_normal((st.cfg.channels, 4), 96, std=0.5).cuda()
    raw = d["qkv"]
    y, out = torch.zeros_like(raw), torch.empty(2, 90, 4, 128, dtype=BF, device="cuda")
    rma.gdn_conv(st, 0, raw, w, y, lens=ln)
    rma.gdn_prefill(st, 0, y, d["a"], d["b"], d["a_log"], d["dt_bias"], out, st.workspace(90), lens=ln)
    seen = x | {"qkv": y}
    past = delta_check(out, st.delta[0], seen, 2, lens=lens, what="prompt")
    assert past[1, 41:].all()
    for t in range(2):
        nxt = si.gdn_inputs(2, 1, 2, 4, seed=97 + t)
        nx = {k: v.cuda() for k, v in nxt.items()}
        old_conv, old = st.conv[0].clone(), st.delta[0].clone()
        y1, o1 = torch.empty(2, st.cfg.channels, dtype=BF, device="cuda"), torch.empty(2, 4, 128, dtype=BF, device="cuda")
        rma.gdn_conv(st, 0, nx["qkv"], w, y1)
        ref, _ = oracle.conv_silu(f64(nx["qkv"]), f64(old_conv), f64(w))
        close(y1.view(2, 1, -1), ref, 2.0 ** -15 * 40, "conv token")
        rma.gdn_decode_step(st, 0, y1, nx["a"], nx["b"], d["a_log"], d["dt_bias"], o1)
        delta_check(o1, st.delta[0], {"qkv": y1.view(2, 1, -1), "a": nx["a"], "b": nx["b"], "a_log": d["a_log"],
                                      "dt_bias": d["dt_bias"], "state": old}, 2, what=f"token {t}")
    assert (f64(st.conv[0][1, 0]) == f64(raw[1, 40])).all()   # the shorter prompt's last row, two tokens on


def test_rotation_then_attention():
    """qk_norm_rope feeding a prefill block and a decode step of the same layer, positions from the counters:
    the attention matches the oracle on the rotated rows, and the second call's positions follow the first's."""
    rma = lib()
    cfg = oracle.Config(batch=2, n_layers=1)
    st, ost = make_pair(cfg, seed=98, pos=[[[40] * 4, [900] * 4]], bank_fill=[[[30] * 4, [600] * 4]], pend_fill=0)
    w, b = si.gate_params(1, 16, 256, seed=98)
    f = (1e6 ** (-torch.arange(32, dtype=torch.float64) / 32)).cuda()
    w_q, w_k = 1 + si.f32_normal((256,), 99, std=0.1).cuda(), 1 + si.f32_normal((256,), 100, std=0.1).cuda()
    start = np.array([40, 900])
    for n in (20, 1, 1):
        x = si.prefill_inputs(2, n, 4, 4, 256, seed=101 + n)
        q, k = x["q"].cuda(), x["k"].cuda()
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        rma.qk_norm_rope(st, 0, q, k, w_q, w_k, f, qr, kr)
        pos = start[:, None] + np.arange(n)
        rope_check(q, k, w_q, w_k, f, qr, kr, pos, pos)
        out = torch.empty_like(q)
        rest = [x[i].cuda() for i in ("v", "cand_k", "cand_v", "cand_score")]
        run, ref = (rma.prefill_block, oracle.prefill_block) if n > 1 else (rma.decode_step, oracle.decode_step)
        run(st, 0, qr, kr, *rest, w[0].cuda(), b[0].cuda(), out, st.workspace(n))
        args = [to_np(t) for t in (qr, kr, *rest)]
        if n == 1:
            args = [t[:, 0] for t in args]
        want = ref(ost, 0, *args, to_np(w[0]), to_np(b[0]))
        assert output_error(to_np(out).reshape(want.shape), want) <= TOL
        start = start + n
    assert rma.get_status(st) == 0
