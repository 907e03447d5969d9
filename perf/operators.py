"""The layer operators around RMA attention: their cases, plain forms and 64-bit definitions.

Four operators of a model that interleaves RMA attention with gated-delta-rule layers:

  rot     RMS norm of each query and key head, then the position rotation (what makes the q and k of a
          decode step or prefill block);
  conv    the short causal depthwise convolution with SiLU and its three-token state;
  step    the gated delta rule, one token for every sequence (recurrent form);
  prompt  the gated delta rule over a block of tokens (chunked form), lengths differing by sequence.

Where ``own`` is false, ``run`` computes them with elementary torch operations in 32 bits; where it is
true it makes the calls a user of bounded_memory_attention_b200 makes.
"""
import math

import torch

own = False

DEV = "cuda"
HEAD = 128          # key and value width of a delta-rule head
WIDTH = 4           # taps of the short convolution
ROT_HEAD = 256      # width of an attention head
CHUNK = 64          # tokens per chunk of the plain chunked form
EPS = 1e-6
L2_EPS = 1e-6


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one sequence's next token at a far position: latency
        {"name": "rot_token_1", "op": "rot", "batch": 1, "tokens": 1, "groups": 4, "rotary": 64, "far": 131072,
         "interleaved": False, "counters": False},
        # a full decode batch, positions taken from the attention state's own counters
        {"name": "rot_token_512", "op": "rot", "batch": 512, "tokens": 1, "groups": 4, "rotary": 64, "far": 131072,
         "interleaved": False, "counters": True},
        # a prefill block of 256 tokens for eight sequences, the whole head rotated
        {"name": "rot_block_8x256", "op": "rot", "batch": 8, "tokens": 256, "groups": 4, "rotary": 256, "far": 32768,
         "interleaved": False, "counters": False},
        # a full decode batch through the convolution
        {"name": "conv_token_512", "op": "conv", "batch": 512, "tokens": 1, "k_heads": 16, "v_heads": 32, "bias": False,
         "ragged": False},
        # four prompts of different lengths in one padded batch
        {"name": "conv_prompt_4x2048", "op": "conv", "batch": 4, "tokens": 2048, "k_heads": 16, "v_heads": 32,
         "bias": True, "ragged": True},
        # one sequence's next token: latency
        {"name": "step_1", "op": "step", "batch": 1, "k_heads": 16, "v_heads": 32},
        # an odd batch of a smaller layer, one value head per key head
        {"name": "step_37", "op": "step", "batch": 37, "k_heads": 6, "v_heads": 6},
        # a full decode batch: 1 GiB of state read and written
        {"name": "step_512", "op": "step", "batch": 512, "k_heads": 16, "v_heads": 32},
        # a short prompt of odd length, from an empty state
        {"name": "prompt_1x100", "op": "prompt", "batch": 1, "tokens": 100, "k_heads": 16, "v_heads": 32,
         "ragged": False, "fresh": True},
        # a prefill block of 256 tokens for eight sequences, going on from their states
        {"name": "prompt_8x256", "op": "prompt", "batch": 8, "tokens": 256, "k_heads": 16, "v_heads": 32,
         "ragged": False, "fresh": False},
        # prompts of different lengths in one padded batch
        {"name": "prompt_6x1000", "op": "prompt", "batch": 6, "tokens": 1000, "k_heads": 8, "v_heads": 32,
         "ragged": True, "fresh": True},
        # one long prompt: the serial chain over the chunks counts
        {"name": "prompt_1x8192", "op": "prompt", "batch": 1, "tokens": 8192, "k_heads": 16, "v_heads": 32,
         "ragged": False, "fresh": True},
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["rot", "conv", "step", "prompt", "prompt"])
    if op == "rot":
        tokens = rng.choice([1, _log_int(rng, 1, 256)])
        return {"op": op, "batch": _log_int(rng, 1, max(1, min(512, 2048 // tokens))), "tokens": tokens,
                "groups": rng.choice([1, 2, 3, 4]), "rotary": 2 * rng.randint(1, 128), "far": _log_int(rng, 16, 262144),
                "interleaved": rng.random() < 0.5, "counters": rng.random() < 0.5}
    k_heads = rng.randint(1, 16)
    v_heads = k_heads * rng.choice([1, 2] + ([3, 4] if k_heads <= 8 else []))
    if op == "conv":
        tokens = rng.choice([1, _log_int(rng, 2, 4096)])
        return {"op": op, "batch": _log_int(rng, 1, max(1, min(512, 8192 // tokens))), "tokens": tokens,
                "k_heads": k_heads, "v_heads": v_heads, "bias": rng.random() < 0.5, "ragged": rng.random() < 0.5}
    if op == "step":
        return {"op": op, "batch": _log_int(rng, 1, 512), "k_heads": k_heads, "v_heads": v_heads}
    tokens = _log_int(rng, 1, 8000)
    return {"op": op, "batch": _log_int(rng, 1, max(1, min(64, 8192 // tokens))), "tokens": tokens,
            "k_heads": k_heads, "v_heads": v_heads, "ragged": rng.random() < 0.5, "fresh": rng.random() < 0.5}


def _channels(case):
    return (2 * case["k_heads"] + case["v_heads"]) * HEAD


# ---------------------------------------------------------------- inputs (from the seed alone)

def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV) * std

    def uniform(low, high, *shape):
        return torch.rand(shape, generator=g, device=DEV) * (high - low) + low

    bf = torch.bfloat16
    d = {}
    B = case["batch"]
    if case["op"] == "rot":
        n, G = case["tokens"], case["groups"]
        # one projection's output row: queries, then keys
        d["qk"] = normal(B, n, 5 * G * ROT_HEAD).to(bf)
        d["w_q"], d["w_k"] = uniform(0.5, 1.5, ROT_HEAD), uniform(0.5, 1.5, ROT_HEAD)
        d["start"] = torch.randint(max(1, case["far"] - case["far"] // 8), case["far"] + 1, (B,), generator=g, device=DEV)
        i = torch.arange(case["rotary"] // 2, device=DEV, dtype=torch.float64)
        d["inv_freq"] = 1e7 ** (-2.0 * i / case["rotary"])
        return d
    C, HV, HK = _channels(case), case["v_heads"], case["k_heads"]
    n = case.get("tokens", 1)
    if case.get("ragged"):
        d["lens"] = torch.randint(max(1, n // 3), n + 1, (B,), generator=g, device=DEV).to(torch.int32)
        d["lens"][0] = n
    if case["op"] == "conv":
        d["x"] = normal(B, n, C).to(bf)
        d["w"] = normal(C, WIDTH, std=0.5)
        d["bias"] = normal(C, std=0.1) if case["bias"] else None
        d["state"] = normal(B, WIDTH - 1, C).to(bf)
        return d
    # what the convolution hands on: SiLU of normal values, queries and keys first
    x = normal(B, n, C)
    d["qkv"] = (x * torch.sigmoid(x)).to(bf)
    d["a"], d["b"] = normal(B, n, HV).to(bf), normal(B, n, HV).to(bf)
    # decay rates from 1 to 16 and time steps from 0.001 to 0.1, as such layers are initialised
    d["a_log"] = torch.log(uniform(1.0, 16.0, HV))
    dt = torch.exp(uniform(math.log(1e-3), math.log(1e-1), HV))
    d["dt_bias"] = dt + torch.log(-torch.expm1(-dt))
    d["state"] = torch.zeros(B, HV, HEAD, HEAD, device=DEV) if case.get("fresh") else normal(B, HV, HEAD, HEAD, std=0.1)
    return d


def prepare(case, seed):
    d = _inputs(case, seed)
    s = dict(d, case=case)
    B, bf = case["batch"], torch.bfloat16
    if case["op"] == "rot":
        n, G = case["tokens"], case["groups"]
        q = 4 * G * ROT_HEAD
        s["q"] = d["qk"][..., :q].view(B, n, 4 * G, ROT_HEAD)
        s["k"] = d["qk"][..., q:].view(B, n, G, ROT_HEAD)
        s["positions"] = (d["start"][:, None] + torch.arange(n, device=DEV)).to(torch.int32)
        s["q_out"] = torch.zeros(B, n, 4 * G, ROT_HEAD, dtype=bf, device=DEV)
        s["k_out"] = torch.zeros(B, n, G, ROT_HEAD, dtype=bf, device=DEV)
        if own:
            import bounded_memory_attention_b200 as rma
            s["rma"] = rma
            s["handle"] = rma.State(rma.Config(batch=B, n_layers=1, n_groups=G, ring_slots=64, bank_slots=64, pend_slots=64))
            s["handle"].counters[0, :, :, 0] = d["start"][:, None]
        return s
    n = case.get("tokens", 1)
    if case["op"] == "conv":
        s["out"] = torch.zeros(B, n, _channels(case), dtype=bf, device=DEV)
    else:
        s["out"] = torch.zeros(B, n, case["v_heads"], HEAD, dtype=bf, device=DEV)
    if own:
        import bounded_memory_attention_b200 as rma
        s["rma"] = rma
        h = rma.GdnState(rma.GdnConfig(batch=B, n_layers=1, n_k_heads=case["k_heads"], n_v_heads=case["v_heads"],
                                       l2_eps=L2_EPS, scale=HEAD ** -0.5))
        view = h.conv if case["op"] == "conv" else h.delta
        view[0].copy_(d["state"])
        s["handle"], s["state"] = h, view[0]
        if case["op"] == "prompt":
            s["ws"] = h.workspace(n)
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_rot(s):
    case = s["case"]
    half = case["rotary"] // 2
    # angles of far positions need 64 bits
    angle = s["positions"].double()[..., None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]

    def one(x, w):
        x = x.float()
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        r = x[..., :2 * half]
        if case["interleaved"]:
            u, v = r[..., 0::2], r[..., 1::2]
            r = torch.stack((u * cos - v * sin, v * cos + u * sin), -1).flatten(-2)
        else:
            u, v = r[..., :half], r[..., half:]
            r = torch.cat((u * cos - v * sin, v * cos + u * sin), -1)
        return torch.cat((r, x[..., 2 * half:]), -1).to(torch.bfloat16)

    return {"q": one(s["q"], s["w_q"]), "k": one(s["k"], s["w_k"])}


def _plain_conv(s):
    x, state, n = s["x"], s["state"], s["x"].shape[1]
    row = torch.cat((state, x), 1).float()
    y = sum(row[:, j:j + n] * s["w"][:, j] for j in range(WIDTH))
    if s["bias"] is not None:
        y = y + s["bias"]
    y = (y / (1 + torch.exp(-y))).to(torch.bfloat16)
    lens = s.get("lens")
    if lens is None:
        s["out"].copy_(y)
        state.copy_(torch.cat((state, x), 1)[:, n:])
    else:
        inside = torch.arange(n, device=DEV)[None, :, None] < lens[:, None, None]
        s["out"].copy_(torch.where(inside, y, s["out"]))
        take = lens.long()[:, None] + torch.arange(WIDTH - 1, device=DEV)
        state.copy_(torch.cat((state, x), 1)[torch.arange(len(lens), device=DEV)[:, None], take])
    return {"out": s["out"], "state": state}


def _plain_parts(s):
    """q, k [B, HV, n, 128] normalised, v, beta, log decay g [B, HV, n], all in 32 bits."""
    case = s["case"]
    HK, HV = case["k_heads"], case["v_heads"]
    x = s["qkv"].float()
    B, n = x.shape[:2]
    q, k, v = x.split((HK * HEAD, HK * HEAD, HV * HEAD), -1)

    def unit(t):
        t = t.reshape(B, n, HK, HEAD)
        return (t / torch.sqrt((t * t).sum(-1, keepdim=True) + L2_EPS)).repeat_interleave(HV // HK, 2).transpose(1, 2)

    z = s["a"].float() + s["dt_bias"]
    soft = z.clamp(min=0) + torch.log1p(torch.exp(-z.abs()))
    g = (-torch.exp(s["a_log"]) * soft).transpose(1, 2)
    beta = (1 / (1 + torch.exp(-s["b"].float()))).transpose(1, 2)
    return unit(q) * HEAD ** -0.5, unit(k), v.reshape(B, n, HV, HEAD).transpose(1, 2), beta, g


def _plain_step(s):
    q, k, v, beta, g = (t[:, :, 0] for t in _plain_parts(s))
    S = s["state"] * torch.exp(g)[..., None, None]
    u = beta[..., None] * (v - (S * k[..., None]).sum(-2))
    S = S + k[..., None] * u[..., None, :]
    s["state"].copy_(S)
    s["out"][:, 0] = (S * q[..., None]).sum(-2)
    return {"out": s["out"], "state": s["state"]}


def _plain_prompt(s):
    q, k, v, beta, g = _plain_parts(s)
    B, H, n = g.shape
    lens = s.get("lens")
    if lens is not None:
        inside = torch.arange(n, device=DEV)[None, None] < lens[:, None, None]
        q, k, v = (torch.where(inside[..., None], t, 0.0) for t in (q, k, v))
        beta, g = torch.where(inside, beta, 0.0), torch.where(inside, g, 0.0)
    N = -(-n // CHUNK)
    fill = N * CHUNK - n

    def cut(t):
        return torch.nn.functional.pad(t, (0, 0, 0, fill) if t.dim() == 4 else (0, fill)).unflatten(2, (N, CHUNK))

    q, k, v, beta, g = (cut(t) for t in (q, k, v, beta, g))
    # decays within a chunk are differences of sums: in 64 bits, where a strong decay hides a weak one otherwise
    G = torch.cumsum(g.double(), -1)
    between = torch.exp((G[..., :, None] - G[..., None, :]).clamp(max=0)).float()
    kk = k @ k.transpose(-1, -2)
    A = torch.tril(beta[..., None] * between * kk, -1)
    # (1 + A)^-1 from the inverses of its diagonal blocks, doubling their size
    T = torch.eye(CHUNK, device=DEV).expand_as(A).clone()
    size = 1
    while size < CHUNK:
        m = torch.arange(CHUNK // (2 * size), device=DEV)
        Ab, Tb = (t.view(B, H, N, len(m), 2 * size, len(m), 2 * size) for t in (A, T))
        D = Tb[:, :, :, m, :, m]
        D[..., size:, :size] = -D[..., size:, size:] @ (Ab[:, :, :, m, :, m][..., size:, :size] @ D[..., :size, :size])
        Tb[:, :, :, m, :, m] = D
        size *= 2
    T = T * beta[..., None, :]
    P = torch.tril(between * (q @ k.transpose(-1, -2)))
    since, until = torch.exp(G).float()[..., None], torch.exp(G[..., -1:] - G).float()[..., None]
    q, kin, kout = q * since, k * since, (k * until).transpose(-1, -2)
    S, o = s["state"].clone(), torch.empty_like(v)
    for c in range(N):  # each chunk starts from the state that the one before leaves
        U = T[:, :, c] @ (v[:, :, c] - kin[:, :, c] @ S)
        o[:, :, c] = q[:, :, c] @ S + P[:, :, c] @ U
        S = S * since[:, :, c, -1:] + kout[:, :, c] @ U
    s["state"].copy_(S)
    o = o.flatten(2, 3)[:, :, :n].transpose(1, 2).to(torch.bfloat16)
    if lens is not None:
        o = torch.where(inside[:, 0, :, None, None], o, s["out"])
    s["out"].copy_(o)
    return {"out": s["out"], "state": s["state"]}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"rot": _plain_rot, "conv": _plain_conv, "step": _plain_step, "prompt": _plain_prompt}[op](s)
    rma = s["rma"]
    if op == "rot":
        rma.qk_norm_rope(s["handle"], 0, s["q"], s["k"], s["w_q"], s["w_k"], s["inv_freq"], s["q_out"], s["k_out"],
                         positions=None if s["case"]["counters"] else s["positions"], eps=EPS,
                         interleaved=s["case"]["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "conv":
        rma.gdn_conv(s["handle"], 0, s["x"], s["w"], s["out"], bias=s["bias"], lens=s.get("lens"))
    elif op == "step":
        rma.gdn_decode_step(s["handle"], 0, s["qkv"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["out"])
    else:
        rma.gdn_prefill(s["handle"], 0, s["qkv"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["out"], s["ws"],
                        lens=s.get("lens"))
    return {"out": s["out"], "state": s["state"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B, n = case["batch"], case.get("tokens", 1)
    if case["op"] == "rot":
        values = B * n * 5 * case["groups"] * ROT_HEAD
        return {"bytes": 4 * values + 4 * B * n, "flops": 8 * values}
    C, HK, HV = _channels(case), case["k_heads"], case["v_heads"]
    # the mean of the ragged lengths
    tokens = B * n if not case.get("ragged") else n + (B - 1) * (n // 3 + n) / 2
    if case["op"] == "conv":
        return {"bytes": 4 * tokens * C + 2 * 2 * 3 * B * C + 16 * C, "flops": 2 * WIDTH * tokens * C}
    row = 2 * (C + HV * HEAD + 2 * HV)
    state = B * HV * HEAD * HEAD
    if case["op"] == "step":
        return {"bytes": B * row + 8 * state, "flops": 7 * state}
    # the recurrence needs S k, k u and S q of each token
    return {"bytes": tokens * row + (4 if case["fresh"] else 8) * state, "flops": 7 * tokens * HV * HEAD * HEAD}


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "rot":
        return _exact_rot(case, d)
    if case["op"] == "conv":
        return _exact_conv(case, d)
    return _exact_delta(case, d)


def _exact_rot(case, d):
    B, n, G, half = case["batch"], case["tokens"], case["groups"], case["rotary"] // 2
    heads = d["qk"].double().view(B, n, 5 * G, ROT_HEAD)
    power = heads.pow(2).sum(-1) / ROT_HEAD + EPS
    weight = torch.cat((d["w_q"].expand(4 * G, -1), d["w_k"].expand(G, -1))).double()
    y = heads * power.pow(-0.5)[..., None] * weight
    place = d["start"].double()[:, None] + torch.arange(n, device=DEV, dtype=torch.float64)
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV), place[..., None] * d["inv_freq"])[:, :, None]
    at = torch.arange(half, device=DEV)
    first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
    z = torch.complex(y[..., first], y[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return {"q": y[:, :, :4 * G].contiguous(), "k": y[:, :, 4 * G:].contiguous()}


def _exact_conv(case, d):
    B, n = case["batch"], case["tokens"]
    lens = d["lens"].tolist() if "lens" in d else [n] * B
    out, states = [], []
    for b in range(B):
        seen = torch.cat((d["state"][b], d["x"][b, :lens[b]])).double()
        y = (seen.unfold(0, WIDTH, 1) * d["w"].double()).sum(-1)
        if d["bias"] is not None:
            y = y + d["bias"].double()
        out.append(torch.nn.functional.pad(y * torch.sigmoid(y), (0, 0, 0, n - lens[b])))
        states.append(seen[lens[b]:])
    return {"out": torch.stack(out), "state": torch.stack(states)}


def _exact_delta(case, d):
    HK, HV = case["k_heads"], case["v_heads"]
    x = d["qkv"].double()
    B, n = x.shape[:2]
    x = x.view(B, n, 2 * HK + HV, HEAD)
    of = torch.arange(HV, device=DEV) // (HV // HK)  # the key head of each value head
    norm = (x[:, :, :2 * HK].pow(2).sum(-1, keepdim=True) + L2_EPS).rsqrt()
    q, k, v = (x[:, :, :HK] * norm[:, :, :HK])[:, :, of] / math.sqrt(HEAD), (x[:, :, HK:2 * HK] * norm[:, :, HK:])[:, :, of], x[:, :, 2 * HK:]
    decay = torch.exp(-torch.exp(d["a_log"].double()) * torch.nn.functional.softplus(d["a"].double() + d["dt_bias"].double(), threshold=1e9))
    beta = torch.sigmoid(d["b"].double())
    lens = d["lens"] if "lens" in d else torch.full((B,), n, device=DEV)
    live = (torch.arange(n, device=DEV)[None] < lens[:, None]).double()[..., None]
    decay, beta = torch.where(live > 0, decay, 1.0), beta * live
    S = d["state"].double()
    out = torch.zeros(B, n, HV, HEAD, dtype=torch.float64, device=DEV)
    for t in range(n):
        S = S * decay[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - torch.einsum("bhkv,bhk->bhv", S, k[:, t]))
        S = torch.addcmul(S, k[:, t, :, :, None], u[:, :, None, :])
        out[:, t] = torch.einsum("bhkv,bhk->bhv", S, q[:, t])
    return {"out": out * live[..., None], "state": S}
