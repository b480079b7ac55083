"""Cases and plain forms of the operators around a paged cache of keys and values.

A step with several new tokens per sequence (one token, or one and its drafts) of layers
that keep a key and a value per head runs them in this order, between the block tables of
the step and the next step's:

* ``rope``: rotary positions of whole tokens' heads: pairs of neighbours or of halves, a part
  of the head, tables scaled for long contexts, and the rotation back (its gradient);
* ``append``: keys (rotated) and values of the packed new tokens into 256-position blocks, the
  queries' rotation in the same pass; the cache holds the layer's type or 8-bit floats;
* ``attn``: softmax attention of the new tokens of each sequence over its blocks, several query
  heads per key head, with the logarithm of the softmax's sum;
* ``verify``: which drafted tokens stand against the target's probabilities, and the token
  that follows them, from given random numbers.

``run`` computes them with elementary torch operations while ``own`` is false, and through
the package's public calls while it is true.
"""
import math

import numpy as np
import torch

own = False
DEV = "cuda"
BLOCK = 256          # token positions of a block
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BASE = 10000.0
FACTOR, ORIG = 16.0, 4096    # scaled tables: ORIG trained positions, FACTOR times as many


# ------------------------------------------------------------------ cases

def _rope(name, n, heads, dim, rot, tail, half, scaled, inverse, fused, dtype, max_pos):
    return {"name": name, "kind": "rope", "n": n, "heads": heads, "dim": dim, "rot": rot,
            "tail": tail, "half": half, "scaled": scaled, "inverse": inverse, "fused": fused,
            "dtype": dtype, "max_pos": max_pos}


def _append(name, batch, new, ctx, heads, kv_heads, dim, rot, half, scaled, dtype, kv):
    return {"name": name, "kind": "append", "batch": batch, "new": new, "ctx": ctx, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "half": half, "scaled": scaled,
            "dtype": dtype, "kv": kv}


def _attn(name, batch, new, ctx, heads, kv_heads, dim, window, ragged, dtype, kv):
    return {"name": name, "kind": "attn", "batch": batch, "new": new, "ctx": ctx, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "window": window, "ragged": ragged, "dtype": dtype,
            "kv": kv}


def _verify(name, batch, drafts, vocab, sampled, ragged, dtype):
    return {"name": name, "kind": "verify", "batch": batch, "drafts": drafts, "vocab": vocab,
            "sampled": sampled, "ragged": ragged, "dtype": dtype}


def listed():
    return [
        # the queries of one new token for each of 8 sequences
        _rope("rope_decode_n8", 8, 64, 128, 128, False, True, "none", False, False, "bf16", 8192),
        # a 4096-token chunk, heads of 512 dims with a 64-dim tail, from a projection's output
        _rope("rope_chunk_n4096", 4096, 64, 512, 64, True, False, "yarn", False, True, "bf16", 65536),
        # gradients rotated back, fp32, an odd number of heads, part of the head
        _rope("rope_back_f32_n333", 333, 5, 96, 32, False, True, "ntk", True, False, "f32", 8192),
        # one new token for each of 8 sequences: keys, values and the queries of 64 heads
        _append("append_decode_b8", 8, 1, 2048, 64, 8, 128, 128, True, "none", "bf16", "bf16"),
        # a 4096-token chunk of each of 2 prompts into an 8-bit cache
        _append("append_chunk_e4m3", 2, 4096, 3000, 64, 8, 128, 64, False, "yarn", "bf16", "e4m3"),
        # a single sequence of 4096 tokens: latency counts
        _attn("attn_b1_ctx4096", 1, 1, 4096, 64, 8, 128, 0, False, "bf16", "bf16"),
        # 8 sequences of 131,072 tokens
        _attn("attn_b8_ctx131072", 8, 1, 131072, 64, 8, 128, 0, False, "bf16", "bf16"),
        # a ragged batch of 64 over an 8-bit cache
        _attn("attn_ragged_b64_e4m3", 64, 1, 32768, 64, 8, 128, 0, True, "bf16", "e4m3"),
        # a token and 4 drafts for each of 16 ragged sequences
        _attn("attn_drafts_b16_t5", 16, 5, 16384, 64, 8, 128, 0, True, "bf16", "bf16"),
        # fp32 layer of small heads, a sliding window
        _attn("attn_window_f32_b3", 3, 2, 5001, 10, 2, 80, 1024, True, "f32", "f32"),
        # 3 greedy drafts for each of 8 sequences
        _verify("verify_greedy_b8", 8, 3, 50021, False, False, "f32"),
        # up to 7 sampled drafts for each of 256 sequences
        _verify("verify_sampled_b256", 256, 7, 131072, True, True, "f32"),
    ]


def _span(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attn", "attn", "attn", "verify"])
    scaled = rng.choice(["none", "linear", "ntk", "yarn"])
    if kind == "rope":
        f32 = rng.random() < 0.3
        dim = rng.choice([64, 80, 96, 128, 192, 256, 512])
        rot = rng.choice([dim, 64, 32, dim // 4 * 2])
        heads = rng.choice([1, 2, 5, 8, 24, 64])
        n = _span(rng, 1, max(2, 4096 * 64 * 512 // (heads * dim * (2 if f32 else 1)) // 4))
        c = _rope("", n, heads, dim, rot, rng.random() < 0.5, rng.random() < 0.5, scaled,
                  rng.random() < 0.3, rng.random() < 0.5, "f32" if f32 else "bf16", 65536)
    elif kind == "append":
        f32 = rng.random() < 0.25
        dim = rng.choice([64, 80, 96, 128, 256])
        kv_heads = rng.choice([1, 2, 4, 8])
        batch, e4m3 = _span(rng, 1, 64), rng.random() < 0.5
        new = rng.choice([1, 1, 2, 5, _span(rng, 2, max(3, 8192 // batch))])
        dtype = "f32" if f32 else "bf16"
        c = _append("", batch, new, _span(rng, 1, 3000), kv_heads * rng.choice([1, 3, 8]), kv_heads,
                    dim, rng.choice([dim, 64, 32]), rng.random() < 0.5, scaled, dtype,
                    "e4m3" if e4m3 else dtype)
    elif kind == "attn":
        f32 = rng.random() < 0.2
        kv_heads, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 16])
        batch = _span(rng, 1, 64)
        new = rng.choice([1, 1, 1, 2, 3, 5, 8])
        ragged, window = rng.random() < 0.6, rng.choice([0, 0, 0, 128, 1000])
        if f32:
            c = _attn("", min(batch, 8), new, _span(rng, 1, 8000), kv_heads * group, kv_heads,
                      rng.choice([64, 80, 128]), window, ragged, "f32", "f32")
        else:
            dim = rng.choice([64, 96, 128, 128, 128, 256])
            most = 8 * 131072 * 8 * 128 // (batch * kv_heads * dim * max(1, new * group // 8))
            c = _attn("", batch, new, _span(rng, 1, max(2, min(131072, most))), kv_heads * group,
                      kv_heads, dim, window, ragged, "bf16", rng.choice(["bf16", "bf16", "e4m3"]))
    else:
        vocab = rng.choice([32000, 50021, 100277, 131072, _span(rng, 100, 131072)])
        c = _verify("", _span(rng, 1, 128), rng.choice([1, 2, 3, 4, 7, 10]), vocab,
                    rng.random() < 0.6, rng.random() < 0.5, rng.choice(["f32", "f32", "bf16"]))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed, *keys):
    g = torch.Generator(device=DEV)
    g.manual_seed((seed * 1000003 + sum((i + 1) * 7919 * k for i, k in enumerate(keys))) & (2**62 - 1))
    return g


def _normal(shape, dtype, g, std=1.0):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
    return x.mul_(std) if std != 1.0 else x


def _i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


def _theta(rot, scaled):
    """Angle per position of each pair (fp64), and the factor of cosines and sines.

    none: theta_i = base^(-2 i / rot). linear: theta_i / factor. ntk: the base times
    factor^(rot / (rot - 2)). yarn: theta_i (g_i + (1 - g_i) / factor), g_i falling from 1 to 0
    between the pairs that turn 32 times and once over the trained positions; cosines and
    sines times 0.1 ln(factor) + 1."""
    i = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    base = BASE * FACTOR ** (rot / (rot - 2)) if scaled == "ntk" else BASE
    theta, mag = base ** (-2.0 * i / rot), 1.0
    if scaled == "linear":
        theta = theta / FACTOR
    elif scaled == "yarn":
        at = lambda turns: rot * math.log(ORIG / (turns * 2 * math.pi)) / (2 * math.log(BASE))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot // 2 - 1)
        g = 1 - ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        theta, mag = theta * (g + (1 - g) / FACTOR), 0.1 * math.log(FACTOR) + 1.0
    return theta, mag


_kept = {}


def _tables(rot, scaled, max_pos):
    """cos and sin [max_pos][rot / 2] in fp32, rounded once."""
    key = (rot, scaled, max_pos)
    if key not in _kept:
        theta, mag = _theta(rot, scaled)
        a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * theta
        _kept[key] = (a.cos().mul(mag).float(), a.sin().mul(mag).float())
    return _kept[key]


def _own_rope(rot, scaled, max_pos, rot_at, half):
    from compressed_kv_sparse_gb300 import lib
    return lib.Rope(n_rot=rot, max_pos=max_pos, base=BASE, rot_at=rot_at, half=half, scaling=scaled,
                    factor=FACTOR, orig_len=ORIG, device=DEV)


def prepare(case, seed):
    return {"rope": _prepare_rope, "append": _prepare_append, "attn": _prepare_attn,
            "verify": _prepare_verify}[case["kind"]](case, seed)


def _prepare_rope(c, seed):
    dt, n, H, D = TYPES[c["dtype"]], c["n"], c["heads"], c["dim"]
    g = _gen(seed, n, H, D)
    s = {"case": c, "rot_at": D - c["rot"] if c["tail"] else 0}
    # fused: the heads are the front of a wider row of the projection's output
    x = _normal((n, H * D + (2 * D if c["fused"] else 0)), dt, g)
    s["x"] = x[:, :H * D].view(n, H, D)
    s["pos"] = torch.randint(0, c["max_pos"], (n,), generator=g, device=DEV, dtype=torch.int32)
    s["y"] = torch.empty((n, H, D), dtype=dt, device=DEV)
    if own:
        s["rope"] = _own_rope(c["rot"], c["scaled"], c["max_pos"], s["rot_at"], c["half"])
    else:
        s["tables"] = _tables(c["rot"], c["scaled"], c["max_pos"])
    return s


def _lengths(c, seed):
    """Contexts before the step and new tokens of each sequence (the case's, in the seed's order)."""
    rng = np.random.default_rng([c["batch"], c["ctx"], c["new"]])
    B, ctx, new = c["batch"], c["ctx"], c["new"]
    if c["kind"] == "append":
        old = rng.integers(0, ctx + 1, B)
        cnt = np.full(B, new)
    elif c["ragged"]:
        total = np.exp(rng.uniform(0, math.log(ctx + 1), B)).astype(np.int64)
        total[0] = ctx
        total = np.clip(total, 1, ctx)
        cnt = np.minimum(rng.integers(1, new + 1, B), total)
        cnt[0] = min(new, ctx)
        old = total - cnt
    else:
        cnt = np.full(B, min(new, ctx))
        old = ctx - cnt
    order = np.random.default_rng([seed & 0xFFFFFFFF, B]).permutation(B)
    return old[order], cnt[order]


def _step(c, seed, g):
    """Positions, packed tokens and the block table of a step."""
    old, cnt = _lengths(c, seed)
    B, M = c["batch"], -(-(int((old + cnt).max())) // BLOCK)
    cu = np.concatenate([[0], np.cumsum(cnt)])
    seq = np.repeat(np.arange(B), cnt)
    t = np.arange(cu[-1]) - cu[seq]
    held = -(-(old + cnt) // BLOCK)
    n_blocks = int(held.sum()) + 3
    perm = torch.randperm(n_blocks, generator=g, device=DEV).cpu().numpy().astype(np.int32)
    table = np.full((B, M), -1, np.int32)
    table[np.arange(M)[None] < held[:, None]] = perm[:int(held.sum())]
    return {"case": c, "old": _i32(old), "cnt": _i32(cnt), "cu": _i32(cu), "seq": _i32(seq), "t": _i32(t),
            "pos": _i32(old[seq] + t), "table": _i32(table), "n_blocks": n_blocks, "M": M,
            "n": int(cu[-1])}


def _prepare_append(c, seed):
    dt, H, K, D = TYPES[c["dtype"]], c["heads"], c["kv_heads"], c["dim"]
    g = _gen(seed, c["batch"], H, K, D)
    s = _step(c, seed, g)
    # queries, keys and values lie in one projection's output, token by token
    qkv = _normal((s["n"], (H + 2 * K) * D), dt, g)
    s["q"] = qkv[:, :H * D].view(s["n"], H, D)
    s["k"] = qkv[:, H * D:(H + K) * D].view(s["n"], K, D)
    s["v"] = qkv[:, (H + K) * D:].view(s["n"], K, D)
    s["q_out"] = torch.empty((s["n"], H, D), dtype=dt, device=DEV)
    s["k_scale"] = torch.rand(K, generator=g, device=DEV) * 0.02 + 0.008
    s["v_scale"] = torch.rand(K, generator=g, device=DEV) * 0.02 + 0.008
    s["max_pos"] = 16384
    shape, kt = (s["n_blocks"], K, BLOCK, D), TYPES[c["kv"]]
    if own:
        from compressed_kv_sparse_gb300 import lib
        e4m3 = c["kv"] == "e4m3"
        s["cache"] = lib.KvCache(
            head_dim=D, n_kv_heads=K, batch=c["batch"], block_table=s["table"], n_blocks=s["n_blocks"],
            dtype=c["dtype"], kv_dtype=c["kv"], k_scale=s["k_scale"] if e4m3 else None,
            v_scale=s["v_scale"] if e4m3 else None,
            rope=_own_rope(c["rot"], c["scaled"], s["max_pos"], 0, c["half"]), device=DEV)
        s["pool_k"], s["pool_v"] = s["cache"].k, s["cache"].v
    else:
        s["tables"] = _tables(c["rot"], c["scaled"], s["max_pos"])
        s["pool_k"] = torch.zeros(shape, device=DEV).to(kt)
        s["pool_v"] = torch.zeros(shape, device=DEV).to(kt)
    return s


def _pool(shape, kt, scale, g):
    if kt != torch.float8_e4m3fn:
        return _normal(shape, kt, g)
    x = torch.empty(shape, dtype=kt, device=DEV)   # (a head at a time: the values are wider)
    inv = 1.0 / scale
    for h in range(shape[1]):
        x[:, h] = (torch.randn((shape[0],) + shape[2:], generator=g, device=DEV) * inv[h]).clamp_(-448, 448).to(kt)
    return x


def _attn_inputs(c, seed):
    dt, kt, H, K, D = TYPES[c["dtype"]], TYPES[c["kv"]], c["heads"], c["kv_heads"], c["dim"]
    g = _gen(seed, c["batch"], H, K, D)
    s = _step(c, seed, g)
    s["q"] = _normal((s["n"], H, D), dt, g, std=1.5)
    s["k_scale"] = torch.rand(K, generator=g, device=DEV) * 0.02 + 0.008
    s["v_scale"] = torch.rand(K, generator=g, device=DEV) * 0.02 + 0.008
    s["pool_k"] = _pool((s["n_blocks"], K, BLOCK, D), kt, s["k_scale"], g)
    s["pool_v"] = _pool((s["n_blocks"], K, BLOCK, D), kt, s["v_scale"], g)
    s["scale"] = 1.0 / math.sqrt(D)
    s["out"] = torch.empty((s["n"], H, D), dtype=dt, device=DEV)
    s["lse"] = torch.empty((s["n"], H), dtype=torch.float32, device=DEV)
    return s


def _prepare_attn(c, seed):
    s = _attn_inputs(c, seed)
    if own:
        from compressed_kv_sparse_gb300 import lib
        e4m3 = c["kv"] == "e4m3"
        s["cache"] = lib.KvCache(
            head_dim=c["dim"], n_kv_heads=c["kv_heads"], batch=c["batch"], block_table=s["table"],
            n_blocks=s["n_blocks"], dtype=c["dtype"], kv_dtype=c["kv"], k_scale=s["k_scale"] if e4m3 else None,
            v_scale=s["v_scale"] if e4m3 else None, k=s["pool_k"], v=s["pool_v"], device=DEV)
        s["cache"].set_seq_pos(s["old"])
        s["ws"] = lib.workspace(s["cache"].attn_workspace_bytes(c["heads"], c["new"]), DEV)
    return s


def _verify_inputs(c, seed):
    dt, B, N, V = TYPES[c["dtype"]], c["batch"], c["drafts"], c["vocab"]
    g = _gen(seed, B, N, V)
    rng = np.random.default_rng([B, N, V])
    cnt = rng.integers(1, N + 2, B) if c["ragged"] else np.full(B, N + 1)   # the last token and its drafts
    cnt = cnt[np.random.default_rng([seed & 0xFFFFFFFF, B]).permutation(B)]
    cu = np.concatenate([[0], np.cumsum(cnt)])
    seq = np.repeat(np.arange(B), cnt)
    s = {"case": c, "cnt": _i32(cnt), "cu": _i32(cu), "n": int(cu[-1])}
    logits = torch.randn((s["n"], V), generator=g, device=DEV) * 2.5
    s["target"] = torch.softmax(logits, -1).to(dt)
    # row of the target's probabilities after i drafts (a sequence with fewer: its last)
    at = np.minimum(cu[:-1, None] + np.arange(N)[None], cu[1:, None] - 1)
    at = torch.tensor(at.reshape(-1), device=DEV)
    s["draft_probs"] = None
    if c["sampled"]:   # a draft model that is near the target
        noise = torch.randn((B * N, V), generator=g, device=DEV) * 0.4
        dp = torch.softmax(logits[at].add_(noise), -1)
        gum = torch.rand((B * N, V), generator=g, device=DEV).clamp_(1e-12, 1 - 1e-7).log_().neg_()
        s["drafts"] = (dp / gum).argmax(-1).int().view(B, N)
        s["draft_probs"] = dp.to(dt).view(B, N, V)
        del noise, gum, dp
    else:              # the likeliest token by the draft model
        s["drafts"] = logits[at].argmax(-1).int().view(B, N)
        wrong = torch.rand((B, N), generator=g, device=DEV) < 0.3
        s["drafts"] = torch.where(wrong, (s["drafts"] + 17) % V, s["drafts"])
    s["u_accept"] = torch.rand((B, N), generator=g, device=DEV)
    s["u_sample"] = torch.rand((B,), generator=g, device=DEV)
    s["old"] = torch.randint(0, 100000, (B,), generator=g, device=DEV, dtype=torch.int32)
    s["seq"] = torch.tensor(seq, device=DEV)
    return s


def _prepare_verify(c, seed):
    s = _verify_inputs(c, seed)
    B, N = c["batch"], c["drafts"]
    s["tokens"] = torch.empty((B, N + 1), dtype=torch.int32, device=DEV)
    s["n_out"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    s["ctx_out"] = torch.empty((B,), dtype=torch.int32, device=DEV)
    return s


# ----------------------------------------------------------------- one pass

def run(state):
    return {"rope": _run_rope, "append": _run_append, "attn": _run_attn,
            "verify": _run_verify}[state["case"]["kind"]](state)


def _rotate(x, pos, cos, sin, rot_at, rot, half, inverse=False):
    """fp32 heads [n][H][D], their dims rot_at .. rot_at + rot - 1 rotated at pos."""
    c, s = cos[pos.long()][:, None], sin[pos.long()][:, None]
    if inverse:
        s = -s
    r = x[..., rot_at:rot_at + rot]
    a, b = (r[..., :rot // 2], r[..., rot // 2:]) if half else (r[..., 0::2], r[..., 1::2])
    y0, y1 = a * c - b * s, a * s + b * c
    out = x.clone()
    out[..., rot_at:rot_at + rot] = torch.cat([y0, y1], -1) if half else torch.stack([y0, y1], -1).flatten(-2)
    return out


def _run_rope(s):
    c = s["case"]
    if own:
        from compressed_kv_sparse_gb300 import lib
        lib.ds4a_rope(s["rope"], s["pos"], s["x"], s["y"], inverse=c["inverse"])
        return s["y"]
    cos, sin = s["tables"]
    y = _rotate(s["x"].float(), s["pos"], cos, sin, s["rot_at"], c["rot"], c["half"], c["inverse"])
    return y.to(TYPES[c["dtype"]])


def _run_append(s):
    c = s["case"]
    if own:
        from compressed_kv_sparse_gb300 import lib
        lib.ds4a_kv_append(s["cache"], s["seq"], s["pos"], s["k"], s["v"], q=s["q"], q_out=s["q_out"])
        return {"k": s["pool_k"], "v": s["pool_v"], "q": s["q_out"]}
    cos, sin = s["tables"]
    dt, kt = TYPES[c["dtype"]], TYPES[c["kv"]]
    q = _rotate(s["q"].float(), s["pos"], cos, sin, 0, c["rot"], c["half"]).to(dt)
    k = _rotate(s["k"].float(), s["pos"], cos, sin, 0, c["rot"], c["half"])
    v = s["v"].float()
    if c["kv"] == "e4m3":   # times the scale's reciprocal, held to the largest value
        k = (k * (1.0 / s["k_scale"])[None, :, None]).clamp(-448, 448)
        v = (v * (1.0 / s["v_scale"])[None, :, None]).clamp(-448, 448)
    blk = s["table"][s["seq"].long(), s["pos"].long() // BLOCK].long()
    r = s["pos"].long() % BLOCK
    bits = torch.uint8 if c["kv"] == "e4m3" else kt
    s["pool_k"].view(bits)[blk, :, r] = k.to(kt).view(bits)
    s["pool_v"].view(bits)[blk, :, r] = v.to(kt).view(bits)
    return {"k": s["pool_k"], "v": s["pool_v"], "q": q}


def _run_attn(s):
    c = s["case"]
    if own:
        from compressed_kv_sparse_gb300 import lib
        lib.ds4a_paged_attn_decode(s["cache"], s["q"], s["out"], s["ws"], max_new=c["new"], cu_len=s["cu"],
                                   lse=s["lse"], window=c["window"], scale=s["scale"])
        return {"out": s["out"], "lse": s["lse"]}
    B, T, H, K, D, M = c["batch"], c["new"], c["heads"], c["kv_heads"], c["dim"], s["M"]
    G, L = H // K, s["M"] * BLOCK
    table = s["table"].clamp(min=0).long()
    at = lambda pool: pool[table.view(-1)].view(B, M, K, BLOCK, D).transpose(1, 2).reshape(B, K, L, D).float()  # noqa: E731
    bits = torch.uint8 if c["kv"] == "e4m3" else None
    if bits is None:
        k, v = at(s["pool_k"]), at(s["pool_v"])
    else:   # (the bytes are gathered, then read as values)
        get = lambda pool: pool.view(bits)[table.view(-1)].view(TYPES["e4m3"]).view(B, M, K, BLOCK, D).transpose(1, 2).float().reshape(B, K, L, D)  # noqa: E731
        k = get(s["pool_k"]) * s["k_scale"][None, :, None, None]
        v = get(s["pool_v"]) * s["v_scale"][None, :, None, None]
    seq, t = s["seq"].long(), s["t"].long()
    q = torch.zeros((B, T, H, D), device=DEV)
    q[seq, t] = s["q"].float()
    q = q.view(B, T, K, G, D).permute(0, 2, 1, 3, 4).reshape(B, K, T * G, D)
    x = (q @ k.transpose(2, 3)).mul_(s["scale"]).view(B, K, T, G, L)
    p = (s["old"].long()[:, None] + torch.arange(T, device=DEV))[..., None]     # [B][T][1]
    key = torch.arange(L, device=DEV)
    seen = key <= p
    if c["window"]:
        seen = seen & (key > p - c["window"])
    x.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    e = x.sub_(top).exp_()
    sum_ = e.sum(-1, keepdim=True)
    o = (e.view(B, K, T * G, L) @ v).view(B, K, T, G, D) / sum_
    lse = (top + sum_.log())[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H, D)[seq, t]
    lse = lse.permute(0, 2, 1, 3).reshape(B, T, H)[seq, t]
    return {"out": o.to(TYPES[c["dtype"]]), "lse": lse}


def _run_verify(s):
    c = s["case"]
    B, N, V = c["batch"], c["drafts"], c["vocab"]
    if own:
        from compressed_kv_sparse_gb300 import lib
        lib.ds4a_verify_drafts(s["target"], s["drafts"], s["u_accept"], s["u_sample"], s["tokens"], s["n_out"],
                               draft_probs=s["draft_probs"], cu_len=s["cu"], seq_pos=s["old"],
                               ctx_out=s["ctx_out"])
        return {"tokens": s["tokens"], "n_out": s["n_out"], "ctx": s["ctx_out"]}
    # (in 64 bits: the sums decide whole numbers)
    row = torch.arange(B, device=DEV)
    i = torch.arange(N, device=DEV)
    there = i < (s["cnt"] - 1)[:, None]
    first = s["cu"][:-1].long()
    at = (first[:, None] + i).clamp(max=s["n"] - 1)
    x = s["drafts"].long()
    p = s["target"][at, x].double()
    q = torch.ones_like(p) if s["draft_probs"] is None else s["draft_probs"][row[:, None], i, x].double()
    ok = (s["u_accept"].double() * q < p) & there
    acc = ok.long().cumprod(1).sum(1)                       # drafts that stand
    refused = acc < s["cnt"] - 1
    w = s["target"][first + acc].double()                   # the row behind them
    j = acc.clamp(max=N - 1)
    if s["draft_probs"] is None:
        cut = w.scatter(1, x[row, j][:, None], 0.0)
    else:
        cut = (w - s["draft_probs"][row, j].double()).clamp(min=0)
    w = torch.where(refused[:, None], cut, w)
    cum = w.cumsum(1)
    new = (cum <= s["u_sample"].double()[:, None] * cum[:, -1:]).sum(1).clamp(max=V - 1)
    col = torch.arange(N + 1, device=DEV)
    pad = torch.cat([x, torch.zeros((B, 1), dtype=torch.long, device=DEV)], 1)
    tokens = torch.where(col < acc[:, None], pad, torch.where(col == acc[:, None], new[:, None], -1))
    return {"tokens": tokens.int(), "n_out": (acc + 1).int(), "ctx": (s["old"] + acc + 1).int()}


# --------------------------------------------------------------------- work

def work(case):
    c = case
    es = {"bf16": 2, "f32": 4, "e4m3": 1}
    if c["kind"] == "rope":
        rows = c["n"] * c["heads"] * c["dim"]
        return {"bytes": 2 * rows * es[c["dtype"]] + c["n"] * (4 + 4 * c["rot"]),
                "flops": 3 * c["n"] * c["heads"] * c["rot"]}
    if c["kind"] == "append":
        n = c["batch"] * c["new"]
        row, kv = c["dim"] * es[c["dtype"]], c["dim"] * es[c["kv"]]
        return {"bytes": n * (2 * c["heads"] * row + 2 * c["kv_heads"] * (row + kv) + 12 + 4 * c["rot"]),
                "flops": 3 * n * (c["heads"] + c["kv_heads"]) * c["rot"]}
    if c["kind"] == "attn":
        old, cnt = _lengths(c, 0)
        lo = np.maximum(old + 1 - c["window"], 0) if c["window"] else np.zeros_like(old)
        keys = int((old + cnt - lo).sum())                      # read for each key head
        seen = 0
        for t in range(c["new"]):
            n = old + t + 1
            seen += int((np.minimum(n, c["window"]) if c["window"] else n)[cnt > t].sum())
        n = int(cnt.sum())
        return {"bytes": 2 * keys * c["kv_heads"] * c["dim"] * es[c["kv"]]
                + n * c["heads"] * (2 * c["dim"] * es[c["dtype"]] + 4),
                "flops": 4 * seen * c["heads"] * c["dim"]}
    # one row of the target for each sequence, and the draft's where a draft fell (about 4 of 5 of
    # them stand one by one)
    e, d = es[c["dtype"]], (c["drafts"] / 2 if c["ragged"] else c["drafts"])
    fell = 1 - 0.8 ** d if c["sampled"] else 0.0
    return {"bytes": int(c["batch"] * (c["vocab"] * e * (1 + fell) + c["drafts"] * (2 * e + 12) + 16)),
            "flops": 2 * c["batch"] * c["vocab"]}


# -------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn,
            "verify": _exact_verify}[case["kind"]](case, seed)


def _turned(x, pos, rot_at, rot, half, scaled, inverse):
    """Each pair as a complex number times mag * exp(i angle)."""
    theta, mag = _theta(rot, scaled)
    ang = pos.double()[:, None] * theta * (-1.0 if inverse else 1.0)
    z = x.double().clone()
    for i in range(rot // 2):
        a, b = (rot_at + i, rot_at + i + rot // 2) if half else (rot_at + 2 * i, rot_at + 2 * i + 1)
        w = torch.complex(x[..., a].double(), x[..., b].double())
        w = w * torch.polar(torch.full_like(ang[:, i], mag), ang[:, i])[:, None]
        z[..., a], z[..., b] = w.real, w.imag
    return z


def _exact_rope(c, seed):
    s = _prepare_rope(c, seed)
    return _turned(s["x"], s["pos"], s["rot_at"], c["rot"], c["half"], c["scaled"], c["inverse"])


def _exact_append(c, seed):
    s = _prepare_append(c, seed)
    turn = lambda x: _turned(x, s["pos"], 0, c["rot"], c["half"], c["scaled"], False)  # noqa: E731
    shape = (s["n_blocks"] * BLOCK, c["kv_heads"], c["dim"])
    out = {"q": turn(s["q"])}
    slot = s["table"][s["seq"].long(), s["pos"].long() // BLOCK].long() * BLOCK + s["pos"].long() % BLOCK
    for name, x in (("k", turn(s["k"])), ("v", s["v"].double())):
        if c["kv"] == "e4m3":
            # the nearest value m * 2^(e - 3), 8 <= m < 16, e >= -6, below 448
            x = (x / s[name + "_scale"].double()[None, :, None]).clamp(-448, 448)
            e = torch.floor(torch.log2(x.abs().clamp(min=2.0**-20))).clamp(min=-6)
            x = torch.round(x * torch.exp2(3 - e)) * torch.exp2(e - 3)
        pool = torch.zeros(shape, dtype=torch.float64, device=DEV)
        pool[slot] = x
        out[name] = pool.view(s["n_blocks"], BLOCK, c["kv_heads"], c["dim"]).transpose(1, 2).contiguous()
    return out


def _exact_attn(c, seed):
    s = _attn_inputs(c, seed)
    old, cnt = _lengths(c, seed)
    H, K, D, W = c["heads"], c["kv_heads"], c["dim"], c["window"]
    G, cu = H // K, np.concatenate([[0], np.cumsum(cnt)])
    out = torch.zeros((s["n"], H, D), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["n"], H), dtype=torch.float64, device=DEV)
    for b in range(c["batch"]):
        n, m = int(old[b] + cnt[b]), int(cnt[b])
        blocks = s["table"][b, :-(-n // BLOCK)].tolist()
        mask = torch.ones((m, n), dtype=torch.bool, device=DEV).tril(n - m)
        if W:
            mask &= ~torch.ones((m, n), dtype=torch.bool, device=DEV).tril(n - m - W)
        for h in range(K):
            rows = lambda p: torch.cat([p[i, h].double() for i in blocks])[:n]  # noqa: E731
            k, v = rows(s["pool_k"]), rows(s["pool_v"])
            if c["kv"] == "e4m3":
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            q = s["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            x = torch.einsum("tgd,nd->gtn", q, k) * s["scale"]
            x = x.masked_fill(~mask, -math.inf)
            z = torch.logsumexp(x, -1)
            out[cu[b]:cu[b + 1], h * G:(h + 1) * G] = torch.einsum("gtn,nd->tgd", (x - z[..., None]).exp(), v)
            lse[cu[b]:cu[b + 1], h * G:(h + 1) * G] = z.T
    return {"out": out, "lse": lse}


def _exact_verify(c, seed):
    s = _verify_inputs(c, seed)
    B, N, V = c["batch"], c["drafts"], c["vocab"]
    cu, x = s["cu"].tolist(), s["drafts"].tolist()
    tokens, n_out = np.full((B, N + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        p = s["target"][cu[b]:cu[b + 1]].double()
        a, m = 0, cu[b + 1] - cu[b] - 1
        d = torch.tensor(x[b][:m], dtype=torch.long, device=DEV)
        r = torch.arange(m, device=DEV)
        q = torch.ones(m, dtype=torch.float64, device=DEV) if s["draft_probs"] is None else s["draft_probs"][b, r, d].double()
        stands = (s["u_accept"][b, :m].double() < p[r, d] / q).tolist()
        while a < m and stands[a]:
            a += 1
        w = p[a].clone()
        if a < m and s["draft_probs"] is None:
            w[x[b][a]] = 0
        elif a < m:
            w = torch.maximum(w - s["draft_probs"][b, a].double(), torch.zeros_like(w))
        cdf = torch.cumsum(w / w.sum(), 0)
        t = int(torch.searchsorted(cdf, s["u_sample"][b].double().view(1), right=True)[0])
        tokens[b, :a], tokens[b, a], n_out[b] = x[b][:a], min(t, V - 1), a + 1
    return {"tokens": tokens, "n_out": n_out, "ctx": (s["old"].cpu().numpy() + n_out).astype(np.int32)}
