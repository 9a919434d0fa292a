"""The prompt path's operators over the shared KV cache, as timed and compared:

* ``rope``     per-head norms and rotation of a fused QKV projection's queries and keys, the keys and values
               written into the cache (``qkv_rope_append``);
* ``prefill``  causal attention of packed prompts of different lengths over the cache (``attn_prefill``);
* ``prefix``   attention of a batch whose sequences share one long prefix (``attn_prefix``).

``run`` computes each of them with elementary torch operations in 32 bits, or, where ``own`` is true, by the
framework's calls.  Every sequence has 128-wide heads and a bf16 cache [batch][kv heads][capacity][128].
"""
import random

import torch

own = False

D = 128


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one drafting pass of 16 sequences: one new token each, Llama-2-7B heads; rotation alone
        _rope("rope draft b16", batch=16, t=1, ragged=False, h_q=32, h_kv=32, ctx=1024, rot=128, norm=False, pairs=False, q32=True),
        # one verifying pass (5 tokens) of 64 sequences, grouped heads, norms of queries and keys
        _rope("rope verify b64 grouped", batch=64, t=5, ragged=False, h_q=32, h_kv=8, ctx=1024, rot=128, norm=True, pairs=False, q32=False),
        # a packed batch of prompts behind cached turns, interleaved pairs, half of the head rotated
        _rope("rope prompts 12x1400", batch=12, t=1400, ragged=True, h_q=64, h_kv=8, ctx=300, rot=64, norm=True, pairs=True, q32=False),
        # one short prompt: what a lone request waits for
        _prefill("prefill 1x200", batch=1, t=200, ragged=False, h_q=32, h_kv=8, ctx=0),
        # prompts of very different lengths in one batch
        _prefill("prefill 16x700 ragged", batch=16, t=700, ragged=True, h_q=32, h_kv=8, ctx=0),
        # the next piece of long prompts whose earlier pieces are cached
        _prefill("prefill 3x1000 cached", batch=3, t=1000, ragged=True, h_q=32, h_kv=32, ctx=4000),
        # one long prompt
        _prefill("prefill 1x8192", batch=1, t=8192, ragged=False, h_q=32, h_kv=8, ctx=0),
        # a few sequences behind a short common instruction
        _prefix("prefix 4x1 p500", batch=4, t=1, ragged=False, h_q=32, h_kv=8, ctx=200, prefix=500),
        # a drafting pass of 32 sequences behind a common document, no grouping
        _prefix("prefix 32x1 p4096", batch=32, t=1, ragged=False, h_q=32, h_kv=32, ctx=700, prefix=4096),
        # a verifying pass of 64 sequences behind a long common document
        _prefix("prefix 64x5 p16384 grouped", batch=64, t=5, ragged=False, h_q=32, h_kv=8, ctx=500, prefix=16384),
        # questions of different lengths behind a common document, read in one call
        _prefix("prefix 24x90 p3000 ragged", batch=24, t=90, ragged=True, h_q=64, h_kv=8, ctx=0, prefix=3000),
    ]


def _rope(name, **k):
    return {"name": name, "op": "rope", "spread": 1, **k}


def _prefill(name, **k):
    return {"name": name, "op": "prefill", "spread": 1, **k}


def _prefix(name, **k):
    return {"name": name, "op": "prefix", "spread": 1, **k}


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


_HEADS = [(32, 32), (32, 8), (64, 8), (8, 8), (14, 2), (12, 4), (16, 1), (5, 5)]


def draw(rng):
    op = rng.choice(["rope", "prefill", "prefill", "prefix", "prefix"])
    h_q, h_kv = rng.choice(_HEADS)
    c = {"op": op, "h_q": h_q, "h_kv": h_kv, "spread": rng.randrange(1 << 20), "ragged": rng.random() < 0.6}
    if op == "rope":
        c["batch"] = _log(rng, 1, 96)
        c["t"] = _log(rng, 1, max(1, min(4096, 16000 // c["batch"])))
        c["ctx"] = rng.choice([0, _log(rng, 1, 2000)])
        c["rot"] = rng.choice([32, 64, 96, 128, 128, 128])
        c["norm"] = rng.random() < 0.6
        c["pairs"] = rng.random() < 0.4
        c["q32"] = rng.random() < 0.3
        return c
    if op == "prefill":
        c["batch"] = _log(rng, 1, 32)
        c["ctx"] = rng.choice([0, 0, _log(rng, 1, 5000)])
        c["t"] = _log(rng, 1, 8000)
        while c["batch"] * h_q * c["t"] * (c["t"] / 2 + c["ctx"]) > 15 * 8192 * 8192:
            c["t"] = c["t"] * 4 // 5
        return c
    c["batch"] = _log(rng, 1, 96)
    c["t"] = rng.choice([1, 1, _log(rng, 2, 17), _log(rng, 2, 300)])
    c["ctx"] = _log(rng, 1, 2000)
    c["prefix"] = _log(rng, 1, 20000)
    while c["batch"] * h_q * c["t"] * (c["t"] / 2 + c["ctx"] + c["prefix"]) > 15 * 8192 * 8192:
        c["t"] = max(1, c["t"] * 4 // 5)
    return c


def _lengths(case):
    """(new tokens, cached positions) of every sequence: plain whole numbers that follow from the case alone."""
    r = random.Random(case["spread"] * 7919 + case["batch"])
    t, ctx = case["t"], case["ctx"]
    new = [t if not case["ragged"] else 1 + int(t * r.random() ** 2) for _ in range(case["batch"])]
    if case["ragged"]:
        new[r.randrange(len(new))] = t  # one is as long as the case says
        new = [min(t, n) for n in new]
    old = [ctx if ctx < 2 else r.randrange(ctx // 2, ctx + 1) for _ in range(case["batch"])]
    return new, old


def work(case):
    new, old = _lengths(case)
    n, h_q, h_kv = sum(new), case["h_q"], case["h_kv"]
    if case["op"] == "rope":
        rows = n * (h_q + 2 * h_kv) * D
        out = n * h_q * D * (4 if case["q32"] else 2) + n * 2 * h_kv * D * 2
        return {"bytes": 4 * rows + out + 4 * n * case["rot"], "flops": 8 * rows}
    p = case.get("prefix", 0)
    pairs = sum(m * (c + p) + m * (m + 1) // 2 for m, c in zip(new, old))  # (token, visible key)
    keys = sum(m + c for m, c in zip(new, old)) + p
    return {"bytes": 4 * n * h_q * D + 4 * keys * h_kv * D, "flops": 4 * pairs * h_q * D}


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    new, old = _lengths(case)
    batch, n, h_q, h_kv = case["batch"], sum(new), case["h_q"], case["h_kv"]
    capacity = max(m + c for m, c in zip(new, old)) + 3

    def normal(*shape, dtype=torch.bfloat16, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)

    s = {"case": case, "new": new, "old": old}
    s["lens"] = torch.tensor(old, dtype=torch.int32, device="cuda")
    starts = [0]
    for m in new:
        starts.append(starts[-1] + m)
    s["cu"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    # every position holds something: what a finished sequence left behind its successor's end stays there
    s["k_cache"] = normal(batch, h_kv, capacity, D)
    s["v_cache"] = normal(batch, h_kv, capacity, D)
    if case["op"] == "rope":
        s["qkv"] = normal(n, (h_q + 2 * h_kv) * D, dtype=torch.float32, scale=2.0)
        positions = torch.arange(capacity, device="cuda", dtype=torch.float64)
        half = case["rot"] // 2
        angle = positions[:, None] * 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        s["table"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        s["q_gamma"] = normal(D, dtype=torch.float32, scale=0.2) + 1 if case["norm"] else None
        s["k_gamma"] = normal(D, dtype=torch.float32, scale=0.2) + 1 if case["norm"] else None
        s["q_out"] = torch.empty(n, h_q * D, device="cuda", dtype=torch.float32 if case["q32"] else torch.bfloat16)
        return s
    s["q"] = normal(n, h_q * D, scale=1.5)
    s["out"] = torch.empty(n, h_q * D, device="cuda", dtype=torch.bfloat16)
    if case["op"] == "prefix":
        s["prefix_k"] = normal(h_kv, case["prefix"] + 5, D)
        s["prefix_v"] = normal(h_kv, case["prefix"] + 5, D)
        s["prefix_len"] = torch.tensor([case["prefix"]], dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if c["op"] == "rope":
        return _run_rope(s, c)
    if own:
        from quantized_speculative_decoding_packed_b200 import qspec
        if c["op"] == "prefill":
            return qspec.attn_prefill(s["q"], s["cu"], s["lens"], s["k_cache"], s["v_cache"], c["h_q"], out=s["out"])
        return qspec.attn_prefix(s["q"], s["lens"], 0, s["k_cache"], s["v_cache"], c["h_q"], s["prefix_k"], s["prefix_v"],
                                 s["prefix_len"], cu=s["cu"] if c["ragged"] else None, out=s["out"])
    return _attend(s, c)


def _run_rope(s, c):
    if own:
        from quantized_speculative_decoding_packed_b200 import qspec
        q = qspec.qkv_rope_append(s["qkv"], s["lens"], 0, s["k_cache"], s["v_cache"], c["h_q"], s["table"],
                                  cu=s["cu"] if c["ragged"] else None, q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], eps=1e-6,
                                  interleaved=c["pairs"], q_out=s["q_out"])
        return q, s["k_cache"], s["v_cache"]
    h_q, h_kv, half = c["h_q"], c["h_kv"], c["rot"] // 2
    qkv = s["qkv"].view(-1, h_q + 2 * h_kv, D)
    token = torch.arange(qkv.shape[0], device=qkv.device)
    b = torch.searchsorted(s["cu"][1:], token, right=True)
    pos = s["lens"][b] + token - s["cu"][b]
    cos, sin = s["table"][pos, None, :half], s["table"][pos, None, half:]

    def turned(x, gamma):
        if gamma is not None:
            x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gamma
        r = x[..., :2 * half]
        a, d = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :half], r[..., half:])
        a, d = a * cos - d * sin, d * cos + a * sin
        r = torch.stack((a, d), -1).flatten(-2) if c["pairs"] else torch.cat((a, d), -1)
        return torch.cat((r, x[..., 2 * half:]), -1)

    q = turned(qkv[:, :h_q], s["q_gamma"])
    s["q_out"].copy_(q.flatten(1))
    s["k_cache"][b, :, pos] = turned(qkv[:, h_q:h_q + h_kv], s["k_gamma"]).to(torch.bfloat16)
    s["v_cache"][b, :, pos] = qkv[:, h_q + h_kv:].to(torch.bfloat16)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _attend(s, c):
    """Every sequence padded to the longest one: scores of all its tokens against its keys, and against the prefix's."""
    h_q, h_kv, batch, t = c["h_q"], c["h_kv"], c["batch"], max(s["new"])
    cu, lens = s["cu"].long(), s["lens"].long()
    at = torch.arange(t, device="cuda")
    there = at[None] < (cu[1:] - cu[:-1])[:, None]                                   # [batch][t]
    row = torch.where(there, cu[:-1, None] + at[None], 0)
    q = s["q"][row].float().view(batch, t, h_kv, h_q // h_kv, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(batch, h_kv, -1, D) * D ** -0.5                                    # rows (head in group, token)
    keys = max(m + o for m, o in zip(s["new"], s["old"]))
    k, v = s["k_cache"][:, :, :keys].float(), s["v_cache"][:, :, :keys].float()
    seen = torch.arange(keys, device="cuda")[None, None] <= (lens[:, None] + at[None])[..., None]   # [batch][t][keys]
    # positions that no token of the sequence sees are not part of it
    v = torch.where((torch.arange(keys, device="cuda")[None] < (lens + cu[1:] - cu[:-1])[:, None])[:, None, :, None], v, 0)
    score = (q @ k.transpose(-1, -2)).view(batch, h_kv, -1, t, keys)
    score = score.masked_fill_(~seen[:, None, None], float("-inf")).view(batch, h_kv, -1, keys)
    top = score.amax(-1, keepdim=True)
    if c["op"] == "prefix":
        pk, pv = s["prefix_k"][:, :c["prefix"]].float(), s["prefix_v"][:, :c["prefix"]].float()
        rows = q.transpose(0, 1).reshape(h_kv, -1, D)
        far = rows @ pk.transpose(-1, -2)
        most = far.amax(-1, keepdim=True).view(h_kv, batch, -1, 1).transpose(0, 1)
        top = torch.maximum(top, most)
        far = far.sub_(top.transpose(0, 1).reshape(h_kv, -1, 1)).exp_()
        score = score.sub_(top).exp_()
        total = score.sum(-1, keepdim=True) + far.sum(-1, keepdim=True).view(h_kv, batch, -1, 1).transpose(0, 1)
        mixed = score @ v + (far @ pv).view(h_kv, batch, -1, D).transpose(0, 1)
    else:
        score = score.sub_(top).exp_()
        total = score.sum(-1, keepdim=True)
        mixed = score @ v
    mixed = (mixed / total).view(batch, h_kv, -1, t, D).permute(0, 3, 1, 2, 4).reshape(batch, t, h_q * D)
    s["out"].copy_(mixed[there])
    return s["out"]


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s, case) if case["op"] == "rope" else _exact_attention(s, case)


def _exact_rope(s, case):
    h_q, h_kv, rot = case["h_q"], case["h_kv"], case["rot"]
    heads = s["qkv"].double().reshape(-1, h_q + 2 * h_kv, D)
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    q_all, first = [], 0
    j = torch.arange(rot // 2, device="cuda")
    lo, hi = (2 * j, 2 * j + 1) if case["pairs"] else (j, j + rot // 2)
    for b, (m, o) in enumerate(zip(s["new"], s["old"])):
        x = heads[first:first + m].clone()
        first += m
        for part, gamma in ((slice(0, h_q), s["q_gamma"]), (slice(h_q, h_q + h_kv), s["k_gamma"])):
            y = x[:, part]
            if gamma is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * gamma.double()
            turn = torch.complex(s["table"][o:o + m, :rot // 2].double(), s["table"][o:o + m, rot // 2:].double())
            z = torch.complex(y[..., lo], y[..., hi]) * turn[:, None]
            y = y.clone()
            y[..., lo], y[..., hi] = z.real, z.imag
            x[:, part] = y
        q_all.append(x[:, :h_q].flatten(1))
        k_cache[b, :, o:o + m] = x[:, h_q:h_q + h_kv].transpose(0, 1)
        v_cache[b, :, o:o + m] = x[:, h_q + h_kv:].transpose(0, 1)
    return torch.cat(q_all), k_cache, v_cache


def _exact_attention(s, case):
    h_q, h_kv = case["h_q"], case["h_kv"]
    out, first = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for b, (m, o) in enumerate(zip(s["new"], s["old"])):
        for h in range(h_q):
            kv = h // (h_q // h_kv)
            k, v = s["k_cache"][b, kv, :o + m].double(), s["v_cache"][b, kv, :o + m].double()
            hidden = torch.ones(m, o + m, dtype=torch.bool, device="cuda").triu(o + 1)
            if case["op"] == "prefix":
                k = torch.cat((s["prefix_k"][kv, :case["prefix"]].double(), k))
                v = torch.cat((s["prefix_v"][kv, :case["prefix"]].double(), v))
                hidden = torch.nn.functional.pad(hidden, (case["prefix"], 0))
            q = s["q"][first:first + m, h * D:(h + 1) * D].double()
            weight = torch.softmax((q @ k.T / D ** 0.5).masked_fill(hidden, float("-inf")), -1)
            out[first:first + m, h * D:(h + 1) * D] = weight @ v
        first += m
    return out
