"""The prompt path on the GPU (norms and rotation with cache append, packed causal attention,
attention behind a shared prefix) against plain 64-bit implementations.

Bound of an attention output, element-wise, with w the exact weights, W = sum_j w_j |v_j| and
A = max_j sum_i |q_i k_ji| / sqrt(128) of its row:
  * the weights are rounded to bf16, at most 2^-8 of each:                    2^-8 W
  * a score is a sum of 128 exact products in fp32 (2^-24 each, taken twice, for the tensor
    cores may cut instead of round): an error of 2^-16 A in the exponent, in weight and sum: 2^-15 A W
  * the sum of weights and the weighted values over n keys in fp32:            n 2^-22 W
  * exp2: a quarter of the weights come from a cubic that is off by up to 7.5e-5, the others from ex2 (2^-22);
    the argument has 2^-24 of at most 2^6 for weights that count.  In a weight and in the sum of weights
    that divides it, 2 (7.5e-5 + 2^-18) = 1.58e-4 < 2.44e-4:                    2^-12 W
  * the output rounded to bf16:                                                2^-8 |out|
The products of these are below 1 % of their sum.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

D = 128
BAD_INPUT = 6


@pytest.fixture(scope="module")
def qs():
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, device="cuda", generator=g) * scale).to(dtype)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _starts(new):
    s = [0]
    for m in new:
        s.append(s[-1] + m)
    return s


def _attention64(q, keys, values, hidden):
    """(out, bound) of one head in 64 bits: q [m][128], hidden [m][n] true where a key is not seen."""
    q, k, v = q.double(), keys.double(), values.double()
    s = (q @ k.T) / math.sqrt(D)
    w = torch.softmax(s.masked_fill(hidden, -math.inf), -1)
    out, mag = w @ v, w @ v.abs()
    a = ((q.abs() @ k.abs().T) / math.sqrt(D)).masked_fill(hidden, 0).amax(-1, keepdim=True)
    n = k.shape[0]
    bound = 1.01 * (2.0 ** -8 * (mag + out.abs()) + mag * (2.0 ** -15 * a + n * 2.0 ** -22 + 2.0 ** -12))
    return out, bound


def _check(out, new, old, q, kc, vc, h_q, pk=None, pv=None, plen=0, rows=None):
    """Every live row of `out` within its bound of the 64-bit attention."""
    h_kv = kc.shape[1]
    first, worst, num, den = 0, 0.0, 0.0, 0.0
    for b, (m, o) in enumerate(zip(new, old)):
        for h in range(h_q):
            if m == 0:
                break
            kv = h // (h_q // h_kv)
            k, v = kc[b, kv, :o + m], vc[b, kv, :o + m]
            hidden = torch.ones(m, o + m, dtype=torch.bool, device="cuda").triu(o + 1)
            if plen:
                k, v = torch.cat((pk[kv, :plen], k)), torch.cat((pv[kv, :plen], v))
                hidden = torch.nn.functional.pad(hidden, (plen, 0))
            ref, bound = _attention64(q[first:first + m, h * D:(h + 1) * D], k, v, hidden)
            got = out[first:first + m, h * D:(h + 1) * D].double()
            assert torch.isfinite(got).all(), (b, h)
            err = (got - ref).abs()
            worst = max(worst, float((err / bound.clamp_min(1e-30)).max()))
            num, den = num + float((err * err).sum()), den + float((ref * ref).sum())
            if worst > 1:
                at = int((err / bound).amax(-1).argmax())
                raise AssertionError(f"sequence {b} head {h} row {at}: {worst:.3g} of the bound")
        first += m
    # each of the two roundings has at most 2^-9 rms of its own size (uniform within half a step: 2^-8 / sqrt 3)
    assert math.sqrt(num / den) <= 2 * 2.0 ** -8, math.sqrt(num / den)


def _case(seed, new, old, h_q, h_kv, extra=3, pad=0, ld_more=0):
    """q, cache (NaN wherever no token sees it), cu, lens."""
    g = _gen(seed)
    n, batch = sum(new), len(new)
    l_max = max(m + o for m, o in zip(new, old)) + extra
    kc = _randn(g, batch, h_kv, l_max, D)
    vc = _randn(g, batch, h_kv, l_max, D)
    for b, (m, o) in enumerate(zip(new, old)):
        kc[b, :, o + m:] = math.nan
        vc[b, :, o + m:] = math.nan
    q = _randn(g, n + pad, h_q * D + ld_more, scale=1.5)[:, :h_q * D]
    return q, kc, vc, _i32(_starts(new)), _i32(old)


# ---------------------------------------------------------------- packed prompts
PREFILL = [
    # new tokens, cached, h_q, h_kv
    ([1], [0], 1, 1),
    ([128], [0], 1, 1),
    ([129], [0], 2, 1),
    ([200], [0], 4, 4),
    ([256], [0], 2, 2),
    ([257], [0], 2, 2),
    ([700], [0], 8, 2),
    ([1], [1000], 4, 1),
    ([5], [300], 32, 8),
    ([3, 0, 130, 1, 64], [0, 7, 5, 0, 200], 4, 2),
    ([17, 33, 400, 1, 129, 128], [0, 0, 0, 0, 0, 0], 8, 8),
    ([100, 50], [127, 128], 14, 2),           # 7 heads a group: 18 tokens a tile, 126 rows
    ([65, 3], [10, 0], 12, 4),                # 3 heads a group
    ([40], [3], 16, 1),
    ([9, 2], [0, 31], 100, 1),                # 100 heads a group: one token a tile
    ([1, 1, 1], [15, 16, 17], 128, 1),
    ([1500], [0], 2, 2),
    ([300, 1, 2000], [1000, 4000, 0], 4, 2),
    ([1] * 20, [150 * b for b in range(20)], 16, 4),          # few items, too long for one CTA each
    ([2] * 9, [1000, 0, 3, 800, 127, 128, 129, 500, 1020], 8, 8),     # and short enough
]


@pytest.mark.parametrize("new,old,h_q,h_kv", PREFILL)
def test_prefill(qs, new, old, h_q, h_kv):
    q, kc, vc, cu, lens = _case(1, new, old, h_q, h_kv)
    out = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    torch.cuda.synchronize()
    _check(out, new, old, q, kc, vc, h_q)


def test_prefill_strides_and_padding_rows(qs):
    """Rows of q and out with gaps; rows behind the last sequence stay as they were."""
    new, old, h_q, h_kv = [70, 200, 0], [5, 0, 9], 8, 2
    q, kc, vc, cu, lens = _case(2, new, old, h_q, h_kv, pad=41, ld_more=24)
    q[sum(new):] = math.nan
    wide = torch.full((q.shape[0], h_q * D + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    out = qs.attn_prefill(q, cu, lens, kc, vc, h_q, out=wide[:, :h_q * D])
    torch.cuda.synchronize()
    _check(out, new, old, q, kc, vc, h_q)
    assert bool((wide[:, h_q * D:] == 7).all()) and bool((wide[sum(new):] == 7).all())


@pytest.mark.parametrize("new,old,h_q,h_kv", [([300, 1, 2000], [1000, 4000, 0], 4, 2), ([1500], [9000], 8, 1),
                                              ([3], [40000], 2, 1)])
def test_prefill_is_the_same_every_time(qs, new, old, h_q, h_kv):
    """Pieces of split items are joined in their order, whichever CTA comes last."""
    q, kc, vc, cu, lens = _case(12, new, old, h_q, h_kv)
    want = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    _check(want, new, old, q, kc, vc, h_q)
    for _ in range(20):
        assert torch.equal(qs.attn_prefill(q, cu, lens, kc, vc, h_q), want)


def test_prefill_extreme_scores(qs):
    """Scores that rise along the keys (the running maximum moves in every tile), fall, and are all equal."""
    h_q = h_kv = 3
    m = 600
    q, kc, vc, cu, lens = _case(3, [m], [0], h_q, h_kv)
    ramp = torch.linspace(-40, 40, m, device="cuda")
    q[:] = 0
    q[:, 0::D] = math.sqrt(D)
    kc[0, :, :m] = 0
    kc[0, 0, :m, 0] = ramp.to(torch.bfloat16)
    kc[0, 1, :m, 0] = (-ramp).to(torch.bfloat16)
    out = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    torch.cuda.synchronize()
    _check(out, [m], [0], q, kc, vc, h_q)


def test_prefill_refuses_bad_lengths_on_the_device(qs):
    """A sequence that does not fit its cache, or with a negative length: zero rows and a status; the others as ever."""
    new, old, h_q, h_kv = [20, 30, 40], [0, 4, 8], 4, 2
    q, kc, vc, cu, lens = _case(4, new, old, h_q, h_kv)
    ref = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    for bad in (-1, kc.shape[2] - 29, 2 ** 31 - 1):
        wrong = lens.clone()
        wrong[1] = bad
        work = torch.zeros(qs.attn_prefill_workspace_size(), dtype=torch.uint8, device="cuda")
        out = torch.full_like(ref, 3.0)
        qs.attn_prefill(q, cu, wrong, kc, vc, h_q, out=out, work=work)
        assert qs.workspace_status(work) == BAD_INPUT and qs.workspace_status(work) == 0
        assert bool((out[20:50] == 0).all())
        _check(out[:20], new[:1], old[:1], q, kc, vc, h_q)
        _check(out[50:], new[2:], old[2:], q[50:], kc[2:], vc[2:], h_q)
    for starts in ([0, 20, 10, 90], [0, 20, 50, 91], [-5, 20, 50, 90]):
        work = torch.zeros(qs.attn_prefill_workspace_size(), dtype=torch.uint8, device="cuda")
        qs.attn_prefill(q, _i32(starts), lens, kc, vc, h_q, work=work)
        assert qs.workspace_status(work) == BAD_INPUT


# ---------------------------------------------------------------- shared prefix
PREFIX = [
    # tokens per sequence (uniform) or list, cached, h_q, h_kv, prefix
    (1, [0], 1, 1, 1),
    (1, [0], 4, 1, 128),
    (1, [5, 300, 17, 128], 32, 8, 500),
    (5, [5, 300, 17, 128], 32, 8, 1000),
    (1, [10] * 40, 4, 4, 129),
    (5, [3, 700, 64] * 20, 8, 2, 3000),
    (17, [100, 0], 14, 2, 255),
    (200, [0, 50], 4, 2, 700),
    (2, [33] * 70, 16, 1, 4000),
    (3, [4, 8], 4, 2, 0),
    ([3, 0, 90, 1, 300], [0, 5, 0, 77, 10], 8, 2, 640),
    ([1] * 300, [7] * 300, 4, 2, 2000),
    ([700, 5], [0, 9], 2, 1, 900),            # long runs behind a prefix that ends inside a tile
    ([1200], [300], 8, 8, 400),
    (300, [0, 130, 70], 4, 4, 1050),
    (16, [40] * 8, 8, 2, 5000),               # few items, too long for one CTA each
    (1, [40] * 30, 4, 4, 900),                # and short enough
]


def _prefix(seed, h_kv, plen, more=5):
    g = _gen(seed)
    pk, pv = _randn(g, h_kv, plen + more, D), _randn(g, h_kv, plen + more, D)
    pk[:, plen:] = math.nan
    pv[:, plen:] = math.nan
    return pk, pv


@pytest.mark.parametrize("t,old,h_q,h_kv,plen", PREFIX)
def test_prefix(qs, t, old, h_q, h_kv, plen):
    packed = isinstance(t, list)
    new = t if packed else [t] * len(old)
    q, kc, vc, cu, lens = _case(5, new, old, h_q, h_kv)
    pk, pv = _prefix(6, h_kv, plen)
    out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu if packed else None)
    torch.cuda.synchronize()
    _check(out, new, old, q, kc, vc, h_q, pk, pv, plen)


def test_prefix_offset_moves_the_window(qs):
    """offset o with lengths l is the call with lengths l + o."""
    new, old, h_q, h_kv, plen = [1] * 3, [20, 7, 130], 4, 2, 200
    q, kc, vc, cu, lens = _case(7, new, old, h_q, h_kv)
    pk, pv = _prefix(8, h_kv, plen)
    a = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]))
    b = qs.attn_prefix(q, lens - 4, 4, kc, vc, h_q, pk, pv, _i32([plen]))
    assert torch.equal(a, b)


def test_prefix_refuses_bad_lengths_on_the_device(qs):
    new, old, h_q, h_kv, plen = [2] * 3, [20, 7, 130], 4, 2, 200
    q, kc, vc, cu, lens = _case(9, new, old, h_q, h_kv)
    pk, pv = _prefix(10, h_kv, plen)
    size = qs.attn_prefix_workspace_size(6, 3, h_q, h_kv)
    for bad in (-1, pk.shape[1] + 1):
        work = torch.zeros(size, dtype=torch.uint8, device="cuda")
        out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([bad]), work=work)
        assert qs.workspace_status(work) == BAD_INPUT
        assert bool((out == 0).all())
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    wrong = lens.clone()
    wrong[0] = -3
    out = qs.attn_prefix(q, wrong, 0, kc, vc, h_q, pk, pv, _i32([plen]), work=work)
    assert qs.workspace_status(work) == BAD_INPUT
    assert bool((out[:2] == 0).all())
    _check(out[2:], new[1:], old[1:], q[2:], kc[1:], vc[1:], h_q, pk, pv, plen)


def test_one_query_sees_a_cache_past_32_bit_offsets(qs):
    """A cache of 2^31 elements: the last head of the last sequence lies behind 2^32 bytes."""
    h_q, h_kv, batch = 2, 2, 2
    l_max = 2 ** 22 + 64
    kc = torch.zeros(batch, h_kv, l_max, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    g = _gen(11)
    old = [100, l_max - 3]
    new = [2, 3]
    for b, (m, o) in enumerate(zip(new, old)):
        lo = max(0, o + m - 5000)
        kc[b, :, lo:o + m] = _randn(g, h_kv, o + m - lo, D, scale=2.0)
        vc[b, :, lo:o + m] = _randn(g, h_kv, o + m - lo, D)
        kc[b, :, :lo, 0] = -300.0                 # their scores are so low that they weigh nothing
    q = _randn(g, 5, h_q * D)
    q[:, 0::D] = 8.0
    out = qs.attn_prefill(q, _i32(_starts(new)), _i32(old), kc, vc, h_q)
    torch.cuda.synchronize()
    for b, (m, o) in enumerate(zip(new, old)):
        lo = max(0, o + m - 5000)
        first = sum(new[:b])
        for h in range(h_q):
            hidden = torch.ones(m, o + m - lo, dtype=torch.bool, device="cuda").triu(o - lo + 1)
            ref, bound = _attention64(q[first:first + m, h * D:(h + 1) * D], kc[b, h, lo:o + m], vc[b, h, lo:o + m], hidden)
            assert bool(((out[first:first + m, h * D:(h + 1) * D].double() - ref).abs() <= bound).all()), (b, h)


# ---------------------------------------------------------------- norms, rotation, append
def _table(qs, rot, positions, base=10000.0):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return qs.rope_table(base ** (-i / (rot // 2)), positions)


@pytest.mark.parametrize("rot,positions", [(8, 1), (64, 777), (128, 200000)])
def test_rope_table(qs, rot, positions):
    """cos and sin in 64 bits, rounded once to fp32: within half a step (values at most 1: 2^-24) and 2^-40."""
    table = _table(qs, rot, positions).double()
    i = torch.arange(rot // 2, dtype=torch.float64)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-i / (rot // 2))
    ref = torch.cat((angle.cos(), angle.sin()), 1).cuda()
    # the frequencies of the two sides may differ by a few 2^-53, which a position multiplies
    assert float((table - ref).abs().max()) <= 2.0 ** -24 + positions * 2.0 ** -50


def _rope64(x, gamma, eps, table, pos, interleaved):
    """(rotated heads, scale of their rounding errors) in 64 bits: x [tokens][heads][128]."""
    x = x.double()
    if gamma is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gamma.double()
    if table is None:
        return x, x.abs()
    rot = table.shape[1]
    c, s = table[pos, :rot // 2].double()[:, None], table[pos, rot // 2:].double()[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, mag = x.clone(), x.abs()
    ra, rb = a * c - b * s, b * c + a * s
    ma, mb = a.abs() * c.abs() + b.abs() * s.abs(), b.abs() * c.abs() + a.abs() * s.abs()
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = ra, rb
        mag[..., 0:rot:2], mag[..., 1:rot:2] = ma, mb
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = ra, rb
        mag[..., :rot // 2], mag[..., rot // 2:rot] = ma, mb
    return y, mag


ROPE = [
    # new, cached, h_q, h_kv, rot, interleaved, q gamma, k gamma, fp32 queries, packed, prefix
    ([1] * 3, [0, 9, 200], 32, 8, 128, False, False, False, False, False, 0),
    ([5] * 2, [0, 9], 4, 4, 128, False, True, True, True, False, 0),
    ([5] * 2, [0, 9], 4, 4, 128, True, True, False, False, False, 70),
    ([3, 0, 40, 1], [5, 0, 0, 8], 14, 2, 64, False, False, True, False, True, 0),
    ([3, 0, 40, 1], [5, 0, 0, 8], 14, 2, 96, True, True, True, True, True, 33),
    ([7], [2], 1, 1, 8, False, False, False, False, True, 0),
    ([2, 2], [2, 4], 64, 8, 0, False, True, True, False, True, 0),
    ([1] * 100, list(range(100)), 8, 8, 128, False, True, True, False, True, 0),
]


@pytest.mark.parametrize("new,old,h_q,h_kv,rot,pairs,gq,gk,q32,packed,pre", ROPE)
def test_rope_append(qs, new, old, h_q, h_kv, rot, pairs, gq, gk, q32, packed, pre):
    """fp32 arithmetic: a norm within 10 fp32 steps (sum of 128, rsqrt, two products), a rotation within
    2 more of its terms' magnitude; then the output's own rounding.  Values are rounded exactly once."""
    g = _gen(21)
    n, batch, pad = sum(new), len(new), 4 if packed else 0
    l_max = max(m + o for m, o in zip(new, old)) + 2
    qkv = _randn(g, n + pad, (h_q + 2 * h_kv) * D + 4, scale=3.0, dtype=torch.float32)[:, :(h_q + 2 * h_kv) * D]
    kc = _randn(g, batch, h_kv, l_max, D)
    vc = _randn(g, batch, h_kv, l_max, D)
    k0, v0 = kc.clone(), vc.clone()
    qg = _randn(g, D, dtype=torch.float32) if gq else None
    kg = _randn(g, D, dtype=torch.float32) if gk else None
    table = _table(qs, rot, l_max + pre) if rot else None
    q_out = torch.full((n + pad, h_q * D), 5.0, dtype=torch.float32 if q32 else torch.bfloat16, device="cuda")
    got = qs.qkv_rope_append(qkv, _i32(old), 0, kc, vc, h_q, table, cu=_i32(_starts(new)) if packed else None,
                             prefix_len=_i32([pre]) if pre else None, q_gamma=qg, k_gamma=kg, eps=1e-5,
                             interleaved=pairs, q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out and bool((q_out[n:] == 5).all())
    seq = torch.tensor([b for b, m in enumerate(new) for _ in range(m)], device="cuda")
    at = torch.tensor([o + i for m, o in zip(new, old) for i in range(m)], device="cuda")
    heads = qkv[:n].reshape(n, h_q + 2 * h_kv, D)
    f32, b16 = 2.0 ** -24, 2.0 ** -8
    ref, mag = _rope64(heads[:, :h_q], qg, 1e-5, table, at + pre, pairs)
    err = (q_out[:n].double().reshape(n, h_q, D) - ref).abs()
    assert bool((err <= 24 * f32 * mag + (f32 if q32 else b16) * ref.abs() * 1.001).all())
    ref, mag = _rope64(heads[:, h_q:h_q + h_kv], kg, 1e-5, table, at + pre, pairs)
    err = (kc[seq, :, at].double() - ref).abs()
    assert bool((err <= 24 * f32 * mag + b16 * ref.abs() * 1.001).all())
    assert torch.equal(vc[seq, :, at], heads[:, h_q + h_kv:].to(torch.bfloat16))
    k0[seq, :, at] = kc[seq, :, at]
    v0[seq, :, at] = vc[seq, :, at]
    assert torch.equal(k0.view(torch.int16), kc.view(torch.int16))       # nothing else is written
    assert torch.equal(v0.view(torch.int16), vc.view(torch.int16))


def test_rope_without_rotation_is_kv_append(qs):
    g = _gen(22)
    qkv = _randn(g, 6, (4 + 2 * 2) * D, dtype=torch.float32)
    lens = _i32([4, 9])
    a = [torch.zeros(2, 2, 20, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    qs.kv_append(qkv, lens, 1, a[0], a[1], 4)
    qs.qkv_rope_append(qkv, lens, 1, a[2], a[3], 4, None)
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])


def test_rope_in_place_feeds_attn_decode(qs):
    """fp32 queries turned where they lie: the projection's other columns stay, attn_decode reads the rows."""
    g = _gen(23)
    h_q, h_kv, lens = 4, 2, _i32([40, 3])
    qkv = _randn(g, 2, (h_q + 2 * h_kv) * D, dtype=torch.float32)
    before = qkv.clone()
    kc, vc = _randn(g, 2, h_kv, 50, D), _randn(g, 2, h_kv, 50, D)
    table = _table(qs, 128, 64)
    apart = qs.qkv_rope_append(qkv, lens, 0, kc.clone(), vc.clone(), h_q, table,
                               q_out=torch.empty(2, h_q * D, dtype=torch.float32, device="cuda"))
    qs.qkv_rope_append(qkv, lens, 0, kc, vc, h_q, table, q_out=qkv[:, :h_q * D])
    assert torch.equal(qkv[:, :h_q * D], apart) and torch.equal(qkv[:, h_q * D:], before[:, h_q * D:])
    out = qs.attn_decode(qkv, lens, 0, kc, vc, h_q, 50)
    q16 = apart.to(torch.bfloat16)
    many = qs.attn_prefill(q16, _i32([0, 1, 2]), lens, kc, vc, h_q)
    torch.cuda.synchronize()
    _check(many, [1, 1], [40, 3], q16, kc, vc, h_q)
    assert float((many.double() - out.double()).norm() / out.double().norm()) < 2e-2      # bf16 queries


def test_rope_skips_positions_outside(qs):
    g = _gen(24)
    h_q = h_kv = 1
    qkv = _randn(g, 4, 3 * D, dtype=torch.float32)
    kc, vc = torch.zeros(2, 1, 8, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, 1, 8, D, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    q = torch.full((4, D), 9.0, dtype=torch.bfloat16, device="cuda")
    qs.qkv_rope_append(qkv, _i32([7, 0]), 0, kc, vc, h_q, _table(qs, 128, 64), q_out=q, work=work)
    assert qs.workspace_status(work) == BAD_INPUT
    assert bool((q[1] == 9).all()) and not bool((q[0] == 9).any())       # position 8 of 8 is refused, 7 is written
    assert bool((kc[1, 0, 2:] == 0).all())
    qs.qkv_rope_append(qkv, _i32([0, 0]), 0, kc, vc, h_q, _table(qs, 128, 1), q_out=q, work=work)
    assert qs.workspace_status(work) == BAD_INPUT                         # the table ends before position 1
    qs.qkv_rope_append(qkv, _i32([-1, 0]), 0, kc, vc, h_q, None, work=work)
    assert qs.workspace_status(work) == BAD_INPUT
    qs.qkv_rope_append(qkv, _i32([0, 0]), 0, kc, vc, h_q, _table(qs, 128, 64), prefix_len=_i32([-1]), work=work)
    assert qs.workspace_status(work) == BAD_INPUT


# ---------------------------------------------------------------- as they are used
def test_two_streams_and_graphs(qs):
    """Calls on two streams at once have workspaces of their own; captured calls give what eager ones give, on
    new inputs in the captured buffers, beside eager calls."""
    new, old, h_q, h_kv, plen = [40, 300, 7], [3, 0, 200], 8, 2, 500
    sets = [_case(30 + i, new, old, h_q, h_kv) for i in range(2)]
    pk, pv = _prefix(40, h_kv, plen)
    plen_d = _i32([plen])

    def both(i):
        q, kc, vc, cu, lens = sets[i]
        return (qs.attn_prefill(q, cu, lens, kc, vc, h_q),
                qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, plen_d, cu=cu),
                qs.attn_prefix(q[:3], lens, 0, kc, vc, h_q, pk, pv, plen_d))

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(both(i))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i]))
    q, kc, vc, cu, lens = [x.clone() for x in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = (qs.attn_prefill(q, cu, lens, kc, vc, h_q), qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, plen_d, cu=cu),
                qs.attn_prefix(q[:3], lens, 0, kc, vc, h_q, pk, pv, plen_d))
    for i in (1, 0, 1):
        for dst, src in zip((q, kc, vc, cu, lens), sets[i]):
            dst.copy_(src)
        graph.replay()
        eager = both(i)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want[i]))
        assert all(torch.equal(x, y) for x, y in zip(eager, want[i]))


def test_captured_call_on_a_forked_stream_has_its_own_workspace(qs):
    """stream= names another stream than the captured one that is current: two calls at once in a graph."""
    new, old, h_q, h_kv = [300, 20], [500, 900], 8, 2
    runs = [_case(seed, new, old, h_q, h_kv) for seed in (41, 42)]
    outs = [torch.empty(sum(new), h_q * D, dtype=torch.bfloat16, device="cuda") for _ in runs]
    want = [qs.attn_prefill(q, cu, lens, kc, vc, h_q) for q, kc, vc, cu, lens in runs]
    torch.cuda.synchronize()
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        side.wait_stream(main)
        for (q, kc, vc, cu, lens), out, stream in zip(runs, outs, (side, None)):
            qs.attn_prefill(q, cu, lens, kc, vc, h_q, out=out, stream=stream)
        main.wait_stream(side)
    for _ in range(3):
        for out in outs:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            assert torch.equal(out, ref)


def test_default_workspace_grows_and_is_kept(qs):
    """A larger call after a captured one: the graph's own buffer is untouched, the eager one is replaced."""
    h_q, h_kv, plen = 4, 2, 100
    pk, pv = _prefix(41, h_kv, plen)
    small = _case(42, [1] * 4, [9] * 4, h_q, h_kv)
    big = _case(43, [1] * 400, [30] * 400, h_q, h_kv)
    call = lambda c: qs.attn_prefix(c[0], c[4], 0, c[1], c[2], h_q, pk, pv, _i32([plen]))   # noqa: E731
    want = call(small)
    _check(call(big), [1] * 400, [30] * 400, big[0], big[1], big[2], h_q, pk, pv, plen)
    assert torch.equal(call(small), want)


def test_prompts_then_rounds_behind_a_prefix(qs):
    """A prefix and prompts are read in, then drafting and verifying passes run, all through one cache: every
    attention against 64 bits from the same cache, the cache and the lengths as the calls say."""
    g = _gen(50)
    h_q, h_kv, batch, gamma, plen, l_max = 8, 2, 3, 2, 77, 200
    width = (h_q + 2 * h_kv) * D
    table = _table(qs, 128, plen + l_max)
    qg, kg = _randn(g, D, dtype=torch.float32), _randn(g, D, dtype=torch.float32)
    # the prefix: a cache of one sequence
    pk = torch.zeros(1, h_kv, 128, D, dtype=torch.bfloat16, device="cuda")
    pv = torch.zeros_like(pk)
    zero = _i32([0])
    qkv = _randn(g, plen, width, dtype=torch.float32)
    q = qs.qkv_rope_append(qkv, zero, 0, pk, pv, h_q, table, cu=_i32([0, plen]), q_gamma=qg, k_gamma=kg)
    out = qs.attn_prefill(q, _i32([0, plen]), zero, pk, pv, h_q)
    _check(out, [plen], [0], q, pk, pv, h_q)
    # the prompts behind it (one slot has none)
    kc = torch.zeros(batch, h_kv, l_max, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    lens, plen_d = _i32([0] * batch), _i32([plen])
    new = [30, 0, 95]
    cu = _i32(_starts(new))
    qkv = _randn(g, sum(new), width, dtype=torch.float32)
    q = qs.qkv_rope_append(qkv, lens, 0, kc, vc, h_q, table, cu=cu, prefix_len=plen_d, q_gamma=qg, k_gamma=kg)
    ref, mag = _rope64(qkv.view(-1, h_q + 2 * h_kv, D)[:, :h_q], qg, 1e-6, table,
                       plen + torch.cat([torch.arange(m, device="cuda") for m in new]), False)
    assert bool(((q.view(-1, h_q, D).double() - ref).abs() <= 24 * 2.0 ** -24 * mag + 1.001 * 2.0 ** -8 * ref.abs()).all())
    out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk[0], pv[0], plen_d, cu=cu)
    _check(out, new, [0] * batch, q, kc, vc, h_q, pk[0], pv[0], plen)
    n_acc = _i32([m - 1 for m in new])
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qs.kv_commit(lens, n_acc, l_max, work=work)
    assert qs.workspace_status(work) == BAD_INPUT          # the slot without a prompt is left as it was
    assert lens.tolist() == new
    at = list(new)
    for accepted in ([2, 0, 1], [0, 1, 2]):
        for j in range(gamma):                             # drafting: one token each
            qkv = _randn(g, batch, width, dtype=torch.float32)
            q = qs.qkv_rope_append(qkv, lens, j, kc, vc, h_q, table, prefix_len=plen_d, q_gamma=qg, k_gamma=kg)
            out = qs.attn_prefix(q, lens, j, kc, vc, h_q, pk[0], pv[0], plen_d)
            _check(out, [1] * batch, [x + j for x in at], q, kc, vc, h_q, pk[0], pv[0], plen)
        qkv = _randn(g, batch * (gamma + 1), width, dtype=torch.float32)      # verifying: gamma + 1 tokens each
        q = qs.qkv_rope_append(qkv, lens, 0, kc, vc, h_q, table, prefix_len=plen_d, q_gamma=qg, k_gamma=kg)
        out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk[0], pv[0], plen_d)
        _check(out, [gamma + 1] * batch, at, q, kc, vc, h_q, pk[0], pv[0], plen)
        qs.kv_commit(lens, _i32(accepted), l_max)
        at = [x + y + 1 for x, y in zip(at, accepted)]
        assert lens.tolist() == at


def test_many_sequences(qs):
    """More sequences than one warp, and than a CTA, looks after; most without tokens."""
    for batch, seed in ((70, 60), (1500, 61)):
        r = torch.Generator().manual_seed(seed)
        new = [int(x) if int(x) < 9 else 0 for x in torch.randint(0, 30, (batch,), generator=r)]
        old = [int(x) for x in torch.randint(0, 40, (batch,), generator=r)]
        h_q, h_kv = 2, 1
        q, kc, vc, cu, lens = _case(seed, new, old, h_q, h_kv)
        out = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
        _check(out, new, old, q, kc, vc, h_q)
        pk, pv = _prefix(seed, h_kv, 150)
        out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([150]), cu=cu)
        _check(out, new, old, q, kc, vc, h_q, pk, pv, 150)


def test_long_context_single_token(qs):
    """One token behind 300000 keys: many pieces of one item."""
    old, h_q, h_kv = [300000], 4, 2
    q, kc, vc, cu, lens = _case(62, [1], old, h_q, h_kv)
    out = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    _check(out, [1], old, q, kc, vc, h_q)
    pk, pv = _prefix(63, h_kv, 250000)
    out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([250000]))
    _check(out, [1], old, q, kc, vc, h_q, pk, pv, 250000)


def test_binding_refuses(qs):
    q, kc, vc, cu, lens = _case(64, [4, 5], [0, 3], 4, 2)
    for bad in (dict(cu=cu[:2]), dict(lens=lens[:1]), dict(q=q.float()), dict(q=q[:, :256]), dict(kc=kc.float()),
                dict(kc=kc[:, :, ::2]), dict(out=torch.empty(8, 512, dtype=torch.bfloat16, device="cuda")),
                dict(lens=lens.cpu()), dict(cu=cu.long()), dict(cu=None)):
        a = dict(q=q, cu=cu, lens=lens, kc=kc, vc=vc, out=None)
        a.update(bad)
        with pytest.raises(ValueError):
            qs.attn_prefill(a["q"], a["cu"], a["lens"], a["kc"], a["vc"], 4, out=a["out"])
    with pytest.raises(qs.QSpecError):
        qs.attn_prefill(q, cu, lens, kc, vc, 4, out=q)                        # over the queries
    with pytest.raises(qs.QSpecError):
        qs.attn_prefill(q, cu, lens, kc, vc, 4, work=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
