"""The prompt path as programs may call it: one token in place, on other streams, from threads, captured, with
starts that are out of order and values that are not finite."""
import math
import threading

import pytest
import torch

from test_gpu_prompt import D, _case, _check, _gen, _i32, _prefix, _randn, _table

pytestmark = pytest.mark.gpu

BAD_INPUT = 6


@pytest.fixture(scope="module")
def qs():
    from quantized_speculative_decoding_packed_b200 import qspec
    return qspec


@pytest.mark.parametrize("more", [0, 4])
def test_one_token_is_turned_in_place(qs, more):
    """A lone sequence drafting: one row of the projection, its queries turned where they lie."""
    g = _gen(1)
    h_q, h_kv, lens = 8, 2, _i32([40])
    qkv = _randn(g, 1, (h_q + 2 * h_kv) * D + more, dtype=torch.float32)
    kc, vc = _randn(g, 1, h_kv, 50, D), _randn(g, 1, h_kv, 50, D)
    ka, va, before, table = kc.clone(), vc.clone(), qkv.clone(), _table(qs, 128, 64)
    rows = qkv[:, :(h_q + 2 * h_kv) * D]
    apart = qs.qkv_rope_append(rows, lens, 0, ka, va, h_q, table,
                               q_out=torch.empty(1, h_q * D, dtype=torch.float32, device="cuda"))
    qs.qkv_rope_append(rows, lens, 0, kc, vc, h_q, table, q_out=qkv[:, :h_q * D])
    torch.cuda.synchronize()
    assert torch.equal(qkv[:, :h_q * D], apart) and torch.equal(qkv[:, h_q * D:], before[:, h_q * D:])
    assert torch.equal(kc, ka) and torch.equal(vc, va)
    out = qs.attn_prefill(apart.to(torch.bfloat16), _i32([0, 1]), lens, kc, vc, h_q)
    _check(out, [1], [40], apart.to(torch.bfloat16), kc, vc, h_q)


# ---------------------------------------------------------------- outputs on another stream
MS = 2_000_000        # about a millisecond of torch.cuda._sleep


def _outputs_of_every_call(qs):
    """name -> a call with a default output on `stream`; all inputs ready beforehand."""
    new, old, h_q, h_kv, plen = [40, 300, 7], [3, 0, 200], 8, 2, 500
    q, kc, vc, cu, lens = _case(2, new, old, h_q, h_kv)
    pk, pv = _prefix(3, h_kv, plen)
    plen_d = _i32([plen])
    g = _gen(4)
    qkv = _randn(g, sum(new), (h_q + 2 * h_kv) * D, dtype=torch.float32)
    ka, va = torch.zeros_like(kc), torch.zeros_like(vc)
    w = _randn(g, 512, 1024, dtype=torch.float32)
    wq, ws = qs.quantize_weights(w)
    x = _randn(g, 16, 1024)
    freq = 10000.0 ** (-torch.arange(64, dtype=torch.float64, device="cuda") / 64)
    table = qs.rope_table(freq, 600)
    size = {op: qs.workspace_size(op, 16, 512, 1024, 128) for op in (qs.OP_GEMM_W4A4, qs.OP_GEMM_W4A16)}
    work = torch.zeros(max(size.values()), dtype=torch.uint8, device="cuda")
    dec = torch.zeros(qs.attn_workspace_size(3, 1, h_q, h_kv, 300), dtype=torch.uint8, device="cuda")
    return {
        "qkv_rope_append": lambda s: qs.qkv_rope_append(qkv, lens, 0, ka, va, h_q, table, cu=cu, stream=s),
        "attn_prefill": lambda s: qs.attn_prefill(q, cu, lens, kc, vc, h_q, stream=s),
        "attn_prefix": lambda s: qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, plen_d, cu=cu, stream=s),
        "rope_table": lambda s: qs.rope_table(freq, 600, stream=s),
        "attn_decode": lambda s: qs.attn_decode(qkv[:3], lens, 0, kc, vc, h_q, 300, work=dec, stream=s),
        "gemm_w4a4": lambda s: qs.gemm_w4a4(x, wq, ws, work=work, stream=s),
        "gemm_w4a16": lambda s: qs.gemm_w4a16(x, wq, ws, work=work, stream=s),
        "cast_bf16": lambda s: qs.cast_bf16(w, stream=s),
    }


CALLS = ["qkv_rope_append", "attn_prefill", "attn_prefix", "rope_table", "attn_decode", "gemm_w4a4", "gemm_w4a16",
         "cast_bf16"]


@pytest.mark.parametrize("name", CALLS)
def test_default_output_is_memory_of_the_named_stream(qs, name):
    """What the current stream still has queued on memory that it freed does not reach an output of another
    stream; and what it reads of the output is not given away while it reads."""
    call = _outputs_of_every_call(qs)[name]
    want = call(None)
    side = torch.cuda.Stream()
    call(side)                                              # (its code is loaded)
    torch.cuda.synchronize()
    late = [torch.empty_like(want) for _ in range(3)]
    torch.cuda._sleep(20 * MS)
    for t in late:
        t.fill_(7)                                          # runs after the sleep ...
    del t, late                                             # ... in memory that is free from here on
    out = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    torch.cuda._sleep(20 * MS)
    got = out.clone()                                       # read after the sleep
    del out
    with torch.cuda.stream(side):
        fresh = [torch.full_like(want, 9) for _ in range(3)]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(fresh) == 3


# ---------------------------------------------------------------- default workspaces
@pytest.fixture
def fresh(qs, monkeypatch):
    """No default workspace from before; the buffers that the test's own thread gets."""
    buffers = qs._StreamBuffers()
    monkeypatch.setattr(qs, "_PROMPT_WS", buffers)
    return buffers


def test_threads_on_one_stream(qs, fresh):
    """Each thread's calls, an attention and a join each, interleave with the others' on the default stream."""
    plen, h_q, h_kv = 700, 8, 2
    pk, pv = _prefix(11, h_kv, plen)
    plen_d = _i32([plen])
    shapes = [([40, 300, 7], [900, 0, 200]), ([1] * 30, [50] * 30), ([600], [1500]), ([5] * 9, [300] * 9)]
    sets = [_case(12 + i, new, old, h_q, h_kv) for i, (new, old) in enumerate(shapes)]

    def both(a):
        q, kc, vc, cu, lens = a
        return (qs.attn_prefill(q, cu, lens, kc, vc, h_q),
                qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, plen_d, cu=cu))

    want = [both(a) for a in sets]
    for (new, old), a, w in zip(shapes, sets, want):
        _check(w[0], new, old, a[0], a[1], a[2], h_q)
        _check(w[1], new, old, a[0], a[1], a[2], h_q, pk, pv, plen)
    torch.cuda.synchronize()
    got, errors = [[] for _ in sets], []

    def run(i):
        try:
            torch.cuda.set_device(0)
            for _ in range(100):
                got[i].append(both(sets[i]))
        except Exception as e:                              # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, outs in enumerate(got):
        assert len(outs) == 100
        for o in outs:
            assert torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1]), i


def test_buffers_of_a_thread_end_with_it(qs, fresh):
    """Short-lived threads, each of which outgrows a buffer, leave none behind."""
    plen, h_q, h_kv = 100, 4, 2
    pk, pv = _prefix(26, h_kv, plen)
    plen_d = _i32([plen])
    sets = [_case(27 + i, [1] * n, [9] * n, h_q, h_kv) for i, n in enumerate((4, 400))]
    want = [qs.attn_prefix(c[0], c[4], 0, c[1], c[2], h_q, pk, pv, plen_d) for c in sets]
    torch.cuda.synchronize()
    same, held = [], []

    def run():
        torch.cuda.set_device(0)
        got = [qs.attn_prefix(c[0], c[4], 0, c[1], c[2], h_q, pk, pv, plen_d) for c in sets]
        torch.cuda.synchronize()
        same.append(all(torch.equal(x, y) for x, y in zip(got, want)))

    for _ in range(6):
        t = threading.Thread(target=run)
        t.start()
        t.join()
        held.append(torch.cuda.memory_allocated())
    assert same == [True] * 6 and held == held[:1] * 6


def test_default_stream_named_where_another_is_current(qs, fresh):
    q, kc, vc, cu, lens = _case(21, [40, 300], [900, 0], 8, 2)
    want = qs.attn_prefill(q, cu, lens, kc, vc, 8)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out = qs.attn_prefill(q, cu, lens, kc, vc, 8, stream=torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(out, want) and len(fresh.of) == 1


def test_workspace_that_is_outgrown_after_a_capture(qs, fresh):
    """A small call eagerly, then captured, then a large one: the eager buffer is replaced and kept, the graph's
    is its own, and the graph is right after others have taken what memory was free."""
    h_q, h_kv, plen = 4, 2, 100
    pk, pv = _prefix(22, h_kv, plen)
    plen_d = _i32([plen])
    small, big = _case(23, [1] * 4, [9] * 4, h_q, h_kv), _case(24, [1] * 400, [30] * 400, h_q, h_kv)
    call = lambda c: qs.attn_prefix(c[0], c[4], 0, c[1], c[2], h_q, pk, pv, plen_d)   # noqa: E731
    want = call(small)
    (key, first), = fresh.of.items()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(small)
    assert fresh.of[key] is first
    _check(call(big), [1] * 400, [30] * 400, big[0], big[1], big[2], h_q, pk, pv, plen)
    assert fresh.of[key].numel() > first.numel() and len(fresh.retired) == 1
    assert fresh.retired[0] is first
    fill = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(64)]
    for _ in range(3):
        out.zero_()
        graph.replay()
        eager = call(small)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(eager, want)
    assert all(bool((f == 255).all()) for f in fill)


def test_status_of_the_default_workspace(qs, fresh):
    """prompt_workspace is the buffer that calls without `work` report to; a captured call reports to its `work`."""
    q, kc, vc, cu, lens = _case(25, [20, 30], [0, 4], 4, 2)
    size = qs.attn_prefill_workspace_size()
    qs.attn_prefill(q, cu, lens, kc, vc, 4)
    ws = qs.prompt_workspace(size, "cuda")
    assert ws is qs.prompt_workspace(256, q.device) and qs.workspace_status(ws) == 0
    qs.attn_prefill(q, cu, lens - 1, kc, vc, 4)
    assert qs.workspace_status(ws) == BAD_INPUT and qs.workspace_status(ws) == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qs.attn_prefill(q, cu, lens - 1, kc, vc, 4, stream=side)
    side.synchronize()
    assert qs.workspace_status(ws) == 0
    assert qs.workspace_status(qs.prompt_workspace(size, "cuda", stream=side), stream=side) == BAD_INPUT
    work, wrong = torch.zeros(size, dtype=torch.uint8, device="cuda"), lens - 1
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qs.attn_prefill(q, cu, wrong, kc, vc, 4, work=work)
    assert qs.workspace_status(work) == 0
    graph.replay()
    assert qs.workspace_status(work) == BAD_INPUT and qs.workspace_status(ws) == 0


# ---------------------------------------------------------------- starts that do not fit
STARTS = [
    # starts of 3 sequences over 90 tokens; by sequence, tokens that are taken for it
    ([0, 20, 10, 90], {0: (0, 10)}),
    ([0, 20, 50, 91], {0: (0, 20), 1: (20, 50)}),
    ([-5, 20, 50, 90], {1: (20, 50), 2: (50, 90)}),
    ([0, 200, 50, 90], {}),
    ([3, 20, 50, 90], {0: (3, 20), 1: (20, 50), 2: (50, 90)}),
    ([0, 30, 30, 2 ** 31 - 1], {0: (0, 30)}),
]


@pytest.mark.parametrize("behind", [0, 60])
@pytest.mark.parametrize("starts,fit", STARTS)
def test_rope_append_reports_starts_that_do_not_fit(qs, starts, fit, behind):
    """The call reports them, and a sequence that fits has its tokens as ever; nothing lies below its length, and
    a sequence that does not fit writes nothing.  `behind`: that many more sequences, without tokens."""
    g = _gen(31)
    h_q, h_kv, n, l_max = 4, 2, 90, 300
    starts = starts + [starts[-1]] * behind
    batch = len(starts) - 1
    lens = _i32([7, 3, 11] + [0] * behind)
    qkv = _randn(g, n, (h_q + 2 * h_kv) * D, dtype=torch.float32)
    table = _table(qs, 128, 400)
    kc, vc = (torch.zeros(batch, h_kv, l_max, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.full((n, h_q * D), 9.0, dtype=torch.bfloat16, device="cuda")
    work = torch.zeros(256, dtype=torch.uint8, device="cuda")
    qs.qkv_rope_append(qkv, lens, 0, kc, vc, h_q, table, cu=_i32(starts), q_out=q, work=work)
    assert qs.workspace_status(work) == BAD_INPUT and qs.workspace_status(work) == 0
    for b, (first, last) in fit.items():
        one = [torch.zeros(1, h_kv, l_max, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        ref = qs.qkv_rope_append(qkv[first:last], lens[b:b + 1] + (first - starts[b]), 0, *one, h_q, table)
        assert torch.equal(q[first:last], ref), b
        at = slice(int(lens[b]) + first - starts[b], int(lens[b]) + last - starts[b])
        assert torch.equal(kc[b, :, at], one[0][0, :, at]) and torch.equal(vc[b, :, at], one[1][0, :, at])
    for b in range(3):
        fits = 0 <= starts[b] <= starts[b + 1] <= n
        assert not kc[b, :, :int(lens[b])].any() and not vc[b, :, :int(lens[b])].any()
        if not fits:
            assert not kc[b].any() and not vc[b].any()
    for i in range(n):
        if not any(0 <= starts[b] <= i < starts[b + 1] <= n for b in range(batch)):
            assert bool((q[i] == 9).all()), i


def test_rope_append_with_fitting_starts_reports_nothing(qs):
    g = _gen(32)
    for starts in ([0, 90], [0, 0, 40, 40, 90], [0] * 50 + [40, 40, 81], [0] * 300 + [7]):
        batch = len(starts) - 1
        qkv = _randn(g, 90, 3 * D, dtype=torch.float32)
        kc, vc = (torch.zeros(batch, 1, 100, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        work = torch.zeros(256, dtype=torch.uint8, device="cuda")
        q = qs.qkv_rope_append(qkv, _i32([4] * batch), 0, kc, vc, 1, None, cu=_i32(starts), work=work,
                               q_out=torch.full((90, D), 9.0, dtype=torch.bfloat16, device="cuda"))
        assert qs.workspace_status(work) == 0
        assert torch.equal(q[:starts[-1]], qkv[:starts[-1], :D].to(torch.bfloat16)) and bool((q[starts[-1]:] == 9).all())


@pytest.mark.parametrize("behind", [0, 40, 70])
@pytest.mark.parametrize("starts", [[0, 20, 10, 90], [0, 90, 0, 90], [0, 50, 49, 49], [-5, 60, 20, 300], [0, 20, 2 ** 31 - 1, 3]])
def test_attention_refuses_starts_out_of_order(qs, starts, behind):
    """Where starts fall a row could belong to two sequences: every row is zero, and the call is reported; the next
    call on the same workspace is as ever.  `behind`: that many more sequences without tokens."""
    new, old, h_q, h_kv, plen = [20, 30, 40], [500, 4, 8], 8, 2, 300
    q, kc, vc, cu, lens = _case(33, new + [0] * behind, old + [0] * behind, h_q, h_kv)
    pk, pv = _prefix(34, h_kv, plen)
    bad = _i32(starts + [starts[-1]] * behind)
    batch = 3 + behind

    def calls(cu, work, out):
        yield lambda: qs.attn_prefill(q, cu, lens, kc, vc, h_q, work=work, out=out)
        yield lambda: qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu, work=work, out=out)

    size = max(qs.attn_prefill_workspace_size(), qs.attn_prefix_workspace_size(90, batch, h_q, h_kv))
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for wrong, right, p in zip(calls(bad, work, out := torch.full_like(q, 3.0)), calls(cu, work, None), (0, plen)):
        out.fill_(3)
        wrong()
        assert qs.workspace_status(work) == BAD_INPUT and qs.workspace_status(work) == 0
        assert bool((out == 0).all())
        _check(right(), new + [0] * behind, old + [0] * behind, q, kc, vc, h_q, pk, pv, p)
        assert qs.workspace_status(work) == 0


def test_attention_refuses_starts_out_of_order_behind_a_prefix_taken_ahead(qs):
    new, old, h_q, h_kv, plen = [100, 130, 200], [500, 4, 8], 8, 2, 300
    q, kc, vc, cu, lens = _case(35, new, old, h_q, h_kv)
    pk, pv = _prefix(36, h_kv, plen)
    work = torch.zeros(qs.attn_prefix_workspace_size(430, 3, h_q, h_kv), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 3.0)
    qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=_i32([0, 300, 200, 430]), work=work, out=out)
    assert qs.workspace_status(work) == BAD_INPUT and bool((out == 0).all())
    qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu, work=work, out=out)
    assert qs.workspace_status(work) == 0
    _check(out, new, old, q, kc, vc, h_q, pk, pv, plen)


# ---------------------------------------------------------------- values that are not finite
def _all_kinds(qs, q, kc, vc, lens, new, h_q, pk, pv, plen):
    """(name, output) of each way that a batch can go: whole items, split ones, a prefix ahead and once."""
    cu = _i32([sum(new[:i]) for i in range(len(new) + 1)])
    yield "prefill", 0, qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    yield "prefix", plen, qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu)


NOT_FINITE = [
    # new, cached, h_q, h_kv, prefix: few items, shares, pieces, one row tile, two, prefix once and ahead
    ([5, 3], [30, 200], 4, 2, 40),
    ([200], [0], 4, 4, 300),
    ([3], [9000], 2, 1, 12000),
    ([1, 1, 1, 1], [5, 300, 2000, 128], 8, 8, 500),
    ([400, 300], [100, 0], 8, 2, 700),
    ([1] * 70, [33] * 70, 4, 2, 200),
]


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("new,old,h_q,h_kv,plen", NOT_FINITE)
def test_a_score_that_is_not_finite_makes_its_row_nan(qs, new, old, h_q, h_kv, plen, what):
    """softmax of scores with a NaN or +inf is NaN: for the rows that see the key, and for no others.  Keys at
    every place modulo 8 of a tile are tried (weights come from two kinds of exponentials)."""
    q, kc, vc, cu, lens = _case(51, new, old, h_q, h_kv)
    q = q.abs() + 0.125                                     # so that a key of +inf has a score of +inf
    pk, pv = _prefix(52, h_kv, plen)
    want = {name: out for name, _, out in _all_kinds(qs, q, kc, vc, lens, new, h_q, pk, pv, plen)}
    group, starts = h_q // h_kv, [sum(new[:i]) for i in range(len(new))]
    last = len(new) - 1
    for back in range(min(9, new[last] + old[last])):
        at = old[last] + new[last] - 1 - back               # a key of the last sequence's, of its last KV head
        kc[last, h_kv - 1, at, 7], kept = what, kc[last, h_kv - 1, at, 7].clone()
        for name, _, out in _all_kinds(qs, q, kc, vc, lens, new, h_q, pk, pv, plen):
            nan = torch.zeros_like(out, dtype=torch.bool)
            first = max(0, at - old[last])                  # the first token that sees it
            nan[starts[last] + first:, (h_q - group) * D:] = True
            assert torch.equal(out.isnan(), nan), (name, back)
            assert torch.equal(out[~nan], want[name][~nan]), (name, back)
        kc[last, h_kv - 1, at, 7] = kept
    for place in (0, plen // 2, plen - 1):                  # a key of the prefix: all rows of its heads
        pk[0, place, 3], kept = what, pk[0, place, 3].clone()
        out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu)
        assert bool(out[:, :group * D].isnan().all()), place
        assert torch.equal(out[:, group * D:], want["prefix"][:, group * D:])
        pk[0, place, 3] = kept


@pytest.mark.parametrize("new,old,h_q,h_kv,plen", NOT_FINITE)
def test_a_query_that_is_not_finite_makes_its_row_nan(qs, new, old, h_q, h_kv, plen):
    q, kc, vc, cu, lens = _case(53, new, old, h_q, h_kv)
    pk, pv = _prefix(54, h_kv, plen)
    want = {name: out for name, _, out in _all_kinds(qs, q, kc, vc, lens, new, h_q, pk, pv, plen)}
    for tok, head in ((0, 0), (sum(new) - 1, h_q - 1), (sum(new) // 2, h_q // 2)):
        bad = q.clone()
        bad[tok, head * D + 5] = float("nan")
        for name, _, out in _all_kinds(qs, bad, kc, vc, lens, new, h_q, pk, pv, plen):
            nan = torch.zeros_like(out, dtype=torch.bool)
            nan[tok, head * D:(head + 1) * D] = True
            assert torch.equal(out.isnan(), nan), (name, tok, head)
            assert torch.equal(out[~nan], want[name][~nan]), (name, tok, head)


def test_scores_of_minus_infinity_weigh_nothing(qs):
    """Keys whose score is -inf, alone and beside others: weight 0; a row with no other key is zero."""
    new, old, h_q, h_kv = [3], [300], 2, 1
    q, kc, vc, cu, lens = _case(55, new, old, h_q, h_kv)
    q = q.abs() + 0.125
    kc[0, 0, :100, 9] = -float("inf")
    out = qs.attn_prefill(q, cu, lens, kc, vc, h_q)
    _check(out, new, [200], q, kc[:, :, 100:], vc[:, :, 100:], h_q)
    kc[0, 0, :303, 9] = -float("inf")
    assert not qs.attn_prefill(q, cu, lens, kc, vc, h_q).any()


def test_values_behind_a_row_weigh_nothing(qs):
    """Values of 2^127 at positions that a row does not see, and at seen ones whose weight is 2^-220 or less of the
    largest (0 in fp32): the rows' outputs are those of the keys that weigh.  Every place modulo 8."""
    for new, old, h_q, h_kv, plen in (([24], [0], 2, 1, 50), ([24], [300], 2, 1, 130), ([150], [40], 4, 4, 10)):
        q, kc, vc, cu, lens = _case(56, new, old, h_q, h_kv)
        pk, pv = _prefix(57, h_kv, plen)
        m, o = new[0], old[0]
        late = m - 17                                       # the last 16 tokens and theirs alone are large
        kc[0, :, :o + m] *= 0.125
        clean = vc.clone()
        clean[0, :, o + late + 1:o + m] = 0
        for i in range(late + 1, m):
            vc[0, :, o + i] = 2.0 ** 127
        for name, p, out in _all_kinds(qs, q, kc, vc, lens, new, h_q, pk, pv, plen):
            ref = dict((n, x) for n, _, x in _all_kinds(qs, q, kc, clean, lens, new, h_q, pk, pv, plen))[name]
            assert torch.equal(out[:late + 1], ref[:late + 1]), (name, new)
            _check(ref[:late + 1], [late + 1], old, q[:late + 1], kc, clean, h_q, pk, pv, p)
    # keys that are seen, with scores 300 below the others (2^-432)
    q, kc, vc, cu, lens = _case(58, [20], [200], 2, 2)
    q[:, 0::D] = 64.0
    kc[0, :, :220, 0] = 0
    kc[0, :, :40, 0] = -53.0                                # -53 64 / sqrt(128) = -299.8
    clean = vc.clone()
    clean[0, :, :40] = 0
    vc[0, :, :40] = 2.0 ** 127
    out, ref = qs.attn_prefill(q, cu, lens, kc, vc, 2), qs.attn_prefill(q, cu, lens, kc, clean, 2)
    assert torch.equal(out, ref)
    _check(ref, [20], [200], q, kc, clean, 2)


@pytest.mark.parametrize("batch,h_q,h_kv", [(64, 32, 8), (3, 14, 2), (5, 8, 8), (2, 100, 1), (4, 200, 2)])
def test_prefix_workspace_size_over_token_counts(qs, batch, h_q, h_kv):
    """The documented rule: it falls at one number of tokens, and the size there or for the largest covers all."""
    each = -(-96 // (h_q // h_kv))                          # tokens a sequence from which the prefix goes ahead
    sizes = [qs.attn_prefix_workspace_size(n, batch, h_q, h_kv) for n in range(1, 4 * batch * each)]
    peak = batch * each - 1
    falls = [n for n in range(1, len(sizes)) if sizes[n] < sizes[n - 1]]
    assert falls == ([peak] if peak > 0 else []) and max(sizes) == (sizes[peak - 1] if peak > 0 else sizes[-1])
    assert min(sizes) >= qs.attn_prefill_workspace_size()


def test_one_workspace_for_all_token_counts(qs):
    """Calls on both sides of the fall on one buffer of the documented size; a smaller one is refused."""
    batch, h_q, h_kv, plen = 4, 8, 2, 200
    pk, pv = _prefix(61, h_kv, plen)
    size = qs.attn_prefix_workspace_size(batch * 24 - 1, batch, h_q, h_kv)
    assert size > qs.attn_prefix_workspace_size(batch * 24, batch, h_q, h_kv)
    work = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for new in ([24] * 4, [24, 24, 24, 23], [1] * 4, [40] * 4, [24, 24, 24, 23]):
        old = [30] * 4
        q, kc, vc, cu, lens = _case(62, new, old, h_q, h_kv)
        out = qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu, work=work)
        _check(out, new, old, q, kc, vc, h_q, pk, pv, plen)
    assert qs.workspace_status(work) == 0
    small = work[:qs.attn_prefix_workspace_size(batch * 24, batch, h_q, h_kv)]
    with pytest.raises(qs.QSpecError) as e:
        qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, _i32([plen]), cu=cu, work=small)
    assert e.value.status == 4


def test_prompts_with_an_empty_slot_are_committed(qs):
    """A batch in which one sequence has no tokens: the prompt calls report nothing, the commit without a workspace
    advances the others, and a sequence that does not fit is told by the prompt calls."""
    g = _gen(71)
    new, h_q, h_kv, l_max = [30, 0, 95], 8, 2, 200
    cu = _i32([0, 30, 30, 125])
    qkv = _randn(g, 125, (h_q + 2 * h_kv) * D, dtype=torch.float32)
    kc, vc = (torch.zeros(3, h_kv, l_max, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    work = torch.zeros(qs.attn_prefill_workspace_size(), dtype=torch.uint8, device="cuda")
    for old, status in (([0, 7, 20], 0), ([0, 7, 150], BAD_INPUT)):
        lens = _i32(old)
        q = qs.qkv_rope_append(qkv, lens, 0, kc, vc, h_q, None, cu=cu, work=work)
        assert qs.workspace_status(work) == status
        out = qs.attn_prefill(q, cu, lens, kc, vc, h_q, work=work)
        assert qs.workspace_status(work) == status
        fits = [m if o + m <= l_max else 0 for m, o in zip(new, old)]
        _check(out, fits, old, q, kc, vc, h_q)
        qs.kv_commit(lens, cu.diff() - 1, l_max)
        assert lens.tolist() == [o + m for o, m in zip(old, fits)]


def test_captured_default_outputs_on_a_forked_stream(qs, fresh):
    """Two calls at once in a graph, one on a forked stream, with outputs and workspaces of their own; the outputs
    are dropped and taken anew by a second graph."""
    new, old, h_q, h_kv = [300, 20], [500, 900], 8, 2
    runs = [_case(81 + i, new, old, h_q, h_kv) for i in range(2)]
    want = [qs.attn_prefill(q, cu, lens, kc, vc, h_q) for q, kc, vc, cu, lens in runs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            outs = [qs.attn_prefill(q, cu, lens, kc, vc, h_q, stream=s) for (q, kc, vc, cu, lens), s in zip(runs, (side, None))]
            main.wait_stream(side)
            sums = [o.float().sum() for o in outs]
        for _ in range(3):
            for o in outs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for o, s, ref in zip(outs, sums, want):
                assert torch.equal(o, ref) and torch.equal(s, ref.float().sum())
        del outs, sums, graph


@pytest.mark.parametrize("h_q,h_kv,rows,slots", [(8, 2, 200, 6), (4, 4, 700, 3), (32, 8, 60, 40), (14, 2, 90, 70)])
def test_one_graph_serves_batches_of_any_shape(qs, h_q, h_kv, rows, slots):
    """Captured once for so many rows and slots, replayed with other token counts (none at all, one long prompt, single
    tokens, empty slots), lengths and prefixes, on padded rows that hold NaN and stay as they were."""
    g = _gen(91)
    r = torch.Generator().manual_seed(92)
    l_max, p_max = rows + 900, 1500
    kc, vc = (_randn(g, slots, h_kv, l_max, D) for _ in range(2))
    pk, pv = (_randn(g, h_kv, p_max, D) for _ in range(2))
    q = torch.empty(rows, h_q * D, dtype=torch.bfloat16, device="cuda")
    cu, lens, plen = _i32([0] * (slots + 1)), _i32([0] * slots), _i32([0])
    out, behind = torch.empty_like(q), torch.empty_like(q)

    def calls(**kw):
        qs.attn_prefill(q, cu, lens, kc, vc, h_q, out=out, **kw)
        qs.attn_prefix(q, lens, 0, kc, vc, h_q, pk, pv, plen, cu=cu, out=behind, **kw)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    few = min(slots, rows)
    spread = torch.rand(slots, generator=r)
    shapes = [[0] * slots, [0] * (slots - 1) + [rows], [rows] + [0] * (slots - 1), [1] * few + [0] * (slots - few),
              [int(x) for x in spread / spread.sum() * rows], [min(3, rows // slots)] * slots]
    for i, new in enumerate(shapes):
        old = [int(x) for x in torch.randint(0, l_max - rows + 1, (slots,), generator=r)]
        p = (0, 1, p_max, 129, 640, 128)[i]
        n = sum(new)
        q.copy_(_randn(g, rows, h_q * D, scale=1.5))
        q[n:] = float("nan")
        cu.copy_(_i32([sum(new[:b]) for b in range(slots + 1)]))
        lens.copy_(_i32(old))
        plen.fill_(p)
        out.fill_(7)
        behind.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((out[n:] == 7).all()) and bool((behind[n:] == 7).all())
        if n:
            _check(out, new, old, q, kc, vc, h_q)
            _check(behind, new, old, q, kc, vc, h_q, pk, pv, p)
