"""Draft verification and batch tables on the GPU against their plain forms: whole numbers,
which have to be equal."""
import pytest
import torch

import attention_harness as ah
import layer_harness as lh
import selective_state_update_ssu_amd as ssu
from test_gpu_layer import Draw

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def case(seed, lengths, window, vocab, io, *, scores, draft, idx=torch.int32, lead=0, tail=0):
    d = Draw(seed)
    cu = lh.starts(lengths, lead)
    rows, B = cu[-1] + tail, len(lengths)
    score = d.normal(rows, vocab) * 2
    drafts = torch.zeros(B, window, dtype=idx)
    probs = torch.zeros(B, window, vocab)
    for b in range(B):
        for i in range(min(lengths[b] - 1, window)):
            probs[b, i] = torch.softmax(score[cu[b] + i] + d.normal(vocab) * 0.5, 0)
            drafts[b, i] = torch.multinomial(probs[b, i], 1, generator=d.g)[0]
    t = d.uniform(0.5, 1.5, B) if scores else None
    if scores and B > 1:
        t[::3] = 0.0
    return dict(target=(score if scores else torch.softmax(score, -1)).to(io), drafts=drafts,
                uniforms=d.uniform(0, 1, B, window + 1), cu=cu, idx=idx,
                probs=probs.to(io) if draft else None, temperature=t)


def run(c, **more):
    got = ssu.verify_drafts(c["target"].to(DEV), c["drafts"].to(DEV), c["uniforms"].to(DEV),
                            torch.tensor(c["cu"], dtype=c["idx"], device=DEV),
                            draft_probs=None if c["probs"] is None else c["probs"].to(DEV),
                            temperature=None if c["temperature"] is None else c["temperature"].to(DEV),
                            **more)
    return got


def check(c, **more):
    tokens, counts, slack = ah.verify(c["target"], c["drafts"], c["uniforms"], c["cu"], c["probs"],
                                      c["temperature"])
    # From scores, probabilities are off by 2^-37 at most (the exponential by 2.2e-12 in a weight and
    # in their sum, all else by some roundings of fp64): no decision here is that near its border.
    assert c["temperature"] is None or min(slack) > 2.0 ** -35
    got, n = run(c, **more)
    assert got.dtype == torch.int32 and n.dtype == torch.int32
    assert n.tolist() == counts
    assert got.tolist() == tokens


LENGTHS = {"one": [1], "mixed": [3, 1, 5, 2, 4, 5, 1], "empty": [0, 2, 0, 0, 5, 1], "long": [6, 2, 7, 5]}


@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("scores", [False, True])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("lengths", sorted(LENGTHS))
@pytest.mark.parametrize("vocab", [1, 7, 1000, 8193, 20001])
def test_verify(io, scores, draft, lengths, vocab):
    check(case(vocab, LENGTHS[lengths], 4, vocab, io, scores=scores, draft=draft, lead=1, tail=2,
               idx=torch.int64 if vocab == 1000 else torch.int32))


@pytest.mark.parametrize("scores", [False, True])
def test_verify_without_a_window(scores):
    """No drafts: a token is drawn for every sequence."""
    check(case(1, [1] * 9, 0, 500, F32, scores=scores, draft=False))


@pytest.mark.parametrize("io,vocab", [(F32, 300001), (BF16, 600007)])
@pytest.mark.parametrize("scores", [False, True])
def test_verify_large_vocabularies(io, vocab, scores):
    """More tiles of a row than a wave has lanes."""
    check(case(3, [2, 1, 3], 2, vocab, io, scores=scores, draft=True))


def test_verify_many_drafts():
    """More drafts than a wave has lanes, all of which stand."""
    c = case(2, [151], 150, 40, F32, scores=False, draft=True)
    c["target"] = torch.cat([c["probs"][0], c["target"][-1:]])
    check(c)
    assert run(c)[1].tolist() == [151]


@pytest.mark.parametrize("u", [0.0, 0.25, 0.5, 1.0 - 2.0 ** -24])
def test_verify_borders_of_the_drawn_number(u):
    """Weights whose sums are exact: a drawn number on a border belongs to the token above it, and
    tokens without weight are never drawn."""
    p = torch.tensor([[0.0, 0.25, 0.0, 0.25, 0.5, 0.0]])
    c = dict(target=p, drafts=torch.zeros(1, 0, dtype=torch.int32), uniforms=torch.tensor([[u]]),
             cu=[0, 1], idx=torch.int32, probs=None, temperature=None)
    check(c)
    assert run(c)[0].tolist() == [[{0.0: 1, 0.25: 3, 0.5: 4}.get(u, 4)]]


def test_verify_takes_equal_distributions():
    """p = q: every draft stands, whatever is drawn; also where u q rounds to p."""
    c = case(3, [5] * 6, 4, 300, F32, scores=False, draft=True)
    for b in range(6):
        c["target"][c["cu"][b]:c["cu"][b] + 4] = c["probs"][b]
    c["uniforms"][:, :4] = 1.0 - 2.0 ** -24
    check(c)
    assert run(c)[1].tolist() == [5] * 6


def test_verify_nothing_left_of_p():
    """A rejected draft with p <= q everywhere: the token comes from p."""
    c = case(4, [2, 2], 1, 50, F32, scores=False, draft=True)
    c["target"][[0, 2]] = c["probs"][:, 0] * 0.5
    c["uniforms"][:, 0] = 0.75
    check(c)
    assert run(c)[1].tolist() == [1, 1]


def test_verify_greedy_ties_and_masked_scores():
    score = torch.tensor([[1.0, 3.0, 3.0, -INF], [-INF, -INF, -INF, -INF], [NAN, 2.0, NAN, 2.0],
                          [INF, 0.0, INF, 1.0]])
    cu = [0, 1, 2, 3, 4]
    for t, want in ((0.0, [[1], [0], [1], [0]]), (0.7, [[1], [-1], [1], [0]])):
        c = dict(target=score, drafts=torch.zeros(4, 0, dtype=torch.int32),
                 uniforms=torch.full((4, 1), 0.2), cu=cu, idx=torch.int32, probs=None,
                 temperature=torch.full((4,), t))
        check(c)
        assert run(c)[0].tolist() == want


def test_verify_very_small_temperature():
    c = case(5, [4, 1, 3], 3, 777, F32, scores=True, draft=True)
    c["temperature"][:] = torch.tensor([1e-30, 1e-6, 1e-38])
    check(c)


def test_verify_values_that_are_no_probabilities():
    c = case(6, [3, 2, 3], 2, 64, F32, scores=False, draft=True)
    c["target"][:, 10:20] = torch.tensor([NAN, -1.0] * 5)
    c["probs"][:, :, 30:40] = NAN
    c["drafts"][0, 0] = 11
    c["drafts"][1, 0] = 33
    c["drafts"][2, 0] = -5
    check(c)
    c["drafts"][2, 0] = 64
    check(c)
    c["target"][:] = 0.0
    check(c)
    assert run(c)[0][:, 0].tolist() == [-1, -1, -1]


def test_verify_bad_ranges():
    c = case(7, [3, 2, 4], 3, 64, F32, scores=True, draft=True)
    for cu in ([0, 3, 2, 9], [0, 3, 5, 10], [-1, 3, 5, 9], [0, 5, 5, 9]):
        c["cu"] = cu
        tokens, counts, _ = ah.verify(c["target"], c["drafts"], c["uniforms"], cu, c["probs"],
                                      c["temperature"])
        got, n = run(c)
        # Where the starts run backwards no row belongs to one sequence alone; what is inert stays so.
        for b in range(3):
            if counts[b] == 0:
                assert n[b] == 0 and got[b].tolist() == tokens[b]


def test_verify_strides():
    """Drafts and their distributions step-major, target columns of a wider buffer."""
    c = case(8, LENGTHS["mixed"], 4, 1001, BF16, scores=True, draft=True)
    tokens, counts, _ = ah.verify(c["target"], c["drafts"], c["uniforms"], c["cu"], c["probs"],
                                  c["temperature"])
    wide = torch.full((c["target"].shape[0], 1017), NAN, dtype=BF16, device=DEV)
    wide[:, 5:1006] = c["target"].to(DEV)
    got, n = ssu.verify_drafts(
        wide[:, 5:1006], c["drafts"].t().contiguous().to(DEV).t(), c["uniforms"].to(DEV),
        torch.tensor(c["cu"], device=DEV),
        draft_probs=c["probs"].transpose(0, 1).contiguous().to(DEV).transpose(0, 1),
        temperature=c["temperature"].to(DEV))
    assert n.tolist() == counts and got.tolist() == tokens


def test_verify_captured():
    c = case(9, LENGTHS["mixed"], 4, 5000, F32, scores=True, draft=True)
    dev = {k: c[k].to(DEV) for k in ("target", "drafts", "uniforms", "probs", "temperature")}
    cu = torch.tensor(c["cu"], device=DEV)

    def call():
        return ssu.verify_drafts(dev["target"], dev["drafts"], dev["uniforms"], cu,
                                 draft_probs=dev["probs"], temperature=dev["temperature"])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, n = call()
    for i in range(3):
        dev["uniforms"].copy_(torch.roll(dev["uniforms"], 1, 0))
        graph.replay()
        torch.cuda.synchronize()
        want, m = call()
        assert torch.equal(got, want) and torch.equal(n, m)


# -------------------------------------------------------------------------- plans

def plan(lengths, rows, chunk=None, nchunks=None, context=None, table=None, block=1, idx=torch.int32):
    def whole(x, dtype=idx):
        return None if x is None else torch.tensor(x, dtype=dtype, device=DEV)

    got = ssu.batch_plan(torch.tensor(lengths, dtype=idx, device=DEV), rows, chunk_size=chunk,
                         nchunks=nchunks, context_lens=whole(context), block_table=whole(table),
                         block_size=block)
    most = nchunks if nchunks is not None else rows // chunk + len(lengths) if chunk else 0
    want = ah.plan(lengths, rows, chunk, most, context, table, block)
    for name, t in got._asdict().items():
        if name not in want:
            assert t is None, name
            continue
        assert t.dtype == (torch.int64 if name == "row_slots" else torch.int32)
        assert t.tolist() == want[name], name


@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
@pytest.mark.parametrize("chunk", [None, 1, 16, 128])
@pytest.mark.parametrize("lengths", [[], [0], [5], [0, 7, 0, 0, 16, 17, 1, 0], [-3, 4, -1, 300],
                                     [1] * 1500, [3, 0] * 1030, [5000, 1, 4096]])
def test_plan(idx, chunk, lengths):
    rows = sum(max(n, 0) for n in lengths) + 3
    g = torch.Generator().manual_seed(len(lengths))
    context = torch.randint(0, 50, (len(lengths),), generator=g).tolist() or None
    table = torch.randint(-1, 900, (len(lengths), 6), generator=g).tolist() or None
    plan(lengths, rows, chunk, idx=idx)
    plan(lengths, rows, chunk, context=context, table=table, block=16, idx=idx)


@pytest.mark.parametrize("n", [4095, 4096, 4097, 9000])
def test_plan_of_many_requests(n):
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(-1, 6, (n,), generator=g).tolist()
    plan(lengths, sum(max(x, 0) for x in lengths) + 5, 2)
    plan(lengths, n, 4)


def test_plan_tables_are_tensors_of_their_own():
    """Tables share an allocation, and nothing else: writing one leaves the others."""
    got = ssu.batch_plan(torch.tensor([3, 0, 4], device=DEV), 9, chunk_size=2,
                         block_table=torch.zeros(3, 9, dtype=torch.int32, device=DEV))
    before = [t.clone() for t in got]
    for i, t in enumerate(got):
        assert t.is_contiguous() and not t.requires_grad
        t.fill_(-7)
        for j, other in enumerate(got):
            assert torch.equal(other, before[j]) == (i != j)
        t.copy_(before[i])


def test_plan_lengths_that_pass_the_rows():
    plan([10, 20, 30], 25, 8)
    plan([10, 20, 30], 25, 8, nchunks=3)
    plan([10, 20], 30, 8, nchunks=0)
    plan([10, 0, 20], 0, 8)


def test_plan_negative_positions():
    plan([4, 5], 12, context=[-2, 3], table=[[7, 8], [9, 1]], block=2)


def test_plan_of_a_strided_table():
    wide = torch.arange(60, dtype=torch.int32, device=DEV).view(3, 20)
    got = ssu.batch_plan(torch.tensor([3, 1, 5], device=DEV), 9, block_table=wide[:, 4:9])
    assert got.row_slots.tolist() == [4, 5, 6, 24, 44, 45, 46, 47, 48]


def test_plan_captured_follows_the_lengths():
    lengths = torch.tensor([5, 9, 0, 2], dtype=torch.int32, device=DEV)
    ssu.batch_plan(lengths, 40, chunk_size=4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ssu.batch_plan(lengths, 40, chunk_size=4)
    for n in ([5, 9, 0, 2], [1, 1, 1, 1], [30, 0, 0, 10]):
        lengths.copy_(torch.tensor(n, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = ah.plan(n, 40, 4, 14, None, None, 1)
        for name in want:
            assert getattr(got, name).tolist() == want[name], name


def test_prefill_on_planned_tables():
    """The prefill on tables built on the GPU, with chunks to spare and a request without rows, is
    that on the host's tables; the empty request's state comes back as it went in."""
    lengths, H, P, N, chunk = [300, 0, 70, 128], 2, 64, 64, 128
    d, T = Draw(21), sum(lengths)
    x, B, C = d.normal(T, H, P, io=BF16), d.normal(T, 1, N, io=BF16), d.normal(T, 1, N, io=BF16)
    x, B, C = x.to(DEV), B.to(DEV), C.to(DEV)
    dt, A = d.uniform(0.01, 0.1, T, H).to(DEV), -d.uniform(0.5, 4, H).to(DEV)
    init = d.normal(4, H, P, N).to(DEV)
    got = ssu.batch_plan(torch.tensor(lengths, device=DEV), T, chunk_size=chunk)
    out = torch.empty_like(x)
    states = ssu.ssd_combined_fwd_varlen(x, dt, A, B, C, chunk, got.cu_seqlens, got.cu_chunk_seqlens,
                                         got.last_chunk_indices, got.seq_idx, out=out,
                                         initial_states=init)
    i32 = dict(dtype=torch.int32, device=DEV)
    want_out = torch.empty_like(x)
    keep = [0, 2, 3]
    want = ssu.ssd_combined_fwd_varlen(
        x, dt, A, B, C, chunk, torch.tensor([0, 300, 370, 498], **i32),
        torch.tensor([0, 128, 256, 300, 370, 498], **i32), torch.tensor([2, 3, 4], **i32),
        torch.tensor([0, 0, 0, 1, 2], **i32), out=want_out, initial_states=init[keep].contiguous())
    assert torch.equal(out, want_out)
    assert torch.equal(states[keep], want)
    assert torch.equal(states[1], init[1])


def test_drafts_verified_and_continued():
    """Two speculative steps as an engine runs them: the tables of the packed rows, linear
    attention and the state update over the window, verification, and the next window from
    the states that stand; the states are those of the accepted tokens alone."""
    B, W, H, K, V, vocab = 3, 4, 2, 64, 64, 200
    d = Draw(31)
    slots = B * W
    refcount = torch.zeros(slots, dtype=torch.int32, device=DEV)
    table = ssu.cache_alloc(refcount, slots).view(B, W)
    attn = (d.normal(slots, H, V, K) * 0.3).to(DEV)
    scan = (d.normal(slots, H, V, K) * 0.3).to(DEV)
    alone_attn, alone_scan = attn[table[:, 0].long()].clone(), scan[table[:, 0].long()].clone()
    accepted = torch.ones(B, dtype=torch.int32, device=DEV)
    g = -d.uniform(0.01, 0.3, H).to(DEV)
    A, ones = -d.uniform(0.5, 2, H).to(DEV), torch.arange(B, dtype=torch.int32, device=DEV)
    for step, lengths in enumerate(([4, 1, 3], [2, 4, 4])):
        p = ssu.batch_plan(torch.tensor(lengths, dtype=torch.int32, device=DEV), sum(lengths))
        rows = sum(lengths)
        q, k, v, x = (d.normal(rows, H, 64, io=BF16).to(DEV) for _ in range(4))
        k = unit_rows(k)
        beta, dt = d.uniform(0, 1, rows, H).to(DEV), d.uniform(0.01, 0.1, rows, H).to(DEV)
        ssu.linear_attention_packed(attn, q, k, v, g, p.cu_seqlens, beta=beta,
                                    num_accepted_tokens=accepted, state_batch_indices=table,
                                    dst_state_batch_indices=table)
        ssu.ssu_packed_varlen(scan, x, dt, A, q, k, p.cu_seqlens, num_accepted_tokens=accepted,
                              state_batch_indices=table, dst_state_batch_indices=table)
        scores = (d.normal(rows, vocab) * 2).to(DEV)
        drafts = torch.zeros(B, W - 1, dtype=torch.int32, device=DEV)
        for b in range(B):  # the best token, which a greedy target accepts, but for one
            n = lengths[b] - 1
            drafts[b, :n] = scores[int(p.cu_seqlens[b]):int(p.cu_seqlens[b]) + n].argmax(-1)
        if step == 0:
            drafts[0, 1] = (drafts[0, 1] + 1) % vocab
        tokens, accepted = ssu.verify_drafts(scores, drafts, torch.rand(B, W, device=DEV), p.cu_seqlens,
                                             temperature=torch.zeros(B, device=DEV))
        assert accepted.tolist() == ([2, 1, 3] if step == 0 else [2, 4, 4])
        # The accepted rows, one at a time.
        for t in range(W):
            on = [b for b in range(B) if t < int(accepted[b])]
            at = [int(p.cu_seqlens[b]) + t for b in on]
            assert all(int(tokens[b, t]) == int(scores[a].argmax()) for b, a in zip(on, at))
            ssu.linear_attention_update(alone_attn, q[at], k[at], v[at], g, beta=beta[at],
                                        state_batch_indices=ones[on])
            ssu.ssu_one_token(alone_scan, x[at], dt[at], A, q[at], k[at], state_batch_indices=ones[on])
        last = table.gather(1, accepted.long()[:, None] - 1)[:, 0].long()
        assert torch.equal(attn[last], alone_attn)
        # The update's two kernels sum in another order (a few roundings of the state).
        torch.testing.assert_close(scan[last], alone_scan, rtol=1e-5, atol=1e-5)


def unit_rows(t):
    f = t.float()
    return (f / f.norm(dim=-1, keepdim=True)).to(t.dtype)
