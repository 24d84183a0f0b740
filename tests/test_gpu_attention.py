"""Linear attention on the GPU against its fp64 form (attention_harness), within the bounds
derived there, at the sizes where it can go wrong: sequences of no, one and few rows, ends
anywhere in a chunk, odd value dimensions, strided rows, inert slots, rows of no sequence."""
import pytest
import torch

import attention_harness as ah
import layer_harness as lh
import selective_state_update_ssu_amd as ssu
from test_gpu_layer import Draw, same

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# Lengths that meet every place in chunks of 32 and 64 rows and their tiles of 16.
LENGTHS = {
    "one": [1],
    "short": [0, 1, 2, 3, 0, 0, 17],
    "ends": [14, 33, 31, 1, 64, 65, 16],
    "long": [130, 0, 63, 200],
    "ones": [1] * 40,
}


def unit(t):
    f = t.float()
    return (f / f.norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(t.dtype)


def inputs(seed, lengths, H, G, K, V, io, st, delta, *, decay="row", lead=0, tail=0, idx=torch.int32,
           inert=(), strided=True, far=1.0, beta_io=False, extra=4):
    d = Draw(seed)
    cu = lh.starts(lengths, lead)
    rows = cu[-1] + tail
    wide = d.normal(rows, 2 * G * K + H * V + 3, io=io)
    q, k, v = (x.unflatten(1, (n, -1)) for x, n in (
        (wide[:, 3:3 + G * K], G), (wide[:, 3 + G * K:3 + 2 * G * K], G), (wide[:, 3 + 2 * G * K:], H)))
    if delta or not strided:
        q, k, v = unit(q).contiguous(), unit(k).contiguous(), v.contiguous() if not strided else v
    g = -far * d.uniform(0.0, 0.7, H) if decay == "head" else -far * d.uniform(0.0, 0.4, rows, H)
    beta = d.uniform(0.0, 1.0, rows, H) if delta else None
    if delta and beta_io:
        beta = beta.to(io)
    nslots = len(lengths) + extra
    return dict(q=q, k=k, v=v, decay=g, beta=beta, scale=K ** -0.5, cu=cu, idx=idx,
                state=(d.normal(nslots, H, V, K) * 0.3).to(st),
                slots=d.slots(len(lengths), nslots, idx, inert), has=d.flags(len(lengths)))


def dev(t):
    """t on the GPU with its strides: a view of a wider buffer stays one."""
    if t is None or t.is_contiguous():
        return None if t is None else t.to(DEV)
    wide = torch.full((t.shape[0], t.stride(0)), NAN, dtype=t.dtype, device=DEV)
    at = t.storage_offset() % t.stride(0)
    view = wide[:, at:at + t[0].numel()].unflatten(1, t.shape[1:])
    view.copy_(t)
    return view


def run(c, call, **more):
    state = c["state"].to(DEV)
    out = torch.full(c["v"].shape, NAN, dtype=c["v"].dtype, device=DEV)
    got = call(state, dev(c["q"]), dev(c["k"]), dev(c["v"]), c["decay"].to(DEV), out=out,
               beta=None if c["beta"] is None else c["beta"].to(DEV), scale=c["scale"], **more)
    assert got is out
    return out, state


def compare(name, c, out, state, ref):
    want, bound, written, after, s_bound, touched = ref
    lh.check(name + " out", out[written.to(DEV)], want[written], bound[written])
    assert out[~written.to(DEV)].isnan().all()
    lh.check(name + " state", state[touched.to(DEV)], after[touched], s_bound[touched])
    assert same(state[~touched.to(DEV)], c["state"][~touched])


def prompts(c, **more):
    out, state = run(c, ssu.linear_attention_varlen,
                     cu_seqlens=torch.tensor(c["cu"], dtype=c["idx"], device=DEV),
                     has_initial_state=c["has"].to(DEV), state_batch_indices=c["slots"].to(DEV), **more)
    begin, end = ah.in_place(c["cu"], c["slots"].tolist(), c["state"].shape[0], c["v"].shape[0])
    ref = ah.attention(c["q"], c["k"], c["v"], c["decay"], c["beta"], c["scale"], c["cu"], c["state"],
                       begin, end, c["has"].tolist())
    compare("prompts", c, out, state, ref)


SHAPES = [(4, 2, 64, 64), (2, 2, 128, 128), (3, 1, 8, 5), (2, 1, 80, 96), (2, 2, 256, 72),
          (1, 1, 136, 256), (6, 2, 16, 1)]


@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("H,G,K,V", SHAPES)
@pytest.mark.parametrize("lengths", ["short", "ends"])
def test_prompts(io, delta, H, G, K, V, lengths):
    n = LENGTHS[lengths]
    c = inputs(K + V, n, H, G, K, V, io, F32, delta, lead=2, tail=3, inert=(0, 3) if K == 64 else ())
    prompts(c)


@pytest.mark.parametrize("st", [F32, F16, BF16])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("lengths,decay,idx,strided,far", [
    ("one", "head", torch.int64, False, 1.0), ("long", "row", torch.int32, True, 1.0),
    ("ones", "head", torch.int32, False, 1.0), ("long", "head", torch.int64, False, 40.0),
    ("long", "row", torch.int32, False, 0.0)])
def test_prompts_states_and_decays(st, delta, lengths, decay, idx, strided, far):
    c = inputs(7, LENGTHS[lengths], 3, 3, 64, 40, BF16, st, delta, decay=decay, idx=idx,
               strided=strided, far=far, beta_io=True)
    prompts(c)


def test_prompts_forget_at_a_decay_of_minus_infinity():
    c = inputs(3, [70, 130], 2, 1, 64, 32, F32, F32, True)
    c["decay"][[0, 5, 69, 100, 133, 199]] = -float("inf")
    prompts(c)


def test_prompts_equal_keys_need_the_whole_inverse():
    """Keys that are all the same make every entry below the diagonal count."""
    c = inputs(4, [64, 200], 2, 1, 64, 32, F32, F32, True, decay="head", far=0.0)
    c["k"] = c["k"][:1].expand_as(c["k"]).contiguous()
    c["beta"] = torch.ones_like(c["beta"])
    prompts(c)


def test_prompts_slots_may_be_left_out():
    c = inputs(5, [10, 70, 0], 2, 2, 64, 64, BF16, F32, False)
    c["slots"] = torch.arange(3, dtype=torch.int32)
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)
    out, state = run(c, ssu.linear_attention_varlen, cu_seqlens=cu)
    begin, end = ah.in_place(c["cu"], None, c["state"].shape[0], c["v"].shape[0])
    ref = ah.attention(c["q"], c["k"], c["v"], c["decay"], None, c["scale"], c["cu"], c["state"], begin,
                       end, [False] * 3)
    compare("prompts", c, out, state, ref)


def test_prompts_bad_ranges_are_inert():
    c = inputs(6, [5, 6, 7], 2, 1, 64, 64, BF16, F32, True)
    for cu in ([7, 0, 11, 18], [0, 5, 11, 19], [-1, 5, 11, 18]):
        c["cu"] = cu
        prompts(c)


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("lengths,H,G,K,V,io,st", [
    ([1500], 2, 1, 64, 40, BF16, F32), ([900, 0, 257, 1, 700], 2, 2, 128, 72, F16, F32),
    ([1100], 1, 1, 256, 256, BF16, BF16), ([300, 1030], 1, 1, 200, 30, F32, F32)])
def test_prompts_cut_into_pieces(delta, lengths, H, G, K, V, io, st):
    """Few heads: sequences of more than 256 rows are cut. Sequences of one, two, three and more
    pieces, ends on a piece's end and one row behind it, inert slots among them."""
    c = inputs(len(lengths) + K, lengths, H, G, K, V, io, st, delta, lead=1, tail=2,
               inert=(1,) if len(lengths) > 2 else ())
    assert ssu.attention_workspace_bytes(c["v"].shape[0], len(lengths), H, K, V, delta) > 255
    prompts(c)


def test_delta_prompts_cut_at_their_longer_pieces():
    """With the delta rule pieces have at least 512 rows."""
    lengths = [512, 1025, 0, 1540, 1, 513]
    c = inputs(77, lengths, 1, 1, 64, 24, BF16, F32, True, lead=3, tail=1, inert=(3,))
    prompts(c)


@pytest.mark.parametrize("delta", [False, True])
def test_prompts_overlapping_ranges_stay_in_the_workspace(delta):
    """Not allowed, with results of no meaning, but nothing outside the workspace is touched: the
    ranges come to more pieces than there is room for."""
    rows, K, V = 2048, 64, 64
    c = inputs(31, [rows], 1, 1, K, V, BF16, F32, delta)
    cu = torch.tensor([0, rows, 0, rows, 0, rows], dtype=torch.int32, device=DEV)
    n = ssu.attention_workspace_bytes(rows, 5, 1, K, V, delta)
    ws = torch.full((n + (1 << 20),), 77, dtype=torch.uint8, device=DEV)
    state = torch.zeros(5, 1, V, K, device=DEV)
    q, k, v, decay = (c[x].to(DEV) for x in ("q", "k", "v", "decay"))
    ssu.linear_attention_varlen(state, q, k, v, decay, cu, workspace=ws,
                                beta=c["beta"].to(DEV) if delta else None)
    torch.cuda.synchronize()
    assert bool((ws[n:] == 77).all())


def test_prompts_workspace():
    c = inputs(30, [700, 400], 2, 1, 64, 64, BF16, F32, True)
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)
    n = ssu.attention_workspace_bytes(1100, 2, 2, 64, 64, True)
    a = run(c, ssu.linear_attention_varlen, cu_seqlens=cu)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    b = run(c, ssu.linear_attention_varlen, cu_seqlens=cu, workspace=ws)
    assert same(a[0], b[0]) and same(a[1], b[1])
    with pytest.raises(ValueError, match="workspace"):
        run(c, ssu.linear_attention_varlen, cu_seqlens=cu, workspace=ws[:-1])


def steps(c):
    out, state = run(c, ssu.linear_attention_update, state_batch_indices=c["slots"].to(DEV))
    rows = c["v"].shape[0]
    cu = list(range(rows + 1))
    begin, end = ah.in_place(cu, c["slots"].tolist(), c["state"].shape[0], rows)
    ref = ah.attention(c["q"], c["k"], c["v"], c["decay"], c["beta"], c["scale"], cu, c["state"], begin, end)
    compare("step", c, out, state, ref)


@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("st", [F32, F16, BF16])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("H,G,K,V", [(4, 2, 128, 128), (3, 1, 8, 5), (2, 1, 80, 33), (1, 1, 256, 256),
                                     (2, 2, 192, 1), (8, 1, 16, 17), (2, 2, 40, 64)])
def test_step(io, st, delta, H, G, K, V):
    c = inputs(K, [1] * 5, H, G, K, V, io, st, delta, decay="head" if K == 80 else "row", inert=(1, 3),
               idx=torch.int64 if K == 80 else torch.int32, strided=K != 128)
    steps(c)


@pytest.mark.parametrize("batch", [0, 1, 300])
def test_step_batches(batch):
    steps(inputs(1, [1] * batch, 2, 1, 64, 64, BF16, F32, True))


def windows(c, W, *, dst, accepted, d):
    nseq = len(c["cu"]) - 1
    nslots = c["state"].shape[0]
    table = torch.randperm(nslots, generator=d.g)[:nseq * W].to(torch.int32).view(nseq, W)
    if dst == "other":
        table = torch.randperm(nslots, generator=d.g)[:2 * nseq * W].to(torch.int32).view(2, nseq, W)
        table, to = table[0], table[1]
    else:
        to = table if dst == "same" else None
    if nseq > 2:
        table[2, 0] = -1
        if to is not None:
            to[1, W - 1] = nslots + 3
    na = torch.randint(1, W + 1, (nseq,), generator=d.g).to(torch.int32) if accepted else None
    if accepted and nseq > 3:
        na[3] = W + 1
    out, state = run(c, ssu.linear_attention_packed,
                     cu_seqlens=torch.tensor(c["cu"], dtype=torch.int32, device=DEV),
                     num_accepted_tokens=None if na is None else na.to(DEV),
                     state_batch_indices=table.to(DEV),
                     dst_state_batch_indices=None if to is None else to.to(DEV))
    begin, end = ah.through_tables(c["cu"], table.tolist(), None if to is None else to.tolist(),
                                   None if na is None else na.tolist(), nslots)
    ref = ah.attention(c["q"], c["k"], c["v"], c["decay"], c["beta"], c["scale"], c["cu"], c["state"],
                       begin, end)
    compare("windows", c, out, state, ref)


@pytest.mark.parametrize("io,st", [(BF16, F32), (F32, F16), (F16, BF16)])
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("dst,accepted", [("same", True), ("other", True), (None, False), ("other", False)])
@pytest.mark.parametrize("lengths", [[3, 0, 2, 4, 1, 4], [1], [6, 4, 1, 3]])
def test_windows(io, st, delta, dst, accepted, lengths):
    W, d = 4, Draw(11)
    c = inputs(9, lengths, 4, 2, 64, 40, io, st, delta, lead=1, tail=2, extra=2 * W * len(lengths))
    windows(c, W, dst=dst, accepted=accepted, d=d)


def test_windows_of_one_row_are_steps():
    """The same rows through both entry points, bit for bit."""
    c = inputs(2, [1] * 9, 4, 2, 128, 64, BF16, F32, True)
    a = run(c, ssu.linear_attention_update, state_batch_indices=c["slots"].to(DEV))
    b = run(c, ssu.linear_attention_packed, cu_seqlens=torch.arange(10, dtype=torch.int32, device=DEV),
            state_batch_indices=c["slots"].to(DEV))
    assert same(a[0], b[0]) and same(a[1], b[1])


def test_prompt_then_tokens_is_one_prompt():
    """A prompt's state carries on in single tokens as in the rest of the prompt."""
    c = inputs(8, [90], 2, 1, 64, 64, F32, F32, True)
    whole, after = run(c, ssu.linear_attention_varlen, cu_seqlens=torch.tensor([0, 90], device=DEV),
                       state_batch_indices=c["slots"].to(DEV))
    state, outs = c["state"].to(DEV), []
    args = [c[x].to(DEV) for x in ("q", "k", "v", "decay", "beta")]
    slots = c["slots"].to(DEV)

    def part(lo, hi):
        q, k, v, g, beta = (x[lo:hi].contiguous() for x in args)
        return q, k, v, g, dict(beta=beta, scale=c["scale"], state_batch_indices=slots)

    q, k, v, g, kw = part(0, 70)
    outs.append(ssu.linear_attention_varlen(state, q, k, v, g, torch.tensor([0, 70], device=DEV), **kw))
    for t in range(70, 90):
        q, k, v, g, kw = part(t, t + 1)
        outs.append(ssu.linear_attention_update(state, q, k, v, g, **kw))
    # Each side is within the bounds of the exact run; together they are within twice them.
    begin, end = ah.in_place(c["cu"], c["slots"].tolist(), c["state"].shape[0], 90)
    _, bound, _, _, s_bound, touched = ah.attention(c["q"], c["k"], c["v"], c["decay"], c["beta"],
                                                    c["scale"], c["cu"], c["state"], begin, end, [False])
    lh.check("out", torch.cat(outs), whole.double().cpu(), 2 * bound)
    lh.check("state", state[touched.to(DEV)], after.double().cpu()[touched], 2 * s_bound[touched])


@pytest.mark.parametrize("entry", ["prompts", "step"])
def test_captured_calls_follow_their_inputs(entry):
    c = inputs(12, [40, 600, 3] if entry == "prompts" else [1] * 6, 4, 2, 64, 64, BF16, F32, True)
    args = [c[x].to(DEV).contiguous() for x in ("q", "k", "v", "decay")]
    beta, slots = c["beta"].to(DEV), c["slots"].to(DEV)
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)

    def call(state):
        kw = dict(beta=beta, scale=c["scale"], state_batch_indices=slots)
        if entry == "prompts":
            return ssu.linear_attention_varlen(state, *args, cu, **kw)
        return ssu.linear_attention_update(state, *args, **kw)

    state = c["state"].to(DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(state.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(state)
    for i in range(3):
        args[2].copy_(torch.roll(args[2], 1 + i, 0))
        state.copy_(c["state"])
        graph.replay()
        torch.cuda.synchronize()
        want_state = c["state"].to(DEV)
        want = call(want_state)
        assert same(out, want) and same(state, want_state)


def test_another_stream():
    c = inputs(13, [40, 100, 3], 4, 2, 64, 64, BF16, F32, False)
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)
    a, sa = run(c, ssu.linear_attention_varlen, cu_seqlens=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b, sb = run(c, ssu.linear_attention_varlen, cu_seqlens=cu, stream=side)
    side.synchronize()
    assert same(a, b) and same(sa, sb)


def test_rows_far_apart():
    """Row offsets past 2^31 elements."""
    rows, stride = 70, 1 << 25
    c = inputs(14, [70], 1, 1, 64, 64, BF16, F32, False, strided=False)
    wide = torch.zeros((rows - 1) * stride + 64, dtype=BF16, device=DEV)
    v = wide.as_strided((rows, 1, 64), (stride, 64, 1))
    v.copy_(c["v"])
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)
    a = ssu.linear_attention_varlen(c["state"].to(DEV), c["q"].to(DEV), c["k"].to(DEV),
                                    c["v"].to(DEV), c["decay"].to(DEV), cu)
    b = ssu.linear_attention_varlen(c["state"].to(DEV), c["q"].to(DEV), c["k"].to(DEV), v,
                                    c["decay"].to(DEV), cu)
    assert same(a, b)
