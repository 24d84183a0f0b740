"""Prompts cut into pieces in calls of more workgroups than the card holds at once: the first
piece of a sequence may start after its last one has ended, in one launch. On the CPU a
model of the launch's order shows that the shape tested here has such sequences; on the GPU the
call is compared with the fp64 form, and with itself."""
import heapq

import pytest
import torch

import attention_harness as ah
import layer_harness as lh
import selective_state_update_ssu_amd as ssu
from layer_harness import TINY, U
from test_gpu_layer import Draw, same

DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
HEADS, DIM, SEQUENCES, SLICES = 20, 64, 24, 1


def lengths():
    """Uneven ones: ends anywhere in a piece, short ones between long ones."""
    g = torch.Generator().manual_seed(5)
    n = torch.randint(100, 1300, (SEQUENCES,), generator=g)
    n[::5] = torch.randint(1, 40, (len(n[::5]),), generator=g)
    return n.tolist()


# ------------------------------------------------------------- the order of a launch

def order(item_count, per_piece, xcds=8):
    """Items of every XCD in the order in which it starts them."""
    share = per_piece // xcds
    if per_piece % xcds == 0:
        def item(xcd, k):
            return (k // share) * per_piece + xcd * share + k % share
    else:
        per, tall = -(-item_count // xcds), item_count % xcds or xcds

        def item(xcd, k):
            return xcd * per + k if xcd < tall else tall * per + (xcd - tall) * (per - 1) + k
    return [[item(x, k) for k in range((item_count - x + xcds - 1) // xcds)] for x in range(xcds)]


def inverted(piece, resident):
    """First pieces that start after their sequence's last one has ended, where a
    workgroup takes as long as its piece has rows and an XCD holds `resident` of them."""
    rows, first, last = [], [], []
    for n in lengths():
        count = -(-n // piece)
        for j in range(count):
            rows.append(min(piece, n - j * piece))
            first.append(len(first) - j)
            last.append(j + 1 == count)
    most = sum(lengths()) // piece + SEQUENCES  # pieces of the launch, the spare ones empty
    per_piece = HEADS * SLICES
    begin, end = {}, {}
    for items in order(most * per_piece, per_piece):
        free = [0.0] * resident
        for i in items:
            p, head = divmod(i, per_piece)
            at = heapq.heappop(free)
            length = rows[p] if p < len(rows) else 0
            begin[p, head], end[p, head] = at, at + length
            heapq.heappush(free, at + length)
    return sum(begin[first[p], h] >= end[p, h] for p in range(len(rows)) for h in range(per_piece)
               if last[p] and first[p] != p)


@pytest.mark.parametrize("delta,piece", [(False, 256), (True, 512)])
def test_the_shape_has_sequences_whose_last_piece_ends_first(delta, piece):
    """So nothing of a launch may read what a last piece writes. (fp32 rows: two workgroups of a
    compute unit, 64 of an XCD.)"""
    each = HEADS * SLICES
    assert SEQUENCES * each < 512  # else nothing is cut
    assert -(-sum(lengths()) * each // 1024) <= piece  # the shortest piece that a call has
    assert inverted(piece, 64) > 0


def touched(launch, j, count):
    """(places read, places written) by the workgroup of piece j of a continued sequence of `count`
    pieces: its slot, and the pieces' places in the workspace."""
    last = j + 1 == count
    if launch == "ends":
        if count == 1:
            return set(), set()
        return {"slot"} if j == 0 or last else set(), {j}
    if launch == "out":
        enters = "slot" if count == 1 else count - 1 if j == 0 else j - 1
        return {enters}, {"slot"} if last else set()


@pytest.mark.parametrize("count", range(1, 8))
def test_no_piece_reads_what_another_of_its_launch_writes(count):
    holds = {"slot": "entering"}  # what a place has, by the launches that ran
    for launch in ("ends", "out"):
        pieces = [touched(launch, j, count) for j in range(count)]
        for i, (read, _) in enumerate(pieces):
            for j, (_, written) in enumerate(pieces):
                assert i == j or not read & written, (launch, i, j)
        if launch == "ends":
            assert all("slot" not in written for _, written in pieces)
            holds.update({j: "entering" if j + 1 == count else f"after {j}" for j in range(count) if count > 1})
        else:
            for j, (read, _) in enumerate(pieces):
                assert [holds[x] for x in read] == ["entering" if j == 0 else f"after {j - 1}"]


# ------------------------------------------------------------------------- the GPU

def problem(delta, io, st):
    d, rows = Draw(41), sum(lengths())
    unit = lambda t: (t.float() / t.float().norm(dim=-1, keepdim=True)).to(t.dtype)  # noqa: E731
    q, k, v = (d.normal(rows, n, DIM, io=io) for n in (HEADS // 2, HEADS // 2, HEADS))
    # Decays so weak that the entering state is felt in every row.
    return dict(q=unit(q), k=unit(k), v=v, decay=-d.uniform(0.0, 2e-3, rows, HEADS),
                beta=d.uniform(0.0, 1.0, rows, HEADS) if delta else None, scale=DIM ** -0.5,
                cu=lh.starts(lengths()), state=(d.normal(SEQUENCES + 3, HEADS, DIM, DIM) * 3).to(st),
                slots=d.slots(SEQUENCES, SEQUENCES + 3))


def on_gpu(c):
    return {name: x.to(DEV) if isinstance(x, torch.Tensor) else x for name, x in c.items()}


def call(g):
    state = g["state"].clone()
    out = ssu.linear_attention_varlen(
        state, g["q"], g["k"], g["v"], g["decay"], torch.tensor(g["cu"], dtype=torch.int32, device=DEV),
        beta=g["beta"], scale=g["scale"], state_batch_indices=g["slots"],
        has_initial_state=torch.ones(SEQUENCES, dtype=torch.bool, device=DEV))
    return out, state


def definition(g):
    """attention_harness.attention's recurrence of values and bounds, all sequences at a time."""
    io, st, K = g["v"].dtype, g["state"].dtype, DIM
    q, k, v, decay = (g[x].double() for x in ("q", "k", "v", "decay"))
    cu = torch.tensor(g["cu"], device=DEV)
    begin, length = cu[:-1], cu[1:] - cu[:-1]
    per = HEADS // q.shape[1]
    S = g["state"][g["slots"].long()].double()
    N, E = S.norm(dim=-1), torch.zeros(SEQUENCES, HEADS, DIM, dtype=torch.float64, device=DEV)
    far = torch.stack([ah.window_decay(decay, g["cu"][b], g["cu"][b + 1]) for b in range(SEQUENCES)])
    c = ((K + 200 + 3 * far) * U)[..., None]
    more = 0.0 if io == F32 else 256 * U
    out, bound = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(int(length.max())):
        on = (t < length).nonzero()[:, 0]
        at = begin[on] + t
        kt, qt = k[at].repeat_interleave(per, 1), q[at].repeat_interleave(per, 1)
        kn, qn = kt.norm(dim=-1)[..., None], qt.norm(dim=-1)[..., None]
        e = torch.exp(decay[at])[..., None]
        now, n = S[on] * e[..., None], N[on]
        r, be = v[at], 0.0
        if g["beta"] is not None:
            be = g["beta"][at].double()[..., None]
            r = be * (r - (now * kt[:, :, None]).sum(-1))
        now = now + r[..., None] * kt[:, :, None]
        local = e * n + r.abs() * kn + be * kn * (v[at].abs() + kn * e * n)
        S[on], N[on], E[on] = now, e * n + r.abs() * kn, e * E[on] + c[on] * local
        y = g["scale"] * (now * qt[:, :, None]).sum(-1)
        out[at] = y
        bound[at] = lh.stored(abs(g["scale"]) * qn * (E[on] + (c[on] + more) * N[on]), y, io)
    return out.cpu(), bound.cpu() + TINY[io], S.cpu(), lh.stored(E[..., None].expand_as(S), S, st).cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("io,st", [(F32, F32), (BF16, F32), (F16, BF16)])
def test_continued_prompts_in_many_pieces(delta, io, st):
    g = on_gpu(problem(delta, io, st))
    want, bound, after, s_bound = definition(g)
    for _ in range(3):
        out, state = call(g)
        lh.check("out", out, want, bound)
        lh.check("state", state[g["slots"].long()], after, s_bound)
        rest = torch.ones(SEQUENCES + 3, dtype=torch.bool, device=DEV)
        rest[g["slots"].long()] = False
        assert same(state[rest], g["state"][rest])


@pytest.mark.gpu
@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("K,V,heads,nseq,most", [
    (64, 64, 20, 24, 1300), (128, 128, 32, 16, 2000), (256, 256, 3, 9, 1500), (128, 128, 32, 3, 90)])
def test_the_same_call_gives_the_same_bits(delta, io, K, V, heads, nseq, most):
    """Cut and uncut calls, more workgroups than the card holds and fewer."""
    d = Draw(K + heads)
    cu = lh.starts(torch.randint(1, most, (nseq,), generator=d.g).tolist())
    rows = cu[-1]
    q, k = (torch.nn.functional.normalize(d.normal(rows, heads, K, io=io).to(DEV).float(), dim=-1).to(io)
            for _ in range(2))
    v, decay = d.normal(rows, heads, V, io=io).to(DEV), -d.uniform(0.0, 0.1, rows, heads).to(DEV)
    beta = d.uniform(0.0, 1.0, rows, heads).to(DEV) if delta else None
    start = d.normal(nseq, heads, V, K).to(DEV)
    has = torch.ones(nseq, dtype=torch.bool, device=DEV)
    starts = torch.tensor(cu, dtype=torch.int32, device=DEV)
    found = None
    for _ in range(8):
        state = start.clone()
        out = ssu.linear_attention_varlen(state, q, k, v, decay, starts, beta=beta, scale=K ** -0.5,
                                          has_initial_state=has)
        if found is None:
            found = out, state
        assert same(out, found[0]) and same(state, found[1])


@pytest.mark.gpu
def test_decays_of_long_pieces():
    """Without values a state is its entering one times a decay, through 12 pieces of 960 rows and one
    of a single row. Its error: 30 chunks of the first piece, each an exponential (one step of fp32,
    2^-23, which also covers the half step of its small argument) and a product (half a step); for each
    of 11 pieces an exponential (a step), its correction, and the product and sum that join (half a
    step each), 2.5 steps; the last chunk like one of the first; half a step when the state is stored,
    which is fp32 anyway."""
    piece, heads, K, V = 960, 80, 64, 64
    rows = 12 * piece + 1
    assert -(-(-(-rows * heads // 1024)) // 64) * 64 == piece  # the length that a call of these sizes cuts at
    d = Draw(9)
    decay = -(0.5 + torch.arange(heads) / (2 * heads)) * 60 / rows
    start = d.uniform(1.0, 2.0, 1, heads, V, K)
    q, k = (torch.nn.functional.normalize(d.normal(rows, heads, K), dim=-1).to(DEV) for _ in range(2))
    state = start.to(DEV)
    ssu.linear_attention_varlen(state, q, k, torch.zeros(rows, heads, V, device=DEV), decay.to(DEV),
                                torch.tensor([0, rows], dtype=torch.int32, device=DEV),
                                has_initial_state=torch.ones(1, dtype=torch.bool, device=DEV))
    want = start.double() * torch.exp(decay.double() * rows)[None, :, None, None]
    steps = 31 * 1.5 + 11 * 2.5 + 0.5
    assert float((state.cpu().double() / want - 1).abs().max()) < steps * 2.0 ** -23
