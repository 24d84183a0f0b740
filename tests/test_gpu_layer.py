"""The layer operators on the GPU against their plain fp64 forms (layer_harness), within the
bounds derived there, at the sizes where they can go wrong: sequences of no, one and
few rows, sequences that begin and end anywhere in a tile, odd channel counts,
strided rows, slots that are padding, rows of no sequence."""
import pytest
import torch

import layer_harness as lh
import selective_state_update_ssu_amd as ssu

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def same(a, b):
    return torch.equal(bits(a.cpu()), bits(b.cpu()))


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator().manual_seed(seed)

    def normal(self, *shape, io=F32, scale=1.0):
        return (torch.randn(*shape, generator=self.g) * scale).to(io)

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.g) * (hi - lo) + lo

    def slots(self, nseq, nslots, dtype=torch.int32, inert=()):
        s = torch.randperm(nslots, generator=self.g)[:nseq].to(dtype)
        for k, b in enumerate(inert):
            s[b] = (-1, nslots, nslots + 7)[k % 3]
        return s

    def flags(self, n):
        return torch.rand(n, generator=self.g) < 0.6


# Lengths that meet every place in tiles of 16 rows.
LENGTHS = {
    "one": [1],
    "short": [0, 1, 2, 3, 4, 5, 0, 0, 6],
    "ends": [14, 5, 13, 1, 1, 1, 29, 17, 15, 2, 16, 1, 31],
    "long": [37, 0, 130, 16, 64, 65],
    "ones": [1] * 70,
}


def conv_inputs(seed, lengths, dim, width, io, *, idx=torch.int32, inert=(), strided=True,
                lead=0, tail=0, bias=True):
    d = Draw(seed)
    cu = lh.starts(lengths, lead)
    rows = cu[-1] + tail
    nslots = len(lengths) + 4
    x = d.normal(rows, 2 * dim + 3, io=io)[:, 3:dim + 3] if strided else d.normal(rows, dim, io=io)
    return dict(x=x, weight=d.uniform(-0.7, 0.7, dim, width).to(io),
                bias=d.normal(dim, io=io, scale=0.3) if bias else None, cu=cu,
                state=d.normal(nslots, width - 1, dim, io=io),
                slots=d.slots(len(lengths), nslots, idx, inert), has=d.flags(len(lengths)), idx=idx)


def strided_copy(t):
    """t on the GPU with the same strides (a view of a wider buffer stays one)."""
    if t is None or t.is_contiguous():
        return None if t is None else t.to(DEV)
    wide = torch.full((t.shape[0], t.stride(0)), NAN, dtype=t.dtype, device=DEV)
    view = wide[:, 3:3 + t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("lengths", sorted(LENGTHS))
@pytest.mark.parametrize("dim,width,strided", [(64, 4, False), (40, 4, True), (33, 3, True),
                                               (1, 2, False), (1032, 4, False), (520, 2, False)])
def test_conv_varlen(io, lengths, dim, width, strided):
    n = LENGTHS[lengths]
    c = conv_inputs(dim + width, n, dim, width, io, strided=strided, lead=2, tail=3,
                    inert=(0, 3) if len(n) > 4 else ())
    ref, bound, written, after = lh.conv(c["x"], c["weight"], c["bias"], c["cu"], c["state"],
                                         c["slots"].tolist(), c["has"].tolist(), True)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    got = ssu.causal_conv1d_varlen(
        state, strided_copy(c["x"]), c["weight"].to(DEV),
        torch.tensor(c["cu"], dtype=torch.int32, device=DEV), out, bias=c["bias"].to(DEV),
        has_initial_state=c["has"].to(DEV), state_batch_indices=c["slots"].to(DEV))
    assert got is out
    lh.check("out", out.cpu()[written], ref[written], bound[written])
    assert torch.isnan(out.cpu()[~written].float()).all()
    assert same(state, after)


@pytest.mark.parametrize("activation", [None, "silu", "swish"])
def test_conv_options(activation):
    """No bias, no activation, 64-bit ids, no history anywhere, no slot table; a slot that
    starts from nothing is not read."""
    c = conv_inputs(5, LENGTHS["ends"], 72, 4, BF16, strided=False, bias=False)
    nseq = len(LENGTHS["ends"])
    c["state"].fill_(NAN)
    ref, bound, written, after = lh.conv(c["x"], c["weight"], None, c["cu"], c["state"],
                                         list(range(nseq)), [False] * nseq, activation is not None)
    state = c["state"].to(DEV)
    out = ssu.causal_conv1d_varlen(state, c["x"].to(DEV), c["weight"].to(DEV),
                                   torch.tensor(c["cu"], device=DEV), activation=activation)
    lh.check("out", out, ref, bound)
    assert same(state, after)


@pytest.mark.parametrize("io", [F32, F16, BF16])
@pytest.mark.parametrize("batch,dim,width", [(1, 64, 4), (5, 1032, 4), (70, 33, 3), (3, 1, 2),
                                             (130, 520, 4)])
def test_conv_update(io, batch, dim, width):
    c = conv_inputs(batch + dim, [1] * batch, dim, width, io, inert=(1,) if batch > 2 else (),
                    idx=torch.int64)
    has = [True] * batch
    ref, bound, written, after = lh.conv(c["x"], c["weight"], c["bias"], c["cu"], c["state"],
                                         c["slots"].tolist(), has, True)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    ssu.causal_conv1d_update(state, strided_copy(c["x"]), c["weight"].to(DEV), out,
                             bias=c["bias"].to(DEV), state_batch_indices=c["slots"].to(DEV))
    lh.check("out", out.cpu()[written], ref[written], bound[written])
    assert torch.isnan(out.cpu()[~written].float()).all()
    assert same(state, after)


def scan_inputs(seed, lengths, dim, N, groups, io, dt, state, *, gate=True, D=True, bias=True,
                inert=(), lead=0, tail=0, idx=torch.int32, nslots=None):
    d = Draw(seed)
    cu = lh.starts(lengths, lead)
    rows = cu[-1] + tail
    nslots = nslots or len(lengths) + 3
    bc = d.normal(rows, 5 + 2 * groups * N, io=io)
    return dict(
        x=d.normal(rows, dim, io=io), z=d.normal(rows, 2 * dim, io=io)[:, dim:] if gate else None,
        dt=d.normal(rows, dim, io=dt) if bias else d.uniform(0.001, 0.2, rows, dim).to(dt),
        dt_bias=d.uniform(-6.0, -2.0, dim) if bias else None,
        B=bc[:, 5:5 + groups * N].unflatten(1, (groups, N)),
        C=bc[:, 5 + groups * N:].unflatten(1, (groups, N)),
        A=-torch.exp(d.uniform(0.0, 2.8, dim, N)), D=d.normal(dim) if D else None,
        state=d.normal(nslots, dim, N, io=state), cu=cu,
        slots=d.slots(len(lengths), nslots, idx, inert), has=d.flags(len(lengths)))


def gpu_scan(c, state, out, *, update=False, softplus=True, stream=None, workspace=None):
    g = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    # B and C as columns of one row, z as half of one.
    rows, (groups, N) = c["x"].shape[0], c["B"].shape[1:]
    bc = torch.zeros(rows, 5 + 2 * groups * N, dtype=c["B"].dtype, device=DEV)
    bc[:, 5:5 + groups * N] = g["B"].flatten(1)
    bc[:, 5 + groups * N:] = g["C"].flatten(1)
    B = bc[:, 5:5 + groups * N].unflatten(1, (groups, N))
    C = bc[:, 5 + groups * N:].unflatten(1, (groups, N))
    z = None
    if g["z"] is not None:
        z = torch.cat([g["z"], g["z"]], 1)[:, c["x"].shape[1]:]
    common = dict(D=g["D"], z=z, dt_bias=g["dt_bias"], dt_softplus=softplus,
                  state_batch_indices=g["slots"], stream=stream)
    if update:
        return ssu.selective_scan_update(state, g["x"], g["dt"], g["A"], B, C, out, **common)
    cu = torch.tensor(c["cu"], dtype=c["slots"].dtype, device=DEV)
    return ssu.selective_scan_varlen(state, g["x"], g["dt"], g["A"], B, C, cu, out,
                                     has_initial_state=g["has"], workspace=workspace, **common)


def check_scan(c, *, update=False, softplus=True):
    has = [True] * len(c["has"]) if update else c["has"].tolist()
    ref, bound, written, after, s_bound, touched = lh.scan(
        c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], softplus, c["cu"],
        c["state"], c["slots"].tolist(), has)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=c["x"].dtype, device=DEV)
    assert gpu_scan(c, state, out, update=update, softplus=softplus) is out
    lh.check("out", out.cpu()[written], ref[written], bound[written])
    assert torch.isnan(out.cpu()[~written].float()).all()
    lh.check("state", state.cpu()[touched], after[touched], s_bound[touched])
    assert same(state.cpu()[~touched], c["state"][~touched])


@pytest.mark.parametrize("N", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("io,dt,state", [(F32, F32, F32), (F16, F32, F16), (BF16, BF16, F32),
                                         (BF16, F32, BF16), (F16, F16, BF16)])
def test_scan_varlen_types(N, io, dt, state):
    check_scan(scan_inputs(N, [3, 0, 70, 1, 16], 66, N, 2, io, dt, state, inert=(3,), lead=1,
                           tail=2))


@pytest.mark.parametrize("lengths", sorted(LENGTHS))
@pytest.mark.parametrize("dim,groups", [(1, 1), (40, 4), (65, 1), (130, 2)])
def test_scan_varlen_lengths(lengths, dim, groups):
    n = LENGTHS[lengths]
    check_scan(scan_inputs(dim, n, dim, 16, groups, BF16, F32, F32,
                           inert=(0, 3) if len(n) > 4 else (), idx=torch.int64))


@pytest.mark.parametrize("kw", [dict(gate=False), dict(D=False), dict(bias=False),
                                dict(gate=False, D=False, bias=False)])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_varlen_options(kw, softplus):
    c = scan_inputs(7, [5, 80, 1, 200], 48, 16, 1, F32, F32, F32, **kw)
    if kw.get("bias", True) and not softplus:
        c["dt"], c["dt_bias"] = c["dt"].abs() * 0.1, c["dt_bias"].abs() * 0.01
    check_scan(c, softplus=softplus)


def test_scan_varlen_many_sequences():
    """Enough sequences that none is cut, one of them long."""
    lengths = [k % 4 for k in range(600)]
    lengths[77] = 150
    check_scan(scan_inputs(8, lengths, 24, 16, 1, BF16, BF16, F32, inert=(4, 9, 13)))


@pytest.mark.parametrize("N", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("io,dt,state", [(F32, F32, F32), (F16, F32, F16), (BF16, BF16, F32),
                                         (BF16, F32, BF16), (F32, F32, BF16), (F16, F16, F32)])
def test_scan_update_types(N, io, dt, state):
    for batch, dim, groups in ((1, 64, 1), (7, 66, 2), (40, 5, 1), (3, 260, 4)):
        check_scan(scan_inputs(N + dim, [1] * batch, dim, N, groups, io, dt, state,
                               inert=(2, 5) if batch > 6 else ()), update=True)


@pytest.mark.parametrize("kw", [dict(gate=False), dict(D=False), dict(bias=False)])
@pytest.mark.parametrize("softplus", [True, False])
def test_scan_update_options(kw, softplus):
    c = scan_inputs(9, [1] * 6, 100, 16, 1, F32, F32, F32, idx=torch.int64, **kw)
    if kw.get("bias", True) and not softplus:
        c["dt"], c["dt_bias"] = c["dt"].abs() * 0.1, c["dt_bias"].abs() * 0.01
    check_scan(c, update=True, softplus=softplus)


def test_softplus_range():
    """dt far below and above zero: v keeps its relative accuracy (down to where 1 + e^d
    is 1 in fp32) and does not overflow."""
    c = scan_inputs(10, [1] * 4, 64, 16, 1, F32, F32, F32, nslots=4)
    c["dt"] = torch.linspace(-80, 60, 256).reshape(4, 64)
    c["dt_bias"].zero_()
    c["A"].fill_(-1e-3)
    check_scan(c, update=True)
    c["has"][:] = True
    check_scan(c)


def test_scan_not_finite_stays_in_its_sequence():
    """Infinite and NaN inputs of one sequence reach no other, a slot that is not an initial
    state is not read, and a state that ends infinite does so past a tile's end too."""
    c = scan_inputs(11, [20, 21, 70, 5], 40, 16, 1, F32, F32, F32)
    c["has"] = torch.tensor([True, False, True, False])
    c["state"][c["slots"][1].item()] = NAN
    c["x"][2, 0], c["x"][115, 3] = NAN, float("inf")
    state = c["state"].to(DEV)
    out = gpu_scan(c, state, None).cpu()
    ref, bound, _, after, s_bound, touched = lh.scan(
        c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], True, c["cu"],
        c["state"], c["slots"].tolist(), c["has"].tolist())
    assert torch.equal(torch.isfinite(out), torch.isfinite(ref))
    fine = torch.isfinite(ref)
    lh.check("out", out[fine], ref[fine], bound[fine])
    got = state.cpu()[touched]
    fine = torch.isfinite(after[touched])
    assert torch.equal(torch.isfinite(got), fine)
    lh.check("state", got[fine], after[touched][fine], s_bound[touched][fine])


def test_prompt_then_tokens():
    """A prompt in one call is the prompt in two and its last rows as single tokens, for the
    convolution bit for bit and for the scan within the bounds."""
    d = Draw(12)
    dim, N, rows = 96, 16, 50
    x = d.normal(rows, dim, io=BF16).to(DEV)
    w, bias = d.uniform(-0.5, 0.5, dim, 4).to(BF16).to(DEV), d.normal(dim, io=BF16).to(DEV)
    whole = torch.full((1, 3, dim), NAN, dtype=BF16, device=DEV)
    out = ssu.causal_conv1d_varlen(whole, x, w, torch.tensor([0, rows], device=DEV), bias=bias)
    parts = torch.full((1, 3, dim), NAN, dtype=BF16, device=DEV)
    yes = torch.ones(1, dtype=torch.bool, device=DEV)
    got = [ssu.causal_conv1d_varlen(parts, x[:2], w, torch.tensor([0, 2], device=DEV), bias=bias),
           ssu.causal_conv1d_varlen(parts, x[2:47], w, torch.tensor([0, 45], device=DEV), bias=bias,
                                    has_initial_state=yes)]
    got += [ssu.causal_conv1d_update(parts, x[t:t + 1], w, bias=bias) for t in range(47, rows)]
    assert same(torch.cat(got), out) and same(parts, whole)

    c = scan_inputs(13, [47], dim, N, 1, BF16, F32, F32, tail=3, nslots=1)
    c["has"][:] = False
    full = dict(c, cu=[0, 50])
    ref, bound, _, after, s_bound, _ = lh.scan(
        full["x"], full["dt"], full["A"], full["B"], full["C"], full["D"], full["z"],
        full["dt_bias"], True, full["cu"], full["state"], [0], [False])
    state = c["state"].to(DEV)
    got = gpu_scan(c, state, None)[:47].cpu()
    for t in range(47, 50):
        one = {k: v[t:t + 1] if k in ("x", "z", "dt", "B", "C") else v for k, v in c.items()}
        got = torch.cat([got, gpu_scan(one, state, None, update=True).cpu()])
    lh.check("out", got, ref, bound)
    lh.check("state", state, after, s_bound)


# ----------------------------------------------------------------------- slots

def cache_set(seed, nslots, shapes, padded=False):
    d = Draw(seed)
    out = []
    for shape, dtype in shapes:
        if dtype in (F32, F16, BF16):
            t = d.normal(nslots, *shape, io=dtype)
        else:
            t = torch.randint(0, 127, (nslots, *shape), generator=d.g).to(dtype)
        if padded:  # slots apart
            flat = torch.zeros(nslots, t[0].numel() + 24, dtype=dtype)
            flat[:, :t[0].numel()] = t.flatten(1)
            t = flat.as_strided((nslots, *shape), (flat.stride(0), *t.stride()[1:]))
        out.append(t)
    return out


def on_gpu(caches):
    out = []
    for c in caches:
        g = torch.empty_strided(c.shape, c.stride(), dtype=c.dtype, device=DEV)
        g.copy_(c)
        out.append(g)
    return out


SHAPES = [((3, 576), BF16), ((8, 64, 16), F32), ((5,), torch.uint8), ((4100,), F16), ((1,), F32),
          ((40, 1000), torch.uint8)]


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("n", [0, 1, 3, 9])
def test_cache_copy(n, padded):
    caches = cache_set(n, 24, SHAPES, padded)
    gpu = on_gpu(caches)
    src, dst = [3, 3, 3, 3, 3, 7, 7, -1, 5][:n], [0, 1, 2, 24, 8, 9, 10, 11, 12][:n]
    lh.copy(caches, src, dst)
    ssu.cache_copy(gpu, torch.tensor(src, dtype=torch.int32, device=DEV),
                   torch.tensor(dst, dtype=torch.int64, device=DEV))
    for i, (a, b) in enumerate(zip(gpu, caches)):
        assert same(a, b), i


@pytest.mark.parametrize("ways", [1, 3, 4, 7])
def test_cache_copy_many_pairs(ways):
    """Enough copies that a workgroup takes four pairs, with sources named 1 to 7 times in a
    row, pairs to skip among them and a last group that is not full."""
    nslots, n = 700, 301
    caches = cache_set(ways, nslots, [((3000,), F32), ((5,), torch.uint8), ((40, 100), BF16)])
    gpu = on_gpu(caches)
    src = [k // ways for k in range(n)]
    dst = [399 + k if k % 11 else -1 for k in range(n)]
    lh.copy(caches, src, dst)
    ssu.cache_copy(gpu, torch.tensor(src, device=DEV), torch.tensor(dst, device=DEV))
    assert all(same(a, b) for a, b in zip(gpu, caches))


def test_cache_copy_many_caches():
    caches = cache_set(20, 6, [((k + 1, 16), F32) for k in range(70)] + [((0,), F32)])
    gpu = on_gpu(caches)
    lh.copy(caches, [0, 2], [5, 1])
    ssu.cache_copy(gpu, torch.tensor([0, 2], device=DEV), torch.tensor([5, 1], device=DEV))
    assert all(same(a, b) for a, b in zip(gpu, caches))


@pytest.mark.parametrize("nslots", [0, 1, 5, 1023, 1024, 1025, 5000])
def test_cache_counts(nslots):
    """Allocation up to more slots than are free, freeing and retaining with repeats, padding
    and free slots among the ids, against the plain loops after every call."""
    d = Draw(nslots)
    ref = torch.randint(0, 3, (nslots,), generator=d.g).tolist()
    if nslots > 3:
        ref[2] = -1
    gpu = torch.tensor(ref, dtype=torch.int32, device=DEV)
    for n in (0, 1, nslots // 4, nslots + 3):
        want = lh.alloc(ref, n)
        assert ssu.cache_alloc(gpu, n).tolist() == want
        assert gpu.tolist() == ref
        ids = torch.randint(-2, nslots + 2, (2 * nslots + 1,), generator=d.g)
        # A slot is freed and retained in calls of their own: the order inside one is free.
        lh.adjust(ref, ids.tolist(), 1)
        ssu.cache_retain(gpu, ids.to(DEV))
        assert gpu.tolist() == ref
        lh.adjust(ref, ids.tolist() + ids.tolist(), -1)
        ssu.cache_free(gpu, torch.cat([ids, ids]).to(torch.int32).to(DEV))
        assert gpu.tolist() == ref


def test_cache_fork():
    caches = cache_set(30, 12, SHAPES)
    gpu = on_gpu(caches)
    ref = [0, 1, 0, 2, 0, 0, 1, 0, 1, 0, 1, 0]
    count = torch.tensor(ref, dtype=torch.int32, device=DEV)
    parents = [3, 3, 1, 1, 1, 6, 8, 8]  # one more than there are free slots
    want = lh.alloc(ref, len(parents))
    assert want[-1] == -1
    lh.copy(caches, parents, want)
    got = ssu.cache_fork(gpu, count, torch.tensor(parents, device=DEV))
    assert got.tolist() == want and count.tolist() == ref
    assert all(same(a, b) for a, b in zip(gpu, caches))


@pytest.mark.parametrize("nslots,used", [(1, 0.5), (2, 0.5), (7, 0.0), (7, 1.0), (24, 0.6),
                                         (40, 0.1), (40, 0.9), (3000, 0.5)])
def test_cache_compact(nslots, used):
    d = Draw(nslots)
    ref = [(1 + k % 3) if r < used else 0
           for k, r in enumerate(torch.rand(nslots, generator=d.g).tolist())]
    shapes = SHAPES if nslots < 100 else [((3,), F32), ((16,), BF16)]
    caches = cache_set(31, nslots, shapes, padded=nslots == 24)
    gpu, count = on_gpu(caches), torch.tensor(ref, dtype=torch.int32, device=DEV)
    want = lh.compact(caches, ref)
    assert ssu.cache_compact(gpu, count).tolist() == want
    assert count.tolist() == ref
    assert all(same(a, b) for a, b in zip(gpu, caches))
    assert ssu.cache_compact(gpu, count).tolist() == [i if r > 0 else -1 for i, r in enumerate(ref)]


# -------------------------------------------------- offsets, streams, graphs, refusals

def test_offsets_past_32_bits():
    """Slots and rows more than 2^31 elements apart."""
    far = (1 << 31) + 64
    big = torch.empty(far + 4096, dtype=BF16, device=DEV)
    d = Draw(40)
    dim, N = 32, 16
    # Two slots of a convolution, and two rows of its input.
    state = big.as_strided((2, 3, dim), (far, dim, 1))
    init = d.normal(2, 3, dim, io=BF16)
    state.copy_(init)
    x = big[2048:].as_strided((2, dim), (far, 1))
    xs = d.normal(2, dim, io=BF16)
    x.copy_(xs)
    w = d.uniform(-0.5, 0.5, dim, 4).to(BF16)
    ref, bound, _, after = lh.conv(xs, w, None, [0, 1, 2], init, [0, 1], [True, True], True)
    # (conv_state and x interleave in one buffer: a copy of x keeps the operands apart.)
    apart = torch.empty(far + 64, dtype=BF16, device=DEV).as_strided((2, dim), (far, 1))
    apart.copy_(x)
    out = ssu.causal_conv1d_update(state, apart, w.to(DEV))
    lh.check("conv out", out, ref, bound)
    assert same(state, after)
    # Two slots of a scan's state.
    c = scan_inputs(41, [1, 1], dim, N, 1, BF16, F32, BF16, nslots=2)
    s = big.as_strided((2, dim, N), (far, N, 1))
    s.copy_(c["state"])
    ref, bound, _, after, s_bound, _ = lh.scan(
        c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], True, c["cu"],
        c["state"], c["slots"].tolist(), [True, True])
    out = gpu_scan(c, s, None, update=True)
    lh.check("scan out", out, ref, bound)
    lh.check("scan state", s, after, s_bound)
    # And a copy between them.
    ssu.cache_copy([s], torch.tensor([0], device=DEV), torch.tensor([1], device=DEV))
    assert same(s[0], s[1])


def test_side_stream():
    """Calls on another stream than the current one, their scratch and out included."""
    c = scan_inputs(50, [90, 3, 140], 70, 16, 1, BF16, F32, F32)
    state = c["state"].to(DEV)
    want = gpu_scan(c, state, None)
    side = torch.cuda.Stream()
    for _ in range(3):
        again = c["state"].to(DEV)
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        got = gpu_scan(c, again, None, stream=side)
        side.synchronize()
        assert same(got, want) and same(again, state)


def test_workspace_argument():
    c = scan_inputs(51, [90, 3, 140], 70, 16, 1, BF16, F32, F32)
    state, again = c["state"].to(DEV), c["state"].to(DEV)
    want = gpu_scan(c, state, None)
    size = ssu.scan_workspace_bytes(233, 3, 70, 16, 1)
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    assert same(gpu_scan(c, again, None, workspace=ws), want) and same(again, state)
    with pytest.raises(ValueError, match="workspace"):
        gpu_scan(c, again, None, workspace=ws[:-1])


def test_graph_replays_match_eager():
    """Prompts, tokens and slot operations recorded into one graph; every replay equals
    one more eager pass, with other work between the replays."""
    c = scan_inputs(60, [30, 200], 48, 16, 1, BF16, F32, F32, nslots=6)
    d = Draw(61)
    x, w = d.normal(230, 48, io=BF16).to(DEV), d.uniform(-0.5, 0.5, 48, 4).to(BF16).to(DEV)
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)
    g = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    slots = torch.tensor([1, 4], dtype=torch.int32, device=DEV)
    yes = torch.ones(2, dtype=torch.bool, device=DEV)

    def make():
        return dict(conv=d0.clone(), state=s0.clone(), count=r0.clone())

    d0 = d.normal(6, 3, 48, io=BF16).to(DEV)
    s0, r0 = c["state"].to(DEV), torch.tensor([0, 1, 0, 0, 1, 0], dtype=torch.int32, device=DEV)

    def step(m):
        u = ssu.causal_conv1d_varlen(m["conv"], x, w, cu, has_initial_state=yes,
                                     state_batch_indices=slots)
        y = ssu.selective_scan_varlen(m["state"], u, g["dt"], g["A"], g["B"], g["C"], cu, D=g["D"],
                                      dt_bias=g["dt_bias"], dt_softplus=True,
                                      has_initial_state=yes, state_batch_indices=slots)
        kids = ssu.cache_fork([m["conv"], m["state"]], m["count"], slots)
        v = ssu.causal_conv1d_update(m["conv"], x[:2], w, state_batch_indices=kids)
        o = ssu.selective_scan_update(m["state"], v, g["dt"][:2], g["A"], g["B"][:2], g["C"][:2],
                                      dt_bias=g["dt_bias"], dt_softplus=True,
                                      state_batch_indices=kids)
        ssu.cache_free(m["count"], kids)
        remap = ssu.cache_compact([m["conv"][:0], m["state"][:0]], m["count"][:0])
        return [y, o, kids, remap]

    eager, graph = make(), make()
    want = step(eager)
    step(graph)  # the workspace exists before the capture
    torch.cuda.synchronize()
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        got = step(graph)
    for i in range(4):
        want = step(eager)
        cg.replay()
        float((torch.randn(1 << 18, device=DEV) * 2).sum())
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want)), i
        assert all(same(graph[k], eager[k]) for k in graph), i


def test_binding_refusals():
    x = torch.zeros(4, 32, dtype=BF16, device=DEV)
    w = torch.zeros(32, 4, dtype=BF16, device=DEV)
    state = torch.zeros(4, 3, 32, dtype=BF16, device=DEV)
    cu = torch.tensor([0, 4], device=DEV)
    bad = [
        (ValueError, "GPU", lambda: ssu.causal_conv1d_update(state.cpu(), x.cpu(), w.cpu())),
        (ValueError, "conv_state", lambda: ssu.causal_conv1d_update(state[:, :2], x, w)),
        (ValueError, "contiguous", lambda: ssu.causal_conv1d_update(state.transpose(1, 2).contiguous().transpose(1, 2), x, w)),
        (ValueError, "weight", lambda: ssu.causal_conv1d_update(state, x, w.float())),
        (ValueError, "bias", lambda: ssu.causal_conv1d_update(state, x, w, bias=w[:, 0])),
        (NotImplementedError, "width", lambda: ssu.causal_conv1d_update(
            torch.zeros(4, 4, 32, dtype=BF16, device=DEV), x, torch.zeros(32, 5, dtype=BF16, device=DEV))),
        (NotImplementedError, "activation", lambda: ssu.causal_conv1d_update(state, x, w, activation="relu")),
        (ValueError, "rows must be contiguous", lambda: ssu.causal_conv1d_update(state, x.t().contiguous().t(), w)),
        (ValueError, "out overlaps", lambda: ssu.causal_conv1d_update(state, x, w, x)),
        (ValueError, "cu_seqlens", lambda: ssu.causal_conv1d_varlen(state, x, w, None)),
        (ValueError, "int32 or int64", lambda: ssu.causal_conv1d_varlen(state, x, w, cu.float())),
        (ValueError, "has_initial_state", lambda: ssu.causal_conv1d_varlen(state, x, w, cu, has_initial_state=cu[:1])),
        (ValueError, "state_batch_indices", lambda: ssu.causal_conv1d_varlen(state, x, w, cu, state_batch_indices=cu)),
        (ValueError, "as many slots", lambda: ssu.causal_conv1d_update(state[:2], x, w)),
    ]
    A = torch.zeros(32, 16, device=DEV)
    B = torch.zeros(4, 1, 16, dtype=BF16, device=DEV)
    s = torch.zeros(4, 32, 16, device=DEV)
    dt = torch.zeros(4, 32, device=DEV)
    bad += [
        (ValueError, "A must", lambda: ssu.selective_scan_update(s, x, dt, A[:, :8], B, B)),
        (ValueError, "A must", lambda: ssu.selective_scan_update(s, x, dt, A.to(BF16), B, B)),
        (ValueError, "C must", lambda: ssu.selective_scan_update(s, x, dt, A, B, B[:, :, :8])),
        (ValueError, "dt must", lambda: ssu.selective_scan_update(s, x, dt.half(), A, B, B)),
        (ValueError, "D must", lambda: ssu.selective_scan_update(s, x, dt, A, B, B, D=A)),
        (ValueError, "groups", lambda: ssu.selective_scan_update(s, x, dt, A, B.expand(4, 3, 16), B)),
        (NotImplementedError, "dstate 24", lambda: ssu.selective_scan_update(
            torch.zeros(4, 32, 24, device=DEV), x, dt, torch.zeros(32, 24, device=DEV),
            torch.zeros(4, 1, 24, dtype=BF16, device=DEV), torch.zeros(4, 1, 24, dtype=BF16, device=DEV))),
        (NotImplementedError, "x dtype", lambda: ssu.selective_scan_update(s, x.double(), dt, A, B, B)),
        (ValueError, "expected", lambda: ssu.selective_scan_update(s, x, dt.cpu(), A, B, B)),
        (ValueError, "out overlaps", lambda: ssu.selective_scan_varlen(s, x, dt, A, B, B, cu, x)),
    ]
    count = torch.zeros(4, dtype=torch.int32, device=DEV)
    ids = torch.zeros(1, dtype=torch.int32, device=DEV)
    bad += [
        (ValueError, "refcount", lambda: ssu.cache_alloc(count.long(), 1)),
        (ValueError, "n must", lambda: ssu.cache_alloc(count, -1)),
        (ValueError, "GPU", lambda: ssu.cache_free(count.cpu(), ids.cpu())),
        (ValueError, "int32 or int64", lambda: ssu.cache_free(count, ids.float())),
        (ValueError, "1-D", lambda: ssu.cache_free(count, ids[None])),
        (ValueError, r"caches\[0\]", lambda: ssu.cache_fork([s[:3]], count, ids)),
        (ValueError, "contiguous inside", lambda: ssu.cache_fork([s.transpose(1, 2)], count, ids)),
        (ValueError, "overlap", lambda: ssu.cache_compact([s[:1].expand(4, 32, 16)], count)),
        (ValueError, "as many entries", lambda: ssu.cache_copy([s], ids, cu)),
    ]
    for kind, match, call in bad:
        with pytest.raises(kind, match=match):
            call()
    torch.cuda.synchronize()
    assert count.tolist() == [0] * 4


def test_serving_example():
    """The example's run: packed prompts, forks, decoding and compaction together give each
    request the scores of a run alone. The library's calls are row by row the same but for the
    join of pieces; the projections are torch's bf16 products, whose shapes differ
    between the two runs: a few bf16 roundings (2^-8 each) of the largest score over the
    layers, far from what a wrong slot would give."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "state_space_serving.py")
    spec = importlib.util.spec_from_file_location("state_space_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert module.main(layers=3, dim=256, tokens=10) < 10 * 2.0 ** -8


# ------------------------------------------------------------- scratch of the scan

def cut_scan(seed, lengths=(90, 3, 140), dim=70):
    """A scan in pieces: a call on its inputs, its starting state and the eager result."""
    c = scan_inputs(seed, list(lengths), dim, 16, 1, BF16, F32, F32)
    g = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    cu = torch.tensor(c["cu"], dtype=torch.int32, device=DEV)
    assert ssu.scan_workspace_bytes(c["cu"][-1], len(lengths), dim, 16, 1) > 255

    def call(state, out=None):
        return ssu.selective_scan_varlen(state, g["x"], g["dt"], g["A"], g["B"], g["C"], cu, out,
                                         D=g["D"], z=g["z"], dt_bias=g["dt_bias"], dt_softplus=True,
                                         has_initial_state=g["has"], state_batch_indices=g["slots"])
    state = g["state"].clone()
    want = call(state)
    torch.cuda.synchronize()
    return call, g["state"], want, state


def test_recorded_scratch_outlives_larger_calls():
    """A graph of a scan in pieces, replayed after larger calls on its stream and a reset of
    the prefill's buffers, with tensors made since then in whatever memory was free: the replays
    give the eager result and leave those tensors alone."""
    call, start, want, after = cut_scan(70)
    larger = cut_scan(71, (300, 250), 200)
    s = torch.cuda.Stream()
    cached = dict(ssu._ssd_workspaces)
    with torch.cuda.stream(s):
        state = start.clone()
        call(state)
        torch.cuda.synchronize()
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg, stream=s):
            got = call(state)
        larger[0](larger[1].clone())
        assert ssu._ssd_workspaces == cached
        ssu.reset_ssd_workspaces()
        torch.cuda.synchronize()
        size = ssu.scan_workspace_bytes(233, 3, 70, 16, 1)
        others = [torch.full((n,), 77, dtype=torch.uint8, device=DEV)
                  for n in (size, size, size - 255, size // 2, 4 * size) for _ in range(4)]
        for i in range(4):
            state.copy_(start)
            cg.replay()
            larger[0](larger[1].clone())
            torch.cuda.synchronize()
            assert same(got, want) and same(state, after), i
            assert all(bool((t == 77).all()) for t in others), i


def test_two_threads_on_one_stream():
    """Two host threads repeat scans in pieces of different inputs on the same stream: every
    result equals the single-threaded one bit for bit."""
    import threading
    runs = [cut_scan(72), cut_scan(73, (200, 20, 90), 70)]
    side = torch.cuda.Stream()
    results, errors = [[], []], []

    def worker(i):
        try:
            call, start = runs[i][:2]
            with torch.cuda.stream(side):
                for _ in range(40):
                    state = start.clone()
                    results[i].append((call(state), state))
        except Exception as e:  # reported below, on the main thread
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for (_, _, want, after), got in zip(runs, results):
        assert len(got) == 40
        assert all(same(y, want) and same(s, after) for y, s in got)


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs two GPUs")
def test_tensors_on_a_gpu_that_is_not_current():
    """Calls on tensors of GPU 1 while GPU 0 is current run on GPU 1's stream and leave GPU 0
    current."""
    c = scan_inputs(80, [1] * 5, 64, 16, 1, BF16, F32, F32)
    on = [{k: v.to(f"cuda:{d}") if isinstance(v, torch.Tensor) else v for k, v in c.items()}
          for d in (0, 1)]
    results = []
    for g in on:
        y = ssu.selective_scan_update(g["state"], g["x"], g["dt"], g["A"], g["B"], g["C"],
                                      dt_bias=g["dt_bias"], dt_softplus=True,
                                      state_batch_indices=g["slots"])
        count = torch.zeros(4, dtype=torch.int32, device=y.device)
        ids = ssu.cache_alloc(count, 2)
        assert torch.cuda.current_device() == 0
        assert y.device == ids.device == g["x"].device
        torch.cuda.synchronize(y.device)
        results.append([y.cpu(), g["state"].cpu(), ids.cpu(), count.cpu()])
    assert all(same(a, b) for a, b in zip(*results))


# --------------------------------------------------- joins of pieces out of fp32's range

def check_join(c, softplus=True):
    """A scan in pieces against the definition: finite values within their bounds, and the
    same infinities and NaNs in the states."""
    state = c["state"].to(DEV)
    out = gpu_scan(c, state, None, softplus=softplus).cpu()
    ref, bound, written, after, s_bound, touched = lh.scan(
        c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], softplus, c["cu"],
        c["state"], c["slots"].tolist(), c["has"].tolist())
    out, ref, bound = out[written], ref[written], bound[written]
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(out), fine)
    lh.check("out", out[fine], ref[fine], bound[fine])
    got, after, s_bound = state.cpu()[touched], after[touched], s_bound[touched]
    fine = torch.isfinite(after)
    assert torch.equal(torch.isnan(got), torch.isnan(after))
    assert torch.equal(got[~fine & ~torch.isnan(after)].double(), after[~fine & ~torch.isnan(after)])
    lh.check("state", got[fine], after[fine], s_bound[fine])


@pytest.mark.parametrize("dim,N", [(40, 16), (70, 64), (20, 256)])
def test_join_keeps_infinite_states(dim, N):
    """Infinite entering states over pieces whose decay underflows, though no row's does."""
    c = scan_inputs(90, [300, 5, 200], dim, N, 1, F32, F32, F32, bias=False)
    c["dt"] = c["dt"].abs() * 0.2 + 0.1
    c["A"] = -Draw(91).uniform(0.5, 16.0, dim, N)
    c["has"][:] = True
    for b, slot in enumerate(c["slots"].tolist()):
        c["state"][slot, b::3] = float("inf")
        c["state"][slot, b + 4::5] = float("-inf")
    check_join(c, softplus=False)


def test_join_of_growing_states():
    """Growth by up to e^144 a piece: states that are zero until late rows, and tiny ones that
    grow into range."""
    dim, N = 40, 16
    c = scan_inputs(92, [300, 200], dim, N, 1, F32, F32, F32, bias=False)
    c["dt"] = torch.full_like(c["dt"], 0.5)
    c["A"] = Draw(93).uniform(2.0, 4.5, dim, N)
    for b in range(2):
        end = c["cu"][b + 1]
        c["x"][c["cu"][b]:end - 3] = 0
    c["has"][:] = False
    check_join(c, softplus=False)
    c["has"][:] = True
    c["state"][:] = 0
    check_join(c, softplus=False)
    # Still, then e^91.2 in the second piece, then still: 2^-120 becomes 2^11.6.
    c["A"].fill_(2.85)
    c["dt"].zero_()
    c["dt"][64:128] = 0.5
    c["cu"] = [0, 200]
    c["slots"], c["has"] = c["slots"][:1], c["has"][:1]
    c["x"].zero_()
    c["state"].fill_(2.0 ** -120)
    check_join(c, softplus=False)


def test_out_beside_inputs():
    """out in columns of the buffer that holds x, for prompts and tokens: the results of a
    buffer of its own."""
    d = Draw(95)
    rows, dim = 37, 64
    cu = torch.tensor([0, 20, 37], dtype=torch.int32, device=DEV)
    w = d.uniform(-0.5, 0.5, dim, 4).to(BF16).to(DEV)
    wide = d.normal(rows, 3 * dim, io=BF16).to(DEV)
    x, out, z = wide[:, :dim], wide[:, dim:2 * dim], wide[:, 2 * dim:]
    c = scan_inputs(96, [20, 17], dim, 16, 1, BF16, F32, F32, nslots=2)
    g = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    history, state = d.normal(2, 3, dim, io=BF16).to(DEV), g["state"]

    def both(conv_out, scan_out, h, s):
        u = ssu.causal_conv1d_varlen(h, x, w, cu, conv_out).clone()
        y = ssu.selective_scan_varlen(s, x, g["dt"], g["A"], g["B"], g["C"], cu, scan_out, z=z).clone()
        u1 = ssu.causal_conv1d_update(h, x[:2], w, None if conv_out is None else conv_out[:2]).clone()
        y1 = ssu.selective_scan_update(s, x[:2], g["dt"][:2], g["A"], g["B"][:2], g["C"][:2],
                                       None if scan_out is None else scan_out[:2], z=z[:2])
        return [u, y, u1, y1.clone(), h, s]

    before = wide.clone()
    want = both(None, None, history.clone(), state.clone())
    got = both(out, out, history.clone(), state.clone())
    assert all(same(a, b) for a, b in zip(got, want))
    assert same(x, before[:, :dim]) and same(z, before[:, 2 * dim:])
    with pytest.raises(ValueError, match="out overlaps x"):
        ssu.causal_conv1d_varlen(history, x, w, cu, wide[:, 1:dim + 1])


def test_allocation_errors_are_torchs():
    """What does not fit raises torch.OutOfMemoryError, as torch's own calls do; more ids than any
    cache has are refused before anything is allocated."""
    x = torch.zeros(1, 512, dtype=BF16, device=DEV).expand(1 << 30, 512)
    w = torch.zeros(512, 4, dtype=BF16, device=DEV)
    state = torch.zeros(1, 3, 512, dtype=BF16, device=DEV)
    cu = torch.tensor([0, 1 << 30], device=DEV)
    with pytest.raises(torch.OutOfMemoryError):
        ssu.causal_conv1d_varlen(state, x, w, cu)
    count = torch.zeros(4, dtype=torch.int32, device=DEV)
    for n in (1 << 31, 1 << 50):
        with pytest.raises(ValueError, match="n must be"):
            ssu.cache_alloc(count, n)
    assert count.tolist() == [0] * 4


def test_a_tensor_is_no_list_of_caches():
    cache = torch.arange(48, dtype=torch.float32, device=DEV).reshape(4, 4, 3)
    before, ids = cache.clone(), torch.tensor([0], dtype=torch.int32, device=DEV)
    count = torch.tensor([1, 0, 1, 0], dtype=torch.int32, device=DEV)
    for call in (lambda: ssu.cache_copy(cache, ids, ids + 1), lambda: ssu.cache_fork(cache, count, ids),
                 lambda: ssu.cache_compact(cache, count)):
        with pytest.raises(ValueError, match="list of tensors"):
            call()
    assert same(cache, before) and count.tolist() == [1, 0, 1, 0]
