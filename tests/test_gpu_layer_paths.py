"""The layer operators' paths for large calls against their plain fp64 forms (layer_harness):
tiles of 16 rows and two sequences per wave in the convolution, whole sequences sorted and
folded over the card and pieces of more than 64 rows in the scan, compactions of more copies
than workgroups. Every test states the rule that its sizes have to meet."""
import pytest
import torch

import layer_harness as lh
import selective_state_update_ssu_amd as ssu
from test_gpu_layer import (BF16, DEV, F16, F32, NAN, Draw, cache_set, check_scan, conv_inputs,
                            gpu_scan, on_gpu, same, scan_inputs, strided_copy)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")


# (io, channels, whether x is at an odd place of wider rows, elements per lane)
CONV = {"f32": (F32, 4100, False, 4), "f16": (F16, 8200, False, 8), "bf16": (BF16, 8200, False, 8),
        "bf16 odd": (BF16, 1101, True, 1), "f32 odd": (F32, 1101, True, 1)}


def conv_lengths(kind):
    if kind == "few":  # fewer than 64; starts at 35 k, every place of a tile
        return [35] * 28 + [1, 2, 3, 0, 16] + [35] * 28 + [100]
    lengths = []  # 19 rows a turn: the turn's short sequences come to every place of a tile
    while sum(lengths) < 2100:
        lengths += [1, 2, 3, 0, 4, 9]
    return lengths + [0, 40]


@pytest.mark.parametrize("kind", ["few", "many"])
@pytest.mark.parametrize("name,width", [("f32", 4), ("f16", 3), ("bf16", 4), ("bf16 odd", 4),
                                        ("f32 odd", 2)])
def test_conv_varlen_long_tiles(name, width, kind):
    """Tiles of 16 rows (2,048 of them over the channel blocks): sequences that start and end at
    every place of a tile, inert ones among them, rows of none before and after."""
    io, dim, strided, vec = CONV[name]
    lengths = conv_lengths(kind)
    c = conv_inputs(dim + width, lengths, dim, width, io, strided=strided, lead=2, tail=5,
                    inert=(0, 3, 9, 20, 21, 40))
    rows = c["x"].shape[0]
    assert (rows + 15) // 16 * -(-dim // (64 * vec)) >= 2048
    starts = {b % 16 for b, n in zip(c["cu"], lengths) if 0 < n}
    assert starts == set(range(16))
    ref, bound, written, after = lh.conv(c["x"], c["weight"], c["bias"], c["cu"], c["state"],
                                         c["slots"].tolist(), c["has"].tolist(), True)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    ssu.causal_conv1d_varlen(
        state, strided_copy(c["x"]), c["weight"].to(DEV),
        torch.tensor(c["cu"], dtype=torch.int32, device=DEV), out, bias=c["bias"].to(DEV),
        has_initial_state=c["has"].to(DEV), state_batch_indices=c["slots"].to(DEV))
    got = out.cpu()
    lh.check("out", got[written], ref[written], bound[written])
    assert torch.isnan(got[~written].float()).all()
    assert same(state, after)


@pytest.mark.parametrize("name,batch,width", [("f32", 513, 3), ("f16", 512, 4), ("bf16", 513, 4),
                                              ("bf16 odd", 457, 2)])
def test_conv_update_two_sequences_per_wave(name, batch, width):
    """8,192 waves and more: a wave takes two sequences, of which the first, the second or both
    may be inert, and the last wave's second may not exist."""
    io, dim, strided, vec = CONV[name]
    assert batch * -(-dim // (64 * vec)) >= 8192
    c = conv_inputs(batch + dim, [1] * batch, dim, width, io, strided=strided,
                    inert=(1, 6, 100, 101, 256))
    ref, bound, written, after = lh.conv(c["x"], c["weight"], c["bias"], c["cu"], c["state"],
                                         c["slots"].tolist(), [True] * batch, True)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    ssu.causal_conv1d_update(state, strided_copy(c["x"]), c["weight"].to(DEV), out,
                             bias=c["bias"].to(DEV), state_batch_indices=c["slots"].to(DEV))
    got = out.cpu()
    lh.check("out", got[written], ref[written], bound[written])
    assert torch.isnan(got[~written].float()).all()
    assert same(state, after)


@pytest.mark.parametrize("nseq,dim,groups,N,io,dt,gate", [
    (20, 1664, 1, 8, BF16, F32, True),      # 520 workgroups: two rounds and a part
    (9, 7300, 2, 16, F32, F32, False),      # 1,044, a last channel block of each group that is not full
    (64, 768, 1, 16, F16, F16, True),       # 768: three rounds
    (16, 4096, 4, 64, BF16, BF16, True),    # 1,024
    (6, 6272, 1, 128, F16, F32, False),     # 588
])
def test_scan_whole_sequences_in_order(nseq, dim, groups, N, io, dt, gate):
    """Up to 64 whole sequences, 512 workgroups and more: taken from the longest to the shortest,
    every second round of the card backwards. Lengths from none to 70, equal ones among them,
    inert sequences too."""
    blocks = -(-(dim // groups) // 64) * groups
    assert nseq * blocks >= 512 and nseq <= 64
    lengths = [(0, 7, 70, 1, 7, 23, 8, 0, 16, 41, 7, 64)[b % 12] for b in range(nseq)]
    check_scan(scan_inputs(nseq + dim, lengths, dim, N, groups, io, dt, F32, gate=gate, lead=1,
                           tail=2, inert=(3, 5)))


def test_scan_whole_sequences_unsorted():
    """More than 64 whole sequences keep their order."""
    lengths = [(b * 7) % 45 for b in range(70)]
    check_scan(scan_inputs(100, lengths, 640, 16, 1, BF16, F32, F32, inert=(0, 69)))


@pytest.mark.parametrize("lengths,dim,N,io", [
    ([1900], 5120, 16, BF16),               # pieces of 104 rows
    ([2500, 0, 700], 7680, 8, F16),         # 256
    ([40, 6000], 7680, 16, BF16),           # 480
    ([3000], 7680, 128, F32),               # 240, eight waves
])
def test_scan_long_pieces(lengths, dim, N, io):
    """Pieces of more than 64 rows, up to 19 of a sequence. The oracle walks the first and the
    last channels, which are independent of the others. A piece's sum of v is a chain of its rows
    over the waves and one of the waves: so many half steps relative, since all v are positive."""
    c = scan_inputs(dim + N, lengths, dim, N, 1, io, F32, F32, tail=3)
    rows, blocks = c["x"].shape[0], -(-dim // 64)
    assert len(lengths) * blocks < 400
    piece = -(-(-(-rows * blocks // 1536)) // 8) * 8
    assert 64 < piece < max(lengths)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    gpu_scan(c, state, out)
    keep = torch.tensor(list(range(5)) + list(range(dim - 68, dim)))
    part = {k: v[:, keep] if k in ("x", "z", "dt", "state") else v[keep] if k in ("A", "D", "dt_bias") else v
            for k, v in c.items()}
    waves = 8 if N > 64 else 4
    ref, bound, written, after, s_bound, touched = lh.scan(
        part["x"], part["dt"], part["A"], part["B"], part["C"], part["D"], part["z"],
        part["dt_bias"], True, part["cu"], part["state"], part["slots"].tolist(),
        part["has"].tolist(), join=piece // waves + waves)
    got = out.cpu()
    lh.check("out", got[written][:, keep], ref[written], bound[written])
    assert torch.isnan(got[~written].float()).all()
    got = state.cpu()
    lh.check("state", got[touched][:, keep], after[touched], s_bound[touched])
    assert same(got[~touched], c["state"][~touched])


def test_compact_more_copies_than_workgroups():
    """Every slot of the upper half moves, in 30 caches: 75,000 items over a grid of 65,536."""
    nslots, half = 20000, 10000
    caches = cache_set(110, nslots, [((k % 5 + 1,), F32) for k in range(28)] +
                       [((9,), torch.uint8), ((4,), BF16)])
    assert -(-half // 4) * len(caches) > 65536
    gpu = on_gpu(caches)
    count = torch.cat([torch.zeros(half), torch.arange(half) % 3 + 1]).to(torch.int32)
    on = count.to(DEV)
    remap = ssu.cache_compact(gpu, on)
    ids = torch.arange(nslots, dtype=torch.int32)
    assert torch.equal(remap.cpu(), torch.where(ids >= half, ids - half, -1))
    assert torch.equal(on.cpu(), torch.cat([count[half:], torch.zeros(half, dtype=torch.int32)]))
    for i, (a, b) in enumerate(zip(gpu, caches)):
        assert same(a, torch.cat([b[half:], b[half:]])), i


@pytest.mark.parametrize("N", [8, 16, 32, 64, 128, 256])
@pytest.mark.parametrize("io,dt,state", [(F32, F32, F32), (F32, F32, F16), (F16, F16, F32),
                                         (F16, F32, F16), (BF16, BF16, F32), (BF16, F32, BF16)])
def test_scan_update_aligned_rows(N, io, dt, state):
    """B and C whose rows are 16-byte aligned are read in pieces of up to 16 bytes."""
    batch, dim, groups = 5, 70, 2
    c = scan_inputs(N, [1] * batch, dim, N, groups, io, dt, state, inert=(2,))
    g = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    bc = torch.cat([g["B"].flatten(1), g["C"].flatten(1)], 1)
    B, C = bc[:, :groups * N].unflatten(1, (groups, N)), bc[:, groups * N:].unflatten(1, (groups, N))
    assert bc.stride(0) * bc.element_size() % 16 == B.data_ptr() % 16 == C.data_ptr() % 16 == 0
    ref, bound, written, after, s_bound, touched = lh.scan(
        c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], c["z"], c["dt_bias"], True, c["cu"],
        c["state"], c["slots"].tolist(), [True] * batch)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    ssu.selective_scan_update(g["state"], g["x"], g["dt"], g["A"], B, C, out, D=g["D"], z=g["z"],
                              dt_bias=g["dt_bias"], dt_softplus=True,
                              state_batch_indices=g["slots"])
    got = out.cpu()
    lh.check("out", got[written], ref[written], bound[written])
    assert torch.isnan(got[~written].float()).all()
    got = g["state"].cpu()
    lh.check("state", got[touched], after[touched], s_bound[touched])
    assert same(got[~touched], c["state"][~touched])


@pytest.mark.parametrize("name,width", [("f32", 2), ("f16", 3), ("bf16", 4)])
@pytest.mark.parametrize("batch", [1, 3, 70])
def test_conv_update_aligned_rows(name, width, batch):
    """Rows that are 16-byte aligned, in batches too small for two sequences per wave."""
    io, vec = CONV[name][0], CONV[name][3]
    dim = 64 * vec + 5 * vec
    c = conv_inputs(batch + width, [1] * batch, dim, width, io, strided=False,
                    inert=(1,) if batch > 1 else ())
    ref, bound, written, after = lh.conv(c["x"], c["weight"], c["bias"], c["cu"], c["state"],
                                         c["slots"].tolist(), [True] * batch, True)
    state = c["state"].to(DEV)
    out = torch.full(c["x"].shape, NAN, dtype=io, device=DEV)
    ssu.causal_conv1d_update(state, c["x"].to(DEV), c["weight"].to(DEV), out,
                             bias=c["bias"].to(DEV), state_batch_indices=c["slots"].to(DEV))
    got = out.cpu()
    lh.check("out", got[written], ref[written], bound[written])
    assert torch.isnan(got[~written].float()).all()
    assert same(state, after)
