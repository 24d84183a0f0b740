"""Timed cases of the layer operators around the state update: the short causal
convolution and the per-channel selective scan (prompts and single tokens), and
the slot operations of the state caches (fork, and free + compact + admit).

`run` computes a case with elementary torch operations in fp32 (own False) or
through the package's entry points (own True). `exact` is the definition in fp64,
token by token and slot by slot.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
DEV = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # Three short prompts of a small fp32 layer with odd sizes: latency.
        dict(name="conv prompts, few tokens", op="conv_prompt", nseq=3, tokens=113, dim=1000,
             width=4, io="f32", continued=False),
        # A prefill step of 8 prompts at the widest layer, later pieces of longer prompts.
        dict(name="conv prompts, prefill", op="conv_prompt", nseq=8, tokens=17885, dim=10240,
             width=4, io="bf16", continued=True),
        # The decode step of three requests.
        dict(name="conv step, 3 sequences", op="conv_step", batch=3, dim=5376, width=4, io="f16",
             slots=16),
        # The decode step of a full batch.
        dict(name="conv step, full batch", op="conv_step", batch=512, dim=10240, width=4,
             io="bf16", slots=1024),
        # One long prompt alone: parallel over channels and positions only.
        dict(name="scan, one prompt", op="scan_prompt", nseq=1, tokens=4096, dim=5120, dstate=16,
             groups=1, io="bf16", dt="bf16", state="f32", continued=False, gate=True),
        # A prefill step of 16 prompts of mixed lengths.
        dict(name="scan, prefill", op="scan_prompt", nseq=16, tokens=17885, dim=5120, dstate=16,
             groups=1, io="bf16", dt="f32", state="f32", continued=True, gate=True),
        # The decode step of two requests.
        dict(name="scan step, 2 sequences", op="scan_step", batch=2, dim=5120, dstate=16, groups=1,
             io="f16", dt="f32", state="f32", slots=8, gate=True),
        # The decode step of a full batch.
        dict(name="scan step, full batch", op="scan_step", batch=512, dim=5120, dstate=16,
             groups=1, io="bf16", dt="bf16", state="f32", slots=1024, gate=True),
        # One request answered four ways, two small layers.
        dict(name="fork, one request", op="fork", parents=1, ways=4, layers=2, slots=16, heads=8,
             headdim=64, dstate=16, conv=576, state="f32", io="bf16"),
        # 16 prompts answered four ways each, eight wide layers.
        dict(name="fork, a batch", op="fork", parents=16, ways=4, layers=8, slots=128, heads=128,
             headdim=64, dstate=128, conv=10240, state="f32", io="bf16"),
        # A few of 24 requests end, two small layers with 16-bit states.
        dict(name="compact, few slots", op="compact", live=24, leaving=5, layers=2, slots=32,
             heads=8, headdim=64, dstate=16, conv=576, state="bf16", io="bf16"),
        # A quarter of 192 requests end, four wide layers.
        dict(name="compact, a batch", op="compact", live=192, leaving=48, layers=4, slots=256,
             heads=80, headdim=64, dstate=128, conv=5376, state="f32", io="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv_prompt", "conv_step", "scan_prompt", "scan_step", "fork", "compact"])
    io = rng.choice(["f32", "f16", "bf16"])
    state = rng.choice(["f32", "f32", "f16", "bf16"])
    if op == "conv_prompt":
        dim = _log(rng, 40, 10240)
        return dict(op=op, nseq=_log(rng, 1, 64), tokens=_log(rng, 1, 17885 if io != "f32" else 8900),
                    dim=dim, width=rng.choice([2, 3, 4]), io=io, continued=rng.random() < 0.5)
    if op == "conv_step":
        batch = _log(rng, 1, 512 if io != "f32" else 256)
        return dict(op=op, batch=batch, dim=_log(rng, 40, 10240), width=rng.choice([2, 3, 4]), io=io,
                    slots=batch + rng.randrange(1, 64))
    if op == "scan_prompt":
        dstate, dim = rng.choice([8, 16, 16, 16, 32, 64, 128]), _log(rng, 40, 5120)
        groups = rng.choice([1, 1, 2, 4])
        dim = max(groups, dim // groups * groups)
        most = min(17885, int(17885 * 5120 * 16 / (dim * dstate)))
        return dict(op=op, nseq=_log(rng, 1, 32), tokens=_log(rng, 1, most), dim=dim, dstate=dstate,
                    groups=groups, io=io, dt=rng.choice(["f32", io]), state=state,
                    continued=rng.random() < 0.5, gate=rng.random() < 0.7)
    if op == "scan_step":
        dstate, dim = rng.choice([8, 16, 16, 16, 32, 64, 128]), _log(rng, 40, 5120)
        groups = rng.choice([1, 1, 2, 4])
        dim = max(groups, dim // groups * groups)
        batch = _log(rng, 1, min(512, int(512 * 5120 * 16 / (dim * dstate))))
        return dict(op=op, batch=batch, dim=dim, dstate=dstate, groups=groups, io=io,
                    dt=rng.choice(["f32", io]), state=state, slots=batch + rng.randrange(1, 64),
                    gate=rng.random() < 0.7)
    layers, heads = rng.randrange(1, 7), _log(rng, 2, 80)
    shape = dict(layers=layers, heads=heads, headdim=64, dstate=rng.choice([16, 64, 128]),
                 conv=heads * 64 + rng.choice([32, 128, 256]), state=state, io=io)
    if op == "fork":
        parents, ways = _log(rng, 1, 12), rng.randrange(1, 5)
        return dict(op=op, parents=parents, ways=ways, slots=parents * (ways + 1) + rng.randrange(1, 40),
                    **shape)
    live = _log(rng, 2, 150)
    return dict(op=op, live=live, leaving=_log(rng, 1, max(1, live // 3)), slots=live + rng.randrange(0, 40),
                **shape)


# ------------------------------------------------------------------- the inputs

class _Draws:
    """One seeded generator on the GPU and one on the host."""

    def __init__(self, seed):
        self.gpu = torch.Generator(device=DEV)
        self.gpu.manual_seed(seed)
        self.host = torch.Generator()
        self.host.manual_seed(seed)

    def normal(self, *shape, io="f32"):
        return torch.randn(*shape, generator=self.gpu, device=DEV).to(_TYPES[io])

    def uniform(self, lo, hi, *shape):
        return torch.rand(*shape, generator=self.gpu, device=DEV) * (hi - lo) + lo

    def permutation(self, n, first):
        return torch.randperm(n, generator=self.host)[:first]

    def starts(self, nseq, tokens):
        """cu_seqlens of nseq prompts of mixed lengths, `tokens` in all (none longer than
        needed: with fewer tokens than prompts some are empty)."""
        cuts = torch.rand(nseq, generator=self.host).double() + 0.15
        ends = torch.round(torch.cumsum(cuts, 0) / cuts.sum() * tokens).to(torch.int32)
        return torch.cat([torch.zeros(1, dtype=torch.int32), ends]).to(DEV)


def _inverse_softplus(v):
    return v + torch.log(-torch.expm1(-v))


def prepare(case, seed):
    d, op = _Draws(seed), case["op"]
    s = dict(op=op)
    if op in ("conv_prompt", "conv_step"):
        dim, width, io = case["dim"], case["width"], case["io"]
        rows = case["tokens"] if op == "conv_prompt" else case["batch"]
        # The convolved columns lie inside the wider rows that the layer's projection makes.
        s["x"] = d.normal(rows, 2 * dim, io=io)[:, dim:]
        s["weight"] = d.uniform(-0.5, 0.5, dim, width).to(_TYPES[io])
        s["bias"] = d.normal(dim, io=io) * 0.1
        nseq = case["nseq"] if op == "conv_prompt" else rows
        slots = case["slots"] if op == "conv_step" else nseq + 3
        s["conv_state"] = d.normal(slots, width - 1, dim, io=io)
        s["slots"] = d.permutation(slots, nseq).to(torch.int32).to(DEV)
        if op == "conv_prompt":
            s["cu"] = d.starts(nseq, rows)
            s["has"] = torch.full((nseq,), case["continued"], dtype=torch.bool, device=DEV)
        return s
    if op in ("scan_prompt", "scan_step"):
        dim, N, G, io = case["dim"], case["dstate"], case["groups"], case["io"]
        rows = case["tokens"] if op == "scan_prompt" else case["batch"]
        nseq = case["nseq"] if op == "scan_prompt" else rows
        slots = case["slots"] if op == "scan_step" else nseq + 3
        # x comes from the convolution, z is one half of the projection's rows, B and C lie
        # behind the step's low-rank part in one narrow row.
        rank = max(8, dim // 16 // 8 * 8)
        bc = d.normal(rows, rank + 2 * G * N, io=io)
        s["x"] = d.normal(rows, dim, io=io)
        s["z"] = d.normal(rows, 2 * dim, io=io)[:, dim:] if case["gate"] else None
        s["B"] = bc[:, rank:rank + G * N].unflatten(1, (G, N))
        s["C"] = bc[:, rank + G * N:].unflatten(1, (G, N))
        s["dt"] = d.normal(rows, dim, io=case["dt"])
        s["dt_bias"] = _inverse_softplus(torch.exp(d.uniform(math.log(1e-3), math.log(0.1), dim)))
        s["A"] = -torch.exp(d.uniform(0.0, math.log(16.0), dim, N))
        s["D"] = d.normal(dim)
        s["state"] = d.normal(slots, dim, N, io=case["state"])
        s["slots"] = d.permutation(slots, nseq).to(torch.int32).to(DEV)
        if op == "scan_prompt":
            s["cu"] = d.starts(nseq, rows)
            s["has"] = torch.full((nseq,), case["continued"], dtype=torch.bool, device=DEV)
        return s
    slots = case["slots"]
    s["caches"] = []
    for _ in range(case["layers"]):
        s["caches"].append(d.normal(slots, 3, case["conv"], io=case["io"]))
        s["caches"].append(d.normal(slots, case["heads"], case["headdim"], case["dstate"],
                                    io=case["state"]))
    refcount = torch.zeros(slots, dtype=torch.int32)
    if op == "fork":
        parents = d.permutation(slots, case["parents"])
        refcount[parents] = 1
        s["parents"] = parents.repeat_interleave(case["ways"]).to(torch.int32).to(DEV)
    else:
        refcount[:case["live"]] = 1
        order = d.permutation(case["live"], case["live"]).to(torch.int32)
        s["leaving"] = order[:case["leaving"]].contiguous().to(DEV)
        s["staying"] = order[case["leaving"]:].contiguous().to(DEV)
        s["admit"] = case["leaving"]
    s["refcount"] = refcount.to(DEV)
    return s


# ---------------------------------------------------------- the plain operators

def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _rows(cu, rows):
    """The sequence of each row, and the row's position in it."""
    t = torch.arange(rows, device=cu.device)
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    return seq, t - cu.long()[seq]


def _conv_prompt(x, weight, bias, cu, conv_state, slots, has):
    rows, width = x.shape[0], weight.shape[1]
    back = torch.arange(width - 1, -1, -1, device=x.device)
    seq, pos = _rows(cu, rows)
    history = conv_state[slots.long()].float() * has[:, None, None]
    xf, begin, length = x.float(), cu.long()[:-1], (cu[1:] - cu[:-1]).long()
    # Value at position p of sequence b: the row begin + p, or for p < 0 the history.
    at = pos[:, None] - back
    window = torch.where((at >= 0)[..., None], xf[(torch.arange(rows, device=x.device)[:, None] - back).clamp(min=0)],
                         history[seq[:, None], (at + width - 1).clamp(max=width - 2)])
    out = _silu((window * weight.float().t()).sum(1) + bias.float())
    last = length[:, None] - back[:-1]
    kept = torch.where((last >= 0)[..., None], xf[(begin[:, None] + last).clamp(min=0, max=max(rows - 1, 0))],
                       history[torch.arange(len(slots), device=x.device)[:, None], (last + width - 1).clamp(max=width - 2)])
    # An empty sequence leaves its slot as it is.
    kept = torch.where((length > 0)[:, None, None], kept, conv_state[slots.long()].float())
    conv_state[slots.long()] = kept.to(conv_state.dtype)
    return out.to(x.dtype)


def _conv_step(x, weight, bias, conv_state, slots):
    window = torch.cat([conv_state[slots.long()].float(), x.float()[:, None]], 1)
    out = _silu((window * weight.float().t()).sum(1) + bias.float())
    conv_state[slots.long()] = window[:, 1:].to(conv_state.dtype)
    return out.to(x.dtype)


def _scan_terms(x, dt, A, B, dt_bias):
    """The decay exp(dt A) and the input dt x B of each row, channel and state element."""
    per = x.shape[1] // B.shape[1]
    step = _softplus(dt.float() + dt_bias)
    decay = torch.exp(step[..., None] * A)
    return decay, (step * x.float())[..., None] * B.float().repeat_interleave(per, 1)


def _scan_out(h, x, C, D, z):
    y = (h * C.float().repeat_interleave(x.shape[1] // C.shape[1], 1)).sum(-1) + D * x.float()
    return (y if z is None else y * _silu(z.float())).to(x.dtype)


def _scan_prompt(x, dt, A, B, C, D, z, dt_bias, cu, state, slots, has):
    """h_t = decay_t h_{t-1} + input_t inside each sequence, by doubling: after the step with
    shift s, (decay_t, input_t) hold the composition of the last 2 s maps up to t. A
    sequence's first map holds the entering state and has decay zero, so none reaches past it."""
    decay, h = _scan_terms(x, dt, A, B, dt_bias)
    begin, end = cu.long()[:-1], cu.long()[1:]
    filled = end > begin
    first = begin.clamp(max=max(x.shape[0] - 1, 0))
    entering = state[slots.long()].float() * (has & filled)[:, None, None]
    h.index_add_(0, first, decay[first] * entering)
    decay[first] *= (~filled)[:, None, None]
    shift = 1
    while shift < x.shape[0]:
        h[shift:] += decay[shift:] * h[:-shift]
        decay = torch.cat([decay[:shift], decay[shift:] * decay[:-shift]])
        shift *= 2
    final = torch.where(filled[:, None, None], h[(end - 1).clamp(min=0)], state[slots.long()].float())
    state[slots.long()] = final.to(state.dtype)
    return _scan_out(h, x, C, D, z)


def _scan_step(x, dt, A, B, C, D, z, dt_bias, state, slots):
    decay, h = _scan_terms(x, dt, A, B, dt_bias)
    h = state[slots.long()].float() * decay + h
    state[slots.long()] = h.to(state.dtype)
    return _scan_out(h, x, C, D, z)


def _lowest_free(refcount, n):
    """The n lowest slots with no user."""
    return torch.sort(refcount != 0, stable=True).indices[:n]


def _move(caches, src, dst):
    for c in caches:
        c[dst] = c[src]


def _fork(caches, refcount, parents):
    children = _lowest_free(refcount, len(parents))
    refcount[children] = 1
    _move(caches, parents.long(), children)
    return children.to(torch.int32)


def _free(refcount, slots):
    refcount.index_add_(0, slots, torch.full_like(slots, -1))


def _compact(caches, refcount):
    ids = torch.arange(len(refcount), device=refcount.device)
    live = refcount > 0
    count = live.sum()
    holes, movers = ((~live) & (ids < count)).nonzero()[:, 0], (live & (ids >= count)).nonzero()[:, 0]
    _move(caches, movers, holes)
    refcount[holes] = refcount[movers]
    refcount[movers] = 0
    remap = torch.where(live, ids, -1)
    remap[movers] = holes
    return remap.to(torch.int32)


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        return _run_own(op, s)
    if op == "conv_prompt":
        out = _conv_prompt(s["x"], s["weight"], s["bias"], s["cu"], s["conv_state"], s["slots"], s["has"])
        return dict(out=out, conv_state=s["conv_state"])
    if op == "conv_step":
        out = _conv_step(s["x"], s["weight"], s["bias"], s["conv_state"], s["slots"])
        return dict(out=out, conv_state=s["conv_state"])
    if op == "scan_prompt":
        out = _scan_prompt(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                           s["cu"], s["state"], s["slots"], s["has"])
        return dict(out=out, state=s["state"])
    if op == "scan_step":
        out = _scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                         s["state"], s["slots"])
        return dict(out=out, state=s["state"])
    if op == "fork":  # the answers start, and end: their slots go back
        children = _fork(s["caches"], s["refcount"], s["parents"])
        _free(s["refcount"], children)
        return dict(children=children, refcount=s["refcount"], caches=s["caches"])
    # Requests end, those that stay move together, new ones are admitted behind them.
    _free(s["refcount"], s["leaving"])
    remap = _compact(s["caches"], s["refcount"])
    admitted = _lowest_free(s["refcount"], s["admit"])
    s["refcount"][admitted] = 1
    return dict(slots=remap[s["staying"].long()], admitted=admitted.to(torch.int32), remap=remap,
                refcount=s["refcount"], caches=s["caches"])


def _run_own(op, s):
    import selective_state_update_ssu_amd as ssu
    if op == "conv_prompt":
        out = ssu.causal_conv1d_varlen(s["conv_state"], s["x"], s["weight"], s["cu"], bias=s["bias"],
                                       has_initial_state=s["has"], state_batch_indices=s["slots"])
        return dict(out=out, conv_state=s["conv_state"])
    if op == "conv_step":
        out = ssu.causal_conv1d_update(s["conv_state"], s["x"], s["weight"], bias=s["bias"],
                                       state_batch_indices=s["slots"])
        return dict(out=out, conv_state=s["conv_state"])
    if op == "scan_prompt":
        out = ssu.selective_scan_varlen(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], s["cu"],
                                        D=s["D"], z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True,
                                        has_initial_state=s["has"], state_batch_indices=s["slots"])
        return dict(out=out, state=s["state"])
    if op == "scan_step":
        out = ssu.selective_scan_update(s["state"], s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"],
                                        z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True,
                                        state_batch_indices=s["slots"])
        return dict(out=out, state=s["state"])
    if op == "fork":
        children = ssu.cache_fork(s["caches"], s["refcount"], s["parents"])
        ssu.cache_free(s["refcount"], children)
        return dict(children=children, refcount=s["refcount"], caches=s["caches"])
    ssu.cache_free(s["refcount"], s["leaving"])
    remap = ssu.cache_compact(s["caches"], s["refcount"])
    admitted = ssu.cache_alloc(s["refcount"], s["admit"])
    return dict(slots=remap[s["staying"].long()], admitted=admitted, remap=remap,
                refcount=s["refcount"], caches=s["caches"])


# ------------------------------------------------------------------- accounting

def work(case):
    op = case["op"]
    if op in ("conv_prompt", "conv_step"):
        b, dim, width = _SIZE[case["io"]], case["dim"], case["width"]
        rows = case["tokens"] if op == "conv_prompt" else case["batch"]
        nseq = case["nseq"] if op == "conv_prompt" else rows
        reads = 1 if op == "conv_step" or case["continued"] else 0
        state = nseq * (width - 1) * dim * b * (1 + reads)
        return dict(bytes=2 * rows * dim * b + state + dim * (width + 1) * b + nseq * 9,
                    flops=rows * dim * (2 * width + 4))
    if op in ("scan_prompt", "scan_step"):
        b, dim, N, G = _SIZE[case["io"]], case["dim"], case["dstate"], case["groups"]
        rows = case["tokens"] if op == "scan_prompt" else case["batch"]
        nseq = case["nseq"] if op == "scan_prompt" else rows
        reads = 1 if op == "scan_step" or case["continued"] else 0
        row = dim * b * (3 if case["gate"] else 2) + dim * _SIZE[case["dt"]] + 2 * G * N * b
        state = nseq * dim * N * _SIZE[case["state"]] * (1 + reads)
        return dict(bytes=rows * row + state + dim * (N + 2) * 4 + nseq * 9,
                    flops=rows * dim * (7 * N + 12))
    slot = case["layers"] * (3 * case["conv"] * _SIZE[case["io"]] +
                             case["heads"] * case["headdim"] * case["dstate"] * _SIZE[case["state"]])
    if op == "fork":
        n = case["parents"] * case["ways"]
        # Each parent is read once, each child written once.
        return dict(bytes=(case["parents"] + n) * slot + 8 * case["slots"] + 8 * n, flops=case["slots"])
    # Of the leaving slots, live - leaving of `live` lie below the new end, on average.
    moved = max(1, round(case["leaving"] * (case["live"] - case["leaving"]) / case["live"]))
    return dict(bytes=2 * moved * slot + 12 * case["slots"] + 8 * case["live"], flops=case["slots"])


# ----------------------------------------------------------- the definitions, fp64

def _gate64(z):
    return z * torch.sigmoid(z)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "conv_prompt" or op == "conv_step":
        return _conv64(s, op)
    if op == "scan_prompt" or op == "scan_step":
        return _scan64(s, op)
    return _slots64(s, op)


def _conv64(s, op):
    x, w, state = s["x"].double(), s["weight"].double(), s["conv_state"].double()
    rows, width, slots = x.shape[0], w.shape[1], s["slots"].tolist()
    cu = s["cu"].tolist() if op == "conv_prompt" else list(range(rows + 1))
    has = s["has"].tolist() if op == "conv_prompt" else [True] * rows
    out = torch.empty_like(x)
    for b, slot in enumerate(slots):
        if cu[b + 1] == cu[b]:
            continue
        before = state[slot] if has[b] else torch.zeros_like(state[slot])
        line = torch.cat([before, x[cu[b]:cu[b + 1]]])
        n = cu[b + 1] - cu[b]
        acc = s["bias"].double().expand(n, -1).clone()
        for k in range(width):
            acc += line[k:k + n] * w[:, k]
        out[cu[b]:cu[b + 1]] = _gate64(acc)
        state[slot] = line[-(width - 1):]
    return dict(out=out, conv_state=state)


def _scan64(s, op):
    x, state, slots = s["x"].double(), s["state"].double(), s["slots"].long()
    rows, dim = x.shape
    cu = s["cu"].long() if op == "scan_prompt" else torch.arange(rows + 1, device=DEV)
    begin, length = cu[:-1], cu[1:] - cu[:-1]
    v = torch.nn.functional.softplus(s["dt"].double() + s["dt_bias"].double(), threshold=700.0)
    A = s["A"].double()
    per = dim // s["B"].shape[1]
    B, C = s["B"].double(), s["C"].double()
    out = torch.zeros_like(x)
    h = state[slots]
    if op == "scan_prompt":
        h = h * s["has"][:, None, None]
    for t in range(int(length.max())):
        on = t < length
        at = (begin + t).clamp(max=rows - 1)
        step = v[at]
        grown = h * torch.exp(step[..., None] * A) + (
            (step * x[at])[..., None] * B[at].repeat_interleave(per, 1))
        h = torch.where(on[:, None, None], grown, h)
        y = (h * C[at].repeat_interleave(per, 1)).sum(-1)
        out.index_add_(0, at, torch.where(on[:, None], y, torch.zeros_like(y)))
    out += s["D"].double() * x
    if s["z"] is not None:
        out *= _gate64(s["z"].double())
    state[slots] = torch.where((length > 0)[:, None, None], h, state[slots])
    return dict(out=out, state=state)


def _slots64(s, op):
    users = s["refcount"].tolist()
    caches = [c.double() for c in s["caches"]]

    def admit():
        slot = users.index(0)
        users[slot] = 1
        return slot

    def copy(pairs):
        for c in caches:
            for a, b in pairs:
                c[b] = c[a]

    def whole(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    if op == "fork":
        parents = s["parents"].tolist()
        children = [admit() for _ in parents]
        copy(list(zip(parents, children)))
        for slot in children:
            users[slot] -= 1
        return dict(children=whole(children), refcount=whole(users), caches=caches)
    for slot in s["leaving"].tolist():
        users[slot] -= 1
    remap = [i if n > 0 else -1 for i, n in enumerate(users)]
    count = sum(n > 0 for n in users)
    pairs, low = [], 0
    for high in range(count, len(users)):
        if users[high] > 0:
            while users[low] > 0:
                low += 1
            pairs.append((high, low))
            users[low], users[high], remap[high] = users[high], 0, low
    copy(pairs)
    admitted = [admit() for _ in range(s["admit"])]
    return dict(slots=whole([remap[i] for i in s["staying"].tolist()]), admitted=whole(admitted),
                remap=whole(remap), refcount=whole(users), caches=caches)
