"""Plain fp64 forms of the operators of include/layer.h on the CPU, token by token and
slot by slot, with running bounds of what fp32 arithmetic and one rounding per
stored value may be off by. u = 2^-24 is half a step of fp32.

Bounds. The hardware's exp2, log2 and reciprocal are within one step (2 u) of their
argument's result, and an argument of size a in an exponential adds a few a u.
  silu(z)       relative (6 + 3 |z|) u
  softplus(d)   relative (12 + 3 |d|) u, with the rounding of d = dt + bias in it
  exp(v A)      relative |v A| (r + 43 u) + 4 u, r that of v; 40 u of it cover the
                join of pieces of up to 128 rows, whose sums of v are four chains of
                at most 32 values, joined by 3 more additions; for longer pieces the
                caller of scan() names the length of the chains as `join`
  sums          n terms: n u times the sum of the magnitudes
Every stored value adds half a step of its type, and where that is coarser half
of the type's smallest subnormal.
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}


def f64(t):
    return None if t is None else t.detach().cpu().double()


def stored(err, ref, dtype):
    """Bound of a value within err of ref that was rounded to dtype."""
    return err + HALF[dtype] * (ref.abs() + err) + TINY[dtype]


def silu(z):
    return z * torch.sigmoid(z)


def silu_rel(z):
    return (6 + 3 * z.abs()) * U


def check(name, got, ref, bound):
    got = got.detach().cpu().double()
    err = (got - ref).abs()
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(err[bad].max()),
                           float((err / bound)[bad].max()), bad.nonzero()[0].tolist())
    return float((err / bound).max()) if err.numel() else 0.0


def ranges(cu, nseq, rows, slots, nslots, pad=-1):
    """(b, begin, end, slot) of every sequence that takes part."""
    for b in range(nseq):
        begin, end = cu[b], cu[b + 1]
        slot = slots[b] if slots is not None else b
        if slot == pad or not 0 <= slot < nslots or not 0 <= begin <= end <= rows:
            continue
        yield b, begin, end, slot


# ---------------------------------------------------------------- convolution

def conv(x, weight, bias, cu, state, slots, has, act):
    """(out, bound, rows written, state) of a call; state is exact (copied values)."""
    io = x.dtype
    x, weight, bias = f64(x), f64(weight), f64(bias)
    rows, dim = x.shape
    width = weight.shape[1]
    state = state.detach().cpu().clone()
    out, bound = torch.zeros(rows, dim, dtype=torch.float64), torch.zeros(rows, dim, dtype=torch.float64)
    written = torch.zeros(rows, dtype=torch.bool)
    xt = x.to(state.dtype)
    for b, begin, end, slot in ranges(cu, len(cu) - 1, rows, slots, state.shape[0]):
        if begin == end:
            continue
        before = state[slot].double() if has[b] else torch.zeros(width - 1, dim, dtype=torch.float64)
        line = torch.cat([before, x[begin:end]])
        n = end - begin
        acc = torch.zeros(n, dim, dtype=torch.float64)
        mag = torch.zeros(n, dim, dtype=torch.float64)
        if bias is not None:
            acc, mag = acc + bias, mag + bias.abs()
        for k in range(width):
            term = line[k:k + n] * weight[:, k]
            acc, mag = acc + term, mag + term.abs()
        err = (width + 1) * U * mag
        if act:
            err = 1.1 * err + silu(acc).abs() * silu_rel(acc)
            acc = silu(acc)
        out[begin:end], bound[begin:end] = acc, stored(err, acc, io)
        written[begin:end] = True
        kept = torch.cat([state[slot] if has[b] else torch.zeros_like(state[slot]), xt[begin:end]])
        state[slot] = kept[-(width - 1):]
    return out, bound, written, state


# ------------------------------------------------------------------------ scan

def scan(x, dt, A, B, C, D, z, dt_bias, softplus, cu, state, slots, has, join=40):
    """(out, bound, rows written, state, its bound, slots written)."""
    io, st = x.dtype, state.dtype
    x, dt, A, B, C, D, z, dt_bias = (f64(t) for t in (x, dt, A, B, C, D, z, dt_bias))
    rows, dim = x.shape
    G, N = B.shape[1:]
    per = dim // G
    state = f64(state)
    s_bound = torch.zeros_like(state)
    out, bound = torch.zeros(rows, dim, dtype=torch.float64), torch.zeros(rows, dim, dtype=torch.float64)
    written = torch.zeros(rows, dtype=torch.bool)
    touched = torch.zeros(state.shape[0], dtype=torch.bool)
    for b, begin, end, slot in ranges(cu, len(cu) - 1, rows, slots, state.shape[0]):
        if begin == end:
            continue
        s = state[slot].clone() if has[b] else torch.zeros(dim, N, dtype=torch.float64)
        e_s = torch.zeros_like(s)
        for t in range(begin, end):
            d = dt[t] + (dt_bias if dt_bias is not None else 0)
            r_v = U * torch.ones_like(d)
            v = d
            if softplus:
                v = torch.nn.functional.softplus(d, threshold=700.0)
                r_v = (12 + 3 * d.abs()) * U
            elif dt_bias is not None:
                # The rounding of the sum, absolute in |d|, is relative u of d.
                r_v = 2 * U * torch.ones_like(d)
            arg = v[:, None] * A
            e = torch.exp(arg)
            r_e = arg.abs() * (r_v[:, None] + (3 + join) * U) + 4 * U
            u = (v * x[t])[:, None] * B[t].repeat_interleave(per, 0)
            e_s = e * e_s * (1 + r_e) + (e * s).abs() * (r_e + U) + u.abs() * (r_v[:, None] + 4 * U)
            s = e * s + u
            Ct = C[t].repeat_interleave(per, 0)
            terms = Ct * s
            y, mag = terms.sum(1), terms.abs().sum(1)
            if D is not None:
                y, mag = y + D * x[t], mag + (D * x[t]).abs()
            err = (Ct.abs() * e_s).sum(1) + (N + 4) * U * mag
            if z is not None:
                gate = silu(z[t])
                err = err * gate.abs() * (1 + silu_rel(z[t])) + (y * gate).abs() * silu_rel(z[t])
                y = y * gate
            out[t], bound[t] = y, stored(err, y, io)
            written[t] = True
        state[slot], s_bound[slot] = s, stored(e_s, s, st)
        touched[slot] = True
    return out, bound, written, state, s_bound, touched


# ----------------------------------------------------------------------- slots

def alloc(refcount, n):
    ids = [i for i, r in enumerate(refcount) if r <= 0][:n]
    for i in ids:
        refcount[i] = 1
    return ids + [-1] * (n - len(ids))


def adjust(refcount, slots, delta):
    for s in slots:
        if 0 <= s < len(refcount) and refcount[s] > 0:
            refcount[s] += delta


def copy(caches, src, dst):
    for c in caches:
        for a, b in zip(src, dst):
            if 0 <= a < len(c) and 0 <= b < len(c):
                c[b] = c[a]


def compact(caches, refcount):
    used = [i for i, r in enumerate(refcount) if r > 0]
    k = len(used)
    remap = [i if r > 0 else -1 for i, r in enumerate(refcount)]
    leave = [i for i in used if i >= k]
    fill = [i for i in range(k) if refcount[i] <= 0]
    assert len(leave) == len(fill)
    copy(caches, leave, fill)
    for a, b in zip(leave, fill):
        remap[a], refcount[b], refcount[a] = b, refcount[a], 0
    return remap


def starts(lengths, first=0):
    cu = [first]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu
