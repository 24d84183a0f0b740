"""Plain fp64 forms of the operators of include/attention.h and include/batch.h on the CPU,
token by token, with running bounds of what the kernels' arithmetic may be off by.
u = 2^-24 is half a step of fp32.

Bounds of linear attention. Per head and value row, N bounds the magnitudes that meet in
a state row: N <- e^g N + |r| |k| (2-norms of key vectors, exact r). One row's arithmetic is off
by at most c u times its magnitudes, where c counts what is summed and rounded on the way: key_dim
terms of a product with the state, up to 64 rows of a chunk twice (scores, values), 16 terms of a
diagonal block's inverse against right-hand sides of up to beta (|v| + |k| N), and a few single
roundings (the parts of a product leave out less than 2 u of it): c = key_dim + 200. What reaches
only a 16-bit out goes in as two parts of 8 bits, which leaves out 2^-17 of either factor: 256 u. An
exponential of a sum x of decays is off by 3 |x| u relative, |x| at most the decays of 64 rows, and
no more than 88 of them before it is 0 in fp32. The errors E of a state row (2-norm)
come forward through e^g (1 - beta k k^T), whose norm is at most e^g where beta |k|^2 lies in
[0, 2], so that
    E <- e^g E + c u (e^g N + |r| |k| + beta |k| (|v| + |k| N))
    out: scale |q| (E + (c + 256 for 16 bits) u N), half a step of its type on top.
"""
import torch

from layer_harness import TINY, U, f64, ranges, stored


def window_decay(g, begin, end):
    """The largest sum of |g| over 64 rows of one sequence, per head, at most 88."""
    total = torch.cumsum(g[begin:end].abs(), 0)
    total = torch.cat([torch.zeros_like(total[:1]), total])
    n = total.shape[0]
    lo = torch.arange(n) - 64
    return (total - total[lo.clamp(min=0)]).max(0).values.clamp(max=88.0)


def attention(q, k, v, decay, beta, scale, cu, state, begin_of, end_of, has=None):
    """(out, its bound, rows written, state, its bound, slots written). begin_of(b): the slot
    that sequence b starts from or None (inert); end_of(b, t, last): the slot of the state after
    its row t, or None. `has`: sequences that start from their slot (None: all)."""
    io, st = v.dtype, state.dtype
    q, k, v, decay, beta = (f64(x) for x in (q, k, v, decay, beta))
    rows, H, V = v.shape
    per, K = H // q.shape[1], q.shape[2]
    g = decay.expand(rows, H).clamp(min=-300.0)
    more = 0.0 if io == torch.float32 else 256 * U
    state = f64(state).clone()
    before = state.clone()
    s_bound = torch.zeros_like(state)
    out, bound = torch.zeros_like(v), torch.zeros_like(v)
    written = torch.zeros(rows, dtype=torch.bool)
    touched = torch.zeros(state.shape[0], dtype=torch.bool)
    for b in range(len(cu) - 1):
        begin, end, slot = cu[b], cu[b + 1], begin_of(b)
        if slot is None or not 0 <= begin < end <= rows:
            continue
        S = before[slot].clone() if has is None or has[b] else torch.zeros(H, V, K, dtype=torch.float64)
        N, E = S.norm(dim=-1), torch.zeros(H, V, dtype=torch.float64)
        c = ((K + 200 + 3 * window_decay(g, begin, end)) * U)[:, None]
        for t in range(begin, end):
            kt, qt = k[t].repeat_interleave(per, 0), q[t].repeat_interleave(per, 0)
            kn, qn = kt.norm(dim=-1)[:, None], qt.norm(dim=-1)[:, None]
            e = torch.exp(g[t])[:, None]
            S = S * e[..., None]
            r, be = v[t], 0.0
            if beta is not None:
                be = beta[t][:, None]
                r = be * (r - (S * kt[:, None]).sum(-1))
            S = S + r[..., None] * kt[:, None]
            local = e * N + r.abs() * kn + be * kn * (v[t].abs() + kn * e * N)
            E = e * E + c * local
            N = e * N + r.abs() * kn
            y = scale * (S * qt[:, None]).sum(-1)
            out[t], bound[t] = y, stored(abs(scale) * qn * (E + (c + more) * N), y, io)
            written[t] = True
            to = end_of(b, t - begin, t + 1 == end)
            if to is not None:
                state[to], touched[to] = S, True
                s_bound[to] = stored(E[..., None].expand_as(S), S, st)
    return out, bound + TINY[io], written, state, s_bound, touched


def in_place(cu, slots, nslots, rows, pad=-1):
    """begin_of and end_of of prompts and single tokens."""
    valid = {b: slot for b, _, _, slot in ranges(cu, len(cu) - 1, rows, slots, nslots, pad)}
    return valid.get, lambda b, t, last: valid.get(b) if last else None


def through_tables(cu, src, dst, accepted, nslots, pad=-1):
    """begin_of and end_of of windows: src and dst are lists of rows (dst may be None)."""
    def real(s):
        return s if s != pad and 0 <= s < nslots else None

    def begin_of(b):
        n = 1 if accepted is None else accepted[b]
        return real(src[b][n - 1]) if 1 <= n <= len(src[b]) else None

    def end_of(b, t, last):
        if dst is None:
            return begin_of(b) if last else None
        return real(dst[b][t]) if t < len(dst[b]) else None

    return begin_of, end_of


# ------------------------------------------------------------------------ batches

def verify(target, drafts, uniforms, cu, probs, temperature):
    """(tokens, num_accepted, slack): slack is, per sequence, the least distance of a decision from
    its border, relative to the probabilities in it."""
    nseq, window = len(cu) - 1, drafts.shape[1]
    rows, vocab = target.shape
    tokens, counts, slack = [], [], []
    for b in range(nseq):
        begin, n = cu[b], cu[b + 1] - cu[b] - 1
        if begin < 0 or cu[b + 1] > rows or n < 0 or n > window:
            tokens.append([-1] * (window + 1))
            counts.append(0)
            slack.append(1.0)
            continue
        got, least = [], 1.0
        for i in range(n + 1):
            p = target[begin + i].double()
            if temperature is not None:
                p = torch.where(torch.isnan(p), -float("inf"), p)
                t = float(temperature[b])
                if t > 0:
                    most = p.max()
                    e = torch.where(p == most, 1.0, torch.exp((p - most) / t))
                    p = e / e.sum() if most > -float("inf") else torch.zeros_like(p)
                else:
                    p = torch.zeros_like(p).index_fill(0, (p == p.max()).nonzero()[0], 1.0)
            p = torch.where(p > 0, p, 0.0)
            w = p
            if i < n:
                x = int(drafts[b, i])
                q = torch.zeros_like(p)
                if probs is not None:
                    q = probs[b, i].double()
                elif 0 <= x < vocab:
                    q[x] = 1.0
                if 0 <= x < vocab:
                    a, c = float(uniforms[b, i]) * float(q[x]), float(p[x])
                    if temperature is not None and float(temperature[b]) > 0:
                        least = min(least, abs(a - c) / max(a, c, 1e-300))
                    if a < c:
                        got.append(x)
                        continue
                w = torch.where(p - q > 0, p - q, 0.0)
                if not float(w.sum()) > 0:
                    w = p
            sums = torch.cumsum(w, 0)
            total = float(sums[-1])
            if not total > 0:
                got.append(-1)
                break
            aim = float(uniforms[b, window]) * total
            hit = ((sums > aim) & (w > 0)).nonzero()
            token = int(hit[0]) if len(hit) else int((w > 0).nonzero()[-1])
            low = float(sums[token] - w[token])
            least = min(least, abs(float(sums[token]) - aim) / total,
                        1.0 if low == 0 else abs(aim - low) / total)
            got.append(token)
            break
        tokens.append(got + [-1] * (window + 1 - len(got)))
        counts.append(len(got))
        slack.append(least)
    return tokens, counts, slack


def plan(lengths, rows, chunk, nchunks, context, table, block):
    """The tables of a batch as lists."""
    cu, seq, pos, begin, owner, last = [0], [], [], [], [], []
    for b, n in enumerate(max(x, 0) for x in lengths):
        if chunk:
            for first in range(0, max(n, 1), chunk):
                begin.append(cu[-1] + first)
                owner.append(b)
            last.append(len(owner) - 1 if len(owner) <= nchunks else -1)
        seq += [b] * n
        pos += [(context[b] if context else 0) + i for i in range(n)]
        cu.append(cu[-1] + n)
    behind = max(rows - len(seq), 0)
    found = dict(cu_seqlens=cu, row_seq=(seq + [-1] * behind)[:rows],
                 row_pos=(pos + [-1] * behind)[:rows])
    if chunk:
        found["cu_chunk_seqlens"] = (begin + [cu[-1]] * (nchunks + 1))[:nchunks + 1]
        found["seq_idx"] = (owner + [-1] * nchunks)[:nchunks]
        found["last_chunk_indices"] = last
    if table is not None:
        def place(b, p):
            if b < 0 or p < 0 or p // block >= len(table[b]) or table[b][p // block] < 0:
                return -1
            return table[b][p // block] * block + p % block
        found["row_slots"] = [place(b, p) for b, p in zip(found["row_seq"], found["row_pos"])]
    return found
