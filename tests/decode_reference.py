"""Plain 64-bit statements of the operators around the verify step (beam
selection, state reordering, slot planning, path commit), on the CPU."""
import numpy as np


def beam_select(x, scores, K, finished=None, eos=0):
    """x [B, W, V] and scores [B, W] as float64 (the stored values) ->
    (scores [B, K] float64, parents, tokens [B, K], values of all candidates
    [B, W V]).  A request with an undefined score or row: NaN, -1, -1."""
    B, W, V = x.shape
    s_out = np.full((B, K), -np.inf)
    p_out = np.full((B, K), -1, np.int32)
    t_out = np.full((B, K), -1, np.int32)
    values = np.full((B, W * V), -np.inf)
    for b in range(B):
        c = np.full((W, V), -np.inf)
        bad = False
        for w in range(W):
            s = scores[b, w]
            if np.isnan(s) or s == np.inf:
                bad = True
            elif s > -np.inf:
                if finished is not None and finished[b, w]:
                    c[w, eos] = s
                    continue
                row = x[b, w]
                if np.isnan(row).any() or (row == np.inf).any():
                    bad = True
                    continue
                m = row.max()
                if m == -np.inf:
                    continue
                z = np.exp(row - m)
                c[w] = s + (row - m) - np.log(np.sort(z).sum())
        if bad:
            s_out[b] = np.nan
            values[b] = np.nan
            continue
        flat = c.ravel()
        values[b] = flat
        order = np.argsort(-flat, kind="stable")[:K]
        n = int((flat[order] > -np.inf).sum())
        s_out[b, :n] = flat[order[:n]]
        p_out[b, :n] = order[:n] // V
        t_out[b, :n] = order[:n] % V
    return s_out, p_out, t_out, values


def reorder_states(src, dst, parents, lengths, time_dim=3):
    """dst with the reordered rows of src written (both numpy arrays)."""
    out = dst.copy()
    T = src.shape[time_dim]
    W = parents.shape[1]
    for b in range(parents.shape[0]):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        for i in range(W):
            p = int(parents[b, i])
            if 0 <= p < W:
                if time_dim == 3:
                    out[:, b, i, :n] = src[:, b, p, :n]
                else:
                    out[:, b, i, :, :n] = src[:, b, p, :, :n]
    return out


def commit_path(src, al, nodes, dst, dst_slots, src_slots=None):
    out = dst.copy()
    N1 = src.shape[2] if src_slots is None else src_slots.shape[1]
    for b in range(len(al)):
        for j in range(min(int(al[b]), nodes.shape[1]) + 1):
            c = 0 if j == 0 else int(nodes[b, j - 1])
            d = int(dst_slots[b, j])
            if not 0 <= c < N1 or not 0 <= d < dst.shape[1]:
                continue
            if src_slots is None:
                out[:, d] = src[:, b, c]
            elif 0 <= int(src_slots[b, c]) < src.shape[1]:
                out[:, d] = src[:, int(src_slots[b, c])]
    return out


def plan_slots(lens, tables, held, ring, state, bs, k=0, offsets=None, total=0, accept=None, release=None, fill=-7):
    """Returns (lens, held, state, positions, slots, tables, ring); rows that
    are not written hold `fill`."""
    B, cols = tables.shape
    tables, ring = tables.copy(), ring.copy()
    head, count = int(state[0]), int(state[1])
    cap = len(ring)
    rows = B * (k + 1) if offsets is None else B + total
    pos, slots = np.full(rows, fill, np.int64), np.full(rows, fill, np.int64)
    new_lens, new_held = np.zeros(B, np.int32), np.zeros(B, np.int32)
    asked = taken = returned = 0
    free = [int(ring[(head + i) % cap]) for i in range(count)]
    for b in range(B):
        if offsets is None:
            n, row0 = k + 1, b * (k + 1)
        else:
            o0, o1 = int(offsets[b]), int(offsets[b + 1])
            ok = 0 <= o0 <= o1 <= min(int(offsets[B]), total) and o1 - o0 <= k
            n, row0 = (o1 - o0 + 1, o0 + b) if ok else (0, 0)
        h = min(max(int(held[b]), 0), cols)
        if release is not None and release[b]:
            for i in range(h):
                if count + returned < cap:
                    ring[(head + count + returned) % cap] = tables[b, i]
                    returned += 1
            pos[row0:row0 + n] = -1
            slots[row0:row0 + n] = -1
            continue
        length = max(int(lens[b]), 0)
        if accept is not None and accept[b] >= 0:
            length += int(accept[b]) + 1
        length = min(length, 2**31 - 1)
        need = -(-(length + n) // bs) if n else 0
        grow = need - h if h < need <= cols else 0
        asked += grow
        if asked <= count:
            tables[b, h:h + grow] = free[taken:taken + grow]
            taken += grow
        else:
            grow = 0
        new_lens[b], new_held[b] = length, h + grow
        for j in range(n):
            p = length + j
            pos[row0 + j] = p
            page = p // bs
            block = int(tables[b, page]) if page < h + grow else -1
            slots[row0 + j] = block * bs + p % bs if block >= 0 else -1
    return new_lens, new_held, np.array([(head + taken) % cap, count - taken + returned], np.int32), pos, slots, tables, ring
