"""Tree attention, page mass and eviction in 64 bits, from their definitions,
on the values the oracle says a cache holds."""
import numpy as np


def tree_rows(ref, q, scale, k_tree=None, v_tree=None, sees=None, nodes=None, max_len=None):
    """ref: an OracleCache; q float [B, T, Hq, D]; k_tree, v_tree float [B, T, Hkv, D];
    sees bool [B, T, T].  Returns (out, lse, page_lse, slack): 64-bit results, and
    for each row sum_c |q_c k_c| at its largest key and sum_j p_j |v_j| (what the
    error bounds are relative to)."""
    B, T, Hq, D = q.shape
    G = Hq // ref.Hkv
    max_len = int(ref.seq_lens.max()) if max_len is None else max_len
    P = -(-max_len // 16)
    out = np.zeros((B, T, Hq, D))
    lse = np.full((B, T, Hq), -np.inf)
    page = np.full((B, T, Hq, P), -np.inf)
    reach = np.zeros((B, T, Hq))
    weight = np.zeros((B, T, Hq, D))
    for b in range(B):
        L = min(int(ref.seq_lens[b]), max_len)
        n = T if nodes is None else min(max(int(nodes[b]), 0), T)
        for h in range(ref.Hkv):
            k = ref.dequantize(b, h, 0, 0, L).astype(np.float64)
            v = ref.dequantize(b, h, 1, 0, L).astype(np.float64)
            for t in range(n):
                kk, vv = k, v
                if k_tree is not None:
                    js = [j for j in range(n) if (sees[b, t, j] if sees is not None else j <= t)]
                    kk = np.concatenate([k, np.asarray(k_tree[b, js, h], np.float64).reshape(-1, D)])
                    vv = np.concatenate([v, np.asarray(v_tree[b, js, h], np.float64).reshape(-1, D)])
                if len(kk) == 0:
                    continue
                for g in range(G):
                    r = h * G + g
                    qr = q[b, t, r].astype(np.float64)
                    a = scale * (kk @ qr)
                    top = a.max()
                    e = np.exp(a - top)
                    lse[b, t, r] = top + np.log(e.sum())
                    out[b, t, r] = (e @ vv) / e.sum()
                    weight[b, t, r] = (e @ np.abs(vv)) / e.sum()
                    reach[b, t, r] = (np.abs(kk) @ np.abs(qr)).max()
                    for p in range(-(-L // 16)):
                        c = a[16 * p:min(16 * p + 16, L)]
                        page[b, t, r, p] = c.max() + np.log(np.exp(c - c.max()).sum())
    return out, lse, page, (reach, weight)


def page_mass(lse, page_lse, mass, decay, on):
    """on: bool [B, T]."""
    w = np.exp(np.where(np.isneginf(lse)[..., None], -np.inf, page_lse.astype(np.float64) -
                        np.where(np.isneginf(lse), 0.0, lse.astype(np.float64))[..., None]))
    out = decay * mass.astype(np.float64)
    out[:, :page_lse.shape[-1]] += (w * on[:, :, None, None]).sum((1, 2))
    return out


def evict(table, lens, mass, keep, sink, recent, unit=1):
    """Rows one by one: (table, lens, mass, evicted)."""
    table, mass, lens = table.copy(), mass.copy(), lens.copy()
    P = table.shape[1]
    gone_n = np.zeros(len(lens), np.int32)
    for b, L in enumerate(lens):
        full, used = L // (16 * unit), -(-L // 16)
        w = [np.float32(0)] * full
        with np.errstate(invalid="ignore"):   # inf - inf
            for u in range(full):
                for j in range(unit):
                    w[u] = mass[b, u * unit] if j == 0 else np.float32(w[u] + mass[b, u * unit + j])
        if full <= keep // unit:
            mass[b, used:] = 0
            continue
        s, r = sink // unit, recent // unit
        fixed = list(range(s)) + list(range(full - r, full))
        free = [u for u in range(full) if u not in set(fixed)]
        free.sort(key=lambda u: (np.isnan(w[u]), -w[u] if not np.isnan(w[u]) else 0, u))
        stay = sorted(fixed + free[:keep // unit - len(fixed)])
        gone = sorted(set(range(full)) - set(stay))
        pages = lambda us: [u * unit + j for u in us for j in range(unit)]
        rest = list(range(full * unit, P))
        m = np.zeros(P, np.float32)
        order = pages(stay) + rest[:used - full * unit]
        m[:len(order)] = mass[b, order]
        table[b] = table[b, pages(stay) + rest + pages(gone)]
        mass[b] = m
        gone_n[b] = unit * len(gone)
        lens[b] -= 16 * gone_n[b]
    return table, lens, mass, gone_n


def sees_from_parents(parents):
    """[B, T] parent indices -> bool [B, T, T]: a node sees itself and its ancestors."""
    B, T = parents.shape
    s = np.zeros((B, T, T), bool)
    for b in range(B):
        for t in range(T):
            if parents[b, t] >= 0:
                s[b, t] = s[b, parents[b, t]]
            s[b, t, t] = True
    return s


def words(sees):
    """bool [..., T, T] -> int64 ancestor words [..., T]."""
    T = sees.shape[-1]
    return (sees.astype(np.uint64) << np.arange(T, dtype=np.uint64)).sum(-1, dtype=np.uint64).view(np.int64)
