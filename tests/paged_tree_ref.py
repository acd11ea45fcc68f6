"""Plain 64-bit attention over a paged cache for any sets of visible keys (test
infrastructure): which keys a drafted token of a tree sees, and the outputs with
what they may be off, derived as in paged_ref.attend."""
import torch

D = 128


def tree_keys(parents, base, n, window, sinks):
    """For each of n drafted tokens the key indices that it sees, ascending; base: tokens before the tree."""
    depth, out = [], []
    for i in range(n):
        depth.append(0 if parents[i] < 0 else depth[parents[i]] + 1)
        p = base + depth[i]
        keys = [j for j in range(base) if not window or j > p - window or j < sinks]
        path, a = [], i
        while a >= 0:
            at = base + depth[a]
            if not window or at > p - window or at < sinks:
                path.append(base + a)
            a = parents[a]
        out.append(torch.tensor(keys + path[::-1], dtype=torch.long))
    return out


def attend(q, k, v, table, cu, keys, scale, w_step):
    """(out, bound, weights) for pages' values k, v [NP, Hkv, PS, 128]; keys: one list a
    query token; weights: the softmax [Hkv, G, n] of each token."""
    T, Hq, _ = q.shape
    Hkv, PS = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    bound = torch.zeros(T, Hq, D, dtype=torch.float64)
    weights = [None] * T
    q = q.double()
    for b in range(table.shape[0]):
        for t in range(int(cu[b]), int(cu[b + 1])):
            j = keys[t]
            if len(j) == 0:
                weights[t] = torch.zeros(Hkv, G, 0, dtype=torch.float64)
                continue
            pg = table[b].long()[j // PS]
            kh, vh = k[pg, :, j % PS].transpose(0, 1), v[pg, :, j % PS].transpose(0, 1)  # [Hkv, n, D]
            qt = q[t].view(Hkv, G, D).transpose(1, 2)                                    # [Hkv, D, G]
            w = torch.softmax(kh @ qt * scale, 1).transpose(1, 2)
            weights[t] = w
            out[t] = (w @ vh).reshape(Hq, D)
            d = 2.0 ** -24 * 140 * (kh.abs() @ qt.abs()).amax(1) * abs(scale) + 2.0 ** -20
            small = len(j) * 2.0 ** -32 * vh.abs().amax(1, keepdim=True)
            u = w_step + 2 * torch.expm1(d) + len(j) ** 0.5 * 2.0 ** -22
            bound[t] = (u[..., None] * (w @ vh.abs()) + small).reshape(Hq, D)
    return out, bound, weights
