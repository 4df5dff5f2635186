"""The causal serving operators from their definitions, in 64 bits, for the
tests: a token-by-token recurrence and page moves one after another (torch on
the CPU; nothing of the library)."""
import torch


def step_sizes(dt, bias=None, lo=0.0, hi=float("inf")):
    dt = dt.double().cpu()
    if bias is None:
        return dt
    u = dt + bias.double().cpu()
    return (u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))).clamp(lo, hi)


def scan(x, dt, A, B, C, D, h, steps=None):
    """x (L, H, P), dt (L, H) step sizes, B, C (L, G, N), h (H, P, N): outputs (L, H, P) and the last state."""
    x, B, C, A = (t.double().cpu() for t in (x, B, C, A))
    D = None if D is None else D.double().cpu()
    dt, h = dt.double().cpu(), h.double().cpu().clone()
    H = x.shape[1]
    group = torch.arange(H) // (H // B.shape[1])
    y = torch.zeros_like(x)
    for t in range(x.shape[0] if steps is None else steps):
        h = torch.exp(dt[t] * A)[:, None, None] * h + (dt[t][:, None] * x[t])[:, :, None] * B[t, group][:, None, :]
        y[t] = (h * C[t, group][:, None, :]).sum(-1)
        if D is not None:
            y[t] += D[:, None] * x[t]
    return y, h


def fwd(x, dt, A, B, C, D, starts, lens):
    """Ragged batch: outputs (zero behind each sequence) and end states, row by row."""
    ys, hs = zip(*(scan(x[b], dt[b], A, B[b], C[b], D, starts[b], lens[b]) for b in range(x.shape[0])))
    return torch.stack(ys), torch.stack(hs)


def copy(pool, src, dst):
    """The list of copies, in order, on a CPU copy of the pool."""
    pool = pool.cpu().clone()
    for s, d in zip(src.tolist(), dst.tolist()):
        if not (-1 <= s < pool.shape[1]) or not (0 <= d < pool.shape[1]):
            continue
        pool[:, d] = 0 if s == -1 else pool[:, s].clone()
    return pool


def compact(pool, table):
    """(pool, table, live): named pages from `live` on go to the unnamed ones below it, both in rising order."""
    pool = pool.cpu().clone()
    n = pool.shape[1]
    rows = [t if 0 <= t < n else -1 for t in table.tolist()]
    used = sorted({t for t in rows if t >= 0})
    live = len(used)
    holes = [p for p in range(live) if p not in set(used)]
    to = {p: p for p in used}
    for hole, p in zip(holes, [p for p in used if p >= live]):
        pool[:, hole] = pool[:, p].clone()
        to[p] = hole
    return pool, [to.get(t, -1) for t in rows], live
