"""The serving operators of the causal (forward-only) SSD scan, as they are measured.

Four operators and the cache they share, a pool of fp32 states (slots, H, P, N):

  fwd      ssd_causal_fwd: prompts. h_t = exp(dt_t A) h_{t-1} + dt_t B_t x_t^T,
           y_t = C_t^T h_t + D x_t over whole (ragged) sequences, in chunks; the
           output and the state after each sequence's last token
  step     ssd_causal_step: the same recurrence for one token of each sequence,
           states read from and written to the rows of a pool
  copy     ssd_cache_copy: pages of a pool copied, forked (one source, several
           destinations) and freed (zeroed), in every layer
  compact  ssd_cache_compact: live pages moved to the front of a pool with the
           fewest moves, and the table of pages that goes with it

A case is a dict of plain values; "op" names the operator. Where `own` is false
run() computes the plain forms below, in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
DT_MIN, DT_MAX = 1e-3, 0.1


# --------------------------------------------------------------------- cases
def _fwd(name, batch, L, H, P, N, G, dtype, ragged=False, slots=0, raw=False, packed=False, init=False, D=True):
    return dict(name=name, op="fwd", batch=batch, L=L, H=H, P=P, N=N, G=G, dtype=dtype, ragged=ragged, slots=slots,
                raw=raw, packed=packed, init=init, D=D)


def _step(name, batch, H, P, N, G, dtype, slots, pad=0, raw=False, packed=False, D=True):
    return dict(name=name, op="step", batch=batch, H=H, P=P, N=N, G=G, dtype=dtype, slots=slots, pad=pad, raw=raw,
                packed=packed, D=D)


def _copy(name, layers, slots, H, P, N, sources, fan, freed):
    return dict(name=name, op="copy", layers=layers, slots=slots, H=H, P=P, N=N, sources=sources, fan=fan, freed=freed)


def _compact(name, layers, slots, H, P, N, live, moves, shared=0):
    return dict(name=name, op="compact", layers=layers, slots=slots, H=H, P=P, N=N, live=live, moves=moves,
                shared=shared)


def listed():
    return [
        # the 130M mixer's full batch as a prompt batch, B and C per head
        _fwd("fwd_130m_b32_L1024", 32, 1024, 24, 64, 128, 24, "bf16"),
        # one long prompt: few units, a long axis
        _fwd("fwd_long_b1_L65536", 1, 65536, 24, 64, 128, 24, "bf16"),
        # a serving batch of prompts of different lengths: views of one projection, raw step sizes, states
        # continued from and kept in a pool, B and C shared by all heads
        _fwd("fwd_ragged_b16_L1000_pool", 16, 1000, 24, 64, 128, 1, "bf16", ragged=True, slots=40, raw=True,
             packed=True, init=True),
        # one short prompt, where latency counts
        _fwd("fwd_short_b1_L100", 1, 100, 24, 64, 128, 24, "bf16"),
        # fp32 prompts of odd lengths, two head-width halves per head, grouped B and C
        _fwd("fwd_f32_b4_L777", 4, 777, 8, 128, 64, 2, "f32", ragged=True, init=True, D=False),
        # one sequence generating alone
        _step("step_b1", 1, 24, 64, 128, 24, "bf16", slots=1),
        # a serving batch out of a larger pool, padded to a fixed size, views of one projection, raw step sizes
        _step("step_b250_pool", 250, 24, 64, 128, 1, "bf16", slots=400, pad=6, raw=True, packed=True),
        # a large decode batch, fp32 activations
        _step("step_f32_b512", 512, 32, 64, 128, 8, "f32", slots=512),
        # a prompt's state forked for three continuations, two old ones freed, in a 12-layer model
        _copy("copy_fork3_12l", 12, 16, 24, 64, 128, 1, 3, 2),
        # a beam's worth of pages moved about in a 24-layer pool
        _copy("copy_b32_24l", 24, 96, 24, 64, 128, 16, 2, 8),
        # a small pool with a hole to close
        _compact("compact_small_2l", 2, 24, 24, 64, 64, 13, 3),
        # a 12-layer pool, half of it live
        _compact("compact_12l_128", 12, 128, 24, 64, 128, 64, 30, shared=6),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], evenly over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _draw(rng)
    del case["name"]
    return case


def _draw(rng):
    op = rng.choice(["fwd", "fwd", "step", "step", "copy", "compact"])
    H = rng.choice([1, 3, 4, 8, 12, 24, 32])
    P = rng.choice([64, 64, 64, 128])
    N = rng.choice([64, 128, 128])
    G = rng.choice([g for g in range(1, H + 1) if H % g == 0])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    raw, packed, D = rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.7
    if op == "fwd":
        # at most half the largest listed case's tokens x heads x head width, so that no draw costs more than it
        most = 32 * 1024 * 24 * 64 // 2 // (2 if dtype == "f32" else 1)
        L = _between(rng, 1, min(40000, most // (H * P)))
        batch = _between(rng, 1, max(1, min(200, most // (L * H * P))))
        ragged = batch > 1 and rng.random() < 0.5
        slots = batch + rng.randint(0, 20) if rng.random() < 0.4 else 0
        return _fwd("", batch, L, H, P, N, G, dtype, ragged, slots, raw, packed, slots > 0 or rng.random() < 0.5, D)
    if op == "step":
        batch = _between(rng, 1, max(1, 512 * 32 * 64 // (H * P)) if H * P > 512 else 1000)
        pad = rng.randint(0, batch // 8)
        return _step("", batch, H, P, N, G, dtype, batch + rng.randint(0, 60), pad, raw, packed, D)
    layers = _between(rng, 1, 24)
    page = layers * H * P * N * 4
    if op == "copy":
        pairs = _between(rng, 1, max(1, min(100, (40 * 24 * 24 * 64 * 128 * 4) // page)))
        fan = rng.choice([1, 1, 2, 3])
        sources = max(1, pairs // fan)
        freed = rng.randint(0, 3)
        return _copy("", layers, sources + sources * fan + freed + rng.randint(0, 10), H, P, N, sources, fan, freed)
    live = _between(rng, 1, max(1, min(200, (64 * 12 * 24 * 64 * 128 * 4) // page)))
    moves = rng.randint(0, live // 2)
    return _compact("", layers, live + moves + rng.randint(0, live), H, P, N, live, moves, rng.randint(0, 3))


# -------------------------------------------------------------------- inputs
def _lengths(case):
    """The prompts' lengths before they are put in order: spread evenly up to L, one of a single token."""
    b, L = case["batch"], case["L"]
    if not case["ragged"]:
        return [L] * b
    return [1] + [max(1, L * (i + 1) // b) for i in range(1, b)]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    rand = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=g, device=dev)  # noqa: E731
    H, P, N = case["H"], case["P"], case["N"]
    st = {"case": case}
    if case["op"] in ("copy", "compact"):
        st["pool"] = randn(case["layers"], case["slots"], H, P, N)
        if case["op"] == "copy":
            ns, fan, nf = case["sources"], case["fan"], case["freed"]
            order = perm(case["slots"]).to(torch.int32)
            src = order[:ns].repeat_interleave(fan)
            st["src"] = torch.cat([src, torch.full((nf,), -1, dtype=torch.int32, device=dev)])
            st["dst"] = order[ns:ns + ns * fan + nf].contiguous()
        else:
            n, m = case["live"], case["moves"]
            inside = perm(n)[:n - m]
            behind = n + perm(case["slots"] - n)[:m]
            pages = torch.cat([inside, behind])
            pages = torch.cat([pages, pages[:min(case["shared"], n)], torch.full((2,), -1, device=dev)])
            st["table"] = pages[perm(pages.numel())].to(torch.int32)
        return st
    io = DTYPES[case["dtype"]]
    G, b = case["G"], case["batch"]
    lead = (b, case["L"]) if case["op"] == "fwd" else (b,)
    nx, nb = H * P, G * N
    x, B, C = randn(*lead, nx), randn(*lead, nb) / 8, randn(*lead, nb) / 8
    if case["packed"]:
        # what a layer's input projection gives: x, B and C side by side, taken as views
        proj = torch.cat([x, B, C], -1).to(io)
        x, B, C = proj[..., :nx], proj[..., nx:nx + nb], proj[..., nx + nb:]
    st["x"], st["B"], st["C"] = (t.to(io).unflatten(-1, s) for t, s in ((x, (H, P)), (B, (G, N)), (C, (G, N))))
    if case["raw"]:
        st["dt"] = randn(*lead, H).to(io)
        st["dt_bias"] = rand(H) * 4.7 - 7.0
    else:
        st["dt"] = torch.log1p(torch.exp(randn(*lead, H) - 4.0)).clamp(DT_MIN, DT_MAX).to(io)
        st["dt_bias"] = None
    st["A"] = -torch.exp(rand(H) * math.log(16.0))
    st["D"] = randn(H) if case["D"] else None
    if case["op"] == "step" or case["slots"]:
        st["pool"] = randn(case["slots"], H, P, N) * 0.3
        st["after"] = st["pool"].clone()
        slots = perm(case["slots"])[:b].to(torch.int32)
        if case.get("pad"):
            slots[perm(b)[:case["pad"]]] = -1
        st["slots"] = slots
    elif case["init"]:
        st["init"] = randn(b, H, P, N) * 0.3
    if case["op"] == "fwd" and case["ragged"]:
        st["seqlens"] = torch.tensor(_lengths(case), dtype=torch.int32, device=dev)[perm(b)].contiguous()
    return st


# --------------------------------------------------------------- plain forms
def _step_sizes(st):
    dt = st["dt"].float()
    if st["dt_bias"] is None:
        return dt
    return torch.logaddexp(dt + st["dt_bias"], torch.zeros((), device=dt.device)).clamp(DT_MIN, DT_MAX)


def _plain_fwd(st):
    case = st["case"]
    b, L, H, P, N, G = (case[k] for k in ("batch", "L", "H", "P", "N", "G"))
    Q = min(128, L)
    nc = -(-L // Q)
    x, B, C, dt = st["x"].float(), st["B"].float(), st["C"].float(), _step_sizes(st)
    lens = st["seqlens"] if "seqlens" in st else torch.full((b,), L, device=x.device)
    inside = torch.arange(L, device=x.device)[None, :] < lens[:, None]
    dt = torch.where(inside[..., None], dt, torch.zeros_like(dt))
    tail = nc * Q - L
    cut = lambda t: torch.cat([t, t.new_zeros(b, tail, *t.shape[2:])], 1).unflatten(1, (nc, Q))  # noqa: E731
    xc, Bc, Cc, dtc = cut(x), cut(B), cut(C), cut(dt)
    a = torch.cumsum(dtc * st["A"], 2).transpose(2, 3)                      # (b, nc, H, Q)
    w = dtc.transpose(2, 3)
    low = torch.ones(Q, Q, dtype=torch.bool, device=x.device).tril()
    decay = torch.exp((a[..., :, None] - a[..., None, :]).masked_fill(~low, -math.inf)) * w[..., None, :]
    Bh, Ch = (t.permute(0, 1, 3, 2, 4).repeat_interleave(H // G, 2) for t in (Bc, Cc))   # (b, nc, H, Q, N)
    xh = xc.permute(0, 1, 3, 2, 4)                                          # (b, nc, H, Q, P)
    y = ((Ch @ Bh.transpose(-1, -2)) * decay) @ xh
    own_state = (xh * (torch.exp(a[..., -1:] - a) * w)[..., None]).transpose(-1, -2) @ Bh   # (b, nc, H, P, N)
    # the states entering every chunk and the last one leaving: start state and chunk states, decayed
    if "pool" in st:
        start = st["pool"][st["slots"].long()]
    else:
        start = st["init"] if "init" in st else x.new_zeros(b, H, P, N)
    total = torch.cumsum(a[..., -1].double(), 1)                            # (b, nc, H)
    edge = torch.cat([torch.zeros_like(total[:, :1]), total], 1).transpose(1, 2)          # (b, H, nc + 1)
    span = (edge[..., :, None] - edge[..., None, :]).masked_fill(
        ~torch.ones(nc + 1, nc + 1, dtype=torch.bool, device=x.device).tril(), -math.inf)
    carry = torch.exp(span).float()                                         # (b, H, nc + 1, nc + 1)
    given = torch.cat([start[:, None], own_state], 1).transpose(1, 2).flatten(3)          # (b, H, nc + 1, P N)
    states = (carry @ given).unflatten(3, (P, N))
    y = y + (Ch * torch.exp(a)[..., None]) @ states[:, :, :-1].transpose(1, 2).transpose(-1, -2)
    y = y.permute(0, 1, 3, 2, 4).flatten(1, 2)[:, :L]
    if st["D"] is not None:
        y = y + x * st["D"][:, None]
    y = torch.where(inside[..., None, None], y, torch.zeros_like(y)).to(st["x"].dtype)
    if "pool" in st:
        st["after"][st["slots"].long()] = states[:, :, -1]
        return y, st["after"]
    return y, states[:, :, -1].contiguous()


def _plain_step(st):
    x, B, C, dt = st["x"].float(), st["B"].float(), st["C"].float(), _step_sizes(st)
    per = st["case"]["H"] // st["case"]["G"]
    B, C = B.repeat_interleave(per, 1), C.repeat_interleave(per, 1)
    used = st["slots"] >= 0
    rows = st["slots"].clamp(min=0).long()
    h = st["pool"][rows] * torch.exp(dt * st["A"])[..., None, None] + (x * dt[..., None])[..., None] * B[:, :, None]
    y = (h * C[:, :, None]).sum(-1)
    if st["D"] is not None:
        y = y + x * st["D"][:, None]
    y = torch.where(used[:, None, None], y, torch.zeros_like(y)).to(st["x"].dtype)
    st["after"][rows[used]] = h[used]
    return y, st["after"]


def _plain_copy(st):
    pool, src, dst = st["pool"], st["src"].long(), st["dst"].long()
    pages = pool[:, src.clamp(min=0)]
    pool[:, dst] = torch.where((src >= 0)[None, :, None, None, None], pages, torch.zeros_like(pages))
    return pool


def _plain_compact(st):
    pool, table = st["pool"], st["table"].long()
    slots = pool.shape[1]
    used = torch.zeros(slots, dtype=torch.bool, device=pool.device)
    used[table[table >= 0]] = True
    live = used.sum()
    at = torch.arange(slots, device=pool.device)
    holes, behind = at[~used & (at < live)], at[used & (at >= live)]
    pool[:, holes] = pool[:, behind]
    to = at.clone()
    to[behind] = holes
    new = torch.where(table >= 0, to[table.clamp(min=0)], table).to(torch.int32)
    return pool, new, live.to(torch.int32).reshape(1)


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        import bidirectional_mamba_ssd_b200 as ssd
        if op in ("fwd", "step"):
            kw = {} if st["dt_bias"] is None else dict(dt_bias=st["dt_bias"], dt_min=DT_MIN, dt_max=DT_MAX)
            if "pool" in st:
                kw |= dict(slots=st["slots"], state_out=st["after"])
        if op == "fwd":
            return ssd.ssd_causal_fwd(st["x"], st["dt"], st["A"], st["B"], st["C"], st["D"],
                                      st.get("pool", st.get("init")), seqlens=st.get("seqlens"), **kw)
        if op == "step":
            y = ssd.ssd_causal_step(st["x"], st["dt"], st["A"], st["B"], st["C"], st["D"], st["pool"], **kw)
            return y, st["after"]
        if op == "copy":
            return ssd.ssd_cache_copy(st["pool"], st["src"], st["dst"])
        table, live = ssd.ssd_cache_compact(st["pool"], st["table"])
        return st["pool"], table, live
    return {"fwd": _plain_fwd, "step": _plain_step, "copy": _plain_copy, "compact": _plain_compact}[op](st)


def work(case):
    H, P, N = case["H"], case["P"], case["N"]
    page = H * P * N * 4
    if case["op"] == "copy":
        pairs = case["sources"] * case["fan"]
        return {"bytes": case["layers"] * page * (case["sources"] + pairs + case["freed"]) + 8 * (pairs + case["freed"]), "flops": 0}
    if case["op"] == "compact":
        rows = case["live"] + min(case["shared"], case["live"]) + 2
        return {"bytes": case["layers"] * page * 2 * case["moves"] + 8 * rows, "flops": 0}
    e = 2 if case["dtype"] == "bf16" else 4
    inputs = (H * P + H + 2 * case["G"] * N) * e
    if case["op"] == "step":
        rows = case["batch"] - case["pad"]
        return {"bytes": rows * (inputs + 2 * page) + case["batch"] * H * P * e, "flops": rows * H * P * N * 5}
    tokens = sum(_lengths(case))
    states = (2 if case["init"] else 1) * case["batch"] * page
    # the recurrence's own operations: the chunked forms do more
    return {"bytes": tokens * inputs + case["batch"] * case["L"] * H * P * e + states, "flops": tokens * H * P * N * 5}


# --------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    """The recurrence, token by token, in 64 bits."""
    if case["op"] in ("copy", "compact"):
        return None
    st = prepare(case, seed)
    H, G = case["H"], case["G"]
    head = torch.arange(H, device="cuda") // (H // G)
    dt = st["dt"].double()
    if st["dt_bias"] is not None:
        u = dt + st["dt_bias"].double()
        dt = (u.clamp(min=0) + torch.log1p(torch.exp(-u.abs()))).clamp(DT_MIN, DT_MAX)
    A = st["A"].double()
    D = st["D"].double()[:, None] if st["D"] is not None else 0.0

    def token(h, x, dt, B, C):
        x, B, C = x.double(), B.double()[:, head], C.double()[:, head]
        h = torch.exp(dt * A)[..., None, None] * h
        h += (dt[..., None] * x)[..., None] * B[:, :, None, :]
        return h, torch.matmul(h, C[..., None])[..., 0] + D * x

    pool = st["after"].double() if "after" in st else None
    if case["op"] == "step":
        y = torch.zeros(st["x"].shape, dtype=torch.float64, device="cuda")
        rows = torch.nonzero(st["slots"] >= 0)[:, 0]
        at = st["slots"][rows].long()
        pool[at], y[rows] = token(st["pool"][at].double(), st["x"][rows], dt[rows], st["B"][rows], st["C"][rows])
        return y, pool
    b, L = case["batch"], case["L"]
    if pool is not None:
        h = st["pool"][st["slots"].long()].double()
    elif "init" in st:
        h = st["init"].double()
    else:
        h = torch.zeros(b, H, case["P"], case["N"], dtype=torch.float64, device="cuda")
    lens = st["seqlens"].tolist() if "seqlens" in st else [L] * b
    # longest first, so that the sequences still running are the first ones
    order = sorted(range(b), key=lambda i: -lens[i])
    back = torch.tensor(order, device="cuda")
    h = h[back]
    y = torch.zeros(b, L, H, case["P"], dtype=torch.float64, device="cuda")
    xs, dts, Bs, Cs = st["x"][back], dt[back], st["B"][back], st["C"][back]
    n = b
    for t in range(max(lens)):
        while lens[order[n - 1]] <= t:
            n -= 1
        h[:n], y[:n, t] = token(h[:n], xs[:n, t], dts[:n, t], Bs[:n, t], Cs[:n, t])
    out, last = torch.empty_like(y), torch.empty_like(h)
    out[back], last[back] = y, h
    if pool is None:
        return out, last
    pool[st["slots"].long()] = last
    return out, pool
