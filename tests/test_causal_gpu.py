"""GPU tests of the causal serving operators (ssd_causal_fwd, ssd_causal_step)
against the recurrence in 64 bits (causal_ref).

Tolerances. Outputs: paritylib's bars (fp32 1e-4 relative, floored at the RMS;
bf16 2e-2 of the RMS beyond half a step of the output's own rounding, and an
RMS error of 3e-3). End states are fp32 whatever the I/O type and are held to
5e-5 relative, floored at the RMS: a state is a sum of tokens whose products
carry at least 24 bits; adding a tile's 128 of them in fp32 loses at most 128 x
2^-23 = 1.5e-5 of the largest partial sum, which is taken as up to three times
the end value or the RMS (a decaying sum of random signs); the decays' own
exponents, at most 60 in magnitude where they still matter, add 60 x 2^-24 =
0.4e-5.
"""
import threading

import numpy as np
import pytest
import torch

import causal_ref as ref
import ssd_inputs as si
from paritylib import check, err_f32, rms_err

pytestmark = pytest.mark.gpu

TOL_STATE = 5e-5
DT_LO, DT_HI = 1e-3, 0.1


@pytest.fixture(scope="module")
def ssd():
    import bidirectional_mamba_ssd_b200 as m
    return m


def inputs(lead, H, P, N, G, io, seed, raw=False, packed=False):
    """x, dt, B, C with the leading dimensions `lead`, A, D, dt_bias, by ssd_inputs' recipe."""
    dev = "cuda"
    dtype = si.DTYPES[io]
    g = torch.Generator(device=dev).manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, B, C = rn(*lead, H * P), rn(*lead, G * N) / 8, rn(*lead, G * N) / 8
    if packed:
        proj = torch.cat([x, B, C], -1).to(dtype)
        x, B, C = proj[..., :H * P], proj[..., H * P:H * P + G * N], proj[..., H * P + G * N:]
    d = dict(x=x.to(dtype).unflatten(-1, (H, P)), B=B.to(dtype).unflatten(-1, (G, N)), C=C.to(dtype).unflatten(-1, (G, N)))
    if raw:
        d["dt"] = rn(*lead, H).to(dtype)
        d["dt_bias"] = torch.rand(H, generator=g, device=dev) * 4.7 - 7.0
    else:
        d["dt"] = torch.nn.functional.softplus(rn(*lead, H) - 4.0).clamp(DT_LO, DT_HI).to(dtype)
        d["dt_bias"] = None
    d["A"] = -torch.exp(torch.rand(H, generator=g, device=dev) * np.log(16.0))
    d["D"] = rn(H)
    d["g"] = g
    return d


def opts(d):
    return {} if d["dt_bias"] is None else dict(dt_bias=d["dt_bias"], dt_min=DT_LO, dt_max=DT_HI)


def sizes(d):
    return ref.step_sizes(d["dt"], d["dt_bias"], DT_LO, DT_HI)


def check_state(h, o, what):
    h = h.detach().double().cpu().numpy()
    assert np.isfinite(h).all(), f"{what}: non-finite state"
    e = err_f32(h, o.numpy())
    assert e <= TOL_STATE, f"{what}: state err {e:.3e} (rms {rms_err(h, o.numpy()):.2e})"


def check_out(y, o, io, what):
    check(y.detach().double().cpu().numpy(), o.numpy(), si.DTYPES[io], what)


# batch, L, H, P, N, G, io, with start states, D, raw step sizes, views of one projection
SHAPES = [
    (1, 1, 4, 64, 128, 4, "bf16", True, True, False, False),
    (2, 2, 2, 64, 64, 1, "bf16", False, True, False, True),
    (3, 17, 4, 64, 128, 2, "bf16", True, False, True, True),
    (1, 127, 3, 64, 128, 3, "bf16", False, True, False, False),
    (2, 128, 2, 64, 64, 2, "bf16", True, True, False, False),
    (2, 129, 2, 128, 128, 1, "bf16", True, True, True, True),
    (1, 777, 6, 64, 128, 2, "bf16", True, True, False, False),
    (5, 300, 4, 64, 64, 4, "bf16", False, True, True, False),
    (1, 3000, 2, 64, 128, 1, "bf16", True, True, False, True),
    (2, 200, 1, 256, 64, 1, "bf16", True, True, True, True),
    (160, 20, 1, 64, 64, 1, "bf16", True, True, False, False),
    (30, 300, 6, 64, 128, 1, "bf16", True, True, False, True),
    (1, 1, 4, 64, 128, 4, "f32", True, True, False, False),
    (3, 17, 4, 64, 128, 2, "f32", True, False, True, True),
    (2, 129, 2, 128, 64, 1, "f32", True, True, True, True),
    (1, 777, 3, 192, 128, 3, "f32", False, True, False, False),
    (1, 2500, 2, 64, 64, 2, "f32", True, True, False, True),
]


def paths_of(ssd, io):
    return [ssd.SSD_PATH_AUTO] + ([ssd.SSD_PATH_SIMT] if io == "bf16" else [])


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "b%d_L%d_H%d_P%d_N%d_G%d_%s_%d%d%d%d" % s)
def test_fwd_against_recurrence(ssd, shape):
    batch, L, H, P, N, G, io, init, skip, raw, packed = shape
    d = inputs((batch, L), H, P, N, G, io, seed=L + 7 * H, raw=raw, packed=packed)
    D = d["D"] if skip else None
    h0 = torch.randn(batch, H, P, N, generator=d["g"], device="cuda") * 0.3 if init else None
    starts = h0 if init else torch.zeros(batch, H, P, N)
    o, oh = ref.fwd(d["x"], sizes(d), d["A"], d["B"], d["C"], D, starts, [L] * batch)
    for path in paths_of(ssd, io):
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], D, h0, path=path, **opts(d))
        torch.cuda.synchronize()
        assert ssd.ssd_get_device_status() == 0
        check_out(y, o, io, f"path {path} {shape}")
        check_state(h, oh, f"path {path} {shape}")


RAGGED = [(6, 300, 2, 64, 128, 1, "bf16", (300, 0, 1, 128, 129, 257)),
          (4, 100, 2, 128, 64, 2, "bf16", (99, 100, 0, 5)),
          (3, 2000, 1, 64, 128, 1, "bf16", (2000, 130, 1024)),
          (5, 200, 2, 64, 64, 1, "f32", (200, 0, 16, 17, 129)),
          (3, 1500, 1, 64, 128, 1, "f32", (0, 1400, 300))]


@pytest.mark.parametrize("case", RAGGED, ids=lambda c: "b%d_L%d_H%d_P%d_N%d_G%d_%s" % c[:7])
def test_fwd_ragged_with_nan_behind_the_sequences(ssd, case):
    """Lengths 0 and 1 among them; what lies behind a sequence is NaN and infinity."""
    batch, L, H, P, N, G, io, lens = case
    d = inputs((batch, L), H, P, N, G, io, seed=5, raw=True)
    h0 = torch.randn(batch, H, P, N, generator=d["g"], device="cuda") * 0.3
    o, oh = ref.fwd(d["x"], sizes(d), d["A"], d["B"], d["C"], d["D"], h0, lens)
    behind = torch.arange(L, device="cuda")[None, :] >= torch.tensor(lens, device="cuda")[:, None]
    for k, v in (("x", float("nan")), ("B", float("inf")), ("C", float("nan")), ("dt", float("inf"))):
        d[k][behind] = v
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for path in paths_of(ssd, io):
        out = torch.full_like(d["x"], 7.0)
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], h0, seqlens=seqlens, out=out,
                                  path=path, **opts(d))
        torch.cuda.synchronize()
        assert ssd.ssd_get_device_status() == 0
        assert y is out and (y[behind] == 0).all(), "rows behind a sequence are zero"
        for b in range(batch):
            if lens[b]:
                check_out(y[b, :lens[b]], o[b, :lens[b]], io, f"path {path} row {b}")
            check_state(h[b], oh[b], f"path {path} row {b}")
        assert torch.equal(h[[b for b in range(batch) if lens[b] == 0]], h0[[b for b in range(batch) if lens[b] == 0]])


@pytest.mark.parametrize("io,L", [("bf16", 150), ("bf16", 1700), ("f32", 40), ("f32", 1300)])
def test_fwd_pool_slots(ssd, io, L):
    """Pages by slot, in place and into another pool; padding rows, bad and repeated slots."""
    batch, H, P, N, G, nslots = 6, 2, 64, 128, 1, 9
    d = inputs((batch, L), H, P, N, G, io, seed=L)
    pool = torch.randn(nslots, H, P, N, generator=d["g"], device="cuda") * 0.3
    slots = torch.tensor([4, -1, 8, 9, 4, 0], dtype=torch.int32, device="cuda")   # 9: out of range, 4: named twice
    good = [0, 2, 5]
    starts = torch.stack([pool[s] if 0 <= s < nslots else torch.zeros_like(pool[0]) for s in slots.tolist()])
    o, oh = ref.fwd(d["x"][good], sizes(d)[good], d["A"], d["B"][good], d["C"][good], d["D"], starts[good], [L] * 3)
    for path in paths_of(ssd, io):
        for inplace in (True, False):
            src = pool.clone()
            dst = src if inplace else torch.full_like(pool, 3.0)
            y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], src, slots=slots,
                                      state_out=None if inplace else dst, path=path)
            torch.cuda.synchronize()
            assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX
            assert ssd.ssd_get_device_status() == 0           # read and cleared
            assert h is dst
            for k, b in enumerate(good):
                check_out(y[b], o[k], io, f"row {b}")
                check_state(dst[slots[b]], oh[k], f"row {b}")
            assert (y[[1, 3, 4]] == 0).all()
            rest = [s for s in range(nslots) if s not in (4, 8, 0)]
            assert torch.equal(dst[rest], pool[rest] if inplace else torch.full_like(pool[rest], 3.0))
            if not inplace:
                assert torch.equal(src, pool)


def test_fwd_orders_and_strides(ssd):
    """Token-major tensors (L, batch, ...), sliced batches, dt with a stride of its own; refused ones."""
    batch, L, H, P, N, G = 3, 140, 2, 64, 64, 1
    d = inputs((L, 2 * batch), H, P, N, G, "bf16", seed=3)
    v = {k: d[k].transpose(0, 1)[::2] for k in ("x", "dt", "B", "C")}
    o, oh = ref.fwd(v["x"], v["dt"].double().cpu(), d["A"], v["B"], v["C"], d["D"], torch.zeros(batch, H, P, N), [L] * batch)
    y, h = ssd.ssd_causal_fwd(v["x"], v["dt"], d["A"], v["B"], v["C"], d["D"])
    torch.cuda.synchronize()
    check_out(y, o, "bf16", "token-major")
    check_state(h, oh, "token-major")
    assert y.is_contiguous()
    with pytest.raises(ValueError, match="contiguous"):
        ssd.ssd_causal_fwd(v["x"].transpose(2, 3).contiguous().transpose(2, 3), v["dt"], d["A"], v["B"], v["C"])
    with pytest.raises(ssd.SSDError):                       # a batch stride of zero
        ssd.ssd_causal_fwd(v["x"][:1].expand(3, -1, -1, -1), v["dt"], d["A"], v["B"], v["C"])
    wide = torch.zeros(batch, L, H * P + 4, dtype=torch.bfloat16, device="cuda")[..., :H * P].unflatten(-1, (H, P))
    with pytest.raises(ssd.SSDError):                       # rows 8 bytes off a 16-byte step
        ssd.ssd_causal_fwd(wide, v["dt"], d["A"], v["B"], v["C"])


def test_fwd_empty(ssd):
    d = inputs((2, 0), 2, 64, 64, 1, "bf16", seed=1)
    h0 = torch.randn(2, 2, 64, 64, device="cuda")
    y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], h0)
    assert y.shape == (2, 0, 2, 64) and torch.equal(h, h0)
    y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"])
    assert (h == 0).all()
    d = inputs((0, 5), 2, 64, 64, 1, "bf16", seed=1)
    y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"])
    assert y.shape == (0, 5, 2, 64) and h.shape == (0, 2, 64, 64)


def test_fwd_strong_and_no_decay(ssd):
    """A of zero (a plain running sum) and of -1e4 (nothing carried), in both I/O types."""
    for io in ("bf16", "f32"):
        d = inputs((1, 260), 3, 64, 64, 1, io, seed=9)
        d["A"] = torch.tensor([0.0, -1e4, -3.0], device="cuda")
        o, oh = ref.fwd(d["x"], sizes(d), d["A"], d["B"], d["C"], d["D"], torch.zeros(1, 3, 64, 64), [260])
        for path in paths_of(ssd, io):
            y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], path=path)
            torch.cuda.synchronize()
            for k in range(3):
                check_out(y[:, :, k], o[:, :, k], io, f"{io} head {k}")
                check_state(h[:, k], oh[:, k], f"{io} head {k}")


def test_fwd_decay_ranges(ssd):
    """Step sizes of 0.1 throughout: a tile of 128 tokens decays by e^-64, e^-147, e^-154, e^-282, e^-320, e^-512
    (both sides of the spans where the masked matrix changes its references), with start states."""
    A = torch.tensor([-5.0, -11.5, -12.0, -22.0, -25.0, -40.0], device="cuda")
    d = inputs((1, 300), 6, 64, 128, 2, "bf16", seed=12)
    d["dt"].fill_(0.1)
    h0 = torch.randn(1, 6, 64, 128, generator=d["g"], device="cuda")
    o, oh = ref.fwd(d["x"], sizes(d), A, d["B"], d["C"], d["D"], h0, [300])
    y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], A, d["B"], d["C"], d["D"], h0)
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0
    for k in range(6):
        check_out(y[:, :, k], o[:, :, k], "bf16", f"A {A[k].item()}")
        check_out(y[:, :1, k], o[:, :1, k], "bf16", f"first token, A {A[k].item()}")
        check_state(h[:, k], oh[:, k], f"A {A[k].item()}")


STEPS = [(1, 4, 64, 128, 4, "bf16", False, False), (7, 2, 64, 64, 1, "bf16", True, True), (33, 8, 128, 128, 2, "bf16", False, True),
         (300, 4, 64, 128, 1, "bf16", True, False), (5, 3, 64, 64, 3, "f32", False, False), (130, 12, 192, 128, 4, "f32", True, True)]


@pytest.mark.parametrize("case", STEPS, ids=lambda c: "b%d_H%d_P%d_N%d_G%d_%s_%d%d" % c)
def test_step_against_recurrence(ssd, case):
    batch, H, P, N, G, io, raw, packed = case
    d = inputs((batch,), H, P, N, G, io, seed=batch, raw=raw, packed=packed)
    h0 = torch.randn(batch, H, P, N, generator=d["g"], device="cuda")
    dt = sizes(d)
    one = lambda t: t[:, None]  # noqa: E731
    for D in (d["D"], None):
        o, oh = ref.fwd(one(d["x"]), one(dt), d["A"], one(d["B"]), one(d["C"]), D, h0, [1] * batch)
        st = h0.clone()
        y = ssd.ssd_causal_step(d["x"], d["dt"], d["A"], d["B"], d["C"], D, st, **opts(d))
        other = torch.empty_like(h0)
        keep = h0.clone()
        y2 = ssd.ssd_causal_step(d["x"], d["dt"], d["A"], d["B"], d["C"], D, keep, state_out=other, **opts(d))
        torch.cuda.synchronize()
        check_out(y, o[:, 0], io, f"{case}")
        check_state(st, oh, f"{case}")
        assert torch.equal(y, y2) and torch.equal(st, other) and torch.equal(keep, h0)


@pytest.mark.parametrize("batch", [6, 2500])
def test_step_pool_slots(ssd, batch):
    H, P, N, G, nslots = 1, 64, 64, 1, batch + 3
    d = inputs((batch,), H, P, N, G, "bf16", seed=8)
    pool = torch.randn(nslots, H, P, N, generator=d["g"], device="cuda")
    slots = torch.randperm(nslots, generator=d["g"], device="cuda")[:batch].to(torch.int32)
    slots[1], slots[3], slots[4] = -1, -2, slots[0]         # padding, out of range, named twice
    good = [b for b in range(batch) if b not in (1, 3, 4)]
    one = lambda t: t[good][:, None]  # noqa: E731
    o, oh = ref.fwd(one(d["x"]), one(sizes(d).cuda()), d["A"], one(d["B"]), one(d["C"]), d["D"], pool[slots[good].long()],
                    [1] * len(good))
    st = pool.clone()
    y = ssd.ssd_causal_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], st, slots)
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX
    check_out(y[good], o[:, 0], "bf16", "pool")
    check_state(st[slots[good].long()], oh, "pool")
    assert (y[[1, 3, 4]] == 0).all()
    rest = sorted(set(range(nslots)) - set(slots[good].tolist()))
    assert torch.equal(st[rest], pool[rest])


def test_refusals(ssd):
    d = inputs((2, 10), 2, 64, 64, 1, "bf16", seed=1)
    a = [d[k] for k in ("x", "dt", "A", "B", "C", "D")]
    pool = torch.zeros(4, 2, 64, 64, device="cuda")
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    f = ssd.ssd_causal_fwd
    cases = [
        (ValueError, lambda: f(*a, slots=slots)),                                   # slots without a pool
        (ValueError, lambda: f(*a, pool, slots=slots.long())),                      # slots int64
        (ValueError, lambda: f(*a, pool)),                                          # 4 pages for 2 rows
        (ValueError, lambda: f(*a, pool, slots=slots, state_out=pool[:3])),         # pools of two sizes
        (ValueError, lambda: f(*a, seqlens=slots[:1])),
        (ValueError, lambda: f(*a, seqlens=slots.cpu())),
        (ValueError, lambda: f(a[0].half(), *a[1:])),
        (ValueError, lambda: f(a[0], a[1].float(), *a[2:])),
        (ValueError, lambda: f(*a[:2], a[2].to(torch.bfloat16), *a[3:])),
        (ValueError, lambda: f(*a, out=torch.empty(2, 10, 2, 64, device="cuda"))),
        (ssd.SSDError, lambda: f(*a, dt_bias=a[2], dt_min=0.2, dt_max=0.1)),
        (ssd.SSDError, lambda: f(*a, path=ssd.SSD_PATH_PAIR)),
    ]
    big = torch.zeros(5, 2, 64, 64, device="cuda")
    cases.append((ValueError, lambda: f(*a, big[:4], slots=slots, state_out=big[1:])))   # overlapping pools
    n32 = inputs((2, 10), 2, 64, 32, 1, "bf16", seed=1)
    cases.append((ssd.SSDError, lambda: f(*(n32[k] for k in ("x", "dt", "A", "B", "C", "D")))))
    p32 = inputs((2, 10), 2, 32, 64, 1, "bf16", seed=1)
    cases.append((ssd.SSDError, lambda: f(*(p32[k] for k in ("x", "dt", "A", "B", "C", "D")))))
    s = inputs((2,), 2, 64, 64, 1, "bf16", seed=1)
    b = [s[k] for k in ("x", "dt", "A", "B", "C", "D")]
    cases += [
        (ValueError, lambda: ssd.ssd_causal_step(*b, pool)),
        (ValueError, lambda: ssd.ssd_causal_step(*b, pool.to(torch.bfloat16), slots)),
        (ValueError, lambda: ssd.ssd_causal_step(*b, pool[:2], state_out=big[:3])),
        (ValueError, lambda: ssd.ssd_causal_step(*b, big[:2], state_out=big[1:3])),
    ]
    for exc, call in cases:
        with pytest.raises(exc):
            call()
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0


def test_streams_threads_and_graphs(ssd):
    """Calls from two threads on one stream, on a side stream, and two graphs whose replays overlap."""
    d = inputs((1, 2000), 2, 64, 128, 1, "bf16", seed=4)
    a = [d[k] for k in ("x", "dt", "A", "B", "C", "D")]
    y0, h0 = ssd.ssd_causal_fwd(*a)
    other = [t.flip(0) if t is not None else None for t in a]
    torch.cuda.synchronize()
    got = {}

    def work(i):
        for _ in range(20):
            got[i] = ssd.ssd_causal_fwd(*a)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in ts]
    [t.join() for t in ts]
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i][0], y0) and torch.equal(got[i][1], h0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y1, h1 = ssd.ssd_causal_fwd(*a)
    side.synchronize()
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ssd.ssd_causal_fwd(*other))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    yo, ho = ssd.ssd_causal_fwd(*other)
    torch.cuda.synchronize()
    for y, h in outs:
        assert torch.equal(y, yo) and torch.equal(h, ho)
    assert ssd.ssd_get_device_status() == 0


def test_serving_run(ssd):
    """A run as a server makes it: ragged prompts into a pool, single tokens, a fork, a freed page, a compaction,
    more tokens; every output and page against the recurrence."""
    layers, nslots, H, P, N, G, io = 2, 8, 2, 64, 128, 1, "bf16"
    pool = torch.randn(layers, nslots, H, P, N, device="cuda")
    lens = [140, 3, 77]
    table = torch.tensor([6, 1, 4], dtype=torch.int32, device="cuda")
    ssd.ssd_cache_copy(pool, torch.full((3,), -1, dtype=torch.int32, device="cuda"), table)   # new pages start at zero
    state = {}
    for l in range(layers):
        d = inputs((3, 140), H, P, N, G, io, seed=l, raw=True)
        y, _ = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool[l], slots=table,
                                  seqlens=torch.tensor(lens, dtype=torch.int32, device="cuda"), **opts(d))
        o, oh = ref.fwd(d["x"], sizes(d), d["A"], d["B"], d["C"], d["D"], torch.zeros(3, H, P, N), lens)
        for b in range(3):
            check_out(y[b, :lens[b]], o[b, :lens[b]], io, f"prompt {b}")
            state[l, b] = oh[b]

    def tokens(table, names, seed):
        for l in range(layers):
            d = inputs((len(table),), H, P, N, G, io, seed=100 * seed + l, raw=True)
            y = ssd.ssd_causal_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool[l], table, **opts(d))
            dt = sizes(d)
            for r, name in enumerate(names):
                if name is None:
                    assert (y[r] == 0).all()
                    continue
                o, state[l, name] = ref.scan(d["x"][r][None], dt[r][None], d["A"], d["B"][r][None], d["C"][r][None], d["D"],
                                             state[l, name])
                check_out(y[r][None], o, io, f"token {seed} row {r}")

    tokens(table, [0, 1, 2], 1)
    tokens(table, [0, 1, 2], 2)
    # row 0 forks into pages 7 and 2; row 1 ends
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ssd.ssd_cache_copy(pool, i32(6, 6, -1), i32(7, 2, 1))
    assert (pool[:, 1] == 0).all()
    for l in range(layers):
        state[l, 3], state[l, 4] = state[l, 0], state[l, 0]
    table = i32(6, -1, 4, 7, 2)
    tokens(table, [0, None, 2, 3, 4], 3)
    table, live = ssd.ssd_cache_compact(pool, table)
    assert live.item() == 4 and sorted(table.tolist()) == [-1, 0, 1, 2, 3]
    tokens(table, [0, None, 2, 3, 4], 4)
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0
    for l in range(layers):
        for r, name in enumerate([0, None, 2, 3, 4]):
            if name is not None:
                check_state(pool[l, table[r]], state[l, name], f"layer {l} row {r}")


def test_block_diffusion_cache_rows(ssd):
    """BlockDiffusionCache.copy and .compact on the cache that prefill fills."""
    from bidirectional_mamba_ssd_b200.blockdiff import BlockDiffusionCache
    layers, batch, H, N, L = 2, 6, 2, 64, 40
    cache = BlockDiffusionCache(layers, batch, H, 64, N, device="cuda")
    per = [inputs((batch, L), H, 64, N, 1, "bf16", seed=l) for l in range(layers)]
    st = lambda k: torch.stack([p[k] for p in per]).contiguous()  # noqa: E731
    before = cache.prefill(st("x"), st("dt"), st("A"), st("B")).clone()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.copy(i32(5, -1), i32(1, 2))
    want = before.clone()
    want[:, 1], want[:, 2] = before[:, 5], 0
    torch.cuda.synchronize()
    assert torch.equal(cache.state, want)
    table, live = cache.compact(i32(5, 1, -1, 3))
    torch.cuda.synchronize()
    assert live.item() == 3 and table.tolist() == [2, 1, -1, 0]
    assert torch.equal(cache.state[:, 0], want[:, 3]) and torch.equal(cache.state[:, 2], want[:, 5])


def test_offsets_past_32_bits(ssd):
    """x and out of more than 2^31 elements, and pages of a pool more than 2^32 bytes apart: the last row against a
    call of its own, the last page against the recurrence."""
    batch, L, H, P, N = 2, 16500, 512, 128, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(batch, L, H, P, generator=g, device="cuda", dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    d = inputs((batch, L), H, 64, N, 1, "bf16", seed=4)
    y, h = ssd.ssd_causal_fwd(x, d["dt"], d["A"], d["B"], d["C"], d["D"])
    y1, h1 = ssd.ssd_causal_fwd(x[1:], d["dt"][1:], d["A"], d["B"][1:], d["C"][1:], d["D"])
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0
    assert torch.equal(y[1:], y1) and torch.equal(h[1:], h1)
    del x, y, y1, d
    nslots, H, P, N = 6000, 24, 64, 128
    pool = torch.zeros(nslots, H, P, N, device="cuda")
    assert pool.numel() * 4 > 2 ** 32
    d = inputs((2,), H, P, N, 1, "bf16", seed=5)
    h0 = torch.randn(2, H, P, N, generator=g, device="cuda")
    slots = torch.tensor([nslots - 1, nslots - 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = h0
    one = lambda t: t[:, None]  # noqa: E731
    o, oh = ref.fwd(one(d["x"]), one(sizes(d)), d["A"], one(d["B"]), one(d["C"]), d["D"], h0, [1, 1])
    y = ssd.ssd_causal_step(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool, slots)
    ssd.ssd_cache_copy(pool[None], slots, torch.tensor([1, nslots - 3], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    check_out(y, o[:, 0], "bf16", "last pages")
    check_state(pool[slots.long()], oh, "last pages")
    assert torch.equal(pool[1], pool[nslots - 1]) and torch.equal(pool[nslots - 3], pool[nslots - 2])
    t, live = ssd.ssd_cache_compact(pool[None], slots)
    assert live.item() == 2 and t.tolist() == [1, 0]
    check_state(pool[:2], oh.flip(0), "moved pages")


def test_out_aligned_to_16_bytes_only(ssd):
    """An output 16 bytes off a 32-byte boundary."""
    d = inputs((2, 200), 2, 64, 64, 1, "bf16", seed=6)
    a = [d[k] for k in ("x", "dt", "A", "B", "C", "D")]
    y, h = ssd.ssd_causal_fwd(*a)
    room = torch.zeros(d["x"].numel() + 16, dtype=torch.bfloat16, device="cuda")
    out = room[8:8 + d["x"].numel()].view(d["x"].shape)
    assert out.data_ptr() % 32 == 16
    y2, h2 = ssd.ssd_causal_fwd(*a, out=out)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(h, h2) and (room[:8] == 0).all() and (room[8 + y.numel():] == 0).all()


def test_many_rows_and_all_skipped(ssd):
    """More rows than threads of a block, lengths all over; a batch of padding rows only."""
    batch, L, H, N = 700, 70, 1, 64
    d = inputs((batch, L), H, 64, N, 1, "bf16", seed=13)
    lens = [int(v) for v in torch.randint(0, L + 1, (batch,), generator=torch.Generator().manual_seed(1))]
    lens[300:500] = [0] * 200
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, oh = ref.fwd(d["x"], sizes(d), d["A"], d["B"], d["C"], d["D"], torch.zeros(batch, H, 64, N), lens)
    y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], seqlens=seqlens)
    torch.cuda.synchronize()
    check_out(y, o, "bf16", "many rows")
    check_state(h, oh, "many rows")
    # values outside [0, L] are clamped
    y2, h2 = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"],
                                seqlens=torch.where(seqlens == L, 1 << 30, torch.where(seqlens == 0, -5, seqlens)).to(torch.int32))
    assert torch.equal(y, y2) and torch.equal(h, h2)
    pool = torch.ones(3, H, 64, N, device="cuda")
    none = torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    for path in paths_of(ssd, "bf16"):
        y3, _ = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool, slots=none, path=path)
        torch.cuda.synchronize()
        assert (y3 == 0).all() and (pool == 1).all()
    assert ssd.ssd_get_device_status() == 0


def test_fp32_scan_decay_of_four_tokens(ssd):
    """The CUDA-core scan rescales the state once for four tokens whose decay is at most e^-4: step sizes of 0.1 with
    decays of e^-3.9, e^-4.1 a four, and heads that change within the sequence, at lengths that end inside a four."""
    A = torch.tensor([-9.75, -10.25, -1.0], device="cuda")
    for L in (1, 3, 6, 33, 203):
        d = inputs((1, L), 3, 64, 64, 1, "f32", seed=20 + L)
        d["dt"][:, :, :2] = 0.1
        d["dt"][:, ::7, 2] = 30.0
        h0 = torch.randn(1, 3, 64, 64, generator=d["g"], device="cuda")
        o, oh = ref.fwd(d["x"], sizes(d), A, d["B"], d["C"], d["D"], h0, [L])
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], A, d["B"], d["C"], d["D"], h0)
        torch.cuda.synchronize()
        for k in range(3):
            check_out(y[:, :, k], o[:, :, k], "f32", f"L {L} head {k}")
            check_state(h[:, k], oh[:, k], f"L {L} head {k}")


class _Declines:
    """Stands for the binding's C++ part: leaves every call to the Python way."""
    causal_fwd = causal_step = cache_copy = cache_compact = staticmethod(lambda *a: NotImplemented)


@pytest.mark.parametrize("io,packed,raw", [("bf16", True, True), ("f32", False, False)])
def test_both_ways_of_the_binding(ssd, monkeypatch, io, packed, raw):
    """The C++ and the Python way of the same calls: the same outputs, states, pages and errors; each is taken."""
    from bidirectional_mamba_ssd_b200 import _binding, causal
    d = inputs((3, 70), 2, 64, 64, 1, io, packed=packed, raw=raw, seed=31)
    t = inputs((3,), 2, 64, 64, 1, io, packed=packed, raw=raw, seed=32)
    slots = torch.tensor([4, 1, 3], dtype=torch.int32, device="cuda")
    lens = torch.tensor([70, 0, 33], dtype=torch.int32, device="cuda")
    src, dst = slots, torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    ws = ssd.Workspace(torch.device("cuda", 0))
    ws.get(1 << 24)
    names = ("causal_fwd", "causal_step", "cache_copy", "cache_compact")

    def run():
        pool = torch.ones(2, 6, 2, 64, 64, device="cuda")
        given = torch.empty(3, 2, 64, dtype=t["x"].dtype, device="cuda")
        got = list(ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool[0], slots=slots, seqlens=lens,
                                      workspace=ws, **opts(d)))
        got += list(ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], path=ssd.SSD_PATH_SIMT, workspace=ws, **opts(d)))
        assert got[1].data_ptr() == pool[0].data_ptr()
        ssd.ssd_cache_copy(pool, src, dst, workspace=ws)
        got.append(ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], pool[0], dst, workspace=ws, **opts(t)))
        y = ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], None, pool[1, :3], out=given,
                                state_out=pool[1, 3:], **opts(t))
        assert y is given
        got += [y, pool]
        got += list(ssd.ssd_cache_compact(pool, slots, workspace=ws))
        with pytest.raises(ssd.SSDError):
            ssd.ssd_causal_step(t["x"][..., :32].contiguous(), t["dt"], t["A"], t["B"], t["C"], None, pool[0, :3, :, :32].contiguous())
        with pytest.raises(ValueError):
            ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], None, pool[0, :3], state_out=pool.view(-1)[64:].narrow(
                0, 0, 3 * 2 * 64 * 64).view(3, 2, 64, 64))
        torch.cuda.synchronize()
        assert ws.status() == 0
        return [g.clone() for g in got]

    took = []
    spy = type("Spy", (), {n: staticmethod(lambda *a, n=n: _took(took, n, getattr(_binding, n)(*a))) for n in names})
    monkeypatch.setattr(causal, "_binding", spy)
    first = run()
    assert set(took) == set(names)
    monkeypatch.setattr(causal, "_binding", _Declines)
    for k, (a, b) in enumerate(zip(first, run())):
        assert a.dtype == b.dtype and torch.equal(a, b), f"result {k}"


def _took(took, name, got):
    if got is not NotImplemented:
        took.append(name)
    return got


def test_no_rows_of_a_pool(ssd, monkeypatch):
    """A batch of no rows with slots: the pool comes back as it is, or, with no pool, the call is refused, either way."""
    from bidirectional_mamba_ssd_b200 import causal
    d, t = inputs((0, 5), 2, 64, 64, 1, "f32", seed=1), inputs((0,), 2, 64, 64, 1, "f32", seed=1)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    pool = torch.randn(3, 2, 64, 64, device="cuda")
    was = pool.clone()
    for declines in (False, True):
        if declines:
            monkeypatch.setattr(causal, "_binding", _Declines)
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], None, pool, slots=none)
        assert y.shape == (0, 5, 2, 64) and h is pool
        assert ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], None, pool, none).shape == (0, 2, 64)
        with pytest.raises(ValueError):
            ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], slots=none)
        with pytest.raises((TypeError, ValueError)):
            ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], None, pool)
    assert torch.equal(pool, was)


def test_workspaces_of_the_binding(ssd):
    """A workspace that has yet to be made, one that is too small, one of something else, and one whose lock is held."""
    import threading
    d = inputs((2, 300), 2, 64, 64, 1, "bf16", seed=3)
    call = lambda ws: ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], workspace=ws)  # noqa: E731
    want = call(None)[0]
    ws = ssd.Workspace(torch.device("cuda", 0))
    assert torch.equal(call(ws)[0], want)
    ws.buf = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(ws)[0], want) and ws.buf.numel() > 256
    with pytest.raises(AttributeError):
        call(object())
    got = []
    with ws.lock:
        th = threading.Thread(target=lambda: got.append(call(ws)[0]))
        th.start()
        th.join(0.2)
        assert not got
    th.join()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and ws.status() == 0


def test_first_call_of_a_thread(ssd):
    """A thread whose first CUDA call this is, of each operator: there is no current context yet."""
    import threading
    d, t = inputs((2, 300), 2, 64, 64, 1, "bf16", seed=3), inputs((2,), 2, 64, 64, 1, "bf16", seed=4)
    pool = torch.randn(1, 4, 2, 64, 64, device="cuda")
    idx = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    z = si.bidir_inputs(8, 300, 24, 64, 128, 24, "bf16", seed=5, device="cuda")
    both = [z[k] for k in ("x", "dt", "A", "B", "C", "D")]
    calls = [lambda: ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"])[0],
             lambda: ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], path=ssd.SSD_PATH_SIMT)[0],
             lambda: ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], None, pool[0].clone(), idx),
             lambda: ssd.ssd_cache_copy(pool.clone(), idx, idx + 1), lambda: ssd.ssd_cache_compact(pool.clone(), idx)[0],
             lambda: ssd.ssd_bidir_fwd(*both)]
    for k, call in enumerate(calls):
        want, got = call(), []
        torch.cuda.synchronize()
        th = threading.Thread(target=lambda: got.append(call()))
        th.start()
        th.join()
        torch.cuda.synchronize()
        assert got and torch.equal(got[0], want), f"call {k}"
