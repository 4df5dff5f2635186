"""GPU tests of the causal serving operators at the edges of what a call may be
given, against the recurrence in 64 bits (causal_ref), at the tolerances of
test_causal_gpu where a test derives none of its own."""
import ctypes
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import causal_ref as ref
from test_causal_gpu import check_out, check_state, inputs, opts, paths_of, sizes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssd():
    import bidirectional_mamba_ssd_b200 as m
    return m


def rounding_bound(x, dt, A, B, C, h0, y, o):
    """How far one row's bf16 outputs y (L, H, P) may be from the exact o, element by element, without a skip term.

    A tile of 128 tokens from the state H entering it: y_t = sum_s G_ts e_ts dt_s x_s + e_t C_t H. The kernel rounds G e dt
    and H to bf16 (2^-8 of each at most) and the output (half a step). The rest is fp32: exponents up to 320 that are sums of
    128 step sizes (each addition off by 2^-24 of up to 320: 8 additions a sum are 1.6e-4 = 2^-12.6, and a difference of two
    twice that), and sums of 256 products (256 x 2^-23 = 2^-15 of the products' magnitudes). So, with E the sum of the
    magnitudes of the terms and F the same with every product of C and B by itself,
        |y - o| <= (2^-8 + 2^-11) E + 2^-14 F + half a step of the output."""
    x, dt, A, B, C, h = (t.double().cpu() for t in (x, dt, A, B, C, h0))
    L, H, _ = x.shape
    group = torch.arange(H) // (H // B.shape[1])
    E, F = torch.zeros_like(x), torch.zeros_like(x)
    for t0 in range(0, L, 128):
        t1 = min(L, t0 + 128)
        xs, Bs, Cs, ds = x[t0:t1].transpose(0, 1), B[t0:t1, group].transpose(0, 1), C[t0:t1, group].transpose(0, 1), dt[t0:t1].T
        a = torch.cumsum(ds * A[:, None], 1)
        e = torch.exp((a[:, :, None] - a[:, None, :]).masked_fill(~torch.ones(t1 - t0, t1 - t0, dtype=bool).tril(), -np.inf))
        w, in_ = e * ds[:, None, :], torch.exp(a)[:, :, None]
        at_start = in_ * (Cs.abs() @ h.abs().transpose(1, 2))
        E[t0:t1] = ((((Cs @ Bs.transpose(1, 2)).abs() * w) @ xs.abs()) + at_start).transpose(0, 1)
        F[t0:t1] = ((((Cs.abs() @ Bs.abs().transpose(1, 2)) * w) @ xs.abs()) + at_start).transpose(0, 1)
        h = torch.exp(a[:, -1])[:, None, None] * h + ((ds * torch.exp(a[:, -1:] - a))[:, :, None] * xs).transpose(1, 2) @ Bs
    top = torch.maximum(y.abs(), o.abs()).clamp(min=2.0 ** -126)
    return (2 ** -8 + 2 ** -11) * E + 2 ** -14 * F + 0.5 * torch.exp2(torch.floor(torch.log2(top)) - 7)


# factors on x (and the start state), on B and on C, of the usual inputs (1, 1/8, 1/8)
SCALES = [(1.0, 1.0), (1e-15, 1.0), (1e-8, 1.0), (1e-7, 1.0), (1e4, 80.0), (500.0, 400.0), (1e12, 8.0)]


@pytest.mark.parametrize("scale", SCALES, ids=lambda s: "x%g_bc%g" % s)
def test_fwd_decays_at_any_magnitude(ssd, scale):
    """A tile of 128 tokens decays by e^-60 to e^-320, both sides of the spans where the masked matrix changes its
    references among them, with inputs and start states of any magnitude and no skip term."""
    spans = [60.0, 79.5, 80.5, 120.0, 149.8, 159.0, 161.0, 320.0]
    d = inputs((1, 300), len(spans), 64, 128, 2, "bf16", seed=41)
    d["dt"].fill_(0.1)
    A = -torch.tensor(spans, device="cuda") / (128 * d["dt"][0, 0, 0].float())
    x, B, C = d["x"] * scale[0], d["B"] * scale[1], d["C"] * scale[1]
    h0 = torch.randn(1, len(spans), 64, 128, generator=d["g"], device="cuda") * scale[0]
    o, oh = ref.fwd(x, sizes(d), A, B, C, None, h0, [300])
    assert np.isfinite(o.to(torch.bfloat16).float().numpy()).all()
    y, h = ssd.ssd_causal_fwd(x, d["dt"], A, B, C, None, h0)
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0
    y = y.double().cpu()
    assert torch.isfinite(y).all(), [s for k, s in enumerate(spans) if not torch.isfinite(y[:, :, k]).all()]
    off = (y - o).abs()[0] / rounding_bound(x[0], sizes(d)[0], A, B[0], C[0], h0[0], y[0], o[0])
    for k, s in enumerate(spans):
        assert off[:, k].max() <= 1, f"decay {s}: {off[:, k].max():.2f} of the bound"
        check_state(h[:, k], oh[:, k], f"decay {s}")


@pytest.mark.parametrize("L", [1, 130])
def test_a_tokens_own_term_against_the_skip_term(ssd, L):
    """A token's own C.B dt x and its skip term may nearly cancel (single tokens, or decays that leave nothing else): both are
    kept in fp32. A sum G of 128 products in fp32 is off by at most 128 x 2^-24 of their magnitudes F, the two exponentials
    that make 1 by 2^-20 (2^-21 each), so
        |y - o| <= (2^-17 F + 2^-20 |G|) dt |x| + 2^-23 (|G| dt + |D|) |x| + half a step of the output."""
    B_, H, P, N = 3, 4, 64, 128
    d = inputs((B_, L), H, P, N, H, "bf16", seed=80 + L)
    d["dt"].fill_(0.1)
    d["B"], d["C"] = d["B"][:1, :1].repeat(B_, L, 1, 1), d["C"][:1, :1].repeat(B_, L, 1, 1)     # one G a head
    # L = 1: masks of one factor (decays of e^-0.1, e^-10, e^-70) and of exponentials (e^-120); L = 130: of exponentials, and
    # e^-50 or less is left of a token at the next
    A = -torch.tensor([5e2, 6e2, 1e3, 1e4], device="cuda") if L > 1 else -torch.tensor([1.0, 100.0, 700.0, 1200.0], device="cuda")
    dt = d["dt"].double().cpu()[0, 0]
    Bd, Cd, x = (d[k].double().cpu() for k in ("B", "C", "x"))
    G, F = (Bd[0, 0] * Cd[0, 0]).sum(-1), (Bd[0, 0] * Cd[0, 0]).abs().sum(-1)
    D = (-(G * dt) * (1 - 2 ** -6)).float().cuda()
    o, oh = ref.fwd(d["x"], d["dt"].double().cpu(), A, d["B"], d["C"], D, torch.zeros(B_, H, P, N), [L] * B_)
    y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], A, d["B"], d["C"], D)
    torch.cuda.synchronize()
    y = y.double().cpu()
    unit = ((2 ** -17 * F + 2 ** -20 * G.abs()) * dt + 2 ** -23 * (G.abs() * dt + D.double().cpu().abs()))[:, None] * x.abs()
    top = torch.maximum(y.abs(), o.abs()).clamp(min=2.0 ** -126)
    off = (y - o).abs() / (unit + 0.5 * torch.exp2(torch.floor(torch.log2(top)) - 7))
    for k in range(H):
        assert off[:, :, k].max() <= 1, f"head {k}: {off[:, :, k].max():.2f} of the bound"
    check_state(h, oh, "states")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("hi", [0.1, float("inf")])
def test_nan_in_a_raw_step_size_shows(ssd, io, hi):
    """A raw step size of NaN makes its head's outputs from there on, and its state, NaN; other heads are as they were."""
    d = inputs((2, 300), 3, 64, 64, 1, io, seed=42, raw=True)
    kw = dict(dt_bias=d["dt_bias"], dt_min=0.0, dt_max=hi)
    bad = d["dt"].clone()
    bad[1, 200, 1] = float("nan")
    a = [d[k] for k in ("A", "B", "C", "D")]
    for path in paths_of(ssd, io):
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], *a, path=path, **kw)
        z, g = ssd.ssd_causal_fwd(d["x"], bad, *a, path=path, **kw)
        torch.cuda.synchronize()
        assert torch.isnan(z[1, 200:, 1]).all() and torch.isnan(g[1, 1]).all(), f"path {path}"
        for b, k in ((0, 0), (0, 1), (0, 2), (1, 0), (1, 2)):
            assert torch.equal(z[b, :, k], y[b, :, k]) and torch.equal(g[b, k], h[b, k]), f"path {path}"
    t = [v[:, 200].contiguous() for v in (d["x"], bad, d["B"], d["C"])]
    st = torch.zeros(2, 3, 64, 64, device="cuda")
    y = ssd.ssd_causal_step(t[0], t[1], d["A"], t[2], t[3], d["D"], st, **kw)
    torch.cuda.synchronize()
    assert torch.isnan(y[1, 1]).all() and torch.isnan(st[1, 1]).all()
    assert torch.isfinite(y[0]).all() and torch.isfinite(st[0]).all() and torch.isfinite(y[1, [0, 2]]).all()


# lengths, H, P, N, G: 148 units or more, so that units are cut between neighbouring CTAs
CUT = [([2500, 0, 300, 1, 129, 128, 0, 257, 700, 64, 5, 127, 130, 256, 999, 1500], 10, 64, 128, 1),
       ([1, 7, 3000, 2, 100, 0, 384, 385, 50, 640], 8, 128, 64, 2),
       ([400] * 25, 6, 64, 128, 3)]


@pytest.mark.parametrize("case", CUT, ids=["one_long", "two_halves", "even"])
def test_units_cut_over_several_ctas(ssd, case):
    """Ragged prompts into a pool in place, with padding, bad and repeated slots, of so many units that the tiles of a unit
    are shared by neighbouring CTAs, by three and more of them where one prompt is long; the same again, bit by bit."""
    lens, H, P, N, G = case
    batch, L = len(lens), max(lens)
    nslots = batch + 4
    d = inputs((batch, L), H, P, N, G, "bf16", seed=43 + batch, raw=True, packed=True)
    pool = torch.randn(nslots, H, P, N, generator=d["g"], device="cuda") * 0.3
    slots = torch.randperm(nslots, generator=d["g"], device="cuda")[:batch].to(torch.int32)
    slots[3], slots[4], slots[5] = -1, nslots, slots[0]
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    good = [b for b in range(batch) if b not in (3, 4, 5)]
    behind = torch.arange(L, device="cuda")[None, :] >= seqlens[:, None]
    o, oh = ref.fwd(d["x"][good], sizes(d)[good], d["A"], d["B"][good], d["C"][good], d["D"], pool[slots[good].long()],
                    [lens[b] for b in good])
    for k in ("x", "dt", "B", "C"):
        d[k][behind] = float("nan")
    got = []
    for _ in range(3):
        st, out = pool.clone(), torch.full((batch, L, H, P), 7.0, dtype=torch.bfloat16, device="cuda")
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], st, seqlens=seqlens, slots=slots, out=out,
                                  **opts(d))
        torch.cuda.synchronize()
        assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX and y is out and h is st
        got.append((y, h))
    assert all(torch.equal(a, b) for pair in got[1:] for a, b in zip(pair, got[0]))
    assert (y[behind] == 0).all() and (y[[3, 4, 5]] == 0).all()
    for k, b in enumerate(good):
        if lens[b]:
            check_out(y[b, :lens[b]], o[k, :lens[b]], "bf16", f"row {b}")
        check_state(h[slots[b]], oh[k], f"row {b}")
    rest = sorted(set(range(nslots)) - set(slots[good].tolist()))
    assert torch.equal(h[rest], pool[rest])


def test_fp32_scan_decays_around_its_border(ssd):
    """The CUDA-core scan rescales the state once for four tokens that decay by at most e^-8: step sizes of 0.1 with decays
    of e^-7.8 and e^-8.2 a four, and a head that changes within the sequence, at lengths that end inside a four."""
    A = torch.tensor([-19.5, -20.5, -1.0], device="cuda")
    for L in (1, 3, 6, 33, 203, 700):
        d = inputs((1, L), 3, 64, 64, 1, "f32", seed=60 + L)
        d["dt"][:, :, :2] = 0.1
        d["dt"][:, ::7, 2] = 30.0
        h0 = torch.randn(1, 3, 64, 64, generator=d["g"], device="cuda")
        o, oh = ref.fwd(d["x"], sizes(d), A, d["B"], d["C"], d["D"], h0, [L])
        y, h = ssd.ssd_causal_fwd(d["x"], d["dt"], A, d["B"], d["C"], d["D"], h0)
        torch.cuda.synchronize()
        for k in range(3):
            check_out(y[:, :, k], o[:, :, k], "f32", f"L {L} head {k}")
            check_state(h[:, k], oh[:, k], f"L {L} head {k}")


@pytest.mark.parametrize("io,path", [("f32", "SIMT"), ("bf16", "SIMT"), ("bf16", "AUTO")])
def test_rows_behind_a_sequence_past_31_bits(ssd, io, path):
    """A padded sequence of so many rows that its 16-byte pieces do not count in 31 bits: all rows behind its 300 tokens
    are zero. (x, B and C are one array, of which only the tokens are ever set.)"""
    torch.cuda.empty_cache()
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[io]
    L, lens = 2 ** 31 * 16 // (64 * dtype.itemsize) + 1000, 300
    if torch.cuda.mem_get_info()[0] < 2 * L * 64 * dtype.itemsize + (8 << 30):
        pytest.skip("not enough free memory")
    d = inputs((1, lens), 1, 64, 64, 1, io, seed=70)
    x = torch.empty(1, L, 1, 64, dtype=dtype, device="cuda")
    dt = torch.empty(1, L, 1, dtype=dtype, device="cuda")
    x[:, :lens], dt[:, :lens] = d["x"], d["dt"]
    out = torch.full_like(x, 7.0)
    seqlens = torch.tensor([lens], dtype=torch.int32, device="cuda")
    y, h = ssd.ssd_causal_fwd(x, dt, d["A"], x, x, d["D"], seqlens=seqlens, out=out, path=getattr(ssd, "SSD_PATH_" + path))
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0
    for part in y.view(-1)[lens * 64:].split(1 << 28):
        assert not part.any()
    o, oh = ref.fwd(d["x"], sizes(d), d["A"], d["x"], d["x"], d["D"], torch.zeros(1, 1, 64, 64), [lens])
    check_out(y[:, :lens], o, io, path)
    check_state(h, oh, path)
    del x, out, y, dt
    torch.cuda.empty_cache()


@pytest.mark.parametrize("width", [4, 1])
def test_pools_of_two_sizes_at_once(ssd, width):
    """Copies and compactions of large and of small pools from four threads, on streams and workspaces of their own: the
    kernels' shared memory depends on the number of slots. (Through the C ABI, which gives the other threads the most time
    between a call's steps.)"""
    v, refused = ctypes.c_void_p, []
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731

    def work(nslots, number):
        pool = torch.full((1, nslots, width), float(number), device="cuda")
        pool[0, 2:] = 0.0
        stream, src, dst, live = torch.cuda.Stream(), i32(0, 1), i32(2, 3), i32(0)
        ws, new = torch.zeros(256, dtype=torch.uint8, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        head, tail = (v(pool.data_ptr()), 4 * width, 1, nslots), (v(ws.data_ptr()), 256, v(stream.cuda_stream))
        copy = (*head, v(src.data_ptr()), v(dst.data_ptr()), 2, *tail)
        compact = (*head, v(src.data_ptr()), 2, v(new.data_ptr()), v(live.data_ptr()), *tail)
        for i in range(4000):
            rc = ssd.lib.ssd_cache_copy(*copy), ssd.lib.ssd_cache_compact(*compact)
            if rc != (0, 0):
                refused.append((nslots, i, rc))
        stream.synchronize()
        if not (pool[0, :4] == number).all() or pool[0, 4:].any() or live.item() != 2 or new.tolist() != [0, 1]:
            refused.append((nslots, "pages"))

    ts = [threading.Thread(target=work, args=a) for a in ((200000, 1), (4, 2), (262144, 3), (4, 4))]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not refused, (len(refused), refused[:3])


def _captured_calls(ssd):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t = inputs((2,), 2, 64, 64, 1, "bf16", seed=51)
    d = inputs((2, 300), 2, 64, 64, 1, "bf16", seed=52)
    w = inputs((2500,), 1, 64, 64, 1, "bf16", seed=53)
    pool, wide = torch.zeros(4, 2, 64, 64, device="cuda"), torch.zeros(2600, 1, 64, 64, device="cuda")
    slots, many = i32(1, 0), torch.arange(2500, dtype=torch.int32, device="cuda")
    pages, to = i32(1, 0), i32(3, 2)
    f = ssd.ssd_causal_fwd
    return {
        "step": (slots, lambda: ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], pool, slots)),
        "many": (many, lambda: ssd.ssd_causal_step(w["x"], w["dt"], w["A"], w["B"], w["C"], w["D"], wide, many)),
        "copy": (pages, lambda: ssd.ssd_cache_copy(pool[None], pages, to)),
        "compact": (pages, lambda: ssd.ssd_cache_compact(pool[None], pages)),
        "prompt": (slots, lambda: f(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool, slots=slots)),
        "scan": (slots, lambda: f(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], pool, slots=slots, path=ssd.SSD_PATH_SIMT)),
    }


@pytest.mark.parametrize("name", ["step", "many", "copy", "compact", "prompt", "scan"])
def test_bad_index_in_a_replay_is_reported(ssd, name):
    """Captured without a workspace: an index that is bad at a replay is reported by ssd_get_device_status, once, on
    whatever stream the graph runs; an index that is good again is not."""
    idx, call = _captured_calls(ssd)[name]
    good = idx.clone()
    call()                                    # loads the kernels
    torch.cuda.synchronize()
    assert ssd.ssd_get_device_status() == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            g.replay()
            assert ssd.ssd_get_device_status() == 0
            idx[1] = 100000
            g.replay()
            idx.copy_(good)
            g.replay()
            assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX
            assert ssd.ssd_get_device_status() == 0
            stream.synchronize()


def test_captured_calls_add_no_fill(ssd):
    """A captured single token, copy and compaction are one node each."""
    cudart = ctypes.CDLL("libcudart.so.12")
    for name in ("step", "copy", "compact"):
        _, call = _captured_calls(ssd)[name]
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(g):
            call()
        n = ctypes.c_size_t()
        assert cudart.cudaGraphGetNodes(ctypes.c_void_p(g.raw_cuda_graph()), None, ctypes.byref(n)) == 0
        assert n.value == 1, f"{name}: {n.value} nodes"


FIRST = """
import sys
sys.path.insert(0, %r)
import torch
import bidirectional_mamba_ssd_b200 as ssd
x, dt, bc = (torch.ones(2, *s, device="cuda") for s in ((2, 64), (2,), (1, 64)))
A, pool = -torch.ones(2, device="cuda"), torch.zeros(4, 2, 64, 64, device="cuda")
slots = torch.tensor([1, 9], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = ssd.ssd_causal_step(x, dt, A, bc, bc, None, pool, slots)
    z, _ = ssd.ssd_causal_fwd(x[:, None], dt[:, None], A, bc[:, None], bc[:, None], None, pool, slots=slots)
assert ssd.ssd_get_device_status() == 0
g.replay()
assert ssd.ssd_get_device_status() == ssd.SSD_ERR_INDEX
# h = 1, then exp(-1) + 1; 64 of them a sum
want = torch.tensor([64.0, 64 * (1 + torch.exp(torch.tensor(-1.0)).item())])
assert torch.allclose(torch.stack([y[0, 0, 0], z[0, 0, 0, 0]]).cpu(), want, rtol=1e-5), (y[0, 0, 0], z[0, 0, 0, 0])
assert (y[1] == 0).all() and (z[1] == 0).all()
"""


def test_first_calls_of_a_process_are_captured():
    """Nothing has been called before the capture: neither the kernels nor the library's own header are loaded yet."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST % root], capture_output=True, text=True, timeout=120)
    assert done.returncode == 0, done.stderr[-2000:]


def test_status_outlives_a_larger_workspace(ssd):
    """A bad slot is reported although a later call on the same stream has made the workspace grow since."""
    t = inputs((2,), 2, 64, 64, 1, "bf16", seed=54)
    d = inputs((2, 300), 2, 64, 64, 1, "bf16", seed=55)
    pool = torch.zeros(4, 2, 64, 64, device="cuda")
    slots = torch.tensor([1, 9], dtype=torch.int32, device="cuda")
    for ws in (ssd.Workspace(), None):
        with torch.cuda.stream(torch.cuda.Stream()):
            ssd.ssd_causal_step(t["x"], t["dt"], t["A"], t["B"], t["C"], t["D"], pool, slots, workspace=ws)
            ssd.ssd_causal_fwd(d["x"], d["dt"], d["A"], d["B"], d["C"], d["D"], workspace=ws)
            assert ssd.ssd_get_device_status(ws) == ssd.SSD_ERR_INDEX
            assert ssd.ssd_get_device_status(ws) == 0
