"""Host-only checks of the causal serving operators' C ABI: workspace sizes, and
bad arguments rejected before anything is launched (these calls never reach the
GPU)."""
import ctypes

import pytest

FAKE = 1 << 20  # a 16-byte aligned non-null address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    from bidirectional_mamba_ssd_b200 import build as b
    b.build()
    from bidirectional_mamba_ssd_b200 import _lib
    return _lib.load()


def test_causal_entry_points_reject_bad_arguments(lib):
    v, f = ctypes.c_void_p, ctypes.c_float

    def fwd(ptr=(FAKE,) * 5, A=FAKE, D=0, bias=0, lo=0.0, hi=1.0, lens=0, slots=0, init=0, so=FAKE, st=None, nslots=2,
            batch=2, L=300, H=4, P=64, N=128, G=2, dtype=1, path=0, ws=FAKE, wsb=1 << 40):
        x, dt, B, C, out = ptr
        st = st or [L * H * P, H * P, L * H, H, L * G * N, G * N, L * G * N, G * N]
        return lib.ssd_causal_fwd(v(x), v(dt), v(A), v(B), v(C), v(D), v(bias), f(lo), f(hi), v(lens), v(slots), v(init),
                                  v(so), v(out), *st, nslots, batch, L, H, P, N, G, dtype, path, v(ws), wsb, None)

    assert fwd(P=32) == -2 and fwd(P=96) == -2 and fwd(P=320) == -2
    assert fwd(N=32) == -2 and fwd(dtype=3) == -2 and fwd(G=3) == -1 and fwd(batch=-1) == -1
    assert fwd(batch=1 << 16, L=1 << 16) == -2
    assert fwd(ws=0) == -4 and fwd(wsb=100) == -4 and fwd(ws=FAKE + 4) == -1
    assert fwd(path=5) == -1
    assert fwd(bias=FAKE, lo=0.2, hi=0.1) == -1 and fwd(bias=FAKE, lo=float("nan")) == -1
    assert fwd(slots=FAKE, nslots=-1) == -1 and fwd(slots=FAKE + 2) == -1 and fwd(lens=FAKE + 1) == -1
    assert fwd(init=FAKE + 4) == -1 and fwd(so=FAKE + 4) == -1 and fwd(A=0) == -1
    for i in range(5):
        p = [FAKE] * 5
        p[i] = 0
        assert fwd(ptr=p) == -1, i
        p[i] = FAKE + 1
        assert fwd(ptr=p) == -1, i
    ok = [300 * 256, 256, 300 * 4, 4, 300 * 256, 256, 300 * 256, 256]
    for i, bad in ((0, 0), (0, 255), (1, 252), (1, -256), (2, 3), (3, 0), (4, 128), (5, 257), (6, 1 << 37), (7, 8)):
        st = list(ok)
        st[i] = bad
        assert fwd(st=st) == -1, (i, bad)
    assert fwd(batch=0, ptr=(0,) * 5) == 0
    op = 6
    assert lib.ssd_workspace_bytes(op, 2, 300, 4, 128, 128, 2, 0, 1) >= 512
    assert lib.ssd_workspace_bytes(op, 2, 300, 4, 96, 128, 2, 0, 1) == 0
    # a long sequence in segments needs their states
    assert lib.ssd_workspace_bytes(op, 1, 65536, 4, 64, 128, 4, 0, 0) > 4 * 64 * 128 * 4 * 2


def test_step_and_cache_entry_points_reject_bad_arguments(lib):
    v, f = ctypes.c_void_p, ctypes.c_float

    def step(ptr=(FAKE,) * 7, slots=0, st=(256, 4, 256, 256), nslots=2, batch=2, H=4, P=64, N=128, G=2, dtype=1, ws=0, wsb=0):
        x, dt, B, C, s, so, out = ptr
        return lib.ssd_causal_step(v(x), v(dt), v(FAKE), v(B), v(C), v(0), v(0), f(0), f(1), v(slots), v(s), v(so), v(out),
                                   *st, nslots, batch, H, P, N, G, dtype, v(ws), wsb, None)

    assert step(P=32) == -2 and step(N=96) == -2 and step(G=3) == -1 and step(dtype=9) == -2
    assert step(slots=FAKE) == -4 and step(slots=FAKE, ws=FAKE, wsb=255) == -4
    assert step(slots=FAKE, ws=FAKE, wsb=256, batch=2049) == -4      # resolved rows need room
    assert step(st=(0, 4, 256, 256)) == -1 and step(st=(256, 4, 260, 256)) == -1
    for i in range(7):
        p = [FAKE] * 7
        p[i] = 0
        assert step(ptr=p) == -1, i
    assert step(batch=0, ptr=(0,) * 7) == 0

    def copy(pool=FAKE, page=64, layers=2, nslots=4, src=FAKE, dst=FAKE, n=3, ws=FAKE, wsb=256):
        return lib.ssd_cache_copy(v(pool), page, layers, nslots, v(src), v(dst), n, v(ws), wsb, None)

    assert copy(page=-1) == -1 and copy(n=-1) == -1 and copy(nslots=-1) == -1 and copy(layers=-1) == -1
    assert copy(nslots=(1 << 18) + 1) == -2 and copy(ws=0) == -4 and copy(wsb=8) == -4
    assert copy(pool=0) == -1 and copy(src=0) == -1 and copy(dst=FAKE + 2) == -1
    assert copy(n=0, src=0, dst=0, pool=0) == 0 and copy(page=0, pool=0) == 0

    def compact(pool=FAKE, page=64, layers=2, nslots=4, table=FAKE, rows=3, out=FAKE + 64, live=FAKE, ws=FAKE, wsb=256):
        return lib.ssd_cache_compact(v(pool), page, layers, nslots, v(table), rows, v(out), v(live), v(ws), wsb, None)

    assert compact(rows=-1) == -1 and compact(nslots=(1 << 18) + 1) == -2 and compact(ws=0) == -4
    assert compact(pool=0) == -1 and compact(table=0) == -1 and compact(out=0) == -1 and compact(live=0) == -1
    assert compact(out=FAKE) == -1 and compact(out=FAKE + 8) == -1       # the tables overlap


def test_binding_leaves_what_is_not_its_own():
    """The C++ part of the binding makes no call of CPU tensors or of things that are none, and raises nothing for them."""
    import torch
    from bidirectional_mamba_ssd_b200 import _binding
    x = torch.zeros(2, 3, 4)
    for a in (x, None, 1, "x", torch.zeros(2, 3, 4, 5), torch.empty(3, 4, 5, device="meta")):
        assert _binding.causal_fwd(*[a] * 16) is NotImplemented
        assert _binding.causal_step(*[a] * 14) is NotImplemented
        assert _binding.cache_copy(*[a] * 4) is NotImplemented
        assert _binding.cache_compact(*[a] * 3) is NotImplemented
    with pytest.raises(TypeError):
        _binding.causal_step(x)
