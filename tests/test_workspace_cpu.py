"""Host-only checks of the Workspace class and of who holds its lock (nothing is
launched: the library's calls are replaced by recorders)."""
import copy
import pickle

import pytest
import torch

B, L, H, P, N, G = 2, 8, 2, 64, 64, 1


@pytest.fixture(scope="module")
def ssd():
    import __graft_entry__
    __graft_entry__.build()
    import bidirectional_mamba_ssd_b200 as m
    return m


def calls(ssd, ws):
    """Every entry point that takes a workspace and is called over ctypes, with small CPU tensors."""
    io = torch.bfloat16
    z = lambda *s: torch.zeros(*s, dtype=io)  # noqa: E731
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    x, dt, bc, A = z(B, L, H, P), z(2, B, L, H), z(2, B, L, G, N), f(2, H)
    layers = (x[None], dt[:1], A[:1], bc[:1])
    cin = H * P + 2 * G * N
    block = (z(B, L, cin), x, dt, f(2, cin, 4), f(2, cin), A, A, A, f(H * P))
    return {
        "ssd_bidir_fwd": lambda: ssd.ssd_bidir_fwd(x, dt, A, bc, bc, A, workspace=ws),
        "ssd_bidir_bwd": lambda: ssd.ssd_bidir_bwd(x, dt, A, bc, bc, A, x, workspace=ws),
        "ssd_block_step_bwd": lambda: ssd.ssd_block_step_bwd(x, dt, A, bc, bc, A, None, x, workspace=ws),
        "ssd_bidir_fwd_x2": lambda: ssd.ssd_bidir_fwd_x2(torch.stack([x, x]), dt, A, bc, bc, A, workspace=ws),
        "ssd_prefix_state": lambda: ssd.ssd_prefix_state(x, dt[0], A[0], bc[0], workspace=ws),
        "ssd_prefix_state_layers": lambda: ssd.ssd_prefix_state_layers(*layers, workspace=ws),
        "ssd_block_step": lambda: ssd.ssd_block_step(x, dt, A, bc, bc, A, None, workspace=ws),
        "ssd_segment_states": lambda: ssd.ssd_segment_states(x, dt, A, bc, workspace=ws),
        "ssd_bidir_fwd_seeded": lambda: ssd.ssd_bidir_fwd_seeded(x, dt, A, bc, bc, A, workspace=ws),
        "ssd_bidir_fwd_dtraw": lambda: ssd.ssd_bidir_fwd_dtraw(x, dt, A, A, bc, bc, A, workspace=ws),
        "ssd_mixer_block_fwd": lambda: ssd.ssd_mixer_block_fwd(*block, H, G, N, workspace=ws),
    }


@pytest.mark.parametrize("name", sorted(calls(None, None)))
def test_every_call_holds_its_workspace(ssd, monkeypatch, name):
    """A call's launches share the workspace's buffer: its lock is held from the buffer's choice to the last launch, so that
    no other thread's call on the same stream comes between them."""
    ws = ssd.Workspace("cpu")
    made = []

    class Lib:
        ssd_workspace_bytes = staticmethod(lambda *a: 4096)

        def __getattr__(self, entry):
            def call(*a):
                made.append((entry, ws.lock.locked()))
                return 0
            return call

    monkeypatch.setattr(ssd, "lib", Lib())
    monkeypatch.setattr(ssd, "_need", lambda *a, **k: None)
    monkeypatch.setattr(ssd, "_stream", lambda device: 0)
    calls(ssd, ws)[name]()
    assert made and all(held for _, held in made), made
    assert not ws.lock.locked()


def test_a_larger_buffer_keeps_the_status_header(ssd):
    ws = ssd.Workspace("cpu")
    ws.get(300)[:256] = torch.arange(256, dtype=torch.uint8)
    ws.buf[256:] = 9
    buf = ws.get(1000)
    assert buf.numel() == 1000 and buf[:256].tolist() == list(range(256)) and not buf[256:].any()
    assert ws.get(500) is buf


def test_copies_and_stored_workspaces(ssd):
    """A workspace, and an object that holds one, can be copied and stored; a copy has a buffer and a lock of its own."""
    ws = ssd.Workspace("cpu")
    ws.get(300)[0] = 7
    with ws.lock:
        twins = [copy.deepcopy(ws), pickle.loads(pickle.dumps(ws)), copy.deepcopy({"cache": [ws]})["cache"][0]]
    for w in twins:
        assert w.device == ws.device and w.buf[0] == 7 and w.buf.data_ptr() != ws.buf.data_ptr()
        assert w.lock is not ws.lock and not w.lock.locked()
        assert w.get(400).numel() == 400
    same = copy.copy(ws)
    assert same.buf is ws.buf and same.lock is ws.lock
