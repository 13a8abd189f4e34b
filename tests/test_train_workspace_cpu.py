"""The binding's own workspaces, on a library whose entry points only note their calls."""

import threading
import time

import pytest
import torch

STREAM = 77          # no stream of a device: nothing here reaches one


class Library:
    """Entry points that take a while, as the launches of one call do."""

    def __init__(self, mod, need=4096):
        self.mod, self.need, self.calls, self.running, self.clashes = mod, need, [], set(), []
        self.capture = None

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *shape: self.need

        def call(*args):
            n = 2 if name == "w4a16_gemm_ex" else 0
            ws, size, raw = args[len(args) - n - 3:len(args) - n]
            held = [t.data_ptr() for t in self.mod._workspaces.values()]
            if ws in self.running or ws not in held:
                self.clashes.append(name)
            self.running.add(ws)
            time.sleep(0.003)
            held = [t.data_ptr() for t in self.mod._workspaces.values()]
            if ws not in held:
                self.clashes.append(name + ": its workspace was replaced")
            self.running.discard(ws)
            self.calls.append((name, ws, size, raw))
            return 0
        return call


@pytest.fixture
def mod(monkeypatch):
    import w4a16_int4_weight_amd as m
    monkeypatch.setattr(m, "_lib", Library(m))
    monkeypatch.setattr(m, "_raw_stream", lambda stream, device: STREAM)
    monkeypatch.setattr(m, "_capture_of", lambda raw: m._lib.capture, raising=False)
    monkeypatch.setattr(m, "_captured", {}, raising=False)
    monkeypatch.setattr(m, "_recorded", {}, raising=False)
    monkeypatch.setattr(m, "_workspaces", {(None, STREAM): torch.zeros(4096, dtype=torch.uint8)})
    m._need.cache_clear()

    def grow(device, nbytes, stream=None):
        m._workspaces[(None, STREAM)] = torch.zeros(nbytes, dtype=torch.uint8)
        return m._workspaces[(None, STREAM)]
    monkeypatch.setattr(m, "_default_workspace", grow)
    yield m
    m._need.cache_clear()


def calls(m):
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    y = torch.zeros((4, 64), dtype=torch.bfloat16)
    ids = torch.zeros((4, 3), dtype=torch.int32)
    packed = torch.zeros(1 << 15, dtype=torch.uint8)
    return [lambda: m.w4a16_gemm_grad(y, packed, 256), lambda: m.w4a16_gated(x, packed, 64),
            lambda: m.w4a16_gated_grad(x, y, packed, 64),
            lambda: m.w4a16_cross_entropy(x, ids[:, 0].contiguous(), packed, 1000, grad=True),
            lambda: m.w4a16_distill(x, ids, ids.float(), packed, 1000, grad=True),
            lambda: m.w4a16_gemm(x, packed, 64), lambda: m.w4a16_gemm_ex(x, packed, 64, path="mfma"),
            lambda: m.w4a8_gemm(packed, packed, 4, 256, 64)]


def test_one_call_at_a_time_has_a_streams_workspace(mod):
    # several launches of a call meet in the workspace: another thread's must not come between
    def thread(first):
        ops = calls(mod)
        for i in range(16):
            if i == 8:
                mod._lib.need += 64          # the buffer grows while other threads call
                mod._need.cache_clear()
            ops[(first + i) % len(ops)]()
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(mod._lib.calls) == 64
    assert mod._lib.clashes == []


def test_a_refused_call_gives_the_workspace_back(mod):
    lib = mod._lib
    lib.w4a16_status_str = lambda code: b"refused"
    lib.w4a16_gated = lambda *args: 2
    ops = calls(mod)
    for _ in range(2):
        with pytest.raises(mod.W4A16Error):
            ops[1]()
    done = threading.Thread(target=ops[2], daemon=True)
    done.start()
    done.join(5)
    assert not done.is_alive() and lib.calls[-1][0] == "w4a16_gated_grad"


def test_a_callers_workspace_is_passed_on(mod):
    ws = torch.zeros(8192, dtype=torch.uint8)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    mod._workspaces[(None, 0)] = ws
    mod.w4a16_gated(x, torch.zeros(1 << 15, dtype=torch.uint8), 64, workspace=ws)
    assert mod._lib.calls[-1][1:] == (ws.data_ptr(), 8192, STREAM)


def test_a_capture_has_its_own_workspace(mod):
    lib, op = mod._lib, calls(mod)[3]
    op()
    eager = lib.calls[-1][1]
    lib.capture = 5
    op()
    first = lib.calls[-1][1]
    assert first != eager and bool((mod._captured[(None, STREAM)][1][:512] == 0).all())
    op()                                        # the calls of one capture share one
    assert lib.calls[-1][1] == first
    lib.need = 16384                            # ... which grows with them
    mod._need.cache_clear()
    op()
    assert lib.calls[-1][2] == 16384
    lib.capture = None                          # eager calls keep theirs, and grow it
    op()
    assert lib.calls[-1][1] not in (first, mod._captured[(None, STREAM)][1].data_ptr())
    assert lib.calls[-1][1] == mod._workspaces[(None, STREAM)].data_ptr()
    lib.capture = 6                             # another graph: cleared by that graph again
    kept = mod._captured[(None, STREAM)][1]
    kept.fill_(1)
    op()
    assert mod._captured[(None, STREAM)][1] is not kept
    assert bool((mod._captured[(None, STREAM)][1][:512] == 0).all())


@pytest.mark.parametrize("i", [5, 6, 7])
def test_captured_products_share_a_workspace_that_is_never_replaced(mod, i):
    lib, op = mod._lib, calls(mod)[i]
    lib.capture = 1                              # without a warm-up: the capture's own
    op()
    assert lib.calls[-1][1] == mod._captured[(None, STREAM)][1].data_ptr()
    lib.capture = None
    op()
    eager = lib.calls[-1][1]
    lib.capture = 2
    op()
    shared = lib.calls[-1][1]
    kept = mod._recorded[None][0]
    assert shared == kept.data_ptr() != eager and kept.numel() >= 4096 and int(kept.count_nonzero()) == 0
    calls(mod)[3]()                              # the other entries' calls have their own
    assert lib.calls[-1][1] not in (shared, eager)
    lib.capture = None                           # a larger need brings another; the first stays
    lib.need = 16384
    op()
    lib.capture = 3
    op()
    assert lib.calls[-1][1:3] == (mod._recorded[None][1].data_ptr(), 16384)
    assert mod._recorded[None][0] is kept
    lib.need = 4096
    lib.capture = None
    op()
    assert len(mod._recorded[None]) == 2
