"""The training operators' C ABI without a GPU: every function the header
declares is exported and bound, and bad arguments are refused before any work
is enqueued."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_training.h")

m = pytest.importorskip("moe_token_routing_amd")

V = ctypes.c_void_p
FAKE = V(1 << 20)        # a non-NULL, 256-byte aligned address that is never dereferenced
ODD = V((1 << 20) + 4)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m.LIB_PATH):
        pytest.fail("libmoe_routing.so is not built (run __graft_entry__.build())")
    return m.lib()


def test_every_declared_function_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert names == set(m._TRAINING_SIGNATURES)
    for n in names:
        assert hasattr(lib, n), n


def test_balance_loss_rejects_before_launch(lib):
    def call(logits=FAKE, ids=FAKE, mask=FAKE, off=FAKE, score=0, T=4, E=16, k=2, S=3, losses=FAKE, counts=FAKE,
             probs=FAKE, tokens=FAKE, ws=FAKE, wsb=BIG):
        return lib.moe_balance_loss(logits, ids, mask, off, score, T, E, k, S, losses, counts, probs, tokens, ws, wsb,
                                    None)

    assert call(T=-1) == -2 and call(E=0) == -2 and call(E=4097) == -2 and call(T=(1 << 30) + 1) == -2
    assert call(k=0) == -2 and call(k=17) == -2 and call(k=33, E=64) == -2
    assert call(S=0) == -2 and call(S=65537) == -2
    assert call(T=1 << 30, k=2) == -2                     # counts are int32
    assert call(off=None) == -1                           # S sequences need offsets
    assert call(score=2) == -5 and call(score=-1) == -5
    for name in ("logits", "ids", "mask", "losses", "counts", "probs", "tokens"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -7, name
    need = m.balance_loss_workspace_bytes(400, 16, 3)
    assert need % 256 == 0 and need >= 2 * 4 * 16 * 4
    assert call(T=400, ws=None) == -4 and call(T=400, wsb=need - 1) == -4
    assert call(T=400, ws=V((1 << 20) + 8)) == -4
    assert m.balance_loss_workspace_bytes(4, 16, 3) == 0          # one block, no workspace
    assert m.balance_loss_workspace_bytes(4, 16, 64) > 0 and m.balance_loss_workspace_bytes(4, 4096, 1) > 0
    assert m.balance_loss_workspace_bytes(4, 0, 3) == 0 and m.balance_loss_workspace_bytes(-1, 4, 3) == 0


def test_balance_loss_backward_rejects_before_launch(lib):
    def call(dl=FAKE, logits=FAKE, mask=FAKE, off=None, counts=FAKE, tokens=FAKE, score=0, T=4, E=16, k=2, S=1, acc=0,
             d=FAKE):
        return lib.moe_balance_loss_backward(dl, logits, mask, off, counts, tokens, score, T, E, k, S, acc, d, None)

    assert call(T=-1) == -2 and call(E=4097) == -2 and call(k=0) == -2 and call(k=17) == -2 and call(S=0) == -2
    assert call(S=2) == -1 and call(score=3) == -5
    for name in ("dl", "logits", "mask", "counts", "tokens", "d"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -7, name
    assert call(T=0, logits=None, mask=None, d=None) == 0   # nothing to write


def test_distill_loss_rejects_before_launch(lib):
    def call(logits=FAKE, ids=FAKE, z=FAKE, mask=FAKE, score=0, temp=1.0, T=4, E=16, K=2, loss=FAKE, each=FAKE,
             tokens=FAKE, ws=FAKE, wsb=BIG):
        return lib.moe_distill_loss(logits, ids, z, mask, score, temp, T, E, K, loss, each, tokens, ws, wsb, None)

    assert call(T=-1) == -2 and call(E=0) == -2 and call(E=4097) == -2 and call(K=0) == -2 and call(K=33) == -2
    for temp in (0.0, -1.0, 1e-7, 1e7, float("inf"), float("nan")):
        assert call(temp=temp) == -5
    assert call(score=2) == -5
    for name in ("logits", "ids", "z", "mask", "loss", "each", "tokens"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -7, name
    need = m.distill_loss_workspace_bytes(400, 16)
    assert call(T=400, ws=None) == -4 and call(T=400, wsb=need - 1) == -4
    assert m.distill_loss_workspace_bytes(4, 16) == 0 and m.distill_loss_workspace_bytes(4, 4096) > 0
    assert m.distill_loss_workspace_bytes(4, 4097) == 0


def test_distill_loss_backward_rejects_before_launch(lib):
    def call(dl=FAKE, logits=FAKE, ids=FAKE, z=FAKE, mask=FAKE, tokens=FAKE, score=0, temp=1.0, T=4, E=16, K=2, acc=0,
             d=FAKE):
        return lib.moe_distill_loss_backward(dl, logits, ids, z, mask, tokens, score, temp, T, E, K, acc, d, None)

    assert call(T=-1) == -2 and call(E=4097) == -2 and call(K=33) == -2 and call(temp=0.0) == -5
    assert call(score=-1) == -5
    for name in ("dl", "logits", "ids", "z", "mask", "tokens", "d"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -7, name
    assert call(T=0, logits=None, ids=None, z=None, mask=None, d=None) == 0


def test_route_backward_rejects_before_launch(lib):
    def call(dw=FAKE, aux=FAKE, hidden=FAKE, dtype=1, W=FAKE, logits=FAKE, ids=FAKE, w=FAKE, mask=FAKE, scale=1.0,
             T=4, H=64, E=16, k=2, dl=FAKE, dh=FAKE, dW=FAKE, ws=FAKE, wsb=BIG):
        return lib.moe_route_backward(dw, aux, hidden, dtype, W, logits, ids, w, mask, scale, T, H, E, k, dl, dh, dW,
                                      ws, wsb, None)

    assert call(T=-1) == -2 and call(H=24) == -2 and call(H=0) == -2 and call(H=16400) == -2
    assert call(E=0) == -2 and call(E=4097) == -2 and call(k=0) == -2 and call(k=17) == -2 and call(k=33, E=64) == -2
    assert call(dtype=2) == -3 and call(scale=float("nan")) == -5
    assert call(dw=None, aux=None) == -1
    for name in ("logits", "ids", "w", "mask", "W", "dl"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -7, name
    for name in ("dw", "aux", "hidden", "dh", "dW"):
        assert call(**{name: ODD}) == -7, name
    assert call(hidden=None) == -1                        # no input, yet its gradients are wanted
    need = m.route_backward_workspace_bytes(400, 64, 16, m.MOE_DTYPE_BF16)
    assert need % 256 == 0 and need > 0
    assert call(T=400, ws=None) == -4 and call(T=400, wsb=need - 1) == -4
    assert call(T=400, ws=V((1 << 20) + 16)) == -4
    assert m.route_backward_workspace_bytes(400, 64, 16, m.MOE_DTYPE_F32) > need
    assert m.route_backward_workspace_bytes(400, 64, 16, m.MOE_DTYPE_BF16, logits_in=True) == 0
    assert m.route_backward_workspace_bytes(4, 64, 16, m.MOE_DTYPE_BF16) == 0     # few tokens: no workspace
    assert m.route_backward_workspace_bytes(32, 64, 4096, m.MOE_DTYPE_BF16) > 0   # too many experts for that
    assert m.route_backward_workspace_bytes(4, 24, 16, m.MOE_DTYPE_BF16) == 0
    assert call(T=0, dW=None, ws=None) == 0


def test_combine_backward_rejects_before_launch(lib):
    def call(y=FAKE, x=FAKE, R=8, slots=FAKE, w=FAKE, nw=FAKE, gc=0.0, eps=1e-6, T=4, H=64, k=2, dx=FAKE, dw=FAKE,
             dn=FAKE, ws=FAKE, wsb=BIG):
        return lib.moe_combine_backward(y, x, R, slots, w, nw, gc, eps, T, H, k, dx, dw, dn, ws, wsb, None)

    assert call(H=63) == -2 and call(H=0) == -2 and call(H=16392) == -2 and call(k=0) == -2 and call(k=33) == -2
    assert call(T=-1) == -2 and call(R=-1) == -2 and call(T=1 << 30, k=2) == -2
    assert call(eps=-1.0) == -5 and call(eps=float("nan")) == -5 and call(gc=float("inf")) == -5
    for name in ("y", "x", "slots", "w", "nw", "dx", "dw"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: ODD}) == -7, name
    assert call(dn=ODD) == -7
    need = m.combine_backward_workspace_bytes(4, 8, 64)
    assert need % 256 == 0 and need > 0
    assert call(ws=None) == -4 and call(wsb=need - 1) == -4
    assert m.combine_backward_workspace_bytes(4, 8, 63) == 0


def test_binding_makes_the_tensors_device_current(monkeypatch):
    """The library launches on the current device: with another one current the
    call runs inside torch.cuda.device(dev), and its stream is looked up there."""
    import torch
    from moe_token_routing_amd import training as tr
    now, log = [0], []

    class Device:
        def __init__(self, dev):
            self.dev = dev

        def __enter__(self):
            self.was, now[0] = now[0], self.dev.index

        def __exit__(self, *_):
            now[0] = self.was

    class Lib:
        def moe_something(self, *args):
            log.append((now[0], args))
            return 0

    monkeypatch.setattr(tr, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(tr, "_stream", lambda dev: "stream of %d" % dev.index)
    monkeypatch.setattr(tr, "lib", Lib)
    tr._call("moe_something", torch.device("cuda", 0), 1, 2)
    tr._call("moe_something", torch.device("cuda", 3), 4)
    assert log == [(0, (1, 2, "stream of 0")), (3, (4, "stream of 3"))] and now[0] == 0


def test_binding_refuses_cpu_tensors():
    import torch
    l, ids, mask = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        m.balance_loss(l, ids, mask)
    with pytest.raises(ValueError):
        m.distill_loss(l, ids, torch.zeros(4, 2), mask)
    with pytest.raises(ValueError):
        m.route_backward(None, None, None, None, None, None, mask)
    with pytest.raises(ValueError):
        m.combine_backward(torch.zeros(4, 8).bfloat16(), torch.zeros(8, 8).bfloat16(), ids, torch.zeros(4, 2),
                           torch.zeros(8), 0.0, 1e-6)
