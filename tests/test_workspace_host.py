"""Workspaces handed to the binding, without a GPU: the entry points get the
address and numel() bytes of the tensor, so one whose bytes do not lie together
(strided, expanded) has to be refused before the call."""
import pytest
import torch

from linear_attention_recurrence_04_b200 import gdn

BYTES = 4096
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


class FakeLibrary:
    """Takes every call as done and keeps the arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_workspace_size"):
                return BYTES
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    """The binding with host tensors let through to a fake library."""
    fake = FakeLibrary()
    monkeypatch.setattr(gdn, "load_library", lambda path=None: fake)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(gdn, "_check", lambda *a: None)
    monkeypatch.setattr(gdn, "_enter", lambda dev, stream: (0, None))
    monkeypatch.setattr(gdn, "_call", lambda device, fn, *args: fn(*args))
    monkeypatch.setattr(gdn, "_stream", lambda device, stream: 0)
    return fake


B, T, D, Hk, Hv, K = 1, 2, 64, 1, 1, 4
C = 2 * Hk * 128 + Hv * 128


def layer(w):
    z = torch.zeros
    return ([z(C, D, dtype=w), z(Hv * 128, D, dtype=w), z(2 * Hv, D, dtype=w), z(D, Hv * 128, dtype=w)],
            [z(B, K - 1, C), z(C, K), z(Hv), z(Hv), z(128), z(B, Hv, 128, 128)])


def forward_batch(ws):
    w, rest = layer(BF)
    gdn.forward_batch(torch.zeros(B, T, D, dtype=BF), *w, *rest, workspace=ws, Hk=Hk)


def forward_batch_i8(ws):
    w, rest = layer(I8)
    scales = [torch.zeros(t.shape[0]) for t in w]
    pairs = [t for both in zip(w, scales) for t in both]
    gdn.forward_batch_i8(torch.zeros(B, T, D, dtype=I8), torch.zeros(B, T), *pairs, *rest,
                         workspace=ws, Hk=Hk)


def short_conv(fn, hidden, *rings):
    def call(ws):
        fn(torch.zeros(*hidden, dtype=BF), torch.zeros(3 * D, D, dtype=BF),
           torch.zeros(D, D, dtype=BF), *(torch.zeros(B, K - 1, D) for _ in rings),
           torch.zeros(D, K), workspace=ws)
    return call


CALLS = {"forward_batch": forward_batch, "forward_batch_i8": forward_batch_i8,
         "short_conv_forward_batch": short_conv(gdn.short_conv_forward_batch, (B, T, D), 0),
         "short_conv_forward": short_conv(gdn.short_conv_forward, (B, D), 0),
         "short_conv_pair": short_conv(gdn.short_conv_pair, (B, 2, D), 0, 1)}


@pytest.mark.parametrize("name", CALLS)
def test_workspace(lib, name):
    call = CALLS[name]
    whole = torch.zeros(2 * BYTES, dtype=torch.uint8)
    for ws in (None, whole[:BYTES], whole[BYTES:], whole.view(2, -1)):
        call(ws)
    assert [n for n, _ in lib.calls] == ["gdn_" + name] * 4
    del lib.calls[:]
    for ws in (whole[::2], torch.zeros(1, dtype=torch.uint8).expand(BYTES),
               whole.view(64, -1).t(), whole.view(64, -1)[:, :64]):
        assert ws.numel() >= BYTES
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call(ws)
    for ws in (torch.zeros(BYTES, dtype=I8), torch.zeros(BYTES, dtype=torch.uint8, device="meta")):
        with pytest.raises(TypeError):
            call(ws)
    assert lib.calls == []
