"""What the layer's and the adapters' gradient calls refuse, without a GPU: the
kernels' calls are replaced by records of their arguments."""
import pytest
import torch

import fp8_blockwise_routed_b200 as fm
from fp8_blockwise_routed_b200 import adapters

T, E, H, I, K = 6, 8, 256, 128, 2


@pytest.fixture
def calls(monkeypatch):
    seen = []
    for name in ("moe_route_quant", "moe_quant_act_mx", "moe_route", "moe_grouped_ffn", "moe_grouped_ffn_mx",
                 "moe_combine", "moe_balance_loss", "moe_route_backward"):
        monkeypatch.setattr(fm, name, lambda *a, _n=name, **k: seen.append((_n, a)))
    for name in ("moe_permute", "moe_lora", "moe_lora_backward"):
        monkeypatch.setattr(adapters, name, lambda *a, _n=name, **k: seen.append((_n, a)))
    monkeypatch.setattr(fm, "moe_mx_pack_scales", lambda s: s)
    return seen


def _layer(cls):
    u8 = torch.uint8
    w = [torch.zeros(s, dtype=u8) for s in ((E, I, H), (E, I, H), (E, H, I))]
    s = [torch.zeros((E, 1, 1))] * 3
    return cls(w[0], s[0], w[1], s[1], w[2], s[2], K, 1.0, 16)


def _refused(call, *args, **kw):
    with pytest.raises(fm.MoeError) as e:
        call(*args, **kw)
    assert e.value.code == 1
    return str(e.value)


@pytest.mark.parametrize("cls", [fm.RoutedMoE, fm.RoutedMoEMX])
def test_gradient_of_another_batch_than_the_counts(calls, cls):
    layer = _layer(cls)
    x, z, dl = torch.zeros((T, H), dtype=torch.bfloat16), torch.zeros((T, E)), torch.ones((2,))
    dout = torch.zeros((T, H), dtype=torch.bfloat16)
    assert "forward comes first" in _refused(layer.router_backward, z, dout)
    assert "forward comes first" in _refused(layer.balance_loss, z)
    layer.forward(x, z, stream=0)
    layer.router_backward(z, dout)                         # through the weights alone: no counts needed
    assert "balance_loss comes first" in _refused(layer.router_backward, z, dout, dl)
    layer.balance_loss(z)
    layer.router_backward(z, dout, dl)
    layer.router_backward(z, None, dl)
    layer.forward(x, z, stream=0)
    assert "balance_loss comes first" in _refused(layer.router_backward, z, dout, dl)
    layer.balance_loss(z)
    layer.router_backward(z, dout, dl)
    assert "was of 6 tokens, not 5" in _refused(layer.router_backward, z[:5], dout[:5])
    assert "was of 6 tokens, not 5" in _refused(layer.balance_loss, z[:5])
    n = len(calls)
    layer._captured = True                                 # replays are not seen: nothing is refused
    layer.router_backward(z[:5], dout[:5], dl)
    assert len(calls) == n + 1


def test_adapter_gradient_of_another_batch(calls):
    a, b = torch.zeros((2, 4, 16), dtype=torch.bfloat16), torch.zeros((2, 4, 8), dtype=torch.bfloat16)
    ad, batch = adapters.LoraAdapters(a, b, None, 16), adapters.LoraBatch(2, 16, device="cpu")
    ids = torch.zeros((T,), dtype=torch.int32)
    x, dout = torch.zeros((T, 16), dtype=torch.bfloat16), torch.zeros((T, 8), dtype=torch.bfloat16)
    assert not ad.v.any()                                  # a gradient before any forward is of zero rows
    ad.backward(batch.assign(ids), x, dout)
    ad.forward(batch, x, None, torch.zeros((T, 8)))
    ad.backward(batch, x, dout)
    batch.assign(ids[:4])
    assert "was of 6 tokens, not 4" in _refused(ad.backward, batch, x[:4], dout[:4])
    ad.forward(batch, x[:4], None, torch.zeros((4, 8)))
    ad.backward(batch, x[:4], dout[:4])
    assert [c[0] for c in calls].count("moe_lora_backward") == 3


def test_gradients_of_micro_batches_are_kept(calls):
    """Buffers given by the caller take the gradients; the object's own are
    made only where they are used, and are the same ones every time."""
    a, b = torch.zeros((2, 4, 16), dtype=torch.bfloat16), torch.zeros((2, 4, 8), dtype=torch.bfloat16)
    ad, batch = adapters.LoraAdapters(a, b, None, 16), adapters.LoraBatch(2, 16, device="cpu")
    x, dout = torch.zeros((T, 16), dtype=torch.bfloat16), torch.zeros((T, 8), dtype=torch.bfloat16)
    ad.forward(batch.assign(torch.zeros((T,), dtype=torch.int32)), x, None, torch.zeros((T, 8)))
    mine = [(torch.zeros(a.shape), torch.zeros(b.shape)) for _ in range(2)]
    for d_a, d_b in mine:
        got = ad.backward(batch, x, dout, d_a=d_a, d_b=d_b)
        assert got[0] is d_a and got[1] is d_b
        assert calls[-1][0] == "moe_lora_backward" and calls[-1][1][10] is d_a and calls[-1][1][11] is d_b
    assert ad._grad is None
    one = ad.backward(batch, x, dout)
    assert one[0].shape == a.shape and one[1].shape == b.shape and one[0].dtype == torch.float32
    two = ad.backward(batch, x, dout, d_b=mine[0][1])
    assert two[0] is one[0] and two[1] is mine[0][1]


def test_batch_on_another_device_than_the_current_one(monkeypatch):
    """assign groups on the device of the ids: its kernels are launched with
    that device (and so its current stream) current."""
    current = [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, current[0] = current[0], self.index

        def __exit__(self, *exc):
            current[0] = self.before

    class Ids:                                             # a tensor on the second device
        shape, dtype, device, is_cuda = (T,), torch.int32, "cuda:1", True

        def is_contiguous(self):
            return True

        def get_device(self):
            return 1

        def view(self, *shape):
            return self

    seen = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(adapters, "moe_permute", lambda *a: seen.append(current[0]))
    batch = adapters.LoraBatch(2, 16, device="cpu")

    class Offsets:
        device = "cuda:1"

    batch.offsets = Offsets()
    batch.assign(Ids())
    assert seen == [1] and current == [0]
    current[0] = 1
    batch.assign(Ids())
    assert seen == [1, 1] and current == [1]


def test_missing_and_misshapen_tensors_are_named():
    z = torch.zeros
    lg, off, cnt = z((4, 8)), z(9, dtype=torch.int32), z(9, dtype=torch.int32)
    x, a = z((4, 16), dtype=torch.bfloat16), z((1, 2, 16), dtype=torch.bfloat16)
    o1, tok = z(2, dtype=torch.int32), z(4, dtype=torch.int32)
    loss = fm.moe_balance_loss
    assert "logits is missing" in _refused(loss, None, off, z(2), cnt, z(8), z(64, dtype=torch.uint8))
    assert "logits: expected 2 dimensions" in _refused(loss, z(8), off, z(2), cnt, z(8), z(64, dtype=torch.uint8))
    grad = fm.moe_route_backward
    assert "logits is missing" in _refused(grad, None, None, None, None, None, 1.0, cnt, z(2), lg)
    assert "logits: expected 2 dimensions" in _refused(grad, z(8), None, None, None, None, 1.0, cnt, z(2), lg)
    lora = fm.moe_lora
    assert "x is missing" in _refused(lora, None, a, a, None, o1, tok, None, z((4, 2)), z((4, 16)))
    assert "x: expected 2 dimensions" in _refused(lora, x[0], a, a, None, o1, tok, None, z((4, 2)), z((4, 16)))
    assert "lora_b is missing" in _refused(lora, x, a, None, None, o1, tok, None, z((4, 2)), z((4, 16)))
    back = fm.moe_lora_backward
    assert "lora_b: expected 3 dimensions" in _refused(back, x, a, a[0], None, o1, tok, z((4, 2)), x, None, None, a, a, tok)
    assert "x is missing" in _refused(back, None, a, a, None, o1, tok, z((4, 2)), x, None, None, a, a, tok)
    assert "ws is missing" in _refused(fm._bytes, "moe_balance_loss", None, 0)
