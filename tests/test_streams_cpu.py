"""Which stream a call's own tensors are made on (CPU: torch's streams are replaced by records)."""
import torch

from head_latent_attention_04_b200 import mla


class FakeStream:
    def __init__(self, handle, device=None):
        self.cuda_stream, self.device = handle, device


def test_a_raw_handle_belongs_to_the_tensors_device(monkeypatch):
    """A handle alone does not say its device: taken for the current one's, the tensors of a call on another
    device would be made on that device's current stream, not on the call's."""
    seen = []
    monkeypatch.setattr(torch.cuda, "ExternalStream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: seen.append(s) or mla._SAME_DEVICE)
    mla._made_on(0x1234, torch.device("cuda", 1))
    assert seen[0].cuda_stream == 0x1234 and seen[0].device == torch.device("cuda", 1)
    own = FakeStream(7, torch.device("cuda", 2))
    mla._made_on(own, torch.device("cuda", 1))
    assert seen[1] is own
    assert mla._made_on(None, torch.device("cuda", 1)) is mla._SAME_DEVICE and len(seen) == 2
