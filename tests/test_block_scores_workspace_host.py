"""The workspace of block scores, as the binding takes it: its bytes have to be the tensor's own. Tensors are stood in
for, so that nothing is launched."""
import pytest
import torch

from dit_transformer_block_gb300 import h3


class Stub:
    """What the binding reads of a CUDA tensor."""

    def __init__(self, shape, dtype, contiguous=True, device=0):
        self.shape, self.dtype, self.contiguous, self.dev = torch.Size(shape), dtype, contiguous, device
        self.device = f"cuda:{device}"

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.contiguous

    def stride(self):
        return torch.empty(self.shape, device="meta").stride()

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.element_size()


@pytest.fixture
def calls(monkeypatch):
    made = []

    class Lib:
        @staticmethod
        def h3_block_scores(*a):
            made.append(a)
            return 0

    monkeypatch.setattr(h3, "_lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    return made


def score(workspace):
    q, k = Stub((300, 4, 128), torch.bfloat16), Stub((200, 2, 128), torch.bfloat16)
    h3.block_scores(q, k, Stub((4, 2, 4), torch.float32), workspace, k_block=64)


def test_bytes_of_the_tensor(calls):
    score(Stub((8192,), torch.uint8))
    score(Stub((32, 64), torch.float32))
    assert [a[-2] for a in calls] == [8192, 8192]


def test_strided_and_expanded_ones_are_refused(calls):
    # a view of every second byte, or one byte expanded to many, has fewer bytes in a row than elements
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        score(Stub((8192,), torch.uint8, contiguous=False))
    assert not calls


def test_another_device_is_refused(calls):
    with pytest.raises(ValueError, match="workspace must be on the current CUDA device"):
        score(Stub((8192,), torch.uint8, device=1))
    assert not calls
