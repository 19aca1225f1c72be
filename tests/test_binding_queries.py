"""The binding's queries of torch's current device and stream, with and without the private entry points."""
import types

import mixed_precision_expert_b200 as mpe


def fake(private):
    C = types.SimpleNamespace(**({"_cuda_getDevice": lambda: 3, "_cuda_getCurrentRawStream": lambda d: 100 + d}
                                 if private else {}))
    cuda = types.SimpleNamespace(current_device=lambda: 5,
                                 current_stream=lambda d: types.SimpleNamespace(cuda_stream=200 + d))
    return types.SimpleNamespace(_C=C, cuda=cuda)


def test_private_entry_points():
    device, stream = mpe._queries(fake(True))
    assert device() == 3 and stream(1) == 101


def test_public_ones_where_a_torch_lacks_them():
    device, stream = mpe._queries(fake(False))
    assert device() == 5 and stream(1) == 201
