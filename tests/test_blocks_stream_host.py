"""A stream of another device than the tensors' is refused before anything is launched on it."""
import pytest

import selective_state_space_79_amd as ssm


class Stream:
    cuda_stream, device_index = 0x1234, 1


@pytest.mark.parametrize("name,count", [("ssm_linattn_fwd", 9), ("ssm_linattn_step", 7), ("ssm_gated_norm_fwd", 4)])
def test_stream_of_another_device(name, count, monkeypatch):
    calls = []
    monkeypatch.setitem(ssm.blocks._bound, name, lambda *a: calls.append(a) or 0)
    with pytest.raises(ValueError, match="stream"):
        ssm.blocks._call(name, (None,) * count, 0, Stream())
    assert not calls
