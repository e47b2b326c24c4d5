"""The native check of a tensor argument answers as the questions asked in Python do, and only for tensors that pass."""
import pytest
import torch

from fp8_block_scaled_amd import _args, serving

F32 = (torch.float32,)


def test_anything_else_is_left_to_python():
    t = torch.zeros(2, 3)
    for args in ((t, F32, (2, 3), -1), (t, F32, (2, 3), 0), (None, F32, (2, 3), 0), ([1], F32, (1,), 0), (t.to("meta"), F32, (2, 3), 0),
                 (t, F32, [2, 3], 0), (t, F32, (2, 3), None), (t, F32, (2, 1 << 70), 0), (t, F32, (2, "3"), 0), (t, F32, (2,), 0)):
        assert _args.address(*args) is None
    with pytest.raises(TypeError):
        _args.address(t, F32, (2, 3))
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        serving._ptr(None, "x", F32, (2, 3), torch.device("cuda", 0))
    with pytest.raises(ValueError, match="is on cpu"):
        serving._ptr(t, "x", F32, (2, 3), torch.device("cuda", 0))


@pytest.mark.gpu
def test_answers_as_python_does(monkeypatch):
    device = torch.device("cuda", 0)
    t = torch.zeros(6, 8, device=device)
    cases = [(t, F32, (6, 8)), (t, F32, t.shape), (t, {torch.float32: 1}, (6, 8)), (t, (torch.int32,), (6, 8)), (t, F32, (8, 6)), (t, F32, (48,)),
             (t[:, :4], F32, (6, 4)), (t.t(), F32, (8, 6)), (t[2:], F32, (4, 8)), (t[:1, :3], F32, (1, 3)), (t[:0], F32, (0, 8)),
             (t[0, 0], F32, ()), (torch.nn.Parameter(t), F32, (6, 8)), (t.cpu(), F32, (6, 8)), (t.to(torch.float8_e4m3fn), serving._F8, (6, 8))]

    def answers():
        out = []
        for c in cases:
            try:
                out.append(serving._ptr(*c[:1], "x", *c[1:], device))
            except (TypeError, ValueError) as e:
                out.append((type(e), str(e)))
        return out

    native = answers()
    assert _args.address(t, F32, (6, 8), 0) == t.data_ptr() and _args.address(t, F32, (6, 8), 1) is None
    monkeypatch.setattr(serving, "_address", lambda *a: None)
    assert native == answers()
