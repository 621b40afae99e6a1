"""What the paged wrappers refuse or arrange before the library is called (CPU)."""
import pytest
import torch

from relation_token_mixing_gb300 import binding as rb


def _i32(*s):
    return torch.zeros(*s, dtype=torch.int32)


def _bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


@pytest.mark.parametrize("theta", [torch.zeros(2, dtype=torch.float64), torch.zeros(2, dtype=torch.bfloat16),
                                   torch.zeros(1), torch.zeros(3), torch.zeros(0)])
def test_store_refuses_a_theta_that_is_not_float32_of_half_the_cache_heads(theta):
    with pytest.raises(ValueError, match="theta"):
        rb.paged_store(_bf(3, 8, 64), _bf(3, 4, 64), _bf(3, 4, 64), theta, 0, 1e4, _i32(3), _i32(3).long(),
                       _bf(3, 8, 64), _bf(8, 4, 16, 64), _bf(8, 4, 16, 64))


@pytest.mark.parametrize("given", [False, True])
def test_forward_allocates_from_the_stream_it_runs_on(given, monkeypatch):
    """The workspace is freed when the call returns: allocated from another stream, its memory could be handed to that
    stream's next work while the kernels still use it.  Y is marked as used by the caller's stream."""
    entered, seen, recorded = [], {}, []

    class Entered:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            entered.append(self.stream)

        def __exit__(self, *exc):
            entered.pop()

    empty_like = torch.empty_like

    def noted(name, make):
        seen[name] = entered[-1] if entered else None
        return make()

    monkeypatch.setattr(torch.cuda, "stream", Entered)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "caller's")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: recorded.append(s))
    monkeypatch.setattr(torch, "empty_like", lambda x: noted("Y", lambda: empty_like(x)))
    monkeypatch.setattr(rb, "paged_workspace", lambda *a: noted("workspace", lambda: torch.empty(16)))
    monkeypatch.setattr(rb, "relation_paged_fwd", lambda *a: seen.update(ran=a[-1]))
    stream = "side" if given else None
    rb.paged_fwd(_bf(3, 4, 64), _bf(8, 2, 16, 64), _bf(8, 2, 16, 64), _i32(1, 4), _i32(2), _i32(1), 0, 1.0, 0.5,
                 stream=stream)
    assert seen == {"Y": stream, "workspace": stream, "ran": stream}
    assert recorded == (["caller's"] if given else [])
