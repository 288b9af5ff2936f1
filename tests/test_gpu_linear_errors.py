"""Failing calls of the linear attention and the norm: what they leave behind."""
import ctypes

import pytest
import torch

from gated_delta_rule_108_b200 import kda

pytestmark = pytest.mark.gpu


class _Capturing:
    """A capture in progress on a stream that the default stream waits for: until it ends, work
    on the default stream is refused on the host (and ends the capture; nothing of it runs)."""

    def __enter__(self):
        self.cu, self.stream = ctypes.CDLL("libcuda.so.1"), ctypes.c_void_p()
        assert self.cu.cuStreamCreate(ctypes.byref(self.stream), 0) == 0
        assert self.cu.cuStreamBeginCapture_v2(self.stream, 2) == 0     # relaxed
        return self.stream.value

    def __exit__(self, *_):
        graph = ctypes.c_void_p()
        self.cu.cuStreamEndCapture(self.stream, ctypes.byref(graph))    # reports that the capture was ended
        assert not graph.value
        assert self.cu.cuStreamDestroy_v2(self.stream) == 0


def _layer(dtype=torch.bfloat16, B=2, T=100, H=2, d=128):
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = {n: r(B, T, H, d).to(dtype) for n in "qkv"}
    out = dict(o=torch.empty_like(x["v"]), final_state=torch.empty(B, H, d, d, device="cuda"))
    return x, out, -torch.rand(H, generator=g, device="cuda")


@pytest.mark.parametrize("failing", ["launch", "status"])
@pytest.mark.parametrize("after", ["step", "norm", "norm gradients", "packed", "kda step"])
def test_a_failed_call_does_not_fail_the_next(cuda_device, failing, after):
    """The next call on the thread does its work once and says so."""
    x, out, l = _layer()
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    kda.linear_chunk_fwd(**x, log_decay=l, **out, workspace=ws)
    S = out["final_state"].clone()
    one = {n: t[:, 0].contiguous() for n, t in x.items()}
    cu = torch.tensor([0, 30, 100], dtype=torch.int32, device="cuda")
    w = torch.ones(128, device="cuda")
    beta, la = torch.rand(2, 2, device="cuda"), -torch.rand(2, 2, 128, device="cuda")

    def call():
        if after == "step":
            s = S.clone()
            return kda.linear_recurrent_step(one["q"], one["k"], one["v"], l, s), s
        if after == "norm":
            return kda.qk_norm_rope(x["q"], x["k"], w, w)
        if after == "norm gradients":
            return tuple(kda.qk_norm_rope_bwd(x["q"], x["k"], x["q"], x["k"], w, w).values())
        if after == "packed":
            return kda.linear_chunk_fwd(*(x[n][:1] for n in "qkv"), l, cu_seqlens=cu, check=False)
        s = S.clone()
        return kda.recurrent_step(one["q"], one["k"], one["v"], la, beta, s), s

    expected = call()
    torch.cuda.synchronize()
    with _Capturing() as capturing:
        if failing == "launch":
            with pytest.raises(kda.KDAError, match="launch failed"):
                kda.linear_chunk_fwd(**x, log_decay=l, **out, workspace=ws)
        else:       # waiting for a stream that captures is refused
            assert kda.lib().kda_workspace_status(ws.data_ptr(), ws.nbytes, capturing) != 0
    got = call()
    assert len(got) == len(expected) and all(torch.equal(a, b) for a, b in zip(got, expected))


def test_a_chain_of_segments_gives_up_once(cuda_device):
    """Segments that follow one another: the ones behind a wait that has run out do not wait for themselves."""
    cap = 40_000_000      # cycles, some 20 ms
    took = {}
    for name, (B, T, H, segments) in dict(one=(1, 100, 2, 1), chain=(5, 16384, 32, 8)).items():
        x, out, l = _layer(B=B, T=T, H=H, d=64)
        ws = torch.empty(kda.linear_chunk_fwd_workspace_size(B, T, H, 64, 64, B, False, torch.bfloat16), dtype=torch.uint8,
                         device="cuda")
        assert segments == 1 or ws.nbytes >= segments * B * H * 64 * 64 * 4
        kda.linear_chunk_fwd(**x, log_decay=l, **out, workspace=ws)
        good = out["o"].clone()
        assert kda.workspace_status(ws) == 0
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        kda.linear_debug_drop_copy(cap)
        start.record()
        kda.linear_chunk_fwd(**x, log_decay=l, **out, workspace=ws)
        end.record()
        assert kda.workspace_status(ws) == 4      # KDA_ERR_TIMEOUT
        took[name] = start.elapsed_time(end)
        kda.linear_chunk_fwd(**x, log_decay=l, **out, workspace=ws, check=True)
        assert torch.equal(out["o"], good)
    # 160 first segments on 148 SMs run out of time in two turns; 8 x 160 segments would in nine
    assert took["one"] > 10 and took["chain"] < 3.5 * took["one"], took
