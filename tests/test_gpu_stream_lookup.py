"""The current stream without torch's private lookup of it, should a version lack that
(the other one, of the current device, is what torch.cuda.current_device calls)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import activation_sparse_gemm_token_amd as rtl  # noqa: E402
from activation_sparse_gemm_token_amd import rotary, training, w4  # noqa: E402

DEV = "cuda:0"


def test_the_public_lookup_gives_the_same_stream(monkeypatch):
    q, pos, f = torch.randn(8, 2, 32, device=DEV).bfloat16(), torch.arange(8, device=DEV), rotary.frequencies(32).to(DEV)
    weight = w4.pack(torch.zeros(16, 32, dtype=torch.uint8, device=DEV), torch.ones(16, 2, device=DEV).bfloat16(), group=32)
    x = torch.randn(4, 64, device=DEV).bfloat16()
    run = lambda: (rotary.rope(q, pos, f), w4.linear(x, weight), training.checkpoint(x).unpack(), rtl.dense_linear(x, x))  # noqa: E731
    want, stream = run(), torch.cuda.Stream()
    torch.cuda.synchronize()
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream")
    for s in (torch.cuda.default_stream(), stream):
        with torch.cuda.stream(s):
            assert rtl._stream() == s.cuda_stream and rtl._here(q) in (None, s.cuda_stream)
            got = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
