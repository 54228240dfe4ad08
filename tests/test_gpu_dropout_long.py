"""Dropout of more elements than one dimension of a grid counts threads for."""
import pytest

from oracle import layers as ol

from .test_gpu_norm import tpc  # noqa: F401  (the module's fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_dropout_beyond_2_to_32_threads(tpc):
    """2^35 + 8,211 bfloat16 elements (64 GiB, in place): 2^32 threads and five workgroups more, the
    last one's last thread with three elements."""
    n = (1 << 35) + 8211
    print("dropout 2^35", flush=True)
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    out = tpc.dropout_forward(x, tpc.Dropout(0.5, 9, 1), out=x)
    torch.cuda.synchronize()
    for at in (0, (1 << 33) - 4, 1 << 33, 3 << 33, (1 << 35) - 4, 1 << 35, (1 << 35) + 8208):
        words = ol.philox_block(at // 4, 9, 1)[:min(4, n - at)]
        assert out[at:at + 4].float().cpu().tolist() == [2.0 if w >= 2 ** 31 else 0.0 for w in words], at
    # nothing left as it was: every element is 0 or 2
    for part in out.split(1 << 32):
        assert not (part == 1).any()
