"""Guard canaries for the convolution, the scan and the 4-bit products: what a call writes lies between bands that stay as they were."""
import pytest
import torch

from layer_helpers import BF, F32
from test_gpu_guards import Guarded
from test_gpu_ssm_scan import cu_of, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    from gated_deltanet_linear_03_gb300 import gdn, linear, ssm
    gdn.load_library()
    return gdn, linear, ssm


@pytest.mark.parametrize("width", [2, 4])
@pytest.mark.parametrize("lens", [[1, 1, 1], [5, 0, 33, 1, 0], [3000, 1, 0, 2500, 7]])
@pytest.mark.parametrize("channels", [8, 1016])
def test_convolution(pkg, lens, width, channels):
    gdn, _, ssm = pkg
    x, w = torch.randn(sum(lens), channels, device="cuda").to(BF), torch.randn(channels, width, device="cuda")
    past = torch.randn(len(lens), width - 1, channels, device="cuda").to(BF)
    for cu in ([cu_of(lens)] + ([None] if max(lens) == 1 else [])):
        out, state = Guarded(tuple(x.shape), BF), Guarded(tuple(past.shape), BF)
        ssm.short_conv(x, w, cu, state_in=past, state_out=state.tensor, out=out.tensor)
        torch.cuda.synchronize()
        assert out.intact() and state.intact() and gdn.device_error() == 0


@pytest.mark.parametrize("n_state", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [[1, 1, 1], [41, 0, 3], [1801, 1, 0, 700]])
@pytest.mark.parametrize("channels,groups", [(8, 1), (120, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scan(pkg, lens, n_state, channels, groups, dtype):
    gdn, _, ssm = pkg
    i = inputs(lens, channels, n_state, groups)
    for cu in ([cu_of(lens)] + ([None] if max(lens) == 1 else [])):
        out, state = Guarded((sum(lens), channels), dtype), Guarded(tuple(i["past"].shape), F32)
        need = ssm.scan_workspace_size(len(lens), sum(lens), channels, n_state, groups, max(lens)) if cu is not None else 0
        ws = Guarded((max(need, 1),), torch.uint8)
        ssm.scan(i["x"], i["dt"], i["a"], i["b"], i["c"], cu, d=i["d"], z=i["z"], dt_bias=i["bias"], state_in=i["past"], state_out=state.tensor,
                 max_len=max(lens), out=out.tensor, workspace=ws.tensor if need else None)
        torch.cuda.synchronize()
        assert out.intact() and state.intact() and ws.intact() and gdn.device_error() == 0


@pytest.mark.parametrize("group,offsets", [(64, True), (128, False), (128, True)])
@pytest.mark.parametrize("rows,n_out,k", [(1, 7, 128), (2, 1001, 2048), (3, 17, 640), (12, 333, 4096), (16, 4101, 8192), (24, 45, 1152), (33, 4099, 4096),
                                          (61, 129, 384), (130, 259, 2176), (509, 1201, 1920), (70, 20001, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_products(pkg, rows, n_out, k, group, offsets, dtype):
    gdn, linear, _ = pkg
    w = linear.quantize(torch.randn(n_out, k, device="cuda"), group, offsets)
    x = torch.randn(rows, k, device="cuda").to(BF)
    need = linear.workspace_size(rows, n_out, k, group, dtype)
    for call in (lambda **kw: linear.q4_linear(x, w, **kw), lambda **kw: linear.q4_gated(x, w, w, **kw)):
        out, ws = Guarded((rows, n_out), dtype), Guarded((max(need, 1),), torch.uint8)
        call(out=out.tensor, workspace=ws.tensor if need else None)
        torch.cuda.synchronize()
        assert out.intact() and ws.intact() and gdn.device_error() == 0
