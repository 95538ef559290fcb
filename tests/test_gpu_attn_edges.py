"""The attention half at its edges on the GPU: refusals that need a device, wrong data that has to be
recorded, values that are not finite, and batches that reach every branch of the schedules."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import top_routing_grouped_router_gb300 as moe  # noqa: E402
from attn_ref import make_batch  # noqa: E402
from test_gpu_attn import ATTN, Dev  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from top_routing_grouped_router_gb300 import build
    build.build()


def test_a_call_without_a_workspace_is_refused():
    d = Dev(make_batch(*ATTN["few tokens"], seed=1))
    with pytest.raises(moe.MoEError) as e:
        moe.moe_paged_attention(d.shape, d.q, d.cache, d.batch, d.out)
    assert e.value.status == -4
    with pytest.raises(moe.MoEError) as e:
        moe.moe_rope_append(d.shape, moe.make_rope(128), d.q, d.q[:, :4].contiguous(), d.q[:, 4:].contiguous(), d.cache,
                            d.batch, d.out)
    assert e.value.status == -4
