"""A wait of the experts' grouped kernel that runs out: the status reaches the host, nothing unfinished is stored, and the context
and the next call are as ever."""
import pytest
import torch

from tests.test_gpu_experts import expert_weights, normal, offsets_of
from weight_only_quantization_act_b200 import awq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    awq.load_library()


@pytest.fixture
def short_limit():
    awq.set_wait_limit_ns(5_000_000)
    yield
    awq.set_experts_stall(-1)
    awq.set_wait_limit_ns(2_000_000_000)


def status(workspace):
    torch.cuda.synchronize()
    return awq.load_library().awq_search_status(workspace.data_ptr(), workspace.numel(), None)


def test_a_stalled_tile_is_reported_and_not_stored(short_limit):
    """Expert 2's second token tile of the first 256 weight rows stalls: its rows 160 to 299 keep their first 256 columns, all
    else is written."""
    counts, K, O = [12, 3, 300], 640, 1000
    _, W = expert_weights(3, O, K, 80)
    X, offsets = normal((315, K), 81).cuda(), offsets_of(counts).cuda()
    ws = awq.w4a16_experts_workspace(W[0], 315)
    clean = awq.w4a16_experts(X, offsets, *W, workspace=ws)
    assert status(ws) == 0
    want = clean.clone()
    want[15 + 160:, :256] = 7.0
    out = torch.full_like(clean, 7.0)
    awq.set_experts_stall(4 + 1)
    awq.w4a16_experts(X, offsets, *W, out=out, workspace=ws)
    assert status(ws) == 5 and "site 5" in awq.load_library().awq_last_error().decode()
    assert torch.equal(out, want)
    # until the workspace is zeroed, experts of more than 8 rows are left alone
    awq.set_experts_stall(-1)
    out = torch.full_like(clean, 7.0)
    awq.w4a16_experts(X, offsets, *W, out=out, workspace=ws)
    assert status(ws) == 5
    assert torch.equal(out[12:15], clean[12:15]) and bool((out[:12] == 7.0).all()) and bool((out[15:] == 7.0).all())
    ws.zero_()
    assert torch.equal(awq.w4a16_experts(X, offsets, *W, workspace=ws), clean) and status(ws) == 0


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,tile", [(300, 0), (40, 3), (12, 39), (190, 10)])
def test_a_pair_with_more_tiles_ends(short_limit, rows, tile, gated):
    """Tiles of two, three and four groups in flight, more of them than CTA pairs: what is stored is what a whole call stores."""
    E, K, O = 8, 1152, 5120
    _, W = expert_weights(E, O, K, 82)
    X, offsets = normal((E * rows, K), 83).cuda(), offsets_of([rows] * E).cuda()
    ws = awq.w4a16_experts_workspace(W[0], E * rows)
    clean = awq.w4a16_experts(X, offsets, *W, gated=gated, workspace=ws)
    out = torch.full_like(clean, 7.0)
    awq.set_experts_stall(tile)
    awq.w4a16_experts(X, offsets, *W, gated=gated, out=out, workspace=ws)
    assert status(ws) == 5
    awq.set_experts_stall(-1)
    left = out == 7.0
    assert bool(left.any()) and bool((left | (out == clean)).all())
    ws.zero_()
    assert torch.equal(awq.w4a16_experts(X, offsets, *W, gated=gated, workspace=ws), clean) and status(ws) == 0
