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


def test_status_from_python():
    """A status word set from the host: reported, the rows left alone, and right again once the workspace is zeroed; through the
    block too, on the device of the workspace and on another stream."""
    counts, K, O = [12, 3], 256, 200
    _, W = expert_weights(2, O, K, 84)
    X, offsets = normal((15, K), 85).cuda(), offsets_of(counts).cuda()
    ws = awq.w4a16_experts_workspace(W[0], 15)
    clean = awq.w4a16_experts(X, offsets, *W, workspace=ws)
    assert awq.w4a16_status(ws) == 0
    ws[0] = 5
    out = torch.full_like(clean, 7.0)
    awq.w4a16_experts(X, offsets, *W, out=out, workspace=ws)
    assert awq.w4a16_status(ws) == 5 and awq.STATUS_NAMES[5] == "AWQ_ERR_TIMEOUT"
    torch.cuda.synchronize()
    assert awq.w4a16_status(ws, stream=torch.cuda.Stream()) == 5
    assert bool((out[:12] == 7.0).all()) and torch.equal(out[12:], clean[12:])
    ws.zero_()
    awq.w4a16_experts(X, offsets, *W, out=out, workspace=ws)
    assert awq.w4a16_status(ws) == 0 and torch.equal(out, clean)


def test_status_of_a_block(short_limit):
    E, K, I, T = 2, 256, 128, 40
    _, gate_up = expert_weights(E, 2 * I, K, 86)
    _, down = expert_weights(E, K, I, 87)
    X, ids = normal((T, K), 88).cuda(), (torch.arange(T)[:, None] % E).cuda()
    weights = torch.ones(T, 1).cuda()
    ws = (awq.w4a16_experts_workspace(gate_up[0], T), awq.w4a16_experts_workspace(down[0], T))
    clean = awq.w4a16_moe(X, ids, weights, gate_up, down, workspaces=ws)
    assert [awq.w4a16_status(w) for w in ws] == [0, 0]
    awq.set_experts_stall(0)
    awq.w4a16_moe(X, ids, weights, gate_up, down, workspaces=ws)
    assert [awq.w4a16_status(w) for w in ws] == [5, 5]
    awq.set_experts_stall(-1)
    for w in ws:
        w.zero_()
    assert torch.equal(awq.w4a16_moe(X, ids, weights, gate_up, down, workspaces=ws), clean)
