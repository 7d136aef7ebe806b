"""The gated feed-forward's forward where it is walked over in tiles: more than 152 tiles of 128 rows and 128 columns, as a
training step has (calls of fewer take another kernel).  (1100, 72, 2568) goes in tiles of 64 columns of G and U,
(2100, 328, 2568) in tiles of 128; both have an odd number of row tiles, a last one that is not full, and columns that are
no multiple of a tile.  Bounds as for the other sizes: h 4e-3, gradients 8e-3 of the largest value; copies of the same
numbers, the same bits."""
import pytest
import torch

from selective_state_space_ssd_gb300 import binding
from test_ffn_gpu import check, compare, make, reference

pytestmark = pytest.mark.gpu
SIZES = [(1100, 72, 2568), (2100, 328, 2568)]


def cuda(c):
    return {k: t.cuda() for k, t in c.items()}


@pytest.mark.parametrize("stash", [True, False])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,d,f", SIZES)
def test_matches_float64(m, d, f, act, stash):
    compare(make(m, d, f, 21), act, stash=stash)


@pytest.mark.parametrize("m,d,f", SIZES)
def test_stash_changes_no_bit(m, d, f):
    c = make(m, d, f, 22)
    a, b = compare(c, "gelu"), compare(c, "gelu", stash=False)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("m,d,f", SIZES)
def test_strided_rows_and_leading_dimensions(m, d, f):
    d_ = cuda(make(m, d, f, 23))
    x, wg, wu, dh = (d_[k] for k in ("x", "wg", "wu", "dh"))

    def passes(rows):
        stash = binding.ffn_stash(rows, wg)
        h = binding.ffn_forward(rows, wg, wu, stash=stash)
        return [h, *binding.ffn_backward(dh, rows, wg, wu, stash=stash).values()]

    want = passes(x)
    room = torch.full((m, 2 * d + 24), float("nan"), device="cuda", dtype=torch.bfloat16)
    room[:, d + 8:2 * d + 8] = x
    assert all(torch.equal(a, b) for a, b in zip(passes(room[:, d + 8:2 * d + 8]), want))
    assert torch.equal(binding.ffn_forward(x.view(20, m // 20, d), wg, wu).view(m, f), want[0])


@pytest.mark.parametrize("row", [0, 500, 1099])
@pytest.mark.parametrize("m,d,f", SIZES)
def test_a_nan_stays_in_its_row(m, d, f, row):
    c = make(m, d, f, 24)
    ref = reference(c, "silu")
    c["x"][row, 5] = float("nan")
    d_ = cuda(c)
    stash = binding.ffn_stash(d_["x"], d_["wg"])
    h = binding.ffn_forward(d_["x"], d_["wg"], d_["wu"], stash=stash)
    dx = binding.ffn_backward(d_["dh"], d_["x"], d_["wg"], d_["wu"], stash=stash)["dx"]
    rest = [r for r in range(m) if r != row]
    assert h[row].isnan().all() and dx[row].isnan().all()
    check("h", h[rest], ref["h"][rest], 4e-3)
    check("dx", dx[rest], ref["dx"][rest], 8e-3)


# (with dx's sums in pieces too, an odd number of row tiles and one)
@pytest.mark.parametrize("m,d,f", SIZES + [(300, 72, 4104), (1, 8, 1024)])
def test_rows_behind_the_last_are_left_alone(m, d, f):
    d_ = cuda(make(m, d, f, 25))
    x, wg, wu, dh = (d_[k] for k in ("x", "wg", "wu", "dh"))
    prob = binding.ffn_problem(x, wg)
    h = torch.full((m + 40, f), 7.0, device="cuda", dtype=torch.bfloat16)
    dx = torch.full((m + 40, d), 7.0, device="cuda", dtype=torch.bfloat16)
    dwg, dwu = (torch.full((f + 40, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    stash = torch.full((binding.ssd_ffn_stash_size(prob) + 4096,), 77, dtype=torch.uint8, device="cuda")
    n = max(binding.ssd_ffn_workspace_size(prob, False, True), binding.ssd_ffn_workspace_size(prob, True, True))
    ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    binding.ssd_ffn_forward(prob, x, wg, wu, h, stash, stash.numel(), ws, n)
    binding.ssd_ffn_backward(prob, dh, x, wg, wu, dx, dwg, dwu, stash, stash.numel(), ws, n)
    assert (h[m:] == 7).all() and (dx[m:] == 7).all() and (dwg[f:] == 7).all() and (dwu[f:] == 7).all()
    assert (stash[-4096:] == 77).all() and (ws[n:] == 77).all()
    kept = binding.ffn_stash(x, wg)
    assert torch.equal(h[:m], binding.ffn_forward(x, wg, wu, stash=kept))
    want = binding.ffn_backward(dh, x, wg, wu, stash=kept)
    assert torch.equal(dx[:m], want["dx"]) and torch.equal(dwg[:f], want["dwg"]) and torch.equal(dwu[:f], want["dwu"])
    assert binding.ssd_read_status(ws) == (0, 0)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("m,d,f", SIZES)
def test_same_bits_again_on_another_stream_and_in_a_graph(m, d, f, act):
    d_ = cuda(make(m, d, f, 26))
    x, wg, wu, dh = (d_[k] for k in ("x", "wg", "wu", "dh"))

    def both(stream=None):
        stash = binding.ffn_stash(x, wg)
        h = binding.ffn_forward(x, wg, wu, act, stash=stash, stream=stream)
        return [h, *binding.ffn_backward(dh, x, wg, wu, act, stash=stash, stream=stream).values()]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
