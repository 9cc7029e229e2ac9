"""Inputs and outputs of one call beside each other in one buffer, sharing no element: accepted, with
the results of separate buffers, and nothing but the output written."""
import pytest
import torch

import gradient_sync_zero_gb300 as dps
from test_model_ops_gpu import BF, F32, bits

pytestmark = pytest.mark.gpu

P, T, D, V = 3, 10, 64, 40


def halves(form):
    """(x, out, buffer) views [P, T, D] of one buffer."""
    if form == "rows of each rank":
        buf = torch.randn(P, 2 * T, D, device="cuda")
        return buf[:, :T], buf[:, T:], buf
    if form == "every second row":
        buf = torch.randn(P, 2 * T, D, device="cuda")
        return buf[:, ::2], buf[:, 1::2], buf
    if form == "columns of rows by rank":
        buf = torch.randn(T, P, 2 * D, device="cuda")
        v = buf.transpose(0, 1)
        return v[..., :D], v[..., D:], buf
    if form == "rows of other spacing":          # x in every fourth row, out in every second odd one
        buf = torch.randn(P, 4 * T, D, device="cuda")
        return buf[:, ::4], buf[:, 1:2 * T:2], buf
    buf = torch.randn(2, P, T, D, device="cuda")
    return buf[0], buf[1], buf


FORMS = ["rows of each rank", "every second row", "columns of rows by rank", "rows of other spacing", "apart"]


@pytest.mark.parametrize("form", FORMS)
def test_dropout_beside_its_output(form):
    x, out, buf = halves(form)
    keep, mine = x.clone(), torch.zeros_like(buf, dtype=torch.bool)
    mine.as_strided(out.shape, out.stride(), out.storage_offset()).fill_(True)
    before, want = buf.clone(), torch.empty(P, T, D, device="cuda")
    cfg = dps.dropout_cfg(0.3, 5)
    dps.dp_dropout(keep, want, cfg)
    dps.dp_dropout(x, out, cfg)
    assert torch.equal(bits(out), bits(want)) and torch.equal(bits(x), bits(keep))
    assert torch.equal(buf[~mine], before[~mine])


@pytest.mark.parametrize("form", FORMS)
def test_logits_beside_their_gradient(form):
    x, out, _ = halves(form)
    keep, want = x.clone(), torch.empty(P, T, D, device="cuda")
    tokens = torch.randint(0, D, (P, T), device="cuda")
    lp, lse = torch.empty(P, T, device="cuda"), torch.empty(P, T, device="cuda")
    dps.dp_token_logprob(keep, tokens, lp, lse)
    dlogp = torch.randn(P, T, device="cuda")
    dps.dp_token_logprob_backward(keep, tokens, lse, dlogp, want)
    dps.dp_token_logprob_backward(x, tokens, lse, dlogp, out)
    assert torch.equal(bits(out), bits(want)) and torch.equal(bits(x), bits(keep))
    old, stats = lp.clone(), torch.empty(P, 4, device="cuda")
    dps.dp_policy_loss(keep, tokens, old, dlogp, lp, stats, dlogits=want)
    dps.dp_policy_loss(x, tokens, old, dlogp, lp, stats, dlogits=out)
    assert torch.equal(bits(out), bits(want)) and torch.equal(bits(x), bits(keep))


@pytest.mark.parametrize("act", [BF, F32])
def test_embedding_and_activations_in_one_arena(act):
    """[slot | activations] of each rank one after the other, the activations of either type."""
    rank = V * D + 2 * T * D
    arena = torch.randn(P, rank, device="cuda").to(BF)
    slot = arena[:, :V * D].unflatten(1, (V, D))
    x = arena.view(act)[:, (V * D * 2) // act.itemsize:][:, :T * D].unflatten(1, (T, D))
    assert x.untyped_storage().data_ptr() == arena.untyped_storage().data_ptr()
    tokens = torch.randint(-1, V, (P, T), device="cuda")
    table, want = slot.clone(), torch.empty(P, T, D, dtype=act, device="cuda")
    dps.dp_embedding_forward(table, tokens, want, scale=1.5)
    dps.dp_embedding_forward(slot, tokens, x, scale=1.5)
    assert torch.equal(bits(x), bits(want)) and torch.equal(bits(slot), bits(table))
    ws = dps.new_embedding_workspace(P, T, V, D)
    grad, dout = torch.empty_like(table), x.clone()
    dps.dp_embedding_backward(dout, tokens, grad, ws)
    dps.dp_embedding_backward(x, tokens, slot, ws)
    assert torch.equal(bits(slot), bits(grad)) and torch.equal(bits(x), bits(dout))


@pytest.mark.parametrize("rank", [1, 3, 7])
def test_output_of_one_rank_in_the_gaps_of_the_other(rank):
    """Rank 0 owns every second row, rank 1 those between, from row `rank` on."""
    buf = torch.full((2 * T + rank, D), float("nan"), device="cuda")
    out = buf.as_strided((2, T, D), (rank * D, 2 * D, 1))
    x, want = torch.randn(2, T, D, device="cuda"), torch.empty(2, T, D, device="cuda")
    cfg = dps.dropout_cfg(0.3, 5)
    dps.dp_dropout(x, want, cfg)
    dps.dp_dropout(x, out, cfg)
    assert torch.equal(bits(out), bits(want))
    out.fill_(float("nan"))
    assert torch.isnan(buf).all()
