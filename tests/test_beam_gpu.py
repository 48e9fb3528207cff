"""spec_beam_select and spec_beam_reorder against the plain forms
(tests/plain_draft.py), and a candidate tree grown by beams, verified, and its
accepted path's states gathered (needs a GPU)."""
import math

import pytest
import torch

import oracle
import plain_draft as plain
from token_verification_gb300 import api

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def case(B, W, V, dtype, seed, dead=0):
    g = gen(seed)
    x = (torch.randn((B, W, V), generator=g, device="cuda") * 3.0).to(dtype)
    s = -4.0 * torch.rand((B, W), generator=g, device="cuda")
    if dead:
        s[:, torch.randperm(W, generator=g, device="cuda")[:dead]] = -math.inf
    return x, s


def check(x, s, n, moved=None):
    out = api.spec_beam_select(x, s, n)
    torch.cuda.synchronize()
    assert not bool(out.status.any())
    got = plain.check_beam(x, s, n, out)
    if moved is not None:
        assert got <= moved
    return out


@pytest.mark.parametrize("V", [1, 5, 8, 33, 256, 1000, 8193, 32000])
@pytest.mark.parametrize("W,n,dtype", [(1, 1, BF16), (2, 64, F32), (3, 7, BF16), (5, 10, F32),
                                       (8, 16, BF16), (13, 128, BF16)])
def test_sizes(W, n, dtype, V):
    check(*case(2, W, V, dtype, W * V + n), n)


@pytest.mark.parametrize("B,W,V,n,dtype,dead", [
    (2, 8, 128256, 16, BF16, 0), (1, 4, 152064, 8, BF16, 1), (1, 32, 50001, 64, F32, 7),
    (2, 64, 5001, 128, BF16, 20), (90, 2, 3001, 4, F32, 0), (400, 3, 515, 6, BF16, 0),
    (1, 1, 700001, 32, BF16, 0)])
def test_large(B, W, V, n, dtype, dead):
    check(*case(B, W, V, dtype, B + W + V, dead), n)


def test_first_step_and_finished_beams():
    """All beams but one dead; all dead; beams without a finite logit; dead rows are not read."""
    x, s = case(4, 6, 2001, BF16, 1)
    s[0, 1:] = -math.inf
    x[0, 1:] = math.nan
    s[1] = -math.inf
    x[2, :3] = -math.inf
    x[3] = -math.inf
    out = check(x, s, 20, moved=0)
    assert bool((out.tokens[1] == -1).all()) and bool((out.tokens[3] == -1).all())


def test_few_candidates():
    x, s = case(2, 3, 900, F32, 2)
    x[:, :, 5:] = -math.inf
    out = check(x, s, 40)
    assert int((out.tokens[0] >= 0).sum()) == 15


@pytest.mark.parametrize("V", [300, 1003, 12001])
def test_ties(V):
    """Equal rows with equal scores: equal candidates go by ascending beam and token (odd V:
    the beams' rows start at different alignments); constant rows: every candidate is equal."""
    x, s = case(3, 6, V, BF16, 3)
    x[0] = x[0, :1]
    s[0] = -1.0
    x[1] = 0.5
    s[1] = -2.0
    x[2] = 1.0
    s[2] = torch.tensor([-3.0, -1.0, -2.0, -1.0, -math.inf, -5.0])
    for n in (1, 50, 128):
        check(x, s, n, moved=0)
        check(x.float(), s, n, moved=0)


def test_bad_requests():
    x, s = case(5, 4, 1500, F32, 4)
    x[0, 2, 1499] = math.nan
    x[1, 0, 0] = math.inf
    s[2, 3] = math.nan
    s[3, 3] = math.inf
    out = api.spec_beam_select(x, s, 9)
    assert out.status.tolist() == [2, 2, 2, 2, 0]
    assert bool((out.tokens[:4] == -1).all()) and bool((out.scores[:4] == -math.inf).all())
    good = api.BeamOutputs(out.tokens[4:], out.parents[4:], out.scores[4:])
    plain.check_beam(x[4:], s[4:], 9, good)


def test_unaligned_base_and_refusals():
    x, s = case(2, 3, 1001, BF16, 5)
    buf = torch.empty(x.numel() + 8, dtype=BF16, device="cuda")
    for shift in (1, 2, 4, 7):
        y = buf[shift:shift + x.numel()].view(x.shape)
        y.copy_(x)
        check(y, s, 11)
    with pytest.raises(ValueError):
        api.spec_beam_select(x, s[:, :2], 4)
    with pytest.raises(TypeError):
        api.spec_beam_select(x, s.double(), 4)
    with pytest.raises(api.VerifyError):
        api.spec_beam_select(x, s, 129)
    with pytest.raises(api.VerifyError):
        api.spec_beam_select(torch.zeros(1, 65, 8, device="cuda"),
                             torch.zeros(1, 65, device="cuda"), 4)


# --- reordering ------------------------------------------------------------

TYPES = [torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.float64]


def states(shape, dtype, seed, order=(0, 1, 2, 3, 4, 5)):
    """A [G, B, W, H, L, D] view whose memory lies in the given order of dimensions."""
    g = gen(seed)
    mem = [shape[i] for i in order]
    x = torch.randint(0, 255, mem, generator=g, device="cuda").to(dtype)
    back = [order.index(i) for i in range(6)]
    return x.permute(back)


def check_reorder(state, parents, out, lens=None):
    d = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    p = torch.tensor(parents, dtype=torch.int32, device="cuda")
    want = plain.reorder(state.cpu(), p.cpu(), out.cpu(), lens)
    status = torch.full((state.shape[1],), 77, dtype=torch.int32, device="cuda")
    assert api.spec_beam_reorder(state, p, out, lens=d, status=status) is out
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    return status.tolist()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [1, 3, 8, 80])
@pytest.mark.parametrize("order", [(0, 1, 2, 3, 4, 5), (0, 1, 3, 2, 4, 5), (4, 1, 2, 0, 3, 5)])
def test_reorder(dtype, D, order):
    B, W, Wo, L = 3, 4, 6, 21
    state = states((2, B, W, 3, L, D), dtype, D, order)
    out = states((2, B, Wo, 3, L, D), dtype, D + 1, order)
    parents = [[0, 0, 3, -1, 2, 1], [3, 2, 1, 0, -1, -1], [1, 1, 1, 1, 1, 1]]
    assert check_reorder(state, parents, out, [L, 7, 0]) == [0, 0, 0]
    assert check_reorder(state, parents, out) == [0, 0, 0]


def test_reorder_mixed_layouts_and_expanded_state():
    state = states((1, 2, 4, 2, 9, 16), BF16, 1, (0, 1, 3, 2, 4, 5))
    out = states((1, 2, 4, 2, 9, 16), BF16, 2)
    check_reorder(state, [[3, 2, 1, 0], [0, 0, 1, 1]], out, [9, 4])
    one = states((1, 2, 1, 2, 9, 16), BF16, 3).expand(1, 2, 4, 2, 9, 16)
    check_reorder(one, [[3, 2, 1, 0], [0, -1, 1, 1]], out)
    odd = states((1, 2, 4, 2, 9, 17), BF16, 4)[..., 1:]
    check_reorder(odd, [[3, 2, 1, 0], [0, -1, 1, 1]], out, [1, 8])


def test_reorder_large_and_status():
    state = states((2, 5, 8, 4, 300, 64), BF16, 5)
    out = states((2, 5, 8, 4, 300, 64), BF16, 6)
    parents = torch.randint(0, 8, (5, 8), generator=gen(7), device="cuda").tolist()
    parents[2][3] = 8
    parents[3][0] = -2
    assert check_reorder(state, parents, out, [300, 299, 150, 301, -1]) == [0, 0, 16, 20, 4]


def test_reorder_new_output_and_refusals():
    state = states((1, 2, 3, 1, 1, 8), F32, 8)
    p = torch.tensor([[2, -1], [0, 1]], dtype=torch.int32, device="cuda")
    out = api.spec_beam_reorder(state, p)
    assert torch.equal(out[0, 0, 0], state[0, 0, 2]) and not bool(out[0, 0, 1].any())
    with pytest.raises(ValueError):
        api.spec_beam_reorder(state, p[:1])
    with pytest.raises(ValueError):
        api.spec_beam_reorder(states((1, 2, 3, 1, 1, 8), F32, 8, (0, 1, 2, 3, 5, 4))[:, :, :, :, :, ::2],
                              p)
    with pytest.raises(TypeError):
        api.spec_beam_reorder(state, p, out.to(BF16))
    with pytest.raises(api.VerifyError):  # in place
        api.spec_beam_reorder(state, torch.zeros((2, 3), dtype=torch.int32, device="cuda"), state)
    with pytest.raises(api.VerifyError):  # an output that folds onto itself
        api.spec_beam_reorder(state, p, out[:, :, :1].expand(1, 2, 2, 1, 1, 8))


def test_reorder_moves_block_tables():
    """A paged cache moves by its block table: int32 rows of any odd length."""
    table = states((1, 4, 5, 1, 1, 37), torch.int32, 9)
    out = torch.zeros_like(table)
    check_reorder(table, [[4, 3, 2, 1, 0]] * 4, out)


# --- together ----------------------------------------------------------------

def test_beams_grow_a_tree_that_is_verified_and_compacted():
    """Each level's selection gives the tree's next nodes (token, parent) and moves the draft's
    states; the grown tree goes through greedy verification (checked against the oracle) and
    the accepted path's states are gathered out of the nodes' states."""
    B, W, V, depth, H = 6, 4, 900, 3, 16
    g = gen(21)
    target_of = torch.randn((V, V), generator=g, device="cuda") * 3
    draft_of = target_of + 0.7 * torch.randn((V, V), generator=g, device="cuda")
    embed = torch.randn((V, H), generator=g, device="cuda")
    root = torch.randint(0, V, (B,), generator=g, device="cuda")
    tokens = root[:, None].expand(B, W).contiguous()
    scores = torch.full((B, W), -math.inf, device="cuda")
    scores[:, 0] = 0.0
    state = embed[tokens]  # the draft's state: the sum of its path's embeddings
    node_state = [embed[root][:, None]]
    parents, nodes = [], []
    for d in range(depth):
        logits = draft_of[tokens].to(BF16)
        out = api.spec_beam_select(logits, scores, W)
        plain.check_beam(logits, scores, W, out)
        assert bool((out.tokens >= 0).all())
        moved = api.spec_beam_reorder(state[None, :, :, None, None], out.parents)[0, :, :, 0, 0]
        tokens, scores = out.tokens.long(), out.scores
        state = moved + embed[tokens]
        node_state.append(state)
        nodes.append(out.tokens)
        parents.append(torch.zeros_like(out.parents) if d == 0
                       else 1 + (d - 1) * W + out.parents)
    parent, node_tokens = torch.cat(parents, 1).contiguous(), torch.cat(nodes, 1).contiguous()
    ctx = torch.cat([root[:, None], node_tokens.long()], 1)
    target = target_of[ctx].to(BF16).contiguous()
    out = api.spec_verify_tree(target, parent, node_tokens, depth)
    bits = target.view(torch.int16).cpu().numpy().view("uint16")
    for b in range(B):
        ref = oracle.tree(bits[b:b + 1], parent[b].cpu().numpy(), node_tokens[b:b + 1].cpu().numpy(),
                          depth)
        assert (out.tokens[b].cpu().numpy() == ref["tokens"][0]).all()
    assert int(out.accept_len.max()) > 1
    all_states = torch.cat(node_state, 1)  # [B, 1 + depth W, H]
    got = api.spec_beam_reorder(all_states[None, :, :, None, None], out.path)[0, :, :, 0, 0]
    for b in range(B):
        n = int(out.accept_len[b])
        assert torch.equal(got[b, :n], all_states[b, out.path[b, :n].long()])
        assert not bool(got[b, n:].any())
        path = torch.cat([root[b:b + 1], out.tokens[b, :n - 1].long()])
        # sums of the path's embeddings, added in the same order
        want = embed[path[0]]
        for d in range(1, n):
            want = want + embed[path[d]]
            assert torch.equal(got[b, d], want)


def test_every_candidate_equal_in_wide_beams():
    """64 beams of constant rows, 128 kept: the merge of 8192 equal candidates."""
    x = torch.full((2, 64, 9001), 0.25, dtype=BF16, device="cuda")
    s = torch.full((2, 64), -1.5, device="cuda")
    s[1, ::2] = -math.inf
    check(x, s, 128, moved=0)


def test_two_graphs_on_two_streams():
    """Each captured call has scratch of its own: two graphs replay at once."""
    ins = [case(24, 16, 9001, BF16, 50 + i, dead=3) for i in range(2)]
    graphs, outs, streams = [], [], []
    for x, s in ins:
        api.spec_beam_select(x, s, 32)
        g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=st):
            outs.append(api.spec_beam_select(x, s, 32))
        graphs.append(g)
        streams.append(st)
    for i, (x, s) in enumerate(ins):
        y, r = case(24, 16, 9001, BF16, 60 + i, dead=3)
        x.copy_(y)
        s.copy_(r)
    torch.cuda.synchronize()
    for _ in range(4):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (x, s), out in zip(ins, outs):
        want = api.spec_beam_select(x, s, 32)
        assert torch.equal(out.tokens, want.tokens) and torch.equal(out.parents, want.parents)
        assert torch.equal(out.scores, want.scores)
        few = api.BeamOutputs(out.tokens[:2], out.parents[:2], out.scores[:2])
        plain.check_beam(x[:2], s[:2], 32, few)


def test_reorder_offsets_past_32_bits():
    D = (1 << 30) + 16
    state = torch.zeros((1, 1, 5, 1, 1, D), dtype=torch.uint8, device="cuda")
    for w in range(5):
        state[0, 0, w, 0, 0, 0] = w + 1
        state[0, 0, w, 0, 0, -1] = 10 * (w + 1)
        state[0, 0, w, 0, 0, D // 2 + 7] = w + 100
    p = torch.tensor([[4, 0, 4, -1]], dtype=torch.int32, device="cuda")
    out = api.spec_beam_reorder(state, p)
    for w, q in enumerate([4, 0, 4]):
        assert torch.equal(out[0, 0, w, 0, 0], state[0, 0, q, 0, 0])
    assert not bool(out[0, 0, 3].any())


def test_binding_and_long_way_agree():
    """Outputs given by the caller take the Python checks, new ones the compiled binding."""
    x, s = case(2, 4, 3001, BF16, 70)
    a = api.spec_beam_select(x, s, 9)
    b = api.BeamOutputs(*(torch.empty_like(t) for t in (a.tokens, a.parents, a.scores, a.status)))
    api.spec_beam_select(x, s, 9, out=b)
    for f in ("tokens", "parents", "scores", "status"):
        assert torch.equal(getattr(a, f), getattr(b, f))
    assert api.spec_beam_select(x, s, 9, status=False).status is None
    with pytest.raises(api.VerifyError):  # the C call's own refusal, through the binding
        api.spec_beam_select(torch.zeros((1, 65, 8), device="cuda"),
                             torch.zeros((1, 65), device="cuda"), 4)
    import numpy as np
    assert torch.equal(api.spec_beam_select(x, s, np.int64(9)).tokens, a.tokens)


@pytest.mark.parametrize("W", [4, 16])
def test_lowest_value_masks(W):
    """Masks of the type's lowest value beside ordinary logits, and whole rows of it: their
    tokens are the last candidates, in order."""
    x, s = case(2, W, 2000, F32, 80 + W)
    x[0, :, 40:] = torch.finfo(F32).min
    x[1] = torch.finfo(F32).min
    out = api.spec_beam_select(x, s, 128)
    assert not bool(out.status.any())
    first = min(128, 40 * W)
    plain.check_beam(x[:1, :, :40].contiguous(), s[:1], first, api.BeamOutputs(
        out.tokens[:1, :first], out.parents[:1, :first], out.scores[:1, :first]))
    best = int(s[1].argmax())  # uniform rows: log-probability -log V each
    assert abs(float(out.scores[1, 0]) - float(s[1].max()) + math.log(2000)) < 1e-4
    assert out.parents[1].tolist() == [best] * 128 and out.tokens[1].tolist() == list(range(128))


@pytest.mark.parametrize("W", [4, 16])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scores_that_cancel(W, dtype):
    """Every other beam has a score of 2^24 and a first token 2^24 above all others: the other
    tokens' scores are differences of those, and compete with the other beams'."""
    x, s = case(3, W, 500, dtype, 90 + W)
    x[:, ::2, 0] = 2.0 ** 24
    s[:, ::2] += 2.0 ** 24
    out = api.spec_beam_select(x, s, 96)
    assert not bool(out.status.any())
    plain.check_beam(x, s, 96, out)
