"""Decoder operators at once: two blocks on two streams, and two captured blocks that share their workspaces and
are replayed in turn.  Every result equals that of the same calls by themselves, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
oeq = pytest.importorskip("cg_tensor_product_amd")

HEADS, DIM, TABLE = 4, 32, 700


class Block:
    """Tokens to rows, their norm, causal attention with the norm as queries, keys and values, and all gradients."""

    def __init__(self, lengths, seed, kind):
        gen = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=gen).to("cuda", kind)  # noqa: E731
        rows = sum(lengths)
        self.tokens = torch.randint(-1, TABLE, (rows,), generator=gen).cuda()
        self.table, self.residual, self.grad = rand(TABLE, HEADS * DIM), rand(rows, HEADS * DIM), rand(rows, HEADS, DIM)
        self.weight = torch.randn(HEADS * DIM, generator=gen).cuda()
        self.ptr = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        self.rng = torch.tensor([seed, 5], device="cuda")
        shape = (rows, HEADS, DIM)
        self.sizes = (oeq.oeq_embedding_workspace_size(TABLE, HEADS * DIM, rows, kind),
                      oeq.oeq_rms_norm_workspace_size(rows, HEADS * DIM),
                      *oeq.oeq_causal_attn_workspace_size(shape, shape, len(lengths), kind))

    def run(self, spaces=(None,) * 4):
        x = oeq.oeq_embedding_fwd(self.table, self.tokens)
        y, rstd, total = oeq.oeq_rms_norm_fwd(x, self.weight, self.residual)
        q = y.view(-1, HEADS, DIM)
        args = (q, q, q, self.ptr, self.ptr)
        out, lse = oeq.oeq_causal_attn_fwd(*args, p_drop=0.2, rng=self.rng, workspace=spaces[2])
        gq, gk, gv = oeq.oeq_causal_attn_bwd(*args, out, lse, self.grad, p_drop=0.2, rng=self.rng, workspace=spaces[3])
        gx, gw = oeq.oeq_rms_norm_bwd(total, rstd, gq.view_as(y), self.weight, workspace=spaces[1])
        gt = oeq.oeq_embedding_bwd(self.tokens, gx, TABLE, workspace=spaces[0])
        return out, lse, gq, gk, gv, gx, gw, gt


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


def blocks(kind):
    return Block([900, 3, 0, 260], 1, kind), Block([5, 1400], 2, kind)


@pytest.mark.parametrize("kind", [torch.float32, torch.float16, torch.bfloat16])
def test_on_two_streams(kind):
    pair, streams = blocks(kind), (torch.cuda.Stream(), torch.cuda.Stream())
    want = [b.run() for b in pair]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(3):
        for i, (b, s) in enumerate(zip(pair, streams)):
            with torch.cuda.stream(s):
                got[i].append(b.run())
    torch.cuda.synchronize()
    assert all(same(g, want[i]) for i in range(2) for g in got[i])


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_two_graphs_that_share_workspaces(kind):
    pair = blocks(kind)
    want = [b.run() for b in pair]
    spaces = [torch.zeros(max(sizes), dtype=torch.uint8, device="cuda") if max(sizes) else None
              for sizes in zip(*(b.sizes for b in pair))]
    graphs, got = [], []
    for b in pair:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(b.run(spaces))
        graphs.append(graph)
    for turn in range(4):
        for space in spaces:
            if space is not None:
                space.fill_(17 * turn)  # whatever another call left there
        for i in (turn % 2, 1 - turn % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(same(got[i], want[i]) for i in range(2))
        assert same(pair[0].run(), want[0])  # eager work between the replays
