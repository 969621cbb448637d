"""A serving step as programs run it: pages, trees, rotary writes, attention
and kept rows one after another, over several steps, captured into a graph
whose lengths, trees and pages change, on other streams, in padded batches."""
import math

import pytest
import torch

import tests.pagedref as ref
import tests.stepref as step
from tests.test_gpu_paged import BF16, DTYPES, E4M3, E5M2, batch_of, bits, filled, gen, on_gpu, sz
from tests.test_gpu_step import forest, ints

pytestmark = pytest.mark.gpu


class Server:
    """Sequences that draft a tree in every step and keep one line of it."""

    def __init__(self, dtype, seqs, nodes, H, G, D, P, most, seed):
        m = self.m = sz()
        self.dtype, self.seqs, self.nodes, self.H, self.G, self.D, self.P = dtype, seqs, nodes, H, G, D, P
        width = -(-most // P)
        pages = seqs * width
        self.cache = m.paged_cache(pages, P, H, D, dtype)
        self.pool = m.page_pool(pages, P)
        cuda = dict(dtype=torch.int32, device="cuda")
        T = self.T = seqs * nodes
        self.table, self.lens, self.held = torch.zeros(seqs, width, **cuda), torch.zeros(seqs, **cuda), torch.zeros(seqs, **cuda)
        self.batch = m.PageBatch(self.table, self.lens, torch.arange(0, T + 1, nodes, **cuda), T, max_new=nodes, max_kv=most)
        self.parents = torch.zeros(T, **cuda)
        self.kept, self.counts = torch.zeros(seqs, 5, **cuda), torch.zeros(seqs, **cuda)
        self.x = torch.zeros(T, H * (G + 2), D, dtype=torch.bfloat16, device="cuda")
        self.f = m.rotary_frequencies(D, stretch=4.0, original=512)
        self.rotary = m.Rotary(self.f, amplitude=1.125)
        self.ws, self.aws = m.attention_workspace(self.cache, self.batch, H * G), m.assign_workspace(self.batch)
        self.out, self.lse = torch.zeros(T, H * G, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, H * G, device="cuda")
        self.tree = (torch.zeros(T, m.tree_words(self.batch), dtype=torch.int64, device="cuda"), torch.zeros(T, **cuda))
        self.slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.q = torch.zeros_like(self.out)
        self.g = gen(seed)
        self.past = [0] * seqs
        self.line = [[] for _ in range(seqs)]                # what is kept: (position, key rows, value rows)

    def inputs(self):
        """The next step's lengths, trees, rows and the line that will be kept."""
        n, g = self.nodes, self.g
        trees = [forest("random", n, g) for _ in range(self.seqs)]
        for t in trees:
            t[0] = -1
        self.lens.copy_(ints([p + n for p in self.past]))
        self.parents.copy_(ints(sum(trees, [])))
        self.x.copy_(torch.randn(self.x.shape, generator=g).to(torch.bfloat16))
        lines = []
        for t in trees:
            at, line = int(torch.randint(0, n, (1,), generator=g)), []
            while at >= 0:
                line.append(at)
                at = t[at]
            lines.append(line[::-1][:5])
        rows = torch.zeros(self.seqs, 5, dtype=torch.int32)
        for i, line in enumerate(lines):
            rows[i, :len(line)] = ints(line)
        self.kept.copy_(rows)
        self.counts.copy_(ints([len(line) for line in lines]))
        self.trees, self.lines = trees, lines

    def run(self):
        m, HG, H = self.m, self.H * self.G, self.H
        m.pages_assign(self.pool, self.batch, self.held, slots=self.slots, ws=self.aws, check=False)
        m.draft_tree(self.batch, self.parents, out=self.tree, status=self.cache.status, check=False)
        m.rotary_write(self.cache, self.batch, self.rotary, self.x[:, :HG], self.x[:, HG:HG + H], self.x[:, HG + H:],
                       positions=self.tree[1], out=self.q, check=False)
        m.tree_attention(self.q, self.cache, self.batch, self.tree[0], out=self.out, lse=self.lse, ws=self.ws, check=False)
        m.cache_keep(self.cache, self.batch, self.kept, self.counts, check=False)

    def verify(self):
        """Everything from the rows themselves: each token's line of ancestors
        over what was kept before, in 64 bits."""
        n, H, G, D, P = self.nodes, self.H, self.G, self.D, self.P
        assert int(self.cache.status.item()) == 0 and int(self.pool.status.item()) == 0
        x = self.x.cpu()
        table = self.table.tolist()
        for i, tree in enumerate(self.trees):
            past, at = self.past[i], i * n
            depth = []
            for j, p in enumerate(tree):
                depth.append(0 if p < 0 else depth[p] + 1)
            positions = [past + d for d in depth]
            assert self.tree[1][at:at + n].tolist() == positions
            cos, sin = step.angles(positions, self.f.tolist())
            q, _ = step.turned(x[at:at + n, :H * G], cos, sin, False, 1.125)
            k, _ = step.turned(x[at:at + n, H * G:H * G + H], cos, sin, False, 1.125)
            v = x[at:at + n, H * G + H:].double()
            if self.dtype == BF16:
                k = k.to(torch.bfloat16).double()
            else:
                k = ref.dequantise(*ref.quantise(k.float().double(), self.dtype))
                v = ref.dequantise(*ref.quantise(v, self.dtype))
            q = self.q[at:at + n].double().cpu()             # rounded once; held to its bound by tests of its own
            for j in range(n):
                line, p = [], j
                while p >= 0:
                    line.append(p)
                    p = tree[p]
                line = line[::-1]
                K = torch.stack([r[0] for r in self.line[i]] + [k[p] for p in line])
                V = torch.stack([r[1] for r in self.line[i]] + [v[p] for p in line])
                for h in range(H * G):
                    s = (K[:, h // G] @ q[j, h]) * D ** -0.5
                    p64 = torch.softmax(s, 0)
                    want, a = p64 @ V[:, h // G], p64 @ V[:, h // G].abs()
                    # BF16 keys of BF16 caches may round the other way (2^-7 of a key): as much as their scores move
                    size = float((K[:, h // G].abs() @ q[j, h].abs()).max()) * D ** -0.5
                    e = 2.0 ** -14 * size + 2.0 ** -20
                    tol = (2.0 ** -8 * (a + want.abs()) + 2 * e * a) * 1.01 + 1e-30
                    got = self.out[at + j, h].double().cpu()
                    assert bool(((got - want).abs() <= tol).all()), (i, j, h, float(((got - want).abs() / tol).max()))
                    assert abs(float(self.lse[at + j, h]) - float(torch.logsumexp(s, 0))) <= e + 1e-5
            for j in range(n):
                pos = past + j
                assert int(self.slots[at + j]) == table[i][pos // P] * P + pos % P
            for t in self.lines[i]:
                self.line[i].append((k[t], v[t]))
            self.past[i] += len(self.lines[i])
            # what the cache holds of the line is what was kept
            flat = ref.gather(self.cache.data.cpu(), None if self.cache.scales is None else self.cache.scales.cpu(),
                              self.table.cpu(), i, self.past[i], P)
            K = torch.stack([r[0] for r in self.line[i]])
            assert torch.equal(flat[:, 1], torch.stack([r[1] for r in self.line[i]]))
            if self.dtype == BF16:                           # at most to the next BF16 value
                assert bool(((flat[:, 0] - K).abs() <= 2.0 ** -7 * K.abs() + 1e-6).all())
                self.line[i] = [(flat[r, 0], b) for r, (_, b) in enumerate(self.line[i])]
            else:
                assert torch.equal(flat[:, 0], K)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(3, 7, 2, 4, 128, 16), (2, 20, 1, 2, 64, 32), (5, 1, 2, 2, 64, 16)], ids=str)
def test_steps_with_trees(dtype, shape):
    seqs, nodes, H, G, D, P = shape
    s = Server(dtype, seqs, nodes, H, G, D, P, 200, seqs)
    for rep in range(6):
        print("step", ref.NAMES[dtype], shape, rep, flush=True)
        s.inputs()
        s.run()
        s.verify()


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_steps_with_trees_captured(dtype):
    """The whole step in one graph, replayed with other lengths, trees, pages
    and rows, eager work between the replays."""
    s = Server(dtype, 3, 9, 2, 4, 128, 16, 200, 1)
    stream = torch.cuda.Stream()
    s.inputs()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.run()                                              # the first step, uncaptured
    stream.synchronize()
    s.verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
    for rep in range(6):
        print("replay", ref.NAMES[dtype], rep, flush=True)
        s.inputs()
        torch.cuda.synchronize()
        s.out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        s.verify()


def test_two_graphs_share_workspaces():
    """Steps of two shapes, captured over the same workspaces, replayed in turn."""
    shapes = [(E5M2, 3, 9, 2, 4, 128, 16, 300, 1), (E5M2, 2, 40, 1, 4, 64, 16, 300, 2)]
    servers = [Server(*a) for a in shapes]
    ws = max((s.ws for s in servers), key=lambda t: t.numel())
    aws = max((s.aws for s in servers), key=lambda t: t.numel())
    stream, graphs = torch.cuda.Stream(), []
    for s in servers:
        s.ws, s.aws = ws, aws
        s.inputs()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            s.run()
        stream.synchronize()
        s.verify()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            s.run()
        graphs.append(graph)
    for rep in range(3):
        for s, graph in zip(servers, graphs):
            s.inputs()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            s.verify()


def test_other_streams():
    """Every call on a stream that is not the current one; what Python makes
    for a call (outputs, workspaces) is that stream's until it is done."""
    m = sz()
    dtype, H, G, D, P = E4M3, 2, 4, 128, 16
    lens, new = [300, 90], [20, 20]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=8)
    data, scales = filled(dtype, pages, H, P, D, 5)
    g = gen(2)
    x = torch.randn(T, H * (G + 2), D, generator=g).to(torch.bfloat16).cuda()
    parents = ints(sum([forest("random", n, g) for n in new], [])).cuda()
    rotary = m.Rotary(m.rotary_frequencies(D))
    kept, counts = ints([[1, 5, 9], [0, 19, 0]]).cuda(), ints([3, 2]).cuda()
    side = torch.cuda.Stream()

    def whole(stream):
        cache, batch = on_gpu(dtype, data, scales), batch_of(table, kv, starts, T, max_new=20)
        pool = m.page_pool(40, P)
        held = torch.zeros(2, dtype=torch.int32, device="cuda")
        grown = m.PageBatch(torch.zeros(2, 19, dtype=torch.int32, device="cuda"), kv.cuda(), starts.cuda(), T, max_new=20)
        torch.cuda.synchronize()
        slots = m.pages_assign(pool, grown, held, slots=True, stream=stream, check=False)
        masks, positions = m.draft_tree(batch, parents, stream=stream, check=False)
        if stream is not None:
            stream.synchronize()                             # the tensors were made for the current stream
        q = m.rotary_write(cache, batch, rotary, x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:], positions=positions,
                           stream=stream, check=False)
        if stream is not None:
            stream.synchronize()
        out, lse = m.tree_attention(q, cache, batch, masks, lse=True, stream=stream, check=False)
        m.cache_keep(cache, batch, kept, counts, stream=stream)
        torch.cuda.synchronize()
        return [slots, masks, positions, q, out, lse, cache.data.view(torch.uint8), cache.scales, held, grown.page_table]

    for a, b in zip(whole(None), whole(side)):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    """Steps of two servers on two streams, nothing shared, without waiting."""
    servers = [Server(E4M3, 3, 9, 2, 4, 128, 16, 300, 1), Server(BF16, 2, 40, 1, 4, 64, 16, 300, 2)]
    streams = [torch.cuda.Stream() for _ in servers]
    for rep in range(3):
        for s in servers:
            s.inputs()
        torch.cuda.synchronize()
        for s, stream in zip(servers, streams):
            with torch.cuda.stream(stream):
                s.run()
        torch.cuda.synchronize()
        for s in servers:
            s.verify()


@pytest.mark.parametrize("seqs", [62, 63, 64, 130])
def test_tokens_behind_the_last_sequence_are_left(seqs):
    """A padded batch: rows of tokens that are none's, before the first
    sequence and behind the last, keep what they held."""
    m = sz()
    dtype, H, G, D, P, gap = E5M2, 1, 2, 64, 16, 19
    lens, new = [20 + i % 7 for i in range(seqs)], [1 + i % 3 for i in range(seqs)]
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=8, gap=gap)
    data, scales = filled(dtype, pages, H, P, D, 5)
    cache, batch = on_gpu(dtype, data, scales), batch_of(table, kv, starts, T, max_new=3)
    rest = torch.ones(T, dtype=torch.bool)
    rest[gap:T - gap] = False
    parents = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    masks, positions = torch.full((T, 1), 9, dtype=torch.int64, device="cuda"), torch.full((T,), 9, dtype=torch.int32, device="cuda")
    m.draft_tree(batch, parents, out=(masks, positions))
    x = torch.randn(T, H * (G + 2), D, generator=gen(3)).to(torch.bfloat16).cuda()
    q = torch.full((T, H * G, D), 9.0, dtype=torch.bfloat16, device="cuda")
    m.rotary_write(cache, batch, m.Rotary(m.rotary_frequencies(D)), x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:], out=q)
    out, lse = torch.full_like(q, 9.0), torch.full((T, H * G), 9.0, device="cuda")
    m.tree_attention(q, cache, batch, masks, out=out, lse=lse)
    for t in (masks, positions, q, out, lse):
        assert bool((t[rest.cuda()] == 9).all()) and not bool((t[~rest.cuda()].float() == 9).all())
    written = torch.zeros(pages, P, dtype=torch.bool)
    for i, n in enumerate(lens):
        for p in range(n - new[i], n):
            written[int(table[i, p // P]), p % P] = True
    same = (bits(cache.data) == bits(data)).view(pages, 2, H, P, D).all(-1).all(2).all(1)
    assert bool(same[~written].all())


def test_pages_past_four_gib():
    """Rows whose offsets pass 32 bits: written, attended to and moved."""
    m = sz()
    dtype, H, G, D, P = E4M3, 8, 2, 128, 64
    pages = (5 << 30) // (2 * H * P * D)
    data = torch.zeros(pages, 2, H, P, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    cache = m.PagedCache(dtype, data, torch.full((pages, 2, H, P), 127, dtype=torch.uint8, device="cuda"))
    small = m.paged_cache(4, P, H, D, dtype)
    near = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    far = torch.tensor([[pages - 1, pages - 2], [pages - 9, 1]], dtype=torch.int32, device="cuda")
    lens, starts, T = ints([100, 70]).cuda(), ints([0, 100, 170]).cuda(), 170
    x = torch.randn(T, H * (G + 2), D, generator=gen(3)).to(torch.bfloat16).cuda()
    rotary = m.Rotary(m.rotary_frequencies(D))
    masks = torch.zeros(T, 2, dtype=torch.int64, device="cuda")
    masks[:, 0], masks[:, 1] = -1, 5
    kept, counts = ints([[3, 90], [1, 69]]).cuda(), ints([2, 2]).cuda()
    got = []
    for c, table in ((cache, far), (small, near)):
        batch = m.PageBatch(table, lens, starts, T, max_new=100)
        q = m.rotary_write(c, batch, rotary, x[:, :H * G], x[:, H * G:H * G + H], x[:, H * G + H:])
        out = m.tree_attention(q, c, batch, masks)
        m.cache_keep(c, batch, kept, counts)
        got.append((out, [c.data.view(torch.uint8)[p.long()] for p in table.flatten()], [c.scales[p.long()] for p in table.flatten()]))
    assert torch.equal(got[0][0], got[1][0])
    for k in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(got[0][k], got[1][k]))


def test_instrumentation_names_the_launches():
    m = sz()
    s = Server(E4M3, 3, 9, 2, 4, 128, 16, 200, 1)
    s.inputs()
    m.profile_enable(True)
    s.run()
    torch.cuda.synchronize()
    names = m.profile_collect()
    m.profile_enable(False)
    assert {"sz_pages_assign", "sz_draft_tree", "sz_rotary_write", "sz_cache_keep"} <= set(names)
    assert {"sz_attn_rows", "sz_attn_tiles"} & set(names)
