"""The target-side operators as a verification step uses them: new rows into
the cache, attention over it, logits adjusted, verification, counts and
lengths moved on; eager and as one captured graph, on streams, from threads,
and with the workspaces they share."""

import threading

import numpy as np
import pytest
import torch

import block_speculative_decoding_ctx_gb300 as dfl
from oracle import target as ot
from oracle import verify as over
from target_testutil import F8, Paged, attention_reference, check_attention, rows_tensor, run_attention, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    dfl.lib()


class Target:
    """One layer of a model that verifies blocks: embeddings, projections, an
    attention layer over the paged cache, a head."""

    def __init__(self, B, gamma, V, n_q, n_kv, hd, page, pages, e4m3, seed, lens):
        g = torch.Generator().manual_seed(seed)
        dev = "cuda"
        self.B, self.gamma, self.V, self.n_q, self.n_kv, self.hd = B, gamma, V, n_q, n_kv, hd
        self.embed = torch.randn(V, 64, generator=g).to(torch.bfloat16).to(dev)
        self.w = [(torch.randn(64, n * hd, generator=g) * 0.3).to(torch.bfloat16).to(dev) for n in (n_q, n_kv, n_kv)]
        self.head = (torch.randn(n_q * hd, V, generator=g) * 0.1).to(torch.bfloat16).to(dev)
        width = pages // B
        order = torch.randperm(pages, generator=g)
        self.table = order[:B * width].view(B, width).to(torch.int32).to(dev)
        shape = (pages, n_kv, page, hd)
        kind = F8 if e4m3 else torch.bfloat16
        rows = torch.randn((2,) + shape, generator=g).to(torch.bfloat16)
        if e4m3:
            codes, scale = ot.quantize(rows.float().numpy())
            self.pages = torch.from_numpy(codes).to(dev).view(F8)
            self.scale = torch.from_numpy(scale).to(dev)
        else:
            self.pages, self.scale = rows.to(dev), [None, None]
        assert self.pages.dtype is kind
        self.cache = dfl.paged_cache(self.pages[0], self.pages[1], self.scale[0], self.scale[1])
        i32, n = torch.int32, B * gamma
        self.row_start = (torch.arange(B + 1) * gamma).to(i32).to(dev)
        self.kv_len = torch.tensor(lens, dtype=torch.int64, device=dev)
        self.tokens_in = torch.randint(0, V, (B, gamma), generator=g).to(i32).to(dev)     # anchor, drafts
        self.draft = self.tokens_in[:, 1:].contiguous()
        self.counts = torch.zeros(B, V, dtype=i32, device=dev)
        allow = torch.randint(-2 ** 31, 2 ** 31, (B, gamma, (V + 31) // 32), generator=g)
        self.allow = (allow | torch.randint(-2 ** 31, 2 ** 31, allow.shape, generator=g)).to(i32).to(dev)
        self.pen = {k: (torch.rand(B, generator=g) * 0.4 + o).to(dev) for k, o in
                    (("repetition", 1.0), ("frequency", 0.1), ("presence", 0.0))}
        self.q = torch.empty(n, n_q, hd, dtype=torch.bfloat16, device=dev)
        self.out = torch.empty_like(self.q)
        self.logits = torch.empty(B, gamma, V, device=dev)
        self.adjusted = torch.empty_like(self.logits)
        self.accept = torch.zeros(B, dtype=i32, device=dev)
        self.tokens = torch.zeros(B, gamma, dtype=i32, device=dev)
        self.anchor = torch.zeros(B, dtype=i32, device=dev)
        self.n_append = torch.zeros(B, dtype=i32, device=dev)
        # append, attention and adjustment run one after another: one workspace
        self.ws = dfl.workspace(max(dfl.dflash_paged_attention_workspace_bytes(n_q, n_kv, hd, gamma),
                                    dfl.dflash_paged_workspace_bytes(), dfl.dflash_logits_adjust_workspace_bytes()))
        self.ws_v = dfl.workspace(dfl.dflash_verify_workspace_bytes(B, gamma, V))

    def step(self):
        x = self.embed[self.tokens_in.view(-1).long()]
        self.q.copy_((x @ self.w[0]).view(-1, self.n_q, self.hd))
        k, v = ((x @ w).view(-1, self.n_kv, self.hd) for w in self.w[1:])
        batch = (self.row_start, self.kv_len, self.table)
        dfl.dflash_paged_append(self.cache, k, v, *batch, self.ws)
        dfl.dflash_paged_attention(self.cache, self.q, self.out, *batch, self.gamma, self.ws)
        self.logits.copy_((self.out.view(-1, self.n_q * self.hd) @ self.head).view(self.logits.shape))
        dfl.dflash_logits_adjust(self.logits, self.adjusted, self.ws, counts=self.counts, draft=self.draft,
                                 allow=self.allow, **self.pen)
        dfl.dflash_verify(dfl.DFLASH_VERIFY_GREEDY, self.adjusted, self.draft, self.accept, self.tokens, self.ws_v,
                          next_anchor=self.anchor, n_append=self.n_append)

    def move_on(self):
        """Counts and lengths after verification; the accepted tokens become
        the next block's input (a drafter would fill the rest)."""
        ok = self.tokens >= 0
        self.counts.scatter_add_(1, self.tokens.clamp(min=0).long(), ok.to(torch.int32))
        # rows of rejected drafts fall off, the next block's come
        self.kv_len += self.n_append.long()
        nxt = torch.where(ok, self.tokens, self.tokens_in)
        self.tokens_in.copy_(nxt.roll(1, 1))
        self.tokens_in[:, 0] = self.anchor
        self.draft.copy_(self.tokens_in[:, 1:])

    def state(self):
        t = [self.kv_len, self.counts, self.tokens, self.accept, self.out, self.adjusted,
             self.pages.view(torch.uint8)] + [s for s in self.scale if s is not None]
        return [x.clone() for x in t]


ARGS = dict(B=3, gamma=5, V=777, n_q=6, n_kv=2, hd=64, page=16, pages=30)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_step_against_the_oracle(e4m3):
    m = Target(**ARGS, e4m3=e4m3, seed=3, lens=[40, 5, 131])
    for cycle in range(2):
        counts = m.counts.cpu().numpy()
        m.step()
        torch.cuda.synchronize()
        assert dfl.dflash_read_status(m.ws) == 0 and dfl.dflash_read_status(m.ws_v) == 0

        class P:  # what attention_reference reads
            lens, start_np = m.kv_len.tolist(), m.row_start.cpu().numpy()
            page, dtype, table_np = 16, torch.bfloat16, m.table.cpu().numpy()
            host = staticmethod(lambda: tuple(to64(t) for t in (m.pages[0], m.pages[1], m.scale[0], m.scale[1])))
        P.e4m3 = e4m3
        want, _, bound, _ = attention_reference(P, m.q, True, 0, 0.125)
        assert (np.abs(to64(m.out) - want) <= bound).all()
        words = m.allow.cpu().numpy()
        allow = np.unpackbits(words.view(np.uint8), axis=-1, bitorder="little")[:, :, :m.V].astype(bool)
        adj, size = ot.adjust(to64(m.logits), counts=counts, draft=m.draft.cpu().numpy(), allow=allow,
                              **{k: v.cpu().numpy() for k, v in m.pen.items()})
        got = to64(m.adjusted)
        fine = np.isfinite(adj)
        np.testing.assert_array_equal(np.isfinite(got), fine)
        assert (np.abs(got[fine] - adj[fine]) <= 7 * 2.0 ** -24 * size[fine]).all()
        n, tok = over.greedy(m.adjusted.cpu().numpy(), m.draft.cpu().numpy())
        np.testing.assert_array_equal(m.accept.cpu().numpy(), n)
        np.testing.assert_array_equal(m.tokens.cpu().numpy(), tok)
        m.move_on()


@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_steps_equal_eager_ones(e4m3):
    eager = Target(**ARGS, e4m3=e4m3, seed=3, lens=[40, 5, 100])
    for _ in range(4):
        eager.step()
        eager.move_on()
    torch.cuda.synchronize()
    m = Target(**ARGS, e4m3=e4m3, seed=3, lens=[40, 5, 100])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):                         # library warm-up on this stream, then all state as it was
        m.step()
        m.move_on()
    torch.cuda.current_stream().wait_stream(s)
    fresh = Target(**ARGS, e4m3=e4m3, seed=3, lens=[40, 5, 100])
    for name, t in vars(fresh).items():
        if isinstance(t, torch.Tensor) and t.is_cuda:
            (getattr(m, name).view(torch.uint8) if t.dtype is F8 else getattr(m, name)).copy_(
                t.view(torch.uint8) if t.dtype is F8 else t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.step()
        m.move_on()
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert dfl.dflash_read_status(m.ws) == 0
    for a, b in zip(eager.state(), m.state()):
        assert torch.equal(a, b)


def test_two_graphs_that_share_a_workspace():
    p = [Paged([300, 40], [8, 8], 2, 64, 32, seed=1), Paged([70, 900], [8, 8], 2, 64, 32, seed=2, e4m3=True)]
    q = [rows_tensor(16, 8, 64, torch.bfloat16, 5 + i) for i in range(2)]
    want = [run_attention(a, b)[0].clone() for a, b in zip(p, q)]
    ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(8, 2, 64, 8))
    out = [torch.zeros_like(x) for x in q]
    graphs = []
    for a, x, o in zip(p, q, out):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dfl.dflash_paged_attention(a.cache, x, o, *a.batch, 8, ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        assert torch.equal(o, w)


def test_streams_and_threads_with_workspaces_of_their_own():
    cases = [(Paged([2000, 64, 5], [16, 1, 5], 2, 128, 64, seed=i, e4m3=i % 2 == 1),
              rows_tensor(22, 10, 128, torch.bfloat16, 9 + i)) for i in range(4)]
    want = [run_attention(p, q)[0].clone() for p, q in cases]
    got, errors = [None] * 4, []

    def work(i):
        try:
            torch.cuda.set_device(0)
            p, q = cases[i]
            s = torch.cuda.Stream()
            ws = dfl.workspace(dfl.dflash_paged_attention_workspace_bytes(10, 2, 128, 16))
            s.wait_stream(torch.cuda.default_stream())
            for _ in range(20):
                out = torch.zeros_like(q)
                s.wait_stream(torch.cuda.current_stream())
                dfl.dflash_paged_attention(p.cache, q, out, *p.batch, 16, ws, stream=s)
                s.synchronize()
            got[i] = out
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_many_requests_of_every_kind_at_once():
    """Single tokens, blocks, a prompt chunk, empty and new requests, in one
    call with more items than SMs."""
    rng = np.random.default_rng(0)
    lens, rows = [], []
    for i in range(90):
        n = int(rng.choice([0, 1, 1, 4, 8]))
        lens.append(int(n + rng.choice([0, 3, 127, 128, 500])) if i % 9 else n)
        rows.append(n)
    lens += [330, 260]
    rows += [300, 129]
    for e4m3 in (False, True):
        p = Paged(lens, rows, 2, 64, 16, e4m3=e4m3, seed=4)
        q = rows_tensor(p.n_rows, 6, 64, torch.bfloat16, 3, extra=1)
        out, lse, status = run_attention(p, q)
        assert status == 0
        check_attention(p, q, out, lse)
